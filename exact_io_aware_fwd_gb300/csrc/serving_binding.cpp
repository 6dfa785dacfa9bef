// Python binding of the operators around attention (fa_rope_table excepted): argument checks,
// output and workspace allocation, and the C-ABI call, in one compiled step.
//
// The kernels behind these calls take a few microseconds in the smallest cases (a decoding step of
// a small batch); the same checks and allocations in Python with ctypes took 20 to 30 us a call
// on the GPU's host, the compiled ones 3 to 6.  Nothing is computed here and nothing is kept
// between calls.  The library's entry points come from the Python side (bind), so that there is
// one loaded instance of it.
#include <Python.h>

#include <algorithm>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace {

// ---- the library's entry points, and the exception of a refused call
decltype(&fa_qk_norm_rope_fwd) p_rope_fwd;
decltype(&fa_qk_norm_rope_bwd) p_rope_bwd;
decltype(&fa_qk_norm_rope_bwd_workspace_size) p_rope_bwd_ws;
decltype(&fa_kv_append) p_append;
decltype(&fa_fwd_paged) p_paged;
decltype(&fa_fwd_paged_workspace_size) p_paged_ws;
decltype(&fa_fwd_shared_prefix) p_prefix;
decltype(&fa_fwd_shared_prefix_workspace_size) p_prefix_ws;
decltype(&fa_tree_mask) p_tree_mask;
decltype(&fa_fwd_paged_tree) p_tree;
decltype(&fa_page_bounds) p_bounds;
decltype(&fa_select_pages) p_select;
decltype(&fa_select_pages_workspace_size) p_select_ws;
decltype(&fa_fwd_paged_selected) p_selected;
decltype(&fa_fwd_paged_selected_workspace_size) p_selected_ws;
decltype(&fa_kv_weights) p_weights;
decltype(&fa_kv_evict) p_evict;
PyObject* fa_error;  // FAError(status, where)

struct Refused : std::runtime_error {  // becomes ValueError
  using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const std::string& why) { throw Refused(why); }

struct Status {  // becomes FAError
  int code;
  const char* where;
};
void check(fa_status st, const char* where) {
  if (st != FA_OK) throw Status{static_cast<int>(st), where};
}

// ---- arguments
const at::Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor_or_none(o, name);
  if (t == nullptr) refuse(std::string(name) + " must be a tensor");
  return *t;
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int int32_of(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return static_cast<int>(v);
}
int dim32(int64_t v) {
  if (v > INT32_MAX) refuse("a dimension is out of range");
  return static_cast<int>(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// Address of a contiguous tensor of `shape`; nullptr for None.
void* array(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape, at::Device dev,
            const char* name) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != type || t->sizes() != shape || t->device() != dev || !t->is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) +
           " tensor of shape " + shape_text(shape) + " on " + dev.str());
  return t->data_ptr();
}
int32_t* ints(const at::Tensor* t, at::IntArrayRef shape, at::Device dev, const char* name) {
  return static_cast<int32_t*>(array(t, at::kInt, shape, dev, name));
}

at::Device cuda_device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return t.device();
}

enum Order { kNH, kBNH, kBHN };  // dimensions before the head's elements: batch, token, head

// View of a bf16 tensor with contiguous rows.
fa_view rows(const at::Tensor& t, Order order, at::Device dev, const char* name) {
  const int lead = order == kNH ? 2 : 3;
  if (t.scalar_type() != at::kBFloat16 || t.device() != dev || t.dim() != lead + 1)
    refuse(std::string(name) + " must be a bfloat16 tensor on " + dev.str() + " of " +
           std::to_string(lead + 1) + " dimensions");
  int64_t s[3] = {0, 0, 0};  // batch, token, head
  const int place[3][3] = {{1, 2, 0}, {0, 1, 2}, {0, 2, 1}};
  bool ok = t.stride(lead) == 1;
  for (int i = 0; i < lead; ++i) {
    if (t.size(i) <= 1) continue;  // the stride of a dimension of one element does not matter
    s[place[order][i]] = t.stride(i);
    ok = ok && t.stride(i) % 8 == 0;
  }
  void* p = t.data_ptr();
  if (!ok || reinterpret_cast<uintptr_t>(p) % 16 != 0)
    refuse(std::string(name) + " must have contiguous rows, 16-byte aligned, at strides that are "
                               "multiples of 8 elements");
  return {p, s[0], s[1], s[2]};
}

// A new tensor, without the dispatcher's detour: between other calls of a program, whose code has
// taken its place in the host's caches, each such step costs more than in a loop of its own.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return at::Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}

// Rows [first, first + n) of dimension `dim` of a new tensor, as a tensor of its own.
at::Tensor part_of(const at::Tensor& t, int64_t dim, int64_t first, int64_t n) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(t.storage()),
                                                   t.key_set(), t.dtype());
  c10::SmallVector<int64_t, 5> sizes(t.sizes().begin(), t.sizes().end());
  sizes[dim] = n;
  impl->set_sizes_and_strides(sizes, t.strides(), t.storage_offset() + first * t.stride(dim));
  return at::Tensor(std::move(impl));
}

// An output: the caller's, whose elements must be distinct (no expanded or overlapping
// dimensions), or a new contiguous tensor.
at::Tensor own_rows(const at::Tensor* given, at::IntArrayRef shape, Order order, at::Device dev,
                    const char* name, fa_view& v) {
  at::Tensor t = given != nullptr ? *given : fresh(shape, at::kBFloat16, dev);
  if (given != nullptr) {
    if (t.sizes() != shape) refuse(std::string(name) + " must have shape " + shape_text(shape));
    int64_t reach = 1;
    std::vector<bool> seen(static_cast<size_t>(t.dim()), false);
    for (int64_t k = 0; k < t.dim(); ++k) {  // dimensions by ascending stride
      int64_t best = -1;
      for (int64_t i = 0; i < t.dim(); ++i)
        if (!seen[i] && (best < 0 || t.stride(i) < t.stride(best))) best = i;
      seen[best] = true;
      if (t.size(best) <= 1) continue;
      if (t.stride(best) < reach) refuse(std::string(name) + " must not overlap itself");
      reach += t.stride(best) * (t.size(best) - 1);
    }
  }
  v = rows(t, order, dev, name);
  return t;
}
at::Tensor own_array(const at::Tensor* given, at::IntArrayRef shape, at::ScalarType type,
                     at::Device dev, const char* name) {
  if (given == nullptr) return fresh(shape, type, dev);
  array(given, type, shape, dev, name);
  return *given;
}

// The caller's workspace, whose size counts in bytes, or a new one (kept until the call has been
// launched; the allocator orders its reuse on the current stream).
struct Workspace {
  c10::DataPtr own;
  void* p = nullptr;
  size_t bytes = 0;
};
Workspace workspace(const at::Tensor* given, size_t need, at::Device dev) {
  Workspace w;
  if (given == nullptr) {
    w.bytes = need;
    if (need > 0) w.own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
    w.p = w.own.get();
    return w;
  }
  if (given->device() != dev || !given->is_contiguous())
    refuse("workspace must be a contiguous tensor on " + dev.str());
  w.bytes = static_cast<size_t>(given->numel()) * given->element_size();
  w.p = given->data_ptr();
  return w;
}

// Calls launch on the device's current stream, on which their outputs are allocated too.
void* stream_of(at::Device dev) {
  return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}

fa_qk_transform transform(PyObject* table_o, PyObject* interleaved, PyObject* wq_o, PyObject* wk_o,
                          PyObject* eps, int64_t d, at::Device dev) {
  fa_qk_transform t{};
  const at::Tensor* table = tensor_or_none(table_o, "table");
  if (table != nullptr) {
    if (table->dim() != 2) refuse("table must be a tensor [positions, rot]");
    const int64_t n = table->size(0), rot = table->size(1);
    t.table = static_cast<const float*>(array(table, at::kFloat, {n, rot}, dev, "table"));
    if (n < 1 || rot < 16 || rot > d || rot % 16 != 0)
      refuse("the rotated part must be a multiple of 16 elements, at most d");
    t.n_pos = dim32(n);
    t.rot = static_cast<int>(rot);
  }
  const at::Tensor* wq = tensor_or_none(wq_o, "q_weight");
  const at::Tensor* wk = tensor_or_none(wk_o, "k_weight");
  if ((wq == nullptr) != (wk == nullptr)) refuse("q_weight and k_weight go together");
  t.q_weight = static_cast<const float*>(array(wq, at::kFloat, {d}, dev, "q_weight"));
  t.k_weight = static_cast<const float*>(array(wk, at::kFloat, {d}, dev, "k_weight"));
  const int truth = PyObject_IsTrue(interleaved);
  if (truth < 0) throw python_error();
  t.interleaved = truth;
  t.eps = real(eps);
  return t;
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* wrap_all(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (o == nullptr) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Runs a binding with its exceptions as Python's: Refused as ValueError, Status as FAError, and
// PyTorch's own (out of memory among them) as PyTorch raises them.
template <PyObject* (*kBody)(PyObject* const*)>
PyObject* guarded(PyObject* const* a) {
  HANDLE_TH_ERRORS
  try {
    return kBody(a);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Status& s) {
    PyObject* e = PyObject_CallFunction(fa_error, "is", s.code, s.where);
    if (e != nullptr) {
      PyErr_SetObject(fa_error, e);
      Py_DECREF(e);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*kBody)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  return guarded<kBody>(a);
}

// ---- q, k, v, table, positions, interleaved, q_weight, k_weight, eps, q_out, k_out, v_out
PyObject* norm_rope_fwd(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const at::Tensor& k = tensor(a[1], "k");
  const at::Tensor* v = tensor_or_none(a[2], "v");
  const at::Device dev = cuda_device(q, "q");
  const int64_t nd = q.dim();
  if ((nd != 3 && nd != 4) || k.dim() != nd || k.size(-1) != q.size(-1) || k.size(0) != q.size(0) ||
      (nd == 4 && k.size(1) != q.size(1)))
    refuse("q and k must be [B, N, heads, d] or packed [total, heads, d], alike in tokens and head "
           "dimension");
  if (v != nullptr && v->sizes() != k.sizes()) refuse("v must have k's shape");
  const int64_t H = q.size(-2), Hkv = k.size(-2), d = q.size(-1);
  const int64_t B = nd == 4 ? q.size(0) : 1, N = nd == 4 ? q.size(1) : q.size(0);
  const Order in_order = nd == 4 ? kBNH : kNH, out_order = nd == 4 ? kBHN : kNH;
  auto shape = [&](int64_t h) {
    return nd == 4 ? std::vector<int64_t>{B, h, N, d} : std::vector<int64_t>{N, h, d};
  };
  const fa_qk_transform t = transform(a[3], a[5], a[6], a[7], a[8], d, dev);
  const int32_t* pos = ints(tensor_or_none(a[4], "positions"), q.sizes().slice(0, nd - 2), dev, "positions");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  fa_view in[3] = {rows(q, in_order, dev, "q"), rows(k, in_order, dev, "k"), {}}, out[3] = {};
  if (v != nullptr) in[2] = rows(*v, in_order, dev, "v");
  at::Tensor qo = own_rows(tensor_or_none(a[9], "q_out"), shape(H), out_order, dev, "q_out", out[0]);
  at::Tensor ko = own_rows(tensor_or_none(a[10], "k_out"), shape(Hkv), out_order, dev, "k_out", out[1]);
  at::Tensor vo;
  if (v != nullptr)
    vo = own_rows(tensor_or_none(a[11], "v_out"), shape(Hkv), out_order, dev, "v_out", out[2]);
  if (B == 0 || N == 0) return wrap_all({qo, ko, vo});
  check(p_rope_fwd(in, out, pos, dim32(B), dim32(N), dim32(H), dim32(Hkv), dim32(d), &t,
                   stream_of(dev)),
        "fa_qk_norm_rope_fwd");
  return wrap_all({qo, ko, vo});
}

// ---- dq, dk, dv, q, k, table, positions, interleaved, q_weight, k_weight, eps, dq_in, dk_in,
//      dv_in, workspace
PyObject* norm_rope_bwd(PyObject* const* a) {
  const at::Tensor& dq = tensor(a[0], "dq");
  const at::Tensor& dk = tensor(a[1], "dk");
  const at::Tensor* dv = tensor_or_none(a[2], "dv");
  const at::Device dev = cuda_device(dq, "dq");
  const int64_t nd = dq.dim();
  if ((nd != 3 && nd != 4) || dk.dim() != nd)
    refuse("dq and dk must be [B, heads, N, d] or packed [total, heads, d]");
  const int64_t B = nd == 4 ? dq.size(0) : 1, N = nd == 4 ? dq.size(2) : dq.size(0);
  const int64_t H = dq.size(1), Hkv = dk.size(1), d = dq.size(-1);
  if (dk.size(0) != dq.size(0) || dk.size(-1) != d || (nd == 4 && dk.size(2) != N) ||
      (dv != nullptr && dv->sizes() != dk.sizes()))
    refuse("dk and dv must agree with dq");
  const Order order = nd == 4 ? kBHN : kNH, out_order = nd == 4 ? kBNH : kNH;
  auto shape = [&](int64_t h) {  // of the projection's side
    return nd == 4 ? std::vector<int64_t>{B, N, h, d} : std::vector<int64_t>{N, h, d};
  };
  const fa_qk_transform t = transform(a[5], a[7], a[8], a[9], a[10], d, dev);
  const std::vector<int64_t> lead = nd == 4 ? std::vector<int64_t>{B, N} : std::vector<int64_t>{N};
  const int32_t* pos = ints(tensor_or_none(a[6], "positions"), lead, dev, "positions");
  const at::Tensor* q = tensor_or_none(a[3], "q");
  const at::Tensor* k = tensor_or_none(a[4], "k");
  const bool norm = t.q_weight != nullptr;
  if (norm && (q == nullptr || k == nullptr || q->sizes() != at::IntArrayRef(shape(H)) ||
               k->sizes() != at::IntArrayRef(shape(Hkv))))
    refuse("q and k (the forward's inputs) are needed with norms");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  at::Tensor out_t[3];
  const at::Tensor* given[3] = {tensor_or_none(a[11], "dq_in"), tensor_or_none(a[12], "dk_in"),
                                tensor_or_none(a[13], "dv_in")};
  if (given[0] == nullptr && given[1] == nullptr && given[2] == nullptr) {
    // the gradient of a fused projection: slices of one tensor
    const at::Tensor fused = fresh(shape(H + (dv != nullptr ? 2 : 1) * Hkv), at::kBFloat16, dev);
    out_t[0] = part_of(fused, nd - 2, 0, H);
    out_t[1] = part_of(fused, nd - 2, H, Hkv);
    if (dv != nullptr) out_t[2] = part_of(fused, nd - 2, H + Hkv, Hkv);
    for (int i = 0; i < 3; ++i) given[i] = out_t[i].defined() ? &out_t[i] : nullptr;
  }
  const bool empty = B == 0 || N == 0;
  fa_view grad[3] = {}, x[2] = {}, out[3] = {};
  const char* names[3] = {"dq_in", "dk_in", "dv_in"};
  for (int i = 0; i < (dv != nullptr ? 3 : 2); ++i) {
    const at::Tensor& z = i == 0 ? dq : (i == 1 ? dk : *dv);
    grad[i] = rows(z, order, dev, i == 0 ? "dq" : (i == 1 ? "dk" : "dv"));
    out_t[i] = own_rows(given[i], shape(i == 0 ? H : Hkv), out_order, dev, names[i], out[i]);
    if (norm && i < 2) x[i] = rows(i == 0 ? *q : *k, out_order, dev, i == 0 ? "q" : "k");
  }
  at::Tensor dwq, dwk;
  Workspace ws;
  if (norm) {
    const at::Tensor dw = fresh({2 * d}, at::kFloat, dev);
    dwq = part_of(dw, 0, 0, d);
    dwk = part_of(dw, 0, d, d);
    ws = workspace(tensor_or_none(a[14], "workspace"), p_rope_bwd_ws(dim32(d)), dev);
  }
  check(p_rope_bwd(grad, norm ? x : nullptr, out, norm ? dwq.data_ptr<float>() : nullptr,
                   norm ? dwk.data_ptr<float>() : nullptr, pos, B > 0 ? dim32(B) : 1,
                   empty ? 0 : dim32(N), dim32(H), dim32(Hkv), dim32(d), &t,
                   ws.p, ws.bytes, stream_of(dev)),
        "fa_qk_norm_rope_bwd");
  return wrap_all({out_t[0], out_t[1], out_t[2], dwq, dwk});
}

// ---- the cache's tensors: k_cache, v_cache, block_table, kv_lens
struct Cache {
  fa_paged_kv kv;
  int64_t B, Hkv, d, pages, page_size;
};
// block_table and kv_lens alone
Cache table_of(PyObject* const* a, at::Device dev) {
  const at::Tensor& table = tensor(a[0], "block_table");
  const at::Tensor& lens = tensor(a[1], "kv_lens");
  if (table.dim() != 2) refuse("block_table must be [B, max_pages]");
  Cache c{};
  c.B = table.size(0);
  c.pages = table.size(1);
  c.kv.block_table = ints(&table, {c.B, c.pages}, dev, "block_table");
  c.kv.max_pages = dim32(c.pages);
  c.kv.kv_lens = ints(&lens, {c.B}, dev, "kv_lens");
  return c;
}
// with keys (and values, unless v is nullptr)
Cache keys_of(PyObject* k_o, PyObject* v_o, PyObject* const* table, at::Device dev) {
  const at::Tensor& k = tensor(k_o, "k_cache");
  Cache c = table_of(table, dev);
  if (k.dim() != 4) refuse("k_cache must be [pages, Hkv, page_size, d]");
  c.Hkv = k.size(1);
  c.page_size = k.size(2);
  c.d = k.size(3);
  c.kv.k_cache = array(&k, at::kBFloat16, k.sizes(), dev, "k_cache");
  if (v_o != nullptr)
    c.kv.v_cache = array(&tensor(v_o, "v_cache"), at::kBFloat16, k.sizes(), dev, "v_cache");
  c.kv.num_pages = dim32(k.size(0));
  c.kv.page_size = dim32(c.page_size);
  return c;
}
Cache cache_of(PyObject* const* a, at::Device dev) { return keys_of(a[0], a[1], a + 2, dev); }

// The keys of a sequence that a block table reaches.
int reach_of(const Cache& c) {
  const int64_t reach = c.pages * c.page_size;
  return static_cast<int>(reach < INT32_MAX ? reach : INT32_MAX);
}
const int32_t* token_offsets(PyObject* o, const Cache& c, int64_t total, at::Device dev) {
  const at::Tensor* cu = tensor_or_none(o, "cu_seqlens");
  if (cu == nullptr && total != c.B) refuse("without cu_seqlens there is one token per sequence");
  return ints(cu, {c.B + 1}, dev, "cu_seqlens");
}

// ---- q, k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens, pos_offset, table,
//      interleaved, q_weight, k_weight, eps, q_out
PyObject* kv_append(PyObject* const* a) {
  const at::Tensor* q = tensor_or_none(a[0], "q");
  const at::Tensor& k = tensor(a[1], "k");
  const at::Tensor& v = tensor(a[2], "v");
  const at::Device dev = cuda_device(k, "k");
  const Cache c = cache_of(a + 3, dev);
  if (k.dim() != 3 || k.size(1) != c.Hkv || k.size(2) != c.d || v.sizes() != k.sizes())
    refuse("k and v must be [total, Hkv, d] with the cache's heads");
  const int64_t total = k.size(0);
  if (q != nullptr && (q->dim() != 3 || q->size(0) != total || q->size(2) != c.d))
    refuse("q must be [total, H, d]");
  const int64_t H = q != nullptr ? q->size(1) : c.Hkv;
  const int32_t* cu = token_offsets(a[7], c, total, dev);
  const int32_t* offset = ints(tensor_or_none(a[8], "pos_offset"), {c.B}, dev, "pos_offset");
  const fa_qk_transform t = transform(a[9], a[10], a[11], a[12], a[13], c.d, dev);
  const c10::cuda::OptionalCUDAGuard guard(dev);
  at::Tensor qo;
  fa_view in[3] = {}, out{};
  if (q != nullptr) {
    in[0] = rows(*q, kNH, dev, "q");
    qo = own_rows(tensor_or_none(a[14], "q_out"), {total, H, c.d}, kNH, dev, "q_out", out);
  }
  in[1] = rows(k, kNH, dev, "k");
  in[2] = rows(v, kNH, dev, "v");
  if (total > 0)
    check(p_append(in, &out, &c.kv, cu, offset, dim32(c.B), dim32(total), dim32(H), dim32(c.Hkv),
                   dim32(c.d), &t, stream_of(dev)),
          "fa_kv_append");
  return wrap(qo);
}

// ---- q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_q, max_kv, causal, scale, out,
//      lse, workspace; with a prefix: prefix_table, prefix_lens, group_cu, max_prefix too; with a
//      tree: its mask
enum Kind { kPlain, kPrefix, kTree };
template <Kind kKind>
PyObject* attend(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const at::Device dev = cuda_device(q, "q");
  const Cache c = cache_of(a + 1, dev);
  if (q.dim() != 3 || q.size(2) != c.d || c.Hkv < 1 || q.size(1) % c.Hkv != 0)
    refuse("q must be [total, H, d] with H a multiple of the cache's heads");
  const int64_t total = q.size(0), H = q.size(1);
  const void* qp = array(&q, at::kBFloat16, q.sizes(), dev, "q");
  const int32_t* cu = token_offsets(a[5], c, total, dev);
  int max_q = 1;
  if (a[6] != Py_None) max_q = int32_of(a[6], "max_q");
  else if (cu != nullptr) max_q = total > 1 ? dim32(total) : 1;
  const int max_kv = a[7] != Py_None ? int32_of(a[7], "max_kv") : reach_of(c);
  const int causal = PyObject_IsTrue(a[8]);
  if (causal < 0) throw python_error();
  const float scale = a[9] == Py_None ? -1.f : real(a[9]);
  fa_prefix pre{};
  const uint64_t* mask = nullptr;
  int words = 1;
  if (kKind == kTree) {
    const at::Tensor& m = tensor(a[13], "tree_mask");
    if (m.dim() != 2) refuse("tree_mask must be [total, words]");
    mask = static_cast<const uint64_t*>(array(&m, at::kLong, {total, m.size(1)}, dev, "tree_mask"));
    words = dim32(m.size(1));
  }
  if (kKind == kPrefix) {
    const at::Tensor& table = tensor(a[13], "prefix_table");
    if (table.dim() != 2) refuse("prefix_table must be [groups, pages]");
    const int64_t groups = table.size(0), pages = table.size(1), most = pages * c.page_size;
    pre.table = ints(&table, {groups, pages}, dev, "prefix_table");
    pre.max_pages = dim32(pages);
    pre.lens = ints(&tensor(a[14], "prefix_lens"), {groups}, dev, "prefix_lens");
    pre.group_cu = ints(&tensor(a[15], "group_cu"), {groups + 1}, dev, "group_cu");
    pre.groups = dim32(groups);
    pre.max_len = a[16] != Py_None ? int32_of(a[16], "max_prefix")
                                   : static_cast<int>(most < INT32_MAX ? most : INT32_MAX);
  }
  const c10::cuda::OptionalCUDAGuard guard(dev);
  const at::Tensor out = own_array(tensor_or_none(a[10], "out"), q.sizes(), at::kBFloat16, dev, "out");
  const at::Tensor lse = own_array(tensor_or_none(a[11], "lse"), {H, total}, at::kFloat, dev, "lse");
  if (c.B == 0 && total == 0) return wrap_all({out, lse});  // an empty batch
  const int B = dim32(c.B), T = dim32(total), h = dim32(H), hkv = dim32(c.Hkv), d = dim32(c.d);
  const Workspace ws =
      workspace(tensor_or_none(a[12], "workspace"),
                kKind == kPrefix ? p_prefix_ws(B, pre.groups, T, h, hkv, d)
                                 : p_paged_ws(B, T, h, hkv, d),
                dev);
  void* stream = stream_of(dev);
  if (kKind == kTree)
    check(p_tree(qp, &c.kv, mask, words, out.data_ptr(), lse.data_ptr<float>(), cu, B, max_q, max_kv, T,
                 h, hkv, d, scale, ws.p, ws.bytes, stream),
          "fa_fwd_paged_tree");
  else if (kKind == kPrefix)
    check(p_prefix(qp, &c.kv, &pre, out.data_ptr(), lse.data_ptr<float>(), cu, B, max_q, max_kv, T,
                   h, hkv, d, causal, scale, ws.p, ws.bytes, stream),
          "fa_fwd_shared_prefix");
  else
    check(p_paged(qp, &c.kv, out.data_ptr(), lse.data_ptr<float>(), cu, B, max_q, max_kv, T, h, hkv,
                  d, causal, scale, ws.p, ws.bytes, stream),
          "fa_fwd_paged");
  return wrap_all({out, lse});
}

// ---- parents, cu_seqlens, max_q, out
PyObject* tree_mask(PyObject* const* a) {
  const at::Tensor& parents = tensor(a[0], "parents");
  const at::Device dev = cuda_device(parents, "parents");
  if (parents.dim() != 1) refuse("parents must be [total]");
  const int64_t total = parents.size(0);
  const int32_t* p = ints(&parents, {total}, dev, "parents");
  const at::Tensor* cu = tensor_or_none(a[1], "cu_seqlens");
  if (cu != nullptr && (cu->dim() != 1 || cu->size(0) < 1)) refuse("cu_seqlens must be [B + 1]");
  const int64_t B = cu != nullptr ? cu->size(0) - 1 : total;
  const int32_t* offsets = ints(cu, {B + 1}, dev, "cu_seqlens");
  int64_t most = cu != nullptr ? total : 1;
  if (a[2] != Py_None) most = int32_of(a[2], "max_q");
  const int words = most > 0 ? dim32((most + 63) / 64) : 1;
  const c10::cuda::OptionalCUDAGuard guard(dev);
  const at::Tensor out =
      own_array(tensor_or_none(a[3], "out"), {total, words}, at::kLong, dev, "out");
  if (B > 0 && total > 0)
    check(p_tree_mask(p, offsets, dim32(B), dim32(total), words,
                      static_cast<uint64_t*>(out.data_ptr()), stream_of(dev)),
          "fa_tree_mask");
  return wrap(out);
}

// ---- k_cache, block_table, kv_lens, bounds, cu_seqlens, total
PyObject* page_bounds(PyObject* const* a) {
  const at::Device dev = cuda_device(tensor(a[0], "k_cache"), "k_cache");
  const Cache c = keys_of(a[0], nullptr, a + 1, dev);
  const at::Tensor& bounds = tensor(a[3], "bounds");
  void* p = array(&bounds, at::kBFloat16, {c.kv.num_pages, c.Hkv, 2, c.d}, dev, "bounds");
  const at::Tensor* cu = tensor_or_none(a[4], "cu_seqlens");
  // without a count, any that the block table has room for
  int64_t total = c.B;
  if (cu != nullptr) {
    const int64_t most = c.B * c.pages * c.page_size;
    total = a[5] != Py_None ? integer(a[5]) : (most < INT32_MAX ? most : INT32_MAX);
    if (total == 0) total = 1;  // launched, so that offsets that say otherwise are reported
  } else if (a[5] != Py_None && integer(a[5]) != c.B) {
    refuse("without cu_seqlens there is one token per sequence");
  }
  const int32_t* offsets = ints(cu, {c.B + 1}, dev, "cu_seqlens");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  if (c.B > 0)
    check(p_bounds(&c.kv, p, offsets, dim32(c.B), dim32(total), dim32(c.Hkv), dim32(c.d),
                   stream_of(dev)),
          "fa_page_bounds");
  return wrap(bounds);
}

// ---- q, bounds, block_table, kv_lens, page_size, top, first, last, cu_seqlens, max_kv, out,
//      workspace
PyObject* select_pages(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const at::Tensor& bounds = tensor(a[1], "bounds");
  const at::Device dev = cuda_device(q, "q");
  Cache c = table_of(a + 2, dev);
  if (bounds.dim() != 4 || bounds.size(2) != 2) refuse("bounds must be [pages, Hkv, 2, d]");
  c.Hkv = bounds.size(1);
  c.d = bounds.size(3);
  c.kv.num_pages = dim32(bounds.size(0));
  c.kv.page_size = int32_of(a[4], "page_size");
  c.page_size = c.kv.page_size;
  if (c.page_size < 1) refuse("page_size is out of range");
  const void* bp = array(&bounds, at::kBFloat16, bounds.sizes(), dev, "bounds");
  if (q.dim() != 3 || q.size(2) != c.d || c.Hkv < 1 || q.size(1) % c.Hkv != 0)
    refuse("q must be [total, H, d] with H a multiple of the bounds' heads");
  const int64_t total = q.size(0), H = q.size(1);
  const void* qp = array(&q, at::kBFloat16, q.sizes(), dev, "q");
  const int top = int32_of(a[5], "top"), first = int32_of(a[6], "first"), last = int32_of(a[7], "last");
  const int32_t* cu = token_offsets(a[8], c, total, dev);
  const int max_kv = a[9] != Py_None ? int32_of(a[9], "max_kv") : reach_of(c);
  if (top < 1) refuse("top must be positive");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  const at::Tensor out =
      own_array(tensor_or_none(a[10], "out"), {total, c.Hkv, top}, at::kInt, dev, "out");
  if (c.B == 0 && total == 0) return wrap(out);  // an empty batch
  const int B = dim32(c.B), T = dim32(total), hkv = dim32(c.Hkv);
  const Workspace ws = workspace(tensor_or_none(a[11], "workspace"),
                                 p_select_ws(B, T, hkv, c.kv.page_size, max_kv), dev);
  check(p_select(qp, bp, &c.kv, out.data_ptr<int32_t>(), top, first, last, cu, B, max_kv, T, dim32(H),
                 hkv, dim32(c.d), ws.p, ws.bytes, stream_of(dev)),
        "fa_select_pages");
  return wrap(out);
}

// ---- q, k_cache, v_cache, block_table, kv_lens, pages, cu_seqlens, scale, out, lse, workspace
PyObject* attend_selected(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const at::Device dev = cuda_device(q, "q");
  const Cache c = cache_of(a + 1, dev);
  if (q.dim() != 3 || q.size(2) != c.d || c.Hkv < 1 || q.size(1) % c.Hkv != 0)
    refuse("q must be [total, H, d] with H a multiple of the cache's heads");
  const int64_t total = q.size(0), H = q.size(1);
  const void* qp = array(&q, at::kBFloat16, q.sizes(), dev, "q");
  const at::Tensor& pages = tensor(a[5], "pages");
  if (pages.dim() != 3) refuse("pages must be [total, Hkv, top]");
  const int top = dim32(pages.size(2));
  const int32_t* pp = ints(&pages, {total, c.Hkv, pages.size(2)}, dev, "pages");
  const int32_t* cu = token_offsets(a[6], c, total, dev);
  const float scale = a[7] == Py_None ? -1.f : real(a[7]);
  const c10::cuda::OptionalCUDAGuard guard(dev);
  const at::Tensor out = own_array(tensor_or_none(a[8], "out"), q.sizes(), at::kBFloat16, dev, "out");
  const at::Tensor lse = own_array(tensor_or_none(a[9], "lse"), {H, total}, at::kFloat, dev, "lse");
  if (c.B == 0 && total == 0) return wrap_all({out, lse});  // an empty batch
  const int T = dim32(total), h = dim32(H), hkv = dim32(c.Hkv), d = dim32(c.d);
  const Workspace ws = workspace(tensor_or_none(a[10], "workspace"), p_selected_ws(T, h, hkv, d), dev);
  check(p_selected(qp, &c.kv, pp, top, out.data_ptr(), lse.data_ptr<float>(), cu, dim32(c.B), T, h, hkv,
                   d, scale, ws.p, ws.bytes, stream_of(dev)),
        "fa_fwd_paged_selected");
  return wrap_all({out, lse});
}

// ---- q, lse, k_cache, block_table, kv_lens, weights, cu_seqlens, max_q, max_kv, causal, scale, out
PyObject* kv_weights(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const at::Device dev = cuda_device(q, "q");
  const Cache c = keys_of(a[2], nullptr, a + 3, dev);
  if (q.dim() != 3 || q.size(2) != c.d || c.Hkv < 1 || q.size(1) % c.Hkv != 0)
    refuse("q must be [total, H, d] with H a multiple of the cache's heads");
  const int64_t total = q.size(0), H = q.size(1);
  const void* qp = array(&q, at::kBFloat16, q.sizes(), dev, "q");
  const float* lse = static_cast<const float*>(
      array(&tensor(a[1], "lse"), at::kFloat, {H, total}, dev, "lse"));
  const int32_t* cu = token_offsets(a[6], c, total, dev);
  int max_q = 1;
  if (a[7] != Py_None) max_q = int32_of(a[7], "max_q");
  else if (cu != nullptr) max_q = total > 1 ? dim32(total) : 1;
  const int max_kv = a[8] != Py_None ? int32_of(a[8], "max_kv") : reach_of(c);
  const int causal = PyObject_IsTrue(a[9]);
  if (causal < 0) throw python_error();
  const float scale = a[10] == Py_None ? -1.f : real(a[10]);
  const at::Tensor* in = tensor_or_none(a[5], "weights");
  const at::Tensor* given = tensor_or_none(a[11], "out");
  if (max_kv < 0) refuse("max_kv is out of range");
  int64_t cap = max_kv;  // columns: those of weights, of out, or max_kv
  for (const at::Tensor* t : {given, in}) {
    if (t == nullptr) continue;
    if (t->dim() != 3) refuse("weights and out must be [B, Hkv, capacity]");
    cap = t->size(2);
  }
  const float* w = static_cast<const float*>(array(in, at::kFloat, {c.B, c.Hkv, cap}, dev, "weights"));
  const c10::cuda::OptionalCUDAGuard guard(dev);
  const at::Tensor out = own_array(given, {c.B, c.Hkv, cap}, at::kFloat, dev, "out");
  if (c.B > 0)
    check(p_weights(qp, lse, &c.kv, w, out.data_ptr<float>(), dim32(cap), cu, dim32(c.B), max_q, max_kv,
                    dim32(total), dim32(H), dim32(c.Hkv), dim32(c.d), causal, scale, stream_of(dev)),
          "fa_kv_weights");
  return wrap(out);
}

// ---- weights, k_cache, v_cache, block_table, kv_lens, new_table, budget, recent, max_kv
PyObject* kv_evict(PyObject* const* a) {
  const at::Tensor& w = tensor(a[0], "weights");
  const at::Device dev = cuda_device(w, "weights");
  const Cache c = cache_of(a + 1, dev);
  if (w.dim() != 3) refuse("weights must be [B, Hkv, capacity]");
  const int64_t cap = w.size(2);
  const float* wp = static_cast<const float*>(array(&w, at::kFloat, {c.B, c.Hkv, cap}, dev, "weights"));
  const at::Tensor& table = tensor(a[5], "new_table");
  if (table.dim() != 2) refuse("new_table must be [B, pages]");
  const int32_t* tp = ints(&table, {c.B, table.size(1)}, dev, "new_table");
  const int budget = int32_of(a[6], "budget"), recent = int32_of(a[7], "recent");
  const int max_kv = a[8] != Py_None ? int32_of(a[8], "max_kv") : reach_of(c);
  if (budget < 1 || recent < 0 || recent > budget) refuse("0 <= recent <= budget and 1 <= budget");
  if (table.size(1) * c.page_size < std::min<int64_t>({budget, max_kv, cap}))
    refuse("new_table must have pages for the keys that may be kept");
  const c10::cuda::OptionalCUDAGuard guard(dev);
  const at::Tensor lens = fresh({c.B}, at::kInt, dev);
  const at::Tensor kept = fresh({c.B, c.Hkv, budget}, at::kInt, dev);
  const at::Tensor left = fresh({c.B, c.Hkv, budget}, at::kFloat, dev);
  if (c.B > 0)
    check(p_evict(wp, dim32(cap), &c.kv, tp, dim32(table.size(1)), budget, recent,
                  lens.data_ptr<int32_t>(), kept.data_ptr<int32_t>(), left.data_ptr<float>(), dim32(c.B),
                  max_kv, dim32(c.Hkv), dim32(c.d), stream_of(dev)),
          "fa_kv_evict");
  return wrap_all({lens, kept, left});
}

// ---- error class, then the entry points' addresses in the order below
PyObject* bind(PyObject* const* a) {
  Py_INCREF(a[0]);
  Py_XDECREF(fa_error);
  fa_error = a[0];
  auto at = [&](int i) { return reinterpret_cast<void*>(static_cast<intptr_t>(integer(a[i]))); };
  p_rope_fwd = reinterpret_cast<decltype(p_rope_fwd)>(at(1));
  p_rope_bwd = reinterpret_cast<decltype(p_rope_bwd)>(at(2));
  p_rope_bwd_ws = reinterpret_cast<decltype(p_rope_bwd_ws)>(at(3));
  p_append = reinterpret_cast<decltype(p_append)>(at(4));
  p_paged = reinterpret_cast<decltype(p_paged)>(at(5));
  p_paged_ws = reinterpret_cast<decltype(p_paged_ws)>(at(6));
  p_prefix = reinterpret_cast<decltype(p_prefix)>(at(7));
  p_prefix_ws = reinterpret_cast<decltype(p_prefix_ws)>(at(8));
  p_tree_mask = reinterpret_cast<decltype(p_tree_mask)>(at(9));
  p_tree = reinterpret_cast<decltype(p_tree)>(at(10));
  p_bounds = reinterpret_cast<decltype(p_bounds)>(at(11));
  p_select = reinterpret_cast<decltype(p_select)>(at(12));
  p_select_ws = reinterpret_cast<decltype(p_select_ws)>(at(13));
  p_selected = reinterpret_cast<decltype(p_selected)>(at(14));
  p_selected_ws = reinterpret_cast<decltype(p_selected_ws)>(at(15));
  p_weights = reinterpret_cast<decltype(p_weights)>(at(16));
  p_evict = reinterpret_cast<decltype(p_evict)>(at(17));
  Py_RETURN_NONE;
}

#define FA_METHOD(name, body, args)                                                         \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<body, args>)), \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_METHOD("bind", bind, 18),
                         FA_METHOD("norm_rope_fwd", norm_rope_fwd, 12),
                         FA_METHOD("norm_rope_bwd", norm_rope_bwd, 15),
                         FA_METHOD("kv_append", kv_append, 15),
                         FA_METHOD("fwd_paged", attend<kPlain>, 13),
                         FA_METHOD("fwd_shared_prefix", attend<kPrefix>, 17),
                         FA_METHOD("fwd_paged_tree", attend<kTree>, 14),
                         FA_METHOD("tree_mask", tree_mask, 4),
                         FA_METHOD("page_bounds", page_bounds, 6),
                         FA_METHOD("select_pages", select_pages, 12),
                         FA_METHOD("fwd_paged_selected", attend_selected, 11),
                         FA_METHOD("kv_weights", kv_weights, 12),
                         FA_METHOD("kv_evict", kv_evict, 9),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__serving_binding() {
  return PyModule_Create(&module);
}
