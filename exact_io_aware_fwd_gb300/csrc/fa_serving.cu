// C-ABI entry points (declared in include/fa.h) of the operators around attention: the norm and
// rotation pass, the paged cache and the attention that reads it.  Every argument is checked
// before the first launch; nothing here allocates device memory.
#include <cmath>
#include <limits>

#include "fa.h"
#include "fa_host.h"
#include "fa_internal.h"
#include "fa_paged.h"
#include "serving_checks.h"

namespace {

using fa::aligned_to;
using fa::check_cache;
using fa::check_heads;
using fa::device_ready;
using fa::kMaxInt;
using fa::kMaxKeys;
using fa::make_pool_map;
using fa::page_shift;
using fa::status_of;
using fa::up256;

constexpr float kLog2e = 1.4426950408889634f;

// A view that rows of 16-byte pieces can be read from or written to; the stride of a dimension
// of one element does not matter.
bool view_ok(const fa_view& v, int B, int N, int H) {
  return v.data != nullptr && aligned_to(v.data, 16) && (B == 1 || v.batch % 8 == 0) &&
         (N == 1 || v.token % 8 == 0) && (H == 1 || v.head % 8 == 0);
}
fa::RowView row_view(const fa_view& v) {
  return {static_cast<__nv_bfloat16*>(v.data), v.batch, v.token, v.head};
}

fa_status check_transform(const fa_qk_transform* t, int d) {
  if (t == nullptr) return FA_ERR_INVALID_ARG;
  if (t->table != nullptr) {
    if (t->rot < 16 || t->rot > d || t->rot % 16 != 0 || t->n_pos < 1) return FA_ERR_INVALID_ARG;
    if (!aligned_to(t->table, 16)) return FA_ERR_INVALID_ARG;
  }
  if ((t->q_weight == nullptr) != (t->k_weight == nullptr)) return FA_ERR_INVALID_ARG;
  if (!aligned_to(t->q_weight, 16) || !aligned_to(t->k_weight, 16)) return FA_ERR_INVALID_ARG;
  if (t->q_weight != nullptr && !(std::isfinite(t->eps) && t->eps >= 0.f))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

void set_transform(fa::RopeArgs& a, const fa_qk_transform& t) {
  a.table = t.table;
  a.n_pos = t.n_pos;
  a.rot = t.table != nullptr ? t.rot : 0;
  a.wq = t.q_weight;
  a.wk = t.k_weight;
  a.eps = t.eps;
}

// Query rows per key/value head above which a list goes to the tensor-core kernel.  The other
// kernel reads the keys once per 16 rows: 16 sequences of 8192 keys take it 85 us with 12 to 16 rows
// and 154 with 24, the tensor-core kernel 89 with 24; at d = 64 it takes 51 with 12 rows and 81 with
// 20 or 32, the tensor-core kernel 67.  With two lists and d = 64, where a row tile's second slot
// rests (82), it takes over above 32.
constexpr long long mma_rows(int d, int lists) { return d == 64 && lists == 2 ? 32 : 16; }

// Keys up to which no entry is split, so that there is nothing to join.  Few rows: a warp takes
// 0.27 us a tile (16 keys), the join 4 to 5 us, so 128 keys; where the segments keep half of the
// warps busy, 256 (64 sequences of 8 heads and 256 keys: 13.4 and, split, 15.2 us).  The
// tensor-core kernel: 512 (4 sequences of 40 tokens and 300 keys 13.4 and 15.5 us, 32 of 500 keys
// 28.6 and 44).
int unsplit_keys(bool mma, int count, int Hkv) {
  if (mma) return 512;
  return static_cast<long long>(count) * Hkv >= 2 * fa::kPagedCtas ? 256 : 128;
}

// How a call with shared prefixes divides the SMs (lists of both kinds of row tiles): a key tile of
// the tensor-core kernel counts as this many of the other's.  One works at the tensor core's pace
// and the other at memory's, so at once they take less than one after the other: 128 sequences of
// 1..1024 keys behind two prefixes of 32768 133 us instead of 148 (138 with 14 or 24, 160 with 30),
// 64 of 512 keys behind 4096 47 instead of 65; d = 64, 64 of 1024 behind 32768 56 instead of 80 (63
// with 18, 70 with 14). 
constexpr float mma_tile_cost(int d) { return d == 64 ? 30.f : 20.f; }

// Key tiles that a segment of the tensor-core kernel counts besides its own in a call with a tree: a CTA
// takes 7.4 us longer for each piece of its share, as for 3.6 key tiles (queries to load, the pipeline
// to empty and fill, a result to write).  32 trees of 48 to 64 tokens, 8 heads and 2048 to 8192 keys:
// 164.2 us (of a version 1% faster, whose maxima were not exact: 162.1, with 3 163.0, 2 165.3, 0
// 172.9); 64 of them over 512 to 2048 keys 128 and, with 0, 144; of 20 to 30 tokens, 64 over 2048 to
// 8192 keys, 236 and 251.  With fewer sequences and heads than CTAs the parts are what costs: 4 trees
// over 700 keys 22.3 us, with 2 20.6, over 2000 26.3 and 24.6 (with 0 28.9).  Calls without a mask keep
// their division of the work, and with it their results bit for bit.
int tree_extra(int B, int Hkv) { return static_cast<long long>(B) * Hkv >= fa::kPagedCtas ? 4 : 2; }

// Few rows: whether a CTA takes whole segments, its warps an eighth of the keys each, so that there
// is nothing to join.  With a segment per SM at most, up to 1024 keys (d = 128, 8 heads, split and
// whole: one sequence of 128 keys 8.7 and 5.3 us, 500 keys 8.9 and 7.4, 1000 keys 10.2 and 10.2; 16
// sequences of 1000 keys 15.2 and 11.1); with two, from 64 to 512 (32 sequences of 256 keys 12.4
// and 10.4, of 500 15.4 and 13.6, of 32, a warp each, 5.8 and 8.4).  Longer ones would be as slow
// as the longest, and more segments take turns (48 sequences of 256 keys 13.5 and 14.2).
// The first rule holds for more than 16 rows as well (13 sequences of 4 to 9 tokens, 8 heads on one
// and 253 keys: 7.5 us, tensor-core kernel 9.1; one of 256 tokens, 8 heads and 1000 keys: 12.1 and
// 18.4).
bool whole_segments(long long segments, bool many_rows, int max_kv) {
  if (segments <= fa::kPagedCtas) return max_kv <= 1024;
  return segments <= 2 * fa::kPagedCtas && !many_rows && max_kv > 64 && max_kv <= 512;
}

// Few segments that are split: whether CTAs are the workers, an eighth of the parts to join (split
// over warps and over CTAs: one segment of 4000 keys 10.6 and 8.8 us, of 16000 18.1 and 10.1, of
// 64000 32.8 and 14.1; 8 segments of 2000 keys 10.8 and 11.5, of 32000 31.5 and 27.5; 16 of 8000
// 14.5 and 16.0).  Segments of up to 64 tiles are whole.
constexpr int kUnsplitTilesTogether = 64;
bool cta_workers(long long segments, int max_kv) {
  return segments <= 8 && max_kv >= 500 * segments;
}

// The same behind a shared prefix, which is then read (from L2) for each sequence: 0.55 us per 100
// keys and turn at d = 128, 0.4 at d = 64, against 10 to 20 us of two lists and a join.  d = 128, 8
// heads, prefix + own keys, two lists and whole: 4 sequences of 256 + 16 10.5 and 7.6 us, of 1000 +
// 24 12.5 and 12.2, 16 of 1000 + 24 17.2 and 12.5, 38 of 500 + 64 (two turns) 23.0 and 16.0 but of
// 1000 + 24 19.6 and 21.8, 48 of 256 + 256 (three) 28 and 20; d = 64, 8 of 1500 + 64 13.5 and 11.7.
bool whole_with_prefix(long long segments, int d, long long max_keys) {
  const long long turns = (segments + fa::kPagedCtas - 1) / fa::kPagedCtas;
  if (turns == 1) return max_keys <= (d == 64 ? 1536 : 1152);
  return (turns == 2 && max_keys <= 640) || (turns == 3 && max_keys <= 512);
}

// Groups of 8 lanes per row of the join.  A group reads its parts two at a time (four where
// several share a row), so few rows, which have many parts, take more groups: 128 rows of 39 parts 292 us with 16, 306 with 1 (4 x 131072
// keys); 1472 rows of 19 parts 36 with 4, 41 with 1, 40 with 16; 4096 rows of 6 parts 135 with 1,
// 141 with 4, 160 with 16.
int join_split(long long rows) {
  return rows <= 4 * fa::kPagedCtas ? 16 : (rows <= 16 * fa::kPagedCtas ? 4 : 1);
}

// Workspace of a paged call: the spans and slots of each list, then (joined lists) row buffers.
// Which kernel a list takes is decided by the query rows of an entry (of the sequences by max_q, of
// the groups by their average) and by the rules for whole segments above; with few rows in all it
// cannot be the tensor-core one, whose slots are larger.
struct PagedWorkspace {
  size_t spans[2], slots[2], rowbuf[2], total;
};
PagedWorkspace paged_workspace(const int (&count)[2], int lists, int total, int H, int Hkv, int d) {
  PagedWorkspace w{};
  size_t at = 0;
  size_t slots = static_cast<size_t>(fa::kPagedCtas) * fa::kPagedWarps * 2 * fa::kPagedRows *
                 (d + 2) * 4;
  if (static_cast<long long>(total) * (H / Hkv) > mma_rows(d, lists)) {
    const size_t mma = static_cast<size_t>(fa::kPagedCtas) * 2 * fa::kPagedMmaRows * (d + 2) * 4;
    if (mma > slots) slots = mma;
  }
  for (int i = 0; i < lists; ++i) {
    w.spans[i] = at;
    at += up256(static_cast<size_t>(Hkv) *
                fa::row_tiles_bound(total, H / Hkv, fa::kPagedRows, count[i]) * sizeof(int2));
    w.slots[i] = at;
    at += up256(slots);
    if (lists > 1) {
      w.rowbuf[i] = at;
      at += up256(static_cast<size_t>(total) * H * (d + 2) * 4);
    }
  }
  w.total = at;
  return w;
}

fa_status check_paged_sizes(int B, int total, int H, int Hkv, int d) {
  fa_status st = check_heads(H, Hkv, d);
  if (st != FA_OK) return st;
  if (B <= 0 || total < 0 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (H / Hkv > 128) return FA_ERR_UNSUPPORTED;
  // rows of every tile and the index of a (token, head) row fit 32 bits
  if ((static_cast<long long>(total) + B) * H + 256LL * B > kMaxInt) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// never quite 0 (a scale of 0): a hidden key's score of -inf has to stay -inf when scaled
float scale_log2_of(float scale, int d) {
  return std::fmax(fa::resolve_scale(scale, d) * kLog2e, std::numeric_limits<float>::denorm_min());
}

// tree: the mask of a tree of new tokens (causal is then 0), or nullptr.
fa_status paged_impl(const void* Q, const fa_paged_kv* cache, const fa_prefix* prefix,
                     const uint64_t* tree, int tree_words, void* O, float* LSE, const int32_t* cu,
                     int B, int max_q, int max_kv, int total, int H, int Hkv, int d, int causal,
                     float scale, void* ws, size_t ws_bytes, cudaStream_t s) {
  fa_status st = check_paged_sizes(B, total, H, Hkv, d);
  if (st != FA_OK) return st;
  if (max_q < 1 || max_kv < 0 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (cu == nullptr && total != B) return FA_ERR_INVALID_ARG;
  if ((st = check_cache(cache)) != FA_OK) return st;
  if (prefix != nullptr &&
      (prefix->groups < 1 || prefix->max_len < 0 || prefix->max_pages < 0 ||
       (prefix->max_pages > 0 && prefix->table == nullptr) || prefix->lens == nullptr ||
       prefix->group_cu == nullptr))
    return FA_ERR_INVALID_ARG;
  if (total == 0) return FA_OK;
  if (!Q || !O || !LSE || !aligned_to(Q, 16) || !aligned_to(O, 16)) return FA_ERR_INVALID_ARG;
  const int lists = prefix != nullptr ? 2 : 1;
  const int count[2] = {B, prefix != nullptr ? prefix->groups : 0};
  // pages x heads is a tensor-map coordinate
  if (static_cast<long long>(cache->num_pages) * Hkv > kMaxInt) return FA_ERR_INVALID_ARG;
  if (lists == 2 && (static_cast<long long>(total) + count[1]) * H + 256LL * count[1] > kMaxInt)
    return FA_ERR_INVALID_ARG;
  bool mma[2];
  bool twin = false, whole = false;
  long long segments = 0;  // of 16 rows at most
  long long units[2];
  for (int i = 0; i < lists; ++i) {
    // query rows of an entry: at most those of max_q tokens; of a group, its share of the batch
    const long long tokens = i == 0 && max_q < total ? max_q : total;
    const long long rows = (i == 0 ? tokens : (total + count[i] - 1) / count[i]) * (H / Hkv);
    mma[i] = rows > mma_rows(d, lists);
    if (i == 0) {
      segments = B * ((rows + fa::kPagedRows - 1) / fa::kPagedRows) * Hkv;
      whole = lists == 1 ? whole_segments(segments, mma[0], max_kv)
                         : whole_with_prefix(segments, d,
                                             static_cast<long long>(max_kv) + prefix->max_len);
      mma[0] = mma[0] && !whole;
      twin = lists == 1 && rows <= 128;
    }
    // row tiles over all entries x heads x key tiles: the units of a launch, which fit 32 bits
    const long long keys = i == 0 ? max_kv : prefix->max_len;
    units[i] = Hkv * static_cast<long long>(fa::row_tiles_bound(
                         total, H / Hkv, mma[i] ? fa::kPagedMmaRows : fa::kPagedRows, count[i])) *
               (keys / (mma[i] ? fa::kPagedMmaKeys : fa::kPagedKeys) + 1 + (tree != nullptr && mma[i] ? tree_extra(B, Hkv) : 0));
    if (units[i] > kMaxInt) return FA_ERR_UNSUPPORTED;
  }
  const PagedWorkspace w = paged_workspace(count, lists, total, H, Hkv, d);
  if ((st = fa::check_workspace(ws, ws_bytes, w.total)) != FA_OK) return st;
  int* status = nullptr;
  if ((st = device_ready(status)) != FA_OK) return st;

  char* base = static_cast<char*>(ws);
  fa::PagedArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(Q);
  a.k_cache = static_cast<const __nv_bfloat16*>(cache->k_cache);
  a.v_cache = static_cast<const __nv_bfloat16*>(cache->v_cache);
  a.o = static_cast<__nv_bfloat16*>(O);
  a.lse = LSE;
  a.cu = cu;
  a.B = B;
  a.total = total;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.num_pages = cache->num_pages;
  a.page_shift = page_shift(cache->page_size);
  a.scale_log2 = scale_log2_of(scale, d);
  a.status = status;
  a.tree = reinterpret_cast<const uint32_t*>(tree);
  a.tree_words = 2 * tree_words;
  const fa::KeyMode mode = tree != nullptr ? fa::kTreeKeys : fa::kAllKeys;
  fa::JoinArgs j{};
  j.o = a.o;
  j.lse = LSE;
  j.cu = cu;
  j.B = B;
  j.total = total;
  j.H = H;
  j.Hkv = Hkv;
  j.G = a.G;
  j.lists = lists;
  CUtensorMap tk, tv;
  const bool any_mma = !whole && (mma[0] || (lists > 1 && mma[1]));
  if (any_mma &&
      (!make_pool_map(&tk, cache->k_cache, *cache, Hkv, d) ||
       !make_pool_map(&tv, cache->v_cache, *cache, Hkv, d)))
    return FA_ERR_CUDA;
  for (int i = 0; i < lists; ++i) {
    fa::KeyList& l = a.list[i];
    l.count = count[i];
    l.lens = i == 0 ? cache->kv_lens : prefix->lens;
    l.table = i == 0 ? cache->block_table : prefix->table;
    l.max_pages = i == 0 ? cache->max_pages : prefix->max_pages;
    l.max_len = i == 0 ? max_kv : prefix->max_len;
    if (l.max_len > kMaxKeys) l.max_len = kMaxKeys;
    l.max_q = i == 0 ? max_q : kMaxInt;
    l.group_cu = i == 0 ? nullptr : prefix->group_cu;
    l.causal = i == 0 && causal ? 1 : 0;
    l.mma = mma[i];
    l.unsplit = unsplit_keys(mma[i], l.count, Hkv) / (mma[i] ? fa::kPagedMmaKeys : fa::kPagedKeys);
    l.extra = tree != nullptr && mma[i] ? tree_extra(B, Hkv) : 0;
    a.rowbuf[i] = lists > 1 ? reinterpret_cast<float*>(base + w.rowbuf[i]) : nullptr;
    fa::PartialLayout& p = a.part[i];
    p.R = mma[i] ? fa::kPagedMmaRows : fa::kPagedRows;
    p.workers = fa::kPagedCtas * (mma[i] ? 1 : fa::kPagedWarps);
    p.span_tiles = fa::row_tiles_bound(total, a.G, p.R, l.count);
    p.spans = reinterpret_cast<int2*>(base + w.spans[i]);
    p.slots = reinterpret_cast<float*>(base + w.slots[i]);
    j.list[i] = l;
    j.part[i] = p;
    j.rowbuf[i] = a.rowbuf[i];
  }
  a.mma_cost = mma_tile_cost(d);
  if (whole) {
    a.list[0].unsplit = kMaxInt;
    return status_of(fa::launch_paged_cta(d, mode, a, lists, segments, s));
  }
  const long long all = units[0] + (lists > 1 ? units[1] : 0);
  const bool together = lists == 1 && !mma[0] && cta_workers(segments, max_kv);
  if (together) {
    a.part[0].workers = j.part[0].workers = fa::kPagedCtas;
    a.list[0].unsplit = j.list[0].unsplit = kUnsplitTilesTogether;
  }
  const cudaError_t e =
      together ? fa::launch_paged_cta(d, mode, a, 1, all, s)
      : any_mma ? fa::launch_paged_mma(d, mode, tk, tv, a, lists, twin, all, fa::wait_timeout_ns(), s)
              : fa::launch_paged(d, mode, a, lists, all, s);
  if ((st = status_of(e)) != FA_OK) return st;
  // no entry can have been split (lengths are clamped to max_kv): every result is final
  if (lists == 1 && max_kv <= unsplit_keys(mma[0], B, Hkv))
    return FA_OK;
  return status_of(fa::launch_paged_join(d, j, join_split(static_cast<long long>(total) * H), s));
}

// Attention over selected pages: every token is an entry of its own with top * page_size keys.
fa_status selected_impl(const void* Q, const fa_paged_kv* cache, const int32_t* pages, int top,
                        void* O, float* LSE, const int32_t* cu, int B, int total, int H, int Hkv,
                        int d, float scale, void* ws, size_t ws_bytes, cudaStream_t s) {
  if (B <= 0 || total < 0 || top < 1 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  fa_status st = check_paged_sizes(total > 0 ? total : 1, total, H, Hkv, d);
  if (st != FA_OK) return st;
  if (cu == nullptr && total != B) return FA_ERR_INVALID_ARG;
  if ((st = check_cache(cache)) != FA_OK) return st;
  if (total == 0) return FA_OK;
  if (!Q || !O || !LSE || !pages || !aligned_to(Q, 16) || !aligned_to(O, 16))
    return FA_ERR_INVALID_ARG;
  const long long keys = static_cast<long long>(top) * cache->page_size;
  const int count[2] = {total, 0}, G = H / Hkv;
  const long long units = Hkv * static_cast<long long>(fa::row_tiles_bound(total, G, fa::kPagedRows, total)) *
                          (keys / fa::kPagedKeys + 1);
  if (keys > kMaxKeys || units > kMaxInt) return FA_ERR_UNSUPPORTED;
  const PagedWorkspace w = paged_workspace(count, 1, total, H, Hkv, d);
  if ((st = fa::check_workspace(ws, ws_bytes, w.total)) != FA_OK) return st;
  int* status = nullptr;
  if ((st = device_ready(status)) != FA_OK) return st;

  char* base = static_cast<char*>(ws);
  fa::PagedArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(Q);
  a.k_cache = static_cast<const __nv_bfloat16*>(cache->k_cache);
  a.v_cache = static_cast<const __nv_bfloat16*>(cache->v_cache);
  a.o = static_cast<__nv_bfloat16*>(O);
  a.lse = LSE;
  a.B = total;
  a.total = total;
  a.H = H;
  a.Hkv = Hkv;
  a.G = G;
  a.num_pages = cache->num_pages;
  a.page_shift = page_shift(cache->page_size);
  a.scale_log2 = scale_log2_of(scale, d);
  a.status = status;
  a.pages = pages;
  a.top = top;
  a.seq_cu = cu;
  a.seq_lens = cache->kv_lens;
  a.seqs = B;
  fa::KeyList& l = a.list[0];
  l.count = total;
  l.table = cache->block_table;
  l.max_pages = cache->max_pages;
  l.max_len = static_cast<int>(keys);
  l.max_q = kMaxInt;
  const long long segments = static_cast<long long>(total) * ((G + fa::kPagedRows - 1) / fa::kPagedRows) * Hkv;
  const bool whole = whole_segments(segments, false, l.max_len);
  const bool together = !whole && cta_workers(segments, l.max_len);
  l.unsplit = whole      ? kMaxInt
              : together ? kUnsplitTilesTogether
                         : unsplit_keys(false, total, Hkv) / fa::kPagedKeys;
  fa::PartialLayout& p = a.part[0];
  p.R = fa::kPagedRows;
  p.workers = fa::kPagedCtas * (together ? 1 : fa::kPagedWarps);
  p.span_tiles = fa::row_tiles_bound(total, G, p.R, total);
  p.spans = reinterpret_cast<int2*>(base + w.spans[0]);
  p.slots = reinterpret_cast<float*>(base + w.slots[0]);
  if (whole) return status_of(fa::launch_paged_cta(d, fa::kSelectedKeys, a, 1, segments, s));
  const cudaError_t e = together ? fa::launch_paged_cta(d, fa::kSelectedKeys, a, 1, units, s)
                                 : fa::launch_paged(d, fa::kSelectedKeys, a, 1, units, s);
  if ((st = status_of(e)) != FA_OK) return st;
  if (l.max_len / fa::kPagedKeys <= l.unsplit) return FA_OK;  // every result is final
  fa::JoinArgs j{};
  j.o = a.o;
  j.lse = LSE;
  j.B = total;
  j.total = total;
  j.H = H;
  j.Hkv = Hkv;
  j.G = G;
  j.lists = 1;
  j.list[0] = l;
  j.part[0] = p;
  j.seq_cu = cu;
  j.seqs = B;
  return status_of(fa::launch_paged_join(d, j, join_split(static_cast<long long>(total) * H), s));
}

}  // namespace

extern "C" {

fa_status fa_rope_table(const double* inv_freq, int rot, int n_pos, float amplitude,
                        float* table, void* stream) {
  if (!inv_freq || !table || rot < 2 || rot > 1024 || rot % 2 != 0 || n_pos < 1)
    return FA_ERR_INVALID_ARG;
  if (!aligned_to(inv_freq, 8) || !aligned_to(table, 4) || !std::isfinite(amplitude))
    return FA_ERR_INVALID_ARG;
  const fa_status st = fa::check_device();
  if (st != FA_OK) return st;
  return status_of(fa::launch_rope_table(inv_freq, rot, n_pos, amplitude, table,
                                         static_cast<cudaStream_t>(stream)));
}

fa_status fa_qk_norm_rope_fwd(const fa_view in[3], const fa_view out[3],
                              const int32_t* positions, int B, int N, int H, int Hkv, int d,
                              const fa_qk_transform* t, void* stream) {
  fa_status st = check_heads(H, Hkv, d);
  if (st != FA_OK) return st;
  if ((st = check_transform(t, d)) != FA_OK) return st;
  if (B <= 0 || N < 0 || static_cast<long long>(B) * N > kMaxInt) return FA_ERR_INVALID_ARG;
  if (N == 0) return FA_OK;
  if (t->table != nullptr && positions == nullptr && N > t->n_pos) return FA_ERR_INVALID_ARG;
  if (in == nullptr || out == nullptr) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (i == 2 && in[2].data == nullptr) break;  // no V
    if (!view_ok(in[i], B, N, i == 0 ? H : Hkv) || !view_ok(out[i], B, N, i == 0 ? H : Hkv))
      return FA_ERR_INVALID_ARG;
  }
  fa::RopeArgs a{};
  if ((st = device_ready(a.status)) != FA_OK) return st;
  set_transform(a, *t);
  a.q = row_view(in[0]);
  a.k = row_view(in[1]);
  a.v = row_view(in[2]);
  a.qo = row_view(out[0]);
  a.ko = row_view(out[1]);
  a.vo = row_view(out[2]);
  a.B = B;
  a.N = N;
  a.tokens = B * N;
  a.H = H;
  a.Hkv = Hkv;
  a.positions = positions;
  return status_of(fa::launch_rope_fwd(d, t->interleaved != 0, /*paged=*/false, a,
                                       static_cast<cudaStream_t>(stream)));
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  return static_cast<size_t>(fa::kRopeBwdBlocks + 2) * d * sizeof(float);
}

fa_status fa_qk_norm_rope_bwd(const fa_view grad[3], const fa_view x[2], const fa_view out[3],
                              float* dq_weight, float* dk_weight, const int32_t* positions,
                              int B, int N, int H, int Hkv, int d, const fa_qk_transform* t,
                              void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_heads(H, Hkv, d);
  if (st != FA_OK) return st;
  if ((st = check_transform(t, d)) != FA_OK) return st;
  if (B <= 0 || N < 0 || static_cast<long long>(B) * N > kMaxInt) return FA_ERR_INVALID_ARG;
  const bool norm = t->q_weight != nullptr;
  if (norm) {
    if (!dq_weight || !dk_weight) return FA_ERR_INVALID_ARG;
    if ((st = fa::check_workspace(workspace, workspace_bytes,
                                  fa_qk_norm_rope_bwd_workspace_size(d))) != FA_OK)
      return st;
  }
  if (N == 0 && !norm) return FA_OK;
  if (t->table != nullptr && positions == nullptr && N > t->n_pos) return FA_ERR_INVALID_ARG;
  if (N > 0) {
    if (grad == nullptr || out == nullptr || (norm && x == nullptr)) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
      const int h = i == 0 ? H : Hkv;
      if (i == 2 && grad[2].data == nullptr) break;  // no V
      if (!view_ok(grad[i], B, N, h) || !view_ok(out[i], B, N, h)) return FA_ERR_INVALID_ARG;
      if (norm && i < 2 && !view_ok(x[i], B, N, h)) return FA_ERR_INVALID_ARG;
    }
  }
  fa::RopeArgs a{};
  if ((st = device_ready(a.status)) != FA_OK) return st;
  set_transform(a, *t);
  if (N > 0) {
    a.q = row_view(grad[0]);
    a.k = row_view(grad[1]);
    a.v = row_view(grad[2]);
    a.qo = row_view(out[0]);
    a.ko = row_view(out[1]);
    a.vo = row_view(out[2]);
    if (norm) {
      a.qx = row_view(x[0]);
      a.kx = row_view(x[1]);
    }
  }
  a.B = B;
  a.N = N;
  a.tokens = B * N;
  a.H = H;
  a.Hkv = Hkv;
  a.positions = positions;
  a.partial = static_cast<float*>(workspace);
  return status_of(fa::launch_rope_bwd(d, t->interleaved != 0, a, dq_weight, dk_weight,
                                       static_cast<cudaStream_t>(stream)));
}

fa_status fa_kv_append(const fa_view in[3], const fa_view* q_out, const fa_paged_kv* cache,
                       const int32_t* cu_seqlens, const int32_t* pos_offset, int B, int total,
                       int H, int Hkv, int d, const fa_qk_transform* t, void* stream) {
  fa_status st = check_heads(H, Hkv, d);
  if (st != FA_OK) return st;
  if ((st = check_transform(t, d)) != FA_OK) return st;
  if ((st = check_cache(cache)) != FA_OK) return st;
  if (B <= 0 || total < 0 || cache->max_pages < 1) return FA_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr && total != B) return FA_ERR_INVALID_ARG;
  if (total == 0) return FA_OK;
  if (in == nullptr || !view_ok(in[1], 1, total, Hkv) || !view_ok(in[2], 1, total, Hkv))
    return FA_ERR_INVALID_ARG;
  const bool with_q = in[0].data != nullptr;
  if (with_q && (q_out == nullptr || !view_ok(in[0], 1, total, H) || !view_ok(*q_out, 1, total, H)))
    return FA_ERR_INVALID_ARG;
  fa::RopeArgs a{};
  if ((st = device_ready(a.status)) != FA_OK) return st;
  set_transform(a, *t);
  a.q = row_view(in[0]);
  a.k = row_view(in[1]);
  a.v = row_view(in[2]);
  if (with_q) a.qo = row_view(*q_out);
  a.B = 1;
  a.N = total;
  a.tokens = total;
  a.H = H;
  a.Hkv = Hkv;
  a.k_cache = static_cast<__nv_bfloat16*>(cache->k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(cache->v_cache);
  a.block_table = cache->block_table;
  a.kv_lens = cache->kv_lens;
  a.cu = cu_seqlens;
  a.pos_offset = pos_offset;
  a.max_pages = cache->max_pages;
  a.num_pages = cache->num_pages;
  a.page_shift = page_shift(cache->page_size);
  a.seqs = B;
  return status_of(fa::launch_rope_fwd(d, t->interleaved != 0, /*paged=*/true, a,
                                       static_cast<cudaStream_t>(stream)));
}

size_t fa_fwd_paged_workspace_size(int B, int total, int H, int Hkv, int d) {
  if (check_paged_sizes(B, total, H, Hkv, d) != FA_OK) return 0;
  const int count[2] = {B, 0};
  return paged_workspace(count, 1, total, H, Hkv, d).total;
}

fa_status fa_fwd_paged(const void* Q, const fa_paged_kv* cache, void* O, float* LSE,
                       const int32_t* cu_seqlens, int B, int max_q, int max_kv, int total, int H,
                       int Hkv, int d, int causal, float scale, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return paged_impl(Q, cache, nullptr, nullptr, 0, O, LSE, cu_seqlens, B, max_q, max_kv, total, H, Hkv, d,
                    causal, scale, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

fa_status fa_fwd_paged_tree(const void* Q, const fa_paged_kv* cache, const uint64_t* tree_mask,
                            int mask_words, void* O, float* LSE, const int32_t* cu_seqlens, int B,
                            int max_q, int max_kv, int total, int H, int Hkv, int d, float scale,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (mask_words < 1 || mask_words > (1 << 24)) return FA_ERR_INVALID_ARG;
  if (total > 0 && (!tree_mask || !aligned_to(tree_mask, 8))) return FA_ERR_INVALID_ARG;
  return paged_impl(Q, cache, nullptr, total > 0 ? tree_mask : nullptr, mask_words, O, LSE, cu_seqlens,
                    B, max_q, max_kv, total, H, Hkv, d, 0, scale, workspace, workspace_bytes,
                    static_cast<cudaStream_t>(stream));
}

size_t fa_fwd_paged_selected_workspace_size(int total, int H, int Hkv, int d) {
  if (check_paged_sizes(total > 0 ? total : 1, total, H, Hkv, d) != FA_OK) return 0;
  const int count[2] = {total, 0};
  return paged_workspace(count, 1, total, H, Hkv, d).total;
}

fa_status fa_fwd_paged_selected(const void* Q, const fa_paged_kv* cache, const int32_t* pages,
                                int top, void* O, float* LSE, const int32_t* cu_seqlens, int B,
                                int total, int H, int Hkv, int d, float scale, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return selected_impl(Q, cache, pages, top, O, LSE, cu_seqlens, B, total, H, Hkv, d, scale,
                       workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

size_t fa_fwd_shared_prefix_workspace_size(int B, int groups, int total, int H, int Hkv, int d) {
  if (check_paged_sizes(B, total, H, Hkv, d) != FA_OK || groups < 1) return 0;
  if ((static_cast<long long>(total) + groups) * H + 256LL * groups > kMaxInt) return 0;
  const int count[2] = {B, groups};
  return paged_workspace(count, 2, total, H, Hkv, d).total;
}

fa_status fa_fwd_shared_prefix(const void* Q, const fa_paged_kv* cache, const fa_prefix* prefix,
                               void* O, float* LSE, const int32_t* cu_seqlens, int B, int max_q,
                               int max_kv, int total, int H, int Hkv, int d, int causal,
                               float scale, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (prefix == nullptr) return FA_ERR_INVALID_ARG;
  return paged_impl(Q, cache, prefix, nullptr, 0, O, LSE, cu_seqlens, B, max_q, max_kv, total, H, Hkv, d,
                    causal, scale, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
