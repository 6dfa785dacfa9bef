// Norms and rotary positions of queries and keys: one pass from the projection's rows to the
// attention layout (or into a paged cache), and its backward.
//
// A row is one head of one token, d bf16 elements.
//   forward:   r = rsqrt(mean(x^2) + eps),  y = x r w,  (a, b) -> (a cos - b sin, a sin + b cos)
//   backward:  g = the inverse rotation of dz,  dw = sum over rows of g x r,
//              u = g w,  dx = r (u - x r mean(u x r))
// Bound by memory: a row is read and written once and nothing else of size moves.  D / 8 lanes
// hold a row, 8 elements each, arranged so that both elements of every rotation pair are in one
// lane: with interleaved pairs a lane holds 8 consecutive elements (one 16-byte access); with
// the half layout it holds 4 consecutive elements of the first half and their 4 partners (two
// 8-byte accesses, each coalesced over the lanes).  A lane group keeps its token's cos and sin in
// registers and walks over heads, four rows at a time so that four rows' loads are in flight.
// A CTA's rows are all of Q, of K or of V: one set of weights, and no choice per row.  The
// arithmetic is in packed pairs: with scalar operations and a choice of weights per row the
// instructions, not memory, set the pace (16384 tokens of 48 heads, forward 82, backward 171 us).
#include "fa_internal.h"
#include "fa_paged.h"
#include "sm103.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = 4;  // rows of a lane group in flight

// The pairs 4j .. 4j+3 of lane j: element offsets of its two groups of four elements (half
// layout) or of its eight (interleaved: off0, off0 + 4).
template <int D, bool kInter>
struct LanePairs {
  int off0, off1;
  bool turned;  // inside the rotated part
  __device__ LanePairs(int j, int rot) {
    if (kInter) {
      off0 = 8 * j;
      off1 = off0 + 4;
      turned = off0 < rot;
    } else {
      const int p = 4 * j, half = rot >> 1;  // rot is a multiple of 16: groups do not straddle
      turned = p < half;
      off0 = turned ? p : rot + (p - half);
      off1 = off0 + (turned ? half : (D - rot) >> 1);
    }
  }
};

struct Row8 {
  uint2 a, b;  // the lane's two groups of four bf16
};

template <bool kInter>
__device__ __forceinline__ Row8 load_row(const __nv_bfloat16* row, int gap) {
  Row8 r;
  if (kInter) {
    const uint4 v = *reinterpret_cast<const uint4*>(row);
    r.a = make_uint2(v.x, v.y);
    r.b = make_uint2(v.z, v.w);
  } else {
    r.a = *reinterpret_cast<const uint2*>(row);
    r.b = *reinterpret_cast<const uint2*>(row + gap);
  }
  return r;
}
template <bool kInter>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int gap, const Row8& r) {
  if (kInter) {
    *reinterpret_cast<uint4*>(row) = make_uint4(r.a.x, r.a.y, r.b.x, r.b.y);
  } else {
    *reinterpret_cast<uint2*>(row) = r.a;
    *reinterpret_cast<uint2*>(row + gap) = r.b;
  }
}

// The lane's eight values as four packed pairs, in memory order.
struct Vec8 {
  float2 v[4];
};
__device__ __forceinline__ float2 pair_of(uint32_t u) {
  return make_float2(bf16_lo(u), bf16_hi(u));
}
__device__ __forceinline__ Vec8 unpack(const Row8& r) {
  return {{pair_of(r.a.x), pair_of(r.a.y), pair_of(r.b.x), pair_of(r.b.y)}};
}
__device__ __forceinline__ Row8 pack(const Vec8& x) {
  Row8 r;
  r.a = make_uint2(pack_bf16(x.v[0].x, x.v[0].y), pack_bf16(x.v[1].x, x.v[1].y));
  r.b = make_uint2(pack_bf16(x.v[2].x, x.v[2].y), pack_bf16(x.v[3].x, x.v[3].y));
  return r;
}
__device__ __forceinline__ float dot(const Vec8& a, const Vec8& b) {
  float2 s = mul2(a.v[0], b.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(a.v[i], b.v[i], s);
  return s.x + s.y;
}

// cos and sin of the lane's four pairs.
struct Angles {
  float2 c[2], s[2];
};

// Rotates the lane's pairs; lanes outside the rotated part keep their elements untouched (not
// multiplied by 1 and 0: an infinity there must not reach its neighbour).
template <bool kInter>
__device__ __forceinline__ void turn(Vec8& x, const Angles& t, bool turned) {
  if (!turned) return;
  if (kInter) {  // v[i] is pair i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = i & 1 ? t.c[i / 2].y : t.c[i / 2].x, s = i & 1 ? t.s[i / 2].y : t.s[i / 2].x;
      const float a = x.v[i].x, b = x.v[i].y;
      x.v[i] = fma2(make_float2(-b, a), make_float2(s, s), mul2(make_float2(a, b), make_float2(c, c)));
    }
  } else {  // v[i] and v[i + 2] are the first and second elements of pairs 2i, 2i + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = x.v[i], b = x.v[i + 2];
      x.v[i] = fma2(make_float2(-b.x, -b.y), t.s[i], mul2(a, t.c[i]));
      x.v[i + 2] = fma2(b, t.c[i], mul2(a, t.s[i]));
    }
  }
}

// Sum over the L lanes of a row's lane group (`mask`: those lanes of the warp).
template <int L>
__device__ __forceinline__ float group_sum(float v, unsigned mask) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

__device__ __forceinline__ Vec8 load_weight(const float* w, int off0, int off1) {
  const float4 a = *reinterpret_cast<const float4*>(w + off0);
  const float4 b = *reinterpret_cast<const float4*>(w + off1);
  return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}

// cos and sin of the lane's pairs at position pos (clamped to the table).
__device__ __forceinline__ Angles load_angles(const RopeArgs& a, int pos, int j, bool turned,
                                              bool report) {
  Angles t{};
  if (a.table == nullptr) return t;
  if (pos < 0 || pos >= a.n_pos) {
    if (report) atomicCAS(a.status, 0, kErrIndex);
    pos = pos < 0 ? 0 : a.n_pos - 1;
  }
  if (!turned) return t;
  const float* row = a.table + static_cast<int64_t>(pos) * a.rot + 4 * j;
  const float4 c = *reinterpret_cast<const float4*>(row);
  const float4 s = *reinterpret_cast<const float4*>(row + (a.rot >> 1));
  t.c[0] = make_float2(c.x, c.y);
  t.c[1] = make_float2(c.z, c.w);
  t.s[0] = make_float2(s.x, s.y);
  t.s[1] = make_float2(s.z, s.w);
  return t;
}

// Address of row (b, n, head) of a view.
__device__ __forceinline__ __nv_bfloat16* row_of(const RowView& v, int b, int n, int h) {
  return v.p + b * v.batch + n * v.token + h * v.head;
}

// Rows h0 .. h1 - 1 of Q, K or V: kind 0, 1, 2.
struct HeadRange {
  int kind, h0, h1;
};
__host__ __device__ inline int chunks_of(int heads, int chunk) { return (heads + chunk - 1) / chunk; }
__device__ __forceinline__ HeadRange head_range(const RopeArgs& a, int i) {
  HeadRange r{0, i * a.chunk, 0};
  const int cq = chunks_of(a.H, a.chunk), ck = chunks_of(a.Hkv, a.chunk);
  if (i >= cq) {
    r.kind = i < cq + ck ? 1 : 2;
    r.h0 = (i - cq - (r.kind == 2 ? ck : 0)) * a.chunk;
  }
  r.h1 = min(r.h0 + a.chunk, r.kind == 0 ? a.H : a.Hkv);
  return r;
}

// Forward.  Block: kThreads / (D / 8) tokens; grid y: chunks of heads (q, then k, then v).
template <int D, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const RopeArgs a) {
  constexpr int L = D / 8;
  begin_launch();
  const int j = threadIdx.x % L;
  const int64_t t64 = static_cast<int64_t>(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
  if (t64 >= a.tokens) return;
  const int t = static_cast<int>(t64);
  const unsigned lane = threadIdx.x & 31u;
  const unsigned mask = ((1u << L) - 1u) << (lane & ~(L - 1u));
  const HeadRange hr = head_range(a, blockIdx.y);
  const RowView& in = hr.kind == 0 ? a.q : (hr.kind == 1 ? a.k : a.v);
  if (in.p == nullptr) return;  // no Q, or no V

  int b, n, pos;
  int64_t slot = -1;  // paged: element offset of the token's first head, or -1
  if constexpr (kPaged) {
    const int seq = token_sequence_group<L>(a.cu, a.seqs, t, j, mask);
    if (seq < 0) return;  // behind the last sequence
    int start, count;
    token_bounds(a.cu, seq, a.tokens, start, count);
    if (t < start || t >= start + count) {  // offsets that do not ascend
      if (j == 0) atomicCAS(a.status, 0, kErrIndex);
      return;
    }
    const int64_t limit = static_cast<int64_t>(a.max_pages) << a.page_shift;
    const int len = __ldg(a.kv_lens + seq);
    const int key = max(len, 0) - count + (t - start);
    b = 0;
    n = t;
    pos = key;
    if (a.pos_offset != nullptr) {  // a sum past 32 bits is past the table as well
      const int64_t p = static_cast<int64_t>(key) + __ldg(a.pos_offset + seq);
      pos = p < 0 ? -1 : (p < a.n_pos ? static_cast<int>(p) : a.n_pos);
    }
    if (key >= 0) {
      const int page =
          key < limit ? resolve_page(a.block_table + static_cast<int64_t>(seq) * a.max_pages,
                                     a.max_pages, a.num_pages, a.page_shift, key)
                      : -1;
      if (page >= 0)
        slot = ((static_cast<int64_t>(page) * a.Hkv << a.page_shift) +
                (key & ((1 << a.page_shift) - 1))) * D;
      else if (j == 0)
        atomicCAS(a.status, 0, kErrIndex);
    } else if (len < 0 && j == 0) {
      atomicCAS(a.status, 0, kErrIndex);
    }
    if (key < 0) pos = 0;  // never written; its Q row is still defined
  } else {
    b = t / a.N;
    n = t - b * a.N;
    pos = a.positions != nullptr ? __ldg(a.positions + t) : n;
  }

  const LanePairs<D, kInter> lp(j, a.rot);
  const bool turned = a.table != nullptr && lp.turned;
  const int gap = lp.off1 - lp.off0;
  const __nv_bfloat16* src = row_of(in, b, n, hr.h0) + lp.off0;
  __nv_bfloat16* dst;
  int64_t src_step = in.head, dst_step;
  if (kPaged && hr.kind != 0) {
    if (slot < 0) return;
    dst_step = static_cast<int64_t>(D) << a.page_shift;
    dst = (hr.kind == 1 ? a.k_cache : a.v_cache) + slot + hr.h0 * dst_step + lp.off0;
  } else {
    const RowView& out = hr.kind == 0 ? a.qo : (hr.kind == 1 ? a.ko : a.vo);
    dst_step = out.head;
    dst = row_of(out, b, n, hr.h0) + lp.off0;
  }
  const float* weight = hr.kind == 0 ? a.wq : a.wk;
  const bool norm = weight != nullptr;
  Angles angles{};
  Vec8 w{};
  if (hr.kind != 2) {
    angles = load_angles(a, pos, j, turned, j == 0);
    if (norm) w = load_weight(weight, lp.off0, lp.off1);
  }

  for (int h = hr.h0; h < hr.h1; h += kRows) {
    const int rows = hr.h1 - h;
    Row8 r[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i < rows) r[i] = load_row<kInter>(src + i * src_step, gap);
    if (hr.kind != 2) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i >= rows) break;
        Vec8 x = unpack(r[i]);
        if (norm) {
          const float rs = rsqrtf(group_sum<L>(dot(x, x), mask) * (1.f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < 4; ++e) x.v[e] = mul2(x.v[e], mul2(w.v[e], make_float2(rs, rs)));
        }
        turn<kInter>(x, angles, turned);
        r[i] = pack(x);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i < rows) store_row<kInter>(dst + i * dst_step, gap, r[i]);
    src += kRows * src_step;
    dst += kRows * dst_step;
  }
}

// ---- backward
// Work items are (token group, head chunk).  The grid is persistent and split between Q, K and V
// (blocks [0, first_k), [first_k, first_v) and the rest), so that with norms a thread sums the
// weight gradients of its eight elements over all its rows, a block leaves one partial [D], and
// the sum over blocks (rope_dw_kernel) has a fixed order.  Rows come through a ring of
// shared-memory stages filled by cp.async, one stage ahead of the arithmetic; a lane group reads
// back only its own rows, so a warp-level barrier a stage is all the ring needs.  16384 tokens of
// 48 heads: 97 us (548 MB, 5.6 TB/s); with each lane copying the two 8-byte halves that it reads,
// through L1, 103, with loads into registers 110; 5 blocks an SM 97, 4 blocks 100, 6 blocks (no L1
// left) 101; three stages 102, half as many rows a stage 109; 4 or 16 heads an item 19% and 4%
// slower (an item's rows are far apart in the attention layout and next to each other in the
// projection's).
constexpr int kBwdRows = 4;    // rows of a stage
constexpr int kBwdStages = 2;
constexpr uint32_t kBwdStage = kBwdRows * 2 * 16 * kThreads;  // dz and x, 16 bytes a thread and row
constexpr uint32_t kBwdSmem = kBwdStages * kBwdStage;
constexpr int kBwdBlocksPerSm = 5;

__device__ __forceinline__ void copy16(uint32_t dst, const __nv_bfloat16* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The lane's two groups of four of a row in shared memory.
template <bool kInter>
__device__ __forceinline__ Row8 read_row(uint32_t row, int off0, int off1) {
  Row8 r;
  if (kInter) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.b.x), "=r"(r.b.y)
                 : "r"(row + 2 * off0)
                 : "memory");
  } else {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                 : "=r"(r.a.x), "=r"(r.a.y)
                 : "r"(row + 2 * off0)
                 : "memory");
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                 : "=r"(r.b.x), "=r"(r.b.y)
                 : "r"(row + 2 * off1)
                 : "memory");
  }
  return r;
}

// Walks a lane group's rows, kBwdRows at a time.
template <int G>
struct RowCursor {
  int64_t it, items, step;
  int grp, heads, chunks;
  int b, n, t, h, h1;  // current token and the heads that are left of the item

  __device__ bool settle(const RopeArgs& a) {  // moves to the first item from `it` that has a token
    for (; it < items; it += step) {
      const int64_t t64 = it / chunks * G + grp;
      if (t64 >= a.tokens) continue;
      t = static_cast<int>(t64);
      h = static_cast<int>(it % chunks) * a.chunk;
      h1 = min(h + a.chunk, heads);
      b = t / a.N;
      n = t - b * a.N;
      return true;
    }
    return false;
  }
  __device__ bool next(const RopeArgs& a) {
    h += kBwdRows;
    if (h < h1) return true;
    it += step;
    return settle(a);
  }
};

template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, kBwdBlocksPerSm) rope_bwd_kernel(const RopeArgs a) {
  constexpr int L = D / 8, G = kThreads / L;
  extern __shared__ __align__(16) uint8_t ring[];
  begin_launch();
  const int j = threadIdx.x % L, grp = threadIdx.x / L;
  const unsigned lane = threadIdx.x & 31u;
  const unsigned mask = ((1u << L) - 1u) << (lane & ~(L - 1u));
  const LanePairs<D, kInter> lp(j, a.rot);
  const bool turned = a.table != nullptr && lp.turned;
  const int gap = lp.off1 - lp.off0;
  const int block = blockIdx.x;
  const int kind = block < a.first_k ? 0 : (block < a.first_v ? 1 : 2);
  const int b0 = kind == 0 ? 0 : (kind == 1 ? a.first_k : a.first_v);
  const int b1 = kind == 0 ? a.first_k : (kind == 1 ? a.first_v : static_cast<int>(gridDim.x));
  const RowView& in = kind == 0 ? a.q : (kind == 1 ? a.k : a.v);
  const RowView& out = kind == 0 ? a.qo : (kind == 1 ? a.ko : a.vo);
  const RowView& fwd = kind == 0 ? a.qx : a.kx;
  const float* weight = kind == 0 ? a.wq : a.wk;
  const bool norm = kind != 2 && weight != nullptr;
  Vec8 w{}, dw{};
  if (norm) w = load_weight(weight, lp.off0, lp.off1);
  // row i of dz (k = 0) or x (k = 1) of the lane group: + (2 i + k) 16 kThreads
  const uint32_t base = smem_u32(ring) + grp * (D * 2);

  RowCursor<G> load;
  load.heads = kind == 0 ? a.H : a.Hkv;
  load.chunks = chunks_of(load.heads, a.chunk);
  load.items = (static_cast<int64_t>(a.tokens) + G - 1) / G * load.chunks;
  load.it = block - b0;
  load.step = b1 - b0;
  load.grp = grp;
  RowCursor<G> work = load;
  bool loading = load.settle(a), working = work.settle(a);
  int filled = 0, done = 0;  // stages
  auto fill = [&]() {
    if (loading) {
      const uint32_t st = base + filled % kBwdStages * kBwdStage;
      const __nv_bfloat16* src = row_of(in, load.b, load.n, load.h) + 8 * j;
      const __nv_bfloat16* xs = norm ? row_of(fwd, load.b, load.n, load.h) + 8 * j : nullptr;
#pragma unroll
      for (int i = 0; i < kBwdRows; ++i) {
        if (load.h + i >= load.h1) break;
        copy16(st + i * 2 * 16 * kThreads + 16 * j, src + i * in.head);
        if (norm) copy16(st + (i * 2 + 1) * 16 * kThreads + 16 * j, xs + i * fwd.head);
      }
      loading = load.next(a);
    }
    ++filled;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kBwdStages - 1; ++i) fill();
  Angles angles{};
  int token = -1;
  while (working) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kBwdStages - 2) : "memory");
    __syncwarp(mask);  // the group's copies of this stage are here, its reads of the last one done
    const uint32_t st = base + done % kBwdStages * kBwdStage;
    if (kind != 2 && token != work.t) {
      token = work.t;
      angles = load_angles(a, a.positions != nullptr ? __ldg(a.positions + work.t) : work.n, j,
                           turned, j == 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) angles.s[e] = make_float2(-angles.s[e].x, -angles.s[e].y);
    }
    fill();  // into the stage read one round ago
    __nv_bfloat16* dst = row_of(out, work.b, work.n, work.h) + lp.off0;
#pragma unroll
    for (int i = 0; i < kBwdRows; ++i) {
      if (work.h + i >= work.h1) break;
      Row8 r = read_row<kInter>(st + i * 2 * 16 * kThreads, lp.off0, lp.off1);
      if (kind != 2) {
        Vec8 g = unpack(r);
        turn<kInter>(g, angles, turned);
        if (norm) {
          const Vec8 x = unpack(read_row<kInter>(st + (i * 2 + 1) * 16 * kThreads, lp.off0, lp.off1));
          Vec8 u;
#pragma unroll
          for (int e = 0; e < 4; ++e) u.v[e] = mul2(g.v[e], w.v[e]);
          const float ss = group_sum<L>(dot(x, x), mask), ux = group_sum<L>(dot(u, x), mask);
          const float rs = rsqrtf(ss * (1.f / D) + a.eps);
          // with x r, of the size of 1, in place of x: no power of r, which leaves float32's range
          // long before dx does (rows of rms 1e-13 or 1e15)
          const float c = -(rs * ux) * (1.f / D);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 xr = mul2(x.v[e], make_float2(rs, rs));
            dw.v[e] = fma2(g.v[e], xr, dw.v[e]);
            g.v[e] = mul2(fma2(xr, make_float2(c, c), u.v[e]), make_float2(rs, rs));
          }
        }
        r = pack(g);
      }
      store_row<kInter>(dst + i * out.head, gap, r);
    }
    ++done;
    working = work.next(a);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!norm) return;  // uniform over the block
  __syncthreads();    // the ring becomes [G][D] sums
  float* part = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int at = grp * D + (e < 2 ? lp.off0 + 2 * e : lp.off1 + 2 * (e - 2));
    part[at] = dw.v[e].x;
    part[at + 1] = dw.v[e].y;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) sum += part[g * D + i];
    a.partial[static_cast<int64_t>(block) * D + i] = sum;
  }
}

// dw[q or k][e] = sum over the blocks [0, first_k) or [first_k, first_v): 32 columns a block, 32
// row lanes, joined in a fixed order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* partial, int first_k,
                                                       int first_v, int D, float* dwq, float* dwk) {
  __shared__ float sm[32][33];
  begin_launch();
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const bool of_k = blockIdx.x * 32 >= D;
  const int col = blockIdx.x * 32 + x - (of_k ? D : 0);
  float sum = 0.f;
#pragma unroll 8
  for (int r = (of_k ? first_k : 0) + y; r < (of_k ? first_v : first_k); r += 32)
    sum += partial[static_cast<int64_t>(r) * D + col];
  sm[y][x] = sum;
  __syncthreads();
  if (y == 0) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) s += sm[r][x];
    (of_k ? dwk : dwq)[col] = s;
  }
}

// cos / sin of p * inv_freq[i]: the product and the functions in float64 (a far position times a
// frequency keeps 2^-53 relative precision; in float32 position 10^6 would be off by 0.06 rad).
__global__ void __launch_bounds__(256) rope_table_kernel(const double* inv_freq, int half,
                                                         int64_t count, float amplitude,
                                                         float* table) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= count) return;
  const int64_t p = i / half;
  const int f = static_cast<int>(i - p * half);
  double sn, cs;
  sincos(static_cast<double>(p) * inv_freq[f], &sn, &cs);
  table[p * 2 * half + f] = static_cast<float>(amplitude * cs);
  table[p * 2 * half + half + f] = static_cast<float>(amplitude * sn);
}

// Heads of one work item, at most `most`.  A lane group that walks over many heads loads its
// token's angles and weights once (forward, 16384 tokens of 48 heads: 65 us with 16, 63 with 32);
// few tokens need more groups to cover memory latency.
int head_chunk(int64_t tokens, int heads, int groups_per_block, int most) {
  // about 152 SMs x 8 blocks of lane groups before a group takes more than kRows heads
  const int64_t want = 152ll * 8 * groups_per_block;
  int chunk = kRows;
  while (chunk < most && chunk < heads && tokens * ((heads + 2 * chunk - 1) / (2 * chunk)) >= want)
    chunk *= 2;
  return chunk;
}

template <int D, bool kInter, bool kPaged>
cudaError_t fwd_t(RopeArgs a, cudaStream_t s) {
  constexpr int G = kThreads / (D / 8);
  a.chunk = head_chunk(a.tokens, a.H + 2 * a.Hkv, G, 32);
  const dim3 grid((a.tokens + G - 1) / G, chunks_of(a.H, a.chunk) + 2 * chunks_of(a.Hkv, a.chunk));
  return launch_chained(rope_fwd_kernel<D, kInter, kPaged>, grid, kThreads, 0, s, a);
}

template <int D, bool kInter>
cudaError_t bwd_t(RopeArgs a, float* dwq, float* dwk, cudaStream_t s) {
  constexpr int G = kThreads / (D / 8);
  a.chunk = head_chunk(a.tokens, a.H + 2 * a.Hkv, G, 8);
  const int64_t groups = (static_cast<int64_t>(a.tokens) + G - 1) / G;
  const int64_t items[3] = {groups * chunks_of(a.H, a.chunk), groups * chunks_of(a.Hkv, a.chunk),
                            a.v.p != nullptr ? groups * chunks_of(a.Hkv, a.chunk) : 0};
  // blocks in proportion to a kind's stages and the bytes of their rows (with norms Q and K rows
  // read x too): a stage of one head takes about as long as one of four (11912 tokens of 4 + 1 + 1
  // heads: 14 us, by bytes alone 19; with norms 19 and 25)
  const double cost = a.wq != nullptr ? 3 : 2;
  const double bytes[3] = {cost * chunks_of(a.H, kBwdRows), cost * chunks_of(a.Hkv, kBwdRows),
                           a.v.p != nullptr ? 2.0 * chunks_of(a.Hkv, kBwdRows) : 0.0};
  const double all = bytes[0] + bytes[1] + bytes[2];
  int blocks[3];
  for (int i = 0; i < 3; ++i) {
    int64_t n = static_cast<int64_t>(kRopeBwdBlocks * bytes[i] / all);
    if (n < 1) n = 1;
    blocks[i] = static_cast<int>(n < items[i] ? n : items[i]);
  }
  a.first_k = blocks[0];
  a.first_v = blocks[0] + blocks[1];
  const int grid = a.first_v + blocks[2];
  if (grid > 0) {
    cudaError_t e = ensure_smem_limit<rope_bwd_kernel<D, kInter>>(kBwdSmem);
    if (e != cudaSuccess) return e;
    e = launch_chained(rope_bwd_kernel<D, kInter>, grid, kThreads, kBwdSmem, s, a);
    if (e != cudaSuccess) return e;
  }
  if (a.wq == nullptr) return cudaSuccess;
  return launch_chained(rope_dw_kernel, 2 * D / 32, 1024, 0, s, static_cast<const float*>(a.partial),
                        a.first_k, a.first_v, D, dwq, dwk);
}

}  // namespace

cudaError_t launch_rope_table(const double* inv_freq, int rot, int n_pos, float amplitude,
                              float* table, cudaStream_t s) {
  const int64_t count = static_cast<int64_t>(n_pos) * (rot / 2);
  rope_table_kernel<<<static_cast<unsigned>((count + 255) / 256), 256, 0, s>>>(
      inv_freq, rot / 2, count, amplitude, table);
  return cudaGetLastError();
}

cudaError_t launch_rope_fwd(int d, bool interleaved, bool paged, const RopeArgs& a,
                            cudaStream_t s) {
  if (d == 64) {
    if (paged) return interleaved ? fwd_t<64, true, true>(a, s) : fwd_t<64, false, true>(a, s);
    return interleaved ? fwd_t<64, true, false>(a, s) : fwd_t<64, false, false>(a, s);
  }
  if (paged) return interleaved ? fwd_t<128, true, true>(a, s) : fwd_t<128, false, true>(a, s);
  return interleaved ? fwd_t<128, true, false>(a, s) : fwd_t<128, false, false>(a, s);
}

cudaError_t launch_rope_bwd(int d, bool interleaved, const RopeArgs& a, float* dwq, float* dwk,
                            cudaStream_t s) {
  if (d == 64)
    return interleaved ? bwd_t<64, true>(a, dwq, dwk, s) : bwd_t<64, false>(a, dwq, dwk, s);
  return interleaved ? bwd_t<128, true>(a, dwq, dwk, s) : bwd_t<128, false>(a, dwq, dwk, s);
}

}  // namespace fa
