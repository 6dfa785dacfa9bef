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
// registers and walks over heads, four rows at a time so that four loads are in flight.
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
__device__ __forceinline__ Row8 load_row(const __nv_bfloat16* row, int off0, int off1) {
  Row8 r;
  if (kInter) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + off0);
    r.a = make_uint2(v.x, v.y);
    r.b = make_uint2(v.z, v.w);
  } else {
    r.a = *reinterpret_cast<const uint2*>(row + off0);
    r.b = *reinterpret_cast<const uint2*>(row + off1);
  }
  return r;
}
template <bool kInter>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int off0, int off1, const Row8& r) {
  if (kInter) {
    *reinterpret_cast<uint4*>(row + off0) = make_uint4(r.a.x, r.a.y, r.b.x, r.b.y);
  } else {
    *reinterpret_cast<uint2*>(row + off0) = r.a;
    *reinterpret_cast<uint2*>(row + off1) = r.b;
  }
}
__device__ __forceinline__ void unpack(const Row8& r, float (&x)[8]) {
  x[0] = bf16_lo(r.a.x); x[1] = bf16_hi(r.a.x); x[2] = bf16_lo(r.a.y); x[3] = bf16_hi(r.a.y);
  x[4] = bf16_lo(r.b.x); x[5] = bf16_hi(r.b.x); x[6] = bf16_lo(r.b.y); x[7] = bf16_hi(r.b.y);
}
__device__ __forceinline__ Row8 pack(const float (&x)[8]) {
  Row8 r;
  r.a = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  r.b = make_uint2(pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  return r;
}

// Pair e of the lane is elements (first(e), second(e)) of x.
template <bool kInter>
__device__ __forceinline__ constexpr int first_of(int e) { return kInter ? 2 * e : e; }
template <bool kInter>
__device__ __forceinline__ constexpr int second_of(int e) { return kInter ? 2 * e + 1 : e + 4; }

// Rotates the lane's four pairs by the angle of (c, s); lanes outside the rotated part keep their
// elements untouched (not multiplied by 1 and 0: an infinity there must not reach its neighbour).
template <bool kInter>
__device__ __forceinline__ void turn(float (&x)[8], const float (&c)[4], const float (&s)[4],
                                     bool turned) {
  if (!turned) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = x[first_of<kInter>(e)], b = x[second_of<kInter>(e)];
    x[first_of<kInter>(e)] = a * c[e] - b * s[e];
    x[second_of<kInter>(e)] = a * s[e] + b * c[e];
  }
}

// Sum over the L lanes of a row's lane group (`mask`: those lanes of the warp).
template <int L>
__device__ __forceinline__ float group_sum(float v, unsigned mask) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

__device__ __forceinline__ void load_weight(const float* w, int off0, int off1, float (&r)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(w + off0);
  const float4 b = *reinterpret_cast<const float4*>(w + off1);
  r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
  r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
}

// cos and sin of the lane's pairs at position pos (clamped to the table).
__device__ __forceinline__ void load_angle(const RopeArgs& a, int pos, int j, bool turned,
                                           bool report, float (&c)[4], float (&s)[4]) {
  if (a.table == nullptr) return;
  if (pos < 0 || pos >= a.n_pos) {
    if (report) atomicCAS(a.status, 0, kErrIndex);
    pos = pos < 0 ? 0 : a.n_pos - 1;
  }
  if (!turned) return;
  const float* t = a.table + static_cast<int64_t>(pos) * a.rot + 4 * j;
  const float4 cv = *reinterpret_cast<const float4*>(t);
  const float4 sv = *reinterpret_cast<const float4*>(t + (a.rot >> 1));
  c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
  s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
}

// Address of row (b, n, head) of a view.
__device__ __forceinline__ __nv_bfloat16* row_of(const RowView& v, int b, int n, int h) {
  return v.p + b * v.batch + n * v.token + h * v.head;
}

// Forward.  Block: kThreads / (D / 8) tokens; grid y: chunks of heads (q, then k, then v).
template <int D, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const RopeArgs a) {
  constexpr int L = D / 8;
  begin_launch(true);
  const int j = threadIdx.x % L;
  const int64_t t64 = static_cast<int64_t>(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
  if (t64 >= a.tokens) return;
  const int t = static_cast<int>(t64);
  const unsigned lane = threadIdx.x & 31u;
  const unsigned mask = ((1u << L) - 1u) << (lane & ~(L - 1u));
  const int h0 = blockIdx.y * a.chunk;
  const int h1 = min(h0 + a.chunk, a.H + 2 * a.Hkv);

  int b, n, pos;
  int64_t slot = -1;  // paged: element offset of the token's first head, or -1
  if constexpr (kPaged) {
    const int seq = token_sequence(a.cu, a.seqs, t);
    if (seq < 0) return;  // behind the last sequence
    int start, count;
    token_bounds(a.cu, seq, a.tokens, start, count);
    const int64_t limit = static_cast<int64_t>(a.max_pages) << a.page_shift;
    const int len = __ldg(a.kv_lens + seq);
    const int key = len - count + (t - start);
    b = 0;
    n = t;
    pos = key + (a.pos_offset != nullptr ? __ldg(a.pos_offset + seq) : 0);
    if (key >= 0) {
      const int page = key < limit ? resolve_page(a.block_table + static_cast<int64_t>(seq) * a.max_pages,
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
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  load_angle(a, pos, j, turned, j == 0, c, s);
  float wq[8], wk[8];
  const bool norm = a.wq != nullptr;
  if (norm) {
    load_weight(a.wq, lp.off0, lp.off1, wq);
    load_weight(a.wk, lp.off0, lp.off1, wk);
  }

  for (int h = h0; h < h1; h += kRows) {
    Row8 r[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int hh = h + i;
      if (hh >= h1) break;
      const RowView& v = hh < a.H ? a.q : (hh < a.H + a.Hkv ? a.k : a.v);
      const int hv = hh < a.H ? hh : (hh < a.H + a.Hkv ? hh - a.H : hh - a.H - a.Hkv);
      if (v.p != nullptr) r[i] = load_row<kInter>(row_of(v, b, n, hv), lp.off0, lp.off1);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int hh = h + i;
      if (hh >= h1) break;
      const bool is_q = hh < a.H, is_v = hh >= a.H + a.Hkv;
      if ((is_q && a.q.p == nullptr) || (is_v && a.v.p == nullptr)) continue;
      if (!is_v) {
        float x[8];
        unpack(r[i], x);
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
          const float rs = rsqrtf(group_sum<L>(ss, mask) * (1.f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * rs * (is_q ? wq[e] : wk[e]);
        }
        turn<kInter>(x, c, s, turned);
        r[i] = pack(x);
      }
      if (is_q) {
        store_row<kInter>(row_of(a.qo, b, n, hh), lp.off0, lp.off1, r[i]);
      } else {
        const int hk = is_v ? hh - a.H - a.Hkv : hh - a.H;
        if constexpr (kPaged) {
          if (slot >= 0)
            store_row<kInter>((is_v ? a.v_cache : a.k_cache) + slot +
                                  (static_cast<int64_t>(hk) << a.page_shift) * D,
                              lp.off0, lp.off1, r[i]);
        } else {
          store_row<kInter>(row_of(is_v ? a.vo : a.ko, b, n, hk), lp.off0, lp.off1, r[i]);
        }
      }
    }
  }
}

// Backward.  Work items are (token group, head chunk); with norms the grid is persistent and a
// thread sums the weight gradients of its elements over all its rows, so that a block leaves one
// partial [2][D] and the sum over blocks (rope_dw_kernel) has a fixed order.
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const RopeArgs a) {
  constexpr int L = D / 8, G = kThreads / L;
  constexpr int kR = 2;  // rows in flight: each brings a gradient and an input
  begin_launch(true);
  const int j = threadIdx.x % L, grp = threadIdx.x / L;
  const unsigned lane = threadIdx.x & 31u;
  const unsigned mask = ((1u << L) - 1u) << (lane & ~(L - 1u));
  const LanePairs<D, kInter> lp(j, a.rot);
  const bool turned = a.table != nullptr && lp.turned;
  const bool norm = a.wq != nullptr;
  float wq[8], wk[8], dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  if (norm) {
    load_weight(a.wq, lp.off0, lp.off1, wq);
    load_weight(a.wk, lp.off0, lp.off1, wk);
  }
  const int heads = a.H + 2 * a.Hkv;
  const int chunks = (heads + a.chunk - 1) / a.chunk;
  const int64_t items = (static_cast<int64_t>(a.tokens) + G - 1) / G * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t t64 = it / chunks * G + grp;
    if (t64 >= a.tokens) continue;  // whole lane groups; nothing below is block-wide
    const int t = static_cast<int>(t64);
    const int h0 = static_cast<int>(it % chunks) * a.chunk;
    const int h1 = min(h0 + a.chunk, heads);
    const int b = t / a.N, n = t - b * a.N;
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    load_angle(a, a.positions != nullptr ? __ldg(a.positions + t) : n, j, turned, j == 0, c, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = -s[e];  // the transpose of the rotation
    for (int h = h0; h < h1; h += kR) {
      Row8 r[kR], xr[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const int hh = h + i;
        if (hh >= h1) break;
        const bool is_q = hh < a.H, is_v = hh >= a.H + a.Hkv;
        const int hv = is_q ? hh : (is_v ? hh - a.H - a.Hkv : hh - a.H);
        const RowView& v = is_q ? a.q : (is_v ? a.v : a.k);
        if (v.p != nullptr) r[i] = load_row<kInter>(row_of(v, b, n, hv), lp.off0, lp.off1);
        if (norm && !is_v)
          xr[i] = load_row<kInter>(row_of(is_q ? a.qx : a.kx, b, n, hv), lp.off0, lp.off1);
      }
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const int hh = h + i;
        if (hh >= h1) break;
        const bool is_q = hh < a.H, is_v = hh >= a.H + a.Hkv;
        const int hv = is_q ? hh : (is_v ? hh - a.H - a.Hkv : hh - a.H);
        if (is_v && a.v.p == nullptr) continue;
        if (!is_v) {
          float g[8];
          unpack(r[i], g);
          turn<kInter>(g, c, s, turned);
          if (norm) {
            float x[8];
            unpack(xr[i], x);
            float ss = 0.f, ux = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              ss = fmaf(x[e], x[e], ss);
              ux = fmaf(g[e] * (is_q ? wq[e] : wk[e]), x[e], ux);
            }
            ss = group_sum<L>(ss, mask);
            ux = group_sum<L>(ux, mask);
            const float rs = rsqrtf(ss * (1.f / D) + a.eps);
            const float m = ux * rs * (1.f / D);  // mean(u x r)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float xh = x[e] * rs;
              if (is_q) dwq[e] = fmaf(g[e], xh, dwq[e]);
              else dwk[e] = fmaf(g[e], xh, dwk[e]);
              g[e] = rs * (g[e] * (is_q ? wq[e] : wk[e]) - xh * m);
            }
          }
          r[i] = pack(g);
        }
        store_row<kInter>(row_of(is_q ? a.qo : (is_v ? a.vo : a.ko), b, n, hv), lp.off0, lp.off1,
                          r[i]);
      }
    }
  }
  if (!norm) return;
  __shared__ float part[G][2][D];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int at = e < 4 ? lp.off0 + e : lp.off1 + e - 4;
    part[grp][0][at] = dwq[e];
    part[grp][1][at] = dwk[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) sum += part[g][i / D][i % D];
    a.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = sum;
  }
}

// dw[q or k][e] = sum over blocks: 32 columns a block, 32 row lanes, joined in a fixed order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* partial, int blocks, int D,
                                                       float* dwq, float* dwk) {
  __shared__ float sm[32][33];
  begin_launch(true);
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + x;
  float sum = 0.f;
  for (int r = y; r < blocks; r += 32) sum += partial[static_cast<int64_t>(r) * 2 * D + col];
  sm[y][x] = sum;
  __syncthreads();
  if (y == 0) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) s += sm[r][x];
    (col < D ? dwq[col] : dwk[col - D]) = s;
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

// Heads of one work item.  A lane group that walks over many heads loads its token's angles and
// weights once; few tokens need more groups to cover memory latency.
int head_chunk(int64_t tokens, int heads, int groups_per_block) {
  // about 152 SMs x 8 blocks of lane groups before a group takes more than kRows heads
  const int64_t want = 152ll * 8 * groups_per_block;
  int chunk = kRows;
  while (chunk < 16 && chunk < heads && tokens * ((heads + 2 * chunk - 1) / (2 * chunk)) >= want)
    chunk *= 2;
  return chunk;
}

template <int D, bool kInter, bool kPaged>
cudaError_t fwd_t(RopeArgs a, cudaStream_t s) {
  constexpr int G = kThreads / (D / 8);
  const int heads = a.H + 2 * a.Hkv;
  a.chunk = head_chunk(a.tokens, heads, G);
  const dim3 grid((a.tokens + G - 1) / G, (heads + a.chunk - 1) / a.chunk);
  return launch_chained(rope_fwd_kernel<D, kInter, kPaged>, grid, kThreads, 0, s, a);
}

template <int D, bool kInter>
cudaError_t bwd_t(RopeArgs a, float* dwq, float* dwk, cudaStream_t s) {
  constexpr int G = kThreads / (D / 8);
  const int heads = a.H + 2 * a.Hkv;
  a.chunk = head_chunk(a.tokens, heads, G);
  const int64_t items = (static_cast<int64_t>(a.tokens) + G - 1) / G * ((heads + a.chunk - 1) / a.chunk);
  const int blocks = static_cast<int>(items < kRopeBwdBlocks ? items : kRopeBwdBlocks);
  if (blocks > 0) {
    const cudaError_t e = launch_chained(rope_bwd_kernel<D, kInter>, blocks, kThreads, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  if (a.wq == nullptr) return cudaSuccess;
  return launch_chained(rope_dw_kernel, 2 * D / 32, 1024, 0, s, static_cast<const float*>(a.partial),
                        blocks, D, dwq, dwk);
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
