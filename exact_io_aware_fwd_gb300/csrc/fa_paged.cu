// Attention of a few query rows over a paged key/value cache, and the join of partial results.
//
// O = softmax(scale q K^T) V for the queries of one sequence that share a key/value head (group
// members x new tokens), 16 rows at a time: each K, V element is used by at most 16 rows, so the
// kernel is bound by reading the cache once.  A warp takes 16 keys of every 64-key tile and is a
// pipeline of its own: it copies its keys' rows with cp.async into a private ring of
// shared-memory stages (keys past the length become zeros, whatever the page holds there), and
// computes S (m16n8k16), the online softmax and O += P V from the ring, with no barrier between
// warps until a segment's end, where the four partial (m, l, O) are merged through shared memory.
// mma.sync is enough here: 16 rows x 4 flops per element and 2 bytes is 32 flops a byte, a few
// percent of the tensor pipe at full memory bandwidth.
#include "fa_internal.h"
#include "fa_paged.h"
#include "paged_plan.cuh"
#include "sm103.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int R = kPagedRows;
constexpr int kKeys = 16;             // keys of a warp's step
constexpr int KT = kKeys * kWarps;    // keys of a tile
constexpr int kDirectTiles = kPagedUnsplitKeys / KT;  // one CTA for a whole segment
constexpr float kLn2 = 0.693147180559945309f;

template <int D>
struct PagedLayout {
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr uint32_t kHalf = kKeys * D * 2u;                // K or V of a step
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kRing = kWarps * kStages * kStage;
  static constexpr int kPad = D + 4;                               // floats per merged row
  static constexpr uint32_t kMerge = kWarps * R * (kPad + 2) * 4u;
  static constexpr uint32_t kBytes = kRing > kMerge ? kRing : kMerge;
  static constexpr int kCtasPerSm = D == 128 ? 2 : 3;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0: the 16 bytes become zeros, src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte granule g of key row r in a step's K or V: granules are permuted within
// each 128 bytes by the row, so the eight rows of an ldmatrix fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t step_offset(uint32_t r, uint32_t g) {
  return r * (D * 2u) + ((g ^ (r & 7u)) << 4);  // the xor stays within the granule's 128 bytes
}

template <int D>
__global__ void __launch_bounds__(kThreads, PagedLayout<D>::kCtasPerSm)
    paged_kernel(const PagedArgs a) {
  using L = PagedLayout<D>;
  constexpr int S = L::kStages, GR = D / 8;  // granules of a row
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Share sh = make_share<R, KT, kThreads, kDirectTiles>(a);
  if (sh.u0 >= sh.u1) return;
  const KeyList& l = a.list;
  const uint32_t ring = smem_u32(smem) + warp * (S * L::kStage);

  Walk<R, KT> walk(sh, a);
  Piece piece;
  while (walk.next(a, piece)) {
    const Entry& e = walk.e;
    const int b = walk.b, hk = piece.hk, rtile = piece.r;
    const int tile_a = piece.ta, tile_e = piece.te;
    const bool whole = piece.whole;

    // ---- the rows' queries as A fragments: thread holds rows lane / 4 and lane / 4 + 8
    const int rows = min(R, e.nc * a.G - rtile * R);
    uint32_t qf[D / 16][4];
    int lim[2];  // keys below it are visible to the row
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = (lane >> 2) + 8 * i;
      const int row = rtile * R + rr;
      const int tok = row / a.G;
      lim[i] = rr < rows ? row_limit(e, l.causal, a.G, row) : e.len;
      const __nv_bfloat16* qp =
          a.q + (static_cast<int64_t>(e.start + tok) * a.H + hk * a.G + (row - tok * a.G)) * D +
          (lane & 3) * 2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][i] = rr < rows ? *reinterpret_cast<const uint32_t*>(qp + k * 16) : 0u;
        qf[k][i + 2] = rr < rows ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + 8) : 0u;
      }
    }
    // smallest limit of the tile: its first token's
    const int lim_min = row_limit(e, l.causal, a.G, rtile * R);

    // ---- this warp's steps: keys [(t * kWarps + warp) * kKeys, + kKeys) of tiles t
    const int32_t* trow = l.table + static_cast<int64_t>(b) * l.max_pages;
    const int first = tile_a * kWarps + warp;  // 16-key block of step 0
    const int blocks = (e.len + kKeys - 1) / kKeys;
    int steps = tile_e - tile_a;
    while (steps > 0 && first + (steps - 1) * kWarps >= blocks) --steps;
    int pages = -1;          // lane i: page of step (issue & ~31) + i
    uint32_t missing = 0;    // bit s: the page of stage s is out of range
    auto issue = [&](int st) {
      if (st < steps) {
        if ((st & 31) == 0) {
          const int blk = first + (st + lane) * kWarps;
          pages = st + lane < steps ? resolve_page(trow, l.max_pages, a.num_pages, a.page_shift,
                                                   blk * kKeys)
                                    : 0;
        }
        const int page = __shfl_sync(~0u, pages, st & 31);
        const int key0 = (first + st * kWarps) * kKeys;
        const int slot = st % S;
        missing = page < 0 ? missing | (1u << slot) : missing & ~(1u << slot);
        if (page < 0 && lane == 0) atomicCAS(a.status, 0, kErrIndex);
        const int64_t base =
            (((static_cast<int64_t>(max(page, 0)) * a.Hkv + hk) << a.page_shift) +
             (key0 & ((1 << a.page_shift) - 1))) * D;
        const uint32_t dst = ring + slot * L::kStage;
#pragma unroll
        for (int i = 0; i < kKeys * GR / 32; ++i) {
          const int r = (i * 32 + lane) / GR, g = (i * 32 + lane) % GR;
          const bool valid = page >= 0 && key0 + r < e.len;
          const int64_t off = valid ? base + r * D + g * 8 : 0;
          cp_async16(dst + step_offset<D>(r, g), a.k_cache + off, valid);
          cp_async16(dst + L::kHalf + step_offset<D>(r, g), a.v_cache + off, valid);
        }
      }
      cp_commit();
    };

    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    for (int st = 0; st < S - 1; ++st) issue(st);
    for (int st = 0; st < steps; ++st) {
      cp_wait<S - 2>();
      __syncwarp();
      const uint32_t kb = ring + (st % S) * L::kStage, vb = kb + L::kHalf;
      // S = Q K^T: 16 rows x 16 keys
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const uint32_t r = (lane & 7) + ((lane >> 4) << 3), gh = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t f[4];
          ldsm4(kb + step_offset<D>(r, 2 * k + gh), f);
          mma16816(s[0], qf[k], f[0], f[1]);
          mma16816(s[1], qf[k], f[2], f[3]);
        }
      }
      const int key0 = (first + st * kWarps) * kKeys;
      if (key0 + kKeys > lim_min || ((missing >> (st % S)) & 1u)) {
        const bool gone = (missing >> (st % S)) & 1u;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = key0 + n * 8 + (lane & 3) * 2 + (c & 1);
            if (gone || key >= lim[c >> 1]) s[n][c] = -INFINITY;
          }
      }
      // online softmax; the row maximum is shared by the four lanes of a row, the sum is joined
      // at the end
      bool moved = false;
      float alpha[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2)) * a.scale_log2;
        alpha[i] = 1.f;
        if (mx > m[i]) {
          alpha[i] = ex2(m[i] - mx);
          m[i] = mx;
          moved = true;
        }
        const float ref = m[i] == -INFINITY ? 0.f : m[i];
        float part = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // a masked score stays -inf whatever the scale (0 * inf would be NaN)
            const float x = s[n][2 * i + c];
            const float p = x == -INFINITY ? 0.f : ex2(fmaf(x, a.scale_log2, -ref));
            s[n][2 * i + c] = p;
            part += p;
          }
        sum[i] = sum[i] * alpha[i] + part;
      }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][0] *= alpha[0];
          o[n][1] *= alpha[0];
          o[n][2] *= alpha[1];
          o[n][3] *= alpha[1];
        }
      }
      // O += P V; P rounded to bf16 (relative 2^-9, as in fa_fwd), its sum is not
      const uint32_t pf[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]),
                              pack_bf16(s[1][0], s[1][1]), pack_bf16(s[1][2], s[1][3])};
      {
        const uint32_t r = lane & 15, gh = lane >> 4;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t f[4];
          ldsm4_t(vb + step_offset<D>(r, 2 * n + gh), f);
          mma16816(o[2 * n], pf, f[0], f[1]);
          mma16816(o[2 * n + 1], pf, f[2], f[3]);
        }
      }
      __syncwarp();  // every lane has read stage st % S before it is filled again
      issue(st + S - 1);
    }
    cp_wait<0>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] += __shfl_xor_sync(~0u, sum[i], 1);
      sum[i] += __shfl_xor_sync(~0u, sum[i], 2);
    }

    // ---- the four warps' parts meet in shared memory (over the ring)
    __syncthreads();
    float* mo = reinterpret_cast<float*>(smem);           // [warp][row][kPad]
    float* mm = mo + kWarps * R * L::kPad;                // [warp][row]
    float* ml = mm + kWarps * R;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = (lane >> 2) + 8 * i;
      float* dst = mo + (warp * R + rr) * L::kPad + (lane & 3) * 2;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
      if ((lane & 3) == 0) {
        mm[warp * R + rr] = m[i];
        ml[warp * R + rr] = sum[i];
      }
    }
    __syncthreads();
    const int tile = row_tile0(e.start, a.G, R, b) + rtile;
    if (tid == 0 && tile_a == 0)  // this CTA began the segment
      a.part.spans[static_cast<int64_t>(hk) * a.part.span_tiles + tile] = span_of(sh, piece);
    {
      const int rr = tid / 8, c8 = tid % 8;  // 8 threads a row
      float w[kWarps], mx = -INFINITY, lsum = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, mm[i * R + rr]);
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        w[i] = mx == -INFINITY ? 0.f : ex2(mm[i * R + rr] - mx);
        lsum = fmaf(w[i], ml[i * R + rr], lsum);
      }
      const int row = rtile * R + rr, tok = row / a.G;
      const int head = hk * a.G + (row - tok * a.G);
      const int64_t at = static_cast<int64_t>(e.start + tok) * a.H + head;
      const bool final_out = whole && a.rowbuf == nullptr;
      const float inv = lsum > 0.f ? 1.f / lsum : (lsum == 0.f ? 0.f : lsum);  // NaN stays NaN
      float* slot = whole ? a.rowbuf + at * D
                          : a.part.slots + (static_cast<int64_t>(blockIdx.x) * 2 + (tile_a == 0)) *
                                               (R * (D + 2)) + rr * D;
      if (rr < rows) {
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
          const int col = g * 32 + c8 * 4;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(mo + (i * R + rr) * L::kPad + col);
            acc.x = fmaf(w[i], v.x, acc.x);
            acc.y = fmaf(w[i], v.y, acc.y);
            acc.z = fmaf(w[i], v.z, acc.z);
            acc.w = fmaf(w[i], v.w, acc.w);
          }
          if (final_out)
            *reinterpret_cast<uint2*>(a.o + at * D + col) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
          else
            *reinterpret_cast<float4*>(slot + col) = acc;
        }
        if (c8 == 0) {
          if (final_out) {
            a.lse[static_cast<int64_t>(head) * a.total + e.start + tok] =
                lsum == 0.f ? -INFINITY : (mx + log2f(lsum)) * kLn2;
          } else if (whole) {
            float* st = a.rowbuf + static_cast<int64_t>(a.total) * a.H * D;
            st[at] = mx;
            st[static_cast<int64_t>(a.total) * a.H + at] = lsum;
          } else {
            float* st = a.part.slots + (static_cast<int64_t>(blockIdx.x) * 2 + (tile_a == 0)) *
                                           (R * (D + 2)) + R * D;
            st[rr] = mx;
            st[R + rr] = lsum;
          }
        }
      }
    }
    __syncthreads();  // the ring is free again
  }
}

// Joins the parts of each output row: O = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i, in the order
// of the keys.  One warp per (token, head); D / 32 elements a lane.
template <int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const JoinArgs a) {
  constexpr int E = D / 32;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= static_cast<int64_t>(a.total) * a.H) return;
  const int t = static_cast<int>(id / a.H), head = static_cast<int>(id % a.H);
  const int hk = head / a.G;
  const int seq = token_sequence(a.cu, a.B, t);
  if (seq < 0) return;
  float m = -INFINITY, lsum = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  auto add = [&](const float* po, float pm, float pl) {
    if (pm == -INFINITY && pl == 0.f) return;  // no visible key
    float v[E];
    if constexpr (E == 4) {
      const float4 x = *reinterpret_cast<const float4*>(po + lane * 4);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(po + lane * 2);
      v[0] = x.x; v[1] = x.y;
    }
    const float top = fmaxf(m, pm);
    const float wa = m == -INFINITY ? 0.f : ex2(m - top), wb = ex2(pm - top);
    lsum = lsum * wa + pl * wb;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * wa + v[i] * wb;
    m = top;
  };
  for (int li = 0; li < a.lists; ++li) {
    const KeyList& l = a.list[li];
    const PartialLayout& p = a.part[li];
    int b = seq, start, n;
    if (l.group_cu != nullptr) {
      b = token_sequence(l.group_cu, l.count, seq);
      if (b < 0) continue;  // a sequence of no group has no prefix
      const int s0 = min(max(__ldg(l.group_cu + b), 0), a.B);
      start = a.cu != nullptr ? min(max(__ldg(a.cu + s0), 0), a.total) : s0;
      n = 0x7fffffff;
    } else {
      token_bounds(a.cu, b, a.total, start, n);
      n = min(n, l.max_q);
    }
    if (t - start >= n) return;  // beyond max_q: not computed
    const int row = (t - start) * a.G + (head - hk * a.G);
    const int tile = row_tile0(start, a.G, p.R, b) + row / p.R, rr = row % p.R;
    if (tile < 0 || tile >= p.span_tiles) continue;
    const int2 span = p.spans[static_cast<int64_t>(hk) * p.span_tiles + tile];
    // a launch that gave up leaves no span: nothing out of range is read
    if (span.x < 0 || span.y < 1 || span.x + span.y > p.ctas) continue;
    if (span.y == 1) {
      if (a.rowbuf[li] == nullptr) return;  // already final
      const float* st = a.rowbuf[li] + static_cast<int64_t>(a.total) * a.H * D;
      add(a.rowbuf[li] + id * D, st[id], st[static_cast<int64_t>(a.total) * a.H + id]);
      continue;
    }
    for (int i = 0; i < span.y; ++i) {
      const float* slot = p.slots + (static_cast<int64_t>(span.x + i) * 2 + (i == 0)) *
                                        (p.R * (D + 2));
      add(slot + rr * D, slot[p.R * D + rr], slot[p.R * D + p.R + rr]);
    }
  }
  const float inv = lsum > 0.f ? 1.f / lsum : (lsum == 0.f ? 0.f : lsum);
  __nv_bfloat16* dst = a.o + id * D;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst + lane * 4) =
        make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst + lane * 2) = pack_bf16(o[0] * inv, o[1] * inv);
  if (lane == 0)
    a.lse[static_cast<int64_t>(head) * a.total + t] =
        lsum == 0.f ? -INFINITY : (m + log2f(lsum)) * kLn2;
}

template <int D>
cudaError_t launch_paged_d(const PagedArgs& a, int64_t max_units, cudaStream_t s) {
  using L = PagedLayout<D>;
  cudaError_t e = ensure_smem_limit<paged_kernel<D>>(L::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t most = 152 * L::kCtasPerSm;
  const int64_t ctas = max_units < most ? max_units : most;
  paged_kernel<D><<<static_cast<unsigned>(ctas), kThreads, L::kBytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged(int d, const PagedArgs& a, int64_t max_units, cudaStream_t s) {
  return d == 64 ? launch_paged_d<64>(a, max_units, s) : launch_paged_d<128>(a, max_units, s);
}

cudaError_t launch_paged_join(int d, const JoinArgs& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.total) * a.H;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (d == 64) paged_join_kernel<64><<<grid, 128, 0, s>>>(a);
  else paged_join_kernel<128><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
