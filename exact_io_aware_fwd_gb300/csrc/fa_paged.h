// Internal interface of the operators around attention: the norm + rotation pass, the paged
// cache and the attention that reads it.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace fa {

enum : int { kErrIndex = 6 };  // FA_ERR_INDEX in the status word

// Launches that may be scheduled while the kernel ahead of them on the stream still runs, so that
// their launch and their CTAs' start overlap its end.  Nothing is read or written before it has
// completed (begin_launch; the join looks up where its rows' parts are before it waits, from inputs
// that were complete before the kernel ahead of it began).
template <typename K, typename... Args>
cudaError_t launch_chained(K kernel, dim3 grid, unsigned threads, uint32_t smem, cudaStream_t s,
                           const Args&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}
#ifdef __CUDACC__
// The next kernel on the stream may be scheduled.
__device__ __forceinline__ void let_next_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// The kernel ahead on the stream has completed and its writes are visible.
__device__ __forceinline__ void wait_for_last_launch() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void begin_launch() {
  wait_for_last_launch();
  let_next_launch();
}
#endif

// Page that holds key `key` of a sequence whose block-table row is `row` (max_pages entries), or
// -1 when the entry or the page lies outside its range.
__host__ __device__ inline int resolve_page(const int32_t* row, int max_pages, int num_pages,
                                            int page_shift, int key) {
  const int i = key >> page_shift;
  if (key < 0 || i >= max_pages) return -1;
  const int p = row[i];
  return (p < 0 || p >= num_pages) ? -1 : p;
}

// Tokens [s0, s1) of `total`, clamped.
__host__ __device__ inline void clamp_tokens(int s0, int s1, int total, int& start, int& n) {
  s0 = s0 < 0 ? 0 : (s0 > total ? total : s0);
  s1 = s1 < s0 ? s0 : (s1 > total ? total : s1);
  start = s0;
  n = s1 - s0;
}
// Bounds of new tokens [cu[b], cu[b + 1]) in packed tensors of `total` tokens, clamped like
// seq_bounds (cu == nullptr: one token per sequence).
__host__ __device__ inline void token_bounds(const int32_t* cu, int b, int total, int& start,
                                             int& n) {
  clamp_tokens(cu != nullptr ? cu[b] : b, cu != nullptr ? cu[b + 1] : b + 1, total, start, n);
}
// Search for the last of the n offsets cu[lo], ..., that is <= t, by `lanes` lanes: lane i looks at
// cu[lo + i * step()] (none past the n), offsets ascend, so the lanes that find one <= t are the
// first `hits` ones.
struct OffsetSearch {
  int lo, n;
  __host__ __device__ int step(int lanes) const { return (n + lanes - 1) / lanes; }
  __host__ __device__ void narrow(int step, int hits) {
    const int skip = (hits - 1) * step, left = n - skip;
    n = step < left ? step : left;
    lo += skip;
  }
};

// Sequence whose tokens include t: the last b with cu[b] <= t (empty sequences skipped), or -1
// when t lies behind cu[B] or before cu[0] (cu == nullptr: one token per sequence).
#ifdef __CUDACC__
// By a group of kLanes lanes (`mask`: its lanes of the warp).
template <int kLanes>
__device__ __forceinline__ int token_sequence_group(const int32_t* cu, int B, int t, int sub,
                                                    unsigned mask) {
  if (cu == nullptr) return t < B ? t : -1;
  OffsetSearch s{0, B + 1};
  while (true) {
    const int step = s.step(kLanes);
    const bool le = sub * step < s.n && __ldg(cu + s.lo + sub * step) <= t;
    const int hits = __popc(__ballot_sync(mask, le) & mask);
    if (hits == 0) return -1;  // before cu[0]
    s.narrow(step, hits);
    if (step == 1) break;
  }
  return s.lo < B ? s.lo : -1;  // behind cu[B]
}
#endif
// The same search on the host, lane by lane (checked against every answer in the tests).
template <int kLanes = 8>
inline int token_sequence(const int32_t* cu, int B, int t) {
  if (cu == nullptr) return t < B ? t : -1;
  OffsetSearch s{0, B + 1};
  while (true) {
    const int step = s.step(kLanes);
    int hits = 0;
    for (int sub = 0; sub < kLanes; ++sub) hits += sub * step < s.n && cu[s.lo + sub * step] <= t;
    if (hits == 0) return -1;
    s.narrow(step, hits);
    if (step == 1) break;
  }
  return s.lo < B ? s.lo : -1;
}

// ---- norm + rotation pass (fa_rope.cu)
struct RowView {
  __nv_bfloat16* p;
  int64_t batch, token, head;
};

struct RopeArgs {
  RowView q, k, v;     // inputs (backward: gradients of the outputs); q.p / v.p may be null
  RowView qo, ko, vo;  // outputs (backward: gradients of the inputs); paged: qo alone
  RowView qx, kx;      // backward with norms: the forward's inputs
  int B, N, H, Hkv;
  int tokens;          // B * N
  int chunk;           // heads of one work item
  const int32_t* positions;
  const float* table;
  int n_pos, rot;
  const float *wq, *wk;
  float eps;
  float* partial;      // backward with norms: [blocks][d] weight-gradient partials
  int first_k, first_v;  // backward: first blocks of K's and V's rows
  // paged destination of K and V
  __nv_bfloat16 *k_cache, *v_cache;
  const int32_t *block_table, *kv_lens, *cu, *pos_offset;
  int max_pages, num_pages, page_shift, seqs;
  int* status;
};

constexpr int kRopeBwdBlocks = 152 * 5;  // blocks of the backward (at most two more: one a kind)

cudaError_t launch_rope_table(const double* inv_freq, int rot, int n_pos, float amplitude,
                              float* table, cudaStream_t s);
cudaError_t launch_rope_fwd(int d, bool interleaved, bool paged, const RopeArgs& a,
                            cudaStream_t s);
cudaError_t launch_rope_bwd(int d, bool interleaved, const RopeArgs& a, float* dwq, float* dwk,
                            cudaStream_t s);

// ---- attention over the paged cache (fa_paged.cu)
//
// A list of key ranges: the sequences of a batch with their own pages, or the groups of a batch
// with the pages of their shared prefix (group_cu set).  Entry b has packed query tokens [start,
// start + n) and len keys.
struct KeyList {
  int count;                // entries
  const int32_t* lens;      // [count]
  const int32_t* table;     // [count][max_pages]
  int max_pages, max_len, max_q;
  const int32_t* group_cu;  // groups: [count + 1] over sequences, or nullptr
  int causal;
  int mma;                  // row tiles and key tiles of the tensor-core kernel
  int unsplit;              // no segment is split where none has more key tiles
};

// Partial results of one list.  Its rows (query token x head of the key/value head's group) are
// cut into tiles of R rows; tile r of entry b has index row_tile0(b) + r in [0, row_tiles()).
// spans[hk][tile] = (first worker, number of workers) that had the tile's keys.  One: it wrote
// the result (a joined list: into the row buffer).  Several: worker i left its part in slot
// 2 i + (1 when it began the tile's keys), and the join kernel adds them up in key order.
struct PartialLayout {
  int R;
  int2* spans;
  int span_tiles;  // tiles per key/value head
  float* slots;    // [workers][2][R * (D + 2)]: unnormalised O, then m (log2 units), then l
  int workers;
};
__host__ __device__ inline int row_tiles_bound(int total, int G, int R, int count) {
  return (total * G + R - 1) / R + count;
}
__host__ __device__ inline int row_tile0(int start, int G, int R, int b) {
  return (start * G + R - 1) / R + b;  // never overlaps entry b - 1's tiles
}

// Whether a span read from the workspace names workers whose slots exist.  A launch that gave up
// leaves spans of its rows unwritten, and the workspace may hold anything: nothing is added that
// could leave 32 bits.
__host__ __device__ inline bool span_ok(int first, int count, int workers) {
  return first >= 0 && first < workers && count >= 1 && count <= workers - first;
}

// One launch works on one list, or on both lists of a call with shared prefixes (list 0: the
// sequences, list 1: the groups) at once, each on its own part of the SMs.
struct PagedArgs {
  const __nv_bfloat16 *q, *k_cache, *v_cache;
  __nv_bfloat16* o;
  float* lse;
  const int32_t* cu;
  int B, total, H, Hkv, G;
  int num_pages, page_shift;
  float scale_log2;
  KeyList list[2];
  PartialLayout part[2];
  float mma_cost;    // a key tile of the tensor-core kernel in key tiles of the other one
  float* rowbuf[2];  // joined lists: [total * H] rows of O, then m, then l; else nullptr
  int* status;
};

struct JoinArgs {
  __nv_bfloat16* o;
  float* lse;
  const int32_t* cu;
  int B, total, H, Hkv, G;
  KeyList list[2];
  PartialLayout part[2];
  const float* rowbuf[2];
  int lists;
};

constexpr int kPagedRows = 16;           // rows of a tile
constexpr int kPagedCtas = 152;          // CTAs of a launch: one per SM
constexpr int kPagedWarps = 8;           // warps of a CTA, each a worker
constexpr int kPagedKeys = 16;           // keys of a tile
constexpr int kPagedMmaRows = 256;       // the tensor-core kernel, whose CTAs are the workers
constexpr int kPagedMmaKeys = 128;

cudaError_t launch_paged(int d, const PagedArgs& a, int lists, int64_t max_units, cudaStream_t s);
// Few segments: list 0, with its prefixes (lists == 2: segments are then not split).  max_units: as
// many CTAs as have work.
cudaError_t launch_paged_cta(int d, const PagedArgs& a, int lists, int64_t max_units,
                             cudaStream_t s);
// twin: one list, and no entry has more than 128 rows
cudaError_t launch_paged_mma(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedArgs& a, int lists, bool twin, int64_t max_units,
                             uint64_t timeout_ns, cudaStream_t s);
// split: groups of 8 lanes that share a row (1, 4 or 16)
cudaError_t launch_paged_join(int d, const JoinArgs& a, int split, cudaStream_t s);

}  // namespace fa
