// Segments of a packed scan: how one call's sequences are cut along time, the
// same for every scan kernel.
//
// Cuts lie at multiples of `seg` tokens on an axis that starts at the last
// multiple of `align` before a sequence's first token (counted with ctx), so
// chunks of `align` tokens inside a segment end where snapshots may be wanted.
// Work items are numbered without the lengths: sequence r's begin at
//     base(r) = floor(cu[r] / seg) + 2 r,
// which leaves room for its ceil((ctx % align + len) / seg) segments, as that is
// at most 1 + ceil(len / seg) <= floor(cu[r + 1] / seg) - floor(cu[r] / seg) + 2
// while align <= seg.  Items between a sequence's last segment and the next
// base have no work.
#pragma once
#include "kda_serve.cuh"

namespace kda {

constexpr int kAlign = 128;     // `align` of the tensor-core kernel: its chunks
constexpr int kSimtAlign = 16;  // of the CUDA-core kernel: the tokens that it stages at a time

// Items of a call (seg 0: one for each sequence).
inline int64_t scan_items(int R, int rows, int seg) { return seg == 0 ? R : (int64_t)rows / seg + 2 * (int64_t)R; }

__device__ __forceinline__ int seg_base(const Requests &q, int r, int seg) {
  if (seg == 0) return r;
  const int start = q.cu ? q.cu[r] : r * q.T;
  return start / seg + 2 * r;
}

struct Item {
  Seq s;
  int r;
  int index, count;    // segment of the sequence, and how many it has
  int begin, end;      // its tokens, counted from the sequence's first one
  int64_t item;        // its number (workspace entry)
};

// Requests of a packed call up to which whole sequences run longest first.  Every block
// finds its sequence for itself: 0.9 us of each at R = 40, 3 us at R = 256, while one late long
// sequence costs a call of many blocks less and less.
constexpr int kMaxRanked = 64;

// Sequence of rank `item` by length, longest first (ties: lower index first), so that the
// longest do not begin when the machine is already running dry: 9 sequences of 362 to
// 7,305 tokens, 32 heads: 254 us in the order of the call, 185 us longest first.
// `scratch`: kMaxRanked + 1 ints of shared memory.  Every thread of the block calls it.
__device__ __forceinline__ int sequence_of_rank(const Requests &q, int item, int *scratch) {
  for (int r = threadIdx.x; r < q.R; r += blockDim.x) scratch[r] = q.cu[r + 1] - q.cu[r];
  __syncthreads();
  for (int r = threadIdx.x; r < q.R; r += blockDim.x) {
    const int len = scratch[r];
    int rank = 0;
    for (int k = 0; k < q.R; ++k) rank += scratch[k] > len || (scratch[k] == len && k < r);
    if (rank == item) scratch[kMaxRanked] = r;
  }
  __syncthreads();
  const int r = scratch[kMaxRanked];
  __syncthreads();  // (the caller may use the scratch for something else)
  return r;
}

// The block's work item; false: none.  Every thread of the block must call it;
// `scratch` as above.
__device__ __forceinline__ bool item_of(const Requests &q, int item, int seg, int align, bool tell, int *scratch, Item &it) {
  if (tell && item == 0) tell_offsets(q);
  if (seg == 0) {
    it.r = q.cu && q.R > 1 && q.R <= kMaxRanked ? sequence_of_rank(q, item, scratch) : item;
  } else {
    it.r = block_count_le(q.R, [&](int i) { return seg_base(q, i, seg); }, item) - 1;
    if (it.r < 0) return false;
  }
  it.s = seq_of(q, it.r, tell);
  it.item = item;
  const int len = it.s.end - it.s.start;
  if (!it.s.ok || len == 0) return false;
  const int off = it.s.ctx % align;
  it.index = seg == 0 ? 0 : item - seg_base(q, it.r, seg);
  it.count = seg == 0 ? 1 : (int)(((int64_t)off + len + seg - 1) / seg);
  if (it.index < 0 || it.index >= it.count) return false;
  it.begin = it.index == 0 ? 0 : it.index * seg - off;
  it.end = it.index == it.count - 1 ? len : (it.index + 1) * seg - off;
  return true;
}

// Workspace of a segmented call: [items][H][N * P] states, then [items][H] decays.
// The state pass leaves there what each segment adds to a zero state and how it
// decays one; launch_segment_states turns the states into the entering ones.
inline float *seg_states(const SsmArgs &a) { return (float *)a.workspace; }
inline float *seg_decays(const SsmArgs &a, int64_t items) { return seg_states(a) + items * a.H * a.N * a.P; }
inline size_t seg_workspace(int64_t items, int H, int N, int P) {
  return (size_t)((items * H * ((int64_t)N * P + 1) * 4 + 15) & ~(int64_t)15);
}
cudaError_t launch_segment_states(const SsmArgs &a, int seg, int align, cudaStream_t st);

// Tokens up to which the tensor-core kernel runs an item token by token.
constexpr int kShort = 16;

// The tensor-core scan (bf16, 16-byte aligned rows), and whether a call's arrays fit it.
bool ssm_tc_fits(const SsmArgs &a);
cudaError_t launch_ssm_tc(const SsmArgs &a, int seg, cudaStream_t st);

// Time step d and the pool entry of a snapshot, shared by the scan kernels.
template <typename T>
__device__ __forceinline__ float time_step(const SsmArgs &a, int64_t row, int h) {
  float d = as_float(((const T *)a.dt)[row * a.dt_stride + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f);
  return a.softplus ? softplus(d) : d;
}

// Snapshot of sequence r after `pos` tokens (counted with ctx, so below 2^32): its place, or null.
__device__ __forceinline__ float *snapshot(const SsmArgs &a, int r, int h, uint32_t pos, bool tell) {
  if (a.page == 0 || pos % (uint32_t)a.page != 0) return nullptr;
  const uint32_t j = pos / (uint32_t)a.page - 1;  // (pos 0 gives a block behind every table)
  if (j >= (uint32_t)a.table_stride) return nullptr;
  const int p = a.table[(int64_t)r * a.table_stride + j];
  if (p < 0) return nullptr;
  if (p >= a.n_pages) {
    if (tell) record_bounds(a.q.status);
    return nullptr;
  }
  return a.pages + ((int64_t)p * a.H + h) * ((int64_t)a.N * a.P);
}

}  // namespace kda
