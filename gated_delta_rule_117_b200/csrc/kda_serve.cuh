// Launch interface and device helpers of the packed-request operators (block
// map, short convolution, selective scan).  Not installed; the public
// interface is include/kda.h.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_internal.cuh"

namespace kda {

// The requests of a call: see "Packed requests" in include/kda.h.
struct Requests {
  const int *cu, *ctx, *slots;
  int R, rows, T, n_slots;  // T: tokens of a sequence without cu; n_slots 0: no pool
  unsigned *status;
};

struct MapArgs {
  const int *len, *ctx, *free_pages;
  int n_free;
  int *table;
  int table_stride, page;
  int *cu;
  int64_t *token_slots;
  int *used;
  int R, rows;
};

struct ConvArgs {
  Requests q;
  const void *x, *w, *bias;
  void *state, *y;
  int64_t x_stride, y_stride;
  int C, K, d;  // d: head dimension (norm, head-major output), else 0
  int log2_d, heads;
  int bf16, silu, norm, head_major;
  int vec;  // four channels can be moved at once everywhere
  float eps;
};

struct SsmArgs {
  Requests q;
  const void *x, *dt, *B, *C;
  const float *A, *D, *dt_bias;
  float *state;
  void *y;
  int64_t x_stride, dt_stride, b_stride, c_stride, y_stride;
  int H, G, N, P, bf16, softplus;
  // snapshots
  const int *table;
  int table_stride;
  float *pages;
  int n_pages, page;
  void *workspace;
};

cudaError_t launch_block_map(const MapArgs &a, cudaStream_t s);
cudaError_t launch_short_conv(const ConvArgs &a, cudaStream_t s);
cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t s);
cudaError_t launch_ssm_step(const SsmArgs &a, cudaStream_t s);
// How a scan cuts its sequences: seg[tensor cores][packed] tokens (0: whole sequences).
struct ScanPlan {
  int seg[2][2];
  size_t workspace;
};
ScanPlan plan_ssm_scan(int R, int rows, int H, int N, int P, int bf16);
cudaError_t launch_ssm_scan(const SsmArgs &a, const ScanPlan &plan, cudaStream_t s);

// ---- device side ---------------------------------------------------------------

// One sequence of a call, with everything that may not be followed found out.
struct Seq {
  int start, end;  // rows
  int slot;        // pool entry, valid when the call has a pool and ok
  int ctx;         // tokens behind it, >= 0
  bool ok;         // to be computed
};

__device__ __forceinline__ void record_bounds(unsigned *status) { atomicCAS(status, kDevOk, kDevBounds); }

// Offsets that lead outside the rows, whether or not any block comes to the sequence (one thread
// of a call does this).
__device__ __forceinline__ void tell_offsets(const Requests &q) {
  if (q.cu && (q.cu[0] < 0 || q.cu[q.R] > q.rows)) record_bounds(q.status);
}

// Rows and slot of sequence r.  `tell`: record values that lead outside.
__device__ __forceinline__ Seq seq_of(const Requests &q, int r, bool tell) {
  Seq s;
  if (q.cu) {
    s.start = q.cu[r];
    s.end = q.cu[r + 1];
  } else {
    s.start = r * q.T;
    s.end = s.start + q.T;
  }
  s.slot = q.slots ? q.slots[r] : r;
  s.ctx = q.ctx ? max(q.ctx[r], 0) : 0;
  s.ok = true;
  if (s.start < 0 || s.end < s.start || s.end > q.rows || (q.n_slots > 0 && s.slot >= q.n_slots)) {
    s.ok = false;
    if (tell) record_bounds(q.status);
  }
  if (s.slot < 0) s.ok = false;
  return s;
}

// Number of entries i in [0, n) with key(i) <= v, key non-decreasing, found by the
// whole block (every thread gets it; holds barriers): each step samples one entry a
// thread and keeps the gap between two samples.
template <typename F>
__device__ __forceinline__ int block_count_le(int n, F key, int v) {
  int lo = 0, hi = n;  // the count lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo - 1) / (int)blockDim.x + 1;
    const int64_t i = lo + (int64_t)threadIdx.x * step;
    const int c = __syncthreads_count(i < hi && key((int)i) <= v);
    if (c == 0) return lo;
    hi = (int)min((int64_t)hi, lo + (int64_t)c * step);
    lo += (c - 1) * step + 1;
  }
  return lo;
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T as_type(float x);
template <>
__device__ __forceinline__ float as_type<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 as_type<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// log(1 + e^v) without overflow or cancellation.
__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

}  // namespace kda
