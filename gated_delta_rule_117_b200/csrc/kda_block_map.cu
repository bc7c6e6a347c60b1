// Block tables and token slots from request lengths (include/kda.h,
// kda_block_map): sequence offsets, the blocks that the new tokens need, and
// the pool slot of every new token.
//
// The work is prefix sums over the requests (tokens, and new blocks) and one
// lookup a token, so a launch's latency and the 8 bytes a token bound it.
// One launch does all: every block forms the prefix sums itself (R lengths and
// contexts from L2, three integers a request in shared memory) instead of
// waiting for another block, takes its own tile of rows, and finds a row's
// request by bisection in shared memory.  A token in a new block takes the
// block from free_pages, not from the table, so no block waits for the
// table's update, which is spread over all threads block by block.
#include "kda_serve.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerBlock = 1024;
constexpr int kMaxR = 16384;

// Blocks of `tokens` tokens (a context and new tokens: below 2^32, so 32-bit divisions do).
__device__ __forceinline__ uint32_t blocks_of(uint32_t tokens, uint32_t page) {
  return tokens ? (tokens - 1) / page + 1 : 0;
}

__device__ __forceinline__ int saturate(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int)v; }

__global__ void __launch_bounds__(kThreads) block_map_kernel(MapArgs a) {
  // [R + 1] offsets of rows, of new blocks, and of new blocks that the table has room for
  extern __shared__ int sh[];
  int *s_cu = sh, *s_new = s_cu + a.R + 1, *s_put = s_new + a.R + 1;
  __shared__ int64_t w_tok[kThreads / 32], w_blk[kThreads / 32], w_put[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // exclusive prefix sums, kThreads requests at a time (64 bits: garbage lengths must not wrap)
  int64_t tok0 = 0, blk0 = 0, put0 = 0;
  for (int r0 = 0; r0 < a.R; r0 += kThreads) {
    const int r = r0 + tid;
    int64_t n = 0, b = 0, p = 0;
    if (r < a.R) {
      const uint32_t len = max(a.len[r], 0), c = a.ctx ? max(a.ctx[r], 0) : 0;
      n = len;
      const int64_t old = blocks_of(c, a.page);
      b = blocks_of(c + len, a.page) - old;
      p = max(min(b, a.table_stride - old), (int64_t)0);
    }
    int64_t in = n, ib = b, ip = p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, in, o), y = __shfl_up_sync(~0u, ib, o), z = __shfl_up_sync(~0u, ip, o);
      if (lane >= o) { in += x; ib += y; ip += z; }
    }
    if (lane == 31) { w_tok[warp] = in; w_blk[warp] = ib; w_put[warp] = ip; }
    __syncthreads();
    int64_t bt = tok0, bb = blk0, bp = put0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) { bt += w_tok[w]; bb += w_blk[w]; bp += w_put[w]; }
      tok0 += w_tok[w];
      blk0 += w_blk[w];
      put0 += w_put[w];
    }
    if (r < a.R) {
      s_cu[r] = saturate(bt + in - n);
      s_new[r] = saturate(bb + ib - b);
      s_put[r] = saturate(bp + ip - p);
    }
    __syncthreads();
  }
  if (tid == 0) {
    s_cu[a.R] = saturate(tok0);
    s_new[a.R] = saturate(blk0);
    s_put[a.R] = saturate(put0);
  }
  __syncthreads();

  if (blockIdx.x == 0) {
    for (int r = tid; r <= a.R; r += kThreads) a.cu[r] = s_cu[r];
    if (tid == 0) a.used[0] = s_new[a.R];
  }
  // the request that owns entry v of a prefix sum: sum[lo] <= v < sum[lo + 1]
  auto owner = [&](const int *sum, int v) {
    int lo = 0, hi = a.R;
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (sum[m] <= v) lo = m; else hi = m;
    }
    return lo;
  };
  // new table entries, one a thread, whoever's they are (256 single tokens with 90 new
  // blocks: 7.9 us with a warp a request, 4.2 us so); there are no more than the table holds
  for (int64_t e = (int64_t)blockIdx.x * kThreads + tid; e < s_put[a.R]; e += (int64_t)gridDim.x * kThreads) {
    const int r = owner(s_put, (int)e), k = (int)e - s_put[r];
    const int64_t f = (int64_t)s_new[r] + k, j = (int64_t)blocks_of(a.ctx ? max(a.ctx[r], 0) : 0, a.page) + k;
    a.table[(int64_t)r * a.table_stride + j] = f < a.n_free ? a.free_pages[f] : -1;
  }
  const int row0 = blockIdx.x * kRowsPerBlock;
  for (int i = tid; i < kRowsPerBlock; i += kThreads) {
    const int row = row0 + i;
    if (row >= a.rows) break;
    int64_t slot = -1;
    if (row < s_cu[a.R]) {
      const int lo = owner(s_cu, row);
      const uint32_t c = a.ctx ? max(a.ctx[lo], 0) : 0, page_size = a.page;
      const uint32_t pos = c + (uint32_t)(row - s_cu[lo]);
      const uint32_t j = pos / page_size, old = blocks_of(c, page_size);
      if (j < (uint32_t)a.table_stride) {
        int64_t page = -1;
        if (j < old) {
          page = a.table[(int64_t)lo * a.table_stride + j];
        } else {
          const int64_t f = (int64_t)s_new[lo] + (j - old);
          if (f < a.n_free) page = a.free_pages[f];
        }
        if (page >= 0) slot = page * a.page + (pos - j * page_size);
      }
    }
    a.token_slots[row] = slot;
  }
}

}  // namespace

cudaError_t launch_block_map(const MapArgs &a, cudaStream_t st) {
  // The attribute is the kernel's, not the call's: always the most that a call may need, so that
  // calls of several host threads agree on it.
  constexpr int kMaxSmem = 3 * sizeof(int) * (kMaxR + 1);
  static_assert(kMaxSmem <= 200 * 1024, "prefix sums in shared memory");
  const size_t smem = 3 * sizeof(int) * ((size_t)a.R + 1);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(block_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  const int grid = max(1, (int)(((int64_t)a.rows + kRowsPerBlock - 1) / kRowsPerBlock));
  block_map_kernel<<<grid, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
