// Short causal convolution (include/kda.h, kda_short_conv and
// kda_short_conv_step; Kimi K3 report, section 2.1.1, Eq. 2 without the
// projections): K taps a channel, Swish, L2 norm of each head.
//
// Bytes bound both: an input element is read once and an output element
// written once for about 2 K + 8 operations.  A thread owns a vector of V
// channels (16 bytes) and walks down a tile of rows with the last K - 1 inputs
// in registers, so an input is loaded once a tile (plus K - 1 rows of halo).
// Tiles are cut over the packed rows, not over the sequences, so the grid
// needs no lengths on the host; a tile walks through the sequences that it
// meets.
//
// The pool is read where a sequence starts and written where it ends, which
// may be different tiles: the tile with the last row therefore also computes
// the first K - 1 outputs of a sequence that reads the pool, so one thread
// reads the old entry and writes the new one, in that order.
#include "kda_serve.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// V elements from p (16-byte aligned if VEC), zeros behind the first n.
template <typename T, bool VEC>
__device__ __forceinline__ void load_v(const T *p, int n, float (&v)[kVec<T>]) {
  if constexpr (VEC) {
    union { uint4 u; T t[kVec<T>]; } b;
    b.u = n > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) v[j] = as_float(b.t[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) v[j] = j < n ? as_float(p[j]) : 0.f;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_v(T *p, int n, const float (&v)[kVec<T>]) {
  if constexpr (VEC) {
    union { uint4 u; T t[kVec<T>]; } b;
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) b.t[j] = as_type<T>(v[j]);
    if (n > 0) *reinterpret_cast<uint4 *>(p) = b.u;
  } else {
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j)
      if (j < n) p[j] = as_type<T>(v[j]);
  }
}

// v Sigmoid(v).  The fast forms are off by a few 2^-22, far below a bf16 step.
__device__ __forceinline__ float swish(float v, __nv_bfloat16) { return __fdividef(v, 1.f + __expf(-v)); }
__device__ __forceinline__ float swish(float v, float) { return v / (1.f + expf(-v)); }

template <typename T, int K>
struct Taps {
  float w[K][kVec<T>], b[kVec<T>];
};

template <typename T, int K, bool VEC>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c0, int n, Taps<T, K> &t) {
  const T *w = (const T *)a.w + (int64_t)c0 * K;
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) t.w[i][j] = j < n ? as_float(w[j * K + i]) : 0.f;
#pragma unroll
  for (int j = 0; j < kVec<T>; ++j) t.b[j] = a.bias && j < n ? as_float(((const T *)a.bias)[c0 + j]) : 0.f;
}

// Output of one row from its K inputs, oldest first.  A head's channels lie in
// d / V neighbouring lanes, so its norm is a butterfly over them: every lane of
// the warp must come here.
template <typename T, int K>
__device__ __forceinline__ void conv_row(const ConvArgs &a, const Taps<T, K> &t, const float *const (&u)[K],
                                         float (&o)[kVec<T>]) {
  constexpr int V = kVec<T>;
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float v = t.b[j];
#pragma unroll
    for (int i = 0; i < K; ++i) v = fmaf(t.w[i][j], u[i][j], v);
    if (a.silu) v = swish(v, T());
    o[j] = v;
    ss = fmaf(v, v, ss);
  }
  if (a.norm) {
    for (int off = 1; off < a.d / V; off <<= 1) ss += __shfl_xor_sync(~0u, ss, off);
    const float f = 1.f / sqrtf(ss + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] *= f;
  }
}

template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(kThreads) short_conv_kernel(ConvArgs a, int tile) {
  constexpr int V = kVec<T>;
  constexpr int NB = 4;  // rows whose loads are in flight together
  const Requests &q = a.q;
  const int row0 = (int)((int64_t)blockIdx.x * tile);
  const int c0 = (blockIdx.y * kThreads + threadIdx.x) * V;
  const int n = min(V, a.C - c0);  // <= 0: nothing of this thread's exists
  const T *x = (const T *)a.x + c0;
  T *pool = a.state ? (T *)a.state + c0 : nullptr;
  const int64_t xs = a.x_stride;

  int total = q.rows, r;
  if (q.cu) {
    total = min(q.cu[q.R], q.rows);
    r = block_count_le(q.R, [&](int i) { return q.cu[i]; }, row0) - 1;
  } else {
    r = row0 / (q.rows / q.R);
  }
  const int rend = min((int64_t)row0 + tile, (int64_t)total);
  int row = row0;
  if (r < 0) {
    r = 0;
    row = q.cu[0];
  }
  if (row >= rend) return;
  Taps<T, K> taps;
  load_taps<T, K, VEC>(a, c0, n, taps);

  auto put = [&](int rr, const Seq &s, int at, const float (&o)[V]) {
    T *y = (T *)a.y;
    if (a.head_major) {
      const int len = s.end - s.start, h = c0 / a.d;
      y += (((int64_t)rr * (a.C / a.d) + h) * len + (at - s.start)) * a.d + c0 % a.d;
    } else {
      y += (int64_t)at * a.y_stride + c0;
    }
    store_v<T, VEC>(y, n, o);
  };

  while (row < rend) {
    while (r < q.R && q.cu && q.cu[r + 1] <= row) ++r;
    if (r >= q.R) break;
    const Seq s = seq_of(q, r, blockIdx.y == 0 && threadIdx.x == 0);
    const int stop = min(s.end, rend);
    if (!s.ok || row < s.start) {  // (row < start: offsets that decrease)
      row = max(stop, row + 1);
      ++r;
      continue;
    }
    const bool carry = pool && s.ctx > 0, here = s.end <= rend;
    T *entry = pool ? pool + (int64_t)s.slot * (K - 1) * a.C : nullptr;
    float h[K - 1][V];  // the K - 1 inputs before `row`, oldest first
    // (a sequence that reads the pool and ends in a later tile: that tile computes the outputs
    // that need it)
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int at = row - (K - 1) + i;
      if (at >= s.start) {
        load_v<T, VEC>(x + at * xs, n, h[i]);
      } else if (carry && here) {
        load_v<T, VEC>(entry + (int64_t)(at - s.start + K - 1) * a.C, n, h[i]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] = 0.f;
      }
    }
    if (carry && here && row > s.start) {  // its first rows, in earlier tiles
      for (int at = s.start; at < min(row, s.start + K - 1); ++at) {
        float u[K][V], o[V];
        const float *up[K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const int p = at - (K - 1) + i - s.start;
          load_v<T, VEC>(p >= 0 ? x + (s.start + p) * xs : entry + (int64_t)(p + K - 1) * a.C, n, u[i]);
          up[i] = u[i];
        }
        conv_row<T, K>(a, taps, up, o);
        put(r, s, at, o);
      }
    }
    const int first = carry && !here ? s.start + K - 1 : row;  // rows before it are another tile's
    while (row < stop) {
      float u[NB][V];
#pragma unroll
      for (int b = 0; b < NB; ++b) load_v<T, VEC>(x + (row + b) * xs, row + b < stop ? n : 0, u[b]);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (row + b < stop) {
          float o[V];
          const float *up[K];
#pragma unroll
          for (int i = 0; i < K; ++i) up[i] = b + i < K - 1 ? h[b + i < K - 1 ? b + i : 0] : u[b + i - (K - 1) >= 0 ? b + i - (K - 1) : 0];
          conv_row<T, K>(a, taps, up, o);
          if (row + b >= first) put(r, s, row + b, o);
        }
      }
      const int nb = min(NB, stop - row);
      if (nb == NB) {
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) h[i][j] = u[NB - (K - 1) + i][j];
      } else {
        for (int b = 0; b < nb; ++b) {
#pragma unroll
          for (int i = 0; i + 1 < K - 1; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) h[i][j] = h[i + 1][j];
#pragma unroll
          for (int j = 0; j < V; ++j) h[K - 2][j] = b == 0 ? u[0][j] : b == 1 ? u[1][j] : u[2][j];
        }
      }
      row += nb;
    }
    if (here && pool) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) store_v<T, VEC>(entry + (int64_t)i * a.C, n, h[i]);
    }
    ++r;
  }
}

template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(ConvArgs a) {
  constexpr int V = kVec<T>;
  const int r = blockIdx.x;
  const int c0 = (blockIdx.y * kThreads + threadIdx.x) * V;
  const int n = min(V, a.C - c0);
  const int slot = a.q.slots ? a.q.slots[r] : r;
  if (slot < 0) return;
  if (slot >= a.q.n_slots) {
    if (blockIdx.y == 0 && threadIdx.x == 0) record_bounds(a.q.status);
    return;
  }
  T *entry = (T *)a.state + (int64_t)slot * (K - 1) * a.C + c0;
  float u[K][V], o[V];
  const float *up[K];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) load_v<T, VEC>(entry + (int64_t)i * a.C, n, u[i]);
  load_v<T, VEC>((const T *)a.x + r * a.x_stride + c0, n, u[K - 1]);
  Taps<T, K> taps;
  load_taps<T, K, VEC>(a, c0, n, taps);
#pragma unroll
  for (int i = 0; i < K; ++i) up[i] = u[i];
  conv_row<T, K>(a, taps, up, o);
  store_v<T, VEC>((T *)a.y + r * a.y_stride + c0, n, o);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) store_v<T, VEC>(entry + (int64_t)i * a.C, n, u[i + 1]);
}

// f(T, K, VEC) for the call's type, taps and alignment.
template <typename F>
cudaError_t dispatch(const ConvArgs &a, F f) {
#define KDA_CONV_CASE(TT, KK)                                   \
  if (a.K == KK) return a.vec ? f.template run<TT, KK, true>() : f.template run<TT, KK, false>();
  if (a.bf16) {
    KDA_CONV_CASE(__nv_bfloat16, 2) KDA_CONV_CASE(__nv_bfloat16, 3) KDA_CONV_CASE(__nv_bfloat16, 4)
  } else {
    KDA_CONV_CASE(float, 2) KDA_CONV_CASE(float, 3) KDA_CONV_CASE(float, 4)
  }
#undef KDA_CONV_CASE
  return cudaErrorInvalidValue;
}

struct RunConv {
  const ConvArgs &a;
  cudaStream_t st;
  template <typename T, int K, bool VEC>
  cudaError_t run() const {
    const int tile = 16;
    const dim3 grid((unsigned)(((int64_t)a.q.rows + tile - 1) / tile), (a.C + kThreads * kVec<T> - 1) / (kThreads * kVec<T>));
    short_conv_kernel<T, K, VEC><<<grid, kThreads, 0, st>>>(a, tile);
    return cudaGetLastError();
  }
};

struct RunStep {
  const ConvArgs &a;
  cudaStream_t st;
  template <typename T, int K, bool VEC>
  cudaError_t run() const {
    const dim3 grid(a.q.R, (a.C + kThreads * kVec<T> - 1) / (kThreads * kVec<T>));
    short_conv_step_kernel<T, K, VEC><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_short_conv(const ConvArgs &a, cudaStream_t st) { return dispatch(a, RunConv{a, st}); }

cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t st) { return dispatch(a, RunStep{a, st}); }

}  // namespace kda
