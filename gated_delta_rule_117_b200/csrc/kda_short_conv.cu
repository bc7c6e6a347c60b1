// Short causal convolution (include/kda.h, kda_short_conv and
// kda_short_conv_step; Kimi K3 report, section 2.1.1, Eq. 2 without the
// projections): K taps a channel, Swish, L2 norm of each head.
//
// Bytes bound both: an input element is read once and an output element
// written once for about 2 K + 8 operations.  A thread owns four channels (8 or
// 16 bytes; a warp moves 256 or 512 bytes of a row) and walks down a tile of rows
// with the last K - 1 inputs in registers, so an input is loaded once a tile (plus
// K - 1 rows of halo), sixteen rows ahead of their use.  Eight channels a thread took
// 168 registers, which left 3 blocks an SM and 1.8 TB/s at 65,536 x 4,352 bf16.
// Tiles are cut over the packed rows, not over the sequences, so the grid needs no
// lengths on the host; a tile walks through the sequences that it meets.
//
// The pool is read where a sequence starts and written where it ends, which
// may be different tiles: the tile with the last row therefore also computes
// the first K - 1 outputs of a sequence that reads the pool, so one thread
// reads the old entry and writes the new one, in that order.
#include "kda_serve.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
// Blocks an SM: 6 leave 80 registers (7 and 8 spill: 225 and 253 us against 216 at 65,536 x
// 4,352 bf16), 5 leave the norm of four rows at a time its 96.
constexpr int blocks_of(bool norm) { return norm ? 5 : 6; }
constexpr int V = 4;  // channels of a thread

// Four elements as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ float2 lo() const { return pair(u.x); }
  __device__ __forceinline__ float2 hi() const { return pair(u.y); }
  static __device__ __forceinline__ float2 pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <>
struct Raw<float> {
  float4 u;
  __device__ __forceinline__ float2 lo() const { return make_float2(u.x, u.y); }
  __device__ __forceinline__ float2 hi() const { return make_float2(u.z, u.w); }
};

struct F4 {
  float2 a, b;
};
template <typename T>
__device__ __forceinline__ F4 widen(const Raw<T> &r) { return F4{r.lo(), r.hi()}; }

__device__ __forceinline__ Raw<__nv_bfloat16> narrow(const F4 &v, __nv_bfloat16) {
  const __nv_bfloat162 a = __float22bfloat162_rn(v.a), b = __float22bfloat162_rn(v.b);
  return Raw<__nv_bfloat16>{make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b))};
}
__device__ __forceinline__ Raw<float> narrow(const F4 &v, float) {
  return Raw<float>{make_float4(v.a.x, v.a.y, v.b.x, v.b.y)};
}

// Four elements from p (aligned to them if VEC); zeros behind the first n.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load4(const T *p, int n) {
  union { Raw<T> r; T t[V]; };
  if constexpr (VEC) {
    if (n > 0) return *reinterpret_cast<const Raw<T> *>(p);
#pragma unroll
    for (int j = 0; j < V; ++j) t[j] = as_type<T>(0.f);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) t[j] = j < n ? p[j] : as_type<T>(0.f);
  }
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store4(T *p, int n, const F4 &v) {
  union { Raw<T> r; T t[V]; };
  r = narrow(v, T());
  if constexpr (VEC) {
    if (n > 0) *reinterpret_cast<Raw<T> *>(p) = r;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) p[j] = t[j];
  }
}

// v Sigmoid(v).  The bf16 form takes the hardware's 2^x and 1/x (2^-22 relative, far
// below a bf16 step; results below the normal range are 0): nine instructions a pair.
__device__ __forceinline__ float2 swish(float2 v, __nv_bfloat16) {
  float2 e = __fmul2_rn(v, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  e = __fadd2_rn(e, make_float2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  return __fmul2_rn(v, e);
}
__device__ __forceinline__ float2 swish(float2 v, float) {
  return make_float2(v.x / (1.f + expf(-v.x)), v.y / (1.f + expf(-v.y)));
}

// 1 / sqrt(v); the bf16 form is off by at most two units in the last place.
__device__ __forceinline__ float inverse_root(float v, __nv_bfloat16) { return rsqrtf(v); }
__device__ __forceinline__ float inverse_root(float v, float) { return 1.f / sqrtf(v); }

template <int K>
struct Taps {
  F4 w[K], b;
};

template <typename T, int K, bool VEC>
__device__ __forceinline__ Taps<K> load_taps(const ConvArgs &a, int c0, int n) {
  Taps<K> t;
  union { Raw<T> r[K]; T e[V * K]; };  // channel by channel, as in memory
  const T *w = (const T *)a.w + (int64_t)c0 * K;
  union { Raw<T> rb; T eb[V]; };
#pragma unroll
  for (int i = 0; i < K; ++i) r[i] = load4<T, VEC>(w + V * i, VEC ? n : n * K - V * i);
  rb = load4<T, VEC>((const T *)a.bias + c0, a.bias ? n : 0);
#pragma unroll
  for (int i = 0; i < K; ++i)
    t.w[i] = F4{make_float2(as_float(e[i]), as_float(e[K + i])), make_float2(as_float(e[2 * K + i]), as_float(e[3 * K + i]))};
  t.b = F4{make_float2(as_float(eb[0]), as_float(eb[1])), make_float2(as_float(eb[2]), as_float(eb[3]))};
  return t;
}

// A thread's own queue of its tile's rows in flight, in shared memory: kDepth rows
// asynchronous copies ahead, across the borders of sequences, without a register or a
// barrier for them (every thread reads only what it asked for).  65,536 x 4,352 bf16:
// 283 us with four rows ahead in registers.
constexpr int kGroup = 4, kGroups = 4, kDepth = kGroup * kGroups;
template <typename T>
struct Queue {
  Raw<T> *mine;    // [kDepth][kThreads], this thread's column
  const T *from;   // the next row to ask for
  int64_t xs;
  int left;        // rows of the tile that are not asked for yet
  int i;           // rows taken of the oldest group
  int head;        // its first place
  // Ask for the next kGroup rows, into the places from `to` on.
  __device__ __forceinline__ void ask(int to) {
    uint32_t p = (uint32_t)__cvta_generic_to_shared(mine + to);
#pragma unroll
    for (int b = 0; b < kGroup; ++b, from += xs)
      if (b < left)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(p + b * kThreads * (int)sizeof(Raw<T>)), "l"(from),
                     "n"((int)sizeof(Raw<T>))
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    left -= kGroup;
  }
  // Rows from p on, `rows` of them.
  __device__ __forceinline__ void begin(const T *p, int rows) {
    asm volatile("cp.async.wait_all;" ::: "memory");  // nothing may still land in the places
    from = p;
    left = rows;
    i = head = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) ask(g * kGroup * kThreads);
  }
  // The oldest group that was asked for has arrived.
  __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 1) : "memory"); }
  // Row b of it.
  __device__ __forceinline__ Raw<T> row(int b) const { return mine[head + b * kThreads]; }
  // The group is used up: its places take the next rows.
  __device__ __forceinline__ void next_group() {
    ask(head);
    i = 0;
    head = head == (kGroups - 1) * kGroup * kThreads ? 0 : head + kGroup * kThreads;
  }
};

// The convolution and Swish of one row from its K inputs, oldest first.
template <typename T, int K>
__device__ __forceinline__ F4 conv_row(const ConvArgs &a, const Taps<K> &t, const F4 (&u)[K]) {
  F4 o = t.b;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    o.a = __ffma2_rn(t.w[i].a, u[i].a, o.a);
    o.b = __ffma2_rn(t.w[i].b, u[i].b, o.b);
  }
  if (a.silu) {
    o.a = swish(o.a, T());
    o.b = swish(o.b, T());
  }
  return o;
}

// The L2 norm of NR rows' heads.  A head's channels lie in d / V neighbouring lanes, so
// its sum is a butterfly over them, the rows' in step: every lane of the warp must come
// here.
template <typename T, int NR>
__device__ __forceinline__ void norm_rows(const ConvArgs &a, F4 (&o)[NR]) {
  float ss[NR];
#pragma unroll
  for (int b = 0; b < NR; ++b) {
    const float2 q = __ffma2_rn(o[b].a, o[b].a, __fmul2_rn(o[b].b, o[b].b));
    ss[b] = q.x + q.y;
  }
  for (int off = 1; off < a.d / V; off <<= 1)
#pragma unroll
    for (int b = 0; b < NR; ++b) ss[b] += __shfl_xor_sync(~0u, ss[b], off);
#pragma unroll
  for (int b = 0; b < NR; ++b) {
    const float f = inverse_root(ss[b] + a.eps, T());
    o[b].a = __fmul2_rn(o[b].a, make_float2(f, f));
    o[b].b = __fmul2_rn(o[b].b, make_float2(f, f));
  }
}

template <typename T, int K, bool VEC, bool NORM>
__global__ void __launch_bounds__(kThreads, blocks_of(NORM)) short_conv_kernel(ConvArgs a, int tile) {
  __shared__ Raw<T> rows_ahead[VEC ? kDepth * kThreads : 1];
  Queue<T> queue;
  queue.mine = rows_ahead + (VEC ? threadIdx.x : 0);
  const Requests &q = a.q;
  const int row0 = (int)((int64_t)blockIdx.x * tile);
  const int c0 = (blockIdx.y * kThreads + threadIdx.x) * V;
  const int n = min(V, a.C - c0);  // <= 0: nothing of this thread's exists
  const T *x = (const T *)a.x + c0;
  T *pool = a.state ? (T *)a.state + c0 : nullptr;
  const int64_t xs = a.x_stride;

  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) tell_offsets(q);
  int total = q.rows, r;
  if (q.cu) {
    total = min(q.cu[q.R], q.rows);
    r = block_count_le(q.R, [&](int i) { return q.cu[i]; }, row0) - 1;
  } else {
    r = row0 / q.T;
  }
  const int rend = min((int64_t)row0 + tile, (int64_t)total);
  int row = row0;
  if (r < 0) {
    r = 0;
    row = q.cu[0];
  }
  if (row >= rend) return;
  queue.xs = xs;
  auto ahead = [&]() {
    if (VEC && row < rend) queue.begin(x + row * xs, n > 0 ? rend - row : 0);
  };
  ahead();
  // the rows before the tile, asked for before it is known whose they are
  Raw<T> before[K - 1];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) before[i] = load4<T, VEC>(x + (row - (K - 1) + i) * xs, row - (K - 1) + i >= 0 ? n : 0);
  bool at_start = true;
  const Taps<K> taps = load_taps<T, K, VEC>(a, c0, n);

  while (row < rend) {
    while (r < q.R && q.cu && q.cu[r + 1] <= row) ++r;
    if (r >= q.R) break;
    const Seq s = seq_of(q, r, blockIdx.y == 0 && threadIdx.x == 0);
    const int stop = min(s.end, rend);
    if (!s.ok || row < s.start) {  // (row < start: offsets that decrease)
      row = max(stop, row + 1);
      ++r;
      at_start = false;
      ahead();
      continue;
    }
    const bool carry = pool && s.ctx > 0, here = s.end <= rend;
    T *entry = pool ? pool + (int64_t)s.slot * (K - 1) * a.C : nullptr;
    // where the sequence's row 0 goes, and the step from row to row
    T *y = (T *)a.y;
    int64_t ys = a.y_stride;
    if (a.head_major) {
      ys = a.d;
      y += (((int64_t)r * a.heads + (c0 >> a.log2_d)) * q.T << a.log2_d) + (c0 & (a.d - 1));
    } else {
      y += s.start * ys + c0;
    }
    F4 h[K - 1];  // the K - 1 inputs before `row`, oldest first
    // (a sequence that reads the pool and ends in a later tile: that tile computes the outputs
    // that need it)
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int at = row - (K - 1) + i;
      const F4 zero = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      // (only the tile's first sequence can have begun before it)
      h[i] = at >= s.start    ? (at_start ? widen(before[i]) : zero)
             : carry && here ? widen(load4<T, VEC>(entry + (int64_t)(at - s.start + K - 1) * a.C, n))
                             : zero;
    }
    at_start = false;
    if (carry && here && row > s.start) {  // its first rows, in earlier tiles
      for (int at = s.start; at < min(row, s.start + K - 1); ++at) {
        F4 u[K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const int p = at - (K - 1) + i - s.start;
          u[i] = widen(load4<T, VEC>(p >= 0 ? x + (s.start + p) * xs : entry + (int64_t)(p + K - 1) * a.C, n));
        }
        F4 o[1] = {conv_row<T, K>(a, taps, u)};
        if (NORM) norm_rows<T>(a, o);
        store4<T, VEC>(y + (at - s.start) * ys, n, o[0]);
      }
    }
    const int first = carry && !here ? s.start + K - 1 : row;  // rows before it are another tile's
    T *yr = y + (row - s.start) * ys;
    // one row before its norm: its inputs are h and `in`, which then moves into h
    auto step = [&](const Raw<T> &in) {
      F4 w[K];
#pragma unroll
      for (int i = 0; i < K - 1; ++i) w[i] = h[i];
      w[K - 1] = widen(in);
#pragma unroll
      for (int i = 0; i < K - 1; ++i) h[i] = w[i + 1];
      return conv_row<T, K>(a, taps, w);
    };
    while (row < stop) {
      if (VEC && queue.i == 0 && row + kGroup <= stop && row >= first) {  // a whole group
        queue.wait();
        F4 o[kGroup];
#pragma unroll
        for (int b = 0; b < kGroup; ++b) {
          o[b] = step(queue.row(b));
          if (!NORM) {
            store4<T, VEC>(yr, n, o[b]);
            yr += ys;
          }
        }
        queue.next_group();
        if (NORM) {
          norm_rows<T>(a, o);
#pragma unroll
          for (int b = 0; b < kGroup; ++b, yr += ys) store4<T, VEC>(yr, n, o[b]);
        }
        row += kGroup;
      } else if constexpr (VEC) {
        if (queue.i == 0) queue.wait();
        F4 o[1] = {step(queue.row(queue.i))};
        if (NORM) norm_rows<T>(a, o);
        if (row >= first) store4<T, VEC>(yr, n, o[0]);
        if (++queue.i == kGroup) queue.next_group();
        ++row;
        yr += ys;
      } else {
        Raw<T> in[kGroup];  // element by element, a group's loads in flight together
#pragma unroll
        for (int b = 0; b < kGroup; ++b) in[b] = load4<T, VEC>(x + (row + b) * xs, row + b < stop ? n : 0);
#pragma unroll
        for (int b = 0; b < kGroup; ++b)
          if (row + b < stop) {
            F4 o[1] = {step(in[b])};
            if (NORM) norm_rows<T>(a, o);
            if (row + b >= first) store4<T, VEC>(yr + b * ys, n, o[0]);
          }
        row += kGroup;
        yr += kGroup * ys;
      }
    }
    row = stop;
    if (here && pool) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) store4<T, VEC>(entry + (int64_t)i * a.C, n, h[i]);
    }
    ++r;
  }
  if (VEC) asm volatile("cp.async.wait_all;" ::: "memory");  // nothing in flight at the block's end
}

template <typename T, int K, bool VEC, bool NORM>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(ConvArgs a) {
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
  F4 u[K];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) u[i] = widen(load4<T, VEC>(entry + (int64_t)i * a.C, n));
  u[K - 1] = widen(load4<T, VEC>((const T *)a.x + r * a.x_stride + c0, n));
  const Taps<K> taps = load_taps<T, K, VEC>(a, c0, n);
  F4 o[1] = {conv_row<T, K>(a, taps, u)};
  if (NORM) norm_rows<T>(a, o);
  store4<T, VEC>((T *)a.y + r * a.y_stride + c0, n, o[0]);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) store4<T, VEC>(entry + (int64_t)i * a.C, n, u[i + 1]);
}

// f(T, K, VEC, NORM) for the call's type, taps, alignment and norm.
template <typename F>
cudaError_t dispatch(const ConvArgs &a, F f) {
#define KDA_CONV_CASE(TT, KK)                                                                            \
  if (a.K == KK)                                                                                       \
    return a.norm ? (a.vec ? f.template run<TT, KK, true, true>() : f.template run<TT, KK, false, true>()) \
                  : (a.vec ? f.template run<TT, KK, true, false>() : f.template run<TT, KK, false, false>());
  if (a.bf16) {
    KDA_CONV_CASE(__nv_bfloat16, 2) KDA_CONV_CASE(__nv_bfloat16, 3) KDA_CONV_CASE(__nv_bfloat16, 4)
  } else {
    KDA_CONV_CASE(float, 2) KDA_CONV_CASE(float, 3) KDA_CONV_CASE(float, 4)
  }
#undef KDA_CONV_CASE
  return cudaErrorInvalidValue;
}

// Rows of a tile: 64, or as few as let all tiles run at once, but 8 at
// least, as a tile costs about eight rows' instructions to begin.  4,096 x 2,048 with
// norms: tiles of 16 rows (1,024 of them, a second wave of 136) took 18.3 us, of 20
// 14 us.
int conv_tile(const ConvArgs &a) {
  const int64_t columns = (a.C + kThreads * V - 1) / (kThreads * V), at_once = blocks_of(a.norm) * 148;
  const int64_t tile = (columns * a.q.rows + at_once - 1) / at_once;
  return (int)(tile >= 64 ? 64 : tile <= 8 ? 8 : (tile + kGroup - 1) / kGroup * kGroup);
}

struct RunConv {
  const ConvArgs &a;
  cudaStream_t st;
  template <typename T, int K, bool VEC, bool NORM>
  cudaError_t run() const {
    const int tile = conv_tile(a);
    const dim3 grid((unsigned)(((int64_t)a.q.rows + tile - 1) / tile), (a.C + kThreads * V - 1) / (kThreads * V));
    short_conv_kernel<T, K, VEC, NORM><<<grid, kThreads, 0, st>>>(a, tile);
    return cudaGetLastError();
  }
};

struct RunStep {
  const ConvArgs &a;
  cudaStream_t st;
  template <typename T, int K, bool VEC, bool NORM>
  cudaError_t run() const {
    const dim3 grid(a.q.R, (a.C + kThreads * V - 1) / (kThreads * V));
    short_conv_step_kernel<T, K, VEC, NORM><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_short_conv(const ConvArgs &a, cudaStream_t st) { return dispatch(a, RunConv{a, st}); }

cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t st) { return dispatch(a, RunStep{a, st}); }

}  // namespace kda
