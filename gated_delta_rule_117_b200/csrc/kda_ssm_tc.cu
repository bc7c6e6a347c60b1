// Selective state space scan on the sm_100a tensor cores (tcgen05 + TMEM +
// TMA): bf16, chunks of Q = 128 tokens, 64 state columns a CTA.
//
// Mathematics.  With l_t = d_t A log2(e) and, inside a chunk, L_t = l_0 + .. + l_t,
//     y_t  = sum_{s <= t} (C_t . B_s) d_s 2^{L_t - L_s} x_s  +  2^{L_t} C_t S  +  D x_t
//     S'   = 2^{L_127} S + sum_s B_s (d_s 2^{L_127 - L_s} x_s)^T
// so a chunk is four products (M x N x K):
//     G  = C B^T      128 x 128 x N      scores
//     Yx = C S        128 x 64 x N       what the entering state gives
//     dS = B^T wx     128 x 64 x 128     (wx = d 2^{L_127 - L} x, as bf16 hi + lo)
//     Yi = W x        128 x 64 x 128     (W = G masked and decayed, A operand in TMEM)
// Every exponent is a sum of l over consecutive tokens, formed from sums inside
// blocks of 32 tokens and whole-block totals, never as a difference of long
// sums: decays as small as those of one token keep their relative accuracy, and
// none overflows (l <= 0).  Below the diagonal blocks the decay factors into a
// row and a column part, so exponentials are taken for the diagonal blocks only.
//
// Rounding.  The state lives in fp32 registers; what is added to it is split into
// bf16 hi + lo (16 bits), as one bf16 would put 2^-9 of every update into it for
// good.  W and the copy of S that outputs read are single bf16: each costs an
// output about what its own rounding to bf16 does, and nothing carries on.
//
// What bounds it: 1.5 K cycles of tensor-core work a chunk against 32 KB of x and
// y from HBM (0.74 us at the copy rate); the roles below overlap, so the tensor
// pipe's 0.8 us and the handovers between roles set the pace.
//
// Work split: one CTA a (segment, head, 64 columns of P), 16 warps:
//   warp 0     producer: TMA loads of C, B, x (two stages), TMA stores of y
//   warp 1     decays: d, sums of l, the factors of every role (two stages)
//   warp 2     issues every MMA
//   warps 4-7  scores: thread t owns row t of G; writes W to TMEM
//   warps 8-11 tokens: thread t owns row t of x; writes wx, later the output row
//   warps 12-15 state: thread n owns row n of S (64 fp32 registers); writes the
//              bf16 copy, the snapshots and the final state
// Columns of S are independent, so P = 128 is two CTAs (which form G twice: it
// is a third of the tensor work and saves any exchange).  Rows behind a chunk's
// last token are zeroed in the operands that sum over tokens, and not stored;
// values that are not finite spoil their chunk's outputs, earlier tokens included.
//
// Handovers are mbarriers, one completion a chunk; a barrier is a ring of two
// where a waiter may fall a whole chunk behind.  Every wait is bounded: one that
// gives up records KDA_ERR_TIMEOUT, and the CTA drains and returns.
#include <cuda_bf16.h>

#include "kda_ssm_seg.cuh"
#include "kda_tmap.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int Q = 128;    // tokens of a chunk
constexpr int PC = 64;    // state columns of a CTA
constexpr int NT = 512;
static_assert(Q == kAlign, "snapshots fall on chunk ends");

// ---- shared memory (byte offsets from a 1024-aligned base) -------------------
// Tiles of 128-byte rows in the 128-byte swizzle; [rows x 128] tiles are two
// blocks of 64 columns (16 KB each).
constexpr int kC = 0;              // [2] C, 32 KB
constexpr int kB = 65536;          // [2] B, 32 KB
constexpr int kX = 131072;         // [2] x, 16 KB; later the chunk's y
constexpr int kW = 163840;         // wx hi | lo, 16 KB each
constexpr int kS = 196608;         // S as bf16 [n][p], 16 KB
constexpr int kDec = 212992;       // [2] Decays
constexpr int kBarOff = 219264;
constexpr int kMisc = 219520;       // TMEM base address, abort flag
constexpr int kSmemBytes = 219584 + 1024;

struct Decays {
  float d[Q];        // step (0 behind the last token)
  float pre[Q];      // sum of l from the token's block's first token to the token
  float w[Q];        // d 2^(sum of l behind the token, to the chunk's end)
  float col[3][Q];   // d 2^(sum behind the token to the start of the block i + 1, i + 2, i + 3 of its own i)
  float before[4];   // 2^(sum of l of the blocks before block i)
  float all;         // 2^(sum of l of the chunk)
  float pad[3];
};
static_assert(kDec + 2 * sizeof(Decays) <= kBarOff && kSmemBytes <= 232448, "shared memory layout");

enum {
  F_CB = 0,   // [2] C and B landed
  F_X = 2,    // [2] x landed
  DEC = 4,    // [2] decays written
  DEC_FREE = 6,  // [2] decays read by every role
  G_DONE = 8, // G in TMEM
  W_READY,    // W in TMEM (and G read)
  WX_READY,   // wx written, tail rows zeroed
  DS_DONE,    // dS in TMEM (and wx and S read)
  DS_READ,    // dS read
  S_READY,    // bf16 S of the chunk written
  Y_DONE,     // [2] Yi and Yx in TMEM (and W read)
  Y_READ = Y_DONE + 2,  // [2] they are read
  CB_FREE = Y_READ + 2, // [2] every MMA of the chunk done: C and B may be replaced
  X_FREE = CB_FREE + 2, // [2] x read (y staged in its place, in output runs)
  DRAIN = X_FREE + 2,   // every MMA issued is done
  BARS
};
static_assert(kBarOff + 8 * BARS <= kMisc, "barriers");

// TMEM columns
constexpr uint32_t kCols = 512;
constexpr uint32_t tG = 0, tW = 128, tDS = 192;
__device__ __forceinline__ uint32_t tYi(int i) { return 256u + 128u * (i & 1); }
__device__ __forceinline__ uint32_t tYx(int i) { return tYi(i) + 64u; }

struct TcArgs {
  SsmArgs a;
  int seg;
  float *ws, *decays;
  uint64_t wait_ns;
};

struct Cta {
  unsigned char *sm;
  uint64_t *bar;
  volatile int *abort;
  unsigned *status;
  uint64_t wait_ns;

  __device__ __noinline__ bool wait_slow(int b, uint32_t parity) const {
    const uint64_t t0 = global_ns();
    for (;;) {
      if (mbar_try_wait_sleep(&bar[b], parity, 1000000u)) return true;
      if (*abort) return false;
      if (global_ns() - t0 > wait_ns) break;
    }
    *abort = 1;
    atomicExch(status, kDevTimeout);
    return false;
  }
  // Phase `k` (0, 1, ...) of barrier b; the whole warp calls it.
  __device__ __forceinline__ bool wait(int b, int k) const {
    // the same answer for the whole warp: warp-wide instructions follow
    bool ok = mbar_try_wait(&bar[b], k & 1);
    if (__all_sync(~0u, ok)) return true;
    ok = ok || wait_slow(b, k & 1);
    return __all_sync(~0u, ok);
  }
  // Phase k / 2 of entry k % 2 of a ring.
  __device__ __forceinline__ bool wait2(int b, int k) const { return wait(b + (k & 1), k >> 1); }
  __device__ __forceinline__ void arrive(int b) const { mbar_arrive(&bar[b]); }
  __device__ __forceinline__ Decays &dec(int i) const { return *reinterpret_cast<Decays *>(sm + kDec + (i & 1) * sizeof(Decays)); }
};

// Chunk i of an item: its first token (counted from the sequence's first) and its tokens.
struct Chunks {
  int begin, end, base;  // tokens; base: the multiple of Q (counted with ctx) at or before begin, minus ctx
  int n;
  __device__ __forceinline__ explicit Chunks(const Item &it) {
    begin = it.begin;
    end = it.end;
    const int off = it.s.ctx % Q;
    base = (begin + off) / Q * Q - off;
    n = (end - base + Q - 1) / Q;
  }
  __device__ __forceinline__ int first(int i) const { return max(begin, base + Q * i); }
  __device__ __forceinline__ int count(int i) const { return min(end, base + Q * (i + 1)) - first(i); }
};

__device__ __forceinline__ float4 f4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// v as bf16 hi + lo: returns packed hi (rounded), writes packed lo.
__device__ __forceinline__ uint32_t split(float2 v, uint32_t &lo) {
  const __nv_bfloat162 h = __float22bfloat162_rn(v);
  const float2 b = __bfloat1622float2(h);
  lo = pack_bf16x2(v.x - b.x, v.y - b.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// kOut: the run that writes y, snapshots and final states; else the state pass,
// which leaves each segment's S~ and decay in the workspace.
template <bool kOut>
__global__ void __launch_bounds__(NT, 1)
    ssm_tc_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mb,
                  const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap my, const TcArgs p) {
  extern __shared__ __align__(1024) unsigned char smraw[];
  const SsmArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = (a.P + PC - 1) / PC;
  const int p0 = (int)(blockIdx.x % slices) * PC, h = (int)(blockIdx.x / slices % a.H);
  const bool tell = kOut && p0 == 0 && h == 0 && tid == 0;
  Item it;
  if (!item_of(a.q, blockIdx.x / (slices * a.H), p.seg, tell, it)) return;
  if (!kOut && it.index == it.count - 1) return;  // nothing follows it
  const Chunks ch(it);
  const int n = ch.n, g = h / (a.H / a.G), nk = a.N / 16;

  Cta x;
  unsigned char *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  x.sm = sm;
  x.bar = reinterpret_cast<uint64_t *>(sm + kBarOff);
  x.abort = reinterpret_cast<volatile int *>(sm + kMisc + 4);
  x.status = a.q.status;
  x.wait_ns = p.wait_ns;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + kMisc);
  const uint32_t sbase = smem_u32(sm);
  if (tid == 0) {
    for (int i = 0; i < BARS; ++i) {
      uint32_t count = 1;  // TMA and MMA completions
      if (i == DEC || i == DEC + 1) count = 32;
      if (i == DEC_FREE || i == DEC_FREE + 1) count = kOut ? 384 : 256;
      if (i == W_READY || i == WX_READY || i == DS_READ || i == S_READY || i == Y_READ || i == Y_READ + 1 ||
          i == X_FREE || i == X_FREE + 1)
        count = 128;
      mbar_init(&x.bar[i], count);
    }
    *x.abort = 0;
    mbar_init_fence();
  }
  if (warp == 3) {
    tmem_alloc(tslot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = *tslot;
  const uint32_t tl = tb + ((uint32_t)(32 * (warp & 3)) << 16);  // this warp's lanes
  const int row_of_seq = it.s.start;

  if (warp == 0) {
    // ======================= producer =======================
    const uint32_t cb_bytes = (kOut ? 2u : 1u) * (a.N > 64 ? 32768u : 16384u);
    int cb = 0, xs = 0;  // loads issued
    bool ok = true;
    auto store = [&](int i) {  // y of chunk i, staged in its x tile (ragged chunks are stored by the token warps)
      if (kOut && ch.count(i) == Q) {
        tma_store_3d_warp(&my, sm + kX + (i & 1) * 16384, p0, h, row_of_seq + ch.first(i));
        bulk_commit_warp();
        bulk_wait_read_all();
        __syncwarp();
      }
    };
    for (int i = 0; i < n; ++i) {
      const int st = i & 1, row = row_of_seq + ch.first(i);
      if (i >= 2 && !(ok = x.wait2(CB_FREE, i - 2))) break;
      mbar_arrive_expect_tx_warp(&x.bar[F_CB + st], cb_bytes);
      for (int c = 0; c < a.N; c += 64) {
        if (kOut) tma_load_3d_warp(sm + kC + st * 32768 + c * 256, &mc, &x.bar[F_CB + st], c, g, row);
        tma_load_3d_warp(sm + kB + st * 32768 + c * 256, &mb, &x.bar[F_CB + st], c, g, row);
      }
      cb = i + 1;
      if (i >= 2) {
        if (!(ok = x.wait2(X_FREE, i - 2))) break;
        store(i - 2);
      }
      mbar_arrive_expect_tx_warp(&x.bar[F_X + st], 16384u);
      tma_load_3d_warp(sm + kX + st * 16384, &mx, &x.bar[F_X + st], p0, h, row);
      xs = i + 1;
    }
    for (int i = max(0, n - 2); ok && i < n; ++i) {
      if (!(ok = x.wait2(X_FREE, i))) break;
      store(i);
    }
    if (!ok) {  // loads in flight must land before shared memory is given up
      const uint64_t t0 = global_ns();
      for (int k = 0; k < 4; ++k) {
        const int issued = k < 2 ? cb : xs, b = (k < 2 ? F_CB : F_X) + (k & 1);
        const int last = issued - 1 - ((issued - 1 - (k & 1)) & 1);  // the last chunk of this stage
        if (last < 0) continue;
        while (!mbar_try_wait_sleep(&x.bar[b], (last >> 1) & 1, 1000000u))
          if (global_ns() - t0 > p.wait_ns) break;
      }
    }
  } else if (warp == 1) {
    // ======================= decays =======================
    const float A2 = a.A[h] * 1.4426950408889634f;
    const __nv_bfloat16 *dt = (const __nv_bfloat16 *)a.dt + h;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    float raw[4];
    auto fetch = [&](int i) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = 32 * b + lane;
        raw[b] = i < n && t < ch.count(i) ? __bfloat162float(dt[(int64_t)(row_of_seq + ch.first(i) + t) * a.dt_stride]) : 0.f;
      }
    };
    fetch(0);
    float total = 0.f;
    for (int i = 0; i < n; ++i) {
      const int count = ch.count(i);
      float d[4], pre[4], suf[4], L[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float v = raw[b] + bias;
        if (a.softplus) v = softplus(v);
        d[b] = 32 * b + lane < count ? v : 0.f;
      }
      fetch(i + 1);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float l = d[b] * A2;
        float up = l, dn = l;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float u = __shfl_up_sync(~0u, up, o), v = __shfl_down_sync(~0u, dn, o);
          if (lane >= o) up += u;
          if (lane + o < 32) dn += v;
        }
        const float after = __shfl_down_sync(~0u, dn, 1);
        pre[b] = up;
        suf[b] = lane < 31 ? after : 0.f;
        L[b] = __shfl_sync(~0u, up, 31);
      }
      if (i >= 2 && !x.wait2(DEC_FREE, i - 2)) break;
      Decays &D = x.dec(i);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = 32 * b + lane;
        D.d[t] = d[b];
        D.pre[t] = pre[b];
        float s = suf[b];
#pragma unroll
        for (int k = b + 1; k < 4; ++k) {
          D.col[k - b - 1][t] = d[b] * exp2f(s);
          s += L[k];
        }
        D.w[t] = d[b] * exp2f(s);
      }
      const float all = L[0] + L[1] + L[2] + L[3];
      total += all;
      if (lane == 0) {
        D.before[0] = 1.f;
        D.before[1] = exp2f(L[0]);
        D.before[2] = exp2f(L[0] + L[1]);
        D.before[3] = exp2f(L[0] + L[1] + L[2]);
        D.all = exp2f(all);
      }
      x.arrive(DEC + (i & 1));
    }
    if (!kOut && lane == 0 && p0 == 0) p.decays[it.item * a.H + h] = exp2f(total);
  } else if (warp == 2) {
    // ======================= MMA issue =======================
    const uint32_t idG = idesc_bf16(128, 128, false, false, false);
    const uint32_t idYx = idesc_bf16(128, 64, false, true, false);
    const uint32_t idDS = idesc_bf16(128, 64, true, true, false);
    const uint64_t dS = sdesc_sw128(sbase + kS, 16, 1024);
    const uint64_t dW = sdesc_sw128(sbase + kW, 16, 1024);
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const uint64_t dC = sdesc_sw128(sbase + kC + st * 32768, 16, 1024);
      const uint64_t dB = sdesc_sw128(sbase + kB + st * 32768, 16, 1024);
      const uint64_t dBt = sdesc_sw128(sbase + kB + st * 32768, 16384, 1024);
      const uint64_t dX = sdesc_sw128(sbase + kX + st * 16384, 16, 1024);
      auto koff = [](int k) { return (uint32_t)((k >> 2) * 16384 + (k & 3) * 32); };
      if (!x.wait2(F_CB, i)) break;
      if (kOut) {
        // (G was read before W of the chunk before was ready)
        tc_fence_after();
        for (int k = 0; k < nk; ++k) mma_bf16_warp(tb + tG, sdesc_add(dC, koff(k)), sdesc_add(dB, koff(k)), idG, k > 0);
        mma_commit_warp(&x.bar[G_DONE]);
        if (i >= 2 && !x.wait2(Y_READ, i - 2)) break;
        if (!x.wait(S_READY, i)) break;
        tc_fence_after();
        for (int k = 0; k < nk; ++k)
          mma_bf16_warp(tb + tYx(i), sdesc_add(dC, koff(k)), sdesc_add(dS, k * 2048), idYx, k > 0);
      }
      if (!x.wait2(F_X, i) || !x.wait(WX_READY, i)) break;
      if (i >= 1 && !x.wait(DS_READ, i - 1)) break;
      tc_fence_after();
      for (int k = 0; k < 16; ++k)
        mma_bf16_warp(tb + tDS, sdesc_add(dBt, (k & 7) * 2048), sdesc_add(dW, k * 2048), idDS, k > 0);
      mma_commit_warp(&x.bar[DS_DONE]);
      if (kOut) {
        if (!x.wait(W_READY, i)) break;
        tc_fence_after();
        for (int k = 0; k < 8; ++k)
          mma_bf16_ts_warp(tb + tYi(i), tb + tW + k * 8, sdesc_add(dX, k * 2048), idYx, k > 0);
        mma_commit_warp(&x.bar[Y_DONE + st]);
      }
      mma_commit_warp(&x.bar[CB_FREE + st]);
    }
    mma_commit_warp(&x.bar[DRAIN]);
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait_sleep(&x.bar[DRAIN], 0, 1000000u))
      if (global_ns() - t0 > p.wait_ns) break;
  } else if (warp >= 4 && warp < 8) {
    // ======================= scores =======================
    if (kOut) {
      const int b = warp - 4;  // this warp's rows are block b
      const int t = 32 * b + lane;
      {  // tokens behind this warp's block: zeros, once
        uint32_t z[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = 0;
        for (int c = b + 1; c < 4; ++c) tmem_st16(tl + tW + 16 * c, z);
        tmem_st_wait();
      }
      for (int i = 0; i < n; ++i) {
        if (!x.wait2(DEC, i) || !x.wait(G_DONE, i)) break;
        if (i >= 1 && !x.wait2(Y_DONE, i - 1)) break;  // W is read
        tc_fence_after();
        const Decays &D = x.dec(i);
        const float pre = D.pre[t], rowf = exp2f(pre);
        for (int c = 0; c <= b; ++c) {
          float v[32];
          uint32_t w[16];
          tmem_ld32(tl + tG + 32 * c, v);
          tmem_ld_wait(v);
          if (c < b) {
            const float *col = D.col[b - c - 1] + 32 * c;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 f = f4(col + j);
              const float2 r2 = make_float2(rowf, rowf);
              const float2 lo = __fmul2_rn(__fmul2_rn(make_float2(v[j], v[j + 1]), r2), make_float2(f.x, f.y));
              const float2 hi = __fmul2_rn(__fmul2_rn(make_float2(v[j + 2], v[j + 3]), r2), make_float2(f.z, f.w));
              w[j / 2] = pack_bf16x2(lo.x, lo.y);
              w[j / 2 + 1] = pack_bf16x2(hi.x, hi.y);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 f = f4(D.pre + 32 * c + j), d = f4(D.d + 32 * c + j);
              const float e0 = j <= lane ? v[j] * (d.x * exp2f(pre - f.x)) : 0.f;
              const float e1 = j + 1 <= lane ? v[j + 1] * (d.y * exp2f(pre - f.y)) : 0.f;
              const float e2 = j + 2 <= lane ? v[j + 2] * (d.z * exp2f(pre - f.z)) : 0.f;
              const float e3 = j + 3 <= lane ? v[j + 3] * (d.w * exp2f(pre - f.w)) : 0.f;
              w[j / 2] = pack_bf16x2(e0, e1);
              w[j / 2 + 1] = pack_bf16x2(e2, e3);
            }
          }
          tmem_st16(tl + tW + 16 * c, w);
        }
        tmem_st_wait();
        tc_fence_before();
        x.arrive(W_READY);
        x.arrive(DEC_FREE + (i & 1));
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // ======================= tokens =======================
    const int t = 32 * (warp - 8) + lane;
    const float skip = kOut && a.D ? a.D[h] : 0.f;
    const float2 skip2 = make_float2(skip, skip);
    auto output = [&](int i) {  // y of chunk i, row t
      if (!x.wait2(Y_DONE, i)) return false;
      tc_fence_after();
      const Decays &D = x.dec(i);
      const float f = D.before[t >> 5] * exp2f(D.pre[t]);
      const float2 f2 = make_float2(f, f);
      unsigned char *xt = sm + kX + (i & 1) * 16384;
      const int count = ch.count(i);
      __nv_bfloat16 *yrow = (__nv_bfloat16 *)a.y + (int64_t)(row_of_seq + ch.first(i) + t) * a.y_stride + h * a.P + p0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float yi[32], yx[32];
        tmem_ld32(tl + tYi(i) + 32 * c, yi);
        tmem_ld32(tl + tYx(i) + 32 * c, yx);
        tmem_ld_wait(yi);
        tmem_ld_touch(yx);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint4 *at = reinterpret_cast<uint4 *>(xt + sw128_chunk(t, 4 * c + k));
          uint4 v = *at;
          uint32_t *u = &v.x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 8 * k + 2 * j;
            const float2 xv = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[j]));
            const float2 s = __ffma2_rn(f2, make_float2(yx[e], yx[e + 1]), make_float2(yi[e], yi[e + 1]));
            const float2 o = __ffma2_rn(skip2, xv, s);
            u[j] = pack_bf16x2(o.x, o.y);
          }
          *at = v;
          const int col = 32 * c + 8 * k;
          if (count < Q && t < count && p0 + col < a.P) *reinterpret_cast<uint4 *>(yrow + col) = v;
        }
      }
      tc_fence_before();
      x.arrive(Y_READ + (i & 1));
      fence_proxy_async_smem();
      x.arrive(X_FREE + (i & 1));
      x.arrive(DEC_FREE + (i & 1));
      return true;
    };
    int i = 0;
    for (; i < n; ++i) {
      if (!x.wait2(DEC, i) || !x.wait2(F_X, i)) break;
      if (i >= 1 && !x.wait(DS_DONE, i - 1)) break;  // wx is read
      const int count = ch.count(i);
      const bool live = t < count;
      const float f = x.dec(i).w[t];
      const float2 f2 = make_float2(f, f);
      unsigned char *xt = sm + kX + (i & 1) * 16384;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t at = sw128_chunk(t, k);
        const uint4 v = *reinterpret_cast<const uint4 *>(xt + at);
        const uint32_t *u = &v.x;
        uint4 hi, lo;
        uint32_t *ph = &hi.x, *pl = &lo.x;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ph[j] = split(__fmul2_rn(f2, __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[j]))), pl[j]);
        if (!live) hi = lo = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(sm + kW + at) = hi;
        *reinterpret_cast<uint4 *>(sm + kW + 16384 + at) = lo;
      }
      if (count < Q) {  // rows behind the last token: x and B sum over tokens, so they must be zeros
        if (!x.wait2(F_CB, i)) break;
        if (!live) {
          const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t at = sw128_chunk(t, k);
            if (kOut) *reinterpret_cast<uint4 *>(xt + at) = z;
            *reinterpret_cast<uint4 *>(sm + kB + (i & 1) * 32768 + at) = z;
            *reinterpret_cast<uint4 *>(sm + kB + (i & 1) * 32768 + 16384 + at) = z;
          }
        }
      }
      fence_proxy_async_smem();
      x.arrive(WX_READY);
      if (kOut) {
        if (i >= 1 && !output(i - 1)) break;
      } else {
        x.arrive(X_FREE + (i & 1));
        x.arrive(DEC_FREE + (i & 1));
      }
    }
    if (kOut && i == n) output(n - 1);
  } else if (warp >= 12) {
    // ======================= state =======================
    const int row = 32 * (warp - 12) + lane;
    const bool live = row < a.N;
    const int cols = min(PC, a.P - p0);
    const int64_t np = (int64_t)a.N * a.P, at = (int64_t)row * a.P + p0;
    float S[PC];
    const float *from = nullptr;
    if (kOut && live) {
      if (p.seg != 0) from = p.ws + (it.item * a.H + h) * np + at;
      else if (a.state && it.s.ctx > 0) from = a.state + ((int64_t)it.s.slot * a.H + h) * np + at;
    }
#pragma unroll
    for (int j = 0; j < PC; j += 4) {
      const float4 v = from && j < cols ? f4(from + j) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
    }
    auto save = [&](float *to) {
      if (!live) return;
#pragma unroll
      for (int j = 0; j < PC; j += 4)
        if (j < cols) *reinterpret_cast<float4 *>(to + at + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
    };
    int i = 0;
    for (; i < n; ++i) {
      if (kOut) {  // (the products that read the copy before this one are done: DS_DONE)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint4 v;
          v.x = pack_bf16x2(S[8 * k + 0], S[8 * k + 1]);
          v.y = pack_bf16x2(S[8 * k + 2], S[8 * k + 3]);
          v.z = pack_bf16x2(S[8 * k + 4], S[8 * k + 5]);
          v.w = pack_bf16x2(S[8 * k + 6], S[8 * k + 7]);
          *reinterpret_cast<uint4 *>(sm + kS + sw128_chunk(row, k)) = v;
        }
        fence_proxy_async_smem();
        x.arrive(S_READY);
      }
      if (!x.wait2(DEC, i)) break;
      const float keep = x.dec(i).all;
      x.arrive(DEC_FREE + (i & 1));
      if (!x.wait(DS_DONE, i)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v[32];
        tmem_ld32(tl + tDS + 32 * c, v);
        tmem_ld_wait(v);
#pragma unroll
        for (int j = 0; j < 32; ++j) S[32 * c + j] = fmaf(keep, S[32 * c + j], v[j]);
      }
      tc_fence_before();
      x.arrive(DS_READ);
      if (kOut && a.page) {
        const int64_t pos = (int64_t)it.s.ctx + ch.first(i) + ch.count(i);
        if (float *to = snapshot(a, it.r, h, pos, p0 == 0 && row == 0)) save(to);
      }
    }
    if (i == n) {
      if (!kOut) save(p.ws + (it.item * a.H + h) * np);
      else if (a.state && it.index == it.count - 1) save(a.state + ((int64_t)it.s.slot * a.H + h) * np);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) tmem_dealloc(tb, kCols);
}

}  // namespace

bool ssm_tc_fits(const SsmArgs &a) {
  auto row16 = [](const void *p, int64_t stride) { return ((uintptr_t)p & 15) == 0 && stride % 8 == 0; };
  return a.bf16 && row16(a.x, a.x_stride) && row16(a.B, a.b_stride) && row16(a.C, a.c_stride) && row16(a.y, a.y_stride);
}

cudaError_t launch_ssm_tc(const SsmArgs &a, int seg, cudaStream_t st) {
  CUtensorMap mx, mb, mc, my;
  const uint64_t rows = (uint64_t)a.q.rows;
  if (!encode_tmap_bf16_rows(&mx, a.x, a.P, a.H, rows, a.x_stride, PC, Q) ||
      !encode_tmap_bf16_rows(&mb, a.B, a.N, a.G, rows, a.b_stride, 64, Q) ||
      !encode_tmap_bf16_rows(&mc, a.C, a.N, a.G, rows, a.c_stride, 64, Q) ||
      !encode_tmap_bf16_rows(&my, a.y, a.P, a.H, rows, a.y_stride, PC, Q))
    return cudaErrorInvalidValue;
  const int64_t items = scan_items(a.q.R, a.q.rows, seg);
  TcArgs p;
  p.a = a;
  p.seg = seg;
  p.ws = seg ? seg_states(a) : nullptr;
  p.decays = seg ? seg_decays(a, items) : nullptr;
  p.wait_ns = debug_wait_ns();
  const unsigned grid = (unsigned)(items * a.H * ((a.P + PC - 1) / PC));
  cudaError_t e = cudaFuncSetAttribute(ssm_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(ssm_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  if (seg) {
    ssm_tc_kernel<false><<<grid, NT, kSmemBytes, st>>>(mx, mb, mc, my, p);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_segment_states(a, seg, st);
    if (e != cudaSuccess) return e;
  }
  ssm_tc_kernel<true><<<grid, NT, kSmemBytes, st>>>(mx, mb, mc, my, p);
  return cudaGetLastError();
}

}  // namespace kda
