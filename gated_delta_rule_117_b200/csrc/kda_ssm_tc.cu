// Selective state space scan on the sm_100a tensor cores (tcgen05 + TMEM +
// TMA): bf16, chunks of Q = 128 tokens, 64 state columns a CTA.
//
// Mathematics.  With l_t = d_t A log2(e) and, inside a chunk, L_t = l_0 + .. + l_t,
//     y_t  = sum_{s <= t} (C_t . B_s) d_s 2^{L_t - L_s} x_s  +  2^{L_t} C_t S  +  D x_t
//     S'   = 2^{L_127} S + sum_s B_s (d_s 2^{L_127 - L_s} x_s)^T
// so a chunk is four products (M x N x K):
//     G  = C B^T      128 x 128 x N      scores
//     Yx = C S        128 x 64 x N       what the entering state gives
//     dS = B^T wx     128 x 64 x 128     (wx = d 2^{L_127 - L} x, in three bf16 terms)
//     Yi = W x        128 x 64 x 128     (W = G masked and decayed, in two bf16 terms, A operand in TMEM)
// Every exponent is a sum of l over exactly the tokens that it spans, all of one sign,
// never a difference of two sums: decays as small as those of one token keep their
// relative accuracy beside a step that wipes the state out (1e4 and more, where a
// difference of sums loses them), and l = -inf gives 0, not NaN.  Below the
// diagonal blocks of 32 tokens the decay factors into a row and a column part, sums over
// a block's end or beginning and whole blocks between, so exponentials are taken for the
// diagonal blocks only; there a thread adds l up from its row backwards.
//
// Rounding.  The state lives in fp32 registers; what is added to it is split into
// three bf16 terms (24 bits), so the state keeps fp32 accuracy: one bf16 would be off
// by up to 2^-8 of every update for good, and two by 2^-16.  W is split into two (16 bits):
// single, it cost an output up to 2.3e-3 of it in the mean square, where its own rounding to
// bf16 is 1.66e-3 (2.09e-3 at 131,072 tokens of 16 heads, 1.67e-3 with the second term, which
// takes 8 % of the time).  Only the copy of S that outputs read is single bf16, and what it costs is
// not carried on from token to token.  By how much of an output the entering state makes up: 1.66e-3
// to 1.67e-3 at steps d A of -0.1 and beyond, 1.81e-3 at -1e-3 (2.24e-3 without the skip term),
// 2.33e-3 at worst (smaller steps, no skip term; 1.68e-3 with it).  A second term of it was built: y then
// takes x's place in shared memory, 1.66e-3 throughout, and 870 us for those 131,072 tokens against 835.
//
// What bounds it: the score warps' path between G and Yi, and shared memory.  A chunk's
// products read 224 KB (with N = 64 columns an operand pair feeds the tensor core at 48
// cycles a step for its 32), loads and stores by TMA move 96 KB and the roles 128 KB: 3,500
// cycles at 128 bytes a cycle.  Measured, 148 CTAs, N = 128: 4,600 cycles, 2.45 us a chunk
// (against 0.74 us for its 32 KB of x and y at the copy rate), tensor pipe 44 % and issue
// slots 54 % busy.  What was tried and lost: rows of y stored from registers instead of a
// staged tile (2.99 us against 2.33), the outputs' tensor memory read at once (2.42 against
// 2.33), the score warps sharing wx in output runs (3.03), Yx in two places of tensor memory so
// that it need not wait for the outputs (the same), first terms of W cut instead of rounded
// (857 us against 846).  Two terms of wx instead of three are 7 % faster and lose the state's
// last 8 bits.
//
// Work split: one CTA a (segment, head, 64 columns of P), 32 warps of 64 registers:
//   warp 0       producer: TMA loads of B, x (two stages) and C
//   warps 1, 3   decays: steps, sums of l, the factors of every role (up to four
//                chunks ahead); warps 24-27 in a state pass
//   warp 2       issues every MMA
//   warps 4-11   scores: two threads own row t of G, half a block of columns each;
//                they write W in G's place, up to the row's own block (the MMA leaves a row out
//                where W has nothing: 64 columns of zeros a chunk and row need not be written)
//   warps 12-15  tokens: thread t writes row t of wx (with warps 4-11, in a state pass)
//   warps 16-23  state: two threads own row n of S, 32 columns (fp32 registers)
//                each; they write the bf16 copy, the snapshots and the final state
//   warps 24-31  outputs: two threads own row t of y, 32 columns each; a warp stores
//                its tile by TMA
// The order of a chunk's products, Yx, G, dS, Yi, lets the roles work under the tensor
// time of others: scores under dS, the state update under Yi.  C is single-buffered
// (its readers come first), which makes room for wx's third term; B and x have two
// stages.
// Columns of S are independent, so P = 128 is two CTAs (which form G twice: it
// is a third of the tensor work and saves any exchange).  Rows behind a chunk's
// last token are zeroed in the operands that sum over tokens, and not stored.  An x that is not
// finite spoils the outputs of the earlier tokens of its block of 32 (0 times it); other
// inputs that are not finite meet no earlier token.
//
// Handovers are mbarriers, one completion a chunk; a barrier is a ring of two
// where a waiter may fall a whole chunk behind.  Every wait is bounded: one that
// gives up records KDA_ERR_TIMEOUT, and the CTA drains and returns: its loads have
// landed and its MMAs are done before shared and tensor memory are given up, however
// short the limit of the waits is (the drain has a limit of its own).
#include <cuda_bf16.h>

#include "kda_ssm_seg.cuh"
#include "kda_tmap.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int Q = 128;    // tokens of a chunk
constexpr int PC = 64;    // state columns of a CTA
constexpr int NT = 1024;
static_assert(Q == kAlign, "snapshots fall on chunk ends");

// ---- shared memory (byte offsets from a 1024-aligned base) -------------------
// Tiles of 128-byte rows in the 128-byte swizzle; [rows x 128] tiles are two
// blocks of 64 columns (16 KB each).
constexpr int kC = 0;              // C, 32 KB
constexpr int kB = 32768;          // [2] B, 32 KB
constexpr int kX = 98304;          // [2] x, 16 KB
constexpr int kW = 131072;         // wx terms, 3 x 16 KB
constexpr int kS = 180224;         // S as bf16 [n][p], 16 KB
constexpr int kY = 196608;         // y, 16 KB
constexpr int kDec = 212992;       // [4] Decays
constexpr int kBarOff = 227584;
constexpr int kMisc = 227840;      // Misc
constexpr int kSmemBytes = 227968 + 1024;

struct Decays {
  float d[Q];        // step (0 behind the last token)
  float pre[Q];      // sum of l from the token's block's first token to the token
  float mid[Q];      // the same from the token's half block's first token
  float w[Q];        // d 2^(sum behind the token to the chunk's end)
  float col[3][Q];   // d 2^(sum behind the token to the start of the block i + 1, i + 2, i + 3 of its own i)
  float total[4];    // sum of l of each block
  float before[4];   // 2^(sum of l of the blocks before block i)
  float all;         // 2^(sum of l of the chunk)
  float pad[3];
};
static_assert(kDec + 4 * sizeof(Decays) <= kBarOff && kSmemBytes <= 232448, "shared memory layout");

enum {
  F_BX = 0,   // [2] x landed, and B in an output run
  BX_FREE = 2,   // [2] every reader of those is done
  DEC = 4,       // [4] decays written
  DEC_FREE = 8,  // [4] decays read by the other roles
  F_C = 12,   // C landed
  C_FREE,     // C read (Yx done)
  G_DONE,     // G in TMEM
  W_READY,    // W in TMEM (and G read)
  WX_READY,   // [2] wx written, tail rows zeroed; the dS that was in its place is read
  DS_DONE = WX_READY + 2,  // [2] dS in TMEM (and wx and S read)
  YX_READY = DS_DONE + 2,  // bf16 S of the chunk written; the Yi and Yx before are read
  Y_DONE,     // [2] Yi and Yx in TMEM (and W read)
  TOTALS = Y_DONE + 2,  // the blocks' totals are written
  F_B,        // [2] state pass: B landed
  B_FREE = F_B + 2,  // [2] state pass: B read
  DRAIN = B_FREE + 2,  // every MMA issued is done
  NEVER,      // nothing arrives here: the wait of an injected stall (failure-detection tests)
  BARS
};
static_assert(kBarOff + 8 * BARS <= kMisc, "barriers");

// TMEM columns
constexpr uint32_t kCols = 512;
// (state pass: dS twice, at 0 and 192)
constexpr uint32_t tG = 0, tDS = 192, tYi = 384, tYx = 448;  // dS: one block of 64 for each term of wx
// W takes the place of G: the 16 scores of a K step become 8 columns of first terms and 8 of second ones

// A state pass has no C, S or y, so it has room for two wx and two dS: wx of a chunk is
// written while the products of the one before run.  And as its chunks are short against
// the latency of their loads (2,300 cycles from a stage's release to its next tiles), x is
// released when wx is written and B, which only the products read, on its own.  131,072
// tokens, 16 heads of 128, 9 segments: 279 us, against 313 with x and B released
// together and one wx.  Places and depth of each run:
template <bool kOut>
struct Layout {
  static constexpr int B = kOut ? kB : 0, X = kOut ? kX : 65536, W = kOut ? kW : 98304;
  static constexpr int kDeep = kOut ? 1 : 2;
  static __device__ __forceinline__ int w(int i) { return W + (kOut ? 0 : (i & 1) * 49152); }
  static __device__ __forceinline__ uint32_t ds(int i) { return kOut ? tDS : 192u * (i & 1); }
  // entry of a ring of kDeep barriers, and its phase, for chunk i
  static __device__ __forceinline__ int at(int i) { return kOut ? 0 : i & 1; }
  static __device__ __forceinline__ int phase(int i) { return kOut ? i : i >> 1; }
};
static_assert(Layout<false>::W + 2 * 49152 <= kDec, "two wx in a state pass");

struct TcArgs {
  SsmArgs a;
  int seg;
  float *ws, *decays;
  uint64_t wait_ns;
  int stall;  // the MMA warp first waits on a barrier that nothing arrives on (failure-detection tests)
};

// Limit of the drain at the end of a CTA: far beyond what a load or an MMA in flight takes.
constexpr uint64_t kDrainNs = 2000000000ull;

// What a wait needs when it does not succeed at once (shared memory).
struct Misc {
  uint32_t tmem;
  volatile int abort;
  unsigned *status;
  uint64_t wait_ns;
};

// The sleeping part of a wait, one copy for every role (the roles' hot loops together
// should fit the SM's instruction cache: unrolled and inlined to 108 KB, the kernel
// spent a third of its time waiting for instructions, and more on the SMs that share
// a larger cache level with others).  The whole warp calls it and gets the same
// answer, as warp-wide instructions follow.
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, Misc *m) {
  bool ok = false;
  const uint64_t t0 = global_ns();
  for (;;) {
    if ((ok = mbar_try_wait_sleep(bar, parity, 1000000u))) break;
    if (m->abort) break;
    if (global_ns() - t0 > m->wait_ns) {
      m->abort = 1;
      atomicExch(m->status, kDevTimeout);
      break;
    }
  }
  return __all_sync(~0u, ok);
}

// Waits for something that is in flight and ends by itself.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity, unsigned *status) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait_sleep(bar, parity, 1000000u))
    if (global_ns() - t0 > kDrainNs) {
      atomicExch(status, kDevTimeout);
      break;
    }
}

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Misc *m) {
  return __all_sync(~0u, mbar_try_wait(bar, parity)) || wait_slow(bar, parity, m);
}

struct Cta {
  unsigned char *sm;
  uint64_t *bar;
  Misc *m;

  // Phase `k` (0, 1, ...) of barrier b.
  __device__ __forceinline__ bool wait(int b, int k) const { return wait_bar(&bar[b], k & 1, m); }
  // Phase k / 2 of entry k % 2 of a ring.
  __device__ __forceinline__ bool wait2(int b, int k) const { return wait_bar(&bar[b + (k & 1)], (k >> 1) & 1, m); }
  // One arrival for the warp, after what all its lanes did before.
  __device__ __forceinline__ void arrive(int b) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar[b]);
  }
  __device__ __forceinline__ bool wait4(int b, int k) const { return wait_bar(&bar[b + (k & 3)], (k >> 2) & 1, m); }
  __device__ __forceinline__ Decays &dec(int i) const { return *reinterpret_cast<Decays *>(sm + kDec + (i & 3) * sizeof(Decays)); }
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

// 2^v.  The hardware's approximation (2^-22 relative); results below the normal range are 0.
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// log(1 + e^v) = max(v, 0) + log1p(z), z = e^-|v|, by log1p(z) = 2 atanh(z / (2 + z)):
// the argument is at most 1/3, where seven terms of the series s + s^3 / 3 + ... leave 2e-8.
// Four times shorter than log1pf(expf(v)), which the decay warps feel.
__device__ __forceinline__ float softplus_fast(float v) {
  const float z = __expf(-fabsf(v)), s = __fdividef(z, 2.f + z), q = s * s;
  float r = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  r = fmaf(q, r, 1.f / 9.f);
  r = fmaf(q, r, 1.f / 7.f);
  r = fmaf(q, r, 1.f / 5.f);
  r = fmaf(q, r, 1.f / 3.f);
  r = fmaf(q * r, s, s);
  return fmaxf(v, 0.f) + 2.f * r;
}

__device__ __forceinline__ float2 unpack(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// The next bf16 term of v: returns it packed and leaves the exact remainder in v.
__device__ __forceinline__ uint32_t take_term(float2 &v) {
  const uint32_t h = pack_bf16x2(v.x, v.y);
  v = __ffma2_rn(unpack(h), make_float2(-1.f, -1.f), v);
  return h;
}

// An item of at most kShort tokens: token by token in fp32, without the tensor cores.  A
// thread owns one column of NK rows, so state moves in whole lines, and the 16 row groups'
// shares of y are added at the end: the loop over tokens has no barrier.  One wave, N = 128: 5.6 us
// for one token, 0.25 more for each; the chunk form (barriers, tensor memory, three products
// one after another) takes 9.6 us for any number up to 128.
template <int NK>
__device__ __forceinline__ void short_item(const TcArgs &p, const Item &it, unsigned char *sm, int h, int g, int p0) {
  constexpr int N = 16 * NK;
  const SsmArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, c = 32 * (tid >> 5 & 1) + lane, group = tid >> 6;
  const int len = it.end - it.begin;
  float *sB = reinterpret_cast<float *>(sm), *sC = sB + kShort * N, *sx = sC + kShort * N, *part = sx + kShort * PC;
  float *sd = part + kShort * 16 * PC, *sa = sd + kShort;
  static_assert((kShort * (2 * N + 17 * PC + 2)) * 4 <= kSmemBytes - 1024, "shared memory of a short item");
  const bool mine = p0 + c < a.P;
  const int at = group * NK * a.P + p0 + c;  // of this thread's first row
  const int64_t np = (int64_t)N * a.P;
  const float *from = nullptr;
  if (p.seg != 0) from = p.ws + (it.item * a.H + h) * np;
  else if (a.state && it.s.ctx > 0) from = a.state + ((int64_t)it.s.slot * a.H + h) * np;
  float S[NK];
#pragma unroll
  for (int j = 0; j < NK; ++j) S[j] = from && mine ? from[at + j * a.P] : 0.f;
  auto save = [&](float *to) {
#pragma unroll
    for (int j = 0; j < NK; ++j)
      if (mine) to[at + j * a.P] = S[j];
  };
  const int64_t row0 = (int64_t)it.s.start + it.begin;
  auto spread = [](float *to, uint4 v) {  // eight bf16
    const float2 f[4] = {unpack(v.x), unpack(v.y), unpack(v.z), unpack(v.w)};
    *reinterpret_cast<float4 *>(to) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    *reinterpret_cast<float4 *>(to + 4) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  };
  auto eight = [](const void *base, int64_t i) { return *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)base + i); };
  for (int e = tid; e < len * 2 * NK; e += NT) {
    const int t = e / (2 * NK), k = e % (2 * NK) * 8;
    const uint4 b = eight(a.B, (row0 + t) * a.b_stride + g * N + k), q = eight(a.C, (row0 + t) * a.c_stride + g * N + k);
    spread(sB + t * N + k, b);
    spread(sC + t * N + k, q);
  }
  for (int e = tid; e < len * (PC / 8); e += NT) {
    const int t = e / (PC / 8), k = e % (PC / 8) * 8;
    spread(sx + t * PC + k, p0 + k < a.P ? eight(a.x, (row0 + t) * a.x_stride + h * a.P + p0 + k) : make_uint4(0, 0, 0, 0));
  }
  if (tid < len) {
    const float d = time_step<__nv_bfloat16>(a, row0 + tid, h);
    sd[tid] = d;
    sa[tid] = expf(d * a.A[h]);
  }
  __syncthreads();
#pragma unroll 2
  for (int t = 0; t < len; ++t) {
    const float keep = sa[t], dx = sd[t] * sx[t * PC + c], *b = sB + t * N + group * NK, *q = sC + t * N + group * NK;
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      S[j] = fmaf(b[j], dx, keep * S[j]);
      y = fmaf(q[j], S[j], y);
    }
    part[(t * 16 + group) * PC + c] = y;
    if (a.page)
      if (float *to = snapshot(a, it.r, h, (uint32_t)it.s.ctx + (uint32_t)(it.begin + t + 1), p0 == 0 && tid == 0)) save(to);
  }
  if (a.state && it.index == it.count - 1) save(a.state + ((int64_t)it.s.slot * a.H + h) * np);
  __syncthreads();
  const float skip = a.D ? a.D[h] : 0.f;
  for (int e = tid; e < len * (PC / 2); e += NT) {
    const int t = e / (PC / 2), k = e % (PC / 2) * 2;
    if (p0 + k >= a.P) continue;
    const float2 xv = *reinterpret_cast<const float2 *>(sx + t * PC + k);
    float2 y = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) y = __fadd2_rn(y, *reinterpret_cast<const float2 *>(part + (t * 16 + i) * PC + k));
    y = __ffma2_rn(make_float2(skip, skip), xv, y);
    *reinterpret_cast<uint32_t *>((__nv_bfloat16 *)a.y + (row0 + t) * a.y_stride + h * a.P + p0 + k) = pack_bf16x2(y.x, y.y);
  }
}

// kOut: the run that writes y, snapshots and final states; else the state pass,
// which leaves each segment's S~ and decay in the workspace.
// NK: K steps over N (N / 16).
template <bool kOut, int NK>
__global__ void __launch_bounds__(NT, 1)
    ssm_tc_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mb,
                  const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap my, const TcArgs p) {
  using L = Layout<kOut>;
  extern __shared__ __align__(1024) unsigned char smraw[];
  const SsmArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = (a.P + PC - 1) / PC;
  const int p0 = (int)(blockIdx.x % slices) * PC, h = (int)(blockIdx.x / slices % a.H);
  const bool tell = kOut && p0 == 0 && h == 0 && tid == 0;
  unsigned char *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  Item it;
  if (!item_of(a.q, blockIdx.x / (slices * a.H), p.seg, kAlign, tell, reinterpret_cast<int *>(sm + L::W), it)) return;
  if (!kOut && it.index == it.count - 1) return;  // nothing follows it
  const int g = h / (a.H / a.G);
  if (kOut && it.end - it.begin <= kShort) {
    short_item<NK>(p, it, sm, h, g, p0);
    return;
  }
  const Chunks ch(it);
  const int n = ch.n;

  Cta x;
  x.sm = sm;
  x.bar = reinterpret_cast<uint64_t *>(sm + kBarOff);
  x.m = reinterpret_cast<Misc *>(sm + kMisc);
  const uint32_t sbase = smem_u32(sm);
  if (tid == 0) {
    for (int i = 0; i < BARS; ++i) {
      uint32_t count = 1;  // TMA and MMA completions; the others count warps
      if (i == BX_FREE || i == BX_FREE + 1) count = kOut ? 9 : 12;  // the MMAs and the output warps; the token warps
      if (i >= DEC && i < DEC + 4) count = kOut ? 2 : 4;
      if (i >= DEC_FREE && i < DEC_FREE + 4) count = kOut ? 28 : 20;
      if (i == TOTALS) count = kOut ? 2 : 4;
      if (i == W_READY) count = 8;
      if (i == WX_READY || i == WX_READY + 1) count = kOut ? 12 : 20;  // token and state warps
      if (i == YX_READY) count = 16;  // state and output warps
      mbar_init(&x.bar[i], count);
    }
    x.m->abort = 0;
    x.m->status = a.q.status;
    x.m->wait_ns = p.wait_ns;
    mbar_init_fence();
  }
  if (warp == 3) {
    tmem_alloc(&x.m->tmem, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = x.m->tmem;
  const uint32_t tl = tb + ((uint32_t)(32 * (warp & 3)) << 16);  // this warp's lanes
  const int t = 32 * (warp & 3) + lane;  // this thread's row in its role
  const int row_of_seq = it.s.start;

  if (warp == 0) {
    // ======================= producer =======================
    const uint32_t half = NK > 4 ? 32768u : 16384u;  // bytes of a B or C tile that are loaded
    int loads = 0, bloads = 0, cloads = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i & 1, row = row_of_seq + ch.first(i);
      if (i >= 2 && !x.wait2(BX_FREE, i - 2)) break;
      const int f_b = kOut ? F_BX : F_B;
      if (elect_one()) {
        mbar_arrive_expect_tx(&x.bar[F_BX + st], 16384u + (kOut ? half : 0u));
        tma_load_3d(sm + L::X + st * 16384, &mx, &x.bar[F_BX + st], p0, h, row);
      }
      __syncwarp();
      loads = i + 1;
      if (!kOut && i >= 2 && !x.wait2(B_FREE, i - 2)) break;
      if (elect_one()) {
        if (!kOut) mbar_arrive_expect_tx(&x.bar[f_b + st], half);
#pragma unroll
        for (int c = 0; c < 16 * NK; c += 64)
          tma_load_3d(sm + L::B + st * 32768 + c * 256, &mb, &x.bar[f_b + st], c, g, row);
      }
      __syncwarp();
      bloads = i + 1;
      if (kOut) {
        if (i >= 1 && !x.wait(C_FREE, i - 1)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&x.bar[F_C], half);
#pragma unroll
          for (int c = 0; c < 16 * NK; c += 64) tma_load_3d(sm + kC + c * 256, &mc, &x.bar[F_C], c, g, row);
        }
        __syncwarp();
        cloads = i + 1;
      }
      // x of the chunk after the next on its way from HBM (281 us against 285 for 148 heads
      // of 16,384 tokens; B and C are in L2 for the group's other heads: asking for them
      // too cost 284)
      if (i + 2 < n) {
        const int next = row_of_seq + ch.first(i + 2);
        if (elect_one()) tma_prefetch_3d(&mx, p0, h, next);
        __syncwarp();
      }
    }
    // the last loads must land before shared memory is given up (where the other roles gave up they
    // may still be in flight, however few chunks there are)
    for (int k = max(0, loads - 2); k < loads; ++k) drain(&x.bar[F_BX + (k & 1)], (k >> 1) & 1, a.q.status);
    if (!kOut)
      for (int k = max(0, bloads - 2); k < bloads; ++k) drain(&x.bar[F_B + (k & 1)], (k >> 1) & 1, a.q.status);
    if (cloads > 0) drain(&x.bar[F_C], (cloads - 1) & 1, a.q.status);
  } else if (warp == 2) {
    // ======================= MMA issue =======================
    const uint32_t idG = idesc_bf16(128, 128, false, false, false);
    const uint32_t idYx = idesc_bf16(128, 64, false, true, false);
    const uint32_t idDS = idesc_bf16(128, 192, true, true, false);  // the terms of wx side by side
    const uint64_t dS = sdesc_sw128(sbase + kS, 16, 1024);
    const uint64_t dC = sdesc_sw128(sbase + kC, 16, 1024);
    // byte offset of K step k in a [128 x 128] tile, K along its rows
    auto koff = [](int k) { return (uint32_t)((k >> 2) * 16384 + (k & 3) * 32); };
    if (p.stall) x.wait(NEVER, 0);  // (gives up, and every wait after it)
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const uint64_t dB = sdesc_sw128(sbase + L::B + st * 32768, 16, 1024);
      const uint64_t dBt = sdesc_sw128(sbase + L::B + st * 32768, 16384, 1024);
      const uint64_t dX = sdesc_sw128(sbase + L::X + st * 16384, 16, 1024);
      if (!x.wait2(kOut ? F_BX : F_B, i)) break;
      if (kOut) {
        // (the W in G's place is read: YX_READY comes after the outputs of the chunk before)
        // Yx first: it waits longest for what it reads, and C is free for the next chunk once both
        // are done (G first: 2.44 us a chunk against 2.36)
        if (!x.wait(F_C, i) || !x.wait(YX_READY, i)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < NK; ++k) mma_bf16(tb + tYx, sdesc_add(dC, koff(k)), sdesc_add(dS, k * 2048), idYx, k > 0);
#pragma unroll
          for (int k = 0; k < NK; ++k) mma_bf16(tb + tG, sdesc_add(dC, koff(k)), sdesc_add(dB, koff(k)), idG, k > 0);
          mma_commit(&x.bar[G_DONE]);
          mma_commit(&x.bar[C_FREE]);
        }
        __syncwarp();
      }
      if (!x.wait(WX_READY + L::at(i), L::phase(i))) break;
      tc_fence_after();
      const uint64_t dW = sdesc_sw128(sbase + L::w(i), 16384, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16(tb + L::ds(i), sdesc_add(dBt, k * 2048), sdesc_add(dW, k * 2048), idDS, k > 0);
        mma_commit(&x.bar[DS_DONE + L::at(i)]);
        if (!kOut) mma_commit(&x.bar[B_FREE + st]);
      }
      __syncwarp();
      if (kOut) {
        if (!x.wait(W_READY, i)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 16; ++k)  // (rows before the step's block of tokens: no part of W)
            mma_bf16_ts(tb + tYi, tb + tG + 8 * k, sdesc_add(dX, (k >> 1) * 2048), idYx, (1u << (k >> 2)) - 1, k > 0);
          mma_commit(&x.bar[Y_DONE + st]);
          mma_commit(&x.bar[BX_FREE + st]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(&x.bar[DRAIN]);
    __syncwarp();
    drain(&x.bar[DRAIN], 0, a.q.status);
  } else if (kOut && warp >= 4 && warp < 12) {
    // ======================= scores =======================
    const int b = warp & 3, half = (warp - 4) >> 2;  // this warp's rows are block b, its columns a half of each block
    const uint32_t tg = tl + tG + 16 * half;
    const float A2 = a.A[h] * 1.4426950408889634f;
    const int row = lane - 16 * half;  // the diagonal block's columns of this half up to the row
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      if (!x.wait4(DEC, i)) break;
      const Decays &D = x.dec(i);
      const float pre = D.pre[t], rowf = ex2(pre);
      const float2 r2 = make_float2(rowf, rowf);
      // the diagonal block's factors, formed before the scores arrive (131,072 tokens of 16 heads: 838 us
      // formed between them, 824 so): from the half's last column back, with the sum of l from behind
      // the column to the row (0 where the column is behind it)
      float2 e[8];
      float sum = half == 0 && lane >= 16 ? D.mid[t] : 0.f;
#pragma unroll
      for (int j = 6; j >= 0; j -= 2) {
        const float4 d = f4(D.d + 32 * b + 16 * half + 2 * j);
        float f[4];
        const float dd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          f[k] = ex2(sum);
          if (2 * j + k <= row) sum = fmaf(dd[k], A2, sum);
        }
        e[j] = __fmul2_rn(make_float2(d.x, d.y), make_float2(f[0], f[1]));
        e[j + 1] = __fmul2_rn(make_float2(d.z, d.w), make_float2(f[2], f[3]));
      }
      if (!x.wait(G_DONE, i)) break;
      tc_fence_after();
      float v[16];
      uint32_t w[8], rest[8];
      tmem_ld16(tg, v);
#pragma unroll 1
      for (int c = 0; c < b; ++c) {
        const float *col = D.col[b - c - 1] + 32 * c + 16 * half;
        tmem_ld_wait(v);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = f4(col + j);
          float2 lo = __fmul2_rn(make_float2(v[j], v[j + 1]), __fmul2_rn(r2, make_float2(f.x, f.y)));
          float2 hi = __fmul2_rn(make_float2(v[j + 2], v[j + 3]), __fmul2_rn(r2, make_float2(f.z, f.w)));
          w[j / 2] = take_term(lo);
          rest[j / 2] = pack_bf16x2(lo.x, lo.y);
          w[j / 2 + 1] = take_term(hi);
          rest[j / 2 + 1] = pack_bf16x2(hi.x, hi.y);
        }
        tmem_ld16(tg + 32 * (c + 1), v);
        tmem_st16(tg + 32 * c, w, rest);
      }
      tmem_ld_wait(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float2 r = __fmul2_rn(make_float2(v[2 * j], v[2 * j + 1]), e[j]);
        // columns behind the row: zeros, whatever the scores and factors are
        const int behind = 16 * half + 2 * j - lane;
        const uint32_t mask = behind < 0 ? ~0u : behind == 0 ? 0xffffu : 0u;
        w[j] = take_term(r) & mask;
        rest[j] = pack_bf16x2(r.x, r.y) & mask;
      }
      tmem_st16(tg + 32 * b, w, rest);
      tmem_st_wait();
      tc_fence_before();
      x.arrive(W_READY);
      x.arrive(DEC_FREE + (i & 3));
    }
  } else if (kOut ? warp < 4 : warp >= 24 && warp < 28) {
    // ======================= decays =======================
    // two blocks of 32 tokens for each of warps 1 and 3; in a state pass, whose chunks are shorter,
    // one for each of warps 24-27
    constexpr int NB = kOut ? 2 : 1, kAhead = 3;
    const int b0 = kOut ? warp & 2 : warp & 3;  // this warp's blocks: b0 ..
    const float A2 = a.A[h] * 1.4426950408889634f;
    const __nv_bfloat16 *dt = (const __nv_bfloat16 *)a.dt + h;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    // dt of the next chunks, as loaded (a conversion here would wait for the load, which takes about
    // as long as a chunk)
    __nv_bfloat16 raw[NB][kAhead];
    float total = 0.f;
    auto fetch = [&](int i, int to) {
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int tk = 32 * (b0 + k) + lane;
        raw[k][to] = __ushort_as_bfloat16(0);
        if (i < n && tk < ch.count(i)) raw[k][to] = dt[(int64_t)(row_of_seq + ch.first(i) + tk) * a.dt_stride];
      }
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) fetch(j, j);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      float d[NB], up[NB], mid[NB], s[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        d[k] = __bfloat162float(raw[k][0]) + bias;
#pragma unroll
        for (int j = 0; j + 1 < kAhead; ++j) raw[k][j] = raw[k][j + 1];
        if (a.softplus) d[k] = softplus_fast(d[k]);
        if (32 * (b0 + k) + lane >= ch.count(i)) d[k] = 0.f;
        up[k] = s[k] = d[k] * A2;
      }
      fetch(i + kAhead, kAhead - 1);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          if (o == 16) mid[k] = up[k];
          const float u = o < 16 ? __shfl_up_sync(~0u, up[k], o) : __shfl_sync(~0u, up[k], 15);
          const float v = __shfl_down_sync(~0u, s[k], o);
          if (o < 16 ? (lane & 15) >= o : lane >= 16) up[k] += u;
          if (lane + o < 32) s[k] += v;
        }
      }
      if (i >= 4 && !x.wait4(DEC_FREE, i - 4)) break;
      Decays &D = x.dec(i);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float after = __shfl_down_sync(~0u, s[k], 1);
        s[k] = lane < 31 ? after : 0.f;  // behind the token, to its block's end
        if (lane == 31) D.total[b0 + k] = up[k];
        D.d[32 * (b0 + k) + lane] = d[k];
        D.pre[32 * (b0 + k) + lane] = up[k];
        if (kOut) D.mid[32 * (b0 + k) + lane] = mid[k];
      }
      x.arrive(TOTALS);
      if (!x.wait(TOTALS, i)) break;
      const float4 T = f4(D.total);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int tk = 32 * (b0 + k) + lane;
        float sum = s[k];
#pragma unroll
        for (int j = 1; j < 4; ++j) {  // block b0 + k + j
          if (b0 + k + j < 4) {
            if (kOut) D.col[j - 1][tk] = d[k] * ex2(sum);
            const int nb = b0 + k + j;
            sum += nb == 1 ? T.y : nb == 2 ? T.z : T.w;
          }
        }
        D.w[tk] = d[k] * ex2(sum);
      }
      if (b0 == 0 && lane == 0) {
        D.before[0] = 1.f;
        D.before[1] = ex2(T.x);
        D.before[2] = ex2(T.x + T.y);
        D.before[3] = ex2(T.x + T.y + T.z);
        D.all = ex2(T.x + T.y + T.z + T.w);
      }
      total += T.x + T.y + T.z + T.w;
      x.arrive(DEC + (i & 3));
    }
    if (!kOut && b0 == 0 && lane == 0 && p0 == 0) p.decays[it.item * a.H + h] = ex2(total);
  } else if ((warp >= 12 && warp < 16) || (!kOut && warp >= 4 && warp < 12)) {
    // ======================= tokens =======================
    // 16-byte chunks of row t that this thread writes: all, or in a state pass, where the score
    // warps have nothing else to do, two or three of the eight
    const bool first = warp >= 12;
    const int k0 = first ? 0 : 2 + 3 * ((warp - 4) >> 2), k1 = kOut ? 8 : first ? 2 : k0 + 3;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const bool live = t < ch.count(i);
      if (!x.wait4(DEC, i)) break;
      const float w = x.dec(i).w[t];
      x.arrive(DEC_FREE + (i & 3));
      const float2 f2 = make_float2(w, w);
      if (!x.wait2(F_BX, i)) break;
      unsigned char *xt = sm + L::X + (i & 1) * 16384, *wx = sm + L::w(i);
      auto load = [&](int k) {
        return live ? *reinterpret_cast<const uint4 *>(xt + sw128_chunk(t, k)) : make_uint4(0, 0, 0, 0);
      };
      uint4 v = load(k0);
      if (!kOut && first && ch.count(i) < Q && !x.wait2(F_B, i)) break;
      if (first && !live) {  // rows behind the last token: x and B sum over tokens, so they must be zeros
        const uint4 z = make_uint4(0, 0, 0, 0);
        unsigned char *bt = sm + L::B + (i & 1) * 32768;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = sw128_chunk(t, k);
          if (kOut) *reinterpret_cast<uint4 *>(xt + at) = z;
          *reinterpret_cast<uint4 *>(bt + at) = z;
          *reinterpret_cast<uint4 *>(bt + 16384 + at) = z;
        }
      }
      // the wx that was in its place is read
      if (i >= L::kDeep && !x.wait(DS_DONE + L::at(i), L::phase(i - L::kDeep))) break;
#pragma unroll 2
      for (int k = k0; k < k1; ++k) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        v = load((k + 1) & 7);
        uint32_t q0[4], q1[4], q2[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 y = __fmul2_rn(f2, unpack(u[j]));
          q0[j] = take_term(y);
          q1[j] = take_term(y);
          q2[j] = pack_bf16x2(y.x, y.y);
        }
        unsigned char *to = wx + sw128_chunk(t, k);
        *reinterpret_cast<uint4 *>(to) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
        *reinterpret_cast<uint4 *>(to + 16384) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
        *reinterpret_cast<uint4 *>(to + 32768) = make_uint4(q2[0], q2[1], q2[2], q2[3]);
      }
      fence_proxy_async_smem();
      x.arrive(WX_READY + L::at(i));
      if (!kOut) x.arrive(BX_FREE + (i & 1));
    }
  } else if (warp >= 16 && warp < 24) {
    // ======================= state =======================
    const int half = (warp - 16) >> 2;
    const int cols = t < a.N ? min(32, a.P - p0 - 32 * half) : 0;  // columns that exist
    const int at = t * a.P + p0 + 32 * half;
    float2 S[16];
    const float *from = nullptr;
    if (kOut) {
      const int64_t np = (int64_t)a.N * a.P;
      if (p.seg != 0) from = p.ws + (it.item * a.H + h) * np + at;
      else if (a.state && it.s.ctx > 0) from = a.state + ((int64_t)it.s.slot * a.H + h) * np + at;
    }
    auto save = [&](float *to) {
#pragma unroll
      for (int j = 0; j < 16; j += 2)
        if (2 * j < cols) *reinterpret_cast<float4 *>(to + at + 2 * j) = make_float4(S[j].x, S[j].y, S[j + 1].x, S[j + 1].y);
    };
    bool done = false;
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float4 v = from && 2 * j < cols ? f4(from + 2 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[j] = make_float2(v.x, v.y);
      S[j + 1] = make_float2(v.z, v.w);
    }
    auto copy = [&]() {  // the bf16 copy that the next chunk's outputs read
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pack_bf16x2(S[4 * k + j].x, S[4 * k + j].y);
        *reinterpret_cast<uint4 *>(sm + kS + sw128_chunk(t, 4 * half + k)) = make_uint4(v[0], v[1], v[2], v[3]);
      }
      fence_proxy_async_smem();
      x.arrive(YX_READY);
    };
    if (kOut) copy();
    for (int k = 0; k < L::kDeep; ++k) x.arrive(WX_READY + k);  // no dS before the first
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      if (!x.wait4(DEC, i)) break;
      const float keep = x.dec(i).all;
      x.arrive(DEC_FREE + (i & 3));
      if (!x.wait(DS_DONE + L::at(i), L::phase(i))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        float q0[8], q1[8];
        tmem_ld8(tl + L::ds(i) + 128 + 32 * half + c, q0);
        tmem_ld8(tl + L::ds(i) + 64 + 32 * half + c, q1);
        tmem_ld_wait(q0);
        tmem_ld_touch(q1);
        float2 sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sum[j] = __fadd2_rn(make_float2(q0[2 * j], q0[2 * j + 1]), make_float2(q1[2 * j], q1[2 * j + 1]));
        tmem_ld8(tl + L::ds(i) + 32 * half + c, q0);
        tmem_ld_wait(q0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          S[c / 2 + j] = __ffma2_rn(make_float2(keep, keep), S[c / 2 + j], __fadd2_rn(make_float2(q0[2 * j], q0[2 * j + 1]), sum[j]));
      }
      tc_fence_before();
      x.arrive(WX_READY + L::at(i + L::kDeep));
      if (kOut && i + 1 < n) copy();  // (DS_DONE: the products that read the copy before are done)
      if (kOut && a.page) {
        if (float *to = snapshot(a, it.r, h, (uint32_t)it.s.ctx + (uint32_t)(ch.first(i) + ch.count(i)), p0 == 0 && t == 0))
          save(to);
      }
      done = i + 1 == n;
    }
    if (done) {
      if (!kOut) save(p.ws + (it.item * a.H + h) * ((int64_t)a.N * a.P));
      else if (a.state && it.index == it.count - 1) save(a.state + ((int64_t)it.s.slot * a.H + h) * ((int64_t)a.N * a.P));
    }
  } else if (kOut && warp >= 24) {
    // ======================= outputs =======================
    const int half = (warp - 24) >> 2;
    const int col0 = p0 + 32 * half;
    const float skip = a.D ? a.D[h] : 0.f;
    const float2 skip2 = make_float2(skip, skip);
    unsigned char *ytile = sm + kY + (warp - 24) * 2048;  // this warp's 32 rows of 32 columns (64-byte swizzle)
    x.arrive(YX_READY);  // no Yi and Yx before the first
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int count = ch.count(i), first = row_of_seq + ch.first(i);
      if (!x.wait4(DEC, i)) break;
      const float f = x.dec(i).before[warp & 3] * ex2(x.dec(i).pre[t]);
      x.arrive(DEC_FREE + (i & 3));
      const float2 f2 = make_float2(f, f);
      bulk_wait_read_all();  // (the lane that issued the store before)
      __syncwarp();
      if (!x.wait2(F_BX, i) || !x.wait2(Y_DONE, i)) break;
      tc_fence_after();
      const unsigned char *xt = sm + kX + (i & 1) * 16384;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float yi[16], yx[16];
        tmem_ld16(tl + tYi + 32 * half + 16 * c, yi);
        tmem_ld16(tl + tYx + 32 * half + 16 * c, yx);
        tmem_ld_wait(yi);
        tmem_ld_touch(yx);
        if (c == 1) {
          tc_fence_before();
          x.arrive(YX_READY);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 v = *reinterpret_cast<const uint4 *>(xt + sw128_chunk(t, 4 * half + 2 * c + k));
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 8 * k + 2 * j;
            const float2 s = __ffma2_rn(f2, make_float2(yx[e], yx[e + 1]), make_float2(yi[e], yi[e + 1]));
            const float2 r = __ffma2_rn(skip2, unpack(u[j]), s);
            o[j] = pack_bf16x2(r.x, r.y);
          }
          *reinterpret_cast<uint4 *>(ytile + sw64_chunk(lane, 2 * c + k)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      x.arrive(BX_FREE + (i & 1));
      if (col0 >= a.P) continue;
      if (count == Q) {
        fence_proxy_async_smem();
        __syncwarp();
        tma_store_3d_warp(&my, ytile, col0, h, first + 32 * (warp & 3));
        bulk_commit_warp();
      } else if (t < count) {  // a ragged chunk: only its rows
        __nv_bfloat16 *yrow = (__nv_bfloat16 *)a.y + (int64_t)(first + t) * a.y_stride + h * a.P + col0;
#pragma unroll 1
        for (int k = 0; k < 4 && col0 + 8 * k < a.P; ++k)
          *reinterpret_cast<uint4 *>(yrow + 8 * k) = *reinterpret_cast<const uint4 *>(ytile + sw64_chunk(lane, k));
      }
    }
    bulk_wait_read_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) tmem_dealloc(tb, kCols);
}

}  // namespace

bool ssm_tc_fits(const SsmArgs &a) {
  // (a tensor map's strides are below 2^40 bytes)
  auto row16 = [](const void *p, int64_t stride) {
    return ((uintptr_t)p & 15) == 0 && stride % 8 == 0 && stride < (int64_t(1) << 39);
  };
  return a.bf16 && row16(a.x, a.x_stride) && row16(a.B, a.b_stride) && row16(a.C, a.c_stride) && row16(a.y, a.y_stride);
}

namespace {

template <int NK>
cudaError_t launch_nk(const CUtensorMap &mx, const CUtensorMap &mb, const CUtensorMap &mc, const CUtensorMap &my,
                      const TcArgs &p, unsigned grid, cudaStream_t st) {
  constexpr cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(ssm_tc_kernel<true, NK>, smem, kSmemBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(ssm_tc_kernel<false, NK>, smem, kSmemBytes);
  if (e != cudaSuccess) return e;
  if (p.seg) {
    ssm_tc_kernel<false, NK><<<grid, NT, kSmemBytes, st>>>(mx, mb, mc, my, p);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_segment_states(p.a, p.seg, kAlign, st);
    if (e != cudaSuccess) return e;
  }
  ssm_tc_kernel<true, NK><<<grid, NT, kSmemBytes, st>>>(mx, mb, mc, my, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_tc(const SsmArgs &a, int seg, cudaStream_t st) {
  CUtensorMap mx, mb, mc, my;
  const uint64_t rows = (uint64_t)a.q.rows;
  if (!encode_tmap_bf16_rows(&mx, a.x, a.P, a.H, rows, a.x_stride, PC, Q) ||
      !encode_tmap_bf16_rows(&mb, a.B, a.N, a.G, rows, a.b_stride, 64, Q) ||
      !encode_tmap_bf16_rows(&mc, a.C, a.N, a.G, rows, a.c_stride, 64, Q) ||
      !encode_tmap_bf16_rows(&my, a.y, a.P, a.H, rows, a.y_stride, 32, 32))
    return cudaErrorInvalidValue;
  const int64_t items = scan_items(a.q.R, a.q.rows, seg);
  TcArgs p;
  p.a = a;
  p.seg = seg;
  p.ws = seg ? seg_states(a) : nullptr;
  p.decays = seg ? seg_decays(a, items) : nullptr;
  p.wait_ns = debug_wait_ns();
  p.stall = debug_stall();
  const unsigned grid = (unsigned)(items * a.H * ((a.P + PC - 1) / PC));
  switch (a.N) {
    case 16: return launch_nk<1>(mx, mb, mc, my, p, grid, st);
    case 32: return launch_nk<2>(mx, mb, mc, my, p, grid, st);
    case 64: return launch_nk<4>(mx, mb, mc, my, p, grid, st);
    default: return launch_nk<8>(mx, mb, mc, my, p, grid, st);
  }
}

}  // namespace kda
