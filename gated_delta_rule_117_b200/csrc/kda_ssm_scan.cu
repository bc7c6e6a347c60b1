// Selective state space scan of packed prompts (include/kda.h, kda_ssm_scan):
// the CUDA-core kernel (fp32, rows of any alignment, many sequences of a few
// tokens), and the segment bookkeeping that every scan kernel shares.
//
//     S_t = exp(d_t A) S_{t-1} + d_t B_t x_t^T,    y_t = S_t^T C_t + D x_t.
//
// Where the sequences and heads alone do not fill the machine, sequences are
// cut into segments.  The recurrence is linear in the entering state and its
// transition is one number, so a segment maps S to S~ + a S, a = exp(A sum d):
// a first pass computes (S~, a) of every segment but the last of its sequence
// from a zero state, a second walks down the segments and leaves each one's
// entering state, and the last pass runs all segments from those.  No block
// waits for another one.
//
// The CUDA-core kernel: one CTA a (segment, head).  Four neighbouring lanes
// share a state column, each holding a quarter of its N rows in registers, so
// the token loop has no barrier: a token costs 3 N / 4 operations a thread and
// two shuffles.  Tokens are staged in shared memory TB at a time.  Its chain of
// dependent tokens bounds it, not bytes.
#include <math.h>

#include "kda_ssm_seg.cuh"

namespace kda {
namespace {

constexpr int TB = kSimtAlign;  // tokens staged at a time

template <int N, int P, typename T, bool kOut>
__global__ void __launch_bounds__(4 * P) ssm_scan_kernel(SsmArgs a, int seg, float *ws, float *decays) {
  constexpr int NT = 4 * P, J = N / 16;  // a thread holds J blocks of 4 rows
  __shared__ __align__(16) float sB[TB][N];
  __shared__ __align__(16) float sC[kOut ? TB : 1][N];
  __shared__ float sx[TB][P], sy[kOut ? TB : 1][P], sd[TB], sa[TB];
  const int tid = threadIdx.x, p = tid >> 2, quarter = tid & 3;
  const int h = blockIdx.x % a.H;
  const bool tell = kOut && h == 0 && tid == 0;
  Item it;
  __shared__ int scratch[kMaxRanked + 1];
  if (!item_of(a.q, blockIdx.x / a.H, seg, kSimtAlign, tell, scratch, it)) return;
  if (!kOut && it.index == it.count - 1) return;  // nothing follows it
  const int g = h / (a.H / a.G);
  float2 S[J][2];  // rows 16 j + 4 quarter + 0 .. 3
  const int64_t at = (it.item * a.H + h) * (N * P);
  const float *from = nullptr;
  if (kOut) {
    if (seg != 0) from = ws + at;
    else if (a.state && it.s.ctx > 0) from = a.state + ((int64_t)it.s.slot * a.H + h) * (N * P);
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = 16 * j + 4 * quarter + 2 * i;
      S[j][i] = from ? make_float2(from[n * P + p], from[(n + 1) * P + p]) : make_float2(0.f, 0.f);
    }
  auto save = [&](float *to) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = 16 * j + 4 * quarter + 2 * i;
        to[n * P + p] = S[j][i].x;
        to[(n + 1) * P + p] = S[j][i].y;
      }
  };
  const float A = a.A[h], skip = a.D ? a.D[h] : 0.f;
  float total = 0.f;  // sum of d (thread 0)

  // blocks of TB tokens that end at multiples of TB of the position, so snapshots fall on their ends
  for (int t0 = it.begin, nt; t0 < it.end; t0 += nt) {
    nt = min(TB - (int)(((uint32_t)it.s.ctx + (uint32_t)t0) % TB), it.end - t0);
    const int64_t row0 = (int64_t)it.s.start + t0;
    __syncthreads();
    for (int e = tid; e < nt * N; e += NT) {
      const int t = e / N, n = e % N;
      sB[t][n] = as_float(((const T *)a.B)[(row0 + t) * a.b_stride + g * N + n]);
      if (kOut) sC[t][n] = as_float(((const T *)a.C)[(row0 + t) * a.c_stride + g * N + n]);
    }
    for (int e = tid; e < nt * P; e += NT) {
      const int t = e / P, c = e % P;
      sx[t][c] = as_float(((const T *)a.x)[(row0 + t) * a.x_stride + h * P + c]);
    }
    if (tid < nt) {
      const float d = time_step<T>(a, row0 + tid, h);
      sd[tid] = d;
      sa[tid] = expf(d * A);
    }
    __syncthreads();
    if (!kOut && tid == 0)
      for (int t = 0; t < nt; ++t) total += sd[t];
#pragma unroll 4
    for (int t = 0; t < nt; ++t) {
      const float xv = sx[t][p], dx = sd[t] * xv;
      const float2 keep2 = make_float2(sa[t], sa[t]), dx2 = make_float2(dx, dx);
      float2 y0 = make_float2(0.f, 0.f), y1 = y0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float4 b = *reinterpret_cast<const float4 *>(&sB[t][16 * j + 4 * quarter]);
        S[j][0] = __ffma2_rn(make_float2(b.x, b.y), dx2, __fmul2_rn(keep2, S[j][0]));
        S[j][1] = __ffma2_rn(make_float2(b.z, b.w), dx2, __fmul2_rn(keep2, S[j][1]));
        if (kOut) {
          const float4 c = *reinterpret_cast<const float4 *>(&sC[t][16 * j + 4 * quarter]);
          y0 = __ffma2_rn(make_float2(c.x, c.y), S[j][0], y0);
          y1 = __ffma2_rn(make_float2(c.z, c.w), S[j][1], y1);
        }
      }
      if (kOut) {
        float y = (y0.x + y0.y) + (y1.x + y1.y);
        y += __shfl_xor_sync(~0u, y, 1);
        y += __shfl_xor_sync(~0u, y, 2);
        if (quarter == 0) sy[t][p] = fmaf(skip, xv, y);
      }
    }
    if (kOut) {
      if (float *to = snapshot(a, it.r, h, (uint32_t)it.s.ctx + (uint32_t)(t0 + nt), tell)) save(to);
      __syncthreads();
      for (int e = tid; e < nt * P; e += NT) {
        const int t = e / P, c = e % P;
        ((T *)a.y)[(row0 + t) * a.y_stride + h * P + c] = as_type<T>(sy[t][c]);
      }
    }
  }
  if (!kOut) {
    save(ws + at);
    if (tid == 0) decays[it.item * a.H + h] = expf(A * total);
  } else if (a.state && it.index == it.count - 1) {
    save(a.state + ((int64_t)it.s.slot * a.H + h) * (N * P));
  }
}

// Entering states of every segment of a sequence, in place of what the segments
// add to a zero state: S(0) from the pool, S(i + 1) = a_i S(i) + S~_i.
constexpr int kJoinThreads = 128, kAhead = 8;
__global__ void __launch_bounds__(kJoinThreads) segment_states_kernel(SsmArgs a, int seg, int align, float4 *ws,
                                                                      const float *decays) {
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int n4 = a.N * a.P / 4, e = blockIdx.y * kJoinThreads + threadIdx.x;
  const Seq s = seq_of(a.q, r, false);
  const int len = s.end - s.start;
  if (e >= n4 || !s.ok || len == 0) return;
  const int64_t base = seg_base(a.q, r, seg);
  const int count = (int)(((int64_t)(s.ctx % align) + len + seg - 1) / seg);
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.state && s.ctx > 0)
    S = reinterpret_cast<const float4 *>(a.state)[((int64_t)s.slot * a.H + h) * n4 + e];
  float4 *w = ws + (base * a.H + h) * n4 + e;
  const float *dec = decays + base * a.H + h;
  const int64_t step = (int64_t)a.H * n4;
  // kAhead segments' loads in flight together: only the sums depend on one another
  // (16 heads of 128 x 128, 10 segments: 37 us one by one)
  for (int i0 = 0; i0 < count; i0 += kAhead) {
    float4 add[kAhead];
    float keep[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool some = i0 + k + 1 < count;  // (the last segment's is neither computed nor needed)
      add[k] = some ? w[(i0 + k) * step] : make_float4(0.f, 0.f, 0.f, 0.f);
      keep[k] = some ? dec[(int64_t)(i0 + k) * a.H] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i0 + k < count) w[(i0 + k) * step] = S;
      S.x = fmaf(keep[k], S.x, add[k].x);
      S.y = fmaf(keep[k], S.y, add[k].y);
      S.z = fmaf(keep[k], S.z, add[k].z);
      S.w = fmaf(keep[k], S.w, add[k].w);
    }
  }
}

// Segment lengths: those whose blocks cost least, or 0 for whole sequences.  Whole sequences
// run as long as the longest of them; packed ones (whose lengths the host does not see) are
// taken to hold one of twice the mean.  Tried are the mean over 2 to 16 and, from there on, over
// counts an eighth apart: at most 7 % above the cost of the best length by the same model, over
// 4,000 random shapes, for a tenth of the 255 trials (the size query of 4,096 tokens of 32 heads
// 9 to 15 us on the host with all of them, 1.7 so), which a call pays twice.
inline int next_count(int k) { return k < 16 ? k + 1 : k + k / 8; }

// The CUDA-core kernel, in tokens of a block that runs alone (0.16 us for a state of 16 x 16,
// 0.47 for 128 x 64, 0.69 for 128 x 128).  A pass takes its longest block and 16 tokens to begin and
// end, or, where blocks share an SM, their tokens (and 7 each for the state's way in and
// out) over its speed: that of 6.2 lone blocks of 16 x 16, of 0.92 of 128 x 128, a power of N P
// between them.  A state pass takes 0.6 of an output pass, the two more launches 20
// tokens, the join one a segment.  2 x 300 tokens of 4 heads of 128 x 64: 138 us whole, 96 in
// segments of 128, 29 in segments of 16; 4,000 tokens of 4 heads of 64 x 64: 1,092 whole, 66 by 128,
// 55 by 64, 72 by 16.
int simt_segment(int R, int rows, int H, int N, int P, bool packed) {
  packed = packed && R > 1;
  const double mean = (double)rows / R, most = packed ? fmin((double)rows, 2 * mean) : mean;
  const double speed = 6.2 * pow(256.0 / (N * P), 0.46);
  auto pass = [&](double items, double len, double longest) {
    return fmax(longest + 16, ceil(items * H / 148) * (len + 7) / speed);
  };
  double best = pass(R, mean, most);
  int seg = 0;
  if (1.6 * ((double)rows * H / 148) / speed >= best) return 0;  // (no cost below is lower)
  for (int k = 2, len = 0; k <= 256 && len != kSimtAlign; k = next_count(k)) {
    len = ((int)(mean / k) / kSimtAlign + 1) * kSimtAlign;
    const double items = packed ? rows / (double)len + 0.5 * R : (double)R * ceil(mean / len);
    const double cost = 1.6 * pass(items, len, len) + 20 + most / len;
    if (cost < best && scan_items(R, rows, len) * H <= INT32_MAX) {  // (blocks of a launch)
      best = cost;
      seg = len;
    }
  }
  return seg;
}

// The tensor-core kernel, in tokens of an output pass: one block an SM; a chunk takes 2.45 us,
// 1.2 us in the state pass; a block's beginning and end 6 us, the two launches about 10 us.
// 131,072 tokens of 16 heads of 128 in 9 segments: state pass 279 us, join 7 us, outputs 529 us.
int tc_segment(int R, int rows, int H, int P, bool packed) {
  packed = packed && R > 1;
  const double blocks = (double)H * ((P + 63) / 64) / 148, begin = 2.5 * kAlign;
  const double mean = (double)rows / R, most = packed ? fmin((double)rows, 2 * mean) : mean;
  // blocks of unequal length fill the machine as they come: the waves' total, or the longest block
  double best = packed ? fmax(most, (mean + begin) * R * blocks) : ceil(R * blocks) * (mean + begin);
  int seg = 0;
  if (1.49 * rows * blocks >= best) return 0;
  for (int k = 2; k <= 64; k = next_count(k)) {
    const int len = (int)((mean / k + kAlign - 1) / kAlign) * kAlign;
    if (len < 4 * kAlign) break;
    const double items = packed ? rows / (double)len + 0.5 * R : (double)R * ceil(mean / len);
    const double cost = ceil(items * blocks) * (len + begin) * 1.49 + 4 * kAlign;
    if (cost < best) {
      best = cost;
      seg = len;
    }
  }
  return seg;
}

template <int N, int P, typename T>
cudaError_t launch_t(const SsmArgs &a, int seg, cudaStream_t st) {
  const int64_t items = scan_items(a.q.R, a.q.rows, seg);
  float *ws = seg ? seg_states(a) : nullptr, *dec = seg ? seg_decays(a, items) : nullptr;
  const unsigned grid = (unsigned)(items * a.H);
  if (seg) {
    ssm_scan_kernel<N, P, T, false><<<grid, 4 * P, 0, st>>>(a, seg, ws, dec);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_segment_states(a, seg, kSimtAlign, st);
    if (e != cudaSuccess) return e;
  }
  ssm_scan_kernel<N, P, T, true><<<grid, 4 * P, 0, st>>>(a, seg, ws, dec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_segment_states(const SsmArgs &a, int seg, int align, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.q.R * a.H), (a.N * a.P / 4 + kJoinThreads - 1) / kJoinThreads);
  segment_states_kernel<<<grid, kJoinThreads, 0, st>>>(a, seg, align, (float4 *)seg_states(a),
                                                       seg_decays(a, scan_items(a.q.R, a.q.rows, seg)));
  return cudaGetLastError();
}

// The segments of every form that a call of these sizes may take (packed or not, rows that
// fit the tensor-core kernel or not), and workspace enough for any of them.
ScanPlan plan_ssm_scan(int R, int rows, int H, int N, int P, int bf16) {
  ScanPlan p = {};
  for (int packed = 0; packed < 2; ++packed)
    for (int tc = 0; tc <= (bf16 ? 1 : 0); ++tc) {
      int &seg = p.seg[tc][packed];
      if (packed && R == 1) {
        seg = p.seg[tc][0];
        continue;
      }
      seg = tc ? tc_segment(R, rows, H, P, packed) : simt_segment(R, rows, H, N, P, packed);
      const size_t need = seg ? seg_workspace(scan_items(R, rows, seg), H, N, P) : 0;
      p.workspace = need > p.workspace ? need : p.workspace;
    }
  return p;
}

// Whether the CUDA-core kernel should take a call that fits both: many sequences of a few
// tokens, as its blocks are small and several share an SM.  In us, fitted to 1 to 256
// sequences of 1 to 64 tokens, 3 to 32 heads of 16 x 16 to 128 x 128: a state's way in and out
// and a token's work over the machine, the chain of the longest sequence's tokens, and waves of
// the other kernel's blocks.  256 x 32 heads of 128 x 64, one token each: 151 us against 322;
// 16 tokens: 447 against 532; 64 tokens: 1,384 against 501.  The longest of a packed call is
// not known: what is lost if one sequence has all the rows must not exceed what is gained
// if it has twice the mean.
static bool tokens_are_few(const SsmArgs &a) {
  const double states = (double)a.q.R * a.H, np = (double)a.N * a.P, mean = (double)a.q.rows / a.q.R;
  auto simt = [&](double longest) {
    return 4 + states * np * (2.2e-6 + 0.3e-6 * mean) + longest * (0.12 + 0.0028 * a.N * (a.P > 64 ? 1.5 : 1));
  };
  const double waves = fmax(1, states * ((a.P + 63) / 64) / 148);
  const double tc = waves * (mean <= kShort ? 3.8 + 0.015 * a.N + mean * (0.12 + 0.001 * a.N)
                                            : 6 + 0.02 * a.N + 2.45 * floor((mean - 1) / kAlign));
  return a.q.cu ? simt(fmin(a.q.rows, 2 * mean)) * simt(a.q.rows) < tc * tc : simt(mean) < tc;
}

cudaError_t launch_ssm_scan(const SsmArgs &a, const ScanPlan &plan, cudaStream_t st) {
  const bool packed = a.q.cu != nullptr;
  if (ssm_tc_fits(a) && !tokens_are_few(a)) return launch_ssm_tc(a, plan.seg[1][packed], st);
  const int seg = plan.seg[0][packed];
#define KDA_SSM_CASE(NN, PP)    \
  if (a.N == NN && a.P == PP)   \
    return a.bf16 ? launch_t<NN, PP, __nv_bfloat16>(a, seg, st) : launch_t<NN, PP, float>(a, seg, st);
#define KDA_SSM_ROW(NN) KDA_SSM_CASE(NN, 16) KDA_SSM_CASE(NN, 32) KDA_SSM_CASE(NN, 64) KDA_SSM_CASE(NN, 128)
  KDA_SSM_ROW(16) KDA_SSM_ROW(32) KDA_SSM_ROW(64) KDA_SSM_ROW(128)
#undef KDA_SSM_ROW
#undef KDA_SSM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace kda
