// Selective state space step for single tokens (include/kda.h, kda_ssm_step).
//
// Per (sequence, head):  a = exp(d A),  S_ij <- a S_ij + (d B_i) x_j,
//                        y_j = sum_i C_i S_ij + D x_j,   d = softplus(dt + dt_bias).
//
// Bytes bound it: the fp32 state is read and written once (8 N P bytes), the
// token's own inputs are a few hundred bytes.  As in the decode step of the
// delta rule, one CTA owns one (sequence, head), a thread holds float4 pieces
// of rows in registers, every state load is issued before the first use, and
// the column sums over N are joined through shared memory.
#include "kda_serve.cuh"

namespace kda {
namespace {

template <int N, int P>
struct StepShape {
  static constexpr int TPR = P / 4;                           // threads per state row (float4 each)
  static constexpr int RP = (N < 256 / TPR) ? N : 256 / TPR;  // row groups
  static constexpr int NT = TPR * RP;
  static constexpr int RPT = N / RP;  // rows per thread
};

template <int N, int P, typename T>
__global__ void __launch_bounds__(StepShape<N, P>::NT) ssm_step_kernel(SsmArgs a) {
  using Sh = StepShape<N, P>;
  constexpr int TPR = Sh::TPR, RP = Sh::RP, NT = Sh::NT, RPT = Sh::RPT;
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int tid = threadIdx.x, tx = tid % TPR, ty = tid / TPR;
  const int slot = a.q.slots ? a.q.slots[r] : r;
  if (slot < 0) return;
  if (slot >= a.q.n_slots) {
    if (h == 0 && tid == 0) record_bounds(a.q.status);
    return;
  }
  float4 *S4 = reinterpret_cast<float4 *>(a.state + ((int64_t)slot * a.H + h) * (N * P));
  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = S4[(ty + i * RP) * TPR + tx];

  __shared__ float sB[N], sC[N];
  __shared__ float4 red[RP][TPR];
  const int g = h / (a.H / a.G);
  const T *B = (const T *)a.B + r * a.b_stride + g * N, *C = (const T *)a.C + r * a.c_stride + g * N;
  for (int i = tid; i < N; i += NT) {
    sB[i] = as_float(B[i]);
    sC[i] = as_float(C[i]);
  }
  float d = as_float(((const T *)a.dt)[r * a.dt_stride + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f);
  if (a.softplus) d = softplus(d);
  const float keep = expf(d * a.A[h]), skip = a.D ? a.D[h] : 0.f;
  const T *x = (const T *)a.x + r * a.x_stride + h * P + 4 * tx;
  const float4 xv = make_float4(as_float(x[0]), as_float(x[1]), as_float(x[2]), as_float(x[3]));
  const float4 dx = make_float4(d * xv.x, d * xv.y, d * xv.z, d * xv.w);
  __syncthreads();

  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int n = ty + i * RP;
    const float b = sB[n], c = sC[n];
    float4 v = s[i];
    v.x = fmaf(b, dx.x, keep * v.x);
    v.y = fmaf(b, dx.y, keep * v.y);
    v.z = fmaf(b, dx.z, keep * v.z);
    v.w = fmaf(b, dx.w, keep * v.w);
    S4[n * TPR + tx] = v;
    y.x = fmaf(c, v.x, y.x);
    y.y = fmaf(c, v.y, y.y);
    y.z = fmaf(c, v.z, y.z);
    y.w = fmaf(c, v.w, y.w);
  }
  red[ty][tx] = y;
  __syncthreads();
  if (ty == 0) {
#pragma unroll
    for (int i = 1; i < RP; ++i) {
      const float4 t = red[i][tx];
      y.x += t.x; y.y += t.y; y.z += t.z; y.w += t.w;
    }
    T *o = (T *)a.y + r * a.y_stride + h * P + 4 * tx;
    o[0] = as_type<T>(fmaf(skip, xv.x, y.x));
    o[1] = as_type<T>(fmaf(skip, xv.y, y.y));
    o[2] = as_type<T>(fmaf(skip, xv.z, y.z));
    o[3] = as_type<T>(fmaf(skip, xv.w, y.w));
  }
}

template <int N, int P>
cudaError_t launch_np(const SsmArgs &a, cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.q.R * a.H);
  if (a.bf16)
    ssm_step_kernel<N, P, __nv_bfloat16><<<grid, StepShape<N, P>::NT, 0, st>>>(a);
  else
    ssm_step_kernel<N, P, float><<<grid, StepShape<N, P>::NT, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_step(const SsmArgs &a, cudaStream_t st) {
#define KDA_SSM_CASE(NN, PP) \
  if (a.N == NN && a.P == PP) return launch_np<NN, PP>(a, st);
#define KDA_SSM_ROW(NN) KDA_SSM_CASE(NN, 16) KDA_SSM_CASE(NN, 32) KDA_SSM_CASE(NN, 64) KDA_SSM_CASE(NN, 128)
  KDA_SSM_ROW(16) KDA_SSM_ROW(32) KDA_SSM_ROW(64) KDA_SSM_ROW(128)
#undef KDA_SSM_ROW
#undef KDA_SSM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace kda
