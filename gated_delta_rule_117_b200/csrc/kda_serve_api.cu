// C-ABI layer of the packed-request operators: argument validation and
// dispatch.  The interface and its contract are documented in include/kda.h.
#include <math.h>

#include "kda.h"
#include "kda_check.cuh"
#include "kda_serve.cuh"

namespace {

using namespace kda::check;

constexpr int kMaxMapRequests = 16384;
constexpr int kMaxRows = INT32_MAX - 4096;      // rows and what is added to them stay 32-bit
constexpr int kMaxChannels = 1 << 24;  // a block for each 512 of them in a grid's second dimension
constexpr int kMaxHeads = 1 << 24;     // times 128 columns, an element's place in its row stays 32-bit

size_t elem(kda_dtype_t t) { return t == KDA_DTYPE_BF16 ? 2 : 4; }

// Bytes between the first and the last element of a token-major array.
size_t extent(int64_t rows, int64_t stride, int64_t width, size_t e) {
  return rows > 0 ? (size_t)((rows - 1) * stride + width) * e : 0;
}

// Whether a row stride holds `width` elements and the array's extent an int64.
bool stride_fits(int64_t rows, int64_t stride, int64_t width) {
  return stride >= width && stride <= (int64_t(1) << 48) / (rows > 0 ? rows : 1);
}

// Whether any of `outs` overlaps another of them or one of `ins`.
template <int NO, int NI>
bool aliased(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return true;
  }
  return false;
}

bool aligned4(const void *p) { return aligned_to(p, 4); }

// Sizes and pool of a packed call.  `tokens`: rows of the token-major arrays.
kda_status_t check_requests(int R, int rows, const int *cu, const int *ctx, const int *slots, const void *state,
                            int n_slots) {
  if (R < 0 || rows < 0 || n_slots < 0) return KDA_ERR_INVALID_ARG;
  if (rows > kMaxRows || (!cu && R > 0 && rows % R != 0)) return KDA_ERR_SHAPE;
  if ((state != nullptr) != (n_slots > 0)) return KDA_ERR_INVALID_ARG;
  if (state && !slots && n_slots < R) return KDA_ERR_SHAPE;
  if (!aligned4(cu) || !aligned4(ctx) || !aligned4(slots)) return KDA_ERR_ALIGNMENT;
  return KDA_OK;
}

kda_status_t check_conv(int rows, const void *x, int64_t x_stride, const void *w, const void *bias, const void *state, void *y,
                        int64_t y_stride, int C, int K, int head_dim, kda_dtype_t dtype, int flags, float eps) {
  if (C < 0) return KDA_ERR_INVALID_ARG;
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_DTYPE;
  if (K < 2 || K > 4 || C > kMaxChannels) return KDA_ERR_SHAPE;
  if (flags & ~(KDA_CONV_SILU | KDA_CONV_L2NORM | KDA_CONV_HEAD_MAJOR)) return KDA_ERR_INVALID_ARG;
  const bool heads = (flags & (KDA_CONV_L2NORM | KDA_CONV_HEAD_MAJOR)) != 0;
  if (heads && (!supported_d(head_dim) || C % head_dim != 0)) return KDA_ERR_SHAPE;
  if ((flags & KDA_CONV_L2NORM) && (!(eps >= 0.f) || !isfinite(eps))) return KDA_ERR_INVALID_ARG;
  if (!stride_fits(rows, x_stride, C) || (!(flags & KDA_CONV_HEAD_MAJOR) && !stride_fits(rows, y_stride, C)))
    return KDA_ERR_SHAPE;
  const size_t e = elem(dtype);
  const void *ptrs[] = {x, w, bias, state, y};
  for (const void *p : ptrs)
    if (!aligned_to(p, e)) return KDA_ERR_ALIGNMENT;
  return KDA_OK;
}

void set_shape(kda::ConvArgs &a, int C, int K, int head_dim) {
  a.C = C;
  a.K = K;
  a.d = supported_d(head_dim) ? head_dim : 0;
  a.log2_d = a.d == 16 ? 4 : a.d == 32 ? 5 : a.d == 64 ? 6 : 7;
  a.heads = a.d ? C / a.d : 0;
}

// Whether a thread's four channels can be moved at once everywhere.
bool conv_vectors(const kda::ConvArgs &a) {
  const size_t bytes = a.bf16 ? 8 : 16;
  auto fits = [&](const void *p) { return aligned_to(p, bytes); };
  return a.C % 4 == 0 && a.x_stride % 4 == 0 && (a.head_major || a.y_stride % 4 == 0) && fits(a.x) && fits(a.y) &&
         fits(a.state) && fits(a.w) && fits(a.bias);
}

}  // namespace

extern "C" {

kda_status_t kda_block_map(const int *len, const int *ctx, const int *free_pages, int n_free, int *block_table,
                           int table_stride, int page_size, int *cu, int64_t *token_slots, int *pages_used, int R,
                           int rows, kda_stream_t stream) {
  if (R < 0 || rows < 0 || n_free < 0 || table_stride < 0 || page_size < 1) return KDA_ERR_INVALID_ARG;
  if (R > kMaxMapRequests || rows > kMaxRows) return KDA_ERR_SHAPE;
  if (!cu || !pages_used || (R > 0 && !len) || (n_free > 0 && !free_pages) ||
      (R > 0 && table_stride > 0 && !block_table) || (rows > 0 && !token_slots))
    return KDA_ERR_INVALID_ARG;
  const void *ptrs[] = {len, ctx, free_pages, block_table, cu, pages_used};
  for (const void *p : ptrs)
    if (!aligned4(p)) return KDA_ERR_ALIGNMENT;
  if (!aligned_to(token_slots, 8)) return KDA_ERR_ALIGNMENT;
  const size_t r4 = (size_t)R * 4;
  const Range outs[] = {range_of(block_table, r4 * table_stride), range_of(cu, r4 + 4),
                        range_of(token_slots, (size_t)rows * 8), range_of(pages_used, 4)};
  const Range ins[] = {range_of(len, r4), range_of(ctx, ctx ? r4 : 0), range_of(free_pages, (size_t)n_free * 4)};
  if (aliased(outs, ins)) return KDA_ERR_ALIAS;
  const kda_status_t st = check_device();
  if (st != KDA_OK) return st;
  kda::MapArgs a;
  a.len = len; a.ctx = ctx; a.free_pages = free_pages; a.n_free = n_free;
  a.table = block_table; a.table_stride = table_stride; a.page = page_size;
  a.cu = cu; a.token_slots = token_slots; a.used = pages_used;
  a.R = R; a.rows = rows;
  return kda::launch_block_map(a, (cudaStream_t)stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_short_conv(const void *x, int64_t x_stride, const void *w, const void *bias, void *state, int n_slots,
                            const int *slots, const int *ctx, const int *cu, void *y, int64_t y_stride, int R, int rows,
                            int C, int K, int head_dim, kda_dtype_t dtype, int flags, float eps, kda_stream_t stream) {
  kda_status_t st = check_requests(R, rows, cu, ctx, slots, state, n_slots);
  if (st != KDA_OK) return st;
  st = check_conv(rows, x, x_stride, w, bias, state, y, y_stride, C, K, head_dim, dtype, flags, eps);
  if (st != KDA_OK) return st;
  const bool head_major = (flags & KDA_CONV_HEAD_MAJOR) != 0;
  if (head_major && cu) return KDA_ERR_INVALID_ARG;
  if (R == 0 || rows == 0 || C == 0) return KDA_OK;
  if (!x || !w || !y) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(dtype), r4 = (size_t)R * 4;
  const Range outs[] = {range_of(y, head_major ? (size_t)rows * C * e : extent(rows, y_stride, C, e)),
                        range_of(state, (size_t)n_slots * (K - 1) * C * e)};
  const Range ins[] = {range_of(x, extent(rows, x_stride, C, e)), range_of(w, (size_t)C * K * e),
                       range_of(bias, bias ? C * e : 0),          range_of(slots, slots ? r4 : 0),
                       range_of(ctx, ctx ? r4 : 0),               range_of(cu, cu ? r4 + 4 : 0)};
  if (aliased(outs, ins)) return KDA_ERR_ALIAS;
  st = check_device();
  if (st != KDA_OK) return st;
  kda::ConvArgs a;
  a.q = kda::Requests{cu, ctx, slots, R, rows, rows / R, n_slots, kda::device_status_ptr()};
  if (!a.q.status) return KDA_ERR_CUDA;
  a.x = x; a.w = w; a.bias = bias; a.state = state; a.y = y;
  a.x_stride = x_stride; a.y_stride = y_stride;
  set_shape(a, C, K, head_dim);
  a.bf16 = dtype == KDA_DTYPE_BF16;
  a.silu = (flags & KDA_CONV_SILU) != 0;
  a.norm = (flags & KDA_CONV_L2NORM) != 0;
  a.head_major = head_major;
  a.eps = eps;
  a.vec = conv_vectors(a);
  return kda::launch_short_conv(a, (cudaStream_t)stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_short_conv_step(const void *x, int64_t x_stride, const void *w, const void *bias, void *state,
                                 int n_slots, const int *slots, void *y, int64_t y_stride, int R, int C, int K,
                                 int head_dim, kda_dtype_t dtype, int flags, float eps, kda_stream_t stream) {
  kda_status_t st = check_requests(R, R, nullptr, nullptr, slots, state, n_slots);
  if (st != KDA_OK) return st;
  st = check_conv(R, x, x_stride, w, bias, state, y, y_stride, C, K, head_dim, dtype, flags, eps);
  if (st != KDA_OK) return st;
  if (!stride_fits(R, y_stride, C)) return KDA_ERR_SHAPE;
  if (R == 0 || C == 0) return KDA_OK;
  if (!x || !w || !y || !state) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(dtype);
  const Range outs[] = {range_of(y, extent(R, y_stride, C, e)), range_of(state, (size_t)n_slots * (K - 1) * C * e)};
  const Range ins[] = {range_of(x, extent(R, x_stride, C, e)), range_of(w, (size_t)C * K * e),
                       range_of(bias, bias ? C * e : 0), range_of(slots, slots ? (size_t)R * 4 : 0)};
  if (aliased(outs, ins)) return KDA_ERR_ALIAS;
  st = check_device();
  if (st != KDA_OK) return st;
  kda::ConvArgs a;
  a.q = kda::Requests{nullptr, nullptr, slots, R, R, 1, n_slots, kda::device_status_ptr()};
  if (!a.q.status) return KDA_ERR_CUDA;
  a.x = x; a.w = w; a.bias = bias; a.state = state; a.y = y;
  a.x_stride = x_stride; a.y_stride = y_stride;
  set_shape(a, C, K, head_dim);
  a.bf16 = dtype == KDA_DTYPE_BF16;
  a.silu = (flags & KDA_CONV_SILU) != 0;
  a.norm = (flags & KDA_CONV_L2NORM) != 0;
  a.head_major = 0;
  a.eps = eps;
  a.vec = conv_vectors(a);
  return kda::launch_short_conv_step(a, (cudaStream_t)stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"

namespace {

kda_status_t check_ssm_sizes(int H, int G, int N, int P, kda_dtype_t dtype) {
  if (H < 0 || G < 0) return KDA_ERR_INVALID_ARG;
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_DTYPE;
  if (!supported_d(N) || !supported_d(P) || H > kMaxHeads) return KDA_ERR_SHAPE;
  if (H > 0 && (G == 0 || H % G != 0)) return KDA_ERR_SHAPE;
  return KDA_OK;
}

// The blocks of a launch, one for each (segment, head, slice of P), with segments of 128 tokens:
// the tensor-core kernel's are longer, and shorter ones of the CUDA-core kernel are taken only
// where their blocks fit as well.
bool scan_grid_fits(int R, int rows, int H) {
  return ((int64_t)rows / 128 + 2 * (int64_t)R) <= INT32_MAX / (2 * (int64_t)(H > 0 ? H : 1));
}

// The arguments that the scan and the step share.  `rows`: of the token-major arrays.
kda_status_t check_ssm(const kda::SsmArgs &a, int rows, size_t workspace, kda_dtype_t dtype) {
  const int64_t HP = (int64_t)a.H * a.P, GN = (int64_t)a.G * a.N;
  if (!stride_fits(rows, a.x_stride, HP) || !stride_fits(rows, a.y_stride, HP) || !stride_fits(rows, a.dt_stride, a.H) ||
      !stride_fits(rows, a.b_stride, GN) || !stride_fits(rows, a.c_stride, GN))
    return KDA_ERR_SHAPE;
  if (!a.x || !a.dt || !a.A || !a.B || !a.C || !a.y) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(dtype);
  const void *ptrs[] = {a.x, a.dt, a.B, a.C, a.y};
  for (const void *p : ptrs)
    if (!aligned_to(p, e)) return KDA_ERR_ALIGNMENT;
  const void *ptrs4[] = {a.A, a.D, a.dt_bias, a.table};
  for (const void *p : ptrs4)
    if (!aligned4(p)) return KDA_ERR_ALIGNMENT;
  if (!aligned16(a.state) || !aligned16(a.pages) || !aligned16(a.workspace)) return KDA_ERR_ALIGNMENT;
  const size_t h4 = (size_t)a.H * 4, r4 = (size_t)a.q.R * 4, st = (size_t)a.H * a.N * a.P * 4;
  const Range outs[] = {range_of(a.y, extent(rows, a.y_stride, HP, e)), range_of(a.state, a.q.n_slots * st),
                        range_of(a.pages, a.page ? a.n_pages * st : 0), range_of(a.workspace, workspace)};
  const Range ins[] = {range_of(a.x, extent(rows, a.x_stride, HP, e)),
                       range_of(a.dt, extent(rows, a.dt_stride, a.H, e)),
                       range_of(a.B, extent(rows, a.b_stride, GN, e)),
                       range_of(a.C, extent(rows, a.c_stride, GN, e)),
                       range_of(a.A, h4),
                       range_of(a.D, a.D ? h4 : 0),
                       range_of(a.dt_bias, a.dt_bias ? h4 : 0),
                       range_of(a.q.slots, a.q.slots ? r4 : 0),
                       range_of(a.q.ctx, a.q.ctx ? r4 : 0),
                       range_of(a.q.cu, a.q.cu ? r4 + 4 : 0),
                       range_of(a.table, a.page ? r4 * a.table_stride : 0)};
  if (aliased(outs, ins)) return KDA_ERR_ALIAS;
  return check_device();
}

}  // namespace

extern "C" {

size_t kda_ssm_scan_workspace_size(int R, int rows, int H, int G, int N, int P, kda_dtype_t dtype) {
  if (R < 0 || rows < 0 || check_ssm_sizes(H, G, N, P, dtype) != KDA_OK) return (size_t)-1;
  if (R == 0 || rows == 0 || H == 0) return 0;
  if (rows > kMaxRows || !scan_grid_fits(R, rows, H)) return (size_t)-1;
  return kda::plan_ssm_scan(R, rows, H, N, P, dtype == KDA_DTYPE_BF16).workspace;
}

kda_status_t kda_ssm_scan(const void *x, int64_t x_stride, const void *dt, int64_t dt_stride, const float *A,
                          const void *Bm, int64_t b_stride, const void *Cm, int64_t c_stride, const float *D,
                          const float *dt_bias, int softplus, float *state, int n_slots, const int *slots,
                          const int *ctx, const int *cu, const int *block_table, int table_stride, float *pages,
                          int n_pages, int page_size, void *y, int64_t y_stride, int R, int rows, int H, int G, int N,
                          int P, kda_dtype_t dtype, void *workspace, size_t workspace_bytes, kda_stream_t stream) {
  kda_status_t st = check_requests(R, rows, cu, ctx, slots, state, n_slots);
  if (st != KDA_OK) return st;
  st = check_ssm_sizes(H, G, N, P, dtype);
  if (st != KDA_OK) return st;
  if (page_size < 0 || page_size % 128 != 0) return KDA_ERR_INVALID_ARG;
  if (page_size > 0 && (table_stride < 0 || n_pages < 0)) return KDA_ERR_INVALID_ARG;
  if (R == 0 || rows == 0 || H == 0) return KDA_OK;
  if (!scan_grid_fits(R, rows, H)) return KDA_ERR_SHAPE;
  const bool snap = page_size > 0 && table_stride > 0 && n_pages > 0;
  if (snap && (!block_table || !pages)) return KDA_ERR_INVALID_ARG;
  const kda::ScanPlan plan = kda::plan_ssm_scan(R, rows, H, N, P, dtype == KDA_DTYPE_BF16);
  const size_t need = plan.workspace;
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  kda::SsmArgs a;
  a.q = kda::Requests{cu, ctx, slots, R, rows, rows / R, n_slots, nullptr};
  a.x = x; a.dt = dt; a.A = A; a.B = Bm; a.C = Cm; a.D = D; a.dt_bias = dt_bias;
  a.x_stride = x_stride; a.dt_stride = dt_stride; a.b_stride = b_stride; a.c_stride = c_stride;
  a.y = y; a.y_stride = y_stride;
  a.state = state;
  a.H = H; a.G = G; a.N = N; a.P = P;
  a.bf16 = dtype == KDA_DTYPE_BF16;
  a.softplus = softplus != 0;
  a.table = snap ? block_table : nullptr;
  a.table_stride = snap ? table_stride : 0;
  a.pages = snap ? pages : nullptr;
  a.n_pages = snap ? n_pages : 0;
  a.page = snap ? page_size : 0;
  a.workspace = need > 0 ? workspace : nullptr;
  st = check_ssm(a, rows, need, dtype);
  if (st != KDA_OK) return st;
  a.q.status = kda::device_status_ptr();
  if (!a.q.status) return KDA_ERR_CUDA;
  return kda::launch_ssm_scan(a, plan, (cudaStream_t)stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_ssm_step(const void *x, int64_t x_stride, const void *dt, int64_t dt_stride, const float *A,
                          const void *Bm, int64_t b_stride, const void *Cm, int64_t c_stride, const float *D,
                          const float *dt_bias, int softplus, float *state, int n_slots, const int *slots, void *y,
                          int64_t y_stride, int R, int H, int G, int N, int P, kda_dtype_t dtype, kda_stream_t stream) {
  kda_status_t st = check_requests(R, R, nullptr, nullptr, slots, state, n_slots);
  if (st != KDA_OK) return st;
  st = check_ssm_sizes(H, G, N, P, dtype);
  if (st != KDA_OK) return st;
  if (R == 0 || H == 0) return KDA_OK;
  if ((int64_t)R * H > INT32_MAX) return KDA_ERR_SHAPE;
  if (!state) return KDA_ERR_INVALID_ARG;
  kda::SsmArgs a;
  a.q = kda::Requests{nullptr, nullptr, slots, R, R, 1, n_slots, nullptr};
  a.x = x; a.dt = dt; a.A = A; a.B = Bm; a.C = Cm; a.D = D; a.dt_bias = dt_bias;
  a.x_stride = x_stride; a.dt_stride = dt_stride; a.b_stride = b_stride; a.c_stride = c_stride;
  a.y = y; a.y_stride = y_stride;
  a.state = state;
  a.H = H; a.G = G; a.N = N; a.P = P;
  a.bf16 = dtype == KDA_DTYPE_BF16;
  a.softplus = softplus != 0;
  a.table = nullptr; a.table_stride = 0; a.pages = nullptr; a.n_pages = 0; a.page = 0;
  a.workspace = nullptr;
  st = check_ssm(a, R, 0, dtype);
  if (st != KDA_OK) return st;
  a.q.status = kda::device_status_ptr();
  if (!a.q.status) return KDA_ERR_CUDA;
  return kda::launch_ssm_step(a, (cudaStream_t)stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
