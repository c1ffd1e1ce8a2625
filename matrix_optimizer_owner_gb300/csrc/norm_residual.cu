// Residual addition and layer or RMS norm in one pass, with 8-bit results, forward.
//
// Per row of n elements (RMS norm: mu = 0 and no bias):
//     h = x + r,  mu = sum(h) / n,  s = 1 / sqrt(sum((h - mu)^2) / n + eps),  y = (h - mu) s w + b
// h and y leave in the caller's type, in 8 bits (1 x 128 groups), or both, each rounded once from the
// fp32 value.  Bound by memory (8192 x 4096 bf16, RMS, h in bf16 and y in 8 bits: 41 us, 5.7 TB/s; 46 with the
// weight in fp32).  Short rows fill neither it nor the issue slots (16384 x 768, layer norm, h in 8 bits too:
// 23 us, 4.3 TB/s, 37 instructions a value at 60 % of the slots): a warp loads nothing while it reduces its row.
// A row lies in registers over a warp (up to 768 elements) or a block, so neighbouring threads hold a group of
// 128 and its largest value takes a few shuffles.
#include "norm_residual.cuh"

namespace mfsdp {
namespace {

// ---------------------------------------------------------------- forward
// Rows of up to 768 elements: a warp each, eight consecutive elements a lane, K times.  FULL: rows of K
// times 256 elements, every one for 16-byte accesses: no test per chunk remains.
template <typename T, int K, bool FULL>
__global__ void __launch_bounds__(32 * kNormWarps, sizeof(T) == 2 ? 4 : 2)
    norm_residual_forward_kernel(const __grid_constant__ NrArgs p) {
  constexpr int TPR = 32;
  float* red = nullptr;                   // (a warp's sums need no shared memory)
  pdl_launch();
  const int t = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  pdl_wait();
  if (row >= p.rows) return;              // whole warps
  const int n = (int)p.cols;              // (rows this long fit registers)
  const int vec = FULL ? 1 : p.vec, pvec = FULL ? 1 : p.pvec;
  auto col = [&](int k) { return (k * TPR + t) * 8; };
  auto left_of = [&](int k) { return FULL ? 8 : n - col(k); };
  Pack8<T> xp[K], rp[K];
  const T* xr = static_cast<const T*>(p.x) + row * p.ld_x;
#pragma unroll
  for (int k = 0; k < K; ++k) load_chunk(xp[k], xr, col(k), left_of(k), vec);
  if (p.res) {
    const T* rr = static_cast<const T*>(p.res) + row * p.ld_res;
#pragma unroll
    for (int k = 0; k < K; ++k) load_chunk(rp[k], rr, col(k), left_of(k), vec);
  }
  float v[K][8], s = 0.f, zero = 0.f;
  int turn = 0;
#pragma unroll
  for (int k = 0; k < K; ++k) xp[k].get(v[k]);
  if (p.res)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float r[8];
      rp[k].get(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] += r[j];
    }
  // what does not wait for the row's sums
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (p.h) store_part(static_cast<T*>(p.h) + row * p.ld_h, col(k), left_of(k), vec, v[k]);
  float mu = 0.f;
  if (p.layer) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[k][j];
    row_sum2<TPR>(s, zero, red, turn);
    mu = s * p.inv_n;
  }
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = v[k][j] - mu;
    zero_past(d, left_of(k));
#pragma unroll
    for (int j = 0; j < 8; ++j) q = fmaf(d[j], d[j], q);
  }
  zero = 0.f;
  row_sum2<TPR>(q, zero, red, turn);
  const float r = 1.f / sqrtf(fmaf(q, p.inv_n, p.eps));
  if (t == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = r;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = col(k), left = left_of(k);
    float w[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = (v[k][j] - mu) * r;
    if (p.w) {
      load_param8(p.w, p.wbf16, pvec, c, left, 1.f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= w[j];
    }
    if (p.b) {
      load_param8(p.b, p.wbf16, pvec, c, left, 0.f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] += w[j];
    }
    if (p.y) store_part(static_cast<T*>(p.y) + row * p.ld_y, c, left, vec, y);
    zero_past(y, left);
    store_groups(p, row, c, left, y, v[k]);
  }
}

// Rows of more than 768 elements: a block each, sixteen consecutive elements a thread.  Eight lanes hold
// a group of 128, and what a row costs apart from its values falls on twice as many of them (8192 rows
// of 4096: 49 us with eight a thread).
template <typename T, int TPR, bool LAYER>
__global__ void __launch_bounds__(TPR, sizeof(T) == 2 ? 1024 / TPR : 512 / TPR)
    norm_residual_forward_wide_kernel(const __grid_constant__ NrArgs p) {
  __shared__ float red[4 * (TPR / 32)];
  pdl_launch();
  Sixteen at;
  at.row = blockIdx.x;
  at.has = true;
  at.col = threadIdx.x * 16;
  at.group = threadIdx.x >> 3;
  at.width = max(0, min(16, (int)p.cols - (int)threadIdx.x * 16));
  const int left = at.width;
  pdl_wait();
  Pack8<T> raw[2], add[2];
  load_sixteen(raw, static_cast<const T*>(p.x) + at.row * p.ld_x + at.col, left, p.vec);
  if (p.res) load_sixteen(add, static_cast<const T*>(p.res) + at.row * p.ld_res + at.col, left, p.vec);
  float v[16], s = 0.f, zero = 0.f;
  int turn = 0;
  get_sixteen(raw, v);
  if (p.res) {
    float r[16];
    get_sixteen(add, r);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += r[j];
  }
  if (p.h) store_sixteen(static_cast<T*>(p.h) + at.row * p.ld_h + at.col, left, p.vec, v);
  float mu = 0.f;
  if (LAYER) {
#pragma unroll
    for (int j = 0; j < 16; ++j) s += v[j];
    row_sum2<TPR>(s, zero, red, turn);
    mu = s * p.inv_n;
  }
  float q = 0.f;
  if (!LAYER || left == 16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) q = fmaf(v[j] - mu, v[j] - mu, q);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < left) q = fmaf(v[j] - mu, v[j] - mu, q);
  }
  zero = 0.f;
  row_sum2<TPR>(q, zero, red, turn);
  const float r = 1.f / sqrtf(fmaf(q, p.inv_n, p.eps));
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[at.row] = mu;
    if (p.rstd) p.rstd[at.row] = r;
  }
  float y[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = (int)threadIdx.x * 16 + 8 * h, here = left - 8 * h;
    float u[8], w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = (v[8 * h + j] - mu) * r;
    if (p.w) {
      load_param8(p.w, p.wbf16, p.pvec, c, here, 1.f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] *= w[j];
    }
    if (LAYER && p.b) {
      load_param8(p.b, p.wbf16, p.pvec, c, here, 0.f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += w[j];
    }
    zero_past(u, here);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[8 * h + j] = u[j];
  }
  if (p.y) store_sixteen(static_cast<T*>(p.y) + at.row * p.ld_y + at.col, left, p.vec, y);
  if (p.y8.q) quantize_sixteen(at, y, eighth_warp_max(scale_part(largest(y))), p.y8);
  if (p.h8.q) quantize_sixteen(at, v, eighth_warp_max(scale_part(largest(v))), p.h8);
}

// Rows too long for registers: three passes over the row (the second and third hit the L2).
template <typename T>
__global__ void __launch_bounds__(1024)
    norm_residual_forward_long_kernel(const __grid_constant__ NrArgs p) {
  __shared__ float red[4 * 32];
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.x, n = p.cols;
  const T* xr = static_cast<const T*>(p.x) + row * p.ld_x;
  const T* rr = p.res ? static_cast<const T*>(p.res) + row * p.ld_res : nullptr;
  auto left_of = [&](int64_t c) { return (int)max((int64_t)0, min((int64_t)8, n - c)); };
  auto sum = [&](int64_t c, float (&v)[8]) {
    Pack8<T> a;
    load_chunk(a, xr, c, left_of(c), p.vec);
    a.get(v);
    if (!rr) return;
    float r[8];
    load_chunk(a, rr, c, left_of(c), p.vec);
    a.get(r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  };
  int turn = 0;
  float mu = 0.f, zero = 0.f, v[8];
  if (p.layer) {
    float s = 0.f;
    for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
      sum(c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
    row_sum2<1024>(s, zero, red, turn);
    mu = s * p.inv_n;
  }
  float q = 0.f;
  for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
    sum(c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = c + j < n ? v[j] - mu : 0.f;
      q = fmaf(d, d, q);
    }
  }
  zero = 0.f;
  row_sum2<1024>(q, zero, red, turn);
  const float r = 1.f / sqrtf(fmaf(q, p.inv_n, p.eps));
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = r;
  }
  for (int64_t c0 = 0; c0 < n; c0 += 8192) {        // whole warps: groups are reduced by shuffles
    const int64_t c = c0 + threadIdx.x * 8;
    float y[8];
    sum(c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float w = p.w && c + j < n ? load_param(p.w, p.wbf16, c + j) : 1.f;
      const float b = p.b && c + j < n ? load_param(p.b, p.wbf16, c + j) : 0.f;
      y[j] = fmaf((v[j] - mu) * r, w, b);
    }
    const int left = left_of(c);
    if (p.h) store_part(static_cast<T*>(p.h) + row * p.ld_h, c, left, p.vec, v);
    if (p.y) store_part(static_cast<T*>(p.y) + row * p.ld_y, c, left, p.vec, y);
    zero_past(y, left);
    store_groups(p, row, c, left, y, v);
  }
}

// ---------------------------------------------------------------- dispatch
template <typename T, int TPR>
cudaError_t launch_wide(const NrArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)a.rows), block(TPR);
  return a.layer ? launch_pdl(norm_residual_forward_wide_kernel<T, TPR, true>, grid, block, 0, st, a)
                 : launch_pdl(norm_residual_forward_wide_kernel<T, TPR, false>, grid, block, 0, st, a);
}
template <typename T, int K>
cudaError_t launch_warps(const NrArgs& a, dim3 grid, dim3 block, cudaStream_t st) {
  return a.cols == K * 256 && a.vec && a.pvec
             ? launch_pdl(norm_residual_forward_kernel<T, K, true>, grid, block, 0, st, a)
             : launch_pdl(norm_residual_forward_kernel<T, K, false>, grid, block, 0, st, a);
}
template <typename T>
cudaError_t launch_forward(const NrArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.rows + kNormWarps - 1) / kNormWarps)), block(32 * kNormWarps);
  if (a.cols <= 256) return launch_warps<T, 1>(a, grid, block, st);
  if (a.cols <= 512) return launch_warps<T, 2>(a, grid, block, st);
  // (768 in 64 threads of sixteen leaves a quarter of them idle: 29 -> 36 us for 16384 rows; 1024 fills
  // them: 46 -> 32)
  if (a.cols <= 768) return launch_warps<T, 3>(a, grid, block, st);
  if (a.cols <= 1024) return launch_wide<T, 64>(a, st);
  if (a.cols <= 2048) return launch_wide<T, 128>(a, st);
  if (a.cols <= 4096) return launch_wide<T, 256>(a, st);
  if (a.cols <= kRegRowMax) return launch_wide<T, 512>(a, st);
  return launch_pdl(norm_residual_forward_long_kernel<T>, dim3((unsigned)a.rows), dim3(1024), 0, st, a);
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" int mfsdp_norm_residual_forward(
    int32_t kind, int64_t rows, int64_t cols, int32_t dtype, int32_t param_dtype, const void* x,
    int64_t ld_x, const void* residual, int64_t ld_residual, const void* weight, const void* bias,
    float eps, void* h, int64_t ld_h, void* y, int64_t ld_y, const mfsdp_fp8_matrix* y8,
    const mfsdp_fp8_matrix* h8, float* mean, float* rstd, void* stream) {
  int chk = check_shape(kind, rows, cols, dtype, param_dtype);
  if (chk != MFSDP_OK) return chk;
  if (!(eps >= 0.f) || (kind == MFSDP_NORM_RMS && (bias || mean))) return MFSDP_EINVAL;
  if (!y && !y8) return MFSDP_EINVAL;
  if (y8 && (chk = check_fp8(*y8, rows, cols, MFSDP_GROUPS_ROW)) != MFSDP_OK) return chk;
  if (h8 && (chk = check_fp8(*h8, rows, cols, MFSDP_GROUPS_ROW)) != MFSDP_OK) return chk;
  if (rows == 0) return MFSDP_OK;
  if (!x || ld_x < cols || (residual && ld_residual < cols) || (h && ld_h < cols) ||
      (y && ld_y < cols))
    return MFSDP_EINVAL;
  const size_t es = dtype_bytes(dtype), ps = dtype_bytes(param_dtype);
  if (!aligned_to(x, es) || !aligned_to(residual, es) || !aligned_to(h, es) || !aligned_to(y, es) ||
      !aligned_to(weight, ps) || !aligned_to(bias, ps) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return MFSDP_EALIGN;
  if (!distinct({h, y, data_of(h8), bytes_of(h8), data_of(y8), bytes_of(y8), mean, rstd})) return MFSDP_EINVAL;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  NrArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.x = x;
  a.ld_x = ld_x;
  a.res = residual;
  a.ld_res = ld_residual;
  a.w = weight;
  a.b = bias;
  a.h = h;
  a.ld_h = ld_h;
  a.y = y;
  a.ld_y = ld_y;
  a.y8 = ref_of(y8);
  a.h8 = ref_of(h8);
  a.mean = mean;
  a.rstd = rstd;
  a.eps = eps;
  a.inv_n = (float)(1.0 / (double)cols);
  a.layer = kind == MFSDP_NORM_LAYER;
  a.wbf16 = param_dtype == MFSDP_DTYPE_BF16;
  a.pvec = cols % 8 == 0 && aligned_to(weight, 16) && aligned_to(bias, 16);
  a.vec = vector_rows(x, ld_x, dtype) && (!residual || vector_rows(residual, ld_residual, dtype)) &&
          (!h || vector_rows(h, ld_h, dtype)) && (!y || vector_rows(y, ld_y, dtype));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == MFSDP_DTYPE_BF16;
  const cudaError_t e = bf ? launch_forward<bf16_t>(a, st) : launch_forward<float>(a, st);
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}
