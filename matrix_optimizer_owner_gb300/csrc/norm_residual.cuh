// What the two directions of the norm with a residual share: their arguments, and a thread's chunk of
// a row with its edges.
#pragma once

#include "fp8.cuh"
#include "norm_rows.cuh"

namespace mfsdp {
namespace {

struct NrArgs {
  int64_t rows, cols;
  const void *x, *res, *w, *b;    // forward inputs
  void *h, *y;                    // nullable
  int64_t ld_x, ld_res, ld_h, ld_y;
  Fp8Ref h8, y8;                  // q == nullptr: not wanted (backward: h8 instead of h_in)
  float *mean, *rstd;             // nullable
  const void *dy, *dres, *h_in;   // backward inputs; dres nullable
  int64_t ld_dy, ld_dres, ld_dx;
  void* dx;
  const float *mean_in, *rstd_in;
  float* partials;                // [blocks][2][cols]
  float eps, inv_n;
  int layer, wbf16, has_dw, has_db;
  int pvec, vec;                  // 16-byte accesses of the parameters; of every row
};

// Eight consecutive elements of a row from c on, `left` of them (1 to 8; 0 or less: none) in it and
// zeros past its end.
template <typename T>
__device__ __forceinline__ void load_chunk(Pack8<T>& p, const T* row, int64_t c, int left, int vec) {
  if (left >= 8 && vec) {
    p.load(row + c);
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < left ? to_f32(row[c + j]) : 0.f;
    p.set(v);
  }
}
template <typename T>
__device__ __forceinline__ void store_part(T* row, int64_t c, int left, int vec, const float (&v)[8]) {
  if (left >= 8 && vec) {
    Pack8<T> p;
    p.set(v);
    p.store(row + c);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) row[c + j] = from_f32<T>(v[j]);
  }
}
__device__ __forceinline__ void zero_past(float (&v)[8], int left) {
  if (left >= 8) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < left ? v[j] : 0.f;
}
// The parameters of a thread's chunk, `fill` where there are none.
__device__ __forceinline__ void load_param8(const void* src, int is_bf16, int pvec, int64_t c, int left,
                                            float fill, float (&v)[8]) {
  if (src && pvec && left >= 8) {
    if (is_bf16) {
      Pack8<bf16_t> q;
      q.load(static_cast<const bf16_t*>(src) + c);
      q.get(v);
    } else {
      Pack8<float> q;
      q.load(static_cast<const float*>(src) + c);
      q.get(v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = src && j < left ? load_param(src, is_bf16, c + j) : fill;
  }
}
// A thread's parts of a row's 1 x 128 groups of y and of h (zeros past the row's end); 16 neighbouring
// threads call.
__device__ __forceinline__ void store_groups(const NrArgs& p, int64_t row, int64_t c, int left,
                                             float (&y)[8], float (&h)[8]) {
  if (!p.y8.q && !p.h8.q) return;
  uint32_t sy, sh;
  group_scales(y, h, p.y8.e5m2, p.h8.e5m2, sy, sh);
  if (left <= 0) return;
  if (p.y8.q) {
    store_fp8(p.y8.q + row * p.y8.ld + c, pack_fp8(y, inverse_scale(sy), p.y8.e5m2), left);
    if ((threadIdx.x & 15) == 0) p.y8.s[row * p.y8.ld_s + c / kGroup] = (uint8_t)sy;
  }
  if (p.h8.q) {
    store_fp8(p.h8.q + row * p.h8.ld + c, pack_fp8(h, inverse_scale(sh), p.h8.e5m2), left);
    if ((threadIdx.x & 15) == 0) p.h8.s[row * p.h8.ld_s + c / kGroup] = (uint8_t)sh;
  }
}

}  // namespace
}  // namespace mfsdp
