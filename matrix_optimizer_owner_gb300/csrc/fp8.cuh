// 8-bit floating-point matrices with a power-of-two scale per group of 128: the scale's rule, the
// conversions, and the 128 x 128 tiles in which the kernels produce them.
//
// A value is q 2^(s - 127), q e4m3 or e5m2 and s the group's byte (e8m0).  s is the least one that
// brings the group's largest finite magnitude within the type's range (1.75 2^8 or 1.75 2^15), so
// scaling is exact, nothing saturates and the one rounding is q's (to nearest even, relative 2^-4
// or 2^-3; below the least normal value a fixed step).  A power of two costs up to one binade of
// range against a scale of amax / 448 and nothing in precision above the subnormals, and it is what
// the tensor cores apply themselves.  Infinities and NaN become NaN of their own element and take no
// part in the scale.
#pragma once

#include <cuda_fp8.h>

#include <cfloat>

#include "elem.cuh"
#include "mfsdp.h"

namespace mfsdp {

struct Fp8Ref {            // an 8-bit matrix as the kernels see it; q == nullptr: not wanted
  uint8_t* q;
  uint8_t* s;
  int64_t ld, ld_s;
  int32_t e5m2;
  int32_t groups;
};

constexpr int kGroup = 128;

// ---- scales
__device__ __forceinline__ uint32_t scale_byte(float amax, int e5m2) {
  // the exponent, one higher where the significand is above 1.75 (amax is finite and >= 0)
  const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - (e5m2 ? 15 : 8);
  return (uint32_t)max(e, 0);
}
__device__ __forceinline__ float inverse_scale(uint32_t byte) {   // byte <= 247
  return __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Infinities become NaN, which fmaxf passes over.
__device__ __forceinline__ float finite_or_nan(float v) {
  return fabsf(v) <= FLT_MAX ? v : __uint_as_float(0x7FC00000u);
}
// The larger magnitude, NaN if one of them is: what tells a group with values that are not finite from
// the others without looking at each value twice.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// ---- eight consecutive values
__device__ __forceinline__ uint32_t pack4(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x5410); }
__device__ __forceinline__ uint2 pack_fp8(const float (&v)[8], int e5m2) {
  uint32_t w[4];
  if (e5m2) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * k], v[2 * k + 1]), __NV_SATFINITE, __NV_E5M2);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * k], v[2 * k + 1]), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(pack4(w[0], w[1]), pack4(w[2], w[3]));
}
__device__ __forceinline__ uint2 pack_fp8(const float (&v)[8], float inv, int e5m2) {
  float u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = v[j] * inv;
  return pack_fp8(u, e5m2);
}
__device__ __forceinline__ void unpack_fp8(uint2 r, int e5m2, float scale, float (&v)[8]) {
  const uint32_t w[4] = {r.x & 0xFFFFu, r.x >> 16, r.y & 0xFFFFu, r.y >> 16};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[k],
                                                     e5m2 ? __NV_E5M2 : __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * k] = f.x * scale;
    v[2 * k + 1] = f.y * scale;
  }
}
// The first n (1 to 8) bytes of a chunk at p, which starts on an 8-byte boundary.
__device__ __forceinline__ void store_fp8(uint8_t* p, uint2 r, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = r;
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < n) p[j] = (uint8_t)((j < 4 ? r.x >> (8 * j) : r.y >> (8 * (j - 4))) & 0xFFu);
  }
}
__device__ __forceinline__ uint2 load_fp8(const uint8_t* p, int n) {
  if (n >= 8) return *reinterpret_cast<const uint2*>(p);
  uint2 r = make_uint2(0u, 0u);
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) (j < 4 ? r.x : r.y) |= (uint32_t)p[j] << (8 * (j & 3));
  return r;
}

// NaN where a value is not finite (or an infinity).
__device__ __forceinline__ float largest(const float (&v)[8]) {
  float a = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) a = max_nan(a, v[j]);
  return a;
}
// Over the 16 lanes that share a row's group.
__device__ __forceinline__ float half_warp_max(float a) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  return a;
}
// The largest finite magnitude of the group that 16 lanes hold (8 values each); values that are not
// finite become NaN.
__device__ __forceinline__ float group_max(float (&v)[8]) {
  float a = half_warp_max(largest(v));
  if (!(a <= FLT_MAX)) {                           // the same for the half-warp; rare
    a = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = finite_or_nan(v[j]);
      a = fmaxf(a, fabsf(v[j]));
    }
    const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(half, a, o));
  }
  return a;
}

// ---- tiles
// A block of 512 threads holds a tile of 128 x 128 values: a half-warp a row, eight consecutive
// columns a thread, four rows 32 apart.  Row scales come from one shuffle tree, column scales from
// the block's shared memory.
constexpr int kTileThreads = 512;
constexpr int kTileRows = kTileThreads / 16;      // rows per pass
constexpr int kTilePasses = kGroup / kTileRows;
struct TileSmem {
  float col[kTileThreads / 32][kGroup];
  float top[kGroup];
};

struct TileAt {
  int64_t r0;                                      // the tile's first row
  int64_t col;                                     // this thread's first column
  int64_t group;                                   // the tile's column group
  int row16, lane16;
  int left;                                        // the tile's rows from this thread's first one on
  int width;                                       // columns of this thread's chunk, 0 to 8
  int cols_here;                                   // columns of the tile
  __device__ __forceinline__ TileAt(int64_t tile, int64_t rows, int64_t cols)
      : row16(threadIdx.x >> 4), lane16(threadIdx.x & 15) {
    const int64_t tc = (cols + kGroup - 1) / kGroup, tr = tile / tc;
    group = tile - tr * tc;
    r0 = tr * kGroup;
    col = group * kGroup + lane16 * 8;
    left = (int)min((int64_t)kGroup, rows - r0) - row16;
    cols_here = (int)min((int64_t)kGroup, cols - group * kGroup);
    width = max(0, min(8, cols_here - lane16 * 8));
  }
  __device__ __forceinline__ int64_t row() const { return r0 + row16; }      // of pass 0
  __device__ __forceinline__ bool has(int i) const { return i * kTileRows < left; }
};
inline int64_t tiles_of(int64_t rows, int64_t cols) {
  return ((rows + kGroup - 1) / kGroup) * ((cols + kGroup - 1) / kGroup);
}
using TileValues = float[kTilePasses][8];

// One pass of a tile of an f32 or bf16 matrix; zeros past its edges.
template <typename T>
__device__ __forceinline__ void load_pass(Pack8<T>& p, const TileAt& at, int i, const T* src, int64_t ld,
                                          int vec) {
  const T* s = src + (at.row() + i * kTileRows) * ld + at.col;
  if (vec && at.width == 8) {
    if (at.has(i)) p.load(s); else p.zero();
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = at.has(i) && j < at.width ? to_f32(s[j]) : 0.f;
    p.set(v);
  }
}
// A tile's raw values of one matrix: f32 or bf16 ...
template <typename T>
struct TileRaw {
  using Elem = T;
  Pack8<T> p[kTilePasses];
  __device__ __forceinline__ void load(const TileAt& at, const T* src, int64_t ld, int vec) {
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) load_pass(p[i], at, i, src, ld, vec);
  }
  __device__ __forceinline__ void get(int i, float (&v)[8]) const { p[i].get(v); }
};
// ... or 8 bits.
struct TileRaw8 {
  uint2 p[kTilePasses];
  float s[kTilePasses];                            // of the row's group (1 for COL groups)
  __device__ __forceinline__ void load(const TileAt& at, const Fp8Ref& m) {
    const uint8_t* q = m.q + at.row() * m.ld + at.col;
    const bool rows = m.groups == MFSDP_GROUPS_ROW;
    const uint8_t* sp = m.s + (rows ? at.row() : at.r0 / kGroup) * m.ld_s + at.group;
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) {
      const bool in = at.has(i) && at.width > 0;
      p[i] = make_uint2(0u, 0u);
      if (in) p[i] = load_fp8(q + i * (kTileRows * m.ld), at.width);
      s[i] = 1.f;
      if (in && m.groups != MFSDP_GROUPS_COL)
        s[i] = scale_value(sp[rows ? i * (kTileRows * m.ld_s) : 0]);
    }
  }
  __device__ __forceinline__ void get(int i, int e5m2, float (&v)[8]) const {
    unpack_fp8(p[i], e5m2, s[i], v);
  }
};

// The tile as 1 x 128 groups.  Whole half-warps take part.
__device__ __forceinline__ void quantize_row(const TileAt& at, int i, float (&v)[8], const Fp8Ref& m) {
  const uint32_t byte = scale_byte(group_max(v), m.e5m2);
  if (!at.has(i) || at.width == 0) return;
  const int64_t r = at.row() + i * kTileRows;
  store_fp8(m.q + r * m.ld + at.col, pack_fp8(v, inverse_scale(byte), m.e5m2), at.width);
  if (at.lane16 == 0) m.s[r * m.ld_s + at.group] = (uint8_t)byte;
}

// The tile as 128 x 1 groups (COL) or one group (TILE); every thread of the block calls, and values that
// are not finite become NaN.  The shared memory is free again after the block's next barrier.
template <bool WHOLE>
__device__ __forceinline__ void quantize_cols(const TileAt& at, TileSmem& sm, const Fp8Ref& m,
                                              TileValues& v) {
  const int warp = threadIdx.x >> 5;
  float inv[8];
  // the columns' (or the tile's) largest values; once more without those that are not finite, if some are
  for (bool clean = false;; clean = true) {
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = fabsf(v[0][j]);
#pragma unroll
      for (int i = 1; i < kTilePasses; ++i)
        a[j] = clean ? fmaxf(a[j], fabsf(v[i][j])) : max_nan(a[j], v[i][j]);
      if (clean) a[j] = fmaxf(a[j], 0.f);
    }
    bool bad = false;
    if (WHOLE) {
      float t = largest(a);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t = max_nan(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
      if ((threadIdx.x & 31) == 0) sm.top[warp] = t;
      __syncthreads();
      t = sm.top[0];
#pragma unroll
      for (int w = 1; w < kTileThreads / 32; ++w) t = max_nan(t, sm.top[w]);
      bad = !(t <= FLT_MAX);
      if (!bad) {
        const uint32_t byte = scale_byte(t, m.e5m2);
        if (threadIdx.x == 0) m.s[at.r0 / kGroup * m.ld_s + at.group] = (uint8_t)byte;
        inv[0] = inverse_scale(byte);
      } else {
        __syncthreads();                           // the next round writes sm.top again
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = max_nan(a[j], __shfl_xor_sync(0xFFFFFFFFu, a[j], 16));
      if ((threadIdx.x & 16) == 0) {
        float4* d = reinterpret_cast<float4*>(&sm.col[warp][at.lane16 * 8]);
        d[0] = make_float4(a[0], a[1], a[2], a[3]);
        d[1] = make_float4(a[4], a[5], a[6], a[7]);
      }
      __syncthreads();
      if (threadIdx.x < kGroup) {
        float t = sm.col[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kTileThreads / 32; ++w) t = max_nan(t, sm.col[w][threadIdx.x]);
        bad = !(t <= FLT_MAX);
        const uint32_t byte = bad ? 0u : scale_byte(t, m.e5m2);
        sm.top[threadIdx.x] = inverse_scale(byte);
        if (!bad && (int)threadIdx.x < at.cols_here)
          m.s[at.r0 / kGroup * m.ld_s + at.group * kGroup + threadIdx.x] = (uint8_t)byte;
      }
      bad = __syncthreads_or(bad);
#pragma unroll
      for (int j = 0; j < 8; ++j) inv[j] = sm.top[at.lane16 * 8 + j];
    }
    if (!bad) break;
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = finite_or_nan(v[i][j]);
    __syncthreads();
  }
  uint8_t* q = m.q + at.row() * m.ld + at.col;
#pragma unroll
  for (int i = 0; i < kTilePasses; ++i) {
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = v[i][j] * inv[WHOLE ? 0 : j];
    if (at.has(i) && at.width > 0)
      store_fp8(q + i * (kTileRows * m.ld), pack_fp8(u, m.e5m2), at.width);
  }
}

// ---- host checks
inline bool groups_ok(int32_t g) { return g >= MFSDP_GROUPS_ROW && g <= MFSDP_GROUPS_TILE; }
inline int64_t scale_rows(int32_t g, int64_t rows) {
  return g == MFSDP_GROUPS_ROW ? rows : (rows + kGroup - 1) / kGroup;
}
inline int64_t scale_cols(int32_t g, int64_t cols) {
  return g == MFSDP_GROUPS_COL ? cols : (cols + kGroup - 1) / kGroup;
}
// An 8-bit matrix of rows x cols; `groups` < 0: any.
inline int check_fp8(const mfsdp_fp8_matrix& m, int64_t rows, int64_t cols, int32_t groups) {
  if (m.dtype != MFSDP_FP8_E4M3 && m.dtype != MFSDP_FP8_E5M2) return MFSDP_EINVAL;
  if (!groups_ok(m.groups) || (groups >= 0 && m.groups != groups)) return MFSDP_EINVAL;
  if (rows == 0) return MFSDP_OK;
  if (!m.data || !m.scales || m.ld < cols || m.ld_scales < scale_cols(m.groups, cols))
    return MFSDP_EINVAL;
  if (!aligned_to(m.data, 16) || m.ld % 16 != 0) return MFSDP_EALIGN;
  return MFSDP_OK;
}
inline Fp8Ref ref_of(const mfsdp_fp8_matrix* m) {
  if (!m) return Fp8Ref{};
  return Fp8Ref{static_cast<uint8_t*>(m->data), static_cast<uint8_t*>(m->scales), m->ld,
                m->ld_scales, m->dtype == MFSDP_FP8_E5M2, m->groups};
}
// Rows of 16-byte vectors (any number of columns: a row's last chunk goes by element).
inline bool vector_rows(const void* p, int64_t ld, int32_t dtype) {
  return aligned_to(p, 16) && (ld * (int64_t)dtype_bytes(dtype)) % 16 == 0;
}
inline bool shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 1 && rows < (1ll << 31) && cols < (1ll << 31);
}

}  // namespace mfsdp
