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

#include <algorithm>
#include <cfloat>
#include <initializer_list>

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
// (in bf16 every one is exact, 255 a NaN)
__device__ __forceinline__ float scale_value(uint32_t byte) {
  uint32_t r;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"((uint16_t)byte));
  return __uint_as_float(r << 16);
}

// Infinities become NaN, which fmaxf passes over.
__device__ __forceinline__ float finite_or_nan(float v) {
  return fabsf(v) <= FLT_MAX ? v : __uint_as_float(0x7FC00000u);
}
// The largest magnitude of three, NaN if one of them is: what tells a group with values that are not
// finite from the others without looking at each value twice.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) { return max3_nan(a, b, b); }
// The larger of each half.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A partial maximum as what is reduced across threads: its exponent, one higher where the significand
// is above 1.75, so that a group's scale is the largest one less the type's.  kMaybe and above: an
// infinity, a NaN, or a value beyond 1.75 2^127, which are told apart where the group is looked at again.
constexpr uint32_t kMaybe = 255u;
__device__ __forceinline__ uint32_t scale_part(float amax) {
  return (__float_as_uint(amax) + 0x1FFFFFu) >> 23;
}
__device__ __forceinline__ uint32_t scale_of_part(uint32_t part, int e5m2) {
  return (uint32_t)max((int)part - (e5m2 ? 15 : 8), 0);
}

// ---- two values in one instruction, each rounded as by the scalar one
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split_pair(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// ... cut towards zero: what is beyond fp32 becomes its largest value, not infinity.
__device__ __forceinline__ uint64_t mul2_cut(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int N>
__device__ __forceinline__ void scale_pairs(const float (&v)[N], float f, float (&u)[N]) {
  const uint64_t ff = pair_of(f, f);
#pragma unroll
  for (int j = 0; j < N; j += 2) split_pair(mul2(pair_of(v[j], v[j + 1]), ff), u[j], u[j + 1]);
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
  scale_pairs(v, inv, u);
  return pack_fp8(u, e5m2);
}
__device__ __forceinline__ void unpack_fp8(uint2 r, int e5m2, float (&v)[8]) {
  const uint32_t w[4] = {r.x & 0xFFFFu, r.x >> 16, r.y & 0xFFFFu, r.y >> 16};
  __half2_raw h[4];
  if (e5m2) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      h[k] = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[k], __NV_E5M2);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      h[k] = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[k], __NV_E4M3);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack_fp8(uint2 r, int e5m2, float scale, float (&v)[8]) {
  float u[8];
  unpack_fp8(r, e5m2, u);
  scale_pairs(u, scale, v);
}
// The values that 8 bits hold, as fp32 arithmetic goes on with them.  A product with a scale is exact
// wherever fp32 has it, and fp32's largest values, which are 2^128 in 8 bits, are beyond it: cut, they are
// the largest value again, which rounds to 2^128 once more, in both types.
__device__ __forceinline__ float held_value(float q, float scale) { return __fmul_rz(q, scale); }
__device__ __forceinline__ void held_values(uint2 r, int e5m2, float scale, float (&v)[8]) {
  float u[8];
  unpack_fp8(r, e5m2, u);
  const uint64_t ff = pair_of(scale, scale);
#pragma unroll
  for (int j = 0; j < 8; j += 2) split_pair(mul2_cut(pair_of(u[j], u[j + 1]), ff), v[j], v[j + 1]);
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

// The largest magnitude; NaN or an infinity where a value is not finite.
__device__ __forceinline__ float largest(const float (&v)[8]) {
  const float a = max3_nan(v[0], v[1], v[2]), b = max3_nan(v[3], v[4], v[5]);
  return max3_nan(a, b, max_nan(v[6], v[7]));
}
// Two values at a time over the 16 lanes that share a row's group.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t w) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) w = max_u16x2(w, __shfl_xor_sync(0xFFFFFFFFu, w, o));
  return w;
}
// The scale of a group with values that are not finite, which become NaN; the group's 16 lanes call.
__device__ __forceinline__ uint32_t cleaned_scale(float (&v)[8], int e5m2) {
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = finite_or_nan(v[j]);
    a = fmaxf(a, fabsf(v[j]));
  }
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(half, a, o));
  return scale_byte(a, e5m2);
}
// The scales of two groups, 8 values a lane of each; their lanes' largest values are reduced together.
__device__ __forceinline__ void group_scales(float (&u)[8], float (&v)[8], int u_e5m2, int v_e5m2,
                                             uint32_t& su, uint32_t& sv) {
  const uint32_t w = half_warp_max(scale_part(largest(u)) | (scale_part(largest(v)) << 16));
  su = scale_of_part(w & 0xFFFFu, u_e5m2);
  sv = scale_of_part(w >> 16, v_e5m2);
  if ((w & 0xFFFFu) >= kMaybe) su = cleaned_scale(u, u_e5m2);   // the same for the half-warp; rare
  if ((w >> 16) >= kMaybe) sv = cleaned_scale(v, v_e5m2);
}

// ---- sixteen consecutive values a thread, where no group runs down the columns: eight lanes hold a
// group of 128, and what a row costs apart from its values falls on twice as many of them
struct Sixteen {
  int64_t row, col;
  int32_t group;
  int width;                                       // columns of this thread, 0 to 16
  bool has;                                        // the row exists
};
__device__ __forceinline__ float largest(const float (&v)[16]) {
  float a = max3_nan(v[0], v[1], v[2]);
#pragma unroll
  for (int j = 3; j + 1 < 16; j += 2) a = max3_nan(a, v[j], v[j + 1]);
  return max_nan(a, v[15]);
}
__device__ __forceinline__ uint32_t eighth_warp_max(uint32_t w) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) w = max_u16x2(w, __shfl_xor_sync(0xFFFFFFFFu, w, o));
  return w;
}
__device__ __forceinline__ uint32_t cleaned_scale(float (&v)[16], int e5m2) {
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    v[j] = finite_or_nan(v[j]);
    a = fmaxf(a, fabsf(v[j]));
  }
  const uint32_t eighth = 0xFFu << (threadIdx.x & 24);
  for (int o = 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(eighth, a, o));
  return scale_byte(a, e5m2);
}
// Whole warps call; values past the row's end are zero.
__device__ __forceinline__ void quantize_sixteen(const Sixteen& at, float (&v)[16], uint32_t part,
                                                 const Fp8Ref& m) {
  uint32_t byte = scale_of_part(part, m.e5m2);
  if (part >= kMaybe) byte = cleaned_scale(v, m.e5m2);   // the same for the eight lanes; rare
  if (!at.has || at.width <= 0) return;
  const float inv = inverse_scale(byte);
  float lo[8], hi[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo[j] = v[j];
    hi[j] = v[8 + j];
  }
  scale_pairs(lo, inv, lo);
  scale_pairs(hi, inv, hi);
  const uint2 a = pack_fp8(lo, m.e5m2), b = pack_fp8(hi, m.e5m2);
  uint8_t* q = m.q + at.row * m.ld + at.col;
  if (at.width >= 16) {
    *reinterpret_cast<uint4*>(q) = make_uint4(a.x, a.y, b.x, b.y);
  } else {
    store_fp8(q, a, min(at.width, 8));
    if (at.width > 8) store_fp8(q + 8, b, at.width - 8);
  }
  if ((threadIdx.x & 7) == 0) m.s[at.row * m.ld_s + at.group] = (uint8_t)byte;
}
// `count` values (0 to 16) of a row from p on; zeros past them.
template <typename T>
__device__ __forceinline__ void load_sixteen(Pack8<T> (&r)[2], const T* p, int count, int vec) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (vec && count >= 8 * h + 8) {
      r[h].load(p + 8 * h);
    } else {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 8 * h + j < count ? to_f32(p[8 * h + j]) : 0.f;
      r[h].set(v);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store_sixteen(T* p, int count, int vec, const float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = v[8 * h + j];
    if (vec && count >= 8 * h + 8) {
      Pack8<T> k;
      k.set(u);
      k.store(p + 8 * h);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (8 * h + j < count) p[8 * h + j] = from_f32<T>(u[j]);
    }
  }
}
template <typename T>
__device__ __forceinline__ void get_sixteen(const Pack8<T> (&r)[2], float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float u[8];
    r[h].get(u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * h + j] = u[j];
  }
}

// ---- tiles
// A block of 512 threads holds a tile of 128 x 128 values: a half-warp a row, eight consecutive
// columns a thread, four rows 32 apart.  Row scales come from one shuffle tree, column scales from
// the block's shared memory.
constexpr int kTileThreads = 512;
constexpr int kTileRows = kTileThreads / 16;      // rows per pass
constexpr int kTilePasses = kGroup / kTileRows;
template <int N = 1>
struct TileSmem {
  uint32_t col[N][kTileThreads / 32][kGroup / 2];  // a warp's scales, two columns a word
  float top[N][kGroup];                            // the columns' inverse scales
};

// FULL: the tile has all its rows and columns, and every matrix rows for 16-byte accesses: no test per
// value or chunk remains.
template <bool FULL>
struct TileAt {
  static constexpr bool kFull = FULL;
  int64_t r0;                                      // the tile's first row
  int64_t row;                                     // this thread's first row and column
  int64_t col;
  int32_t group;                                   // the tile's column group
  int lane16;
  int left;                                        // the tile's rows from this thread's first one on
  int cols_here;                                   // columns of the tile
  // tile row tr and column group tc
  __device__ __forceinline__ TileAt(int64_t tr, int32_t tc, int64_t rows, int64_t cols)
      : group(tc), lane16(threadIdx.x & 15) {
    const int row16 = threadIdx.x >> 4;
    r0 = tr * kGroup;
    row = r0 + row16;
    col = (int64_t)tc * kGroup + lane16 * 8;
    left = (int)min((int64_t)kGroup, rows - r0) - row16;
    cols_here = (int)min((int64_t)kGroup, cols - (int64_t)tc * kGroup);
  }
  __device__ __forceinline__ bool has(int i) const { return FULL || i * kTileRows < left; }
  __device__ __forceinline__ int width() const {   // columns of this thread's chunk, 0 to 8
    return FULL ? 8 : max(0, min(8, cols_here - lane16 * 8));
  }
};
__device__ __forceinline__ bool full_tile(int64_t tr, int32_t tc, int64_t rows, int64_t cols, int vec) {
  return vec && (tr + 1) * kGroup <= rows && ((int64_t)tc + 1) * kGroup <= cols;
}
// The blocks of a launch: x the column groups, y the tile rows (walked where there are more).
inline dim3 tile_grid(int64_t rows, int64_t cols) {
  return dim3((unsigned)((cols + kGroup - 1) / kGroup),
              (unsigned)std::min<int64_t>((rows + kGroup - 1) / kGroup, 65535));
}
inline int64_t tiles_of(int64_t rows, int64_t cols) {
  return ((rows + kGroup - 1) / kGroup) * ((cols + kGroup - 1) / kGroup);
}
using TileValues = float[kTilePasses][8];

// One pass of a tile of an f32 or bf16 matrix; zeros past its edges.
template <typename T, typename At>
__device__ __forceinline__ void load_pass(Pack8<T>& p, const At& at, int i, const T* src, int64_t ld,
                                          int vec) {
  const T* s = src + (at.row + i * kTileRows) * ld + at.col;
  if (At::kFull || (vec && at.width() == 8)) {
    if (at.has(i)) p.load(s); else p.zero();
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = at.has(i) && j < at.width() ? to_f32(s[j]) : 0.f;
    p.set(v);
  }
}
// A tile's raw values of one matrix: f32 or bf16 ...
template <typename T>
struct TileRaw {
  using Elem = T;
  Pack8<T> p[kTilePasses];
  template <typename At>
  __device__ __forceinline__ void load(const At& at, const T* src, int64_t ld, int vec) {
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) load_pass(p[i], at, i, src, ld, vec);
  }
  __device__ __forceinline__ void get(int i, float (&v)[8]) const { p[i].get(v); }
};
// ... or 8 bits.
struct TileRaw8 {
  uint2 p[kTilePasses];
  float s[kTilePasses];                            // of the row's group (1 for COL groups)
  template <typename At>
  __device__ __forceinline__ void load(const At& at, const Fp8Ref& m) {
    const uint8_t* q = m.q + at.row * m.ld + at.col;
    const bool rows = m.groups == MFSDP_GROUPS_ROW;
    const uint8_t* sp = m.s + (rows ? at.row : at.r0 / kGroup) * m.ld_s + at.group;
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) {
      const bool in = at.has(i) && at.width() > 0;
      p[i] = make_uint2(0u, 0u);
      if (in) p[i] = load_fp8(q + i * (kTileRows * m.ld), at.width());
      s[i] = 1.f;
      if (in && m.groups != MFSDP_GROUPS_COL)
        s[i] = scale_value(sp[rows ? i * (kTileRows * m.ld_s) : 0]);
    }
  }
  __device__ __forceinline__ void get(int i, int e5m2, float (&v)[8]) const {
    held_values(p[i], e5m2, s[i], v);
  }
};

// Two passes of the tile as 1 x 128 groups.  Whole half-warps take part.
template <typename At>
__device__ __forceinline__ void quantize_rows(const At& at, int i, float (&u)[8], float (&v)[8],
                                              const Fp8Ref& m) {
  uint32_t su, sv;
  group_scales(u, v, m.e5m2, m.e5m2, su, sv);
  if (at.width() == 0) return;
  const int64_t r = at.row + i * kTileRows;
  uint8_t* q = m.q + r * m.ld + at.col;
  uint8_t* s = m.s + r * m.ld_s + at.group;
  if (at.has(i)) {
    store_fp8(q, pack_fp8(u, inverse_scale(su), m.e5m2), at.width());
    if (at.lane16 == 0) *s = (uint8_t)su;
  }
  if (at.has(i + 1)) {
    store_fp8(q + kTileRows * m.ld, pack_fp8(v, inverse_scale(sv), m.e5m2), at.width());
    if (at.lane16 == 0) s[kTileRows * m.ld_s] = (uint8_t)sv;
  }
}

// The columns' scales of a thread's four rows, two columns a word.
__device__ __forceinline__ void column_parts(const TileValues& v, bool again, uint32_t (&w)[4]) {
  static_assert(kTilePasses == 4, "four rows a thread");
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = 2 * k + h;
      const float a = again ? fmaxf(fmaxf(fmaxf(fabsf(v[0][j]), fabsf(v[1][j])),
                                          fmaxf(fabsf(v[2][j]), fabsf(v[3][j]))), 0.f)
                            : max_nan(max3_nan(v[0][j], v[1][j], v[2][j]), v[3][j]);
      b[h] = scale_part(a);
    }
    w[k] = b[0] | (b[1] << 16);
  }
}
__device__ __forceinline__ void clean_values(TileValues& v) {
#pragma unroll
  for (int i = 0; i < kTilePasses; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = finite_or_nan(v[i][j]);
}
template <typename At>
__device__ __forceinline__ void store_columns(const At& at, const Fp8Ref& m, const TileValues& v,
                                              const float (&inv)[8]) {
  uint8_t* q = m.q + at.row * m.ld + at.col;
#pragma unroll
  for (int i = 0; i < kTilePasses; ++i) {
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      split_pair(mul2(pair_of(v[i][j], v[i][j + 1]), pair_of(inv[j], inv[j + 1])), u[j], u[j + 1]);
    if (at.has(i)) store_fp8(q + i * (kTileRows * m.ld), pack_fp8(u, m.e5m2), at.width());
  }
}

// N matrices' tiles as 128 x 1 groups, with the barriers of one; every thread of the block calls, and
// values that are not finite become NaN.  Another tile may follow at once: what it writes to the shared
// memory was last read before a barrier that it has passed.
template <int N, int M, typename At>
__device__ __forceinline__ void quantize_cols(const At& at, TileSmem<M>& sm, const Fp8Ref* const (&m)[N],
                                              TileValues* const (&v)[N]) {
  static_assert(N <= M && N <= 2, "one or two");
  const int warp = threadIdx.x >> 5;
  // the columns' scales; once more without the values that are not finite, if some are
  for (bool again = false;; again = true) {
    if (again) {
#pragma unroll
      for (int n = 0; n < N; ++n) clean_values(*v[n]);
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t w[4];
      column_parts(*v[n], again, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = max_u16x2(w[k], __shfl_xor_sync(0xFFFFFFFFu, w[k], 16));
      if ((threadIdx.x & 16) == 0)
        *reinterpret_cast<uint4*>(&sm.col[n][warp][at.lane16 * 4]) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    bool bad = false;
    if (threadIdx.x < N * (kGroup / 2)) {
      const int n = N == 1 ? 0 : threadIdx.x / (kGroup / 2), c = threadIdx.x % (kGroup / 2);
      const int e5m2 = n ? m[N - 1]->e5m2 : m[0]->e5m2;
      uint32_t t = sm.col[n][0][c];
#pragma unroll
      for (int k = 1; k < kTileThreads / 32; ++k) t = max_u16x2(t, sm.col[n][k][c]);
      const uint32_t lo = scale_of_part(t & 0xFFFFu, e5m2), hi = scale_of_part(t >> 16, e5m2);
      bad = ((t & 0xFFFFu) >= kMaybe || (t >> 16) >= kMaybe) && !again;
      sm.top[n][2 * c] = inverse_scale(lo);
      sm.top[n][2 * c + 1] = inverse_scale(hi);
      uint8_t* s = (n ? m[N - 1]->s : m[0]->s) + at.r0 / kGroup * (n ? m[N - 1]->ld_s : m[0]->ld_s) +
                   at.group * kGroup + 2 * c;
      if (2 * c < at.cols_here) s[0] = (uint8_t)lo;
      if (2 * c + 1 < at.cols_here) s[1] = (uint8_t)hi;
    }
    if (!__syncthreads_or(bad)) break;
  }
  if (at.width() == 0) return;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float inv[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 f = reinterpret_cast<const float4*>(sm.top[n])[at.lane16 * 2 + k];
      inv[4 * k] = f.x;
      inv[4 * k + 1] = f.y;
      inv[4 * k + 2] = f.z;
      inv[4 * k + 3] = f.w;
    }
    store_columns(at, *m[n], *v[n], inv);
  }
}

// The tile as one group.  Another tile's shared memory needs a barrier between.
template <typename At>
__device__ __forceinline__ void quantize_whole(const At& at, TileSmem<1>& sm, const Fp8Ref& m,
                                               TileValues& v) {
  uint32_t byte;
  for (bool again = false;; again = true) {
    if (again) {
      clean_values(v);
      __syncthreads();
    }
    uint32_t w[4];
    column_parts(v, again, w);
    uint32_t t = max_u16x2(max_u16x2(w[0], w[1]), max_u16x2(w[2], w[3]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = max_u16x2(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
    if ((threadIdx.x & 31) == 0) sm.col[0][threadIdx.x >> 5][0] = t;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTileThreads / 32; ++k) t = max_u16x2(t, sm.col[0][k][0]);
    const uint32_t part = max(t & 0xFFFFu, t >> 16);
    byte = scale_of_part(part, m.e5m2);
    if (part < kMaybe || again) break;             // the same for all threads
  }
  if (threadIdx.x == 0) m.s[at.r0 / kGroup * m.ld_s + at.group] = (uint8_t)byte;
  if (at.width() == 0) return;
  float inv[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) inv[j] = inverse_scale(byte);
  store_columns(at, m, v, inv);
}

// ---- host checks
// Whether results have buffers of their own (null: not wanted).
inline bool distinct(std::initializer_list<const void*> results) {
  for (auto i = results.begin(); i != results.end(); ++i)
    for (auto j = results.begin(); j != i; ++j)
      if (*i && *i == *j) return false;
  return true;
}
// Whether no result is an input's buffer (inputs may share theirs).
inline bool apart(std::initializer_list<const void*> results, std::initializer_list<const void*> inputs) {
  for (const void* r : results)
    for (const void* i : inputs)
      if (r && r == i) return false;
  return true;
}
inline const void* data_of(const mfsdp_fp8_matrix* m) { return m ? m->data : nullptr; }
inline const void* bytes_of(const mfsdp_fp8_matrix* m) { return m ? m->scales : nullptr; }
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
