// 8-bit matrices from f32 or bf16 ones, from 8-bit ones of another grouping, and back.
//
// One read serves every grouping that is asked for: a block holds a 128 x 128 tile in registers, so
// 1 x 128, 128 x 1 and 128 x 128 groups all end inside it.  A value is scaled by a power of two
// (exact) and rounded once.  From 8 bits to 8 bits a value keeps its significand, and the change of
// groups rounds only what becomes subnormal (held_values: at the top of fp32's range too).  Bound by memory: the source once, a byte per value out
// (8192 x 14336 bf16 into both groupings: 85.5 us, 5.5 TB/s; 4096 x 4096 fp32 into tiles of 128 x 128:
// 16.3 us, 5.1 TB/s; 8192 x 14336 out of 8 bits into bf16: 64 us from ROW groups, 5.5 TB/s, 72 from COL ones).
// Regrouping moves too little for a block to hide a tile's load, maxima and barriers behind another block's
// (8192 x 14336: ROW into COL 68 us, 3.4 TB/s, into TILE 73, COL into ROW 76).
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"

namespace mfsdp {
namespace {

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ld;
  int32_t vec;
  Fp8Ref src;                 // an 8-bit source
  Fp8Ref row, other;          // 1 x 128 groups; 128 x 1 or 128 x 128 ones
};

enum Form : int { kRow = 1, kCol = 2, kTile = 4 };

template <typename Raw, int FORMS, typename At>
__device__ __forceinline__ void quantize_tile(const QuantArgs& p, const At& at, TileSmem<>& sm) {
  TileValues v;
  if constexpr (std::is_same<Raw, TileRaw8>::value) {
    Raw raw;
    raw.load(at, p.src);
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) raw.get(i, p.src.e5m2, v[i]);
    if (p.src.groups == MFSDP_GROUPS_COL) {
      const uint8_t* s = p.src.s + at.r0 / kGroup * p.src.ld_s + at.col;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = j < at.width() ? scale_value(s[j]) : 1.f;
#pragma unroll
        for (int i = 0; i < kTilePasses; ++i) v[i][j] = held_value(v[i][j], f);
      }
    }
  } else {
    Raw raw;
    raw.load(at, static_cast<const typename Raw::Elem*>(p.x), p.ld, p.vec);
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) raw.get(i, v[i]);
  }
  if (FORMS & kRow) {
#pragma unroll
    for (int i = 0; i < kTilePasses; i += 2) quantize_rows(at, i, v[i], v[i + 1], p.row);
  }
  if (FORMS & kCol) quantize_cols<1>(at, sm, {&p.other}, {&v});
  if (FORMS & kTile) quantize_whole(at, sm, p.other, v);
}

template <typename Raw, int FORMS>
__global__ void __launch_bounds__(kTileThreads, 2)
    quantize_kernel(const __grid_constant__ QuantArgs p) {
  __shared__ __align__(16) TileSmem<> sm;
  pdl_launch();
  pdl_wait();
  const int64_t tile_rows = (p.rows + kGroup - 1) / kGroup;
  const int32_t tc = (int32_t)blockIdx.x;
  for (int64_t tr = blockIdx.y; tr < tile_rows; tr += gridDim.y) {
    if (full_tile(tr, tc, p.rows, p.cols, p.vec))
      quantize_tile<Raw, FORMS>(p, TileAt<true>(tr, tc, p.rows, p.cols), sm);
    else
      quantize_tile<Raw, FORMS>(p, TileAt<false>(tr, tc, p.rows, p.cols), sm);
    if ((FORMS & kTile) && tr + gridDim.y < tile_rows) __syncthreads();
  }
}

struct DequantArgs {
  Fp8Ref src;
  int64_t rows, cols, chunks; // 8-column chunks of a row
  void* out;
  int64_t ld;
  int32_t vec;
};

// Eight consecutive values a thread.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(const __grid_constant__ DequantArgs p) {
  pdl_launch();
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * 256, n = p.rows * p.chunks;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += step) {
    const int64_t r = e / p.chunks, c = (e % p.chunks) * 8;
    const int w = (int)min((int64_t)8, p.cols - c);
    float v[8];
    const uint2 q = load_fp8(p.src.q + r * p.src.ld + c, w);
    if (p.src.groups == MFSDP_GROUPS_COL) {
      unpack_fp8(q, p.src.e5m2, 1.f, v);
      const uint8_t* s = p.src.s + r / kGroup * p.src.ld_s + c;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= j < w ? scale_value(s[j]) : 1.f;
    } else {
      const int64_t sr = p.src.groups == MFSDP_GROUPS_ROW ? r : r / kGroup;
      unpack_fp8(q, p.src.e5m2, scale_value(p.src.s[sr * p.src.ld_s + c / kGroup]), v);
    }
    T* o = static_cast<T*>(p.out) + r * p.ld + c;
    if (p.vec && w == 8) {
      Pack8<T> k;
      k.set(v);
      k.store(o);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < w) o[j] = from_f32<T>(v[j]);
    }
  }
}

template <typename Raw>
cudaError_t launch_quantize(const QuantArgs& a, int forms, cudaStream_t st) {
  const dim3 grid = tile_grid(a.rows, a.cols), block(kTileThreads);
  switch (forms) {
    case kRow: return launch_pdl(quantize_kernel<Raw, kRow>, grid, block, 0, st, a);
    case kCol: return launch_pdl(quantize_kernel<Raw, kCol>, grid, block, 0, st, a);
    case kTile: return launch_pdl(quantize_kernel<Raw, kTile>, grid, block, 0, st, a);
    default: return launch_pdl(quantize_kernel<Raw, kRow | kCol>, grid, block, 0, st, a);
  }
}

// The outputs of a call: one of any grouping, or a ROW and a COL one in either order.
int check_outputs(int64_t rows, int64_t cols, const mfsdp_fp8_matrix* out,
                  const mfsdp_fp8_matrix* also, QuantArgs& a, int& forms) {
  if (!out) return MFSDP_EINVAL;
  const mfsdp_fp8_matrix* m[2] = {out, also};
  forms = 0;
  for (int i = 0; i < 2; ++i) {
    if (!m[i]) continue;
    const int st = check_fp8(*m[i], rows, cols, -1);
    if (st != MFSDP_OK) return st;
    const int f = m[i]->groups == MFSDP_GROUPS_ROW ? kRow
                  : m[i]->groups == MFSDP_GROUPS_COL ? kCol : kTile;
    if (forms & f) return MFSDP_EINVAL;
    forms |= f;
    (f == kRow ? a.row : a.other) = ref_of(m[i]);
  }
  return also && forms != (kRow | kCol) ? MFSDP_EINVAL : MFSDP_OK;
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" int mfsdp_quantize_fp8(int64_t rows, int64_t cols, int32_t dtype, const void* x,
                                  int64_t ld_x, const mfsdp_fp8_matrix* out,
                                  const mfsdp_fp8_matrix* also, void* stream) {
  if (!dtype_ok(dtype)) return MFSDP_EINVAL;
  if (!shape_ok(rows, cols)) return MFSDP_ESHAPE;
  QuantArgs a{};
  int forms = 0;
  const int chk = check_outputs(rows, cols, out, also, a, forms);
  if (chk != MFSDP_OK) return chk;
  if (rows == 0) return MFSDP_OK;
  if (!x || ld_x < cols) return MFSDP_EINVAL;
  if (!aligned_to(x, dtype_bytes(dtype))) return MFSDP_EALIGN;
  if (!distinct({x, data_of(out), bytes_of(out), data_of(also), bytes_of(also)})) return MFSDP_EINVAL;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld_x;
  a.vec = vector_rows(x, ld_x, dtype);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MFSDP_DTYPE_BF16
                            ? launch_quantize<TileRaw<bf16_t>>(a, forms, st)
                            : launch_quantize<TileRaw<float>>(a, forms, st);
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}

extern "C" int mfsdp_regroup_fp8(int64_t rows, int64_t cols, const mfsdp_fp8_matrix* src,
                                 const mfsdp_fp8_matrix* out, const mfsdp_fp8_matrix* also,
                                 void* stream) {
  if (!src) return MFSDP_EINVAL;
  if (!shape_ok(rows, cols)) return MFSDP_ESHAPE;
  QuantArgs a{};
  int forms = 0;
  int chk = check_fp8(*src, rows, cols, -1);
  if (chk == MFSDP_OK) chk = check_outputs(rows, cols, out, also, a, forms);
  if (chk != MFSDP_OK) return chk;
  if (rows == 0) return MFSDP_OK;
  if (!distinct({src->data, src->scales, data_of(out), bytes_of(out), data_of(also), bytes_of(also)}))
    return MFSDP_EINVAL;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  a.src = ref_of(src);
  a.rows = rows;
  a.cols = cols;
  a.vec = 1;
  const cudaError_t e = launch_quantize<TileRaw8>(a, forms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}

extern "C" int mfsdp_dequantize_fp8(int64_t rows, int64_t cols, const mfsdp_fp8_matrix* src,
                                    int32_t dtype, void* out, int64_t ld_out, void* stream) {
  if (!src || !dtype_ok(dtype)) return MFSDP_EINVAL;
  if (!shape_ok(rows, cols)) return MFSDP_ESHAPE;
  const int chk = check_fp8(*src, rows, cols, -1);
  if (chk != MFSDP_OK) return chk;
  if (rows == 0) return MFSDP_OK;
  if (!out || ld_out < cols) return MFSDP_EINVAL;
  if (!aligned_to(out, dtype_bytes(dtype))) return MFSDP_EALIGN;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  DequantArgs a{};
  a.src = ref_of(src);
  a.rows = rows;
  a.cols = cols;
  a.chunks = (cols + 7) / 8;
  a.out = out;
  a.ld = ld_out;
  a.vec = vector_rows(out, ld_out, dtype);
  const int64_t blocks = (rows * a.chunks + 255) / 256;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)sms * 32));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MFSDP_DTYPE_BF16
                            ? launch_pdl(dequantize_kernel<bf16_t>, grid, dim3(256), 0, st, a)
                            : launch_pdl(dequantize_kernel<float>, grid, dim3(256), 0, st, a);
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}
