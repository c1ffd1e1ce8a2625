// The activation between two linear layers, with results and checkpoints in 8 bits.
//
//   SwiGLU: y = gate p up,  p = 1 / (1 + exp(-gate));   dgate = dy up p (1 + gate (1 - p)),
//           dup = dy gate p
//   GELU (tanh form): y = gate p,  p = 1 / (1 + exp(-2 u)),  u = sqrt(2 / pi) (gate + 0.044715 gate^3)
//           ((1 + tanh u) / 2 = p);   dgate = dy (p + gate 2 p (1 - p) u')
// Forward reads the inputs once and writes y (in the caller's type, in 8 bits, or both) and the inputs'
// 8-bit checkpoints.  Backward reads dy and the inputs, or their checkpoints, and writes the gradients in
// the caller's type or in 8 bits, in the two groupings that the two products of a layer's backward pass
// take, so that no gradient is written in 16 bits and read again to be quantized.  A block holds a tile of
// 128 x 128 values, which both groupings end inside.
//
// Bound by memory, with little to spare: a value costs two special-function instructions and some forty
// others in the backward pass.
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"

namespace mfsdp {
namespace {

struct ActArgs {
  int64_t rows, cols, tiles;
  const void *gate, *up, *dy;     // inputs (backward: nullable where the checkpoint is given)
  int64_t ld_gate, ld_up, ld_dy;
  void* y;
  int64_t ld_y;
  Fp8Ref y8, gate8, up8;          // forward: results; backward: gate8 and up8 are inputs
  void *dgate, *dup;              // nullable
  int64_t ld_dgate, ld_dup;
  Fp8Ref dgate_row, dgate_col, dup_row, dup_col;
  int32_t vec;
};

// 1 / (1 + exp(-x)).  Beside bf16 rows, whose time leaves room for some twenty instructions a value,
// exp and the division are the special-function unit's (within 2 ulp each); fp32 ones move twice the
// bytes and take the exact ones.
template <typename T>
__device__ __forceinline__ float sigmoid(float x);
template <>
__device__ __forceinline__ float sigmoid<bf16_t>(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-x)));
  return r;
}
template <>
__device__ __forceinline__ float sigmoid<float>(float x) {
  return 1.f / (1.f + expf(-x));
}

constexpr float kGelu = 1.5957691216057308f;           // 2 sqrt(2 / pi)
// The share of the gate that passes.
template <typename T, bool GLU>
__device__ __forceinline__ float gate_of(float g) {
  return sigmoid<T>(GLU ? g : kGelu * g * fmaf(0.044715f, g * g, 1.f));
}
template <typename T, bool GLU>
__device__ __forceinline__ float act(float g, float u) {
  const float y = g * gate_of<T, GLU>(g);
  return GLU ? y * u : y;
}
template <typename T, bool GLU>
__device__ __forceinline__ float grad_gate(float dy, float g, float u) {
  const float p = gate_of<T, GLU>(g);
  if (GLU) return dy * p * u * fmaf(g, 1.f - p, 1.f);
  // beyond 16 p is 0 or 1 in fp32, and the polynomial may be too large for it
  const float slope = fabsf(g) > 16.f ? 0.f : g * kGelu * fmaf(3.f * 0.044715f, g * g, 1.f);
  return dy * fmaf(slope, p * (1.f - p), p);
}

template <typename T>
__device__ __forceinline__ void store_values(T* base, int64_t ld, const TileAt& at, int i, int vec,
                                             const float (&v)[8]) {
  if (!at.has(i)) return;
  T* d = base + (at.row() + i * kTileRows) * ld + at.col;
  if (vec && at.width == 8) {
    Pack8<T> p;
    p.set(v);
    p.store(d);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < at.width) d[j] = from_f32<T>(v[j]);
  }
}

template <typename T, bool GLU>
__global__ void __launch_bounds__(kTileThreads, sizeof(T) == 2 ? 2 : 1)
    activation_forward_kernel(const __grid_constant__ ActArgs p) {
  pdl_launch();
  pdl_wait();
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const TileAt at(tile, p.rows, p.cols);
#pragma unroll
    for (int half = 0; half < kTilePasses; half += 2) {    // (all passes at once would spill)
      Pack8<T> graw[2], uraw[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        load_pass(graw[h], at, half + h, static_cast<const T*>(p.gate), p.ld_gate, p.vec);
        if (GLU) load_pass(uraw[h], at, half + h, static_cast<const T*>(p.up), p.ld_up, p.vec);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = half + h;
        float g[8], u[8], y[8];
        graw[h].get(g);
        if (GLU) uraw[h].get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = act<T, GLU>(g[j], GLU ? u[j] : 0.f);
        if (p.y) store_values(static_cast<T*>(p.y), p.ld_y, at, i, p.vec, y);
        if (p.y8.q) quantize_row(at, i, y, p.y8);
        if (p.gate8.q) quantize_row(at, i, g, p.gate8);
        if (GLU && p.up8.q) quantize_row(at, i, u, p.up8);
      }
    }
  }
}

// The gate's gradient, then up's: one of them in registers at a time, and p computed twice, so that
// two blocks share an SM and one loads while the other computes.
template <typename T, bool GLU, typename Raw>
__global__ void __launch_bounds__(kTileThreads, sizeof(T) == 2 ? 2 : 1)
    activation_backward_kernel(const __grid_constant__ ActArgs p) {
  __shared__ __align__(16) TileSmem sm;
  pdl_launch();
  pdl_wait();
  constexpr bool kKept = std::is_same<Raw, TileRaw8>::value;
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const TileAt at(tile, p.rows, p.cols);
    TileRaw<T> dy;
    Raw gate, up;
    dy.load(at, static_cast<const T*>(p.dy), p.ld_dy, p.vec);
    if constexpr (kKept) {
      gate.load(at, p.gate8);
      if (GLU) up.load(at, p.up8);
    } else {
      gate.load(at, static_cast<const T*>(p.gate), p.ld_gate, p.vec);
      if (GLU) up.load(at, static_cast<const T*>(p.up), p.ld_up, p.vec);
    }
    auto emit = [&](TileValues& v, void* out, int64_t ld, const Fp8Ref& row, const Fp8Ref& col) {
      if (out)
#pragma unroll
        for (int i = 0; i < kTilePasses; ++i)
          store_values(static_cast<T*>(out), ld, at, i, p.vec, v[i]);
      if (row.q)
#pragma unroll
        for (int i = 0; i < kTilePasses; ++i) quantize_row(at, i, v[i], row);
      if (col.q) {
        quantize_cols<false>(at, sm, col, v);
        __syncthreads();
      }
    };
    auto gate_value = [&](int i, float (&g)[8]) {
      if constexpr (kKept) gate.get(i, p.gate8.e5m2, g); else gate.get(i, g);
    };
    TileValues v;
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) {
      float d[8], g[8], u[8];
      dy.get(i, d);
      gate_value(i, g);
      if constexpr (GLU && kKept) up.get(i, p.up8.e5m2, u);
      if constexpr (GLU && !kKept) up.get(i, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = grad_gate<T, GLU>(d[j], g[j], GLU ? u[j] : 0.f);
    }
    emit(v, p.dgate, p.ld_dgate, p.dgate_row, p.dgate_col);
    if (!GLU || !(p.dup || p.dup_row.q || p.dup_col.q)) continue;
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) {
      float d[8], g[8];
      dy.get(i, d);
      gate_value(i, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = d[j] * g[j] * gate_of<T, GLU>(g[j]);
    }
    emit(v, p.dup, p.ld_dup, p.dup_row, p.dup_col);
  }
}

int check_kind(int32_t kind, int64_t rows, int64_t cols, int32_t dtype) {
  if ((kind != MFSDP_ACT_SWIGLU && kind != MFSDP_ACT_GELU) || !dtype_ok(dtype)) return MFSDP_EINVAL;
  return shape_ok(rows, cols) ? MFSDP_OK : MFSDP_ESHAPE;
}
// A matrix of the caller's type (nullable): its pitch, and whether its rows take 16-byte accesses.
int check_rows(const void* p, int64_t ld, int64_t cols, int32_t dtype, int32_t& vec) {
  if (!p) return MFSDP_OK;
  if (ld < cols) return MFSDP_EINVAL;
  if (!aligned_to(p, dtype_bytes(dtype))) return MFSDP_EALIGN;
  vec = vec && vector_rows(p, ld, dtype);
  return MFSDP_OK;
}
int check_group(const mfsdp_fp8_matrix* m, int64_t rows, int64_t cols, int32_t groups) {
  return m ? check_fp8(*m, rows, cols, groups) : MFSDP_OK;
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" int mfsdp_activation_forward(int32_t kind, int64_t rows, int64_t cols, int32_t dtype,
                                        const void* gate, int64_t ld_gate, const void* up,
                                        int64_t ld_up, void* y, int64_t ld_y,
                                        const mfsdp_fp8_matrix* y8, const mfsdp_fp8_matrix* gate8,
                                        const mfsdp_fp8_matrix* up8, void* stream) {
  int chk = check_kind(kind, rows, cols, dtype);
  if (chk != MFSDP_OK) return chk;
  const bool glu = kind == MFSDP_ACT_SWIGLU;
  if ((!y && !y8) || (!glu && (up || up8))) return MFSDP_EINVAL;
  for (const mfsdp_fp8_matrix* m : {y8, gate8, up8})
    if ((chk = check_group(m, rows, cols, MFSDP_GROUPS_ROW)) != MFSDP_OK) return chk;
  if (rows == 0) return MFSDP_OK;
  if (!gate || (glu && !up)) return MFSDP_EINVAL;
  ActArgs a{};
  a.vec = 1;
  if ((chk = check_rows(gate, ld_gate, cols, dtype, a.vec)) != MFSDP_OK ||
      (chk = check_rows(up, ld_up, cols, dtype, a.vec)) != MFSDP_OK ||
      (chk = check_rows(y, ld_y, cols, dtype, a.vec)) != MFSDP_OK)
    return chk;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  a.rows = rows;
  a.cols = cols;
  a.tiles = tiles_of(rows, cols);
  a.gate = gate;
  a.ld_gate = ld_gate;
  a.up = up;
  a.ld_up = ld_up;
  a.y = y;
  a.ld_y = ld_y;
  a.y8 = ref_of(y8);
  a.gate8 = ref_of(gate8);
  a.up8 = ref_of(up8);
  const dim3 grid((unsigned)std::min<int64_t>(a.tiles, 1ll << 30)), block(kTileThreads);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == MFSDP_DTYPE_BF16;
  const cudaError_t e =
      glu ? (bf ? launch_pdl(activation_forward_kernel<bf16_t, true>, grid, block, 0, st, a)
                : launch_pdl(activation_forward_kernel<float, true>, grid, block, 0, st, a))
          : (bf ? launch_pdl(activation_forward_kernel<bf16_t, false>, grid, block, 0, st, a)
                : launch_pdl(activation_forward_kernel<float, false>, grid, block, 0, st, a));
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}

extern "C" int mfsdp_activation_backward(
    int32_t kind, int64_t rows, int64_t cols, int32_t dtype, const void* dy, int64_t ld_dy,
    const void* gate, int64_t ld_gate, const mfsdp_fp8_matrix* gate8, const void* up, int64_t ld_up,
    const mfsdp_fp8_matrix* up8, void* dgate, int64_t ld_dgate, void* dup, int64_t ld_dup,
    const mfsdp_fp8_matrix* dgate_row, const mfsdp_fp8_matrix* dgate_col,
    const mfsdp_fp8_matrix* dup_row, const mfsdp_fp8_matrix* dup_col, void* stream) {
  int chk = check_kind(kind, rows, cols, dtype);
  if (chk != MFSDP_OK) return chk;
  const bool glu = kind == MFSDP_ACT_SWIGLU;
  if (!glu && (up || up8 || dup || dup_row || dup_col)) return MFSDP_EINVAL;
  if (!dgate && !dgate_row && !dgate_col && !dup && !dup_row && !dup_col) return MFSDP_EINVAL;
  for (const mfsdp_fp8_matrix* m : {gate8, up8, dgate_row, dup_row})
    if ((chk = check_group(m, rows, cols, MFSDP_GROUPS_ROW)) != MFSDP_OK) return chk;
  for (const mfsdp_fp8_matrix* m : {dgate_col, dup_col})
    if ((chk = check_group(m, rows, cols, MFSDP_GROUPS_COL)) != MFSDP_OK) return chk;
  // the inputs as they are, or both in 8 bits
  if ((gate && gate8) || (up && up8) || (glu && (gate8 != nullptr) != (up8 != nullptr)))
    return MFSDP_EINVAL;
  if (rows == 0) return MFSDP_OK;
  if (!dy || (!gate && !gate8) || (glu && !up && !up8)) return MFSDP_EINVAL;
  ActArgs a{};
  a.vec = 1;
  if ((chk = check_rows(dy, ld_dy, cols, dtype, a.vec)) != MFSDP_OK ||
      (chk = check_rows(gate, ld_gate, cols, dtype, a.vec)) != MFSDP_OK ||
      (chk = check_rows(up, ld_up, cols, dtype, a.vec)) != MFSDP_OK ||
      (chk = check_rows(dgate, ld_dgate, cols, dtype, a.vec)) != MFSDP_OK ||
      (chk = check_rows(dup, ld_dup, cols, dtype, a.vec)) != MFSDP_OK)
    return chk;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  a.rows = rows;
  a.cols = cols;
  a.tiles = tiles_of(rows, cols);
  a.dy = dy;
  a.ld_dy = ld_dy;
  a.gate = gate;
  a.ld_gate = ld_gate;
  a.gate8 = ref_of(gate8);
  a.up = up;
  a.ld_up = ld_up;
  a.up8 = ref_of(up8);
  a.dgate = dgate;
  a.ld_dgate = ld_dgate;
  a.dup = dup;
  a.ld_dup = ld_dup;
  a.dgate_row = ref_of(dgate_row);
  a.dgate_col = ref_of(dgate_col);
  a.dup_row = ref_of(dup_row);
  a.dup_col = ref_of(dup_col);
  const dim3 grid((unsigned)std::min<int64_t>(a.tiles, 1ll << 30)), block(kTileThreads);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, st, a); };
  const bool bf = dtype == MFSDP_DTYPE_BF16;
  cudaError_t e;
  if (gate8)
    e = glu ? (bf ? go(activation_backward_kernel<bf16_t, true, TileRaw8>)
                  : go(activation_backward_kernel<float, true, TileRaw8>))
            : (bf ? go(activation_backward_kernel<bf16_t, false, TileRaw8>)
                  : go(activation_backward_kernel<float, false, TileRaw8>));
  else
    e = glu ? (bf ? go(activation_backward_kernel<bf16_t, true, TileRaw<bf16_t>>)
                  : go(activation_backward_kernel<float, true, TileRaw<float>>))
            : (bf ? go(activation_backward_kernel<bf16_t, false, TileRaw<bf16_t>>)
                  : go(activation_backward_kernel<float, false, TileRaw<float>>));
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}
