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
// Forward is bound by memory, with little to spare (8192 x 14336 SwiGLU with all three results in 8 bits:
// 163 us, 5.0 TB/s; GELU 128 us).  Backward fills no unit (2048 rows of it: 57 % of the issue slots, 45 % of the
// ALU, 34 % of the memory): a value's four results cost some fifty instructions, and the gradients fill the
// registers for one block of 16 warps an SM, which meet at two barriers a tile (the same size from the
// checkpoints, 8 bytes a value: 242 us, 3.9 TB/s; GELU 152 us).
#include <algorithm>
#include <atomic>

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
// exp and the division are the special-function unit's: the product with log2(e) is rounded before the
// power of two is taken, so exp is within (2 + 1.2 |x|) 2^-23 of itself, the division within 2^-22, and
// results below 2^-126 (x < -87.3) are 0.  fp32 ones move twice the bytes and take the exact ones.
template <typename T>
__device__ __forceinline__ float sigmoid(float x);
template <>
__device__ __forceinline__ float sigmoid<bf16_t>(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
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
__device__ __forceinline__ void act_grads(float dy, float g, float u, float& dg, float& du) {
  const float p = gate_of<T, GLU>(g);
  if (GLU) {
    const float s = dy * p;
    dg = s * u * fmaf(g, 1.f - p, 1.f);
    du = s * g;
  } else {
    // beyond 16 p is 0 or 1 in fp32, and the polynomial may be too large for it
    const float slope = fabsf(g) > 16.f ? 0.f : g * kGelu * fmaf(3.f * 0.044715f, g * g, 1.f);
    dg = dy * fmaf(slope, p * (1.f - p), p);
    du = 0.f;
  }
}

template <typename T, typename At>
__device__ __forceinline__ void store_values(T* base, int64_t ld, const At& at, int i, int vec,
                                             const float (&v)[8]) {
  if (!at.has(i)) return;
  T* d = base + (at.row + i * kTileRows) * ld + at.col;
  if (At::kFull || (vec && at.width() == 8)) {
    Pack8<T> p;
    p.set(v);
    p.store(d);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < at.width()) d[j] = from_f32<T>(v[j]);
  }
}

// A block takes 32 rows of 128 columns, a thread 16 consecutive columns of one.  The results are made one
// after the other from the raw inputs, which keeps a thread within 64 registers.
constexpr int kFwdThreads = 256;
constexpr int kFwdRows = kFwdThreads / 8;
template <typename T, bool GLU>
__global__ void __launch_bounds__(kFwdThreads, sizeof(T) == 2 ? 4 : 2)
    activation_forward_kernel(const __grid_constant__ ActArgs p) {
  pdl_launch();
  Sixteen at;
  at.group = (int32_t)blockIdx.x;
  at.col = (int64_t)at.group * kGroup + (threadIdx.x & 7) * 16;
  at.width = (int)max((int64_t)0, min((int64_t)16, p.cols - at.col));
  pdl_wait();
  const int64_t row_blocks = (p.rows + kFwdRows - 1) / kFwdRows;
  for (int64_t b = blockIdx.y; b < row_blocks; b += gridDim.y) {
    at.row = b * kFwdRows + (threadIdx.x >> 3);
    at.has = at.row < p.rows;
    const int n = at.has ? at.width : 0;
    Pack8<T> graw[2], uraw[2];
    load_sixteen(graw, static_cast<const T*>(p.gate) + at.row * p.ld_gate + at.col, n, p.vec);
    if (GLU) load_sixteen(uraw, static_cast<const T*>(p.up) + at.row * p.ld_up + at.col, n, p.vec);
    {
      float y[16], u[16];
      get_sixteen(graw, y);
      if (GLU) get_sixteen(uraw, u);
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] = act<T, GLU>(y[j], GLU ? u[j] : 0.f);
      if (p.y) store_sixteen(static_cast<T*>(p.y) + at.row * p.ld_y + at.col, n, p.vec, y);
      if (p.y8.q) quantize_sixteen(at, y, eighth_warp_max(scale_part(largest(y))), p.y8);
    }
    if (p.gate8.q) {
      float g[16];
      get_sixteen(graw, g);
      quantize_sixteen(at, g, eighth_warp_max(scale_part(largest(g))), p.gate8);
    }
    if (GLU && p.up8.q) {
      float u[16];
      get_sixteen(uraw, u);
      quantize_sixteen(at, u, eighth_warp_max(scale_part(largest(u))), p.up8);
    }
  }
}

// The inputs of the tiles that a block will need next, copied ahead to shared memory as they lie in
// memory (cp.async where rows start on 16-byte boundaries).  A thread reads back only what it copied, so
// no barrier is needed.
template <typename T, bool GLU, bool KEPT>
struct Ahead {
  static constexpr int P = sizeof(T) / 2;                   // 16-byte planes of eight values
  static constexpr int kInput = KEPT ? 8 : 16 * P;          // bytes of eight values of gate or up
  static constexpr int kPass = kTileThreads * (16 * P + (GLU ? 2 : 1) * kInput);
  static constexpr int kStage = kTilePasses * kPass;
  static constexpr int kDepth = 3 * kStage <= 200 * 1024 ? 3 : 2 * kStage <= 200 * 1024 ? 2 : 1;
  static constexpr int kBytes = kDepth * kStage;
  uint32_t base;
  __device__ __forceinline__ explicit Ahead(const void* smem)
      : base((uint32_t)__cvta_generic_to_shared(smem)) {}
  // matrix m (0 dy, 1 gate, 2 up), plane q of this thread's values of pass i
  __device__ __forceinline__ uint32_t at(int stage, int i, int m, int q) const {
    return base + (uint32_t)(stage * kStage + i * kPass +
                             (m == 0 ? 0 : kTileThreads * (16 * P + (m - 1) * kInput)) +
                             q * kTileThreads * 16) +
           threadIdx.x * (m > 0 && KEPT ? 8 : 16);
  }
  template <typename At>
  __device__ __forceinline__ void copy(int stage, int m, const At& at_, const T* src, int64_t ld,
                                       int vec) const {
    const T* s = src + at_.row * ld + at_.col;
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) {
      if (vec) {
        const int left = at_.has(i) ? at_.width() * (int)sizeof(T) : 0;
#pragma unroll
        for (int q = 0; q < P; ++q) {
          const int bytes = max(0, min(16, left - 16 * q));
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, i, m, q)),
                       "l"(bytes ? reinterpret_cast<const char*>(s + i * (kTileRows * ld)) + 16 * q
                                 : reinterpret_cast<const char*>(src)),
                       "r"(bytes)
                       : "memory");
        }
      } else {
        Pack8<T> p;
        load_pass(p, at_, i, src, ld, 0);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
        for (int q = 0; q < P; ++q)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(stage, i, m, q)),
                       "r"(w[4 * q]), "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                       : "memory");
      }
    }
  }
  template <typename At>
  __device__ __forceinline__ void copy8(int stage, int m, const At& at_, const Fp8Ref& src) const {
    const uint8_t* s = src.q + at_.row * src.ld + at_.col;
#pragma unroll
    for (int i = 0; i < kTilePasses; ++i) {
      const int bytes = at_.has(i) ? at_.width() : 0;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(at(stage, i, m, 0)),
                   "l"(bytes ? s + i * (kTileRows * src.ld) : src.q), "r"(bytes)
                   : "memory");
    }
  }
  __device__ __forceinline__ void get(int stage, int i, int m, float (&v)[8]) const {
    Pack8<T> p;
    uint32_t* w = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
    for (int q = 0; q < P; ++q)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * q]), "=r"(w[4 * q + 1]), "=r"(w[4 * q + 2]), "=r"(w[4 * q + 3])
                   : "r"(at(stage, i, m, q))
                   : "memory");
    p.get(v);
  }
  __device__ __forceinline__ void get8(int stage, int i, int m, int e5m2, uint32_t byte,
                                       float (&v)[8]) const {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                 : "=r"(r.x), "=r"(r.y)
                 : "r"(at(stage, i, m, 0))
                 : "memory");
    held_values(r, e5m2, scale_value(byte), v);
  }
};

// A block walks the tiles with the next ones' inputs under way, and holds both gradients in registers
// (one after the other, with p computed twice, took a fifth more instructions).
template <typename T, bool GLU, bool KEPT>
__global__ void __launch_bounds__(kTileThreads, 1)
    activation_backward_kernel(const __grid_constant__ ActArgs p) {
  using A = Ahead<T, GLU, KEPT>;
  constexpr int D = A::kDepth;
  __shared__ __align__(16) TileSmem<GLU ? 2 : 1> sm;
  extern __shared__ uint4 ahead_smem[];
  const A in(ahead_smem);
  pdl_launch();
  pdl_wait();
  // tiles blockIdx.x, + gridDim.x, ...: a tile row and column group each, carried along (a division per
  // tile would cost as much as a tenth of the tile)
  const int32_t groups = (int32_t)((p.cols + kGroup - 1) / kGroup);
  const int32_t step_r = (int32_t)(gridDim.x / (unsigned)groups);
  const int32_t step_c = (int32_t)(gridDim.x % (unsigned)groups);
  const int64_t tile_rows = (p.rows + kGroup - 1) / kGroup;
  struct Tile {
    int64_t r;
    int32_t c;
  };
  auto after = [&](Tile t) {
    t.r += step_r;
    t.c += step_c;
    if (t.c >= groups) {
      t.c -= groups;
      ++t.r;
    }
    return t;
  };
  auto fetch = [&](const Tile& tile, int stage) {
    if (tile.r < tile_rows) {
      auto all = [&](const auto& at) {
        const int vec = at.kFull || p.vec;
        in.copy(stage, 0, at, static_cast<const T*>(p.dy), p.ld_dy, vec);
        if constexpr (KEPT) {
          in.copy8(stage, 1, at, p.gate8);
          if (GLU) in.copy8(stage, 2, at, p.up8);
        } else {
          in.copy(stage, 1, at, static_cast<const T*>(p.gate), p.ld_gate, vec);
          if (GLU) in.copy(stage, 2, at, static_cast<const T*>(p.up), p.ld_up, vec);
        }
      };
      if (full_tile(tile.r, tile.c, p.rows, p.cols, p.vec))
        all(TileAt<true>(tile.r, tile.c, p.rows, p.cols));
      else
        all(TileAt<false>(tile.r, tile.c, p.rows, p.cols));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  struct Scales {
    uint32_t s[KEPT ? kTilePasses : 1][KEPT && GLU ? 2 : 1];
  };
  auto fetch_scales = [&](const Tile& tile, Scales& v) {
    if (!KEPT || tile.r >= tile_rows) return;
    auto all = [&](const auto& at) {
      const uint8_t* g = p.gate8.s + at.row * p.gate8.ld_s + at.group;
      const uint8_t* u = GLU ? p.up8.s + at.row * p.up8.ld_s + at.group : nullptr;
#pragma unroll
      for (int i = 0; i < kTilePasses; ++i) {
        v.s[KEPT ? i : 0][0] = at.has(i) ? g[i * (kTileRows * p.gate8.ld_s)] : 127u;
        if (GLU) v.s[KEPT ? i : 0][KEPT && GLU ? 1 : 0] = at.has(i) ? u[i * (kTileRows * p.up8.ld_s)] : 127u;
      }
    };
    if (full_tile(tile.r, tile.c, p.rows, p.cols, p.vec))
      all(TileAt<true>(tile.r, tile.c, p.rows, p.cols));
    else
      all(TileAt<false>(tile.r, tile.c, p.rows, p.cols));
  };
  Tile tile{(int64_t)(blockIdx.x / (unsigned)groups), (int32_t)(blockIdx.x % (unsigned)groups)};
  Tile far = tile;                         // the next tile to copy
  Scales cur, next;
#pragma unroll
  for (int i = 0; i < D - 1; ++i, far = after(far)) fetch(far, i);
  fetch_scales(tile, next);
  for (int stage = 0; tile.r < tile_rows; stage = stage + 1 == D ? 0 : stage + 1) {
    const Tile here = tile;
    tile = after(tile);
    cur = next;
    fetch_scales(tile, next);
    fetch(far, stage == 0 ? D - 1 : stage - 1);
    far = after(far);
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    auto process = [&](const auto& at) {
      auto input = [&](int i, int m, float (&v)[8]) {
        if constexpr (KEPT)
          in.get8(stage, i, m, m == 1 ? p.gate8.e5m2 : p.up8.e5m2, cur.s[i][GLU ? m - 1 : 0], v);
        else
          in.get(stage, i, m, v);
      };
      auto emit = [&](TileValues& v, void* out, int64_t ld, const Fp8Ref& row) {
        if (out)
#pragma unroll
          for (int i = 0; i < kTilePasses; ++i)
            store_values(static_cast<T*>(out), ld, at, i, p.vec, v[i]);
        if (row.q)
#pragma unroll
          for (int i = 0; i < kTilePasses; i += 2) quantize_rows(at, i, v[i], v[i + 1], row);
      };
      TileValues dg, du;
#pragma unroll
      for (int i = 0; i < kTilePasses; ++i) {
        float d[8], g[8], u[8];
        in.get(stage, i, 0, d);
        input(i, 1, g);
        if constexpr (GLU) input(i, 2, u);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          act_grads<T, GLU>(d[j], g[j], GLU ? u[j] : 0.f, dg[i][j], du[i][j]);
      }
      emit(dg, p.dgate, p.ld_dgate, p.dgate_row);
      if (GLU) emit(du, p.dup, p.ld_dup, p.dup_row);
      if constexpr (GLU) {
        if (p.dgate_col.q && p.dup_col.q) quantize_cols<2>(at, sm, {&p.dgate_col, &p.dup_col}, {&dg, &du});
        else if (p.dgate_col.q) quantize_cols<1>(at, sm, {&p.dgate_col}, {&dg});
        else if (p.dup_col.q) quantize_cols<1>(at, sm, {&p.dup_col}, {&du});
      } else {
        if (p.dgate_col.q) quantize_cols<1>(at, sm, {&p.dgate_col}, {&dg});
      }
    };
    if (full_tile(here.r, here.c, p.rows, p.cols, p.vec))
      process(TileAt<true>(here.r, here.c, p.rows, p.cols));
    else
      process(TileAt<false>(here.r, here.c, p.rows, p.cols));
  }
}

template <typename T, bool GLU, bool KEPT>
cudaError_t launch_backward(const ActArgs& a, int sms, cudaStream_t st) {
  static std::atomic<bool> done[64];
  constexpr int smem = Ahead<T, GLU, KEPT>::kBytes;
  const auto kernel = activation_backward_kernel<T, GLU, KEPT>;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !done[dev].load())) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) done[dev].store(true);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)std::min<int64_t>(a.tiles, sms)), dim3(kTileThreads), smem, st,
                    a);
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
  if (!distinct({y, data_of(y8), bytes_of(y8), data_of(gate8), bytes_of(gate8), data_of(up8), bytes_of(up8)}))
    return MFSDP_EINVAL;
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
  const dim3 grid((unsigned)((cols + kGroup - 1) / kGroup),
                  (unsigned)std::min<int64_t>((rows + kFwdRows - 1) / kFwdRows, 65535));
  const dim3 block(kFwdThreads);
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
  const std::initializer_list<const void*> results = {
      dgate, dup, data_of(dgate_row), bytes_of(dgate_row), data_of(dgate_col), bytes_of(dgate_col),
      data_of(dup_row), bytes_of(dup_row), data_of(dup_col), bytes_of(dup_col)};
  if (!distinct(results) || !apart(results, {data_of(gate8), bytes_of(gate8), data_of(up8), bytes_of(up8)}))
    return MFSDP_EINVAL;
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
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == MFSDP_DTYPE_BF16;
  cudaError_t e;
  if (gate8)
    e = glu ? (bf ? launch_backward<bf16_t, true, true>(a, sms, st)
                  : launch_backward<float, true, true>(a, sms, st))
            : (bf ? launch_backward<bf16_t, false, true>(a, sms, st)
                  : launch_backward<float, false, true>(a, sms, st));
  else
    e = glu ? (bf ? launch_backward<bf16_t, true, false>(a, sms, st)
                  : launch_backward<float, true, false>(a, sms, st))
            : (bf ? launch_backward<bf16_t, false, false>(a, sms, st)
                  : launch_backward<float, false, false>(a, sms, st));
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}
