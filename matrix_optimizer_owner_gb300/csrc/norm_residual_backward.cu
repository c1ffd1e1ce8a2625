// Backward pass of the norm with a residual, from h as it was kept or from its 8-bit checkpoint.
//
// With z = (h - mu) s and g = dy w, per row of n elements:
//     dx = s (g - sum(g) / n [layer] - z sum(g z) / n) + dres,  dw = sum_rows dy z,  db = sum_rows dy
// dx is the gradient of x and of r.  Bound by memory: a persistent grid walks the rows, each in registers
// over a warp (up to 1024 elements) or a block, with the next rows under way to shared memory; a block's
// column sums stay in registers and are joined by a second launch, in block order.  8192 x 4096 bf16, RMS:
// 51 us, 5.3 TB/s; 16384 x 768, layer norm from the checkpoint: 24 us, 3.7 TB/s, where the sums leave
// registers for one block of eight warps an SM (twelve: 22 us here, and 8.7 instead of 6.1 for 2000 rows).
#include <algorithm>
#include <type_traits>

#include "norm_residual.cuh"

namespace mfsdp {
namespace {

// The rows a thread will need next, copied ahead to shared memory as they lie in memory (dy, dres and
// h or its 8-bit checkpoint; cp.async where rows start on 16-byte boundaries).  A thread reads back
// only what it copied, so no barrier is needed.
template <typename T, int TPR, int K, bool H8>
struct Rows {
  static constexpr int kThreads = TPR == 32 ? 32 * kNormWarps : TPR;
  static constexpr int P = sizeof(T) / 2;                     // 16-byte planes of a chunk
  static constexpr int kChunk = kThreads * (16 * P * (H8 ? 2 : 3) + (H8 ? 8 : 0));
  static constexpr int kStage = K * kChunk;
  // rows a turn: blocks of 128 and 256 threads share the sums' shuffles and barrier between two
  static constexpr int NR = (TPR == 128 || TPR == 256) && sizeof(T) == 2 ? 2 : 1;
  static constexpr int kDepth = kStage * 4 <= 96 * 1024 ? 4 : kStage * 3 <= 96 * 1024 ? 3 : 2;
  static_assert(kDepth > NR || NR == 1, "a turn's rows beside the next one's");
  static constexpr int kBytes = kDepth * kStage;
  uint32_t base;
  __device__ __forceinline__ explicit Rows(const void* smem)
      : base((uint32_t)__cvta_generic_to_shared(smem)) {}
  // matrix m (0 dy, 1 dres, 2 h), plane i
  __device__ __forceinline__ uint32_t at(int stage, int k, int m, int i) const {
    return base + (uint32_t)(stage * kStage + k * kChunk + (m * P + i) * kThreads * 16) +
           threadIdx.x * (H8 && m == 2 ? 8 : 16);
  }
  __device__ __forceinline__ void copy(int stage, int k, int m, const T* row, int64_t c, int64_t n,
                                       int vec) const {
    if (vec) {
      const int left = c < n ? (int)min((int64_t)8, n - c) * (int)sizeof(T) : 0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int bytes = max(0, min(16, left - 16 * i));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, k, m, i)),
                     "l"(bytes ? reinterpret_cast<const char*>(row + c) + 16 * i
                               : reinterpret_cast<const char*>(row)),
                     "r"(bytes)
                     : "memory");
      }
      return;
    }
    Pack8<T> p;
    load_chunk(p, row, c, (int)max((int64_t)0, min((int64_t)8, n - c)), 0);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
    for (int i = 0; i < P; ++i)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(stage, k, m, i)), "r"(w[4 * i]),
                   "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                   : "memory");
  }
  __device__ __forceinline__ void copy8(int stage, int k, const uint8_t* row, int64_t c,
                                        int64_t n) const {
    const int bytes = c < n ? (int)min((int64_t)8, n - c) : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(at(stage, k, 2, 0)),
                 "l"(row + (bytes ? c : 0)), "r"(bytes)
                 : "memory");
  }
  __device__ __forceinline__ void commit() const {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void wait() const {              // the NR oldest groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - NR) : "memory");
  }
  __device__ __forceinline__ void get(int stage, int k, int m, float (&v)[8]) const {
    Pack8<T> p;
    uint32_t* w = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
    for (int i = 0; i < P; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(at(stage, k, m, i))
                   : "memory");
    p.get(v);
  }
  __device__ __forceinline__ void get8(int stage, int k, int e5m2, float (&v)[8]) const {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                 : "=r"(r.x), "=r"(r.y)
                 : "r"(at(stage, k, 2, 0))
                 : "memory");
    unpack_fp8(r, e5m2, v);
  }
};

template <typename T, int TPR, int K, bool H8, bool LAYER>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kNormWarps : TPR)
    norm_residual_backward_kernel(const __grid_constant__ NrArgs p) {
  using R = Rows<T, TPR, K, H8>;
  constexpr int NR = R::NR, D = R::kDepth;
  constexpr int kRowsPerBlock = TPR == 32 ? kNormWarps : 1;
  __shared__ __align__(16) float red[TPR == 32 ? 4 : 8 * (TPR / 32)];
  __shared__ float comb[TPR == 32 ? kNormWarps * 32 * 8 : 1];
  // Warps that hold a row each share the weight in shared memory, where they read it as it is used: in
  // registers beside two sums per column it would leave one block an SM.
  constexpr bool kSharedW = TPR == 32;
  __shared__ __align__(16) float weight[kSharedW ? kWarpRowMax : 4];
  extern __shared__ uint4 ring_smem[];
  pdl_launch();
  pdl_wait();
  const int t = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int sub = TPR == 32 ? (threadIdx.x >> 5) : 0;
  const int64_t n = p.cols, step = (int64_t)gridDim.x * kRowsPerBlock;
  int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + sub;
  int turn = 0;
  const R ring(ring_smem);
  struct Stat {
    float rstd, mean;
    uint32_t byte[H8 ? K : 1];            // the scales of this thread's groups
  };
  auto fetch = [&](int64_t i, int stage) {
    if (i < p.rows)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int64_t c = elem_of<TPR, true>(t, k, 0);
        ring.copy(stage, k, 0, static_cast<const T*>(p.dy) + i * p.ld_dy, c, n, p.vec);
        if (p.dres) ring.copy(stage, k, 1, static_cast<const T*>(p.dres) + i * p.ld_dres, c, n, p.vec);
        if (H8) ring.copy8(stage, k, p.h8.q + i * p.h8.ld, c, n);
        else ring.copy(stage, k, 2, static_cast<const T*>(p.h_in) + i * p.ld_h, c, n, p.vec);
      }
    ring.commit();
  };
  auto fetch_stats = [&](int64_t i, Stat& s) {
    if (i >= p.rows) return;
    s.rstd = p.rstd_in[i];
    s.mean = LAYER ? p.mean_in[i] : 0.f;
    if (H8)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int64_t c = elem_of<TPR, true>(t, k, 0);
        s.byte[H8 ? k : 0] = c < n ? p.h8.s[i * p.h8.ld_s + c / kGroup] : 127u;
      }
  };
  auto wrap = [](int stage) { return stage >= D ? stage - D : stage; };
  Stat stat[NR], next[NR];
#pragma unroll
  for (int i = 0; i < D - NR; ++i) fetch(row + i * step, i);
#pragma unroll
  for (int i = 0; i < NR; ++i) fetch_stats(row + i * step, next[i]);
  float aw[K][8], ab[LAYER ? K : 1][8], w[kSharedW ? 1 : K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[k][j] = ab[LAYER ? k : 0][j] = 0.f;
  if constexpr (kSharedW) {
    for (int e = threadIdx.x; e < kWarpRowMax; e += 32 * kNormWarps)
      weight[e] = p.w && e < n ? load_param(p.w, p.wbf16, e) : 1.f;
    __syncthreads();
  } else {
    load_params<TPR, K, true>(p.w, p.wbf16, p.pvec, n, t, 1.f, w);
  }
  auto weights = [&](int k, float (&v)[8]) {
    if constexpr (kSharedW) {
      Pack8<float> q;
      q.load(weight + elem_of<TPR, true>(t, k, 0));
      q.get(v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = w[k][j];
    }
  };
  auto values = [&](int st, const Stat& s, int k, float (&z)[8], float (&g)[8]) {
    // (an 8-bit h takes its scale and rstd in one factor: a power of two changes no rounding)
    float f = s.rstd;
    if (H8) {
      f *= scale_value(s.byte[H8 ? k : 0]);
      ring.get8(st, k, p.h8.e5m2, z);
    } else {
      ring.get(st, k, 2, z);
    }
    ring.get(st, k, 0, g);
    const float shift = -s.mean * s.rstd;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = LAYER ? fmaf(z[j], f, shift) : z[j] * f;
  };
  // a chunk's part of the row's sums and of the columns' (past the row's end dy is 0)
  auto add = [&](int k, const float (&z)[8], float (&g)[8], float2& s) {
    float wk[8];
    weights(k, wk);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      aw[k][j] = fmaf(g[j], z[j], aw[k][j]);
      if (LAYER) ab[LAYER ? k : 0][j] += g[j];
      g[j] *= wk[j];
      if (LAYER) s.x += g[j];
      s.y = fmaf(g[j], z[j], s.y);
    }
  };
  // (`weighted`: g holds g w already)
  auto finish = [&](int st, int k, int64_t i, const float (&z)[8], float (&g)[8], const float2& s,
                    float r, auto weighted) {
    const float s1 = LAYER ? s.x * p.inv_n : 0.f, s2 = s.y * p.inv_n;
    float d[8];
    if constexpr (!decltype(weighted)::value) {
      float wk[8];
      weights(k, wk);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = fmaf(g[j], wk[j], -s1);
    } else if (LAYER) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] -= s1;
    }
    if (p.dres) {
      ring.get(st, k, 1, d);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = fmaf(fmaf(-z[j], s2, g[j]), r, d[j]);
    {
      const int64_t c = elem_of<TPR, true>(t, k, 0);
      store_part(static_cast<T*>(p.dx) + i * p.ld_dx, c, (int)(n - c), p.vec, g);
    }
  };
  for (int stage = 0; row < p.rows; row += NR * step, stage = wrap(stage + NR)) {
    // the second row of the turn, if there is one (the same for the whole group)
    const bool two = NR == 2 && row + step < p.rows;
    const int other = wrap(stage + 1);
#pragma unroll
    for (int i = 0; i < NR; ++i) stat[i] = next[i];
#pragma unroll
    for (int i = 0; i < NR; ++i) fetch_stats(row + (NR + i) * step, next[i]);
#pragma unroll
    for (int i = 0; i < NR; ++i) fetch(row + (D - NR + i) * step, wrap(stage + D - NR + i));
    ring.wait();
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
    if constexpr (TPR == 32) {
      // a warp's row: z and g w stay in registers over the row's sums
      float z[K][8], g[K][8];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        values(stage, stat[0], k, z[k], g[k]);
        add(k, z[k], g[k], s0);
      }
      row_sum2<TPR>(s0.x, s0.y, red, turn);
#pragma unroll
      for (int k = 0; k < K; ++k)
        finish(stage, k, row, z[k], g[k], s0, stat[0].rstd, std::true_type());
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float z[8], g[8];
        values(stage, stat[0], k, z, g);
        add(k, z, g, s0);
        if (two) {
          values(other, stat[NR - 1], k, z, g);
          add(k, z, g, s1);
        }
      }
      if (NR == 2) row_sum4<TPR>(s0, s1, red, turn);
      else row_sum2<TPR>(s0.x, s0.y, red, turn);
      // (read from the ring again rather than kept: fewer registers, more warps)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float z[8], g[8];
        values(stage, stat[0], k, z, g);
        finish(stage, k, row, z, g, s0, stat[0].rstd, std::false_type());
        if (two) {
          values(other, stat[NR - 1], k, z, g);
          finish(other, k, row + step, z, g, s1, stat[NR - 1].rstd, std::false_type());
        }
      }
    }
  }
  // this block's column sums, its warps added in warp order
  float* part = p.partials + (int64_t)blockIdx.x * 2 * n;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!(h == 0 ? p.has_dw : LAYER && p.has_db)) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (TPR == 32) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          comb[(sub * 8 + j) * 32 + t] = h == 0 ? aw[k][j] : ab[LAYER ? k : 0][j];
        __syncthreads();
        // thread (sub, t) adds element j = sub of lane t over the warps
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kNormWarps; ++i) s += comb[(i * 8 + sub) * 32 + t];
        const int64_t e = elem_of<TPR, true>(t, k, sub);
        if (e < n) part[h * n + e] = s;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t e = elem_of<TPR, true>(t, k, j);
          if (e < n) part[h * n + e] = h == 0 ? aw[k][j] : ab[LAYER ? k : 0][j];
        }
      }
    }
  }
}

// Rows too long for registers: the two row sums, then dx; a block owns whole rows, and its
// column sums live in the workspace (only this block's threads touch its slice).
template <typename T>
__global__ void __launch_bounds__(1024)
    norm_residual_backward_long_kernel(const __grid_constant__ NrArgs p) {
  __shared__ float red[4 * 32];
  pdl_launch();
  pdl_wait();
  const int64_t n = p.cols;
  int turn = 0;
  float* part = p.partials + (int64_t)blockIdx.x * 2 * n;
  for (int64_t e = threadIdx.x; e < n; e += 1024) part[e] = part[n + e] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* gr = static_cast<const T*>(p.dy) + row * p.ld_dy;
    const T* er = p.dres ? static_cast<const T*>(p.dres) + row * p.ld_dres : nullptr;
    T* dr = static_cast<T*>(p.dx) + row * p.ld_dx;
    const float r = p.rstd_in[row], mu = p.layer ? p.mean_in[row] : 0.f;
    auto zed = [&](int64_t e) {
      float h;
      if (p.h8.q) {
        float v[8];
        unpack_fp8(make_uint2(p.h8.q[row * p.h8.ld + e], 0u), p.h8.e5m2, v);
        h = v[0] * scale_value(p.h8.s[row * p.h8.ld_s + e / kGroup]);
      } else {
        h = to_f32((static_cast<const T*>(p.h_in) + row * p.ld_h)[e]);
      }
      return (h - mu) * r;
    };
    float s1 = 0.f, s2 = 0.f;
    for (int64_t e = threadIdx.x; e < n; e += 1024) {
      const float z = zed(e), d = to_f32(gr[e]);
      part[e] = fmaf(d, z, part[e]);
      part[n + e] += d;
      const float g = p.w ? d * load_param(p.w, p.wbf16, e) : d;
      s1 += g;
      s2 = fmaf(g, z, s2);
    }
    row_sum2<1024>(s1, s2, red, turn);
    s1 = p.layer ? s1 * p.inv_n : 0.f;
    s2 *= p.inv_n;
    for (int64_t e = threadIdx.x; e < n; e += 1024) {
      const float z = zed(e), d = to_f32(gr[e]);
      const float g = p.w ? d * load_param(p.w, p.wbf16, e) : d;
      dr[e] = from_f32<T>(fmaf(g - s1 - z * s2, r, er ? to_f32(er[e]) : 0.f));
    }
  }
}

// TPR and K are the smallest that hold the row; f is called with the kernel's shape.
template <typename T, typename F>
cudaError_t by_row_shape(int64_t cols, F&& f) {
  if (cols <= 256) return f.template operator()<T, 32, 1>();
  if (cols <= 512) return f.template operator()<T, 32, 2>();
  if (cols <= 768) return f.template operator()<T, 32, 3>();
  if (cols <= kWarpRowMax) return f.template operator()<T, 32, 4>();
  if (cols <= 2048) return f.template operator()<T, 128, 2>();
  if (cols <= 4096) return f.template operator()<T, 256, 2>();
  return f.template operator()<T, 512, 2>();
}

template <bool H8, bool LAYER>
struct NrBackward {
  const NrArgs& a;
  int max_blocks, sms;
  cudaStream_t st;
  int* blocks;
  template <typename T, int TPR, int K>
  cudaError_t operator()() const {
    const int threads = TPR == 32 ? 32 * kNormWarps : TPR;
    constexpr int smem = Rows<T, TPR, K, H8>::kBytes;
    const auto kernel = norm_residual_backward_kernel<T, TPR, K, H8, LAYER>;
    static std::atomic<int> cache[kCachedDevices];
    const int occ = resident(cache, kernel, threads, smem);
    const int64_t per = TPR == 32 ? kNormWarps : 1, need = (a.rows + per - 1) / per;
    const int64_t g = std::min({(int64_t)sms * occ, (int64_t)max_blocks, need});
    *blocks = (int)g;
    return launch_pdl(kernel, dim3((unsigned)g), dim3(threads), smem, st, a);
  }
};
template <bool H8>
cudaError_t launch_backward(const NrArgs& a, bool bf, int max_blocks, int sms, cudaStream_t st,
                            int* blocks) {
  if (a.layer) {
    const NrBackward<H8, true> f{a, max_blocks, sms, st, blocks};
    return bf ? by_row_shape<bf16_t>(a.cols, f) : by_row_shape<float>(a.cols, f);
  }
  const NrBackward<H8, false> f{a, max_blocks, sms, st, blocks};
  return bf ? by_row_shape<bf16_t>(a.cols, f) : by_row_shape<float>(a.cols, f);
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" int mfsdp_norm_residual_backward(
    int32_t kind, int64_t rows, int64_t cols, int32_t dtype, int32_t param_dtype, const void* dy,
    int64_t ld_dy, const void* dres, int64_t ld_dres, const void* h, int64_t ld_h,
    const mfsdp_fp8_matrix* h8, const void* weight, const float* mean, const float* rstd, void* dx,
    int64_t ld_dx, void* dweight, void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  int chk = check_shape(kind, rows, cols, dtype, param_dtype);
  if (chk != MFSDP_OK) return chk;
  if (kind == MFSDP_NORM_RMS && (mean || dbias)) return MFSDP_EINVAL;
  if (h && h8) return MFSDP_EINVAL;
  if (h8 && (chk = check_fp8(*h8, rows, cols, MFSDP_GROUPS_ROW)) != MFSDP_OK) return chk;
  if (rows > 0 && (!dy || (!h && !h8) || !dx || !rstd || (kind == MFSDP_NORM_LAYER && !mean) ||
                   ld_dy < cols || (dres && ld_dres < cols) || (h && ld_h < cols) || ld_dx < cols))
    return MFSDP_EINVAL;
  if (!workspace) return MFSDP_EINVAL;
  const size_t es = dtype_bytes(dtype), ps = dtype_bytes(param_dtype);
  if (!aligned_to(dy, es) || !aligned_to(dres, es) || !aligned_to(h, es) || !aligned_to(dx, es) ||
      !aligned_to(weight, ps) || !aligned_to(dweight, ps) || !aligned_to(dbias, ps) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(workspace, 256))
    return MFSDP_EALIGN;
  size_t need = 0;
  mfsdp_norm_backward_workspace_bytes(rows, cols, &need);
  if (workspace_bytes < need) return MFSDP_EWORKSPACE;
  if (!distinct({dx, dweight, dbias})) return MFSDP_EINVAL;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  NrArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.dy = dy;
  a.ld_dy = ld_dy;
  a.dres = dres;
  a.ld_dres = ld_dres;
  a.h_in = h;
  a.ld_h = ld_h;
  a.h8 = ref_of(h8);
  a.w = weight;
  a.dx = dx;
  a.ld_dx = ld_dx;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.partials = static_cast<float*>(workspace);
  a.inv_n = (float)(1.0 / (double)cols);
  a.layer = kind == MFSDP_NORM_LAYER;
  a.wbf16 = param_dtype == MFSDP_DTYPE_BF16;
  a.pvec = cols % 8 == 0 && aligned_to(weight, 16);
  a.vec = vector_rows(dy, ld_dy, dtype) && vector_rows(dx, ld_dx, dtype) &&
          (!dres || vector_rows(dres, ld_dres, dtype)) && (!h || vector_rows(h, ld_h, dtype));
  a.has_dw = dweight != nullptr;
  a.has_db = dbias != nullptr;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == MFSDP_DTYPE_BF16;
  cudaError_t e = cudaSuccess;
  int blocks = 0;
  if (rows > 0) {
    if (cols > kRegRowMax) {
      blocks = std::min(blocks_bound(rows), sms);
      e = bf ? launch_pdl(norm_residual_backward_long_kernel<bf16_t>, dim3(blocks), dim3(1024), 0, st, a)
             : launch_pdl(norm_residual_backward_long_kernel<float>, dim3(blocks), dim3(1024), 0, st, a);
    } else {
      e = h8 ? launch_backward<true>(a, bf, blocks_bound(rows), sms, st, &blocks)
             : launch_backward<false>(a, bf, blocks_bound(rows), sms, st, &blocks);
    }
  }
  if (e == cudaSuccess && (dweight || dbias)) {
    const dim3 grid((unsigned)((cols + 31) / 32), 2);
    e = param_dtype == MFSDP_DTYPE_BF16
            ? launch_pdl(norm_param_grad_kernel<bf16_t>, grid, dim3(1024), 0, st, a.partials,
                         blocks, cols, static_cast<bf16_t*>(dweight), static_cast<bf16_t*>(dbias))
            : launch_pdl(norm_param_grad_kernel<float>, grid, dim3(1024), 0, st, a.partials,
                         blocks, cols, static_cast<float*>(dweight), static_cast<float*>(dbias));
  }
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}
