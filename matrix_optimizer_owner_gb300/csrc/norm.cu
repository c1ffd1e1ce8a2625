// Layer norm and RMS norm of the rows of a matrix, forward and backward.
//
// Forward, per row x of n elements (layer norm; RMS norm has mu = 0 and no bias):
//     mu = sum(x) / n,  r = 1 / sqrt(sum((x - mu)^2) / n + eps),  y = (x - mu) r w + b.
// The row is held in registers, so it is read once, and the squares are summed of the centred
// values (no cancellation of large means).  Backward, with z = (x - mu) r and g = dy w:
//     dx = r (g - sum(g) / n [layer] - z sum(g z) / n),  dw = sum_rows dy z,  db = sum_rows dy.
//
// Both directions are bound by memory: forward moves 2 and backward 3 values per element.  Rows of
// up to 1024 elements take a warp each (no block barrier), longer ones a block with 16 elements
// per thread; rows beyond 8192 elements are read in passes.  A persistent grid walks the rows with
// the parameters in registers.  Backward keeps every column's dw and db sums in registers over the
// rows a block walks; the blocks' sums go to the workspace and a second launch adds them in block
// order: no atomics, the result does not depend on timing.
//
// Measured (bf16, all launches of both passes by graph replay, 6.78 TB/s being a copy's rate):
// 16384 rows of 768 in 29 us, 3.5 TB/s of the 101 MB that have to move (15 us); 8192 rows of 4096
// in 67 us, 4.0 TB/s of 268 MB (40 us).  What remains is latency: in the backward kernel memory is
// busy half of the time, and the warps wait on the row sums' shuffles and shared-memory reads.  A
// group of warps per row with one chunk per thread instead, for more warps, was slower at every
// width (768: 65 us, 4096: 145).
#include <algorithm>

#include "norm_rows.cuh"

namespace mfsdp {
namespace {

struct NormArgs {
  int64_t rows, cols;
  const void *x, *dy;
  const void *w, *b;          // nullable
  void *y, *dx;
  int64_t ld_x, ld_y, ld_dy, ld_dx;
  float *mean, *rstd;         // forward: nullable outputs
  const float *mean_in, *rstd_in;
  float* partials;            // [blocks][2][cols]
  float eps, inv_n;
  int layer, wbf16, has_dw, has_db;
  int pvec;                   // the parameters start on 16-byte boundaries
};

template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int64_t n, int t, int k, const float (&v)[8]) {
  if (VEC) {
    const int64_t e = elem_of<TPR, VEC>(t, k, 0);
    Pack8<T> p;
    p.set(v);
    if (e < n) p.store(row + e);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = elem_of<TPR, VEC>(t, k, j);
      if (e < n) row[e] = from_f32<T>(v[j]);
    }
  }
}

// The bf16 rows a thread will need next, as they lie in memory: N matrices (x, or x and dy) with
// K chunks of 8 elements each, copied ahead to shared memory (cp.async, kDepth rows deep).  A
// thread reads back only what it copied, so no barrier is needed, and the bytes in flight do not
// cost registers: with one row ahead in registers, 24 KB per SM were in flight and the 768-wide
// backward pass stayed at 3.8 TB/s.
template <int N, int TPR, int K>
struct Ring {
  static constexpr int kThreads = TPR == 32 ? 32 * kNormWarps : TPR;
  static constexpr int kStage = N * K * kThreads * 16;
  static constexpr int kDepth = kStage * 4 <= 96 * 1024 ? 4 : kStage * 3 <= 96 * 1024 ? 3 : 2;
  static constexpr int kBytes = kDepth * kStage;
  uint32_t base;
  __device__ __forceinline__ explicit Ring(const void* smem) {
    base = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
  }
  __device__ __forceinline__ uint32_t at(int stage, int m, int k) const {
    return base + (uint32_t)(((stage * N + m) * K + k) * kThreads * 16);
  }
  // one matrix's row into a stage; chunks past the end are zero
  __device__ __forceinline__ void copy(int stage, int m, const void* mat, int64_t at_row, int n,
                                       int t) const {
    const bf16_t* row = static_cast<const bf16_t*>(mat) + at_row;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int e = (k * TPR + t) * 8;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, m, k)),
                   "l"(row + (e < n ? e : 0)), "r"(e < n ? 16 : 0)
                   : "memory");
    }
  }
  __device__ __forceinline__ void commit() const {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the NR oldest of kDepth groups have landed
  template <int NR>
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - NR) : "memory");
  }
  __device__ __forceinline__ void get(int stage, int m, int k, float (&v)[8]) const {
    Pack8<bf16_t> p;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(p.a.x), "=r"(p.a.y), "=r"(p.a.z), "=r"(p.a.w)
                 : "r"(at(stage, m, k))
                 : "memory");
    p.get(v);
  }
};

// A thread's share of a row in registers.
template <typename T, int TPR, int K, bool VEC>
struct RowChunks {
  Pack8<T> p[VEC ? K : 1];
  T e[VEC ? 1 : K][8];
  __device__ __forceinline__ void load(const T* row, int64_t n, int t) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (VEC) {
        const int64_t c = elem_of<TPR, VEC>(t, k, 0);
        if (c < n) p[VEC ? k : 0].load(row + c); else p[VEC ? k : 0].zero();
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t c = elem_of<TPR, VEC>(t, k, j);
          e[VEC ? 0 : k][j] = c < n ? row[c] : from_f32<T>(0.f);
        }
      }
    }
  }
  __device__ __forceinline__ void get(int k, float (&v)[8]) const {
    if (VEC) {
      p[VEC ? k : 0].get(v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = to_f32(e[VEC ? 0 : k][j]);
    }
  }
};

// bf16 rows of vectors go through the ring.  fp32 rows are faster in registers: 8192 rows of 2048
// took 79 us for both passes, through the ring 106 (bf16: 54 and 50).
template <typename T, bool VEC>
constexpr bool kRing = VEC && sizeof(T) == 2;

// ---------------------------------------------------------------- forward
template <typename T, int TPR, int K, bool VEC>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kNormWarps : TPR)
    norm_forward_kernel(const __grid_constant__ NormArgs p) {
  constexpr int kRowsPerBlock = TPR == 32 ? kNormWarps : 1;
  __shared__ float red[TPR == 32 ? 1 : 4 * (TPR / 32)];
  pdl_launch();
  pdl_wait();
  const int t = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * kRowsPerBlock;
  int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + (TPR == 32 ? (threadIdx.x >> 5) : 0);
  int turn = 0;
  extern __shared__ uint4 ring_smem[];
  constexpr bool kUseRing = kRing<T, VEC>;
  using R = Ring<1, TPR, K>;
  const R ring(ring_smem);
  RowChunks<T, TPR, kUseRing ? 1 : K, VEC> cur, nxt;
  auto fetch = [&](int64_t i, int stage) {
    if (i < p.rows) ring.copy(stage, 0, p.x, i * p.ld_x, (int)p.cols, t);
    ring.commit();
  };
  if (kUseRing) {
#pragma unroll
    for (int i = 0; i < R::kDepth - 1; ++i) fetch(row + i * step, i);
  } else if (row < p.rows) {
    cur.load(static_cast<const T*>(p.x) + row * p.ld_x, p.cols, t);
  }
  float w[K][8], b[K][8];
  load_params<TPR, K, VEC>(p.w, p.wbf16, p.pvec, p.cols, t, 1.f, w);
  load_params<TPR, K, VEC>(p.b, p.wbf16, p.pvec, p.cols, t, 0.f, b);
  int stage = 0;
  for (; row < p.rows; row += step) {     // whole warps (or the whole block) stay together
    if (kUseRing) {
      fetch(row + (R::kDepth - 1) * step, stage == 0 ? R::kDepth - 1 : stage - 1);
      ring.template wait<1>();
    } else if (row + step < p.rows) {
      nxt.load(static_cast<const T*>(p.x) + (row + step) * p.ld_x, p.cols, t);
    }
    float v[K][8];
    float s = 0.f, zero = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (kUseRing) ring.get(stage, 0, k, v[k]); else cur.get(kUseRing ? 0 : k, v[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[k][j];
    }
    float mu = 0.f;
    if (p.layer) {
      row_sum2<TPR>(s, zero, red, turn);
      mu = s * p.inv_n;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = elem_of<TPR, VEC>(t, k, j) < p.cols ? v[k][j] - mu : 0.f;
        q = fmaf(d, d, q);
      }
    zero = 0.f;
    row_sum2<TPR>(q, zero, red, turn);
    const float r = rsqrtf(fmaf(q, p.inv_n, p.eps));
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = r;
    }
    T* yr = static_cast<T*>(p.y) + row * p.ld_y;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = fmaf((v[k][j] - mu) * r, w[k][j], b[k][j]);
      store_chunk<T, TPR, VEC>(yr, p.cols, t, k, v[k]);
    }
    if (!kUseRing) cur = nxt;
    stage = stage == R::kDepth - 1 ? 0 : stage + 1;
  }
}

// Rows too long for registers: three passes over the row (the second and third hit the L2).
template <typename T>
__global__ void __launch_bounds__(1024) norm_forward_long_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[4 * 32];
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(p.x) + row * p.ld_x;
  T* yr = static_cast<T*>(p.y) + row * p.ld_y;
  int turn = 0;
  float mu = 0.f, zero = 0.f;
  if (p.layer) {
    float s = 0.f;
    for (int64_t e = threadIdx.x; e < p.cols; e += 1024) s += to_f32(xr[e]);
    row_sum2<1024>(s, zero, red, turn);
    mu = s * p.inv_n;
  }
  float q = 0.f;
  zero = 0.f;
  for (int64_t e = threadIdx.x; e < p.cols; e += 1024) {
    const float d = to_f32(xr[e]) - mu;
    q = fmaf(d, d, q);
  }
  row_sum2<1024>(q, zero, red, turn);
  const float r = rsqrtf(fmaf(q, p.inv_n, p.eps));
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = r;
  }
  for (int64_t e = threadIdx.x; e < p.cols; e += 1024) {
    const float w = p.w ? load_param(p.w, p.wbf16, e) : 1.f;
    const float b = p.b ? load_param(p.b, p.wbf16, e) : 0.f;
    yr[e] = from_f32<T>(fmaf((to_f32(xr[e]) - mu) * r, w, b));
  }
}

// ---------------------------------------------------------------- backward
template <typename T, int TPR, int K, bool VEC>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kNormWarps : TPR,
                                  TPR == 32 ? 1 : TPR == 256 && sizeof(T) == 2 && VEC ? 3 : 512 / TPR)
    norm_backward_kernel(const __grid_constant__ NormArgs p) {
  constexpr int kRowsPerBlock = TPR == 32 ? kNormWarps : 1;
  __shared__ __align__(16) float red[TPR == 32 ? 4 : 8 * (TPR / 32)];
  __shared__ float comb[TPR == 32 ? kNormWarps * 32 * 8 : 1];
  pdl_launch();
  pdl_wait();
  const int t = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int sub = TPR == 32 ? (threadIdx.x >> 5) : 0;
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * kRowsPerBlock;
  int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + sub;
  float aw[K][8], ab[K][8], w[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[k][j] = ab[k][j] = 0.f;
  // a chunk's part of the row's sums and of the columns' (past the row's end dy is 0)
  auto add = [&](int k, const float (&z)[8], float (&g)[8], float2& s) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      aw[k][j] = fmaf(g[j], z[j], aw[k][j]);
      ab[k][j] += g[j];
      g[j] *= w[k][j];
      s.x += g[j];
      s.y = fmaf(g[j], z[j], s.y);
    }
  };
  auto finish = [&](int k, int64_t i, const float (&z)[8], float (&g)[8], const float2& s, float r) {
    const float s1 = p.layer ? s.x * p.inv_n : 0.f, s2 = s.y * p.inv_n;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = (fmaf(g[j], w[k][j], -s1) - z[j] * s2) * r;
    store_chunk<T, TPR, VEC>(static_cast<T*>(p.dx) + i * p.ld_dx, p.cols, t, k, g);
  };
  float2 stat[2], stat_next[2];            // (rstd, mean) of the rows, fetched ahead too
  auto fetch_stats = [&](int64_t i, float2& v) {
    if (i < p.rows) v = make_float2(p.rstd_in[i], p.layer ? p.mean_in[i] : 0.f);
  };
  if constexpr (kRing<T, VEC>) {
    // Blocks of 128 and 256 threads take two rows at a time: the sums' shuffles, shared-memory
    // reads and barrier are what their warps wait for, and one set of them serves both (8192 rows
    // of 4096: 79 -> 73 us for both passes; a warp per row 28 -> 30, 512 threads per row 90 ->
    // 96).  z and g are read from the ring again after the sums rather than kept across them:
    // fewer registers, more warps.
    constexpr int NR = TPR == 128 || TPR == 256 ? 2 : 1;
    extern __shared__ uint4 ring_smem[];
    using R = Ring<2, TPR, K>;
    const R ring(ring_smem);
    auto fetch = [&](int64_t i, int stage) {
      if (i < p.rows) {
        ring.copy(stage, 0, p.x, i * p.ld_x, (int)p.cols, t);
        ring.copy(stage, 1, p.dy, i * p.ld_dy, (int)p.cols, t);
      }
      ring.commit();
    };
    auto wrap = [](int stage) { return stage >= R::kDepth ? stage - R::kDepth : stage; };
#pragma unroll
    for (int i = 0; i < R::kDepth - NR; ++i) fetch(row + i * step, i);
#pragma unroll
    for (int i = 0; i < NR; ++i) fetch_stats(row + i * step, stat_next[i]);
    load_params<TPR, K, VEC>(p.w, p.wbf16, p.pvec, p.cols, t, 1.f, w);
    for (int stage = 0; row < p.rows; row += NR * step, stage = wrap(stage + NR)) {
      // the second row of the turn, if there is one (the same for the whole group)
      const bool two = NR == 2 && row + step < p.rows;
      const int other = wrap(stage + 1);
#pragma unroll
      for (int i = 0; i < NR; ++i) stat[i] = stat_next[i];
#pragma unroll
      for (int i = 0; i < NR; ++i) fetch_stats(row + (NR + i) * step, stat_next[i]);
#pragma unroll
      for (int i = 0; i < NR; ++i)
        fetch(row + (R::kDepth - NR + i) * step, wrap(stage + R::kDepth - NR + i));
      ring.template wait<NR>();
      auto values = [&](int st, const float2& rm, int k, float (&z)[8], float (&g)[8]) {
        ring.get(st, 0, k, z);
        ring.get(st, 1, k, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = (z[j] - rm.y) * rm.x;
      };
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float z[8], g[8];
        values(stage, stat[0], k, z, g);
        add(k, z, g, s0);
        if (two) {
          values(other, stat[1], k, z, g);
          add(k, z, g, s1);
        }
      }
      if (NR == 2) row_sum4<TPR>(s0, s1, red, turn);
      else row_sum2<TPR>(s0.x, s0.y, red, turn);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float z[8], g[8];
        values(stage, stat[0], k, z, g);
        finish(k, row, z, g, s0, stat[0].x);
        if (two) {
          values(other, stat[1], k, z, g);
          finish(k, row + step, z, g, s1, stat[1].x);
        }
      }
    }
  } else {
    // the next row is loaded ahead where its raw values fit in registers beside this row's
    constexpr bool kAhead = sizeof(T) * K <= 8;
    using Chunks = RowChunks<T, TPR, K, VEC>;
    Chunks xc, gc, xn, gn;
    auto load_row = [&](Chunks& x, Chunks& g, int64_t i) {
      x.load(static_cast<const T*>(p.x) + i * p.ld_x, p.cols, t);
      g.load(static_cast<const T*>(p.dy) + i * p.ld_dy, p.cols, t);
    };
    if (row < p.rows) load_row(xc, gc, row);
    fetch_stats(row, stat_next[0]);
    load_params<TPR, K, VEC>(p.w, p.wbf16, p.pvec, p.cols, t, 1.f, w);
    for (; row < p.rows; row += step) {
      stat[0] = stat_next[0];
      fetch_stats(row + step, stat_next[0]);
      if (kAhead && row + step < p.rows) load_row(xn, gn, row + step);
      auto values = [&](int k, float (&z)[8], float (&g)[8]) {
        xc.get(k, z);
        gc.get(k, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = (z[j] - stat[0].y) * stat[0].x;
      };
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float z[8], g[8];
        values(k, z, g);
        add(k, z, g, s);
      }
      row_sum2<TPR>(s.x, s.y, red, turn);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float z[8], g[8];
        values(k, z, g);
        finish(k, row, z, g, s, stat[0].x);
      }
      if (kAhead) {
        xc = xn;
        gc = gn;
      } else if (row + step < p.rows) {
        load_row(xc, gc, row + step);
      }
    }
  }
  // this block's column sums, its warps added in warp order
  float* part = p.partials + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!(h == 0 ? p.has_dw : p.has_db)) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (TPR == 32) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          comb[(sub * 8 + j) * 32 + t] = h == 0 ? aw[k][j] : ab[k][j];
        __syncthreads();
        // thread (sub, t) adds element j = sub of lane t over the warps
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kNormWarps; ++i) s += comb[(i * 8 + sub) * 32 + t];
        const int64_t e = elem_of<TPR, VEC>(t, k, sub);
        if (e < p.cols) part[h * p.cols + e] = s;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t e = elem_of<TPR, VEC>(t, k, j);
          if (e < p.cols) part[h * p.cols + e] = h == 0 ? aw[k][j] : ab[k][j];
        }
      }
    }
  }
}

// Rows too long for registers: the two row sums, then dx; a block owns whole rows, and its
// column sums live in the workspace (only this block's threads touch its slice).
template <typename T>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[4 * 32];
  pdl_launch();
  pdl_wait();
  int turn = 0;
  float* part = p.partials + (int64_t)blockIdx.x * 2 * p.cols;
  for (int64_t e = threadIdx.x; e < p.cols; e += 1024) part[e] = part[p.cols + e] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.ld_x;
    const T* gr = static_cast<const T*>(p.dy) + row * p.ld_dy;
    T* dr = static_cast<T*>(p.dx) + row * p.ld_dx;
    const float r = p.rstd_in[row], mu = p.layer ? p.mean_in[row] : 0.f;
    float s1 = 0.f, s2 = 0.f;
    for (int64_t e = threadIdx.x; e < p.cols; e += 1024) {
      const float z = (to_f32(xr[e]) - mu) * r, d = to_f32(gr[e]);
      part[e] = fmaf(d, z, part[e]);
      part[p.cols + e] += d;
      const float g = p.w ? d * load_param(p.w, p.wbf16, e) : d;
      s1 += g;
      s2 = fmaf(g, z, s2);
    }
    row_sum2<1024>(s1, s2, red, turn);
    s1 = p.layer ? s1 * p.inv_n : 0.f;
    s2 *= p.inv_n;
    for (int64_t e = threadIdx.x; e < p.cols; e += 1024) {
      const float z = (to_f32(xr[e]) - mu) * r, d = to_f32(gr[e]);
      const float g = p.w ? d * load_param(p.w, p.wbf16, e) : d;
      dr[e] = from_f32<T>((g - s1 - z * s2) * r);
    }
  }
}

// ---------------------------------------------------------------- dispatch
// TPR and K are the smallest that hold the row; f is called with the kernel's shape.
template <typename T, bool VEC, typename F>
cudaError_t by_shape(int64_t cols, F&& f) {
  auto k_of = [&](int tpr) { return (int)((cols + 8 * tpr - 1) / (8 * tpr)); };
#define MFSDP_NORM_K(TPR)                                                                      \
  switch (k_of(TPR)) {                                                                         \
    case 1: return f.template operator()<T, TPR, 1, VEC>();                                    \
    case 2: return f.template operator()<T, TPR, 2, VEC>();                                    \
    case 3: return f.template operator()<T, TPR, 3, VEC>();                                    \
    default: return f.template operator()<T, TPR, 4, VEC>();                                   \
  }
  if (cols <= kWarpRowMax) { MFSDP_NORM_K(32) }
  if (cols <= 2048) return f.template operator()<T, 128, 2, VEC>();
  if (cols <= 4096) return f.template operator()<T, 256, 2, VEC>();
  return f.template operator()<T, 512, 2, VEC>();
#undef MFSDP_NORM_K
}

struct FwdLaunch {
  const NormArgs& a;
  int sms;
  cudaStream_t st;
  template <typename T, int TPR, int K, bool VEC>
  cudaError_t operator()() const {
    const int threads = TPR == 32 ? 32 * kNormWarps : TPR;
    constexpr int smem = kRing<T, VEC> ? Ring<1, TPR, K>::kBytes : 0;
    static std::atomic<int> cache[kCachedDevices];
    const int occ = resident(cache, norm_forward_kernel<T, TPR, K, VEC>, threads, smem);
    const int64_t per = TPR == 32 ? kNormWarps : 1, need = (a.rows + per - 1) / per;
    const int64_t g = std::min<int64_t>((int64_t)sms * occ, need);
    return launch_pdl(norm_forward_kernel<T, TPR, K, VEC>, dim3((unsigned)g), dim3(threads), smem,
                      st, a);
  }
};

struct BwdLaunch {
  const NormArgs& a;
  int max_blocks, sms;
  cudaStream_t st;
  int* blocks;
  template <typename T, int TPR, int K, bool VEC>
  cudaError_t operator()() const {
    const int threads = TPR == 32 ? 32 * kNormWarps : TPR;
    constexpr int smem = kRing<T, VEC> ? Ring<2, TPR, K>::kBytes : 0;
    static std::atomic<int> cache[kCachedDevices];
    const int occ = resident(cache, norm_backward_kernel<T, TPR, K, VEC>, threads, smem);
    const int64_t per = TPR == 32 ? kNormWarps : 1, need = (a.rows + per - 1) / per;
    const int64_t g = std::min({(int64_t)sms * occ, (int64_t)max_blocks, need});
    *blocks = (int)g;
    return launch_pdl(norm_backward_kernel<T, TPR, K, VEC>, dim3((unsigned)g), dim3(threads), smem,
                      st, a);
  }
};

// 16-byte accesses of eight elements: every row starts on a 16-byte boundary and has whole
// chunks.
bool rows_vec(const void* p, int64_t ld, int64_t cols, int32_t dtype) {
  return aligned_to(p, 16) && cols % 8 == 0 && (ld * (int64_t)dtype_bytes(dtype)) % 16 == 0;
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" int mfsdp_norm_forward(int32_t kind, int64_t rows, int64_t cols, int32_t dtype,
                                  int32_t param_dtype, const void* x, int64_t ld_x,
                                  const void* weight, const void* bias, float eps, void* y,
                                  int64_t ld_y, float* mean, float* rstd, void* stream) {
  const int chk = check_shape(kind, rows, cols, dtype, param_dtype);
  if (chk != MFSDP_OK) return chk;
  if (!(eps >= 0.f) || (kind == MFSDP_NORM_RMS && (bias || mean))) return MFSDP_EINVAL;
  if (rows == 0) return MFSDP_OK;
  if (!x || !y || ld_x < cols || ld_y < cols) return MFSDP_EINVAL;
  const size_t es = dtype_bytes(dtype), ps = dtype_bytes(param_dtype);
  if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(weight, ps) ||
      !aligned_to(bias, ps) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return MFSDP_EALIGN;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  NormArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.x = x;
  a.ld_x = ld_x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.ld_y = ld_y;
  a.mean = mean;
  a.rstd = rstd;
  a.eps = eps;
  a.inv_n = (float)(1.0 / (double)cols);
  a.layer = kind == MFSDP_NORM_LAYER;
  a.wbf16 = param_dtype == MFSDP_DTYPE_BF16;
  a.pvec = aligned_to(weight, 16) && aligned_to(bias, 16);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cols > kRegRowMax) {
    e = dtype == MFSDP_DTYPE_BF16
            ? launch_pdl(norm_forward_long_kernel<bf16_t>, dim3((unsigned)rows), dim3(1024), 0, st, a)
            : launch_pdl(norm_forward_long_kernel<float>, dim3((unsigned)rows), dim3(1024), 0, st, a);
  } else {
    const bool vec = rows_vec(x, ld_x, cols, dtype) && rows_vec(y, ld_y, cols, dtype);
    const FwdLaunch f{a, sms, st};
    if (dtype == MFSDP_DTYPE_BF16)
      e = vec ? by_shape<bf16_t, true>(cols, f) : by_shape<bf16_t, false>(cols, f);
    else
      e = vec ? by_shape<float, true>(cols, f) : by_shape<float, false>(cols, f);
  }
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}

extern "C" int mfsdp_norm_backward_workspace_bytes(int64_t rows, int64_t cols, size_t* bytes_out) {
  if (!bytes_out) return MFSDP_EINVAL;
  if (rows < 0 || cols < 1 || rows >= (1ll << 31) || cols >= (1ll << 31)) return MFSDP_ESHAPE;
  *bytes_out = (size_t)blocks_bound(rows) * 2 * (size_t)cols * sizeof(float);
  return MFSDP_OK;
}

extern "C" int mfsdp_norm_backward(int32_t kind, int64_t rows, int64_t cols, int32_t dtype,
                                   int32_t param_dtype, const void* dy, int64_t ld_dy,
                                   const void* x, int64_t ld_x, const void* weight,
                                   const float* mean, const float* rstd, void* dx, int64_t ld_dx,
                                   void* dweight, void* dbias, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  const int chk = check_shape(kind, rows, cols, dtype, param_dtype);
  if (chk != MFSDP_OK) return chk;
  if (kind == MFSDP_NORM_RMS && (mean || dbias)) return MFSDP_EINVAL;
  if (rows > 0 && (!dy || !x || !dx || !rstd || (kind == MFSDP_NORM_LAYER && !mean) ||
                   ld_dy < cols || ld_x < cols || ld_dx < cols))
    return MFSDP_EINVAL;
  if (!workspace) return MFSDP_EINVAL;
  const size_t es = dtype_bytes(dtype), ps = dtype_bytes(param_dtype);
  if (!aligned_to(dy, es) || !aligned_to(x, es) || !aligned_to(dx, es) ||
      !aligned_to(weight, ps) || !aligned_to(dweight, ps) || !aligned_to(dbias, ps) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(workspace, 256))
    return MFSDP_EALIGN;
  size_t need = 0;
  mfsdp_norm_backward_workspace_bytes(rows, cols, &need);
  if (workspace_bytes < need) return MFSDP_EWORKSPACE;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  NormArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.x = x;
  a.ld_x = ld_x;
  a.dy = dy;
  a.ld_dy = ld_dy;
  a.w = weight;
  a.dx = dx;
  a.ld_dx = ld_dx;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.partials = static_cast<float*>(workspace);
  a.inv_n = (float)(1.0 / (double)cols);
  a.layer = kind == MFSDP_NORM_LAYER;
  a.wbf16 = param_dtype == MFSDP_DTYPE_BF16;
  a.pvec = aligned_to(weight, 16);
  a.has_dw = dweight != nullptr;
  a.has_db = dbias != nullptr;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  int blocks = 0;
  if (rows > 0) {
    if (cols > kRegRowMax) {
      blocks = blocks_bound(rows) < sms ? blocks_bound(rows) : sms;
      e = dtype == MFSDP_DTYPE_BF16
              ? launch_pdl(norm_backward_long_kernel<bf16_t>, dim3(blocks), dim3(1024), 0, st, a)
              : launch_pdl(norm_backward_long_kernel<float>, dim3(blocks), dim3(1024), 0, st, a);
    } else {
      const bool vec = rows_vec(x, ld_x, cols, dtype) && rows_vec(dy, ld_dy, cols, dtype) &&
                       rows_vec(dx, ld_dx, cols, dtype);
      const BwdLaunch f{a, blocks_bound(rows), sms, st, &blocks};
      if (dtype == MFSDP_DTYPE_BF16)
        e = vec ? by_shape<bf16_t, true>(cols, f) : by_shape<bf16_t, false>(cols, f);
      else
        e = vec ? by_shape<float, true>(cols, f) : by_shape<float, false>(cols, f);
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
