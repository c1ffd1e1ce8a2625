// What the norm kernels share: how a row lies over the threads that hold it, the sums over a row, the
// parameters of a thread's columns, and the join of the blocks' parameter gradients.
#pragma once

#include <atomic>

#include "elem.cuh"
#include "mfsdp.h"

namespace mfsdp {
namespace {

constexpr int kNormWarps = 8;         // warps per block of the warp-per-row kernels
constexpr int kWarpRowMax = 1024;     // longest row one warp takes
constexpr int kRegRowMax = 512 * 8 * 2;

__device__ __forceinline__ float load_param(const void* p, int is_bf16, int64_t e) {
  return is_bf16 ? to_f32(static_cast<const bf16_t*>(p)[e]) : static_cast<const float*>(p)[e];
}

// How a row lies over the TPR threads that share it: chunk k of thread t holds 8 consecutive
// elements (VEC) or 8 elements TPR apart (rows without 16-byte alignment); both coalesce.
template <int TPR, bool VEC>
__device__ __forceinline__ int64_t elem_of(int t, int k, int j) {
  return VEC ? ((int64_t)k * TPR + t) * 8 + j : ((int64_t)k * 8 + j) * TPR + t;
}

// The parameters of a thread's columns (`fill` where there are none).
template <int TPR, int K, bool VEC>
__device__ __forceinline__ void load_params(const void* src, int is_bf16, int pvec, int64_t n, int t,
                                            float fill, float (&v)[K][8]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t c = elem_of<TPR, VEC>(t, k, 0);
    if (VEC && src && pvec && c < n) {
      if (is_bf16) {
        Pack8<bf16_t> q;
        q.load(static_cast<const bf16_t*>(src) + c);
        q.get(v[k]);
      } else {
        Pack8<float> q;
        q.load(static_cast<const float*>(src) + c);
        q.get(v[k]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t e = elem_of<TPR, VEC>(t, k, j);
        v[k][j] = src && e < n ? load_param(src, is_bf16, e) : fill;
      }
    }
  }
}

// Sums of two values over the threads of a row, in every one of them.  Block rows use two
// buffers in turn, so one barrier per call is enough.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red, int& turn) {
  // both sums in one tree: the lower half of the warp goes on with a, the upper with b
  const bool upper = threadIdx.x & 16;
  float v = upper ? b : a;
  v += __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (TPR == 32) {
    const float w = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
    a = upper ? w : v;
    b = upper ? v : w;
    return;
  }
  constexpr int W = TPR / 32;
  float* buf = red + turn * 2 * W;
  turn ^= 1;
  if ((threadIdx.x & 15) == 0) buf[(upper ? W : 0) + (threadIdx.x >> 5)] = v;
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    a += buf[i];
    b += buf[W + i];
  }
}

// The same for two rows at a time, (a.x, a.y) and (b.x, b.y), in one tree and with one barrier.
template <int TPR>
__device__ __forceinline__ void row_sum4(float2& a, float2& b, float* red, int& turn) {
  // after two halvings lanes 0-7, 8-15, 16-23 and 24-31 hold one of the four values each
  const bool hi = threadIdx.x & 16, odd = threadIdx.x & 8;
  float x = hi ? b.x : a.x, y = hi ? b.y : a.y;
  x += __shfl_xor_sync(0xFFFFFFFFu, hi ? a.x : b.x, 16);
  y += __shfl_xor_sync(0xFFFFFFFFu, hi ? a.y : b.y, 16);
  float v = odd ? y : x;
  v += __shfl_xor_sync(0xFFFFFFFFu, odd ? x : y, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (TPR == 32) {
    a = make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 8));
    b = make_float2(__shfl_sync(0xFFFFFFFFu, v, 16), __shfl_sync(0xFFFFFFFFu, v, 24));
    return;
  }
  constexpr int W = TPR / 32;
  float* buf = red + turn * 4 * W;
  turn ^= 1;
  if ((threadIdx.x & 7) == 0) buf[threadIdx.x >> 3] = v;
  __syncthreads();
  a = b = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float4 q = reinterpret_cast<const float4*>(buf)[i];
    a.x += q.x;
    a.y += q.y;
    b.x += q.z;
    b.y += q.w;
  }
}

// Adds the blocks' column sums in block order: 32 columns of dw (blockIdx.y = 0) or db (1) per
// block, 32 groups of consecutive blocks whose sums are added in group order.
template <typename P>
__global__ void __launch_bounds__(1024)
    norm_param_grad_kernel(const float* partials, int blocks, int64_t cols, P* dw, P* db) {
  __shared__ float s[32][33];
  pdl_launch();
  pdl_wait();
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5, h = blockIdx.y;
  P* out = h == 0 ? dw : db;
  if (!out) return;
  const int64_t e = (int64_t)blockIdx.x * 32 + c;
  const int per = (blocks + 31) / 32, b0 = g * per, b1 = min(blocks, b0 + per);
  float a = 0.f;
  if (e < cols) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) a += partials[((int64_t)b * 2 + h) * cols + e];
  }
  s[g][c] = a;
  __syncthreads();
  if (g != 0 || e >= cols) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += s[i][c];
  out[e] = from_f32<P>(v);
}

// Raises a kernel's shared-memory limit and counts the blocks that an SM holds (at least 1), once
// per device; `cache` is the kernel's own.
constexpr int kCachedDevices = 64;
template <typename K>
int resident(std::atomic<int>* cache, K kernel, int threads, int smem) {
  int dev = -1, occ = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < kCachedDevices) occ = cache[dev].load();
  if (occ > 0) return occ;
  // (a kernel's static shared memory counts towards the 48 KB that need no raising)
  if (smem > 32 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return 1;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, threads, smem) != cudaSuccess ||
      occ < 1)
    return 1;
  if (dev < kCachedDevices) cache[dev].store(occ);
  return occ;
}

constexpr int kNormMaxBlocks = 152 * 8;   // blocks of one backward launch (bounds the workspace)

inline int check_shape(int32_t kind, int64_t rows, int64_t cols, int32_t dtype, int32_t param_dtype) {
  if (kind != MFSDP_NORM_LAYER && kind != MFSDP_NORM_RMS) return MFSDP_EINVAL;
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return MFSDP_EINVAL;
  if (rows < 0 || cols < 1 || rows >= (1ll << 31) || cols >= (1ll << 31)) return MFSDP_ESHAPE;
  return MFSDP_OK;
}

inline int blocks_bound(int64_t rows) {
  return (int)(rows < kNormMaxBlocks ? (rows < 1 ? 1 : rows) : kNormMaxBlocks);
}

}  // namespace
}  // namespace mfsdp
