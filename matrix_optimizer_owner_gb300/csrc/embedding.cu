// Embedding lookup with a scale, and the gradient of its table.
//
// Forward: out[t] = scale * table[ids[t]].  Backward: dtable[v] = scale * sum of dy[t] over the
// tokens t with ids[t] = v, t ascending; rows of ids that do not occur are zero.
//
// Both are bound by memory.  The gradient must not depend on timing, so the tokens are sorted
// by id first (stable, so each id's tokens stay in order) instead of adding with atomics:
//   1. sort     one cluster of eight blocks runs a stable radix sort of (id, token), least
//               significant digit first.  Per pass each warp counts the digits of its own
//               contiguous share, the blocks exchange their digit totals through distributed
//               shared memory, and every warp then places its share in order.  Cluster barriers
//               separate the steps, so the whole sort is one launch.
//   2. sum      the sorted positions are cut into chunks of kChunkPos.  A chunk sums the runs
//               of equal ids inside it in fp32 and writes each finished row once; a run that
//               crosses a chunk boundary leaves fp32 partial rows in the workspace.  The work
//               per block is the same whether one id owns half the tokens or none repeats.
//               The same launch writes the zero rows (ids that a flag array of the sort marks
//               as absent), so the gradient is written exactly once.
//   3. join     adds the partial rows of the runs that cross chunks, in chunk order.
// The sum is held in fp32 throughout and rounded once, to the gradient's type.
#include "elem.cuh"
#include "mfsdp.h"

#include <algorithm>

namespace mfsdp {
namespace {

constexpr int kSortBlocks = 8;              // cluster size
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitMax = 9;                // bits per pass
constexpr int kBinsMax = 1 << kDigitMax;
constexpr int kSortSmem = (kSortWarps * kBinsMax + kBinsMax + kBinsMax + 32) * 4;
constexpr int kChunkPos = 32;               // sorted positions per chunk
constexpr int kSumThreads = 128;
constexpr int kZeroRows = 8;                // table rows per zero-fill block

struct EmbFwd {
  const void* table;
  const void* ids;
  void* out;
  int64_t ld_table, ld_out, n, vocab;
  int32_t dim, is64;
  float scale;
  int* status;
};

// ---------------------------------------------------------------- lookup
// One thread per 8 elements (VEC) or per element of the output.
template <typename TT, typename TO, bool VEC>
__global__ void __launch_bounds__(256) embedding_forward_kernel(const __grid_constant__ EmbFwd p) {
  pdl_launch();
  pdl_wait();
  const int per_row = VEC ? p.dim / 8 : p.dim;
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = u / per_row;
  if (t >= p.n) return;
  const int c = (int)(u - t * per_row) * (VEC ? 8 : 1);
  const int64_t id = load_index(p.ids, p.is64, t);
  const bool ok = id >= 0 && id < p.vocab;
  if (!ok && c == 0) atomicOr(p.status, kStatusBadIndex);
  const TT* src = static_cast<const TT*>(p.table) + id * p.ld_table + c;
  TO* dst = static_cast<TO*>(p.out) + t * p.ld_out + c;
  if (VEC) {
    Pack8<TT> a;
    if (ok) a.load(src); else a.zero();
    float v[8];
    a.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= p.scale;
    Pack8<TO> b;
    b.set(v);
    b.store(dst);
  } else {
    *dst = from_f32<TO>(ok ? to_f32(*src) * p.scale : 0.f);
  }
}

// ---------------------------------------------------------------- sort
struct SortArgs {
  const void* ids;
  uint32_t *key0, *val0, *key1, *val1;   // ping-pong; the result lands in key1, val1
  uint8_t* present;                      // [vocab] written: 1 where an id occurs
  int64_t vocab, padding;
  int32_t n, is64, passes, digit;
  int* status;
};

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* local, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(local), r, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
}

__global__ void __cluster_dims__(kSortBlocks, 1, 1) __launch_bounds__(kSortThreads)
    embedding_sort_kernel(const __grid_constant__ SortArgs p) {
  extern __shared__ uint32_t sort_smem[];
  uint32_t* hist = sort_smem;                          // [warp][bin], then write positions
  uint32_t* total = hist + kSortWarps * kBinsMax;      // this block's digit totals
  uint32_t* base = total + kBinsMax;                   // first position of (digit, this block)
  uint32_t* scan = base + kBinsMax;
  pdl_launch();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int bins = 1 << p.digit;
  // every warp of the cluster owns one contiguous share of the positions
  const int64_t share = (p.n + kSortBlocks * kSortWarps - 1) / (kSortBlocks * kSortWarps);
  const int64_t i0 = ((int64_t)rank * kSortWarps + warp) * share;
  const int64_t i1 = i0 + share < p.n ? i0 + share : (int64_t)p.n;
  // the flags start at zero (the array has 16-byte alignment and is padded to it)
  for (int64_t i = (int64_t)rank * kSortThreads + tid; i < (p.vocab + 15) / 16;
       i += kSortBlocks * kSortThreads)
    reinterpret_cast<uint4*>(p.present)[i] = make_uint4(0u, 0u, 0u, 0u);

  for (int pass = 0; pass < p.passes; ++pass) {
    // the last pass writes buffer 1
    const bool to1 = ((p.passes - 1 - pass) & 1) == 0;
    const uint32_t* ks = to1 ? p.key0 : p.key1;
    const uint32_t* vs = to1 ? p.val0 : p.val1;
    uint32_t* kd = to1 ? p.key1 : p.key0;
    uint32_t* vd = to1 ? p.val1 : p.val0;
    const int shift = pass * p.digit;
    // ids outside the table and the padding id sort behind every row, as key = vocab
    auto key_at = [&](int64_t i) -> uint32_t {
      if (pass > 0) return ks[i];
      const int64_t id = load_index(p.ids, p.is64, i);
      return id < 0 || id >= p.vocab || id == p.padding ? (uint32_t)p.vocab : (uint32_t)id;
    };
    for (int b = tid; b < kSortWarps * bins; b += kSortThreads) hist[b] = 0u;
    __syncthreads();
    for (int64_t i = i0 + lane; i < i1; i += 32) {
      const uint32_t k = key_at(i);
      if (pass == 0) {
        const int64_t id = load_index(p.ids, p.is64, i);
        if ((id < 0 || id >= p.vocab) && id != p.padding) atomicOr(p.status, kStatusBadIndex);
      }
      atomicAdd(&hist[warp * bins + ((k >> shift) & (bins - 1))], 1u);
    }
    __syncthreads();
    // per digit: exclusive sums over this block's warps, and the block's total
    for (int b = tid; b < bins; b += kSortThreads) {
      uint32_t s = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w * bins + b];
        hist[w * bins + b] = s;
        s += c;
      }
      total[b] = s;
    }
    cluster_barrier();
    // digit b of this block starts after all smaller digits and the same digit of the blocks
    // before it
    uint32_t all = 0, before = 0;
    if (tid < bins)
      for (uint32_t r = 0; r < (uint32_t)kSortBlocks; ++r) {
        const uint32_t c = ld_cluster_u32(total + tid, r);
        all += c;
        if (r < rank) before += c;
      }
    uint32_t x = all;   // inclusive scan over the digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    if (warp == 0) {
      uint32_t s = scan[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += y;
      }
      scan[lane] = s;
    }
    __syncthreads();
    if (tid < bins) base[tid] = x - all + (warp > 0 ? scan[warp - 1] : 0u) + before;
    __syncthreads();
    // place, 32 positions at a time, in order: a lane's rank is the number of lower lanes with
    // its digit
    uint32_t* mine = hist + warp * bins;
    for (int64_t b0 = i0; b0 < i1; b0 += 32) {
      const int64_t i = b0 + lane;
      const bool live = i < i1;
      const uint32_t k = live ? key_at(i) : 0u;
      const uint32_t v = live ? (pass > 0 ? vs[i] : (uint32_t)i) : 0u;
      const uint32_t d = live ? (k >> shift) & (bins - 1) : 0xFFFFFFFFu;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
      const uint32_t below = __popc(same & ((1u << lane) - 1u));
      uint32_t pos = 0;
      if (live) pos = base[d] + mine[d] + below;
      __syncwarp();
      if (live && below == 0) mine[d] += __popc(same);
      __syncwarp();
      if (live) {
        kd[pos] = k;
        vd[pos] = v;
        if (pass == p.passes - 1 && k < (uint32_t)p.vocab) p.present[k] = 1;
      }
    }
    cluster_barrier();   // the pass's output, and the peers' totals, before the next pass
  }
}

// ---------------------------------------------------------------- sum and join
struct SumArgs {
  const uint32_t *key, *val;
  const uint8_t* present;
  const void* dy;
  void* dtable;
  float* part;                 // [chunks][2][dim]: run from before the chunk, run into the next
  int64_t ld_dy, ld_dt, vocab;
  int32_t n, dim, chunks, accumulate;
  int32_t slabs, cols_shift;   // column threads per chunk = 1 << cols_shift
  int32_t sum_blocks;          // blocks of the sum part; the rest write zero rows
  float scale;
};

// The eight elements of column thread c in slab s: consecutive (VEC) or TX apart.
template <bool VEC>
__device__ __forceinline__ int col_of(int slab, int tx, int c, int j) {
  return VEC ? (slab * tx + c) * 8 + j : (slab * 8 + j) * tx + c;
}

template <typename TG, bool VEC>
__device__ __forceinline__ void write_row(const SumArgs& p, uint32_t v, int slab, int tx, int c,
                                          const float (&acc)[8]) {
  TG* row = static_cast<TG*>(p.dtable) + (int64_t)v * p.ld_dt;
  if (VEC) {
    const int e = col_of<VEC>(slab, tx, c, 0);
    if (e >= p.dim) return;
    float o[8];
    Pack8<TG> q;
    if (p.accumulate) {
      q.load(row + e);
      q.get(o);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = p.accumulate ? fmaf(acc[j], p.scale, o[j]) : acc[j] * p.scale;
    q.set(o);
    q.store(row + e);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = col_of<VEC>(slab, tx, c, j);
      if (e < p.dim)
        row[e] = from_f32<TG>(p.accumulate ? fmaf(acc[j], p.scale, to_f32(row[e])) : acc[j] * p.scale);
    }
  }
}

template <typename TD, typename TG, bool VEC>
__global__ void __launch_bounds__(kSumThreads) embedding_sum_kernel(const __grid_constant__ SumArgs p) {
  pdl_launch();
  pdl_wait();
  if ((int)blockIdx.x >= p.sum_blocks) {
    // rows of absent ids
    const int64_t r0 = (int64_t)((int)blockIdx.x - p.sum_blocks) * kZeroRows;
    for (int i = 0; i < kZeroRows; ++i) {
      const int64_t r = r0 + i;
      if (r >= p.vocab || p.present[r]) continue;
      TG* row = static_cast<TG*>(p.dtable) + r * p.ld_dt;
      if (VEC) {
        Pack8<TG> z;
        z.zero();
        for (int e = threadIdx.x * 8; e < p.dim; e += kSumThreads * 8) z.store(row + e);
      } else {
        for (int e = threadIdx.x; e < p.dim; e += kSumThreads) row[e] = from_f32<TG>(0.f);
      }
    }
    return;
  }
  const int tx = 1 << p.cols_shift, ty = kSumThreads >> p.cols_shift;
  const int c = threadIdx.x & (tx - 1);
  const int64_t unit = (int64_t)blockIdx.x * ty + (threadIdx.x >> p.cols_shift);
  const int slab = (int)(unit % p.slabs);
  const int64_t chunk = unit / p.slabs;
  if (chunk >= p.chunks) return;
  const int i0 = (int)(chunk * kChunkPos), i1 = min(p.n, i0 + kChunkPos);
  const uint32_t none = (uint32_t)p.vocab;
  const uint32_t prev = i0 > 0 ? p.key[i0 - 1] : none, next = i1 < p.n ? p.key[i1] : none;
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  uint32_t cur = p.key[i0];
  bool from_before = i0 > 0 && prev == cur;
  float* part = p.part + chunk * 2 * p.dim;
  auto flush = [&](bool to_next) {
    if (cur == none) return;
    if (!from_before && !to_next) {
      write_row<TG, VEC>(p, cur, slab, tx, c, acc);
    } else {
      float* dst = part + (from_before ? 0 : p.dim);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = col_of<VEC>(slab, tx, c, j);
        if (e < p.dim) dst[e] = acc[j];
      }
    }
  };
  constexpr int U = 8;   // rows loaded ahead
  for (int b = i0; b < i1; b += U) {
    uint32_t k[U];
    Pack8<TD> d[U];
    float ds[VEC ? 1 : U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = b + u < i1 ? p.key[b + u] : none;
      const TD* row = static_cast<const TD*>(p.dy) +
                      (k[u] != none ? (int64_t)p.val[b + u] * p.ld_dy : 0);
      if (VEC) {
        const int e = col_of<VEC>(slab, tx, c, 0);
        if (k[u] != none && e < p.dim) d[u].load(row + e); else d[u].zero();
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = col_of<VEC>(slab, tx, c, j);
          ds[VEC ? 0 : u][j] = k[u] != none && e < p.dim ? to_f32(row[e]) : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u >= i1) break;
      if (k[u] != cur) {
        flush(false);
        cur = k[u];
        from_before = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
      }
      float v[8];
      if (VEC) d[u].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += VEC ? v[j] : ds[VEC ? 0 : u][j];
    }
  }
  flush(i1 < p.n && next == cur);
}

// A run that starts in this chunk and goes on: its partial rows, in chunk order.
template <typename TG, bool VEC>
__global__ void __launch_bounds__(kSumThreads) embedding_join_kernel(const __grid_constant__ SumArgs p) {
  pdl_launch();
  pdl_wait();
  const int tx = 1 << p.cols_shift, ty = kSumThreads >> p.cols_shift;
  const int c = threadIdx.x & (tx - 1);
  const int64_t unit = (int64_t)blockIdx.x * ty + (threadIdx.x >> p.cols_shift);
  const int slab = (int)(unit % p.slabs);
  const int64_t chunk = unit / p.slabs;
  if (chunk + 1 >= p.chunks) return;
  const int i0 = (int)(chunk * kChunkPos), i1 = i0 + kChunkPos;
  const uint32_t k = p.key[i1 - 1];
  if (k == (uint32_t)p.vocab || p.key[i1] != k) return;           // ends here
  if (i0 > 0 && p.key[i0 - 1] == k) return;                       // an earlier chunk's run
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = col_of<VEC>(slab, tx, c, j);
    acc[j] = e < p.dim ? p.part[(chunk * 2 + 1) * p.dim + e] : 0.f;
  }
  for (int64_t q = chunk + 1; q < p.chunks && p.key[q * kChunkPos] == k; ++q) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = col_of<VEC>(slab, tx, c, j);
      if (e < p.dim) acc[j] += p.part[q * 2 * p.dim + e];
    }
  }
  write_row<TG, VEC>(p, k, slab, tx, c, acc);
}

// ---------------------------------------------------------------- host
size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct BwdLayout {
  size_t key0, val0, key1, val1, present, part, total;
};
BwdLayout bwd_layout(int64_t vocab, int64_t dim, int64_t n) {
  BwdLayout l{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += up256(bytes);
    return at;
  };
  l.key0 = take((size_t)n * 4);
  l.val0 = take((size_t)n * 4);
  l.key1 = take((size_t)n * 4);
  l.val1 = take((size_t)n * 4);
  l.present = take((size_t)vocab);
  l.part = take((size_t)((n + kChunkPos - 1) / kChunkPos) * 2 * (size_t)dim * 4);
  l.total = off;
  return l;
}

int check_table(int64_t vocab, int64_t dim, int64_t n) {
  if (vocab < 1 || dim < 1 || n < 0 || vocab >= (1ll << 31) - 1 || dim >= (1ll << 27) ||
      n >= (1ll << 31) - kChunkPos)
    return MFSDP_ESHAPE;
  return MFSDP_OK;
}

bool vec_ok(const void* p, int64_t ld, int64_t dim, int32_t dtype) {
  return aligned_to(p, 16) && dim % 8 == 0 && (ld * (int64_t)dtype_bytes(dtype)) % 16 == 0;
}

template <typename TT, typename TO>
cudaError_t run_forward(const EmbFwd& a, bool vec, cudaStream_t st) {
  const int64_t units = a.n * (vec ? a.dim / 8 : a.dim);
  const int64_t grid = (units + 255) / 256;
  if (grid >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  return vec ? launch_pdl(embedding_forward_kernel<TT, TO, true>, dim3((unsigned)grid), dim3(256),
                          0, st, a)
             : launch_pdl(embedding_forward_kernel<TT, TO, false>, dim3((unsigned)grid), dim3(256),
                          0, st, a);
}

template <typename TD, typename TG>
cudaError_t run_sum(const SumArgs& a, bool vec, int64_t grid, int64_t join_grid, cudaStream_t st) {
  cudaError_t e;
  const dim3 b(kSumThreads);
  e = vec ? launch_pdl(embedding_sum_kernel<TD, TG, true>, dim3((unsigned)grid), b, 0, st, a)
          : launch_pdl(embedding_sum_kernel<TD, TG, false>, dim3((unsigned)grid), b, 0, st, a);
  if (e != cudaSuccess || a.chunks < 2) return e;
  return vec ? launch_pdl(embedding_join_kernel<TG, true>, dim3((unsigned)join_grid), b, 0, st, a)
             : launch_pdl(embedding_join_kernel<TG, false>, dim3((unsigned)join_grid), b, 0, st, a);
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" int mfsdp_embedding_forward(int64_t vocab, int64_t dim, int32_t table_dtype,
                                       const void* table, int64_t ld_table, int64_t n_tokens,
                                       int32_t index_dtype, const void* ids, float scale,
                                       int32_t out_dtype, void* out, int64_t ld_out,
                                       void* stream) {
  const int chk = check_table(vocab, dim, n_tokens);
  if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype) ||
      (index_dtype != MFSDP_INDEX_I32 && index_dtype != MFSDP_INDEX_I64))
    return MFSDP_EINVAL;
  if (chk != MFSDP_OK) return chk;
  if (n_tokens == 0) return MFSDP_OK;
  if (!table || !ids || !out || ld_table < dim || ld_out < dim) return MFSDP_EINVAL;
  const bool is64 = index_dtype == MFSDP_INDEX_I64;
  if (!aligned_to(table, dtype_bytes(table_dtype)) || !aligned_to(out, dtype_bytes(out_dtype)) ||
      !aligned_to(ids, is64 ? 8 : 4))
    return MFSDP_EALIGN;
  const bool vec = vec_ok(table, ld_table, dim, table_dtype) && vec_ok(out, ld_out, dim, out_dtype);
  if (n_tokens * (vec ? dim / 8 : dim) > (1ll << 31) * 256 - 256) return MFSDP_ESHAPE;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  EmbFwd a{};
  a.table = table;
  a.ids = ids;
  a.out = out;
  a.ld_table = ld_table;
  a.ld_out = ld_out;
  a.n = n_tokens;
  a.vocab = vocab;
  a.dim = (int32_t)dim;
  a.is64 = is64;
  a.scale = scale;
  a.status = status_word_address();
  if (!a.status) return MFSDP_ECUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool tb = table_dtype == MFSDP_DTYPE_BF16, ob = out_dtype == MFSDP_DTYPE_BF16;
  const cudaError_t e = tb ? (ob ? run_forward<bf16_t, bf16_t>(a, vec, st)
                                 : run_forward<bf16_t, float>(a, vec, st))
                           : (ob ? run_forward<float, bf16_t>(a, vec, st)
                                 : run_forward<float, float>(a, vec, st));
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}

extern "C" int mfsdp_embedding_backward_workspace_bytes(int64_t vocab, int64_t dim,
                                                        int64_t n_tokens, size_t* bytes_out) {
  if (!bytes_out) return MFSDP_EINVAL;
  const int chk = check_table(vocab, dim, n_tokens);
  if (chk != MFSDP_OK) return chk;
  *bytes_out = bwd_layout(vocab, dim, n_tokens).total;
  return MFSDP_OK;
}

extern "C" int mfsdp_embedding_backward(int64_t vocab, int64_t dim, int64_t n_tokens,
                                        int32_t index_dtype, const void* ids,
                                        int64_t padding_idx, float scale, int32_t dy_dtype,
                                        const void* dy, int64_t ld_dy, int32_t accumulate,
                                        int32_t grad_dtype, void* dtable, int64_t ld_dtable,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  const int chk = check_table(vocab, dim, n_tokens);
  if (!dtype_ok(dy_dtype) || !dtype_ok(grad_dtype) ||
      (index_dtype != MFSDP_INDEX_I32 && index_dtype != MFSDP_INDEX_I64))
    return MFSDP_EINVAL;
  if (chk != MFSDP_OK) return chk;
  if (!dtable || ld_dtable < dim || !workspace) return MFSDP_EINVAL;
  if (n_tokens > 0 && (!ids || !dy || ld_dy < dim)) return MFSDP_EINVAL;
  const bool is64 = index_dtype == MFSDP_INDEX_I64;
  if (!aligned_to(dtable, dtype_bytes(grad_dtype)) || !aligned_to(dy, dtype_bytes(dy_dtype)) ||
      !aligned_to(ids, is64 ? 8 : 4) || !aligned_to(workspace, 256))
    return MFSDP_EALIGN;
  const BwdLayout l = bwd_layout(vocab, dim, n_tokens);
  if (workspace_bytes < l.total) return MFSDP_EWORKSPACE;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  int* status = status_word_address();
  if (!status) return MFSDP_ECUDA;
  char* ws = static_cast<char*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);

  SortArgs s{};
  s.ids = ids;
  s.key0 = reinterpret_cast<uint32_t*>(ws + l.key0);
  s.val0 = reinterpret_cast<uint32_t*>(ws + l.val0);
  s.key1 = reinterpret_cast<uint32_t*>(ws + l.key1);
  s.val1 = reinterpret_cast<uint32_t*>(ws + l.val1);
  s.present = reinterpret_cast<uint8_t*>(ws + l.present);
  s.vocab = vocab;
  s.padding = padding_idx;
  s.n = (int32_t)n_tokens;
  s.is64 = is64;
  int bits = 1;
  while ((vocab >> bits) != 0) ++bits;   // keys run to vocab itself (ids that take no part)
  s.passes = (bits + kDigitMax - 1) / kDigitMax;
  s.digit = (bits + s.passes - 1) / s.passes;
  s.status = status;

  SumArgs a{};
  a.key = s.key1;
  a.val = s.val1;
  a.present = s.present;
  a.dy = dy;
  a.dtable = dtable;
  a.part = reinterpret_cast<float*>(ws + l.part);
  a.ld_dy = ld_dy;
  a.ld_dt = ld_dtable;
  a.vocab = vocab;
  a.n = (int32_t)n_tokens;
  a.dim = (int32_t)dim;
  a.chunks = (int32_t)((n_tokens + kChunkPos - 1) / kChunkPos);
  a.accumulate = accumulate ? 1 : 0;
  a.scale = scale;
  const int64_t col_threads = (dim + 7) / 8;
  while ((1 << a.cols_shift) < kSumThreads && (1 << a.cols_shift) < col_threads) ++a.cols_shift;
  const int64_t tx = 1ll << a.cols_shift, ty = kSumThreads / tx;
  a.slabs = (int32_t)((col_threads + tx - 1) / tx);
  const int64_t sum_blocks = ((int64_t)a.chunks * a.slabs + ty - 1) / ty;
  const int64_t zero_blocks = accumulate ? 0 : (vocab + kZeroRows - 1) / kZeroRows;
  if (sum_blocks + zero_blocks >= (1ll << 31)) return MFSDP_ESHAPE;
  a.sum_blocks = (int32_t)sum_blocks;
  if (sum_blocks + zero_blocks == 0) return MFSDP_OK;
  const bool vec = vec_ok(dtable, ld_dtable, dim, grad_dtype) &&
                   (n_tokens == 0 || vec_ok(dy, ld_dy, dim, dy_dtype));

  cudaError_t e = cudaFuncSetAttribute(embedding_sort_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
  if (e == cudaSuccess)
    e = launch_pdl(embedding_sort_kernel, dim3(kSortBlocks), dim3(kSortThreads), kSortSmem, st, s);
  if (e == cudaSuccess) {
    const bool db = dy_dtype == MFSDP_DTYPE_BF16, gb = grad_dtype == MFSDP_DTYPE_BF16;
    const int64_t grid = sum_blocks + zero_blocks;
    e = db ? (gb ? run_sum<bf16_t, bf16_t>(a, vec, grid, sum_blocks, st)
                 : run_sum<bf16_t, float>(a, vec, grid, sum_blocks, st))
           : (gb ? run_sum<float, bf16_t>(a, vec, grid, sum_blocks, st)
                 : run_sum<float, float>(a, vec, grid, sum_blocks, st));
  }
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}
