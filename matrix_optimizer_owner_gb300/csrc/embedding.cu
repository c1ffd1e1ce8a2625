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
//               separate the steps, so the whole sort is one launch.  The sort is bound by
//               latency, so the launch's other blocks meanwhile write zeros over the first
//               kFillBytes of the gradient, about what fits in the sort's time.  Where those are
//               the whole table, up to kRankMax tokens are not sorted: each one's place is
//               counted, by blocks of their own.  Where they are not, one block sorts up to
//               kOneBlock tokens.
//   2. sum      the sorted positions are cut into chunks of 16 or 32.  A chunk sums the runs
//               of equal ids inside it in fp32 and writes each finished row once; a run that
//               crosses a chunk boundary leaves fp32 partial rows in the workspace.  The work
//               per block is the same whether one id owns half the tokens or none repeats.
//               More blocks of the launch zero the other rows that do not occur (the sort
//               marks those that do).
//   3. join     adds the partial rows of the runs that cross chunks, in chunk order.
// The sum is held in fp32 throughout and rounded once, to the gradient's type.
//
// Measured (bf16, graph replay, 6.78 TB/s being a copy's rate): lookup of 16384 rows of 768 in 10
// us, 4.3 TB/s of 45 MB; the gradient of 16384 tokens x 768 over 50257 rows in 36 us, 2.9 TB/s of
// 102 MB, of which 19 us are the sort, bound by the latency of its passes, with most of the zeros
// written beside it; 8192 tokens x 4096 over 128256 rows in 165 us, a copy's rate for the 1.12 GB.
#include "elem.cuh"
#include "mfsdp.h"

#include <algorithm>

namespace mfsdp {
namespace {

constexpr int kSortBlocks = 8;              // cluster size beyond kOneBlock tokens
// Tokens that one block sorts: 1 x 768 of 100000 rows 32 us and with the cluster 36, 300 x 768 33 and
// 37, 512 x 2048 of 32000 31 and 34, 1000 x 768 38 both, 4096 x 768 40 and 38.
constexpr int kOneBlock = 1024;
// Tokens up to which places are counted (their square's comparisons) instead of sorted, where no
// rows have to be marked: 1001 x 301 took 20 us so and 26 sorted, 3000 x 64 22 and 24, 4000 x 768
// 28 both, 8192 x 768 50 and 34.
constexpr int kRankMax = 4096;
constexpr int kRankKeys = 64;               // tokens per block that counts
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitMax = 9;                // bits per pass
constexpr int kBinsMax = 1 << kDigitMax;
constexpr int kSortSmem = (kSortWarps * kBinsMax + kBinsMax + kBinsMax + 32) * 4;
// Sorted positions per chunk: 32, or 16 while 32 would give fewer than kFewChunks blocks' work.
// 4096 tokens x 1024 took 46 us with 32 and 40 with 16, 8192 x 4096 172 and 177.
constexpr int kChunkLong = 32, kChunkShort = 16, kFewChunks = 256;
constexpr int kSumThreads = 128;
constexpr int kZeroRows = 8;                // table rows per zeroing block of the sum launch
constexpr int64_t kFillBytes = 80ll << 20;  // zeros written beside the sort (about 13 us)
constexpr int kKeep = 4;                    // positions per lane the sort keeps in registers

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
// Rows of 16-byte vectors: a unit is 8 elements of the output; a thread takes U of them, a grid
// apart, with their loads in flight together.
template <typename TT, typename TO, int U>
__global__ void __launch_bounds__(256) embedding_forward_kernel(const __grid_constant__ EmbFwd p) {
  pdl_launch();
  pdl_wait();
  const int per_row = p.dim / 8;
  const int64_t units = p.n * per_row, step = (int64_t)gridDim.x * 256;
  const int64_t u0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool small = units < (1ll << 31);
  int64_t t[U], id[U];
  int c[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t u = u0 + i * step;
    t[i] = u >= units ? -1 : small ? (int64_t)((uint32_t)u / (uint32_t)per_row) : u / per_row;
    c[i] = (int)(u - t[i] * per_row) * 8;
    id[i] = t[i] >= 0 ? load_index(p.ids, p.is64, t[i]) : 0;
  }
  Pack8<TT> a[U];
  float scale[U];                          // 0 for a row of zeros, whatever the caller's scale is
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const bool ok = t[i] >= 0 && id[i] >= 0 && id[i] < p.vocab;
    if (t[i] >= 0 && !ok && c[i] == 0) atomicOr(p.status, kStatusBadIndex);
    scale[i] = ok ? p.scale : 0.f;
    if (ok) a[i].load(static_cast<const TT*>(p.table) + id[i] * p.ld_table + c[i]); else a[i].zero();
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (t[i] < 0) continue;
    float v[8];
    a[i].get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= scale[i];
    Pack8<TO> b;
    b.set(v);
    b.store(static_cast<TO*>(p.out) + t[i] * p.ld_out + c[i]);
  }
}

// Other rows: a warp per token and 256 columns, eight elements 32 apart per lane.
constexpr int kSegment = 256;
template <typename TT, typename TO>
__global__ void __launch_bounds__(256)
    embedding_forward_any_kernel(const __grid_constant__ EmbFwd p) {
  pdl_launch();
  pdl_wait();
  const int segs = (p.dim + kSegment - 1) / kSegment;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), t = unit / segs;
  if (t >= p.n) return;
  const int c0 = (int)(unit - t * segs) * kSegment, lane = threadIdx.x & 31;
  const int64_t id = load_index(p.ids, p.is64, t);
  const bool ok = id >= 0 && id < p.vocab;
  if (!ok && c0 == 0 && lane == 0) atomicOr(p.status, kStatusBadIndex);
  const TT* src = static_cast<const TT*>(p.table) + (ok ? id : 0) * p.ld_table;
  TO* dst = static_cast<TO*>(p.out) + t * p.ld_out;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = to_f32(src[min(c0 + 32 * j + lane, p.dim - 1)]);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = c0 + 32 * j + lane;
    if (c < p.dim) dst[c] = from_f32<TO>(ok ? v[j] * p.scale : 0.f);
  }
}

// ---------------------------------------------------------------- sort
struct SortArgs {
  const void* ids;
  uint32_t *key0, *val0, *key1, *val1;   // ping-pong; the result lands in key1, val1
  uint8_t* present;                      // [vocab] written: 1 where an id occurs; nullable
  int64_t vocab, padding;
  int32_t n, is64, passes, digit;
  int* status;
  // the zeros: `fill_rows` rows of `fill_units` stores of 16 bytes (fill_vec) or of one element
  char* fill;
  int64_t fill_rows, fill_units, fill_pitch;   // pitch in bytes
  int32_t fill_vec, elem_bytes;
};

__device__ __forceinline__ void zero_fill(const SortArgs& p, int64_t first, int64_t step) {
  const int64_t total = p.fill_rows * p.fill_units;
  const bool flat = p.fill_rows == 1, small = total < (1ll << 31);
  for (int64_t u = first; u < total; u += step) {
    int64_t row = 0, c = u;
    if (!flat) {
      row = small ? (int64_t)((uint32_t)u / (uint32_t)p.fill_units) : u / p.fill_units;
      c = u - row * p.fill_units;
    }
    char* at = p.fill + row * p.fill_pitch;
    if (p.fill_vec)
      reinterpret_cast<uint4*>(at)[c] = make_uint4(0u, 0u, 0u, 0u);
    else if (p.elem_bytes == 2)
      reinterpret_cast<uint16_t*>(at)[c] = 0;
    else
      reinterpret_cast<uint32_t*>(at)[c] = 0u;
  }
}

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

// B blocks sort (the first cluster where B > 1); the grid's other blocks write zeros.
template <int B>
__global__ void __launch_bounds__(kSortThreads)
    embedding_sort_kernel(const __grid_constant__ SortArgs p) {
  auto barrier = [] {
    if (B > 1) cluster_barrier(); else __syncthreads();
  };
  extern __shared__ uint32_t sort_smem[];
  uint32_t* hist = sort_smem;                          // [warp][bin], then write positions
  uint32_t* total = hist + kSortWarps * kBinsMax;      // this block's digit totals
  uint32_t* base = total + kBinsMax;                   // first position of (digit, this block)
  uint32_t* scan = base + kBinsMax;
  pdl_launch();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x >= B) {                               // whole clusters: zeros only
    zero_fill(p, (int64_t)(blockIdx.x - B) * kSortThreads + tid,
              (int64_t)(gridDim.x - B) * kSortThreads);
    return;
  }
  const uint32_t rank = B > 1 ? cluster_ctarank() : 0u;
  const int bins = 1 << p.digit;
  // every warp of the cluster owns one contiguous share of the positions; a short share's keys
  // stay in registers between counting and placing
  const int64_t share = (p.n + B * kSortWarps - 1) / (B * kSortWarps);
  const int64_t i0 = ((int64_t)rank * kSortWarps + warp) * share;
  const int64_t i1 = i0 + share < p.n ? i0 + share : (int64_t)p.n;
  const bool keep = share <= 32 * kKeep;
  // (the array is padded to its 16-byte stores; a barrier of the first pass precedes the marks)
  if (p.present)
    for (int64_t i = (int64_t)rank * kSortThreads + tid; i < (p.vocab + 15) / 16;
         i += B * kSortThreads)
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
    auto key_at = [&](int64_t i, bool check) -> uint32_t {
      if (pass > 0) return ks[i];
      const int64_t id = load_index(p.ids, p.is64, i);
      const bool in = id >= 0 && id < p.vocab;
      if (check && !in && id != p.padding) atomicOr(p.status, kStatusBadIndex);
      return in && id != p.padding ? (uint32_t)id : (uint32_t)p.vocab;
    };
    auto val_at = [&](int64_t i) -> uint32_t { return pass > 0 ? vs[i] : (uint32_t)i; };
    uint32_t kk[kKeep], vv[kKeep];
    if (keep) {
#pragma unroll
      for (int u = 0; u < kKeep; ++u) {
        const int64_t i = i0 + 32 * u + lane;
        kk[u] = i < i1 ? key_at(i, true) : 0u;
        vv[u] = i < i1 ? val_at(i) : 0u;
      }
    }
    for (int b = tid; b < kSortWarps * bins; b += kSortThreads) hist[b] = 0u;
    __syncthreads();
    uint32_t* mine = hist + warp * bins;
    if (keep) {
#pragma unroll
      for (int u = 0; u < kKeep; ++u)
        if (i0 + 32 * u + lane < i1) atomicAdd(&mine[(kk[u] >> shift) & (bins - 1)], 1u);
    } else {
      for (int64_t i = i0 + lane; i < i1; i += 32)
        atomicAdd(&mine[(key_at(i, true) >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // per digit: exclusive sums over this block's warps, and the block's total
    if (tid < bins) {
      uint32_t c[kSortWarps], s = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * bins + tid];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        hist[w * bins + tid] = s;
        s += c[w];
      }
      total[tid] = s;
    }
    barrier();
    // digit b of this block starts after all smaller digits and the same digit of the blocks
    // before it
    uint32_t all = 0, before = 0;
    if (tid < bins) {
      uint32_t c[B];
#pragma unroll
      for (int q = 0; q < B; ++q) c[q] = B > 1 ? ld_cluster_u32(total + tid, (uint32_t)q) : total[tid];
#pragma unroll
      for (int q = 0; q < B; ++q) {
        all += c[q];
        if ((uint32_t)q < rank) before += c[q];
      }
    }
    uint32_t x = all;   // inclusive scan over the digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    // the sum of the warps before: at most 16 warps hold digits
    uint32_t ahead = 0;
#pragma unroll
    for (int w = 0; w < kBinsMax / 32; ++w) ahead += w < warp ? scan[w] : 0u;
    if (tid < bins) base[tid] = x - all + ahead + before;
    __syncthreads();
    // place, 32 positions at a time, in order: a lane's rank is the number of lower lanes with
    // its digit
    auto place = [&](bool live, uint32_t k, uint32_t v) {
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
        if (p.present && pass == p.passes - 1 && k < (uint32_t)p.vocab) p.present[k] = 1;
      }
    };
    if (keep) {
#pragma unroll
      for (int u = 0; u < kKeep; ++u) place(i0 + 32 * u + lane < i1, kk[u], vv[u]);
    } else {
      for (int64_t b = i0; b < i1; b += 32) {
        const int64_t i = b + lane;
        place(i < i1, i < i1 ? key_at(i, false) : 0u, i < i1 ? val_at(i) : 0u);
      }
    }
    barrier();   // the pass's output, and the peers' totals, before the next pass
  }
}

// Few tokens: a token's place is the number of tokens that go before it, counted by comparing it
// with all of them.  Blocks of kRankKeys tokens count independently, so there is no exchange; the
// grid's other blocks write zeros.
__global__ void __launch_bounds__(kSortThreads)
    embedding_rank_kernel(const __grid_constant__ SortArgs p) {
  constexpr int kParts = kSortThreads / kRankKeys;       // threads per token
  __shared__ alignas(16) uint32_t key[kRankMax];
  __shared__ uint32_t place[kRankKeys];
  pdl_launch();
  pdl_wait();
  const int tid = threadIdx.x, blocks = (p.n + kRankKeys - 1) / kRankKeys;
  if ((int)blockIdx.x >= blocks) {
    zero_fill(p, (int64_t)((int)blockIdx.x - blocks) * kSortThreads + tid,
              (int64_t)((int)gridDim.x - blocks) * kSortThreads);
    return;
  }
  const int first = (int)blockIdx.x * kRankKeys;         // this block's tokens
  // ids outside the table and the padding id go behind every row, as key = vocab
  const int part = (p.n + 4 * kParts - 1) / (4 * kParts) * 4;  // tokens per thread, whole vectors
  for (int i = tid; i < part * kParts; i += kSortThreads) {
    uint32_t k = 0xFFFFFFFFu;                            // past the end: behind everything
    if (i < p.n) {
      const int64_t id = load_index(p.ids, p.is64, i);
      const bool in = id >= 0 && id < p.vocab;
      if (!in && id != p.padding && i >= first && i < first + kRankKeys)
        atomicOr(p.status, kStatusBadIndex);
      k = in && id != p.padding ? (uint32_t)id : (uint32_t)p.vocab;
    }
    key[i] = k;
  }
  if (tid < kRankKeys) place[tid] = 0u;
  __syncthreads();
  const int i = first + tid % kRankKeys, j0 = tid / kRankKeys * part, j1 = j0 + part;
  const uint32_t mine = i < p.n ? key[i] : 0u;
  // earlier tokens go first among equals
  uint32_t before = 0;
  if (j1 <= first || j0 >= first + kRankKeys) {          // uniform in a warp
    const uint32_t limit = mine + (j1 <= first ? 1u : 0u);
#pragma unroll 4
    for (int j = j0; j < j1; j += 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(key + j);
      before += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
    }
  } else {
    for (int j = j0; j < j1; ++j) before += key[j] < mine + (j < i ? 1u : 0u);
  }
  atomicAdd(&place[tid % kRankKeys], before);            // integers: any order
  __syncthreads();
  if (tid < kRankKeys && i < p.n) {
    p.key1[place[tid]] = mine;
    p.val1[place[tid]] = (uint32_t)i;
  }
}

// ---------------------------------------------------------------- sum and join
struct SumArgs {
  const uint32_t *key, *val;
  const uint8_t* present;
  int64_t zero_row0;           // rows from here on: zeroed by the blocks after sum_blocks
  int32_t sum_blocks, row_vec;
  const void* dy;
  void* dtable;
  float* part;                 // [chunks][2][dim]: run from before the chunk, run into the next
  int64_t ld_dy, ld_dt, vocab;
  int32_t n, dim, chunk_len, chunks;
  int32_t slabs, cols_shift;   // column threads per chunk = 1 << cols_shift
  float scale;
};

// The eight elements of column thread c in slab s: consecutive (VEC) or TX apart.
template <bool VEC>
__device__ __forceinline__ int col_of(int slab, int tx, int c, int j) {
  return VEC ? (slab * tx + c) * 8 + j : (slab * 8 + j) * tx + c;
}

// What the table holds in a thread's columns of row v (ACC: the gradient is added to it).
template <typename TG, bool VEC>
struct OldRow {
  Pack8<TG> q;
  TG e[VEC ? 1 : 8];
  __device__ __forceinline__ void load(const SumArgs& p, uint32_t v, int slab, int tx, int c) {
    const TG* row = static_cast<const TG*>(p.dtable) + (int64_t)v * p.ld_dt;
    if (VEC) {
      q.load(row + col_of<VEC>(slab, tx, c, 0));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        e[VEC ? 0 : j] = row[min(col_of<VEC>(slab, tx, c, j), p.dim - 1)];
    }
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    if (VEC) {
      q.get(o);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = to_f32(e[VEC ? 0 : j]);
    }
  }
};

template <typename TG, bool VEC, bool ACC>
__device__ __forceinline__ void write_row(const SumArgs& p, uint32_t v, int slab, int tx, int c,
                                          const float (&acc)[8], const OldRow<TG, VEC>& old) {
  TG* row = static_cast<TG*>(p.dtable) + (int64_t)v * p.ld_dt;
  float o[8];
  if (ACC) old.get(o);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = ACC ? fmaf(acc[j], p.scale, o[j]) : acc[j] * p.scale;
  if (VEC) {
    Pack8<TG> q;
    q.set(o);
    q.store(row + col_of<VEC>(slab, tx, c, 0));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = col_of<VEC>(slab, tx, c, j);
      if (e < p.dim) row[e] = from_f32<TG>(o[j]);
    }
  }
}

template <typename TD, typename TG, bool VEC, bool ACC>
__global__ void __launch_bounds__(kSumThreads) embedding_sum_kernel(const __grid_constant__ SumArgs p) {
  pdl_launch();
  pdl_wait();
  if ((int)blockIdx.x >= p.sum_blocks) {
    const int64_t r0 = p.zero_row0 + (int64_t)((int)blockIdx.x - p.sum_blocks) * kZeroRows;
    const int units = p.row_vec ? p.dim * (int)sizeof(TG) / 16 : p.dim;
    for (int64_t r = r0; r < p.vocab && r < r0 + kZeroRows; ++r) {
      if (p.present[r]) continue;
      TG* row = static_cast<TG*>(p.dtable) + r * p.ld_dt;
      for (int e = threadIdx.x; e < units; e += kSumThreads) {
        if (p.row_vec)
          reinterpret_cast<uint4*>(row)[e] = make_uint4(0u, 0u, 0u, 0u);
        else
          row[e] = from_f32<TG>(0.f);
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
  const int i0 = (int)(chunk * p.chunk_len), i1 = min(p.n, i0 + p.chunk_len);
  if (VEC && col_of<VEC>(slab, tx, c, 0) >= p.dim) return;
  const uint32_t none = (uint32_t)p.vocab;
  const uint32_t prev = i0 > 0 ? p.key[i0 - 1] : none, next = i1 < p.n ? p.key[i1] : none;
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  uint32_t cur = p.key[i0];
  bool from_before = i0 > 0 && prev == cur;
  float* part = p.part + chunk * 2 * p.dim;
  auto flush = [&](bool to_next, const OldRow<TG, VEC>& old) {
    if (cur == none) return;
    if (!from_before && !to_next) {
      write_row<TG, VEC, ACC>(p, cur, slab, tx, c, acc, old);
    } else {
      float* dst = part + (from_before ? 0 : p.dim);
      if (VEC) {
        const int e = col_of<VEC>(slab, tx, c, 0);
        Pack8<float> q;
        q.set(acc);
        if (e < p.dim) q.store(dst + e);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = col_of<VEC>(slab, tx, c, j);
          if (e < p.dim) dst[e] = acc[j];
        }
      }
    }
  };
  constexpr int U = ACC ? 4 : 8;   // rows loaded ahead; with ACC the table's rows beside them
  OldRow<TG, VEC> before, old[ACC ? U : 1];
  for (int b = i0; b < i1; b += U) {
    uint32_t k[U];
    Pack8<TD> d[U];
    float ds[VEC ? 1 : U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // unconditional loads of clamped positions: the batch is in flight together (a row that
      // takes no part is flushed under key `none`, which is not written)
      const int at = min(b + u, i1 - 1);
      k[u] = p.key[at];
      const TD* row = static_cast<const TD*>(p.dy) + (int64_t)p.val[at] * p.ld_dy;
      if (VEC) {
        d[u].load(row + col_of<VEC>(slab, tx, c, 0));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          ds[VEC ? 0 : u][j] = to_f32(row[min(col_of<VEC>(slab, tx, c, j), p.dim - 1)]);
      }
      if (ACC) old[ACC ? u : 0].load(p, k[u] == none ? 0u : k[u], slab, tx, c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u >= i1) break;
      if (k[u] != cur) {
        flush(false, u == 0 ? before : old[ACC ? u - 1 : 0]);
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
    if (ACC)   // the batch's last row
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u == min(U, i1 - b) - 1) before = old[ACC ? u : 0];
  }
  flush(i1 < p.n && next == cur, before);
}

// A run that starts in this chunk and goes on: its partial rows, in chunk order.  A block takes one
// chunk and slab; its groups of column threads (one where rows are wide) add consecutive shares of
// the partial rows, which are then added in order: 30000 x 65 fp32 54 -> 46 us for the gradient,
// wide rows unchanged (with 256 or 512 threads 2 us more there).  Most blocks find no run and leave.
template <typename TG, bool VEC, bool ACC>
__global__ void __launch_bounds__(kSumThreads) embedding_join_kernel(const __grid_constant__ SumArgs p) {
  __shared__ float sums[kSumThreads * 8];
  pdl_launch();
  pdl_wait();
  const int tx = 1 << p.cols_shift, ty = kSumThreads >> p.cols_shift;
  const int c = threadIdx.x & (tx - 1), group = threadIdx.x >> p.cols_shift;
  const int slab = (int)(blockIdx.x % p.slabs);
  const int64_t chunk = blockIdx.x / p.slabs;
  const int i0 = (int)(chunk * p.chunk_len), i1 = i0 + p.chunk_len;
  const uint32_t k = p.key[i1 - 1];
  if (k == (uint32_t)p.vocab || p.key[i1] != k) return;           // ends here
  if (i0 > 0 && p.key[i0 - 1] == k) return;                       // an earlier chunk's run
  // The chunks the run goes on into: every one whose first position still holds the id.  The
  // loads are unconditional (indices are clamped instead), so a batch is in flight together.
  const int64_t last = p.chunks - 1;
  int64_t end = chunk + 2;
  for (bool more = true; more;) {
    constexpr int kAhead = 16;
    uint32_t next[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) next[u] = p.key[min(end + u, last) * p.chunk_len];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      more = more && end <= last && next[u] == k;
      end += more ? 1 : 0;
    }
  }
  const bool in = !VEC || col_of<VEC>(slab, tx, c, 0) < p.dim;
  OldRow<TG, VEC> old;
  if (ACC && group == 0 && in) old.load(p, k, slab, tx, c);
  constexpr int U = VEC ? 12 : 4;   // partial rows loaded ahead
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  const int64_t share = (end - chunk + ty - 1) / ty, q0 = chunk + group * share;
  const int64_t q1 = min(end, q0 + share);
  for (int64_t q = q0; q < q1 && in; q += U) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // the first chunk's partial row is its run into the next chunk, the others' the run from
      // before
      const int64_t at = min(q + u, q1 - 1);
      const float* src = p.part + (at * 2 + (at == chunk ? 1 : 0)) * p.dim;
      if (VEC) {
        Pack8<float> w;
        w.load(src + col_of<VEC>(slab, tx, c, 0));
        w.get(v[u]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[u][j] = src[min(col_of<VEC>(slab, tx, c, j), p.dim - 1)];
      }
    }
    asm volatile("" ::: "memory");  // all of them in flight before the first is added
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += q + u < q1 ? v[u][j] : 0.f;
  }
  if (ty > 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[j * kSumThreads + threadIdx.x] = acc[j];
    __syncthreads();
    if (group != 0) return;
    for (int g = 1; g < ty; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += sums[j * kSumThreads + (g << p.cols_shift) + c];
  }
  if (!in) return;
  write_row<TG, VEC, ACC>(p, k, slab, tx, c, acc, old);
}

// ---------------------------------------------------------------- host
size_t up256(size_t b) { return (b + 255) / 256 * 256; }
int64_t cdiv(int64_t x, int64_t a) { return (x + a - 1) / a; }

// The columns are cut into slabs of at most kSumThreads threads of 8 columns.
int64_t slabs_of(int64_t dim) { return cdiv(cdiv(dim, 8), kSumThreads); }
int64_t chunk_len(int64_t n, int64_t dim) {
  return cdiv(n, kChunkLong) * slabs_of(dim) < kFewChunks ? kChunkShort : kChunkLong;
}

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
  const int64_t len = chunk_len(n, dim);
  l.part = take((size_t)cdiv(n, len) * 2 * (size_t)dim * 4);
  l.total = off;
  return l;
}

int check_table(int64_t vocab, int64_t dim, int64_t n) {
  if (vocab < 1 || dim < 1 || n < 0 || vocab >= (1ll << 31) - 1 || dim >= (1ll << 27) ||
      n >= (1ll << 31) - kChunkLong)
    return MFSDP_ESHAPE;
  return MFSDP_OK;
}

bool vec_ok(const void* p, int64_t ld, int64_t dim, int32_t dtype) {
  return aligned_to(p, 16) && dim % 8 == 0 && (ld * (int64_t)dtype_bytes(dtype)) % 16 == 0;
}

template <typename TT, typename TO>
cudaError_t run_forward(const EmbFwd& a, bool vec, int sms, cudaStream_t st) {
  if (!vec)
    return launch_pdl(embedding_forward_any_kernel<TT, TO>,
                      dim3((unsigned)cdiv(a.n * cdiv(a.dim, kSegment), 8)), dim3(256), 0, st, a);
  // four units per thread once that still fills the GPU
  const int64_t units = a.n * (a.dim / 8);
  if (units > (int64_t)sms * 2048 * 2)
    return launch_pdl(embedding_forward_kernel<TT, TO, 4>, dim3((unsigned)cdiv(units, 1024)),
                      dim3(256), 0, st, a);
  return launch_pdl(embedding_forward_kernel<TT, TO, 1>, dim3((unsigned)cdiv(units, 256)), dim3(256), 0,
                    st, a);
}

template <int B>
cudaError_t launch_sort(const SortArgs& a, int64_t fill_blocks, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(
      embedding_sort_kernel<B>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = B;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(B + cdiv(fill_blocks, B) * B));   // whole clusters
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = kSortSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = B > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, embedding_sort_kernel<B>, a);
}

template <typename TD, typename TG, bool VEC, bool ACC>
cudaError_t launch_sum(const SumArgs& a, int64_t zero_blocks, cudaStream_t st) {
  const dim3 all((unsigned)(a.sum_blocks + zero_blocks)), b(kSumThreads);
  const cudaError_t e = launch_pdl(embedding_sum_kernel<TD, TG, VEC, ACC>, all, b, 0, st, a);
  if (e != cudaSuccess || a.chunks < 2) return e;
  // (the last chunk's runs go nowhere)
  return launch_pdl(embedding_join_kernel<TG, VEC, ACC>,
                    dim3((unsigned)((a.chunks - 1) * a.slabs)), b, 0, st, a);
}

template <typename TD, typename TG>
cudaError_t run_sum(const SumArgs& a, bool vec, bool acc, int64_t zero_blocks, cudaStream_t st) {
  if (vec)
    return acc ? launch_sum<TD, TG, true, true>(a, zero_blocks, st)
               : launch_sum<TD, TG, true, false>(a, zero_blocks, st);
  return acc ? launch_sum<TD, TG, false, true>(a, zero_blocks, st)
             : launch_sum<TD, TG, false, false>(a, zero_blocks, st);
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
  // blocks of the launch
  if ((vec ? cdiv(n_tokens * (dim / 8), 1024) : cdiv(n_tokens * cdiv(dim, kSegment), 8)) >= (1ll << 31))
    return MFSDP_ESHAPE;
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
  a.status = device_status();
  if (!a.status) return MFSDP_ECUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool tb = table_dtype == MFSDP_DTYPE_BF16, ob = out_dtype == MFSDP_DTYPE_BF16;
  auto run = [&](auto in, auto out_t) {
    using TT = decltype(in);
    using TO = decltype(out_t);
    return run_forward<TT, TO>(a, vec, sms, st);
  };
  const cudaError_t e = tb ? (ob ? run(bf16_t(), bf16_t()) : run(bf16_t(), 0.f))
                           : (ob ? run(0.f, bf16_t()) : run(0.f, 0.f));
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
  int* status = device_status();
  if (!status) return MFSDP_ECUDA;
  char* ws = static_cast<char*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);

  SortArgs s{};
  s.ids = ids;
  s.key0 = reinterpret_cast<uint32_t*>(ws + l.key0);
  s.val0 = reinterpret_cast<uint32_t*>(ws + l.val0);
  s.key1 = reinterpret_cast<uint32_t*>(ws + l.key1);
  s.val1 = reinterpret_cast<uint32_t*>(ws + l.val1);
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
  a.dy = dy;
  a.dtable = dtable;
  a.part = reinterpret_cast<float*>(ws + l.part);
  a.ld_dy = ld_dy;
  a.ld_dt = ld_dtable;
  a.vocab = vocab;
  a.n = (int32_t)n_tokens;
  a.dim = (int32_t)dim;
  a.chunk_len = (int32_t)chunk_len(n_tokens, dim);
  a.chunks = (int32_t)cdiv(n_tokens, a.chunk_len);
  a.scale = scale;
  const int64_t col_threads = (dim + 7) / 8;
  while ((1 << a.cols_shift) < kSumThreads && (1 << a.cols_shift) < col_threads) ++a.cols_shift;
  const int64_t tx = 1ll << a.cols_shift, ty = kSumThreads / tx;
  a.slabs = (int32_t)slabs_of(dim);
  const int64_t grid = ((int64_t)a.chunks * a.slabs + ty - 1) / ty;
  if ((int64_t)a.chunks * a.slabs >= (1ll << 31)) return MFSDP_ESHAPE;
  if (n_tokens == 0 && accumulate) return MFSDP_OK;

  // zeros: the first rows beside the sort, the rest beside the sums (all of them beside the
  // sort where there are no sums); a table without gaps is one row
  int64_t fill_blocks = 0, zero_blocks = 0;
  if (!accumulate) {
    const int64_t gb = (int64_t)dtype_bytes(grad_dtype);
    const bool flat = ld_dtable == dim || vocab == 1;
    const int64_t first = std::min(vocab, n_tokens == 0 ? vocab : cdiv(kFillBytes, dim * gb));
    const int64_t row_bytes = (flat ? first * dim : dim) * gb;
    s.fill = static_cast<char*>(dtable);
    s.fill_rows = flat ? 1 : first;
    s.fill_pitch = ld_dtable * gb;
    s.fill_vec = aligned_to(dtable, 16) && row_bytes % 16 == 0 && (flat || s.fill_pitch % 16 == 0);
    s.elem_bytes = (int32_t)gb;
    s.fill_units = row_bytes / (s.fill_vec ? 16 : gb);
    fill_blocks = std::min(cdiv(s.fill_rows * s.fill_units, kSortThreads),
                           (int64_t)(2 * sms - kSortBlocks));
    if (first < vocab) {
      s.present = reinterpret_cast<uint8_t*>(ws + l.present);
      a.present = s.present;
      a.zero_row0 = first;
      a.row_vec = aligned_to(dtable, 16) && (dim * gb) % 16 == 0 && s.fill_pitch % 16 == 0;
      zero_blocks = cdiv(vocab - first, kZeroRows);
    }
  }
  a.sum_blocks = (int32_t)grid;
  if (grid + zero_blocks >= (1ll << 31)) return MFSDP_ESHAPE;
  const bool vec = vec_ok(dtable, ld_dtable, dim, grad_dtype) &&
                   (n_tokens == 0 || vec_ok(dy, ld_dy, dim, dy_dtype));

  // (counting marks no rows: the zeros beside it have to cover the table)
  cudaError_t e = cudaSuccess;
  if (n_tokens <= kRankMax && !s.present) {
    const int64_t blocks = cdiv(n_tokens, kRankKeys) + fill_blocks;
    if (blocks > 0)
      e = launch_pdl(embedding_rank_kernel, dim3((unsigned)blocks), dim3(kSortThreads), 0, st, s);
  } else {
    e = n_tokens <= kOneBlock && s.present ? launch_sort<1>(s, fill_blocks, st)
                                           : launch_sort<kSortBlocks>(s, fill_blocks, st);
  }
  if (e == cudaSuccess && n_tokens > 0) {
    const bool db = dy_dtype == MFSDP_DTYPE_BF16, gb = grad_dtype == MFSDP_DTYPE_BF16;
    e = db ? (gb ? run_sum<bf16_t, bf16_t>(a, vec, accumulate != 0, zero_blocks, st)
                 : run_sum<bf16_t, float>(a, vec, accumulate != 0, zero_blocks, st))
           : (gb ? run_sum<float, bf16_t>(a, vec, accumulate != 0, zero_blocks, st)
                 : run_sum<float, float>(a, vec, accumulate != 0, zero_blocks, st));
  }
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}
