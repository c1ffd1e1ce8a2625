// Softmax cross entropy of an output head, per token, without keeping the logits, and its
// gradient for the hidden states and the head's weight.
//
//     Z = H W^T,  lse_t = log sum_v exp Z_tv,  loss_t = lse_t - Z_{t, label_t}
//     G_tv = (exp(Z_tv - lse_t) - [v = label_t]) dloss_t,  dH = G W,  dW = G^T H
//
// Forward computes Z tile by tile on the tensor cores; a tile's epilogue reduces each row to
// (max, sum of exp(z - max)) and picks the label's logit, so Z never leaves the SM.  A small
// launch then joins the tiles' pairs.  Backward walks the vocabulary in pieces: it recomputes a
// piece of Z from the same operands, writes that piece of G, and multiplies it with W's rows for dH
// and with H for that piece's rows of dW.  dH is summed over the pieces in fp32.  One launch
// multiplies a piece of G and computes the next one (two pieces are kept): the many short tiles of
// Z fill the SMs that the few long ones of dH and dW would leave idle at a launch's end.
//
// On the tensor cores G is rounded to bf16, each entry to within 2^-8: the only rounding between
// the inputs and the gradients, and what lets both products run at the bf16 rate.  dloss enters as
// its ratio to the largest |dloss|, which the gradients are multiplied with in fp32 at the end, so a
// uniform dloss is not rounded at all.  A row of G sums to zero, so what all rows of W have in
// common, c, cancels in dH; of rounded entries it would leave (sum of the rounded row) c, which
// grows with c while dH does not.  That part is taken off: dH = G W - (sum_v G_tv) c, in which no
// error of G meets c any more (any c is exact; the mean of some rows of W is used).  With a common
// part of ten times W's spread and confident labels the relative error of dH is 0.0025 instead of
// 0.021 (rounding dH to bf16 alone is 0.0017).
//
// Tokens with the ignored label are dropped before any product: a first launch copies the live
// rows of H together (padded to whole TMA rows), so they cost nothing, and whatever they hold
// (NaN too) reaches no output.  The number of live rows stays on the device.
//
// bf16 inputs run on the CTA-pair tcgen05 kernel below (256 x 256 tiles, TMA operands,
// accumulators in tensor memory).  fp32 inputs run on the library's fp32 GEMM (3xTF32) with a
// piece of Z in the workspace.  Small products of both run on the CUDA cores.  Up to four tokens
// (forward one and backward two, with bf16 inputs that TMA can read) take one pass over W in each
// direction, without tensor cores.
//
// Training sizes are bound by the tensor cores: four products, forward's Z, its second computation,
// dH and dW.  The second costs 2 K / 1.9e15 s a logit, and storing Z in fp32 and reading it again 8
// / 6.8e12: equal at a width K of 1100, so below it recomputing is the faster way.  Above it (4096
// wide: 1.7 ms of products against 0.5 ms) keeping Z would be, for n x vocab x 4 bytes (1.6 GB) held
// from one pass to the other, which these calls do not ask of the caller.  Measured (bf16, both
// passes, 1910 TFLOP/s being a large library product's rate): 8192 tokens x 768 against 50257 rows
// in 1.57 ms, 1.72 when called back to back, 1.6 and 1.5 PFLOP/s of the four products; 3072 live
// tokens of 4096 x 4096 against 128256 rows in 7.4 to 7.8 ms, 1.65 to 1.75 PFLOP/s, where the power
// limit lowers the clock.  Forward alone runs at 1.85 and 2.0 PFLOP/s; a piece of the backward pass
// at 768 keeps the tensor cores 78 % busy and reads 0.55 GB, the sums of dH and the pieces of G,
// which stay in the L2 in part (72 % hits).  One token against 50257 x 768 takes 19 us for W's 77
// MB where W comes from memory (4.0 TB/s; 11 us at a copy's rate), 14 where it is in the L2.
#include <algorithm>
#include <atomic>
#include <cstring>
#include <new>
#include <type_traits>
#include <vector>

#include "elem.cuh"
#include "mfsdp.h"
#include "umma.cuh"

namespace mfsdp {
namespace {

constexpr int kTile = 256;                 // tile rows and columns of a CTA pair
constexpr int kHeadThreads = 320;          // warp 0 TMA, warp 1 MMA, warps 2-9 epilogue
constexpr int kHeadEpiWarps = 8;
constexpr int kHeadChunks = 4;             // 32-column chunks per epilogue warp
constexpr int kHeadStages = 6;
constexpr uint32_t kHalf = 128 * kBK * 2;  // 16 KB: one operand half of one CTA
constexpr uint32_t kHeadStageBytes = 2 * kHalf;
constexpr uint32_t kHeadStaging = kHeadStages * kHeadStageBytes;
constexpr uint32_t kStagePerWarp = 4096;   // two 32 x 32 bf16 blocks or one of fp32
constexpr uint32_t kHeadBars = kHeadStaging + kHeadEpiWarps * kStagePerWarp;
constexpr uint32_t kHeadSmem = 1024 + kHeadBars + 256;
static_assert(kHeadSmem <= 227 * 1024, "shared memory");
constexpr float kLog2e = 1.4426950408889634f;
// k-blocks added up in tensor memory before the epilogue adds them in registers (forward only).
// The tensor cores' fp32 accumulation does not round to nearest: each of the K / 16 additions
// cuts towards zero, which shrinks a logit by some 2e-9 K of itself.  1024 of K per chunk keeps
// loss and lse within about 1e-6 at any width; the backward pass rounds to bf16 after it.
constexpr int kSumBlocks = 16;

enum Phase : int { kStats = 0, kGrads = 1 };
enum Kind : int { kDh = 0, kDw = 1, kZ = 2 };  // tiles of a kGrads launch (kStats: kZ only)

struct HeadArgs {
  CUtensorMap h_k, h_mn;                   // compacted H: 64 x 128 K-major box, 3D MN-major view
  CUtensorMap w_k, w_mn;                   // W (or the copy of a piece): 64 x 128 box, and 64 x 64
                                           // boxes or the 3D view
  CUtensorMap g_k, g_mn;                   // G pieces: 64 x 128 box, 3D view
  CUtensorMap dw_st, acc_st;               // dW bf16 and dH fp32 32 x 32 stores
  const int32_t* nlive;                    // live rows
  const int32_t* label;                    // [rows] of the compacted rows
  const float* lse2;                       // [rows] lse * log2(e)
  const float* dl;                         // [rows] dloss
  const float* dl_max;                     // [dl_blocks] largest finite |dloss| per gather block
  float* scale;                            // the largest of them, for the last launch
  int32_t dl_blocks;
  float2* part;                            // [column half-tiles][rows] (max, sum)
  float* zlab;                             // [rows] the label's logit
  uint16_t* dw;                            // unaligned dW rows (dw_tma == 0)
  int64_t ld_dw;
  float* gsum;                             // [rows][gsum_parts] a row's sums of rounded G, over the
  int32_t gsum_parts;                      // same half-tile of every piece; null without dH
  uint16_t* g;                             // G pieces, rows of `piece` entries
  int64_t piece;
  int32_t dim;
  // the piece whose G is multiplied and the piece of Z that is computed (kGrads: the next one):
  // columns [v0, v0 + width) of the vocabulary, W's map row of column v0, and the first row of
  // the piece's G; width 0 where there is none
  int32_t v0, width, w_row0, g_row0;
  int32_t z_v0, z_width, z_w_row0, z_g_row0;
  int32_t rows;                            // allocated rows (pitch of part, slices of acc)
  int32_t splits;                          // dH: slices of the piece's columns
  int32_t add;                             // dH: add to the slices instead of writing them
  int32_t want_dh, want_dw, dw_tma;
  int32_t w_3d;                            // w_mn is the 3D MN-major view (whole 64-column chunks)
  int32_t group;                           // tile rows that walk the columns together
  uint64_t wait_limit_ns;
  int* status;
};

struct HeadTile {
  int kind, tm, tn;
  int kb0, nk;                             // k-blocks
  int split;
};

// The tiles of one pair, in order: the kind with the longest contraction first, each kind dealt
// so that the pairs' loads (in k-blocks) stay level.  Dealing a kind of n tiles of k: pairs of
// equal load form a group; every group gets whole rounds up to the mean load, and what is left
// goes one by one to the pairs in order of load.  Within a group the tiles are interleaved, so
// pairs that run at the same time work on neighbouring tiles and share operands in the L2.
template <int PHASE>
struct TileList {
  struct Deal {                            // this pair's share of one kind
    int kind, count, rounds, base, stride, rest;
  };
  static constexpr int kKinds = PHASE == kStats ? 1 : 3;
  static constexpr int kNone = 0x7FFFFFFF; // load of an empty group
  int live, ntm, ntn, ntd, kdh, npairs;
  Deal deal[kKinds];
  int z_step, z_dn, z_dm;                  // a step of npairs Z tiles, in columns and rows

  __device__ __forceinline__ TileList(const HeadArgs& p, int pair, int npairs_) {
    npairs = npairs_;
    live = *p.nlive;
    ntm = (live + kTile - 1) / kTile;
    ntn = (p.z_width + kTile - 1) / kTile;
    ntd = (p.dim + kTile - 1) / kTile;
    z_step = npairs;
    z_dn = ntm > 0 ? npairs / ntm : 0;
    z_dm = npairs - z_dn * ntm;
    const int kbp = (p.width + kBK - 1) / kBK;
    kdh = (kbp + p.splits - 1) / p.splits;
    if (PHASE == kStats) {                 // equal tiles: round robin
      deal[0] = Deal{kZ, ntm * ntn, 0, 0, npairs, pair};
      return;
    }
    int kind[3] = {kDh, kDw, kZ};
    int n[3] = {p.want_dh && p.width > 0 ? ntm * ntd * p.splits : 0,
                p.want_dw ? (p.width + kTile - 1) / kTile * ntd : 0, ntm * ntn};
    int k[3] = {kdh, (live + kBK - 1) / kBK, (p.dim + kBK - 1) / kBK};
#pragma unroll
    for (int a = 0; a < 3; ++a)            // longest contraction first
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (k[b] < k[b + 1]) {
          int t = k[b]; k[b] = k[b + 1]; k[b + 1] = t;
          t = n[b]; n[b] = n[b + 1]; n[b + 1] = t;
          t = kind[b]; kind[b] = kind[b + 1]; kind[b + 1] = t;
        }
    // The groups in order of load, empty ones last.  Every loop runs over all four with constant
    // indices, so they stay in registers: each thread goes through this before its first tile.
    int first[4] = {0, 0, 0, 0}, cnt[4] = {npairs, 0, 0, 0}, load[4] = {0, kNone, kNone, kNone};
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      Deal d{kind[c], n[c], 0, 0, 1, 0};
      const int kc = max(k[c], 1);
      if (n[c] > 0) {
        int64_t total = (int64_t)n[c] * kc;
#pragma unroll
        for (int g = 0; g < 4; ++g) total += (int64_t)cnt[g] * (cnt[g] > 0 ? load[g] : 0);
        int level = total < (1ll << 31) ? (int)((uint32_t)total / (uint32_t)npairs)
                                        : (int)(total / npairs);
        int given, q[4];
        do {                               // lower where a group is above the mean
          given = 0;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            q[g] = cnt[g] > 0 && level > load[g] ? (int)((uint32_t)(level - load[g]) / (uint32_t)kc) : 0;
            given += q[g] * cnt[g];
          }
          level -= kc;
        } while (given > n[c]);
        int base = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (pair >= first[g] && pair < first[g] + cnt[g]) {
            d.rounds = q[g];
            d.base = base + pair - first[g];
            d.stride = cnt[g];
          }
          base += q[g] * cnt[g];
          if (cnt[g] > 0) load[g] += q[g] * kc;
        }
        sort_groups(first, cnt, load);
        // what is left, in order of load
        const int rest = n[c] - base, full = rest < npairs ? 0 : rest / npairs;
        const int extra = rest - full * npairs;
        int before = 0, cut = 0, cut_first = 0, cut_load = kNone;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (pair >= first[g] && pair < first[g] + cnt[g]) d.rest = base + before + pair - first[g];
          const int took = max(0, min(extra - before, cnt[g]));   // pairs of it with one tile more
          before += cnt[g];
          if (cnt[g] == 0) continue;
          load[g] += full * kc;
          if (took > 0 && took < cnt[g]) {                        // at most one group is cut
            cut = cnt[g] - took;
            cut_first = first[g] + took;
            cut_load = load[g];
            cnt[g] = took;
          }
          if (took > 0) load[g] += kc;
        }
        if (cut > 0) {                     // the last place is free: two kinds make three groups
          first[3] = cut_first;
          cnt[3] = cut;
          load[3] = cut_load;
        }
        sort_groups(first, cnt, load);
      }
      deal[c] = d;
    }
  }

  // Four groups by load.
  static __device__ __forceinline__ void sort_groups(int (&first)[4], int (&cnt)[4], int (&load)[4]) {
#pragma unroll
    for (int a = 0; a < 3; ++a)
#pragma unroll
      for (int b = 0; b < 3 - a; ++b)
        if (load[b] > load[b + 1]) {
          int t = load[b]; load[b] = load[b + 1]; load[b + 1] = t;
          t = cnt[b]; cnt[b] = cnt[b + 1]; cnt[b + 1] = t;
          t = first[b]; first[b] = first[b + 1]; first[b + 1] = t;
        }
  }

  // Tiles of this pair in deal c, and the contraction of its i-th one.
  __device__ __forceinline__ int tiles_of(int c) const {
    const Deal& d = deal[c];
    return d.rounds + (d.rest < d.count ? (d.count - d.rest - 1) / npairs + 1 : 0);
  }
  __device__ __forceinline__ int index_of(int c, int i) const {
    const Deal& d = deal[c];
    return i < d.rounds ? d.base + i * d.stride : d.rest + (i - d.rounds) * npairs;
  }
  __device__ __forceinline__ int blocks_of(const HeadArgs& p, int c, int i) const {
    if (deal[c].kind == kZ) return (p.dim + kBK - 1) / kBK;
    if (deal[c].kind == kDw) return (live + kBK - 1) / kBK;
    const int split = p.splits == 1 ? 0 : index_of(c, i) / (ntm * ntd);
    return max(0, min(kdh, (p.width + kBK - 1) / kBK - split * kdh));
  }
  // The tile of an index.  Z tiles are short, so a tile that lies `step` indices after the one
  // in t, in the same group of rows, is found without a division.
  __device__ __forceinline__ void locate(const HeadArgs& p, int kind, int idx, HeadTile& t) const {
    t.kind = kind;
    t.kb0 = 0;
    t.split = 0;
    if (kind == kZ) {
      // groups of `group` tile rows walk the columns together: a W panel is read once per
      // group, and the group's rows of H stay in the L2
      const int per = p.group * ntn, g = idx / per, in = idx - g * per;
      const int rows = min(p.group, ntm - g * p.group);
      t.tn = in / rows;
      t.tm = g * p.group + (in - t.tn * rows);
      t.nk = (p.dim + kBK - 1) / kBK;
    } else if (kind == kDh) {
      t.tm = idx % ntm;
      const int rest = idx / ntm;
      t.tn = rest % ntd;
      t.split = rest / ntd;
      t.kb0 = t.split * kdh;
      t.nk = max(0, min(kdh, (p.width + kBK - 1) / kBK - t.kb0));
    } else {
      t.tm = idx / ntd;
      t.tn = idx - t.tm * ntd;
      t.nk = (live + kBK - 1) / kBK;
    }
  }
};

// Walks the tiles of a pair.
template <int PHASE>
struct TileWalk {
  const TileList<PHASE>& l;
  int c, i, left, idx;                     // deal, position in it, tiles left in it, index
  HeadTile t;
  bool have;
  __device__ __forceinline__ TileWalk(const HeadArgs& p, const TileList<PHASE>& list) : l(list) {
    c = -1;
    i = left = idx = 0;
    t = HeadTile{};
    have = true;
    next(p);
  }
  __device__ __forceinline__ void next(const HeadArgs& p) {
    int kind = kZ, at = 0;
    if (--left > 0) {
      ++i;
#pragma unroll
      for (int k = 0; k < TileList<PHASE>::kKinds; ++k)
        if (k == c) {
          kind = l.deal[k].kind;
          at = l.index_of(k, i);
        }
    } else {
      left = 0;
#pragma unroll
      for (int k = 0; k < TileList<PHASE>::kKinds; ++k)
        if (k > c && left == 0) {
          left = l.tiles_of(k);
          if (left > 0) {
            c = k;
            kind = l.deal[k].kind;
            at = l.index_of(k, 0);
          }
        }
      i = 0;
      if (left == 0) {
        have = false;
        return;
      }
    }
    const int step = at - idx;
    idx = at;
    // the common case of short tiles: the next one of the same, only group of rows
    if (kind == kZ && t.kind == kZ && i > 0 && l.ntm <= p.group && step == l.z_step) {
      t.tn += l.z_dn;
      t.tm += l.z_dm;
      if (t.tm >= l.ntm) {
        t.tm -= l.ntm;
        ++t.tn;
      }
      return;
    }
    l.locate(p, kind, at, t);
  }
};

__device__ __forceinline__ void tma_reduce_add_block(const CUtensorMap* map, uint32_t src, int x,
                                                     int y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];"
      ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(src)
      : "memory");
}

// fp32 staging block, 32 rows x 128 bytes in the 128-byte swizzle of the accumulator's map:
// chunk k (16 bytes) of row r lies at k ^ (r & 7).  The block is 1024-byte aligned.
__device__ __forceinline__ uint32_t stg32_off(int r, int k) {
  return (uint32_t)(r * 128 + ((k ^ (r & 7)) << 4));
}

// 16 consecutive fp32 columns of this thread's TMEM lane; waits for the load to land.
__device__ __forceinline__ void tc_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 2^x to about 2 ulp, one instruction (results below 2^-126 are 0): the terms of a softmax sum.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// lo += the bf16 in w's lower half, hi += the one in its upper half: fp32 sums, one instruction each.
__device__ __forceinline__ void add_bf16x2(uint32_t w, float& lo, float& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n add.rn.f32.bf16 %0, a, %0;\n"
      " add.rn.f32.bf16 %1, b, %1;\n}\n"
      : "+f"(lo), "+f"(hi)
      : "r"(w));
}

template <int PHASE>
__global__ void __launch_bounds__(kHeadThreads, 1) head_gemm_kernel(const __grid_constant__ HeadArgs P) {
  constexpr int S = kHeadStages;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kHeadBars);
  // bars: full[S] | empty[S] | tfull[2] | tempty[2] | drain
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int full0 = 0, empty0 = S, tfull0 = 2 * S, tempty0 = 2 * S + 2, drain = 2 * S + 4;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar(full0 + s), 1);
      mbar_init(bar(empty0 + s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar(tfull0 + a), 1);
      mbar_init(bar(tempty0 + a), 2 * kHeadEpiWarps);
    }
    mbar_init(bar(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the previous launch's results
  const uint32_t tmem_base = *tmem_slot;
  uint32_t peer_base;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(peer_base)
               : "r"(map_rank(smem_u32(tmem_slot), rank ^ 1u))
               : "memory");
  const bool usable = peer_base == tmem_base;
  if (!usable && threadIdx.x == 0) atomicOr(P.status, kStatusTmemMismatch);
  const Guard g{abort_flag, P.wait_limit_ns, P.status};
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const TileList<PHASE> tiles(P, pair, npairs);

  if (!usable) {
    // nothing runs: fall through to the teardown
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producers (both CTAs)
    // One thread issues both operands of every k-block: its copies have warp-uniform operands,
    // where several issuing lanes make the compiler walk the lanes copy by copy (four lanes:
    // 1.66 ms for a 768-wide training step of 8192 tokens, one lane 1.59).  The leader arms the
    // stage's full barrier for the bytes of both CTAs.
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 1;             // of the empty barriers: the first round passes
      uint32_t armed = 0, last_par = 0;
      bool ok = true;
      for (TileWalk<PHASE> walk(P, tiles); walk.have && ok; walk.next(P)) {
        const HeadTile& t = walk.t;
        const int a0 = t.tm * kTile + 128 * (int)rank, b0 = t.tn * kTile + 128 * (int)rank;
        for (int kb = 0; kb < t.nk; ++kb) {
          if (!mbar_wait(bar(empty0 + stage), ph, g)) { ok = false; break; }
          const uint32_t fb_local = bar(full0 + stage), fb = map_rank(fb_local, 0);
          const uint32_t dst = sbase + (uint32_t)stage * kHeadStageBytes;
          const int k0 = (t.kb0 + kb) * kBK;
          expect_tx_p(leader, fb_local, 2u * kHeadStageBytes);
          // Z: A = H rows, B = W rows, both with the contraction contiguous; dH: A = G rows
          // (K-major), B = W (its rows are the contraction: MN-major); dW: A = G and B = H, both
          // MN-major with the tokens as the contraction
          if (PHASE == kStats || t.kind == kZ) {
            tma_load_pair_p(true, dst, &P.h_k, k0, a0, fb);
            tma_load_pair_p(true, dst + kHalf, &P.w_k, k0, P.z_w_row0 + b0, fb);
          } else if (t.kind == kDh) {
            tma_load_pair_p(true, dst, &P.g_k, k0, P.g_row0 + a0, fb);
            if (P.w_3d) {
              tma_load3d_pair_p(true, dst + kHalf, &P.w_mn, 0, P.w_row0 + k0, b0 / 64, fb);
            } else {
              tma_load_pair_p(true, dst + kHalf, &P.w_mn, b0, P.w_row0 + k0, fb);
              tma_load_pair_p(true, dst + kHalf + kBoxBytes, &P.w_mn, b0 + 64, P.w_row0 + k0, fb);
            }
          } else {
            tma_load3d_pair_p(true, dst, &P.g_mn, 0, P.g_row0 + k0, a0 / 64, fb);
            tma_load3d_pair_p(true, dst + kHalf, &P.h_mn, 0, k0, b0 / 64, fb);
          }
          armed |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | ((ph ^ 1u) << stage);
          if (++stage == S) { stage = 0; ph ^= 1u; }
        }
      }
      // teardown: the leader's full barriers count both CTAs' bytes
      if (leader)
        for (int st = 0; st < S; ++st)
          if (armed & (1u << st)) mbar_wait(bar(full0 + st), (last_par >> st) & 1u, g, false);
    }
  } else if (warp == 1 && lane == 0 && leader) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    // One thread issues every MMA, so what it does between them has to stay below the MMAs' own
    // time: the operands' storage is a constant of each loop, and of a tile it needs the number
    // of k-blocks only.
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    auto deal = [&](int c, auto a_mn, auto b_mn) -> bool {
      constexpr int A = decltype(a_mn)::value, B = decltype(b_mn)::value;
      constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)A << 15) |
                                 ((uint32_t)B << 16) | ((uint32_t)(kTile >> 3) << 17) |
                                 ((uint32_t)(kTile >> 4) << 24);
      const int n = tiles.tiles_of(c);
      for (int i = 0; i < n; ++i) {
        int left = tiles.blocks_of(P, c, i);
        do {                                              // once, or a chunk at a time (kStats)
          const int nk = PHASE == kStats ? min(left, kSumBlocks) : left;
          left -= nk;
          if (!mbar_wait_cl(bar(tempty0 + acc), acc_phase ^ 1u, g)) return false;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kTile);
          for (int kb = 0; kb < nk; ++kb) {
            if (!mbar_wait(bar(full0 + stage), phase, g)) return false;
            tc_fence_after();
            const uint32_t sa = sbase + (uint32_t)stage * kHeadStageBytes;
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              tc_mma_pair(d_tmem, operand_desc(sa, A, k), operand_desc(sa + kHalf, B, k), idesc,
                          (kb | k) != 0);
            tc_commit_pair(bar(empty0 + stage), 0x3);
            if (++stage == S) { stage = 0; phase ^= 1u; }
          }
          tc_commit_pair(bar(tfull0 + acc), 0x3);
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        } while (left > 0);
      }
      return true;
    };
    using K0 = std::integral_constant<int, 0>;
    using K1 = std::integral_constant<int, 1>;
#pragma unroll
    for (int c = 0; c < TileList<PHASE>::kKinds; ++c) {
      const int kind = tiles.deal[c].kind;
      if (!(PHASE == kStats || kind == kZ ? deal(c, K0(), K0())
            : kind == kDh                ? deal(c, K0(), K1())
                                         : deal(c, K1(), K1())))
        break;
    }
    tc_commit_pair(bar(drain), 0x1);
    mbar_wait(bar(drain), 0u, g, false);
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // Warp w covers TMEM lane quarter (w & 3), 32 rows of the CTA's 128, and 128 columns.
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t stg0 = sbase + kHeadStaging + (uint32_t)(warp - 2) * kStagePerWarp;
    int acc = 0;
    uint32_t acc_phase = 0;
    float scale = 0.f;                          // largest finite |dloss|
    if (PHASE == kGrads) {
      for (int i = lane; i < P.dl_blocks; i += 32) scale = fmaxf(scale, P.dl_max[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) scale = fmaxf(scale, __shfl_xor_sync(0xFFFFFFFFu, scale, o));
      if (blockIdx.x == 0 && warp == 2 && lane == 0) *P.scale = scale;
    }
    for (TileWalk<PHASE> walk(P, tiles); walk.have; walk.next(P)) {
      const HeadTile& t = walk.t;
      const int rw = t.tm * kTile + 128 * (int)rank + quarter * 32, r = rw + lane;
      const int cb = t.tn * kTile + half * 128;   // first column of this warp
      auto taddr_of = [&](int a) {
        return tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(a * kTile + half * 128);
      };
      const uint32_t taddr = taddr_of(acc);
      if (PHASE == kStats) {
        const bool live = r < tiles.live;
        const int lab = live ? P.label[r] - P.z_v0 : -1;
        float m = -INFINITY, s = 0.f;
        // chunks of columns of this warp that hold columns (and rows)
        const int nq = rw < tiles.live ? min(kHeadChunks, (P.z_width - cb + 31) / 32) : 0;
        uint32_t sum[kHeadChunks][32];
        bool ok = true;
        for (int left = t.nk, first = 1; left > 0; left -= kSumBlocks, first = 0) {
          if (!mbar_wait(bar(tfull0 + acc), acc_phase, g)) { ok = false; break; }
          tc_fence_after();
          const uint32_t ta = taddr_of(acc);
          if (first) {
#pragma unroll
            for (int q = 0; q < kHeadChunks; ++q)
              if (q < nq) tc_ld32_issue(ta + (uint32_t)(32 * q), sum[q]);  // warp-uniform
#pragma unroll
            for (int q = 0; q < kHeadChunks; ++q)
              if (q < nq) tc_ld_wait(sum[q]);
          } else {
#pragma unroll
            for (int q = 0; q < 2 * kHeadChunks; ++q)
              if (q < 2 * nq) {
                float part[16];                           // (32 at a time would spill)
                tc_ld16(ta + (uint32_t)(16 * q), part);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  uint32_t& a = sum[q >> 1][(q & 1) * 16 + k];
                  a = __float_as_uint(__uint_as_float(a) + part[k]);
                }
              }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_rank(bar(tempty0 + acc), 0));
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < kHeadChunks; ++q) {
          if (q < nq) {                                   // warp-uniform
            uint32_t (&a32)[32] = sum[q];
            const int c0 = cb + 32 * q, left = P.z_width - c0;
            if (left < 32) {                              // columns past the end take no part
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k >= left) a32[k] = __float_as_uint(-INFINITY);
            }
            float mc = m;
#pragma unroll
            for (int k = 0; k < 32; ++k) mc = fmaxf(mc, __uint_as_float(a32[k]));
            if (lab >= c0 && lab < c0 + 32) {
              uint32_t z = 0u;
#pragma unroll
              for (int k = 0; k < 32; ++k) z |= a32[k] & (lab - c0 == k ? 0xFFFFFFFFu : 0u);
              P.zlab[r] = __uint_as_float(z);
            }
            const float ref = mc == -INFINITY ? 0.f : mc * kLog2e;
            float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 32; ++k)
              sc[k & 3] += ex2(fmaf(__uint_as_float(a32[k]), kLog2e, -ref));
            s = fmaf(s, ex2(fmaf(m, kLog2e, -ref)), (sc[0] + sc[1]) + (sc[2] + sc[3]));
            m = mc;
          }
        }
        if (live && cb < P.z_width) P.part[(int64_t)(t.tn * 2 + half) * P.rows + r] = make_float2(m, s);
        continue;                                         // the accumulators are released
      } else if (t.kind == kZ) {
        const bool live = r < tiles.live;
        const int lab = live ? P.label[r] - P.z_v0 : -1;
        // a row that holds no token: exp2(z - inf) = 0
        const float lse2 = live ? P.lse2[r] : INFINITY;
        // (no finite dloss but zeros: an infinite or NaN one still reaches the gradients)
        const float dl = live ? P.dl[r] / (scale > 0.f ? scale : 1.f) : 0.f;
        float* gsum = P.gsum && live && cb < P.z_width
                          ? P.gsum + (int64_t)r * P.gsum_parts + (t.tn * 2 + half) : nullptr;
        const float gsum_old = gsum && P.z_v0 > 0 ? *gsum : 0.f;
        float gs[2] = {0.f, 0.f};
        if (!mbar_wait(bar(tfull0 + acc), acc_phase, g)) break;
        tc_fence_after();
        // whole k-blocks of G are written, in both directions: the columns past the end and the
        // rows past the live ones are zero (further rows only meet rows of dH that are not read)
        const int nq = rw < (tiles.live + kBK - 1) / kBK * kBK
                           ? min(kHeadChunks, ((P.z_width + kBK - 1) / kBK * kBK - cb + 31) / 32)
                           : 0;
        uint32_t buf[2][32];
        if (nq > 0) tc_ld32_issue(taddr, buf[0]);
#pragma unroll
        for (int q = 0; q < kHeadChunks; ++q) {
          if (q < nq) {                                   // warp-uniform
            __syncwarp();
            uint32_t (&a32)[32] = buf[q & 1];
            // The block is staged so that a warp's stores cover whole 64-byte rows; the halves
            // of the staging area alternate, so one barrier per chunk is enough.  (By TMA store
            // a chunk waited for the area's last store to have been read.)
            const uint32_t stg = stg0 + (q & 1) * 2048u;
            if (q == 0) {                                 // a product's TMA store may be reading
              if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              __syncwarp();
            }
            tc_ld_wait(a32);
            if (q + 1 < nq) tc_ld32_issue(taddr + (uint32_t)(32 * (q + 1)), buf[(q + 1) & 1]);
            const int c0 = cb + 32 * q, left = P.z_width - c0, hit = lab - c0;
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = ex2(fmaf(__uint_as_float(a32[k]), kLog2e, -lse2));
            if (__any_sync(0xFFFFFFFFu, hit >= 0 && hit < 32)) {
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = fmaf(v[k], dl, k == hit ? -dl : 0.f);
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] *= dl;
            }
            if (left < 32) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k >= left) v[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                w[h] = pack_bf16x2(v[8 * k + 2 * h], v[8 * k + 2 * h + 1]);
                add_bf16x2(w[h], gs[0], gs[1]);
              }
              sts128(stg + stg_off(lane, k), make_uint4(w[0], w[1], w[2], w[3]));
            }
            __syncwarp();
            uint16_t* gp = P.g + (int64_t)(P.z_g_row0 + rw) * P.piece + c0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 8 * i + (lane >> 2), k = lane & 3;
              *reinterpret_cast<uint4*>(gp + (int64_t)row * P.piece + 8 * k) =
                  lds128(stg + stg_off(row, k));
            }
          }
        }
        if (gsum) *gsum = gsum_old + (gs[0] + gs[1]);
      } else {
        if (!mbar_wait(bar(tfull0 + acc), acc_phase, g)) break;
        tc_fence_after();
        const int row_end = t.kind == kDh ? tiles.live : P.width;
#pragma unroll 1
        for (int q = 0; q < kHeadChunks; ++q) {
          const int c0 = cb + 32 * q;
          if (c0 >= P.dim || rw >= row_end) break;        // warp-uniform
          __syncwarp();
          uint32_t a32[32];
          if (t.nk > 0) {
            tc_ld32_issue(taddr + (uint32_t)(32 * q), a32);
          } else {                                        // an empty contraction
#pragma unroll
            for (int k = 0; k < 32; ++k) a32[k] = 0u;
          }
          // both kinds stage in the warp's one 4 KB area: the last store has read it
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
          tc_ld_wait(a32);
          if (t.kind == kDh) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              sts128(stg0 + stg32_off(lane, k),
                     make_uint4(a32[4 * k], a32[4 * k + 1], a32[4 * k + 2], a32[4 * k + 3]));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int h = 0; h < 4; ++h)
                w[h] = pack_bf16x2(__uint_as_float(a32[8 * k + 2 * h]) * scale,
                                   __uint_as_float(a32[8 * k + 2 * h + 1]) * scale);
              sts128(stg0 + stg_off(lane, k), make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          if (t.kind == kDw && !P.dw_tma) {
            // rows without 16-byte alignment: a warp writes one row of the block at a time
            __syncwarp();
            for (int i = 0; i < 32; ++i) {
              if (rw + i >= row_end || c0 + lane >= P.dim) continue;
              const uint32_t w = lds32(stg0 + stg_off(i, lane >> 3) + (uint32_t)((lane & 6) * 2));
              P.dw[(int64_t)(P.v0 + rw + i) * P.ld_dw + c0 + lane] =
                  (uint16_t)(lane & 1 ? w >> 16 : w & 0xFFFFu);
            }
            __syncwarp();
            continue;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (t.kind == kDw)
              tma_store_block(&P.dw_st, stg0, c0, P.v0 + rw);
            else if (P.add)
              tma_reduce_add_block(&P.acc_st, stg0, c0, t.split * P.rows + rw);
            else
              tma_store_block(&P.acc_st, stg0, c0, t.split * P.rows + rw);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_rank(bar(tempty0 + acc), 0));
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // stores done
    __syncwarp();
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while its peer may still use its memory
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u)
                 : "memory");
  }
}

// ---------------------------------------------------------------- live rows
struct GatherArgs {
  const void* labels;
  const void* hidden;
  void* hc;                                // [rows][pitch]
  int64_t ld_h, ignore;
  int32_t n, is64, dim, pitch, vocab, per; // per: tokens per block
  int32_t vec;
  int32_t place;                           // keep every token at its own row, dropped ones zero
  int32_t* nlive;
  int32_t* label;
  int32_t* pos;                            // [n] compacted row of a token, -1: dropped
  int32_t* token;                          // [rows] token of a compacted row
  const float *lse_in, *dloss;             // backward
  float *lse2, *dl, *dl_max;
  float *loss, *lse;                       // forward: zeroed for dropped tokens
  int* status;
  int32_t blocks;                          // blocks that gather; the others average rows of W
  const void* weight;
  int64_t ld_w;
  float* wmean;                            // [pitch] mean of up to kMeanRows evenly spaced rows
};

// What all rows of W have in common, 32 columns per block: 128 rows estimate a column's mean to
// within a tenth of its spread, and a warp has all of its loads in flight at once.
constexpr int kMeanRows = 128;
template <typename T>
__device__ __forceinline__ void mean_rows(const GatherArgs& p, int block) {
  __shared__ float sum[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = block * 32 + lane;
  const int rows = min(p.vocab, kMeanRows);
  const int64_t step = (int64_t)(p.vocab / rows) * p.ld_w;
  const T* w = static_cast<const T*>(p.weight) + min(c, p.dim - 1);
  float v[kMeanRows / 8], a = 0.f;
#pragma unroll
  for (int i = 0; i < kMeanRows / 8; ++i) v[i] = to_f32(w[min(8 * i + warp, rows - 1) * step]);
#pragma unroll
  for (int i = 0; i < kMeanRows / 8; ++i) a += 8 * i + warp < rows ? v[i] : 0.f;
  sum[warp][lane] = a;
  __syncthreads();
  if (warp != 0) return;
  for (int i = 1; i < 8; ++i) a += sum[i][lane];
  p.wmean[c] = c < p.dim ? a / (float)rows : 0.f;
}

// Every block counts the live tokens before its own (the labels are read from the L2), so one
// launch compacts without a scan.  The last of them also zeroes the rows up to the next k-block.
// With `place` (the fp32 path, whose GEMM takes its row count from the host) tokens keep their
// rows; a dropped one gets a zero row and label -1.
template <typename T>
__global__ void __launch_bounds__(256) head_gather_kernel(const __grid_constant__ GatherArgs p) {
  __shared__ int32_t red[8], src[256];
  __shared__ int32_t start_s;
  pdl_launch();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((int)blockIdx.x >= p.blocks) {
    mean_rows<T>(p, (int)blockIdx.x - p.blocks);
    return;
  }
  const int t0 = blockIdx.x * p.per, t1 = min(p.n, t0 + p.per);
  auto live_at = [&](int t, int64_t& lab) {
    lab = load_index(p.labels, p.is64, t);
    return lab != p.ignore && lab >= 0 && lab < p.vocab;
  };
  int cnt = 0;
  for (int t = tid; t < t0 && !p.place; t += 256) {
    int64_t lab;
    cnt += live_at(t, lab);
  }
  cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
  if (lane == 0) red[warp] = cnt;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) base += red[i];
  if (p.place) base = t0;
  T* hc = static_cast<T*>(p.hc);
  float top = 0.f;                         // largest finite |dloss| of this thread's live tokens
  for (int b = t0; b < t1; b += 256) {     // 256 tokens at a time
    __syncthreads();
    const int t = b + tid;
    int64_t lab = 0;
    const bool in = t < t1, live = in && live_at(t, lab);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, live);
    if (lane == 0) red[warp] = __popc(mask);
    __syncthreads();
    int off = __popc(mask & ((1u << lane) - 1u)), total = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < warp) off += red[i];
      total += red[i];
    }
    if (p.place) {
      off = tid;
      total = min(256, t1 - b);
    }
    if (in) {
      p.pos[t] = live ? base + off : -1;
      if (live || p.place) {
        src[off] = live ? t : -1;
        p.label[base + off] = live ? (int32_t)lab : -1;
        p.token[base + off] = t;
        if (p.dl) {
          const float dl = live ? p.dloss[t] : 0.f;
          p.dl[base + off] = dl;
          if (fabsf(dl) < INFINITY) top = fmaxf(top, fabsf(dl));
          p.lse2[base + off] = live ? p.lse_in[t] * kLog2e : 0.f;
        }
      }
      if (!live) {
        if (lab != p.ignore) atomicOr(p.status, kStatusBadIndex);
        if (p.loss) p.loss[t] = 0.f;
        if (p.lse) p.lse[t] = 0.f;
      }
    }
    __syncthreads();
    // copy the live rows, a warp per row; columns past dim are zero
    for (int i = warp; i < total; i += 8) {
      const int dim = src[i] >= 0 ? p.dim : 0;
      const T* s = static_cast<const T*>(p.hidden) + (int64_t)max(src[i], 0) * p.ld_h;
      T* d = hc + (int64_t)(base + i) * p.pitch;
      if (p.vec) {
        for (int e = lane * 8; e < p.pitch; e += 256) {
          Pack8<T> v;
          if (e < dim) v.load(s + e); else v.zero();
          v.store(d + e);
        }
      } else {
        for (int e0 = lane; e0 < p.pitch; e0 += 256) {   // eight loads in flight
          T v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = e0 + 32 * k < dim ? s[e0 + 32 * k] : from_f32<T>(0.f);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (e0 + 32 * k < p.pitch) d[e0 + 32 * k] = v[k];
        }
      }
    }
    base += total;
  }
  if (p.dl_max) {
    __shared__ float tops[8];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, tops[i]);
      p.dl_max[blockIdx.x] = top;
    }
  }
  if ((int)blockIdx.x != p.blocks - 1) return;
  if (tid == 0) {
    *p.nlive = base;
    start_s = base;
  }
  __syncthreads();
  const int r0 = start_s, r1 = p.place ? r0 : (r0 + kBK - 1) / kBK * kBK;
  for (int r = r0 + warp; r < r1; r += 8)
    for (int e = lane; e < p.pitch; e += 32) hc[(int64_t)r * p.pitch + e] = from_f32<T>(0.f);
}

// ---------------------------------------------------------------- join of the row statistics
struct JoinArgs {
  const float2* part;                      // [parts][rows]
  float2* state;                           // [rows] running (max, sum) over the pieces
  const float* zlab;
  const int32_t *nlive, *token;
  float *loss, *lse;                       // nullable
  int32_t parts, rows, first, last;
};

__device__ __forceinline__ void merge_stats(float& m, float& s, float m2, float s2) {
  const float mn = fmaxf(m, m2), ref = mn == -INFINITY ? 0.f : mn;
  s = s * exp2f((m - ref) * kLog2e) + s2 * exp2f((m2 - ref) * kLog2e);
  m = mn;
}

// 32 rows per block; 32 groups of parts per row, joined in group order.
__global__ void __launch_bounds__(1024) head_join_kernel(const __grid_constant__ JoinArgs p) {
  __shared__ float2 sm[32][33];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int r = blockIdx.x * 32 + lane, live = *p.nlive;
  if ((int)blockIdx.x * 32 >= live) return;
  float m = -INFINITY, s = 0.f;
  if (r < live) {
#pragma unroll 4
    for (int i = grp; i < p.parts; i += 32) {
      const float2 v = p.part[(int64_t)i * p.rows + r];
      merge_stats(m, s, v.x, v.y);
    }
  }
  sm[grp][lane] = make_float2(m, s);
  __syncthreads();
  if (grp != 0 || r >= live) return;
  if (!p.first) {
    const float2 v = p.state[r];
    m = v.x;
    s = v.y;
    merge_stats(m, s, sm[0][lane].x, sm[0][lane].y);
  }
  for (int i = 1; i < 32; ++i) merge_stats(m, s, sm[i][lane].x, sm[i][lane].y);
  if (!p.last) {
    p.state[r] = make_float2(m, s);
    return;
  }
  const float l = m + logf(s);
  const int t = p.token[r];
  if (p.lse) p.lse[t] = l;
  if (p.loss) p.loss[t] = l - p.zlab[r];
}

// ---------------------------------------------------------------- few tokens
// One token (up to kFewTokens where the tensor cores would need a copy of W or run 3xTF32) is
// bound by reading W once: a matrix product's 256-row tile would be empty but for it.  One token
// over 128256 x 4096 took 191 us here and 218 on the tensor cores, two 267 and 216.  A warp takes
// kFewRows rows of W at a time (all their loads in flight together), multiplies them with the
// tokens' hidden rows, which the block holds in shared memory in fp32, and keeps each token's
// running (max, sum) in registers.
constexpr int kFewTokens = 4;
constexpr int kFewRows = 4;
constexpr int kFewWarps = 8;

struct FewArgs {
  const void *hidden, *weight, *labels;
  int64_t ld_h, ld_w, ignore;
  float2* part;                            // [blocks][kFewTokens]
  float* zlab;                             // [kFewTokens]
  float *loss, *lse;
  int32_t n, dim, vocab, is64, vec, blocks;
  int* status;
};

template <typename T, int NT>
__global__ void __launch_bounds__(32 * kFewWarps) head_few_kernel(const __grid_constant__ FewArgs p) {
  extern __shared__ float few_h[];         // [NT][dim rounded up to 8]
  __shared__ float2 red[kFewWarps][NT];
  pdl_launch();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int dim8 = (p.dim + 7) / 8 * 8;
  const T* w = static_cast<const T*>(p.weight);
  const int first = (blockIdx.x * kFewWarps + warp) * kFewRows;
  // the warp's first rows of W are on their way to the L2 while the hidden rows arrive (3 tokens x
  // 1024 fp32 against 30000 rows: 52 -> 48 us; rows without vectors 35 -> 40)
  if (p.vec && first < p.vocab)
    for (int e = lane * (128 / (int)sizeof(T)); e < p.dim; e += 32 * (128 / (int)sizeof(T)))
#pragma unroll
      for (int i = 0; i < kFewRows; ++i)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
                         w + (int64_t)min(first + i, p.vocab - 1) * p.ld_w + e)
                     : "memory");
  int lab[NT];
  float m[NT], s[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t l = t < p.n ? load_index(p.labels, p.is64, t) : p.ignore;
    lab[t] = l != p.ignore && l >= 0 && l < p.vocab ? (int)l : -1;
    m[t] = -INFINITY;
    s[t] = 0.f;
    // (loaded whatever the label is, and dropped afterwards: one wait for both)
    const T* h = static_cast<const T*>(p.hidden) + (int64_t)min(t, p.n - 1) * p.ld_h;
    for (int e = threadIdx.x; e < dim8; e += 32 * kFewWarps) {
      const float x = to_f32(h[min(e, p.dim - 1)]);
      few_h[t * dim8 + e] = lab[t] >= 0 && e < p.dim ? x : 0.f;
    }
  }
  __syncthreads();
  const int step = gridDim.x * kFewWarps * kFewRows;
  for (int v0 = first; v0 < p.vocab; v0 += step) {
    float dot[kFewRows][NT];
#pragma unroll
    for (int i = 0; i < kFewRows; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) dot[i][t] = 0.f;
    if (p.vec) {
#pragma unroll 4
      for (int e = lane * 8; e < p.dim; e += 256) {
        Pack8<T> q[kFewRows];
#pragma unroll
        for (int i = 0; i < kFewRows; ++i)
          q[i].load(w + (int64_t)min(v0 + i, p.vocab - 1) * p.ld_w + e);
        float x[kFewRows][8];
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) q[i].get(x[i]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          Pack8<float> hq;
          hq.load(few_h + t * dim8 + e);
          float h[8];
          hq.get(h);
#pragma unroll
          for (int i = 0; i < kFewRows; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) dot[i][t] = fmaf(x[i][k], h[k], dot[i][t]);
        }
      }
    } else {
#pragma unroll 4
      for (int e = lane; e < p.dim; e += 32) {
        float x[kFewRows];
#pragma unroll
        for (int i = 0; i < kFewRows; ++i)
          x[i] = to_f32(w[(int64_t)min(v0 + i, p.vocab - 1) * p.ld_w + e]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < kFewRows; ++i) dot[i][t] = fmaf(x[i], few_h[t * dim8 + e], dot[i][t]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float mc = m[t];
#pragma unroll
      for (int i = 0; i < kFewRows; ++i) {
        dot[i][t] = v0 + i < p.vocab ? warp_sum(dot[i][t]) : -INFINITY;
        mc = fmaxf(mc, dot[i][t]);
        if (lane == 0 && v0 + i == lab[t]) p.zlab[t] = dot[i][t];
      }
      const float ref = mc == -INFINITY ? 0.f : mc * kLog2e;
      s[t] *= ex2(fmaf(m[t], kLog2e, -ref));
#pragma unroll
      for (int i = 0; i < kFewRows; ++i) s[t] += ex2(fmaf(dot[i][t], kLog2e, -ref));
      m[t] = mc;
    }
  }
  if (lane == 0)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[warp][t] = make_float2(m[t], s[t]);
  __syncthreads();
  if (threadIdx.x < NT) {
    float a = -INFINITY, b = 0.f;
    for (int i = 0; i < kFewWarps; ++i)
      merge_stats(a, b, red[i][threadIdx.x].x, red[i][threadIdx.x].y);
    p.part[blockIdx.x * kFewTokens + threadIdx.x] = make_float2(a, b);
  }
}

// A block per token joins the blocks' pairs in a fixed order.
constexpr int kFewJoinThreads = 256;
__global__ void __launch_bounds__(kFewJoinThreads)
    head_few_join_kernel(const __grid_constant__ FewArgs p) {
  constexpr int kWarps = kFewJoinThreads / 32;
  __shared__ float2 red[kWarps];
  pdl_launch();
  pdl_wait();
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t lab = load_index(p.labels, p.is64, t);
  const bool live = lab != p.ignore && lab >= 0 && lab < p.vocab;
  const float zlab = p.zlab[t];            // (not written for a dropped token)
  float m = -INFINITY, s = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x; i < p.blocks; i += kFewJoinThreads) {
    const float2 v = p.part[i * kFewTokens + t];
    merge_stats(m, s, v.x, v.y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    merge_stats(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
  if (lane == 0) red[warp] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < kWarps; ++i) merge_stats(m, s, red[i].x, red[i].y);
  if (!live && lab != p.ignore) atomicOr(p.status, kStatusBadIndex);
  const float l = live ? m + logf(s) : 0.f;
  if (p.lse) p.lse[t] = l;
  if (p.loss) p.loss[t] = live ? l - zlab : 0.f;
}

// The backward pass of few tokens, one pass over W: 16 rows at a time, a warp computes a row's
// logits and G; then every thread takes columns of those rows, for the rows of dW and for its
// sums of dH, which stay in shared memory until the block's last rows.  Bound by memory: W is read
// and dW written once (the columns' second read of a row comes from the L1 or L2).
constexpr int kFewGradWarps = 16;
constexpr int kFewGradThreads = 32 * kFewGradWarps;
struct FewGradArgs {
  const void *hidden, *weight, *labels;
  int64_t ld_h, ld_w, ignore;
  const float *lse, *dloss;
  void *dh, *dw;                           // nullable
  int64_t ld_dh, ld_dw;
  float* acc;                              // [blocks][n][pitch]
  int32_t n, dim, vocab, is64, blocks, pitch;
  int* status;
};

__device__ __forceinline__ int few_label(const FewGradArgs& p, int t, bool& bad) {
  const int64_t l = load_index(p.labels, p.is64, t);
  const bool live = l != p.ignore && l >= 0 && l < p.vocab;
  bad = !live && l != p.ignore;
  return live ? (int)l : -1;
}

template <typename T, int C>
__device__ __forceinline__ void load_columns(const T* p, float (&x)[C]) {
  if constexpr (C == 1) {
    x[0] = to_f32(*p);
  } else if constexpr (sizeof(T) == 2) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(q.x << 16);
    x[1] = __uint_as_float(q.x & 0xFFFF0000u);
    x[2] = __uint_as_float(q.y << 16);
    x[3] = __uint_as_float(q.y & 0xFFFF0000u);
  } else {
    const float4 q = *reinterpret_cast<const float4*>(p);
    x[0] = q.x;
    x[1] = q.y;
    x[2] = q.z;
    x[3] = q.w;
  }
}

template <typename T, int C>
__device__ __forceinline__ void store_columns(T* p, const float (&x)[C]) {
  if constexpr (C == 1)
    *p = from_f32<T>(x[0]);
  else if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  else
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// C columns per thread at a time: 4 where every row is aligned to them, else 1.
template <typename T, int NT, int C>
__global__ void __launch_bounds__(kFewGradThreads)
    head_few_grad_kernel(const __grid_constant__ FewGradArgs p) {
  extern __shared__ float few_h[];         // hidden rows, then the sums: [NT][dim rounded up to 8]
  __shared__ float gs[kFewGradWarps][NT];
  pdl_launch();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int dim8 = (p.dim + 7) / 8 * 8;
  float* sums = few_h + NT * dim8;
  int lab[NT];
  float lse2[NT], dl[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int at = min(t, p.n - 1);
    bool bad;
    lab[t] = few_label(p, at, bad);
    if (bad && t < p.n && blockIdx.x == 0 && tid == 0) atomicOr(p.status, kStatusBadIndex);
    if (t >= p.n) lab[t] = -1;
    lse2[t] = p.lse[at] * kLog2e;
    dl[t] = p.dloss[at];
    const T* h = static_cast<const T*>(p.hidden) + (int64_t)at * p.ld_h;
    for (int e = tid; e < dim8; e += kFewGradThreads) {
      const float x = to_f32(h[min(e, p.dim - 1)]);
      few_h[t * dim8 + e] = lab[t] >= 0 && e < p.dim ? x : 0.f;
      sums[t * dim8 + e] = 0.f;
    }
  }
  __syncthreads();
  const T* w = static_cast<const T*>(p.weight);
  T* dw = static_cast<T*>(p.dw);
  for (int v0 = (int)blockIdx.x * kFewGradWarps; v0 < p.vocab; v0 += p.blocks * kFewGradWarps) {
    const int v = v0 + warp;
    const T* row = w + (int64_t)min(v, p.vocab - 1) * p.ld_w;
    float dot[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) dot[t] = 0.f;
#pragma unroll 8
    for (int e = lane * C; e < p.dim; e += 32 * C) {
      float x[C];
      load_columns<T, C>(row + e, x);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < C; ++k) dot[t] = fmaf(x[k], few_h[t * dim8 + e + k], dot[t]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float z = warp_sum(dot[t]);
      if (lane == 0) {
        float g = 0.f;
        if (lab[t] >= 0 && v < p.vocab) {
          g = exp2f(fmaf(z, kLog2e, -lse2[t]));
          if (v == lab[t]) g -= 1.f;
          g *= dl[t];
        }
        gs[warp][t] = g;
      }
    }
    __syncthreads();
    const int rows = min(kFewGradWarps, p.vocab - v0);
    for (int e = tid * C; e < p.dim; e += kFewGradThreads * C) {
      float h[NT][C], a[NT][C];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < C; ++k) {
          h[t][k] = few_h[t * dim8 + e + k];
          a[t][k] = sums[t * dim8 + e + k];
        }
#pragma unroll 4
      for (int r = 0; r < rows; ++r) {
        float x[C], d[C];
        if (p.dh) load_columns<T, C>(w + (int64_t)(v0 + r) * p.ld_w + e, x);
#pragma unroll
        for (int k = 0; k < C; ++k) d[k] = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float g = gs[r][t];
#pragma unroll
          for (int k = 0; k < C; ++k) {
            d[k] = fmaf(g, h[t][k], d[k]);
            if (p.dh) a[t][k] = fmaf(g, x[k], a[t][k]);
          }
        }
        if (dw) store_columns<T, C>(dw + (int64_t)(v0 + r) * p.ld_dw + e, d);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < C; ++k) sums[t * dim8 + e + k] = a[t][k];   // this thread's columns
    }
    __syncthreads();
  }
  if (!p.dh) return;
  for (int t = 0; t < p.n; ++t)
    for (int e = tid; e < p.dim; e += kFewGradThreads)
      p.acc[((int64_t)blockIdx.x * p.n + t) * p.pitch + e] = sums[t * dim8 + e];
}

// 32 columns of a token's dH: 32 groups add the blocks' sums, then the groups are added in order.
template <typename T>
__global__ void __launch_bounds__(1024)
    head_few_finish_kernel(const __grid_constant__ FewGradArgs p) {
  __shared__ float sm[32][33];
  pdl_launch();
  pdl_wait();
  const int t = blockIdx.y, lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int e = (int)blockIdx.x * 32 + lane, at = min(e, p.dim - 1);
  float v = 0.f;
#pragma unroll 4
  for (int b = grp; b < p.blocks; b += 32) v += p.acc[((int64_t)b * p.n + t) * p.pitch + at];
  sm[grp][lane] = v;
  __syncthreads();
  if (grp != 0 || e >= p.dim) return;
  for (int g = 1; g < 32; ++g) v += sm[g][lane];
  bool bad;
  const bool live = few_label(p, t, bad) >= 0;
  static_cast<T*>(p.dh)[t * p.ld_dh + e] = from_f32<T>(live ? v : 0.f);
}

// ---------------------------------------------------------------- dH: slices to the caller's rows
struct FinishArgs {
  const float* acc;                        // [splits][rows][pitch]
  const float* scale;                      // nullable
  const float *gsum, *wmean;               // nullable: [rows][gsum_parts] and [pitch], taken off
  int32_t gsum_parts;
  const int32_t* pos;
  void* dh;
  int64_t ld_dh;
  int32_t dim, pitch, rows, splits, vec;
};

// A block per token, four columns per thread; the slices are added in order, eight of them in
// flight (the sums' rows are aligned whatever the caller's are).
template <typename T>
__global__ void __launch_bounds__(256) head_finish_kernel(const __grid_constant__ FinishArgs p) {
  pdl_launch();
  pdl_wait();
  const int t = blockIdx.x;
  const int r = p.pos[t];
  const float scale = p.scale ? *p.scale : 1.f;
  T* out = static_cast<T*>(p.dh) + (int64_t)t * p.ld_dh;
  const int64_t slice = (int64_t)p.rows * p.pitch;
  const float* a = p.acc + (int64_t)max(r, 0) * p.pitch;
  float common = 0.f;                      // the sum of the token's row of G
  if (p.gsum && r >= 0) {                  // (every warp for itself: no barrier)
#pragma unroll 8
    for (int i = threadIdx.x & 31; i < p.gsum_parts; i += 32)
      common += p.gsum[(int64_t)r * p.gsum_parts + i];
    common = warp_sum(common);
  }
  for (int e = threadIdx.x * 4; e < p.dim; e += 1024) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r >= 0) {
#pragma unroll 8
      for (int s = 0; s < p.splits; ++s) {
        const float4 x = *reinterpret_cast<const float4*>(a + s * slice + e);
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
      }
      if (p.gsum) {
        const float4 c = *reinterpret_cast<const float4*>(p.wmean + e);
        v[0] = fmaf(-common, c.x, v[0]);
        v[1] = fmaf(-common, c.y, v[1]);
        v[2] = fmaf(-common, c.z, v[2]);
        v[3] = fmaf(-common, c.w, v[3]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] *= scale;
    if (p.vec) {   // whole groups of four, aligned to them
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(out + e) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                        *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        *reinterpret_cast<float4*>(out + e) = make_float4(v[0], v[1], v[2], v[3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e + k < p.dim) out[e + k] = from_f32<T>(v[k]);
    }
  }
}

// Rows [0, rows) x cols of a matrix into a buffer of 16-byte aligned rows; the rows after them
// (whole k-blocks) are zero.  A warp per row, eight words of loads in flight; a bf16 row may start
// at an odd element, so its words are put together from halves.
template <typename T>
__global__ void __launch_bounds__(256)
    head_copy_rows_kernel(const T* src, int64_t ld_src, T* dst, int64_t ld_dst, int rows, int total,
                          int cols) {
  constexpr int E = 4 / (int)sizeof(T), U = 8;   // elements per word
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= total) return;
  const T* from = src + (r < rows ? r : 0) * ld_src;
  T* to = dst + r * ld_dst;
  const int words = (cols + E - 1) / E;
  for (int w0 = lane; w0 < words; w0 += 32 * U) {
    T v[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < E; ++h) v[u][h] = from[min((w0 + 32 * u) * E + h, cols - 1)];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = (w0 + 32 * u) * E;
      if (e >= cols) continue;
      uint32_t word = 0u;
      if (r < rows) {
        if constexpr (E == 2) {
          word = (uint32_t)__bfloat16_as_ushort(v[u][0]);
          if (e + 1 < cols) word |= (uint32_t)__bfloat16_as_ushort(v[u][1]) << 16;
        } else {
          word = __float_as_uint(v[u][0]);
        }
      }
      *reinterpret_cast<uint32_t*>(to + e) = word;
    }
  }
}

// ---------------------------------------------------------------- fp32 path
// One row of a piece of Z: (max, sum) joined into the running state, and the label's logit; the
// last piece writes the loss.
struct Stats32Args {
  const float* z;                          // [rows][ldz]
  float2* state;
  float* zlab;
  const int32_t *label, *token;
  float *loss, *lse;
  int32_t width, v0, first, last;
  int64_t ldz;
};

__global__ void __launch_bounds__(256) head_stats32_kernel(const __grid_constant__ Stats32Args p) {
  __shared__ float2 sm[8];
  pdl_launch();
  pdl_wait();
  const int r = blockIdx.x;
  if (p.label[r] < 0) return;              // dropped
  const float* z = p.z + (int64_t)r * p.ldz;
  float m = -INFINITY, s = 0.f;
  for (int c = threadIdx.x; c < p.width; c += 256) merge_stats(m, s, z[c], 1.f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    merge_stats(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < 8; ++i) merge_stats(m, s, sm[i].x, sm[i].y);
  if (!p.first) merge_stats(m, s, p.state[r].x, p.state[r].y);
  const int lab = p.label[r] - p.v0;
  float zl = p.zlab[r];
  if (lab >= 0 && lab < p.width) p.zlab[r] = zl = z[lab];
  p.state[r] = make_float2(m, s);
  if (!p.last) return;
  const float l = m + logf(s);
  const int t = p.token[r];
  if (p.lse) p.lse[t] = l;
  if (p.loss) p.loss[t] = l - zl;
}

struct Grad32Args {
  float* z;                                // [rows][ldz]: Z in, G out
  float* gt;                               // nullable: [columns][ldt], G transposed
  const int32_t* label;
  const float *lse2, *dl;
  int32_t rows, width, v0;
  int64_t ldz, ldt;
};

// A 32 x 32 block of Z to G, in place and transposed.
__global__ void __launch_bounds__(256) head_grad32_kernel(const __grid_constant__ Grad32Args p) {
  __shared__ float tile[32][33];
  pdl_launch();
  pdl_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, nc = (p.width + 31) / 32;
  const int c0 = (int)(blockIdx.x % nc) * 32, r0 = (int)(blockIdx.x / nc) * 32;
#pragma unroll
  for (int i = y; i < 32; i += 8) {
    const int r = r0 + i, c = c0 + x;
    if (r >= p.rows || c >= p.width) continue;
    float* z = p.z + (int64_t)r * p.ldz + c;
    const int lab = p.label[r];
    float g = 0.f;
    if (lab >= 0) {
      g = exp2f(fmaf(*z, kLog2e, -p.lse2[r]));
      if (c == lab - p.v0) g -= 1.f;
      g *= p.dl[r];
    }
    *z = g;
    tile[i][x] = g;
  }
  if (!p.gt) return;
  __syncthreads();
#pragma unroll
  for (int i = y; i < 32; i += 8)
    if (c0 + i < p.width && r0 + x < p.rows) p.gt[(int64_t)(c0 + i) * p.ldt + r0 + x] = tile[x][i];
}

// dst[c][r] = src[r][c]: the GEMM's fast path takes operands with the contraction contiguous.
__global__ void __launch_bounds__(256)
    head_transpose32_kernel(const float* src, int64_t ld_src, int rows, int cols, float* dst,
                            int64_t ld_dst) {  // one block per 32 x 32, column blocks fastest
  __shared__ float tile[32][33];
  pdl_launch();
  pdl_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, nc = (cols + 31) / 32;
  const int c0 = (int)(blockIdx.x % nc) * 32, r0 = (int)(blockIdx.x / nc) * 32;
#pragma unroll
  for (int i = y; i < 32; i += 8)
    if (r0 + i < rows && c0 + x < cols) tile[i][x] = src[(int64_t)(r0 + i) * ld_src + c0 + x];
  __syncthreads();
#pragma unroll
  for (int i = y; i < 32; i += 8)
    if (c0 + i < cols && r0 + x < rows) dst[(int64_t)(c0 + i) * ld_dst + r0 + x] = tile[x][i];
}

// The GEMM's problem table, written by a launch (its values travel in the launch's arguments,
// so a captured graph replays them).
constexpr int kDescBatch = 48;
struct DescArgs {
  GemmDesc d[kDescBatch];
  int32_t n;
  GemmDesc* out;
};
__global__ void head_descs_kernel(const __grid_constant__ DescArgs p) {
  pdl_launch();
  pdl_wait();
  for (int i = threadIdx.x; i < p.n; i += blockDim.x) p.out[i] = p.d[i];
}

// ---------------------------------------------------------------- small products
// Up to kCoreFlops (bf16: kCoreFlopsBf16) the products run on the CUDA cores, from operands as
// they lie (any alignment, either one contiguous), so there is nothing to copy or transpose, and
// the epilogues are fused: two launches forward and three backward, against four and nine (bf16:
// three and five or more).  G stays in fp32.  Such sizes are bound by latency, so tiles are small
// (32 x 32) and steps long (64 of the contraction): four groups of two warps share a step, 4 x 4
// entries per thread, and add up at the end.  A thread sums its 16 of a step by themselves before
// it adds them.
constexpr int kCoreTile = 32, kCoreK = 64, kCoreThreads = 256;
constexpr int kCorePitch = kCoreTile + 4;  // the loader's banks are 4 k + row
constexpr int kCoreGroups = 4;

struct alignas(16) CoreSmem {
  union {
    struct {
      float a[2][kCoreK][kCorePitch], b[2][kCoreK][kCorePitch];
    };
    float sum[kCoreGroups][kCoreTile][kCorePitch];
  };
};

// Entry i of this thread in a 32 x 64 operand tile.  KMAJOR (the contraction is contiguous): 8 of k
// by 4 rows per warp, whole sectors of memory and all banks of the transposed store.
template <bool KMAJOR>
__device__ __forceinline__ void core_place(int i, int& row, int& k) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  row = KMAJOR ? 4 * warp + (lane >> 3) : lane;
  k = KMAJOR ? 8 * i + (lane & 7) : warp + 8 * i;
}

// Entries outside the matrix, or that `keep` drops, are zero whatever memory holds (indices are
// clamped, so the loads need no branch).
template <bool KMAJOR, typename T, typename Keep>
__device__ __forceinline__ void core_load(const T* src, int64_t ld, int r0, int rows, int k0,
                                          int k1, const Keep& keep, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int row, k;
    core_place<KMAJOR>(i, row, k);
    const int64_t r = min(r0 + row, rows - 1), c = min(k0 + k, k1 - 1);
    const float x = to_f32(src[KMAJOR ? r * ld + c : c * ld + r]);
    v[i] = r0 + row < rows && k0 + k < k1 && keep((int)r, (int)c) ? x : 0.f;
  }
}

template <bool KMAJOR>
__device__ __forceinline__ void core_store(float (&tile)[kCoreK][kCorePitch], const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int row, k;
    core_place<KMAJOR>(i, row, k);
    tile[k][row] = v[i];
  }
}

// out = four columns, 4 (t % 8) on, of row t / 8 of the tile (m0, n0) of A B^T over [k0, k1), which
// is not empty, for thread t.
template <bool AK, bool BK, typename TA, typename TB, typename KeepA, typename KeepB>
__device__ __forceinline__ void core_product(CoreSmem& sm, const TA* a, int64_t lda, int m0,
                                             int m, const KeepA& keep_a, const TB* b, int64_t ldb,
                                             int n0, int n, const KeepB& keep_b, int k0, int k1,
                                             float (&out)[4]) {
  constexpr int kShare = kCoreK / kCoreGroups;
  const int grp = threadIdx.x >> 6, ty = (threadIdx.x >> 3) & 7, tx = threadIdx.x & 7;
  float acc[4][4] = {};
  float va[8], vb[8];
  core_load<AK>(a, lda, m0, m, k0, k1, keep_a, va);
  core_load<BK>(b, ldb, n0, n, k0, k1, keep_b, vb);
  core_store<AK>(sm.a[0], va);
  core_store<BK>(sm.b[0], vb);
  __syncthreads();
  for (int buf = 0; k0 < k1; k0 += kCoreK, buf ^= 1) {
    const bool more = k0 + kCoreK < k1;
    if (more) {
      core_load<AK>(a, lda, m0, m, k0 + kCoreK, k1, keep_a, va);
      core_load<BK>(b, ldb, n0, n, k0 + kCoreK, k1, keep_b, vb);
    }
    float sum[4][4] = {};
#pragma unroll
    for (int kk = 0; kk < kShare; ++kk) {
      const int k = grp * kShare + kk;
      const float4 x = *reinterpret_cast<const float4*>(&sm.a[buf][k][4 * ty]);
      const float4 y = *reinterpret_cast<const float4*>(&sm.b[buf][k][4 * tx]);
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(xs[i], ys[j], sum[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += sum[i][j];
    if (more) {                            // the other buffer was last read before the barrier
      core_store<AK>(sm.a[buf ^ 1], va);
      core_store<BK>(sm.b[buf ^ 1], vb);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(&sm.sum[grp][4 * ty + i][4 * tx]) =
        make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) out[j] = 0.f;
#pragma unroll
  for (int g = 0; g < kCoreGroups; ++g) {
    const float4 x =
        *reinterpret_cast<const float4*>(&sm.sum[g][threadIdx.x >> 3][4 * (threadIdx.x & 7)]);
    out[0] += x.x;
    out[1] += x.y;
    out[2] += x.z;
    out[3] += x.w;
  }
}

struct CoreArgs {
  const void* hidden;
  const void* weight;                      // the piece's first row
  const void* labels;
  int64_t ld_h, ld_w, ignore;
  int32_t n, dim, vocab, is64;
  int32_t v0, width;                       // the piece: vocabulary columns [v0, v0 + width)
  float2* part;                            // forward: [n][parts] (max, sum) of a tile's row
  float* zlab;                             // forward: [n]
  int32_t parts;
  float *loss, *lse;                       // forward, nullable
  const float *lse_in, *dloss;             // backward
  float* g;                                // backward: G of the piece, [n][piece]
  int64_t piece;
  int32_t* pos;                            // backward: [n] the token, -1: dropped
  void* dw;                                // the piece's first row
  int64_t ld_dw;
  int32_t dw_tiles;
  float* acc;                              // dH: [splits][rows][pitch]
  int32_t rows, pitch, kdh, add;
  int* status;
};

__device__ __forceinline__ int live_label(const CoreArgs& p, int t, bool& bad) {
  const int64_t lab = load_index(p.labels, p.is64, t);
  const bool live = lab != p.ignore && lab >= 0 && lab < p.vocab;
  bad = !live && lab != p.ignore;
  return live ? (int)lab : -1;
}

// A tile of Z: forward (max, sum) of its rows and the labels' logits, backward G.
template <typename T, bool GRAD>
__global__ void __launch_bounds__(kCoreThreads)
    head_core_z_kernel(const __grid_constant__ CoreArgs p) {
  __shared__ CoreSmem sm;
  __shared__ int32_t label[kCoreTile];
  pdl_launch();
  pdl_wait();
  const int ntm = (p.n + kCoreTile - 1) / kCoreTile;
  const int tm = (int)blockIdx.x % ntm, tn = (int)blockIdx.x / ntm;
  const int m0 = tm * kCoreTile, n0 = tn * kCoreTile;
  if (threadIdx.x < kCoreTile) {
    const int t = m0 + threadIdx.x;
    bool bad = false;
    const int lab = t < p.n ? live_label(p, t, bad) : -1;
    label[threadIdx.x] = lab;
    if (tn == 0 && p.v0 == 0) {
      if (bad) atomicOr(p.status, kStatusBadIndex);
      if (GRAD && t < p.n) p.pos[t] = lab >= 0 ? t : -1;
    }
  }
  __syncthreads();
  float z[4];
  core_product<true, true>(
      sm, static_cast<const T*>(p.hidden), p.ld_h, m0, p.n,
      [&](int r, int) { return label[r - m0] >= 0; }, static_cast<const T*>(p.weight), p.ld_w, n0,
      p.width, [](int, int) { return true; }, 0, p.dim, z);
  const int row = threadIdx.x >> 3, t = m0 + row, lab = label[row];
  const int c0 = n0 + 4 * (threadIdx.x & 7);
  if (GRAD) {
    if (t >= p.n) return;
    const float lse2 = lab >= 0 ? p.lse_in[t] * kLog2e : 0.f, dl = lab >= 0 ? p.dloss[t] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float g = 0.f;
      if (lab >= 0) {
        g = exp2f(fmaf(z[j], kLog2e, -lse2));
        if (p.v0 + c0 + j == lab) g -= 1.f;
        g *= dl;
      }
      if (c0 + j < p.width) p.g[(int64_t)t * p.piece + c0 + j] = g;
    }
  } else {
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c0 + j >= p.width) continue;
      m = fmaxf(m, z[j]);
      if (c0 + j == lab) p.zlab[t] = z[j];
    }
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + j < p.width) s += exp2f((z[j] - ref) * kLog2e);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)        // the eight threads of the row
      merge_stats(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
    if ((threadIdx.x & 7) == 0 && lab >= 0) p.part[(int64_t)t * p.parts + tn] = make_float2(m, s);
  }
}

// A warp per token: the tiles' pairs to loss and lse.
__global__ void __launch_bounds__(kCoreThreads)
    head_core_join_kernel(const __grid_constant__ CoreArgs p) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, t = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= p.n) return;
  bool bad;
  const bool live = live_label(p, t, bad) >= 0;
  float m = -INFINITY, s = 0.f;
  if (live) {
#pragma unroll 4
    for (int i = lane; i < p.parts; i += 32) {
      const float2 v = p.part[(int64_t)t * p.parts + i];
      merge_stats(m, s, v.x, v.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      merge_stats(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
  }
  if (lane != 0) return;
  const float l = live ? m + logf(s) : 0.f;
  if (p.lse) p.lse[t] = l;
  if (p.loss) p.loss[t] = live ? l - p.zlab[t] : 0.f;
}

// Both products of a piece's G: the tiles of dW, then those of dH's slices.
template <typename T>
__global__ void __launch_bounds__(kCoreThreads)
    head_core_grad_kernel(const __grid_constant__ CoreArgs p) {
  __shared__ CoreSmem sm;
  pdl_launch();
  pdl_wait();
  const int ntd = (p.dim + kCoreTile - 1) / kCoreTile, ntm = (p.n + kCoreTile - 1) / kCoreTile;
  const auto all = [](int, int) { return true; };
  const bool of_w = (int)blockIdx.x < p.dw_tiles;
  const int b = of_w ? (int)blockIdx.x : (int)blockIdx.x - p.dw_tiles;
  const int n0 = b % ntd * kCoreTile, m0 = (of_w ? b / ntd : b / ntd % ntm) * kCoreTile;
  const int r = m0 + (threadIdx.x >> 3), c0 = n0 + 4 * (threadIdx.x & 7);
  float v[4];
  if (of_w) {
    core_product<false, false>(sm, p.g, p.piece, m0, p.width, all, static_cast<const T*>(p.hidden),
                               p.ld_h, n0, p.dim, [&](int, int k) { return p.pos[k] >= 0; }, 0,
                               p.n, v);
    if (r >= p.width) return;
    T* out = static_cast<T*>(p.dw) + r * p.ld_dw + c0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + j < p.dim) out[j] = from_f32<T>(v[j]);
    return;
  }
  const int split = b / (ntd * ntm), k0 = split * p.kdh;
  core_product<true, false>(sm, p.g, p.piece, m0, p.n, all, static_cast<const T*>(p.weight), p.ld_w,
                            n0, p.dim, all, k0, min(p.width, k0 + p.kdh), v);
  if (r >= p.n) return;
  float* out = p.acc + ((int64_t)split * p.rows + r) * p.pitch + c0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c0 + j < p.dim) out[j] = p.add ? out[j] + v[j] : v[j];
}

// ---------------------------------------------------------------- host
int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t cdiv(int64_t x, int64_t a) { return (x + a - 1) / a; }

struct HeadShape {
  int64_t n, dim, vocab;
  int32_t dtype;
  bool backward, copy_w;
  bool few;                                // few tokens: head_few_kernel, head_few_grad_kernel
  bool core;                               // small: on the CUDA cores
  int64_t rows, pitch;                     // compacted H (and dH slices)
  int64_t piece, pieces;                   // columns per piece
  int64_t splits;                          // dH slices
  int64_t kdh;                             // fp32: columns per dH slice
  int64_t buffers;                         // pieces of G (and of a copied W) held at a time
};

struct HeadLayout {
  size_t nlive, label, pos, token, lse2, dl, dl_max, scale, zlab, state, hc, part, g, acc, wcopy;
  size_t gsum, wmean;
  size_t ht, gt, wt, descs, total;
};

constexpr int64_t kWorkBytes = 390ll << 20;   // what the backward pass's buffers may come to
constexpr int64_t kMinBytes = 128ll << 20;   // least of them for a piece's columns
constexpr int64_t kZBytes = 128ll << 20;     // fp32: a piece of Z
constexpr int64_t kPartBytes = 64ll << 20;   // bf16 forward: a piece's partials
constexpr int64_t kMinColumns = 4096;        // least columns of a piece
constexpr int kMaxSplits = 64;
// Largest fp32 product that runs on the CUDA cores, in operations of whole tiles.  Both passes
// there and through the 3xTF32 GEMM: 333 tokens x 100 against 1031 rows (0.1 G) 44 and 102 us, 16 x
// 256 against 20000 (0.3 G) 108 and 126, 128 x 512 against 4000 (0.5 G) 136 and 130, 4096 x 64
// against 1000 (0.5 G) 189 and 292, 256 x 256 against 8000 (1.1 G) 216 and 124.
constexpr int64_t kCoreFlops = 1ll << 29;
// The same for bf16, against the tensor cores: 100 x 100 against 1000 (0.03 G) 30 and 56 us, 4 x
// 70 against 7784 (0.06 G) 43 and 55, 1024 x 64 against 1000 (0.13 G) 65 and 50, 16 x 256 against
// 10000 (0.16 G) 65 and 52.
constexpr int64_t kCoreFlopsBf16 = 64ll << 20;
constexpr int kGatherBlocks = 608;         // blocks of the gather launch, at most
constexpr int kFewBlocks = 1024;           // blocks of the few-token kernel (bounds its workspace)
constexpr int kFewGradBlocks = 304;        // and of its backward pass
constexpr int kLayoutSms = 152;            // the workspace's layout does not ask the device
constexpr int kFewSmem = 200 << 10;        // dynamic shared memory the few-token kernels may take

// Slices of dH that a piece of any width may get (head_shape cuts narrow pieces into fewer).  dH has
// few tiles when there are few tokens: its contraction (the piece's columns) is cut until the tiles
// fill the GPU, in one wave where the fp32 GEMM runs the slices alone (the bf16 launch has other
// tiles too).
int64_t most_splits(const HeadShape& s, int sms) {
  const bool bf = s.dtype == MFSDP_DTYPE_BF16;
  const int64_t units = bf ? sms / 2 : sms;
  const int64_t tiles = cdiv(std::max<int64_t>(s.n, 1), bf ? kTile : 128) * cdiv(s.dim, kTile);
  return std::max<int64_t>(1, std::min<int64_t>(bf ? cdiv(units, tiles) : units / tiles, kMaxSplits));
}

// Columns per piece, whole tiles: what a budget leaves for the buffers that grow with a piece, each
// of them counted.  Every piece is a launch whose last wave and ramp cost some 20 us, so the
// backward pass takes what the rows of H and the slices of dH leave of kWorkBytes: 8192 tokens x 768
// ran in 1.54 ms with 48 Mi entries per piece and in 1.53 with 96, 4096 tokens x 4096 in 7.41 and
// 7.23.  A piece takes kMinBytes, and kMinColumns, where that is more.
// With few tokens a piece's Z has few tiles and leaves most of the GPU idle unless the piece is wide.
// An fp32 piece may therefore come to one wave of them within W's bytes, and a piece that does not
// hold the vocabulary is cut to whole waves where that saves some (64 tokens x 4090 against 128256
// copied bf16 rows, backward: one wave, 19456 columns, 1.84 ms, 24576 columns 1.97, 32768 2.49).
// Holding all of a copied or transposed W would be faster by a few per cent and take its size in
// memory (both passes: 64 x 4096 against 128256 fp32 rows 4.1 ms with 2.3 GB and 4.4 with 0.7, 39 x
// 3143 against 110695 copied bf16 rows 1.6 with 0.8 GB and 1.8 with 0.4).
int64_t piece_columns(const HeadShape& s, int64_t asked, int sms) {
  const bool bf = s.dtype == MFSDP_DTYPE_BF16;
  const int64_t es = bf ? 2 : 4, copy = s.copy_w ? s.pitch * es : 0;
  const int64_t weight = s.vocab * s.pitch * es;
  // Z's tiles (256 x 256 per CTA pair, fp32 128 x 256 per CTA): rows of them, and the columns of a
  // wave
  const int64_t units = bf ? sms / 2 : sms;
  const int64_t ntm = cdiv(std::max<int64_t>(s.n, 1), bf ? kTile : 128), wave = units / ntm * kTile;
  int64_t c = asked;
  if (asked == 0 && s.backward) {
    // bf16: the copy of H and the slices; two pieces of G (their row sums are 1 / 128 of them), two
    // of a copied W.  fp32: H transposed too; Z, G transposed, and W transposed (where a copied W
    // was)
    const int64_t fixed = s.rows * s.pitch * (es * (bf ? 1 : 2) + 4 * most_splits(s, sms));
    const int64_t column = bf ? 2 * (s.rows * es + copy) : (2 * s.rows + s.pitch) * es;
    c = std::max(kWorkBytes - fixed, kMinBytes) / column;
    if (!bf)
      c = std::min(std::max(c, std::min(wave, (weight - fixed) / column)), kZBytes / (s.rows * es));
  } else if (asked == 0) {
    // a half-tile's (max, sum) or Z, and a copied W
    const int64_t bytes = bf ? kPartBytes : kZBytes;
    c = bytes / (bf ? cdiv(8 * s.rows, 128) : s.rows * es);
    if (s.copy_w)
      c = std::min(c, std::max((kWorkBytes - bytes) / copy, bf ? 0 : std::min(wave, weight / copy)));
  }
  if (asked == 0) {
    auto waves = [&](int64_t c) {
      return s.vocab / c * cdiv(ntm * cdiv(c, kTile), units) +
             cdiv(ntm * cdiv(s.vocab % c, kTile), units);
    };
    const int64_t whole = wave > 0 ? c - c % wave : 0;
    if (c < s.vocab && whole >= kMinColumns && waves(whole) < waves(c)) c = whole;
    c = std::max(c, kMinColumns);
  }
  return std::min(up(c, kTile), up(s.vocab, kTile));
}

// The few-token kernels are built for 1, 2 and 4 tokens.
int64_t few_width(int64_t n) { return n <= 2 ? std::max<int64_t>(n, 1) : 4; }

HeadShape head_shape(int64_t n, int64_t dim, int64_t vocab, int32_t dtype, bool backward,
                     const void* weight, int64_t ld_w, int64_t piece, int sms) {
  HeadShape s{};
  s.n = n;
  s.dim = dim;
  s.vocab = vocab;
  s.dtype = dtype;
  s.backward = backward;
  const bool bf = dtype == MFSDP_DTYPE_BF16;
  // TMA reads rows that start on 16-byte boundaries
  s.copy_w = !aligned_to(weight, 16) || ld_w % (bf ? 8 : 4) != 0;
  // (counted as the tiles are; the product of the three would pass 64 bits)
  const bool small = 2 * up(std::max<int64_t>(n, 1), kCoreTile) * up(dim, kCoreK) <=
                     (bf ? kCoreFlopsBf16 : kCoreFlops) / up(vocab, kCoreTile);
  // Few tokens, whose hidden rows (and sums) have to fit in shared memory.  Backward against the
  // other paths: 1 token x 2981 and 3264 fp32 rows 72 and 305 us, 4 x 768 and 50257 fp32 rows 233
  // and 355, 4 x 70 and 7784 bf16 rows 30 and 44.
  // bf16 that the tensor cores can read, both passes of one token (of two): 2048 and 128256 rows
  // 349 and 428 (360 and 447) us, 1024 and 50257 100 and 132 (110 and 144), 256 and 50257 51 and 77,
  // 768 and 32000 75 and 116, but 768 and 50257 115 and 109 (116 and 121), 512 and 128256 197 and
  // 168 (196 and 182), 768 and 128256 258 and 207 (249 and 221), 640 and 80000 153 and 144 (152 and
  // 154).  Between 256 and 1024 columns the rounds of loads are short and threads idle in the second
  // phase, so there the tensor cores take large weights.  (4 x 4096 and 128256: 1150 and 798.)
  const bool tensor = dim > 256 && dim < 1024 && dim * vocab > (n + 1) * (18 << 20);
  s.few = backward ? n >= 1 && n <= kFewTokens &&
                         (!bf || s.copy_w || small || (n <= 2 && !tensor)) &&
                         2 * up(dim, 8) * 4 * few_width(n) <= kFewSmem
                   : n <= (bf && !s.copy_w ? 1 : kFewTokens) &&
                         up(dim, 8) * 4 * kFewTokens <= kFewSmem;
  s.core = !s.few && small;
  if (s.few || s.core) s.copy_w = false;
  s.rows = up(std::max<int64_t>(n, 1), bf ? kTile : 32);   // (the fp32 GEMM takes any count)
  s.pitch = up(dim, 64);
  s.piece = piece_columns(s, piece, sms);
  s.pieces = cdiv(vocab, s.piece);
  s.splits = 1;
  s.buffers = 1;
  if (backward) {
    // a slice keeps at least 1024 columns (fp32: 128, its k-blocks are slower)
    s.splits = std::max<int64_t>(1, std::min(most_splits(s, sms), s.piece / (bf ? 1024 : 128)));
    s.kdh = up(cdiv(std::min(s.piece, vocab), s.splits), kBK);  // no slice of a whole piece is empty
    s.splits = cdiv(std::min(s.piece, vocab), s.kdh);
    if (s.core) {                          // two blocks per SM, slices of at least 128 columns
      const int64_t few_tiles = cdiv(std::max<int64_t>(n, 1), kCoreTile) * cdiv(dim, kCoreTile);
      const int64_t cols = std::min(s.piece, vocab);
      s.splits = std::max<int64_t>(1, std::min({2 * sms / few_tiles, cols / 128,
                                                (int64_t)kMaxSplits}));
      s.kdh = up(cdiv(cols, s.splits), kCoreK);
      s.splits = cdiv(cols, s.kdh);
    }
    s.buffers = bf && s.pieces > 1 ? 2 : 1;
  }
  return s;
}

HeadLayout head_layout(const HeadShape& s) {
  HeadLayout l{};
  size_t off = 0;
  // (the few-token kernel needs its partials and the labels' logits only)
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += (size_t)up(bytes, 1024);
    return at;
  };
  const bool bf = s.dtype == MFSDP_DTYPE_BF16;
  const int64_t es = bf ? 2 : 4;
  if (s.few && s.backward) {
    l.acc = take(kFewGradBlocks * s.n * s.pitch * 4);
    l.total = off;
    return l;
  }
  if (s.few) {
    l.zlab = take(kFewTokens * 4);
    l.part = take(kFewBlocks * kFewTokens * 8);
    l.total = off;
    return l;
  }
  if (s.core) {
    l.pos = take(s.backward ? s.rows * 4 : 0);
    l.zlab = take(s.rows * 4);
    l.part = take(s.backward ? 0 : s.n * cdiv(s.vocab, kCoreTile) * 8);
    l.g = take(s.backward ? s.n * s.piece * 4 : 0);
    l.acc = take(s.backward ? s.splits * s.rows * s.pitch * 4 : 0);
    l.total = off;
    return l;
  }
  l.nlive = take(4);
  l.label = take(s.rows * 4);
  l.pos = take(s.rows * 4);
  l.token = take(s.rows * 4);
  l.lse2 = take(s.backward ? s.rows * 4 : 0);
  l.dl = take(s.backward ? s.rows * 4 : 0);
  l.dl_max = take(s.backward ? kGatherBlocks * 4 : 0);
  l.scale = take(4);
  l.zlab = take(s.rows * 4);
  l.state = take(s.rows * 8);
  l.hc = take(s.rows * s.pitch * es);
  l.part = take(!s.backward && bf ? cdiv(s.piece, 128) * s.rows * 8 : 0);
  l.g = take(s.backward || !bf ? s.buffers * s.rows * s.piece * es : 0);
  l.acc = take(s.backward ? s.splits * s.rows * s.pitch * 4 : 0);
  l.gsum = take(s.backward && bf ? s.rows * cdiv(s.piece, 128) * 4 : 0);
  l.wmean = take(s.backward && bf ? s.pitch * 4 : 0);
  l.wcopy = take(s.copy_w ? s.buffers * s.piece * s.pitch * es : 0);
  const bool t32 = s.backward && !bf;        // fp32: transposed H, G piece and W piece
  l.ht = take(t32 ? s.pitch * s.rows * 4 : 0);
  l.gt = take(t32 ? s.piece * s.rows * 4 : 0);
  // (the transposed piece is made after the copied one's last use, in the same place)
  l.wt = t32 && s.copy_w ? l.wcopy : take(t32 ? s.pitch * s.piece * 4 : 0);
  l.descs = take(bf ? 0 : (int64_t)sizeof(GemmDesc) * (s.pieces * (2 + s.splits)));
  l.total = off;
  return l;
}

// CTA pairs of the tensor-core kernel that run at the same time (the grid's size).
int head_pairs(int sms) {
  constexpr int kCached = 64;
  static std::atomic<int> cache[kCached];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  int n = dev < kCached ? cache[dev].load() : 0;
  if (n > 0) return n;
  const void* kernels[2] = {(const void*)head_gemm_kernel<kStats>,
                            (const void*)head_gemm_kernel<kGrads>};
  for (const void* k : kernels)
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kHeadSmem) !=
        cudaSuccess)
      return -1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
  cfg.blockDim = dim3(kHeadThreads, 1, 1);
  cfg.dynamicSmemBytes = kHeadSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, head_gemm_kernel<kGrads>, &cfg) != cudaSuccess || n < 1)
    return -1;
  if (dev < kCached) cache[dev].store(n);
  return n;
}

// Raises a few-token kernel's shared-memory limit, once per device; `done` is the kernel's own.  The
// limit belongs to the kernel, not to a launch: set to what each call needs, a narrow call of one
// host thread would take it from under a wide call of another before that one launches.
constexpr int kFewDevices = 64;
template <typename K>
cudaError_t allow_few_smem(std::atomic<bool>* done, K kernel) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < kFewDevices && done[dev].load())) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  if (e == cudaSuccess && dev < kFewDevices) done[dev].store(true);
  return e;
}

template <int PHASE>
cudaError_t launch_head(const HeadArgs& a, int64_t tiles, int pairs, cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (unsigned)std::max<int64_t>(1, std::min<int64_t>(tiles, pairs)), 1, 1);
  cfg.blockDim = dim3(kHeadThreads, 1, 1);
  cfg.dynamicSmemBytes = kHeadSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, head_gemm_kernel<PHASE>, a);
}

struct HeadCall {
  HeadShape s;
  HeadLayout l;
  char* ws;
  const void *hidden, *weight, *labels;
  int64_t ld_h, ld_w, ignore;
  int32_t index_dtype;
  float *loss, *lse;                       // forward outputs, nullable
  const float *lse_in, *dloss;
  void *dh, *dw;
  int64_t ld_dh, ld_dw;
  int sms;
  int* status;
  cudaStream_t st;

  template <typename T>
  T* at(size_t off) const { return reinterpret_cast<T*>(ws + off); }

  cudaError_t gather() const {
    GatherArgs a{};
    a.labels = labels;
    a.hidden = hidden;
    a.hc = at<void>(l.hc);
    a.ld_h = ld_h;
    a.ignore = ignore;
    a.n = (int32_t)s.n;
    a.is64 = index_dtype == MFSDP_INDEX_I64;
    a.dim = (int32_t)s.dim;
    a.pitch = (int32_t)s.pitch;
    a.vocab = (int32_t)s.vocab;
    a.per = (int32_t)std::max<int64_t>(8, cdiv(s.n, kGatherBlocks));
    a.vec = aligned_to(hidden, 16) && s.dim % 8 == 0 &&
            (ld_h * (int64_t)dtype_bytes(s.dtype)) % 16 == 0;
    a.place = s.dtype == MFSDP_DTYPE_F32;
    a.nlive = at<int32_t>(l.nlive);
    a.label = at<int32_t>(l.label);
    a.pos = at<int32_t>(l.pos);
    a.token = at<int32_t>(l.token);
    if (s.backward) {
      a.lse_in = lse_in;
      a.dloss = dloss;
      a.lse2 = at<float>(l.lse2);
      a.dl = at<float>(l.dl);
      a.dl_max = at<float>(l.dl_max);
    }
    a.loss = loss;
    a.lse = lse;
    a.status = status;
    a.blocks = (int32_t)cdiv(s.n, a.per);
    int64_t mean_blocks = 0;
    if (takes_common()) {
      a.weight = weight;
      a.ld_w = ld_w;
      a.wmean = at<float>(l.wmean);
      mean_blocks = s.pitch / 32;
    }
    const dim3 grid((unsigned)(a.blocks + mean_blocks));
    return s.dtype == MFSDP_DTYPE_BF16
               ? launch_pdl(head_gather_kernel<bf16_t>, grid, dim3(256), 0, st, a)
               : launch_pdl(head_gather_kernel<float>, grid, dim3(256), 0, st, a);
  }

  // G is rounded to bf16 and dH wanted: the common part of W's rows is taken off
  bool takes_common() const {
    return s.backward && s.dtype == MFSDP_DTYPE_BF16 && !s.core && !s.few && dh;
  }
  int32_t gsum_parts() const { return (int32_t)cdiv(std::min(s.piece, s.vocab), 128); }

  cudaError_t finish() const {
    FinishArgs f{};
    if (takes_common()) {
      f.gsum = at<float>(l.gsum);
      f.wmean = at<float>(l.wmean);
      f.gsum_parts = gsum_parts();
    }
    f.acc = at<float>(l.acc);
    f.scale = s.dtype == MFSDP_DTYPE_BF16 && !s.core ? at<float>(l.scale) : nullptr;
    f.pos = at<int32_t>(l.pos);
    f.dh = dh;
    f.ld_dh = ld_dh;
    f.dim = (int32_t)s.dim;
    f.pitch = (int32_t)s.pitch;
    f.rows = (int32_t)s.rows;
    f.splits = (int32_t)s.splits;
    f.vec = aligned_to(dh, 16) && s.dim % 8 == 0 &&
            (ld_dh * (int64_t)dtype_bytes(s.dtype)) % 16 == 0;
    return s.dtype == MFSDP_DTYPE_BF16
               ? launch_pdl(head_finish_kernel<bf16_t>, dim3((unsigned)s.n), dim3(256), 0, st, f)
               : launch_pdl(head_finish_kernel<float>, dim3((unsigned)s.n), dim3(256), 0, st, f);
  }

  // `width` rows of the weight into whole k-blocks of aligned rows
  template <typename T>
  cudaError_t copy_rows(const T* from, T* to, int64_t width) const {
    const int64_t total = up(width, kBK);
    return launch_pdl(head_copy_rows_kernel<T>, dim3((unsigned)cdiv(total, 8)), dim3(256), 0, st, from,
                      ld_w, to, s.pitch, (int)width, (int)total, (int)s.dim);
  }

  template <typename T, int NT>
  cudaError_t launch_few(const FewArgs& a, size_t smem) const {
    if (smem > 48 * 1024) {
      static std::atomic<bool> done[kFewDevices];
      const cudaError_t e = allow_few_smem(done, head_few_kernel<T, NT>);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(head_few_kernel<T, NT>, dim3((unsigned)a.blocks), dim3(32 * kFewWarps), smem, st,
                      a);
  }

  // The forward pass of few tokens (few_tokens() of the shape).
  int run_few() const {
    FewArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.labels = labels;
    a.ld_h = ld_h;
    a.ld_w = ld_w;
    a.ignore = ignore;
    a.part = at<float2>(l.part);
    a.zlab = at<float>(l.zlab);
    a.loss = loss;
    a.lse = lse;
    a.n = (int32_t)s.n;
    a.dim = (int32_t)s.dim;
    a.vocab = (int32_t)s.vocab;
    a.is64 = index_dtype == MFSDP_INDEX_I64;
    a.vec = aligned_to(weight, 16) && s.dim % 8 == 0 &&
            (ld_w * (int64_t)dtype_bytes(s.dtype)) % 16 == 0;
    a.status = status;
    const int nt = s.n == 1 ? 1 : s.n == 2 ? 2 : 4;
    const size_t smem = (size_t)up(s.dim, 8) * 4 * nt;
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(4, kFewSmem / (int64_t)smem));
    a.blocks = (int32_t)std::min<int64_t>(std::min(per_sm * sms, (int64_t)kFewBlocks),
                                          cdiv(s.vocab, kFewWarps * kFewRows));
    cudaError_t e;
    if (s.dtype == MFSDP_DTYPE_BF16)
      e = nt == 1 ? launch_few<bf16_t, 1>(a, smem)
          : nt == 2 ? launch_few<bf16_t, 2>(a, smem) : launch_few<bf16_t, 4>(a, smem);
    else
      e = nt == 1 ? launch_few<float, 1>(a, smem)
          : nt == 2 ? launch_few<float, 2>(a, smem) : launch_few<float, 4>(a, smem);
    if (e == cudaSuccess)
      e = launch_pdl(head_few_join_kernel, dim3((unsigned)s.n), dim3(kFewJoinThreads), 0, st, a);
    return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
  }

  int run_bf16() const {
    const int pairs = head_pairs(sms);
    if (pairs < 1) return MFSDP_ECUDA;
    HeadArgs a{};
    const uint16_t* hc = at<uint16_t>(l.hc);
    bool ok = encode_map(&a.h_k, hc, s.rows, s.pitch, s.pitch, 128u);
    const void* wsrc = s.copy_w ? (const void*)at<uint16_t>(l.wcopy) : weight;
    const int64_t wrows = s.copy_w ? s.buffers * s.piece : s.vocab, wld = s.copy_w ? s.pitch : ld_w;
    ok = ok && encode_map(&a.w_k, wsrc, wrows, s.dim, wld, 128u);
    if (s.backward) {
      ok = ok && encode_map3d(&a.h_mn, hc, s.rows, s.pitch, s.pitch);
      a.w_3d = s.dim % 64 == 0;
      ok = ok && (a.w_3d ? encode_map3d(&a.w_mn, wsrc, wrows, s.dim, wld)
                         : encode_map(&a.w_mn, wsrc, wrows, s.dim, wld, 64u));
      const uint16_t* g = at<uint16_t>(l.g);
      ok = ok && encode_map(&a.g_k, g, s.buffers * s.rows, s.piece, s.piece, 128u);
      ok = ok && encode_map3d(&a.g_mn, g, s.buffers * s.rows, s.piece, s.piece);
      a.g = at<uint16_t>(l.g);
      a.piece = s.piece;
      if (takes_common()) {
        a.gsum = at<float>(l.gsum);
        a.gsum_parts = gsum_parts();
      }
      if (dh)
        ok = ok && encode_map_f32(&a.acc_st, at<float>(l.acc), s.splits * s.rows, s.pitch, s.pitch,
                                  32u);
      a.dw_tma = dw && aligned_to(dw, 16) && ld_dw % 8 == 0;
      if (a.dw_tma) ok = ok && encode_map(&a.dw_st, dw, s.vocab, s.dim, ld_dw, 32u, 32u, false);
    }
    if (!ok) return MFSDP_ECUDA;
    a.nlive = at<int32_t>(l.nlive);
    a.label = at<int32_t>(l.label);
    a.lse2 = at<float>(l.lse2);
    a.dl = at<float>(l.dl);
    a.dl_max = at<float>(l.dl_max);
    a.dl_blocks = (int32_t)cdiv(s.n, std::max<int64_t>(8, cdiv(s.n, kGatherBlocks)));
    a.scale = at<float>(l.scale);
    a.part = at<float2>(l.part);
    a.zlab = at<float>(l.zlab);
    a.dw = static_cast<uint16_t*>(dw);
    a.ld_dw = ld_dw;
    a.dim = (int32_t)s.dim;
    a.rows = (int32_t)s.rows;
    a.splits = (int32_t)s.splits;
    a.want_dh = dh != nullptr;
    a.want_dw = dw != nullptr;
    // a group's rows of H (all of its columns) stay within a share of the L2
    a.group = (int32_t)std::max<int64_t>(4, (32ll << 20) / (kTile * s.pitch * 2));
    a.wait_limit_ns = wait_limit_ns();
    a.status = status;
    const int64_t ntm = cdiv(s.n, kTile), ntd = cdiv(s.dim, kTile);
    // piece i as the one whose Z is computed
    auto set_z = [&](int64_t i) {
      a.z_v0 = (int32_t)(i * s.piece);
      a.z_width = i < s.pieces ? (int32_t)std::min(s.piece, s.vocab - i * s.piece) : 0;
      a.z_w_row0 = s.copy_w ? (int32_t)(i % s.buffers * s.piece) : a.z_v0;
      a.z_g_row0 = (int32_t)(i % s.buffers * s.rows);
      if (i >= s.pieces || !s.copy_w) return cudaSuccess;
      return copy_rows(static_cast<const bf16_t*>(weight) + (int64_t)a.z_v0 * ld_w,
                       at<bf16_t>(l.wcopy) + (int64_t)a.z_w_row0 * s.pitch, a.z_width);
    };
    auto z_tiles = [&] { return ntm * cdiv(a.z_width, kTile); };
    cudaError_t e = gather();
    if (e == cudaSuccess) e = set_z(0);
    if (s.backward && e == cudaSuccess) e = launch_head<kGrads>(a, z_tiles(), pairs, st);
    for (int64_t i = 0; i < s.pieces && e == cudaSuccess; ++i) {
      if (!s.backward) {
        if (i > 0) e = set_z(i);
        if (e == cudaSuccess) e = launch_head<kStats>(a, z_tiles(), pairs, st);
        if (e != cudaSuccess) break;
        JoinArgs j{};
        j.part = a.part;
        j.state = at<float2>(l.state);
        j.zlab = a.zlab;
        j.nlive = a.nlive;
        j.token = at<int32_t>(l.token);
        j.loss = loss;
        j.lse = lse;
        j.parts = (int32_t)cdiv(a.z_width, 128);
        j.rows = a.rows;
        j.first = i == 0;
        j.last = i == s.pieces - 1;
        e = launch_pdl(head_join_kernel, dim3((unsigned)cdiv(s.n, 32)), dim3(1024), 0, st, j);
      } else {
        a.v0 = a.z_v0;
        a.width = a.z_width;
        a.w_row0 = a.z_w_row0;
        a.g_row0 = a.z_g_row0;
        a.add = i > 0;
        e = set_z(i + 1);
        if (e != cudaSuccess) break;
        const int64_t tiles = (dh ? ntm * ntd * s.splits : 0) + (dw ? cdiv(a.width, kTile) * ntd : 0);
        e = launch_head<kGrads>(a, tiles + z_tiles(), pairs, st);
      }
    }
    if (e == cudaSuccess && dh) e = finish();
    return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
  }

  int run() const {
    if (s.few && s.backward)
      return s.dtype == MFSDP_DTYPE_BF16 ? run_few_grad<bf16_t>() : run_few_grad<float>();
    if (s.few) return run_few();
    if (s.core)
      return s.dtype == MFSDP_DTYPE_BF16 ? run_core<bf16_t>() : run_core<float>();
    if (s.dtype == MFSDP_DTYPE_BF16) return run_bf16();
    try {
      return run_f32();
    } catch (const std::bad_alloc&) {  // the problem table of very many pieces
      return MFSDP_ESHAPE;
    }
  }

  template <typename T, int NT, int C>
  cudaError_t launch_few_grad(const FewGradArgs& a, size_t smem) const {
    if (smem > 48 * 1024) {
      static std::atomic<bool> done[kFewDevices];
      const cudaError_t e = allow_few_smem(done, head_few_grad_kernel<T, NT, C>);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(head_few_grad_kernel<T, NT, C>, dim3((unsigned)a.blocks),
                      dim3(kFewGradThreads), smem, st, a);
  }

  template <typename T>
  int run_few_grad() const {
    FewGradArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.labels = labels;
    a.ld_h = ld_h;
    a.ld_w = ld_w;
    a.ignore = ignore;
    a.lse = lse_in;
    a.dloss = dloss;
    a.dh = dh;
    a.dw = dw;
    a.ld_dh = ld_dh;
    a.ld_dw = ld_dw;
    a.acc = at<float>(l.acc);
    a.n = (int32_t)s.n;
    a.dim = (int32_t)s.dim;
    a.vocab = (int32_t)s.vocab;
    a.is64 = index_dtype == MFSDP_INDEX_I64;
    a.pitch = (int32_t)s.pitch;
    a.status = status;
    const bool vec = s.dim % 4 == 0 && aligned_to(weight, 4 * sizeof(T)) && ld_w % 4 == 0 &&
                     (!dw || (aligned_to(dw, 4 * sizeof(T)) && ld_dw % 4 == 0));
    const int nt = (int)few_width(s.n);
    const size_t smem = (size_t)up(s.dim, 8) * 8 * nt;
    const int64_t per_sm = smem <= (100 << 10) ? 2 : 1;
    a.blocks = (int32_t)std::min({per_sm * sms, (int64_t)kFewGradBlocks,
                                  cdiv(s.vocab, kFewGradWarps)});
    cudaError_t e;
    if (vec)
      e = nt == 1   ? launch_few_grad<T, 1, 4>(a, smem)
          : nt == 2 ? launch_few_grad<T, 2, 4>(a, smem)
                    : launch_few_grad<T, 4, 4>(a, smem);
    else
      e = nt == 1   ? launch_few_grad<T, 1, 1>(a, smem)
          : nt == 2 ? launch_few_grad<T, 2, 1>(a, smem)
                    : launch_few_grad<T, 4, 1>(a, smem);
    if (e == cudaSuccess && dh)
      e = launch_pdl(head_few_finish_kernel<T>, dim3((unsigned)cdiv(s.dim, 32), (unsigned)s.n),
                     dim3(1024), 0, st, a);
    return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
  }

  template <typename T>
  int run_core() const {
    CoreArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.labels = labels;
    a.ld_h = ld_h;
    a.ld_w = ld_w;
    a.ignore = ignore;
    a.n = (int32_t)s.n;
    a.dim = (int32_t)s.dim;
    a.vocab = (int32_t)s.vocab;
    a.is64 = index_dtype == MFSDP_INDEX_I64;
    a.zlab = at<float>(l.zlab);
    a.status = status;
    const int64_t ntm = cdiv(s.n, kCoreTile), ntd = cdiv(s.dim, kCoreTile);
    const dim3 threads(kCoreThreads);
    cudaError_t e = cudaSuccess;
    if (!s.backward) {
      a.width = a.vocab;
      a.part = at<float2>(l.part);
      a.parts = (int32_t)cdiv(s.vocab, kCoreTile);
      a.loss = loss;
      a.lse = lse;
      e = launch_pdl(head_core_z_kernel<T, false>, dim3((unsigned)(ntm * a.parts)), threads, 0, st,
                     a);
      if (e == cudaSuccess)
        e = launch_pdl(head_core_join_kernel, dim3((unsigned)cdiv(s.n, 8)), threads, 0, st, a);
      return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
    }
    a.lse_in = lse_in;
    a.dloss = dloss;
    a.g = at<float>(l.g);
    a.piece = s.piece;
    a.pos = at<int32_t>(l.pos);
    a.ld_dw = ld_dw;
    a.acc = at<float>(l.acc);
    a.rows = (int32_t)s.rows;
    a.pitch = (int32_t)s.pitch;
    a.kdh = (int32_t)s.kdh;
    for (int64_t i = 0; i < s.pieces && e == cudaSuccess; ++i) {
      const int64_t v0 = i * s.piece, width = std::min(s.piece, s.vocab - v0);
      a.weight = static_cast<const T*>(weight) + v0 * ld_w;
      a.v0 = (int32_t)v0;
      a.width = (int32_t)width;
      a.dw = dw ? static_cast<T*>(dw) + v0 * ld_dw : nullptr;
      a.dw_tiles = dw ? (int32_t)(cdiv(width, kCoreTile) * ntd) : 0;
      a.add = i > 0;
      // (a narrower last piece may leave slices without columns: nothing to add there)
      const int64_t dh_tiles = dh ? ntm * ntd * cdiv(width, s.kdh) : 0;
      e = launch_pdl(head_core_z_kernel<T, true>, dim3((unsigned)(ntm * cdiv(width, kCoreTile))),
                     threads, 0, st, a);
      if (e == cudaSuccess)
        e = launch_pdl(head_core_grad_kernel<T>, dim3((unsigned)(a.dw_tiles + dh_tiles)), threads, 0,
                       st, a);
    }
    if (e == cudaSuccess && dh) e = finish();
    return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
  }

  int run_f32() const {
    // problem tables of every piece: Z, dW, and dH's slices
    const int64_t per = s.backward ? 2 + s.splits : 1;
    std::vector<GemmDesc> d((size_t)(s.pieces * per));
    GemmDesc* dev = at<GemmDesc>(l.descs);
    const float* hc = at<float>(l.hc);
    float* z = at<float>(l.g);
    float* acc = at<float>(l.acc);
    const float* w = static_cast<const float*>(weight);
    for (int64_t i = 0; i < s.pieces; ++i) {
      const int64_t v0 = i * s.piece, width = std::min(s.piece, s.vocab - v0);
      GemmDesc q{};
      q.a = hc;
      q.lda = (int32_t)s.pitch;
      q.b = s.copy_w ? at<float>(l.wcopy) : w + v0 * ld_w;
      q.ldb = (int32_t)(s.copy_w ? s.pitch : ld_w);
      q.c = z;
      q.ldc = (int32_t)s.piece;
      q.m = (int32_t)s.n;
      q.n = (int32_t)width;
      q.k = (int32_t)s.dim;
      q.alpha = 1.f;
      d[(size_t)(i * per)] = q;
      if (!s.backward) continue;
      q = GemmDesc{};
      q.a = at<float>(l.gt);
      q.lda = (int32_t)s.rows;
      q.b = at<float>(l.ht);
      q.ldb = (int32_t)s.rows;
      q.c = dw ? static_cast<float*>(dw) + v0 * ld_dw : nullptr;
      q.ldc = (int32_t)ld_dw;
      q.m = (int32_t)width;
      q.n = (int32_t)s.dim;
      q.k = (int32_t)s.n;
      q.alpha = 1.f;
      d[(size_t)(i * per + 1)] = q;
      for (int64_t k = 0; k < s.splits; ++k) {
        const int64_t c0 = k * s.kdh, cw = std::min(s.kdh, width - c0);
        q = GemmDesc{};
        q.a = z + c0;
        q.lda = (int32_t)s.piece;
        q.b = at<float>(l.wt) + c0;
        q.ldb = (int32_t)s.piece;
        q.c = acc + k * s.rows * s.pitch;
        q.ldc = (int32_t)s.pitch;
        q.m = (int32_t)s.n;
        q.n = (int32_t)s.dim;
        q.k = (int32_t)std::max<int64_t>(cw, 0);
        q.alpha = 1.f;
        q.beta = i > 0 ? 1.f : 0.f;
        d[(size_t)(i * per + 2 + k)] = q;
      }
    }
    cudaError_t e = cudaSuccess;
    for (size_t b = 0; b < d.size() && e == cudaSuccess; b += kDescBatch) {
      DescArgs t{};
      t.n = (int32_t)std::min<size_t>(kDescBatch, d.size() - b);
      std::memcpy(t.d, d.data() + b, sizeof(GemmDesc) * (size_t)t.n);
      t.out = dev + b;
      e = launch_pdl(head_descs_kernel, dim3(1), dim3(64), 0, st, t);
    }
    if (e == cudaSuccess) e = gather();
    auto transpose = [&](const float* src, int64_t ld, int64_t rows, int64_t cols, float* dst,
                         int64_t ld_dst) {
      return launch_pdl(head_transpose32_kernel, dim3((unsigned)(cdiv(cols, 32) * cdiv(rows, 32))),
                        dim3(256), 0, st, src, ld, (int)rows, (int)cols, dst, ld_dst);
    };
    if (e == cudaSuccess && dw) e = transpose(hc, s.pitch, s.n, s.dim, at<float>(l.ht), s.rows);
    if (e != cudaSuccess) return MFSDP_ECUDA;
    for (int64_t i = 0; i < s.pieces; ++i) {
      const int64_t v0 = i * s.piece, width = std::min(s.piece, s.vocab - v0), at0 = i * per;
      if (s.copy_w && copy_rows(w + v0 * ld_w, at<float>(l.wcopy), width) != cudaSuccess)
        return MFSDP_ECUDA;
      int r = launch_gemm(dev + at0, d.data() + at0, 1, 0, 1, st);
      if (r != MFSDP_OK) return r;
      if (!s.backward) {
        Stats32Args a{};
        a.z = z;
        a.state = at<float2>(l.state);
        a.zlab = at<float>(l.zlab);
        a.label = at<int32_t>(l.label);
        a.token = at<int32_t>(l.token);
        a.loss = loss;
        a.lse = lse;
        a.width = (int32_t)width;
        a.v0 = (int32_t)v0;
        a.first = i == 0;
        a.last = i == s.pieces - 1;
        a.ldz = s.piece;
        e = launch_pdl(head_stats32_kernel, dim3((unsigned)s.n), dim3(256), 0, st, a);
        if (e != cudaSuccess) return MFSDP_ECUDA;
        continue;
      }
      Grad32Args a{};
      a.z = z;
      a.gt = dw ? at<float>(l.gt) : nullptr;
      a.label = at<int32_t>(l.label);
      a.lse2 = at<float>(l.lse2);
      a.dl = at<float>(l.dl);
      a.rows = (int32_t)s.n;
      a.width = (int32_t)width;
      a.v0 = (int32_t)v0;
      a.ldz = s.piece;
      a.ldt = s.rows;
      e = launch_pdl(head_grad32_kernel, dim3((unsigned)(cdiv(width, 32) * cdiv(s.n, 32))),
                     dim3(256), 0, st, a);
      if (e == cudaSuccess && dh)
        e = transpose(w + v0 * ld_w, ld_w, width, s.dim, at<float>(l.wt), s.piece);
      if (e != cudaSuccess) return MFSDP_ECUDA;
      if (dw) {
        r = launch_gemm(dev + at0 + 1, d.data() + at0 + 1, 1, 0, 1, st);
        if (r != MFSDP_OK) return r;
      }
      if (dh) {
        // (a narrower last piece may leave slices without columns: nothing to add there)
        r = launch_gemm(dev + at0 + 2, d.data() + at0 + 2, (int)cdiv(width, s.kdh), 0, 1, st);
        if (r != MFSDP_OK) return r;
      }
    }
    if (dh) e = finish();
    return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
  }
};

int check_head(int64_t n, int64_t dim, int64_t vocab, int32_t dtype, int64_t ld_w, int64_t piece) {
  if (!dtype_ok(dtype) || piece < 0) return MFSDP_EINVAL;
  if (n < 0 || dim < 1 || vocab < 1 || n > (1ll << 28) || dim > (1 << 20) || vocab > (1ll << 30) ||
      piece > (1ll << 30))
    return MFSDP_ESHAPE;
  if (ld_w < dim) return MFSDP_EINVAL;
  // tiles (and the fp32 path's 32 x 32 blocks) of a piece are counted in 32 bits
  const int64_t cols = std::max(std::min(piece, vocab), dim);
  if (ld_w >= (1ll << 31) || cdiv(n, 32) * cdiv(cols, 32) >= (1ll << 31)) return MFSDP_ESHAPE;
  return MFSDP_OK;
}

int check_common(int64_t n, int64_t dim, int32_t dtype, const void* hidden, int64_t ld_h,
                 const void* weight, int32_t index_dtype, const void* labels, const void* ws) {
  if (index_dtype != MFSDP_INDEX_I32 && index_dtype != MFSDP_INDEX_I64) return MFSDP_EINVAL;
  if (!weight || !ws || (n > 0 && (!hidden || !labels || ld_h < dim))) return MFSDP_EINVAL;
  const size_t es = dtype_bytes(dtype);
  if (!aligned_to(hidden, es) || !aligned_to(weight, es) ||
      !aligned_to(labels, index_dtype == MFSDP_INDEX_I64 ? 8 : 4) || !aligned_to(ws, 256))
    return MFSDP_EALIGN;
  return MFSDP_OK;
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" int mfsdp_head_loss_workspace_bytes(int64_t n_tokens, int64_t dim, int64_t vocab,
                                               int32_t dtype, int32_t backward,
                                               const void* weight, int64_t ld_weight,
                                               int64_t piece, size_t* bytes_out) {
  if (!bytes_out) return MFSDP_EINVAL;
  const int chk = check_head(n_tokens, dim, vocab, dtype, ld_weight, piece);
  if (chk != MFSDP_OK) return chk;
  *bytes_out = head_layout(head_shape(n_tokens, dim, vocab, dtype, backward != 0, weight, ld_weight,
                                      piece, kLayoutSms)).total;
  return MFSDP_OK;
}

extern "C" int mfsdp_head_loss_forward(int64_t n_tokens, int64_t dim, int64_t vocab,
                                       int32_t dtype, const void* hidden, int64_t ld_hidden,
                                       const void* weight, int64_t ld_weight,
                                       int32_t index_dtype, const void* labels,
                                       int64_t ignore_index, float* loss, float* lse,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  int chk = check_head(n_tokens, dim, vocab, dtype, ld_weight, 0);
  if (chk == MFSDP_OK)
    chk = check_common(n_tokens, dim, dtype, hidden, ld_hidden, weight, index_dtype, labels, workspace);
  if (chk != MFSDP_OK) return chk;
  if (!aligned_to(loss, 4) || !aligned_to(lse, 4)) return MFSDP_EALIGN;
  HeadCall c{};
  c.s = head_shape(n_tokens, dim, vocab, dtype, false, weight, ld_weight, 0, kLayoutSms);
  c.l = head_layout(c.s);
  if (workspace_bytes < c.l.total) return MFSDP_EWORKSPACE;
  if (n_tokens == 0) return MFSDP_OK;
  const int dst = device_sms(&c.sms);
  if (dst != MFSDP_OK) return dst;
  c.status = device_status();
  if (!c.status) return MFSDP_ECUDA;
  c.ws = static_cast<char*>(workspace);
  c.hidden = hidden;
  c.weight = weight;
  c.labels = labels;
  c.ld_h = ld_hidden;
  c.ld_w = ld_weight;
  c.ignore = ignore_index;
  c.index_dtype = index_dtype;
  c.loss = loss;
  c.lse = lse;
  c.st = static_cast<cudaStream_t>(stream);
  return c.run();
}

extern "C" int mfsdp_head_loss_backward(int64_t n_tokens, int64_t dim, int64_t vocab,
                                        int32_t dtype, const void* hidden, int64_t ld_hidden,
                                        const void* weight, int64_t ld_weight,
                                        int32_t index_dtype, const void* labels,
                                        int64_t ignore_index, const float* lse,
                                        const float* dloss, int64_t piece, void* dhidden,
                                        int64_t ld_dhidden, void* dweight, int64_t ld_dweight,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  int chk = check_head(n_tokens, dim, vocab, dtype, ld_weight, piece);
  if (chk == MFSDP_OK)
    chk = check_common(n_tokens, dim, dtype, hidden, ld_hidden, weight, index_dtype, labels, workspace);
  if (chk != MFSDP_OK) return chk;
  if (n_tokens > 0 && (!lse || !dloss)) return MFSDP_EINVAL;
  if ((dhidden && ld_dhidden < dim) || (dweight && ld_dweight < dim)) return MFSDP_EINVAL;
  if (ld_dweight >= (1ll << 31)) return MFSDP_ESHAPE;
  const size_t es = dtype_bytes(dtype);
  if (!aligned_to(lse, 4) || !aligned_to(dloss, 4) || !aligned_to(dhidden, es) ||
      !aligned_to(dweight, es))
    return MFSDP_EALIGN;
  HeadCall c{};
  c.s = head_shape(n_tokens, dim, vocab, dtype, true, weight, ld_weight, piece, kLayoutSms);
  c.l = head_layout(c.s);
  if (workspace_bytes < c.l.total) return MFSDP_EWORKSPACE;
  if (!dhidden && !dweight) return MFSDP_OK;
  const int dst = device_sms(&c.sms);
  if (dst != MFSDP_OK) return dst;
  c.status = device_status();
  if (!c.status) return MFSDP_ECUDA;
  c.st = static_cast<cudaStream_t>(stream);
  if (n_tokens == 0) {   // no tokens: the weight's gradient is zero
    if (!dweight) return MFSDP_OK;
    return cudaMemset2DAsync(dweight, (size_t)ld_dweight * es, 0, (size_t)dim * es, (size_t)vocab,
                             c.st) == cudaSuccess
               ? MFSDP_OK
               : MFSDP_ECUDA;
  }
  c.ws = static_cast<char*>(workspace);
  c.hidden = hidden;
  c.weight = weight;
  c.labels = labels;
  c.ld_h = ld_hidden;
  c.ld_w = ld_weight;
  c.ignore = ignore_index;
  c.index_dtype = index_dtype;
  c.lse_in = lse;
  c.dloss = dloss;
  c.dh = dhidden;
  c.ld_dh = ld_dhidden;
  c.dw = dweight;
  c.ld_dw = ld_dweight;
  return c.run();
}
