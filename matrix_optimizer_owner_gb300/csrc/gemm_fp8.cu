// Products of 8-bit matrices with a power-of-two scale per 128 of the contraction:
//     C = op(A) op(B),  C_mn = sum_b 2^(sa_mb + sb_nb) sum_{k in block b} qa_mk qb_kn   (fp32 sums)
// on the tensor cores' block-scaled form (tcgen05.mma kind::mxf8f6f4): the products of a block are
// scaled while they are added up, so a tile's accumulator stays in tensor memory and nothing is read
// back between blocks (only every 8192 of k for sums kept in fp32: see most_blocks).  That form wants a
// scale byte per row and 32 of k; a byte serves the four instructions of a block of 128, and the four
// bytes of a 32-bit word four blocks, picked by the instruction's scale id.
//
// Large products are bound by the tensor cores, and where they run back to back by the power limit
// (8192 x 14336 x 4096: 296 us, 3250 TFLOP/s, in a short burst; 342 us in a row); short contractions with a large
// result by writing it (16384 x 2304 x 768: 30 us at 2070 MHz, 35 to 38 at the 1.6 GHz that large products in a
// row leave; 8192 x 4096 x 128: 18 us, 3.8 TB/s); few rows by
// reading the wide operand once (1 x 14336 x 4096: 13 us, 4.5 TB/s); small ones by the latency of their
// steps (333 x 1500 x 1001: 8.7 us).
//
// An operand whose contraction runs down its columns (both of the weight's gradient, the weight of
// the input's gradient) is read as it lies: the tensor cores take it MN-major, no copy is transposed.
#include <algorithm>
#include <atomic>

#include "fp8.cuh"
#include "umma.cuh"

namespace mfsdp {

namespace {

constexpr int kB8 = 128;                    // k of a pipeline stage and of a scale
constexpr uint32_t kBox8 = 128 * 128;       // one operand box: 128 rows of 128 bytes

// ---------------------------------------------------------------- operands
// K-major: rows of 128 k-bytes, eight-row swizzle atoms 1024 bytes apart, the k-step j of 32 starts
// 32 bytes further.  MN-major: 128 output indices a row, one k a row; the k-step j starts 32 rows
// further.
__device__ __forceinline__ uint64_t operand_desc8(uint32_t base, int mn_major, int j) {
  return mn_major ? smem_desc(base + (uint32_t)j * 4096u, kBox8, 1024u)
                  : smem_desc(base + (uint32_t)j * 32u, 16u, 1024u);
}
// The same with the low word's changing part apart: `at` is a stage's offset, in 16 bytes.
struct Desc8 {
  uint32_t lo, hi, step;
  __device__ __forceinline__ Desc8(uint32_t base, int mn_major) {
    const uint64_t d = operand_desc8(base, mn_major, 0);
    lo = (uint32_t)d;
    hi = (uint32_t)(d >> 32);
    step = mn_major ? 4096u >> 4 : 32u >> 4;
  }
  __device__ __forceinline__ uint64_t at(uint32_t off, int j) const {
    return ((uint64_t)hi << 32) | (lo + off + (uint32_t)j * step);
  }
};
// Scale words: 32 rows of 16 bytes, unswizzled (eight rows 128 bytes apart from the next eight).
__device__ __forceinline__ uint64_t scale_desc(uint32_t base) {
  return (uint64_t)((base >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 32) | (1ull << 46);
}
// Instruction descriptor, kind::mxf8f6f4: B's scale id (bits 4-5), the types of A (7-9) and B (10-12;
// e4m3 0, e5m2 1), A / B MN-major (15 / 16), N >> 3 (17-22), e8m0 scales (23), M >> 4 (24-28), A's
// scale id (29-30).
__host__ __device__ constexpr uint32_t idesc8(int a_e5m2, int b_e5m2, int a_mn, int b_mn, int m,
                                              int n) {
  return ((uint32_t)a_e5m2 << 7) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) |
         ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_scale_id(uint32_t idesc, int id) {
  return idesc | ((uint32_t)id << 4) | ((uint32_t)id << 29);
}

template <int CTAS>
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                     uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (CTAS == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 512 bytes of scale words into four columns, the same for all four lane quarters.
template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if (CTAS == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
}
// Arrival on the pair leader's barrier that publishes this CTA's shared memory to the leader's
// thread (which hands it to the tensor cores).
__device__ __forceinline__ void mbar_arrive_leader(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------- scales
enum ScaleForm : int32_t { kBytes = 0, kRowWords = 1, kColWords = 2 };
struct ScaleArgs {
  const uint8_t* s;
  int64_t sr, sk;             // bytes between rows' groups and between blocks of k
  int32_t shift;              // 7: a scale serves 128 rows
  int32_t form;               // kRowWords: four blocks' bytes lie in an aligned word;
                              // kColWords: four rows' do
  int32_t pairs;              // kRowWords: eight blocks' bytes in two aligned words
};

// The scale words of 128 rows from row0 (a multiple of 128) and blocks kb .. kb + 3: word j of lane l
// is that of row row0 + 32 j + l, or with kColWords of row0 + 4 l + j.  Past the end, where the
// operand is zero, scales are 1.  In two steps, the loads and what is made of them, so that a warp has
// all loads of a group under way before it waits for one (addresses are clamped rather than guarded):
// with a wait after each of a group's three loads, the scales took 3400 cycles per four blocks, whose
// products take 2048.
struct ScaleAt {
  int64_t row0;
  int kb, live;               // live: blocks, 1 to 4
  int how;                    // 0 words of four rows, 1 one row group's bytes, 2 words of four blocks,
                              // 3 bytes, 4 one row group's word
  __device__ __forceinline__ ScaleAt(const ScaleArgs& p, int64_t row0_, int64_t rows, int kb_, int nkb)
      : row0(row0_), kb(kb_), live(min(4, nkb - kb_)) {
    how = p.form == kColWords && live == 4 && row0 + 128 <= rows ? 0
          : p.shift ? (p.form == kRowWords && (kb & 3) == 0 && live == 4 ? 4 : 1)
          : p.form == kRowWords && (kb & 3) == 0 && live == 4    ? 2
                                                                 : 3;
  }
};
struct ScaleRaw {
  uint32_t r[16];
};
__device__ __forceinline__ void issue_scales(const ScaleArgs& p, const ScaleAt& at, int64_t rows,
                                             int lane, ScaleRaw& raw) {
  if (at.how == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      raw.r[j] = *reinterpret_cast<const uint32_t*>(p.s + at.row0 + 4 * lane +
                                                    (int64_t)(at.kb + j) * p.sk);
  } else if (at.how == 1 || at.how == 4) {               // the same for all 128 rows
    const uint8_t* s = p.s + (min(at.row0, rows - 1) >> 7) * p.sr + (int64_t)at.kb * p.sk;
    if (at.how == 4) {
      raw.r[0] = *reinterpret_cast<const uint32_t*>(s);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        raw.r[j] = *s;
        s += j + 1 < at.live ? p.sk : 0;
      }
    }
  } else {
    const uint8_t* base = p.s + (int64_t)at.kb * p.sk;
    const int64_t d1 = at.live > 1 ? p.sk : 0, d2 = at.live > 2 ? d1 + p.sk : d1,
                  d3 = at.live > 3 ? d2 + p.sk : d2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = at.row0 + (p.form == kColWords ? 4 * lane + j : 32 * j + lane);
      const uint8_t* s = base + min(r, rows - 1) * p.sr;
      if (at.how == 2) {
        raw.r[j] = *reinterpret_cast<const uint32_t*>(s);
      } else {
        raw.r[4 * j] = s[0];
        raw.r[4 * j + 1] = s[d1];
        raw.r[4 * j + 2] = s[d2];
        raw.r[4 * j + 3] = s[d3];
      }
    }
  }
}
__device__ __forceinline__ void finish_scales(const ScaleAt& at, const ScaleRaw& raw,
                                              uint32_t (&v)[4]) {
  const uint32_t past = at.live < 4 ? 0x7F7F7F7Fu << (8 * at.live) : 0u;
  const uint32_t keep = at.live < 4 ? (1u << (8 * at.live)) - 1u : 0xFFFFFFFFu;
  const uint32_t(&r)[16] = raw.r;
  if (at.how == 0) {
    // from four rows of a block a word to four blocks of a row a word
    const uint32_t a = __byte_perm(r[0], r[1], 0x5140), b = __byte_perm(r[2], r[3], 0x5140);
    const uint32_t c = __byte_perm(r[0], r[1], 0x7362), d = __byte_perm(r[2], r[3], 0x7362);
    v[0] = __byte_perm(a, b, 0x5410);
    v[1] = __byte_perm(a, b, 0x7632);
    v[2] = __byte_perm(c, d, 0x5410);
    v[3] = __byte_perm(c, d, 0x7632);
  } else if (at.how == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = r[j];
  } else if (at.how == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = r[0];
  } else if (at.how == 1) {
    const uint32_t w = ((r[0] | (r[1] << 8) | (r[2] << 16) | (r[3] << 24)) & keep) | past;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = ((r[4 * j] | (r[4 * j + 1] << 8) | (r[4 * j + 2] << 16) | (r[4 * j + 3] << 24)) & keep) |
             past;
  }
}
// Both groups of a stage's eight blocks in one load a row, where the words allow it.
__device__ __forceinline__ bool issue_scale_pairs(const ScaleArgs& p, int64_t row0, int64_t rows, int kb,
                                                  int nkb, int lane, ScaleRaw& lo, ScaleRaw& hi) {
  if (!p.pairs || (kb & 7) != 0 || kb + 8 > nkb) return false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (p.shift && j > 0) break;
    const int64_t r = min(row0 + 32 * j + lane, rows - 1) >> p.shift;
    const uint2 w = *reinterpret_cast<const uint2*>(p.s + r * p.sr + kb);
    lo.r[j] = w.x;
    hi.r[j] = w.y;
  }
  return true;
}
// ... into their 512 bytes of shared memory: row r at 16 (r % 32) + 4 (r / 32).  Rows past the end
// have another row's scales beside zero values; only a NaN among those must not reach them.
__device__ __forceinline__ void store_scales(const ScaleArgs& p, uint32_t dst, int64_t row0,
                                             int64_t rows, int lane, uint32_t (&v)[4]) {
  const bool cols = p.form == kColWords;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (row0 + (cols ? 4 * lane + j : 32 * j + lane) >= rows) v[j] = 0x7F7F7F7Fu;
  if (!cols) {
    sts128(dst + (uint32_t)lane * 16u, make_uint4(v[0], v[1], v[2], v[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t r = 4u * (uint32_t)lane + (uint32_t)j;
      sts32(dst + (r & 31u) * 16u + (r >> 5) * 4u, v[j]);
    }
  }
}

struct Gemm8Args {
  CUtensorMap a, b, cm;       // cm: C in blocks of 32 rows of 64 bytes (PLAIN)
  ScaleArgs sa, sb;
  int32_t m, n, nkb;          // C's sizes and the blocks of k
  int32_t a_mn, b_mn;
  uint32_t idesc;
  int32_t tiles_m, tiles_n;
  int32_t splits, kb_split;   // narrow kernel: slices of k
  void* c;
  int64_t ld_c;
  int32_t c_bf16, accumulate;
  int32_t vec;                // C's rows start on 16-byte boundaries (narrow kernel: on those of four entries)
  int64_t sw, st;             // narrow kernel: C's strides along the wide and the narrow side
  uint64_t wait_limit_ns;
  int* status;
};

// ---------------------------------------------------------------- 256 x 256 tiles
// A pair of CTAs shares a tile, 128 of its rows each, and each half of B's 256 columns: 64 KB of operands
// and 2048 cycles of tensor cores per four blocks.  The grid is persistent: the copies and the scales of
// the next tile run ahead while the epilogue writes this one.
constexpr int kPairThreads = 384;           // warp 0 TMA, 1 MMA, 2-3 scales, 4-11 epilogue
constexpr int kEpi0 = 4, kEpiN = 8;
constexpr int kStages8 = 6;
constexpr uint32_t kStageBytes8 = 2 * kBox8;
constexpr int kSfStages = 4;
constexpr uint32_t kSfBytes = 2 * 3 * 512;  // eight blocks of A's 128 rows and B's 256
constexpr uint32_t kStg8 = kStages8 * kStageBytes8;
constexpr uint32_t kSf8 = kStg8 + kEpiN * 2048;
constexpr uint32_t kBars8 = kSf8 + kSfStages * kSfBytes;
constexpr uint32_t kPairSmem = 1024 + kBars8 + 512;
static_assert(kPairSmem <= 227 * 1024, "shared memory");
// Tensor memory: two accumulators of 256 columns and the scales do not fit 512 columns, so the
// accumulators share the 32 columns 224-255 (the last of the first one, the first of the second).
// The epilogue reads the shared columns of a tile first and says so, and the next tile's products
// wait for that alone.
constexpr uint32_t kAcc1 = 224, kSfCol = 480;
constexpr int kChunk8 = 64;                 // blocks added up in tensor memory (CHUNKED): 8192 of k
constexpr int kRasterRows = 8;              // tile rows that walk the columns together

struct PairTile {
  int tm, tn;
};
__device__ __forceinline__ PairTile pair_tile(const Gemm8Args& P, int i) {
  const int per = kRasterRows * P.tiles_n, group = i / per;
  const int rows = min(kRasterRows, P.tiles_m - group * kRasterRows);
  const int j = i - group * per;
  return PairTile{group * kRasterRows + j % rows, j / rows};
}

// Adds a staging block to C in memory (fp32, to nearest): one addition per element and call, so there is
// no order to depend on.
__device__ __forceinline__ void tma_add_block(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}

// What C held, for this lane's row and 32 columns (added before the rounding).
__device__ __forceinline__ void add_old(const Gemm8Args& P, int64_t r, int64_t c0, float (&v)[32]) {
  if (r >= P.m) return;
  if (P.vec && c0 + 32 <= P.n) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float o[8];
      if (P.c_bf16) {
        Pack8<bf16_t> q;
        q.load(static_cast<const bf16_t*>(P.c) + r * P.ld_c + c0 + 8 * k);
        q.get(o);
      } else {
        Pack8<float> q;
        q.load(static_cast<const float*>(P.c) + r * P.ld_c + c0 + 8 * k);
        q.get(o);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * k + j] += o[j];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (c0 + k < P.n)
        v[k] += P.c_bf16 ? to_f32(static_cast<const bf16_t*>(P.c)[r * P.ld_c + c0 + k])
                         : static_cast<const float*>(P.c)[r * P.ld_c + c0 + k];
  }
}

// 32 columns of a lane's row to C, whatever C's rows, edges and old values are.  Rows without 16-byte
// alignment go through the warp's staging area (2 KB), a row of the block at a time.  What bf16 C held is
// read here, by each lane from its own row, and waited for (16384 x 768 x 2304: 29 us overwritten, 52 added to;
// 4096 x 4096 x 4096: 52 and 60).
template <bool BF16>
__device__ __forceinline__ void put_row(const Gemm8Args& P, int64_t rw, int lane, int64_t c0,
                                        uint32_t stg, float (&v)[32]) {
  const int64_t r = rw + lane;
  constexpr bool f32 = !BF16;
  if (P.accumulate) add_old(P, r, c0, v);
  if (P.vec) {
    if (r >= P.m) return;
    if (!f32) {
      uint32_t w[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
      bf16_t* d = static_cast<bf16_t*>(P.c) + r * P.ld_c + c0;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (c0 + 8 * h + 8 <= P.n) {
          reinterpret_cast<uint4*>(d)[h] =
              make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
        } else {
#pragma unroll
          for (int k = 8 * h; k < 8 * h + 8; ++k)
            if (c0 + k < P.n)
              reinterpret_cast<uint16_t*>(d)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
      }
    } else {
      float* d = static_cast<float*>(P.c) + r * P.ld_c + c0;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (c0 + 8 * h + 8 <= P.n) {
          reinterpret_cast<float4*>(d)[2 * h] =
              make_float4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
          reinterpret_cast<float4*>(d)[2 * h + 1] =
              make_float4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
        } else {
#pragma unroll
          for (int k = 8 * h; k < 8 * h + 8; ++k)
            if (c0 + k < P.n) d[k] = v[k];
        }
      }
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {             // 32 columns of bf16, or 16 of fp32 at a time
    if (!f32 && h == 1) break;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = f32 ? __float_as_uint(v[16 * h + 4 * k + i])
                   : pack_bf16x2(v[8 * k + 2 * i], v[8 * k + 2 * i + 1]);
      sts128(stg + stg_off(lane, k), make_uint4(w[0], w[1], w[2], w[3]));
    }
    __syncwarp();
    // a row of bf16, or two of fp32, at a time
    const int col = f32 ? lane & 15 : lane, row0 = f32 ? lane >> 4 : 0, step = f32 ? 2 : 1;
    const int64_t c = c0 + 16 * h + col;
    const int64_t at = (rw + row0) * P.ld_c + c, next = step * P.ld_c;
    const int rows = c < P.n ? (int)min((int64_t)32, P.m - rw) - row0 : 0;
#pragma unroll 8
    for (int i = 0; i < 32; i += step) {
      const int row = i + row0;
      if (f32) {
        const uint32_t w = lds32(stg + stg_off(row, col >> 2) + (uint32_t)(col & 3) * 4u);
        if (i < rows) static_cast<uint32_t*>(P.c)[at + (i >> 1) * next] = w;
      } else {
        const uint32_t w = lds32(stg + stg_off(row, col >> 3) + (uint32_t)((col & 6) * 2));
        if (i < rows)
          static_cast<uint16_t*>(P.c)[at + i * next] = (uint16_t)(w >> (16 * (col & 1)));
      }
    }
  }
}

// The same where rows start and end on 16-byte boundaries and C in bf16 is not added to: the warp's block
// leaves by TMA, which cuts it at C's edges, 64 bytes of each row at a time.  (Stored by the lanes from registers, 32 bytes of
// a row each: 24.8 us for 8192 x 4096 x 128 against 18.1, 3.8 TB/s, with a fill at 4.0; 35 against 30 for
// 16384 x 2304 x 768.  Two staging blocks a warp, for a stage of operands less, changed nothing.)
template <bool BF16>
__device__ __forceinline__ void put_block(const Gemm8Args& P, int64_t rw, int lane, int64_t c0,
                                          uint32_t stg, const float (&v)[32]) {
  constexpr int kCols = BF16 ? 32 : 16;
#pragma unroll
  for (int h = 0; h < 32 / kCols; ++h) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = BF16 ? pack_bf16x2(v[8 * k + 2 * i], v[8 * k + 2 * i + 1])
                    : __float_as_uint(v[(BF16 ? 0 : 16 * h) + 4 * k + i]);
      sts128(stg + stg_off(lane, k), make_uint4(w[0], w[1], w[2], w[3]));
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (c0 + kCols * h < P.n) {
        if (!BF16 && P.accumulate) tma_add_block(&P.cm, stg, (int)c0 + kCols * h, (int)rw);
        else tma_store_block(&P.cm, stg, (int)c0 + kCols * h, (int)rw);
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
}

// CHUNKED: a tile's contraction is cut into chunks that are added up in registers.
// SPLIT: few tiles with a long contraction.  Two pairs (a cluster of four CTAs) take half of k each of one
// tile; then each takes half of the columns and gets the other's sums of them through its shared memory.
// PLAIN: C's rows start and end on 16-byte boundaries and it is overwritten, or in fp32.  The other forms of the epilogue are
// kernels of their own: beside each other in one kernel they cost its common path up to a sixth (the
// warps wait for instructions).
template <bool CHUNKED, bool SPLIT, bool BF16, bool PLAIN>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ Gemm8Args P) {
  constexpr int S = kStages8, F = kSfStages;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBars8);
  // full[S] | empty[S] | sf_full[F] | sf_empty[F] | sf_free[2] | tfull[2] | tempty[2] | early[2] | drain
  constexpr int full0 = 0, empty0 = S, sf_full0 = 2 * S, sf_empty0 = 2 * S + F,
                sf_free0 = 2 * S + 2 * F, tfull0 = sf_free0 + 2, tempty0 = tfull0 + 2,
                early0 = tempty0 + 2, drain = early0 + 2;
  static_assert((drain + 2) * 8 <= 512, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(bars + i); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cta = cluster_rank(), rank = cta & 1u;  // within the pair
  const uint32_t lead = cta & ~1u;                       // the pair's leader
  const uint16_t both = (uint16_t)(0x3u << lead);
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar(full0 + s), 1);
      mbar_init(bar(empty0 + s), 1);
    }
    for (int s = 0; s < F; ++s) {
      mbar_init(bar(sf_full0 + s), 2);
      mbar_init(bar(sf_empty0 + s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar(sf_free0 + a), 1);
      mbar_init(bar(tfull0 + a), 1);
      mbar_init(bar(tempty0 + a), 2 * kEpiN);
      mbar_init(bar(early0 + a), 2 * (kEpiN / 2));
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
  pdl_wait();
  const uint32_t tmem_base = *tmem_slot;
  uint32_t peer_base;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(peer_base)
               : "r"(map_rank(smem_u32(tmem_slot), cta ^ 1u))
               : "memory");
  const bool usable = peer_base == tmem_base;
  if (!usable && threadIdx.x == 0) atomicOr(P.status, kStatusTmemMismatch);
  const Guard g{abort_flag, P.wait_limit_ns, P.status};
  const int pair = SPLIT ? blockIdx.x >> 2 : blockIdx.x >> 1, npairs = SPLIT ? gridDim.x >> 2 : gridDim.x >> 1;
  // this pair's blocks of k
  const int kb0 = SPLIT && lead ? P.kb_split : 0, nkb = SPLIT ? (lead ? P.nkb - kb0 : P.kb_split) : P.nkb;
  const int tiles = P.tiles_m * P.tiles_n;

  if (!usable) {
    // nothing runs: fall through to the teardown
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 1, armed = 0, last_par = 0;
      bool ok = true;
      for (int w = pair; w < tiles && ok; w += npairs) {
        const PairTile t = pair_tile(P, w);
        const int a0 = t.tm * 256 + 128 * (int)rank, b0 = t.tn * 256 + 128 * (int)rank;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(bar(empty0 + stage), ph, g)) { ok = false; break; }
          const uint32_t fb_local = bar(full0 + stage), fb = map_rank(fb_local, lead);
          const uint32_t dst = sbase + (uint32_t)stage * kStageBytes8;
          const int k0 = (kb0 + kb) * kB8;
          expect_tx_p(leader, fb_local, 2u * kStageBytes8);
          tma_load_pair_p(true, dst, &P.a, P.a_mn ? a0 : k0, P.a_mn ? k0 : a0, fb);
          tma_load_pair_p(true, dst + kBox8, &P.b, P.b_mn ? b0 : k0, P.b_mn ? k0 : b0, fb);
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
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    // One thread issues every product of the pair, so what it does between them has to stay below
    // their own time (512 cycles a block): descriptors differ by a sum in their low word, and a
    // group's four blocks are unrolled with their scale ids.
    if (lane == 0 && leader) {
      int stage = 0, sf = 0, acc = 0, buf = 0;
      uint32_t phase = 0, sf_phase = 0, acc_phase = 0, buf_phase = 1;
      bool ok = true, first = true;
      const Desc8 da(sbase, P.a_mn), db(sbase + kBox8, P.b_mn);
      for (int w = pair; w < tiles && ok; w += npairs) {
        const PairTile t = pair_tile(P, w);
        int in_chunk = 0;                                 // blocks in the accumulator
        for (int kb = 0; kb < nkb && ok; kb += 4) {
          if (in_chunk == 0) {
            // the accumulator, and the columns that it shares with the one before
            if (!mbar_wait_cl(bar(tempty0 + acc), acc_phase ^ 1u, g) ||
                (!first &&
                 !mbar_wait_cl(bar(early0 + (acc ^ 1)), acc ? acc_phase : acc_phase ^ 1u, g))) {
              ok = false;
              break;
            }
            first = false;
          }
          // the scales of four blocks, into the columns that the last but one group has left
          const uint32_t sfa = tmem_base + kSfCol + (uint32_t)buf * 16u, sfb = sfa + 4u;
          if (((kb & 4) == 0 && !mbar_wait_cl(bar(sf_full0 + sf), sf_phase, g)) ||
              !mbar_wait(bar(sf_free0 + buf), buf_phase, g)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t src = sbase + kSf8 + (uint32_t)sf * kSfBytes + (kb & 4 ? 1536u : 0u);
          copy_scales<2>(sfa, scale_desc(src));
          copy_scales<2>(sfb, scale_desc(src + 512u));
          copy_scales<2>(sfb + 4u, scale_desc(src + 1024u));
          if ((kb & 4) || kb + 4 >= nkb) {               // the stage's last group
            tc_commit_pair(bar(sf_empty0 + sf), both);
            if (++sf == F) { sf = 0; sf_phase ^= 1u; }
          }
          const uint32_t d = tmem_base + (acc ? kAcc1 : 0u);
          const int live = min(4, nkb - kb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i < live && ok) {
              ok = mbar_wait(bar(full0 + stage), phase, g);
              if (ok) {
                tc_fence_after();
                const uint32_t at = (uint32_t)stage * (kStageBytes8 >> 4);
                const uint32_t idesc = with_scale_id(P.idesc, i);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  mma8<2>(d, da.at(at, j), db.at(at, j), idesc, sfa, sfb, (in_chunk | i | j) != 0);
                tc_commit_pair(bar(empty0 + stage), both);
                if (++stage == S) { stage = 0; phase ^= 1u; }
              }
            }
          }
          if (!ok) break;
          tc_commit_pair(bar(sf_free0 + buf), (uint16_t)(1u << lead));
          buf ^= 1;
          if (buf == 0) buf_phase ^= 1u;
          in_chunk += 4;
          if (kb + 4 >= nkb || (CHUNKED && in_chunk == kChunk8)) {
            tc_commit_pair(bar(tfull0 + acc), both);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
            in_chunk = 0;
          }
        }
      }
      tc_commit_pair(bar(drain), (uint16_t)(1u << lead));
      mbar_wait(bar(drain), 0u, g, false);
    }
  } else if (warp < kEpi0) {
    // ------------------------------------------------------------ scales (both CTAs)
    // A stage holds the scales of eight blocks; the two warps take the stages in turn, each with all
    // of its loads under way before it waits for one.
    int sf = 0, turn = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int w = pair; w < tiles && ok; w += npairs) {
      const PairTile t = pair_tile(P, w);
      const int64_t a0 = (int64_t)t.tm * 256 + 128 * rank, b0 = (int64_t)t.tn * 256;
      for (int kb = 0; kb < nkb; kb += 8) {
        if (turn == warp - 2) {
          ScaleRaw raw[2][3];
          auto each = [&](auto&& f) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (kb + 4 * h >= nkb) break;
              const int k0 = kb0 + kb + 4 * h;
              f(P.sa, ScaleAt(P.sa, a0, P.m, k0, P.nkb), P.m, h, 0);
              f(P.sb, ScaleAt(P.sb, b0, P.n, k0, P.nkb), P.n, h, 1);
              f(P.sb, ScaleAt(P.sb, b0 + 128, P.n, k0, P.nkb), P.n, h, 2);
            }
          };
          const bool pa = issue_scale_pairs(P.sa, a0, P.m, kb0 + kb, P.nkb, lane, raw[0][0], raw[1][0]);
          const bool pb = issue_scale_pairs(P.sb, b0, P.n, kb0 + kb, P.nkb, lane, raw[0][1], raw[1][1]) &&
                          issue_scale_pairs(P.sb, b0 + 128, P.n, kb0 + kb, P.nkb, lane, raw[0][2], raw[1][2]);
          each([&](const ScaleArgs& p, const ScaleAt& at, int64_t rows, int h, int i) {
            if (!(i == 0 ? pa : pb)) issue_scales(p, at, rows, lane, raw[h][i]);
          });
          ok = mbar_wait(bar(sf_empty0 + sf), ph, g);
          if (!ok) break;
          const uint32_t dst = sbase + kSf8 + (uint32_t)sf * kSfBytes;
          each([&](const ScaleArgs& p, const ScaleAt& at, int64_t rows, int h, int i) {
            uint32_t v[4];
            finish_scales(at, raw[h][i], v);
            store_scales(p, dst + 1536u * h + 512u * i, at.row0, rows, lane, v);
          });
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_leader(map_rank(bar(sf_full0 + sf), lead));
        }
        turn ^= 1;
        if (++sf == F) { sf = 0; ph ^= 1u; }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // Warp w covers TMEM lane quarter (w & 3), 32 rows of the CTA's 128, and 128 columns.
    const int quarter = warp & 3, half = (warp - kEpi0) >> 2;
    const uint32_t stg = sbase + kStg8 + (uint32_t)(warp - kEpi0) * 2048u;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int w = pair; w < tiles && ok; w += npairs) {
      const PairTile t = pair_tile(P, w);
      const int64_t rw = (int64_t)t.tm * 256 + 128 * rank + quarter * 32;
      const int64_t cb = (int64_t)t.tn * 256 + half * 128;
      const int nq = rw < P.m && cb < P.n ? (int)min((int64_t)4, (P.n - cb + 31) / 32) : 0;
      auto put = [&](int q, float (&v)[32]) {
        if (PLAIN) put_block<BF16>(P, rw, lane, cb + 32 * q, stg, v);
        else put_row<BF16>(P, rw, lane, cb + 32 * q, stg, v);
      };
      // the shared columns: this warp's chunk `sh` of this accumulator, if it holds them
      auto shared_chunk = [&]() { return acc == 0 ? (half == 1 ? 3 : -1) : (half == 0 ? 0 : -1); };
      auto base = [&]() {
        return tmem_base + ((uint32_t)(quarter * 32) << 16) + (acc ? kAcc1 : 0u) +
               (uint32_t)(half * 128);
      };
      auto release = [&](int which) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(bar(which + acc), lead));
      };
      if (CHUNKED) {
        float sum[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int k = 0; k < 32; ++k) sum[q][k] = 0.f;
        for (int left = nkb; left > 0; left -= kChunk8) {
          if (!mbar_wait(bar(tfull0 + acc), acc_phase, g)) { ok = false; break; }
          tc_fence_after();
          const int sh = shared_chunk();
          auto add = [&](int q) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t r[16];
              asm volatile(
                  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
                  "%10, %11, %12, %13, %14, %15}, [%16];\ntcgen05.wait::ld.sync.aligned;\n"
                  : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                    "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                    "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                  : "r"(base() + (uint32_t)(32 * q + 16 * h))
                  : "memory");
#pragma unroll
              for (int k = 0; k < 16; ++k) sum[q][16 * h + k] += __uint_as_float(r[k]);
            }
          };
          if (sh == 3) {                                  // warp-uniform
            add(3);
            release(early0);
            add(0);
          } else {
            add(0);
            if (sh == 0) release(early0);
          }
          add(1);
          add(2);
          if (sh != 3) add(3);
          release(tempty0);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < nq) put(q, sum[q]);
      } else if (SPLIT) {
        mbar_wait(bar(tfull0), 0u, g);                    // (the sums are read below)
        tc_fence_after();
      } else {
        if (!mbar_wait(bar(tfull0 + acc), acc_phase, g)) break;
        tc_fence_after();
        const int sh = shared_chunk(), first = sh == 3 ? 3 : 0;   // the shared columns first
        const uint32_t at = base();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int q = (i + first) & 3;
          uint32_t a[32];
          tc_ld32_issue(at + (uint32_t)(32 * q), a);
          tc_ld_wait(a);
          if (q == sh) release(early0);
          if (i == 3) release(tempty0);                   // the last read: the stores can follow it
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(a[k]);
          if (q < nq) put(q, v);
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
  }

  if (SPLIT) {
    // Both pairs' products are done, and with them every copy into the stages, which take the other
    // pair's sums: a warp's 32 columns as eight rows of 512 bytes.  Half 0 of the columns is the first
    // pair's, half 1 the second's.
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    const int quarter = warp & 3, first = ((warp - kEpi0) >> 2) * 2;   // two chunks of a half each
    const int own = (int)(lead >> 1);
    const PairTile t = pair_tile(P, pair);
    const int64_t rw = (int64_t)t.tm * 256 + 128 * rank + quarter * 32;
    const int64_t cb = (int64_t)t.tn * 256 + own * 128;
    const uint32_t at = tmem_base + ((uint32_t)(quarter * 32) << 16);
    auto place = [&](int q, int i) {
      return (uint32_t)(((quarter * 4 + q) * 8 + i) * 512 + lane * 16);
    };
    if (usable && warp >= kEpi0) {
#pragma unroll 1
      for (int q = first; q < first + 2; ++q) {
        uint32_t a[32];
        tc_ld32_issue(at + (uint32_t)((own ^ 1) * 128 + 32 * q), a);
        tc_ld_wait(a);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           map_rank(sbase + place(q, i), cta ^ 2u)),
                       "r"(a[4 * i]), "r"(a[4 * i + 1]), "r"(a[4 * i + 2]), "r"(a[4 * i + 3])
                       : "memory");
      }
    }
    __syncwarp();
    cluster_sync_all();
    if (usable && warp >= kEpi0 && rw < P.m) {
      const uint32_t stg = sbase + kStg8 + (uint32_t)(warp - kEpi0) * 2048u;
#pragma unroll 1
      for (int q = first; q < first + 2; ++q) {
        const int64_t c0 = cb + 32 * q;
        if (c0 >= P.n) break;                             // warp-uniform
        uint32_t a[32];
        tc_ld32_issue(at + (uint32_t)(own * 128 + 32 * q), a);
        tc_ld_wait(a);
        float v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 o = lds128(sbase + place(q, i));
          v[4 * i] = __uint_as_float(a[4 * i]) + __uint_as_float(o.x);   // (a sum of two: any order)
          v[4 * i + 1] = __uint_as_float(a[4 * i + 1]) + __uint_as_float(o.y);
          v[4 * i + 2] = __uint_as_float(a[4 * i + 2]) + __uint_as_float(o.z);
          v[4 * i + 3] = __uint_as_float(a[4 * i + 3]) + __uint_as_float(o.w);
        }
        if (PLAIN) put_block<BF16>(P, rw, lane, c0, stg, v);
        else put_row<BF16>(P, rw, lane, c0, stg, v);
      }
    }
  }

  if (PLAIN) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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

// An empty contraction.
struct ZeroArgs8 {
  void* c;
  int64_t m, n, ld_c;
  int32_t c_bf16;
};
__global__ void __launch_bounds__(256) gemm_fp8_zero_kernel(const __grid_constant__ ZeroArgs8 p) {
  pdl_launch();
  pdl_wait();
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < p.m * p.n; e += (int64_t)gridDim.x * 256) {
    const int64_t at = e / p.n * p.ld_c + e % p.n;
    if (p.c_bf16) static_cast<bf16_t*>(p.c)[at] = from_f32<bf16_t>(0.f);
    else static_cast<float*>(p.c)[at] = 0.f;
  }
}

// ---------------------------------------------------------------- few rows or columns
// The narrow side has up to NT indices.  A CTA takes 128 indices of the wide side (the tensor cores'
// M) and a slice of k; the CTAs of a cluster hold the slices of one tile, and each adds a part of the
// tile over the slices, in order, out of the others' shared memory.  Bound by reading the wide
// operand once: an SM draws some 43 GB/s, and the tiles do not divide among 152 of them (1 x 14336 x 4096:
// 13.0 us, 4.5 TB/s; 1 x 28672 x 8192: 39 us, 6.0 TB/s).  With NT = 128 also small products of any shape,
// which tiles of 256 would leave most SMs idle for.
constexpr int kNarrowThreads = 192;         // warp 0 TMA, 1 MMA, 2 scales, 2-5 epilogue
constexpr int kNarrowSf = 2;
template <int NT>
struct Narrow {
  static constexpr uint32_t kStage = kBox8 + NT * 128u;
  static constexpr int kStages = NT <= 32 ? 5 : NT == 64 ? 4 : 3;
  static constexpr uint32_t kSf = kStages * kStage;
  static constexpr uint32_t kBars = kSf + kNarrowSf * 1024u;
  static constexpr uint32_t kSmem = 1024 + kBars + 256;
  static constexpr uint32_t kCols = NT == 16 ? 32 : NT == 32 ? 64 : NT == 64 ? 128 : 256;
  static_assert(128 * NT * 4 <= kStages * kStage, "the partial sums lie in the stages");
};

template <int NT>
__global__ void __launch_bounds__(kNarrowThreads, 2)
    gemm_fp8_narrow_kernel(const __grid_constant__ Gemm8Args P) {
  using C = Narrow<NT>;
  constexpr int S = C::kStages, F = kNarrowSf;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  constexpr int full0 = 0, empty0 = S, sf_full0 = 2 * S, sf_empty0 = 2 * S + F,
                sf_free0 = 2 * S + 2 * F, done = sf_free0 + 2;
  static_assert((done + 2) * 8 <= 256, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar(full0 + s), 1);
      mbar_init(bar(empty0 + s), 1);
    }
    for (int s = 0; s < F; ++s) {
      mbar_init(bar(sf_full0 + s), 1);
      mbar_init(bar(sf_empty0 + s), 1);
      mbar_init(bar(sf_free0 + s), 1);
    }
    mbar_init(bar(done), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem_base = *tmem_slot;
  const Guard g{abort_flag, P.wait_limit_ns, P.status};
  // the grid's x is (tile, slice) with the slice fastest: a cluster is one tile
  const int split = (int)(blockIdx.x % (unsigned)P.splits);
  const int tile = (int)(blockIdx.x / (unsigned)P.splits);
  const int w0 = tile / P.tiles_n * 128, t0 = tile % P.tiles_n * NT;
  const int kb0 = min(split * P.kb_split, P.nkb), nk = min(P.kb_split, P.nkb - kb0);

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 1, armed = 0, last_par = 0;
      for (int kb = kb0; kb < kb0 + nk; ++kb) {
        if (!mbar_wait(bar(empty0 + stage), ph, g)) break;
        const uint32_t fb = bar(full0 + stage), dst = sbase + (uint32_t)stage * C::kStage;
        const int k0 = kb * kB8;
        expect_tx_p(true, fb, C::kStage);
        tma_load_p(true, dst, &P.a, P.a_mn ? w0 : k0, P.a_mn ? k0 : w0, fb);
        tma_load_p(true, dst + kBox8, &P.b, P.b_mn ? t0 : k0, P.b_mn ? k0 : t0, fb);
        armed |= 1u << stage;
        last_par = (last_par & ~(1u << stage)) | ((ph ^ 1u) << stage);
        if (++stage == S) { stage = 0; ph ^= 1u; }
      }
      for (int st = 0; st < S; ++st)
        if (armed & (1u << st)) mbar_wait(bar(full0 + st), (last_par >> st) & 1u, g, false);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0, sf = 0, buf = 0;
      uint32_t phase = 0, sf_phase = 0, buf_phase = 1;
      for (int kb = 0; kb < nk; ++kb) {
        const uint32_t sfa = tmem_base + NT + (uint32_t)buf * 8u, sfb = sfa + 4u;
        if ((kb & 3) == 0) {
          if (!mbar_wait(bar(sf_full0 + sf), sf_phase, g) ||
              !mbar_wait(bar(sf_free0 + buf), buf_phase, g))
            break;
          tc_fence_after();
          const uint32_t src = sbase + C::kSf + (uint32_t)sf * 1024u;
          copy_scales<1>(sfa, scale_desc(src));
          copy_scales<1>(sfb, scale_desc(src + 512u));
          tc_commit(bar(sf_empty0 + sf));
          if (++sf == F) { sf = 0; sf_phase ^= 1u; }
        }
        if (!mbar_wait(bar(full0 + stage), phase, g)) break;
        tc_fence_after();
        const uint32_t sm_a = sbase + (uint32_t)stage * C::kStage;
        const uint32_t idesc = with_scale_id(P.idesc, kb & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma8<1>(tmem_base, operand_desc8(sm_a, P.a_mn, j), operand_desc8(sm_a + kBox8, P.b_mn, j),
                  idesc, sfa, sfb, (kb | j) != 0);
        tc_commit(bar(empty0 + stage));
        if (++stage == S) { stage = 0; phase ^= 1u; }
        if ((kb & 3) == 3) {
          tc_commit(bar(sf_free0 + buf));
          buf ^= 1;
          if (buf == 0) buf_phase ^= 1u;
        }
      }
      tc_commit(bar(done));
      mbar_wait(bar(done), 0u, g, false);
    }
  } else if (warp == 2) {
    int sf = 0;
    uint32_t ph = 1;
    for (int kb = 0; kb < nk; kb += 4) {
      uint32_t va[4], vb[4];
      const ScaleAt a(P.sa, w0, P.m, kb0 + kb, P.nkb), b(P.sb, t0, P.n, kb0 + kb, P.nkb);
      ScaleRaw ra, rb;
      issue_scales(P.sa, a, P.m, lane, ra);
      issue_scales(P.sb, b, P.n, lane, rb);
      finish_scales(a, ra, va);
      finish_scales(b, rb, vb);
      if (!mbar_wait(bar(sf_empty0 + sf), ph, g)) break;
      const uint32_t dst = sbase + C::kSf + (uint32_t)sf * 1024u;
      store_scales(P.sa, dst, w0, P.m, lane, va);
      store_scales(P.sb, dst + 512u, t0, P.n, lane, vb);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sf_full0 + sf));
      if (++sf == F) { sf = 0; ph ^= 1u; }
    }
  }
  __syncwarp();
  // The products are done (the MMA thread has waited for them), and with them every copy into the
  // stages, whose memory takes the sums now.
  __syncthreads();
  tc_fence_after();
  float* sums = reinterpret_cast<float*>(smem);           // [NT][128]
  if (warp >= 2) {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t ta = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll
    for (int q = 0; q < NT / 16; ++q) {
      uint32_t r[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
          "%10, %11, %12, %13, %14, %15}, [%16];\ntcgen05.wait::ld.sync.aligned;\n"
          : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
            "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
            "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
          : "r"(ta + (uint32_t)(16 * q))
          : "memory");
#pragma unroll
      for (int k = 0; k < 16; ++k)
        sums[(16 * q + k) * 128 + row] = nk > 0 ? __uint_as_float(r[k]) : 0.f;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  {
    // this CTA's share of the tile: narrow indices split, split + splits, ...; a thread adds four
    // consecutive wide indices over the slices, in order, with all loads of two narrow indices under way
    // before it waits for one (one after the other they took 4 us of a small product's 10)
    const int live = min(NT, P.n - t0), wide = min(128, P.m - w0);
    const uint32_t mine = smem_u32(sums);
    const int r = (threadIdx.x & 31) * 4, step = kNarrowThreads / 32 * P.splits;
    auto place = [&](int t) { return (int64_t)(w0 + r) * P.sw + (int64_t)(t0 + t) * P.st; };
    const bool four = P.sw == 1 && P.vec && r + 4 <= wide;
    auto load_old = [&](int t, float (&v)[4]) {
      const int64_t at = place(t);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = 0.f;
      if (four) {
        if (P.c_bf16) {
          const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const bf16_t*>(P.c) + at);
          v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xFFFF0000u);
          v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xFFFF0000u);
        } else {
          const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(P.c) + at);
          v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (r + k >= wide) break;
          v[k] = P.c_bf16 ? to_f32(static_cast<const bf16_t*>(P.c)[at + k * P.sw])
                          : static_cast<const float*>(P.c)[at + k * P.sw];
        }
      }
    };
    auto put = [&](int t, const float (&v)[4]) {
      const int64_t at = place(t);
      if (four) {
        if (P.c_bf16)
          *reinterpret_cast<uint2*>(static_cast<bf16_t*>(P.c) + at) =
              make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(P.c) + at) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (r + k >= wide) break;
          if (P.c_bf16) static_cast<bf16_t*>(P.c)[at + k * P.sw] = from_f32<bf16_t>(v[k]);
          else static_cast<float*>(P.c)[at + k * P.sw] = v[k];
        }
      }
    };
    constexpr int U = 2;                                  // (one: up to 9 % more for tiles of 128)
    if (P.splits == 1 && !P.accumulate) {
      if (r < wide)
#pragma unroll 1
        for (int t = (int)(threadIdx.x >> 5); t < live; t += kNarrowThreads / 32) {
          const float4 o = *reinterpret_cast<const float4*>(sums + t * 128 + r);
          const float v[4] = {o.x, o.y, o.z, o.w};
          put(t, v);
        }
    } else if (r < wide) {
      for (int t = split + (int)(threadIdx.x >> 5) * P.splits; t < live; t += U * step) {
        float o[U][8][4], old[U][4];
        if (P.accumulate)
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (t + u * step < live) load_old(t + u * step, old[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            // (beyond the last slice or index nothing is read)
            asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n"
                         " @p ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n}\n"
                         : "=f"(o[u][i][0]), "=f"(o[u][i][1]), "=f"(o[u][i][2]), "=f"(o[u][i][3])
                         : "r"(map_rank(mine + (uint32_t)((t + u * step) * 128 + r) * 4u,
                                        (uint32_t)min(i, P.splits - 1))),
                           "r"((int)(i < P.splits && t + u * step < live)));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (t + u * step >= live) break;
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = o[u][0][k];
#pragma unroll
            for (int i = 1; i < 8; ++i) v[k] = i < P.splits ? v[k] + o[u][i][k] : v[k];
            v[k] = P.accumulate ? v[k] + old[u][k] : v[k];
          }
          put(t + u * step, v);
        }
      }
    }
  }
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while another may still read its sums
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(C::kCols)
                 : "memory");
  }
}

// ---------------------------------------------------------------- host
constexpr int kPairs = 76;                  // CTA pairs of the device: what the plans count on
// Clusters of so many CTAs, two an SM, that run at a time: sizes that do not divide the SMs of a part of
// the device leave some of them over (1 x 6144 x 4096: 48 clusters of six 12.4 us, of five 7.5).  One cluster
// more is a second round (1 x 16384 of k, 32 and 33 clusters of eight: 10.8 and 13.1 us; 1 x 8192 of k, 96 and 97 of
// three: 15.4 and 19.2; 56 and 57 of five, 46 and 47 of six, 72 and 73 of four alike).
constexpr int kClusters[9] = {0, 304, 152, 96, 72, 56, 46, 32, 32};

struct Gemm8Plan {
  bool narrow = false, swap = false;        // swap: the narrow side is A's
  bool halves = false;                      // two pairs a tile
  int nt = 0;
  int splits = 1, kb_split = 0;
};

// The tensor cores cut each of their additions towards zero, which grows with the contraction: sums that
// are kept in fp32 leave tensor memory every 8192 of k (3e-7 of a Gaussian product's entries, 5e-7 at
// 14336), others where the cuts would come near half a bf16 step.
int most_blocks(bool c_bf16) { return c_bf16 ? 512 : kChunk8; }

// What a call is split into, from its sizes alone.  Times in us, as measured.
Gemm8Plan plan_gemm(int64_t m, int64_t n, int64_t k, bool c_bf16, bool accumulate) {
  Gemm8Plan p;
  const int nkb = (int)((k + kB8 - 1) / kB8);
  const int64_t few = std::min(m, n), wide = std::max(m, n);
  const int least = (nkb + most_blocks(c_bf16) - 1) / most_blocks(c_bf16);   // slices
  if (few <= 64 && least <= 8) {
    p.narrow = true;
    p.swap = m <= n;
    p.nt = few <= 16 ? 16 : few <= 32 ? 32 : 64;
    const int64_t tiles = (wide + 127) / 128;
    // as many slices of k, of two blocks at least, as run at a time: an SM draws some 43 GB/s from
    // memory, whatever it has under way (one, two or three CTAs with 3 to 9 stages each took the same
    // time a block), so what counts is that all of them draw
    int s = 8;
    while (s > 1 && (tiles > kClusters[s] || s > nkb / 2)) --s;
    s = std::max(s, least);
    p.splits = s;
    p.kb_split = (nkb + s - 1) / s;
    return p;
  }
  // 128 x 128 tiles, C's rows the wide side: rounds of two CTAs an SM, up to eight slices of k.  A block of k
  // takes 0.4 us on an SM's only CTA and 0.5 beside another one.  The rest grows with the CTAs: 5.4 us for
  // one and 7 for 256 without slices; 6.8 for 32 and 9.8 for 288 where slices' sums go through distributed
  // shared memory at the same time.  What C holds is read by the CTAs that add it, a few rows at a time.
  const int64_t small = ((m + 127) / 128) * ((n + 127) / 128);
  int ns = 0;
  double narrow = 0.;
  for (int s = std::max(1, least); s <= 8 && s <= std::max(1, nkb); ++s) {
    const int per = (nkb + s - 1) / s;
    const int64_t rounds = (small + kClusters[s] - 1) / kClusters[s];
    const int64_t at_once = std::min<int64_t>(small * s, 4 * kPairs);
    const double rest = s == 1 ? 5.3 + 0.0065 * (double)at_once : 6.2 + 0.0125 * (double)at_once;
    const double old = accumulate ? 10. / s : 0.;
    const double t = (double)rounds * (per * (at_once > 2 * kPairs ? 0.5 : 0.4) + rest + old);
    if (ns == 0 || t < narrow * 0.98) {
      narrow = t;
      ns = s;
    }
  }
  // 256 x 256 tiles on CTA pairs
  const int64_t tiles = ((m + 255) / 256) * ((n + 255) / 256);
  double pair = 7.5 + (double)((tiles + kPairs - 1) / kPairs) * (nkb * 0.3 + 2.);
  // ... or two pairs a tile, where an accumulator takes half of k (longer fp32 sums compare what they run as:
  // 2304 x 768 x 32768 in five slices 69 us, on one pair a tile 98) and the clusters of four, a CTA an SM,
  // run at a time (9216 x 256 x 16384, 36 tiles: 40 us; 37 took 69, without halves 44)
  const int half = ((nkb + 1) / 2 + 7) / 8 * 8;
  if (2 * tiles <= kClusters[4] && nkb >= 16 && half <= most_blocks(c_bf16)) {
    p.kb_split = half;
    const double t = 9. + half * 0.34;
    p.halves = t < pair;
    pair = std::min(pair, t);
  }
  if (ns && narrow < pair) {
    p.halves = false;
    p.narrow = p.swap = true;
    p.nt = 128;
    p.splits = ns;
    p.kb_split = (nkb + ns - 1) / ns;
  }
  return p;
}

int check_sizes(int64_t m, int64_t n, int64_t k) {
  return m < 0 || n < 0 || k < 0 || m >= (1ll << 31) - 512 || n >= (1ll << 31) - 512 ||
                 k >= (1ll << 31) - 512
             ? MFSDP_ESHAPE
             : MFSDP_OK;
}

ScaleArgs scales_of(const mfsdp_fp8_matrix& m, bool along_rows) {
  // along_rows: the contraction runs down the stored rows
  ScaleArgs s{};
  s.s = static_cast<const uint8_t*>(m.scales);
  s.sr = along_rows ? 1 : m.ld_scales;
  s.sk = along_rows ? m.ld_scales : 1;
  s.shift = m.groups == MFSDP_GROUPS_TILE ? 7 : 0;
  if (m.ld_scales % 4 == 0 && aligned_to(m.scales, 4))
    s.form = !along_rows ? kRowWords : s.shift ? kBytes : kColWords;
  s.pairs = s.form == kRowWords && m.ld_scales % 8 == 0 && aligned_to(m.scales, 8);
  return s;
}

template <typename K>
cudaError_t allow_smem(std::atomic<bool>* done, K kernel, uint32_t bytes) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev].load())) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done[dev].store(true);
  return e;
}

cudaError_t launch_clusters(void (*kernel)(const Gemm8Args), unsigned grid, unsigned cluster,
                            unsigned threads, uint32_t smem, cudaStream_t st, const Gemm8Args& a) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool CHUNKED, bool SPLIT, bool PLAIN>
cudaError_t launch_pair(const Gemm8Args& a, int grid, cudaStream_t st) {
  static std::atomic<bool> done[2][64];
  const auto kernel = a.c_bf16 ? gemm_fp8_pair_kernel<CHUNKED, SPLIT, true, PLAIN>
                               : gemm_fp8_pair_kernel<CHUNKED, SPLIT, false, PLAIN>;
  const cudaError_t e = allow_smem(done[a.c_bf16 ? 1 : 0], kernel, kPairSmem);
  return e != cudaSuccess ? e
                          : launch_clusters(kernel, grid, SPLIT ? 4 : 2, kPairThreads, kPairSmem, st, a);
}

template <int NT>
cudaError_t launch_narrow(const Gemm8Args& a, int64_t tiles, cudaStream_t st) {
  static std::atomic<bool> done[64];
  cudaError_t e = allow_smem(done, gemm_fp8_narrow_kernel<NT>, Narrow<NT>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_clusters(gemm_fp8_narrow_kernel<NT>, (unsigned)(tiles * a.splits),
                         (unsigned)a.splits, kNarrowThreads, Narrow<NT>::kSmem, st, a);
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" int mfsdp_gemm_fp8(int64_t m, int64_t n, int64_t k, const mfsdp_fp8_matrix* a,
                              int32_t trans_a, const mfsdp_fp8_matrix* b, int32_t trans_b,
                              int32_t accumulate, int32_t c_dtype, void* c, int64_t ld_c,
                              void* stream) {
  if (!a || !b || !dtype_ok(c_dtype)) return MFSDP_EINVAL;
  int chk = check_sizes(m, n, k);
  if (chk != MFSDP_OK) return chk;
  const bool none = m == 0 || n == 0 || k == 0;           // nothing of A or B is read
  chk = trans_a ? check_fp8(*a, none ? 0 : k, m, -1) : check_fp8(*a, none ? 0 : m, k, -1);
  if (chk == MFSDP_OK)
    chk = trans_b ? check_fp8(*b, none ? 0 : n, k, -1) : check_fp8(*b, none ? 0 : k, n, -1);
  if (chk != MFSDP_OK) return chk;
  // a scale has to be the same for 128 of the contraction
  if (a->groups == (trans_a ? MFSDP_GROUPS_ROW : MFSDP_GROUPS_COL) ||
      b->groups == (trans_b ? MFSDP_GROUPS_COL : MFSDP_GROUPS_ROW))
    return MFSDP_EINVAL;
  if (m == 0 || n == 0) return MFSDP_OK;
  if (!c || ld_c < n) return MFSDP_EINVAL;
  if (!aligned_to(c, dtype_bytes(c_dtype))) return MFSDP_EALIGN;
  const bool c_bf16 = c_dtype == MFSDP_DTYPE_BF16;
  // More of k than eight slices take at fp32's chunks: one such piece after the other, added to C.
  constexpr int64_t piece = 8ll * kChunk8 * kB8;
  if (!c_bf16 && k > piece && plan_gemm(m, n, piece, false, true).narrow) {
    for (int64_t k0 = 0; k0 < k; k0 += piece) {
      mfsdp_fp8_matrix pa = *a, pb = *b;
      auto shift = [&](mfsdp_fp8_matrix& x, bool down) {  // down: the contraction runs down the rows
        x.data = static_cast<uint8_t*>(x.data) + k0 * (down ? x.ld : 1);
        x.scales = static_cast<uint8_t*>(x.scales) + k0 / kB8 * (down ? x.ld_scales : 1);
      };
      shift(pa, trans_a != 0);
      shift(pb, trans_b == 0);
      chk = mfsdp_gemm_fp8(m, n, std::min(piece, k - k0), &pa, trans_a, &pb, trans_b,
                           accumulate || k0 > 0, c_dtype, c, ld_c, stream);
      if (chk != MFSDP_OK) return chk;
    }
    return MFSDP_OK;
  }
  const Gemm8Plan plan = plan_gemm(m, n, k, c_bf16, accumulate != 0);
  if (k == 0 && accumulate) return MFSDP_OK;
  int sms = 0;
  const int dst = device_sms(&sms);
  if (dst != MFSDP_OK) return dst;
  int* status = device_status();
  if (!status) return MFSDP_ECUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (k == 0) {
    const ZeroArgs8 z{c, m, n, ld_c, c_bf16};
    const dim3 grid((unsigned)std::min<int64_t>((m * n + 255) / 256, sms * 16ll));
    return launch_pdl(gemm_fp8_zero_kernel, grid, dim3(256), 0, st, z) == cudaSuccess ? MFSDP_OK
                                                                                      : MFSDP_ECUDA;
  }

  Gemm8Args g{};
  const mfsdp_fp8_matrix *wide = plan.swap ? b : a, *other = plan.swap ? a : b;
  // whether the contraction runs down the stored rows
  const bool a_rows = trans_a != 0, b_rows = trans_b == 0;
  const bool w_rows = plan.swap ? b_rows : a_rows, o_rows = plan.swap ? a_rows : b_rows;
  g.m = (int32_t)(plan.swap ? n : m);
  g.n = (int32_t)(plan.swap ? m : n);
  g.nkb = (int32_t)((k + kB8 - 1) / kB8);
  g.a_mn = w_rows;
  g.b_mn = o_rows;
  const int nt = plan.narrow && o_rows ? 128 : plan.nt;   // MN-major boxes are 128 indices wide
  bool ok = encode_map_u8(&g.a, wide->data, w_rows ? k : g.m, w_rows ? g.m : k, wide->ld, 128u);
  ok = ok && encode_map_u8(&g.b, other->data, o_rows ? k : g.n, o_rows ? g.n : k, other->ld,
                           plan.narrow && !o_rows ? (uint32_t)nt : 128u);
  if (!ok) return MFSDP_ECUDA;
  g.sa = scales_of(*wide, w_rows);
  g.sb = scales_of(*other, o_rows);
  g.idesc = idesc8(wide->dtype == MFSDP_FP8_E5M2, other->dtype == MFSDP_FP8_E5M2, g.a_mn, g.b_mn,
                   plan.narrow ? 128 : 256, plan.narrow ? nt : 256);
  g.splits = plan.splits;
  g.kb_split = plan.kb_split;
  g.c = c;
  g.ld_c = ld_c;
  g.c_bf16 = c_bf16;
  g.accumulate = accumulate != 0;
  // 16-byte accesses of C's rows; the narrow kernel's are of four entries
  g.vec = plan.narrow ? ld_c % 4 == 0 && aligned_to(c, 4 * dtype_bytes(c_dtype))
                      : vector_rows(c, ld_c, c_dtype);
  g.wait_limit_ns = wait_limit_ns();
  g.status = status;
  cudaError_t e;
  if (plan.narrow) {
    g.tiles_m = (g.m + 127) / 128;
    g.tiles_n = (int32_t)((g.n + nt - 1) / nt);
    g.sw = plan.swap ? 1 : ld_c;
    g.st = plan.swap ? ld_c : 1;
    const int64_t tiles = (int64_t)g.tiles_m * g.tiles_n;
    e = nt == 16   ? launch_narrow<16>(g, tiles, st)
        : nt == 32 ? launch_narrow<32>(g, tiles, st)
        : nt == 64 ? launch_narrow<64>(g, tiles, st)
                   : launch_narrow<128>(g, tiles, st);
    return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
  }
  g.tiles_m = (g.m + 255) / 256;
  g.tiles_n = (g.n + 255) / 256;
  const int most = most_blocks(c_bf16);
  const int tiles = g.tiles_m * g.tiles_n;
  const int pairs = std::max(1, std::min(sms / 2, tiles));
  // (A store by TMA writes whole groups of 16 bytes: past the last column, where that is inside one.)
  const bool plain = g.vec && (n * (int64_t)dtype_bytes(c_dtype)) % 16 == 0 && (!g.accumulate || !c_bf16) &&
                     (c_bf16 ? encode_map(&g.cm, c, m, n, ld_c, 32u, 32u, false)
                             : encode_map_f32(&g.cm, static_cast<float*>(c), m, n, ld_c, 32u, 16u));
  if (plan.halves)
    e = plain ? launch_pair<false, true, true>(g, 4 * tiles, st)
              : launch_pair<false, true, false>(g, 4 * tiles, st);
  else if (g.nkb > most)
    e = plain ? launch_pair<true, false, true>(g, 2 * pairs, st)
              : launch_pair<true, false, false>(g, 2 * pairs, st);
  else
    e = plain ? launch_pair<false, false, true>(g, 2 * pairs, st)
              : launch_pair<false, false, false>(g, 2 * pairs, st);
  return e == cudaSuccess ? MFSDP_OK : MFSDP_ECUDA;
}
