// dense_gemm.hpp -- the matrix-product kernel behind the dense operators, for
// gfx950's matrix cores.
//
//   C[m][n] = sum_s sum_k A_s[m][k] B_s[n][k],   s < segs
//
// in 16-bit operands (bf16 or fp16) and fp32 accumulators, with the operators'
// elementwise work done on the accumulators before they are stored (Epi below).
//
// Operand layouts.  Either operand may be stored with the contraction index
// contiguous ("kc": row m holds its k values) or with the output index
// contiguous ("mc": row k holds its m values), so that a projection (kc, kc),
// its input gradient (kc, mc) and its weight gradient (mc, mc) all read the
// tensors as they lie, without transposed copies.  kc tiles are read from LDS
// as 16-byte rows; mc tiles through ds_read_b64_tr_b16, which transposes 4x16
// blocks on the way to the registers.
//
// Segments let one launch sum several products of the same shape: the two
// halves of a gated block's input gradient, the six products of fp32 operands
// split into three bf16 planes, and the three of Newton-Schulz iterates in two
// fp16 planes.
//
// What bounds it (this card): at 8192 x 8192 x 8192 bf16 840 / 808 / 802 us for
// the three layouts, 1309 / 1361 / 1371 TFLOP/s, 52-55% of the nominal peak.
// The matrix cores are busy 68% of the clocks, at 1.9 GHz of the nominal 2.4
// (the card's power); the other clocks go to issuing the loads to LDS, 25 to
// 45 of a wave's clocks each.  Staggering the waves, or their priority, did not
// change it; branching so that waves load in turns cost 18%.  Small products
// are bound by the latency of a tile's trip through LDS (64 x 64: 0.25 us a
// step), and each product pays about 3000 clocks before its first load and
// 2000 (64) to 17000 (256) in its epilogue.
//
// LDS tiles are written by buffer loads straight to LDS (no registers), whose
// range check supplies the zeros beyond the operands' ends: no access leaves
// the operands whatever the sizes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense_epilogue.hpp"
#include "pdr_common.hpp"

namespace pdr {
namespace dense {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) const char lds_char;

constexpr int kBK = 64;  // contraction values per LDS tile (128 bytes of a kc row)
constexpr int kMaxSegs = 12;  // a gated block's input gradient in fp32
constexpr long long kMaxLd = 1 << 22;  // 256 rows' byte offsets stay below 2^31
constexpr uint32_t kOutside = 0x80000000u;  // a byte offset beyond every bound used below

struct GemmArgs {
  const void *a[kMaxSegs];
  const void *b[kMaxSegs];
  int M, N, K;       // K: contraction length of one segment, a multiple of 8 where an operand is kc
  int ka, kb;        // rows that a mc operand has (<= K: the other operand holds zeros there)
  int segs;
  long long lda, ldb;                  // elements between rows, multiples of 8
  long long up_at;                     // dual products: elements from the gate rows to the up rows
  long long batch_a, batch_b;          // elements between the operands of two batches
  int tiles_m, tiles_n, batches;
  int symmetric;                       // kEpiPoly: C is
  int lower;                           // then tiles above the diagonal may be left out, and those
                                       // below it stored on both sides
  int splits;                          // parts that the contraction is cut into
  int steps, steps_more;               // kBK steps of a part; the first steps_more parts take one more
  FastDiv band;                        // by kBand * tiles_n
  float *partial;                      // splits > 1: [split][batch][M][N] fp32
  Epi epi;
};

// c += a b on 16x16 tiles, 32 contraction values.  Written out so that the
// sums stay in accumulation registers: with the builtin, the 256 sums a lane
// holds are moved between register files at every turn of the loop.  The
// instructions on one accumulator are far apart, and settle() stands between
// them and any other use of the accumulators, before and after.
template <int FMT>
__device__ __forceinline__ void mfma(f32x4 &c, s16x8 a, s16x8 b) {
  if constexpr (FMT == kBf16)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
// All but the wave's last LEFT loads to LDS have landed and its LDS reads are
// done; then every wave's.
template <int LEFT>
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// LDS swizzles: 16-byte chunk c of tile row r is stored at chunk c ^ s(r), so
// that the lanes of one read phase fall on different banks (counted: no
// conflicts).  A kc read takes rows 0..15 of one chunk: s = r & 7.  A mc read
// takes 32 bytes of each of 4 rows per 16 lanes: s moves pairs of chunks (of
// the 8 that a row of 64 values has, or within 16).
template <bool MC, int ROWS>
__device__ __forceinline__ int swizzle(int r) {
  return MC ? ((r & 3) << 1) | (ROWS > 64 ? ((r >> 3) & 1) << 3 : 0) : r & 7;
}

// A value that is the same in every lane, told to the compiler.
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return lo | ((uint64_t)hi << 32);
}

// One operand's global-to-LDS copy: ROWS output rows by kBK contraction values
// per tile, NW waves.  It walks the tiles of its segments in order.  Stepping
// from one whole tile to the next is a few scalar instructions (they stand
// between matrix instructions); what is rare, a segment's last and partial
// tile and a change of segment, is worked out in seek().
template <int ROWS, bool MC, int NW, bool DUAL>
struct Loader {
  static constexpr int kBytes = ROWS * kBK * 2;
  static constexpr int kIssues = kBytes / (NW * 1024);
  const void *const *segs;  // where the segments begin,
  long long off;            // and how many bytes further this batch's
  long long ld;
  int row0, rows, K, have;  // first output row, output rows, contraction values, those that a mc operand has
  uint32_t voff[kIssues];
  int chunk_k;              // kc: first contraction value of this lane's chunk
  bool masked;              // chunks past a partial tile's end are turned away in voff
  const char *base;         // this tile's first byte
  uint32_t bytes;           // from there to the operand's end
  uint32_t step, fewer;     // what a whole tile adds to base and takes from bytes
  int seg, kin, plain;      // segment, and tile in it, after the next `plain` - 1 whole tiles
  int more;                 // tiles to come, this one included

  __device__ __forceinline__ void place_lanes(int wave, int lane) {
    masked = false;
#pragma unroll
    for (int i = 0; i < kIssues; ++i) {
      const int blk = i * NW + wave;
      if constexpr (!MC) {
        const int r = blk * 8 + (lane >> 3);
        const int c = (lane & 7) ^ swizzle<false, ROWS>(r);
        chunk_k = c * 8;  // the same for every issue: r % 8 is
        if constexpr (DUAL) {
          // LDS rows 16 j .. 16 j + 7 hold gate columns 8 j .. 8 j + 7, the 8 rows
          // after them the same up columns (a wave loads only one kind)
          const int col = (r >> 4) * 8 + (r & 7);
          voff[i] = row0 + col < rows ? (uint32_t)col * (uint32_t)ld * 2u + c * 16 : kOutside;
        } else {
          voff[i] = (uint32_t)r * (uint32_t)ld * 2u + c * 16;
        }
      } else {
        constexpr int kLanesPerRow = ROWS / 8;
        const int k = blk * (64 / kLanesPerRow) + lane / kLanesPerRow;
        const int c = (lane % kLanesPerRow) ^ swizzle<true, ROWS>(k);
        voff[i] = (uint32_t)k * (uint32_t)ld * 2u + c * 16;
      }
    }
  }
  // Point at tile `kin` of segment `seg`.
  __device__ __forceinline__ void seek(int wave, int lane) {
    const char *first = (const char *)uniform((uint64_t)segs[seg]) + off;
    const int k0 = kin * kBK, whole = K / kBK;
    if (masked) place_lanes(wave, lane);
    plain = kin < whole ? whole - kin : 1;
    if (plain > more) plain = more;
    long long left;
    if constexpr (!MC) {
      base = first + ((long long)row0 * ld + k0) * 2;
      const int r = rows - row0 < ROWS ? rows - row0 : ROWS;
      left = ((long long)(r - 1) * ld + K - k0) * 2;
      step = fewer = kBK * 2;
      if (kin >= whole && chunk_k >= K - k0) {
        // a row goes on beyond K in memory
#pragma unroll
        for (int i = 0; i < kIssues; ++i) voff[i] = kOutside;
      }
      masked = kin >= whole;
    } else {
      base = first + ((long long)k0 * ld + row0) * 2;
      left = ((long long)(have - k0 - 1) * ld + rows - row0) * 2;
      // where more than kOutside bytes are left the bound need not follow
      step = (uint32_t)ld * (kBK * 2u);
      const long long after = left - (long long)plain * step;
      fewer = after > (long long)kOutside ? 0u : step;
      if (left > (long long)kOutside && fewer) plain = 1;
    }
    // The range check turns away whole 4-byte words.  An operand that ends in
    // the middle of one (an odd mc length) is bounded by the word's end: the
    // value beyond is in the same aligned word, so reading it cannot fault, and
    // it belongs to a column that does not exist.
    const uint32_t n = left <= 0                       ? 0u
                       : left >= (long long)kOutside ? kOutside
                                                       : ((uint32_t)left + 3u) & ~3u;
    bytes = (uint32_t)__builtin_amdgcn_readfirstlane((int)n);
    kin += plain;
    if (kin * kBK >= K) {
      kin = 0;
      ++seg;
    }
  }
  // No tiles at all.
  __device__ __forceinline__ void none() {
    base = (const char *)uniform((uint64_t)segs[0]);
    bytes = 0;
    plain = 0;
  }
  __device__ __forceinline__ void next(int wave, int lane) {
    --more;
    if (--plain > 0) {
      base += step;
      bytes -= fewer;
    } else if (more > 0) {
      seek(wave, lane);
    } else {
      bytes = 0;  // zeros from here on
    }
    // both are the same in every lane; without this they move to vector registers
    base = (const char *)uniform((uint64_t)base);
    bytes = (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes);
  }
  __device__ __forceinline__ void load(int i, char *lds, int wave) const {
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)bytes, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(lds + (i * NW + wave) * 1024), 16,
                                             voff[i], 0, 0, 0);
  }
};

// ds_read_b64_tr_b16: of each 16 lanes' 4 rows of 16 values (a row is four
// lanes' 8 bytes), lane t receives column t.  The restrict pointer matters: it
// gives the read the alias information without which the compiler lets it wait
// for every load to LDS in flight, whichever stage that goes to.
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ s16x4 read_transposed(lds_s16x4 *__restrict p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// Register fragments of one operand from its LDS tile.
template <int ROWS, bool MC>
struct Reader {
  static constexpr int kVar = MC ? 8 : 2;
  uint32_t at[kVar];
  // row0: this wave's first output row in the tile
  __device__ __forceinline__ void init(int lane, int row0) {
    const int g = lane >> 4, t = lane & 15;
    if constexpr (!MC) {
      const int r = row0 + t;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) at[ks] = r * 128 + (((ks * 4 + g) ^ swizzle<false, ROWS>(r)) << 4);
    } else {
      const int k = 8 * g + (t >> 2), q = t & 3;
#pragma unroll
      for (int v = 0; v < kVar; ++v) {
        const int c = row0 / 8 + 2 * v + (q >> 1);
        at[v] = k * (ROWS * 2) + ((c ^ swizzle<true, ROWS>(k)) << 4) + (q & 1) * 8;
      }
    }
  }
  // Tile i of 16 output rows, contraction values 32 ks .. 32 ks + 31.
  __device__ __forceinline__ s16x8 get(const char *lds, int i, int ks) const {
    lds_char *p = (lds_char *)lds;
    if constexpr (!MC) {
      return *(const __attribute__((address_space(3))) s16x8 *)(p + at[ks] + i * 2048);
    } else {
      lds_char *b = p + at[i] + ks * 32 * (ROWS * 2);
      const s16x4 lo = read_transposed((lds_s16x4 *)b);
      const s16x4 hi = read_transposed((lds_s16x4 *)(b + 4 * ROWS * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Which tile a workgroup takes.  Consecutive workgroups go to different XCDs,
// each with its own L2: every XCD is given a contiguous run of tiles, and runs
// walk bands of kBand tile rows, so that the tiles in flight on one XCD share
// operand rows.
constexpr int kBand = 4;
__device__ __forceinline__ void pick_tile(const GemmArgs &g, int id, int *tm, int *tn) {
  const int total = g.lower ? g.tiles_m * (g.tiles_m + 1) / 2 : g.tiles_m * g.tiles_n;
  const int xcd = id & 7, at = id >> 3, each = total >> 3, extra = total & 7;
  const int t = xcd * each + (xcd < extra ? xcd : extra) + at;
  if (g.lower) {  // t = tm (tm + 1) / 2 + tn, tn <= tm
    int m = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while (m * (m + 1) / 2 > t) --m;
    while ((m + 1) * (m + 2) / 2 <= t) ++m;
    *tm = m;
    *tn = t - m * (m + 1) / 2;
    return;
  }
  const int band = (int)fdiv((uint32_t)t, g.band), in = t - band * kBand * g.tiles_n;
  const int rows = g.tiles_m - band * kBand;
  if (rows >= kBand) {
    *tm = band * kBand + in % kBand;
    *tn = in / kBand;
  } else {
    *tm = band * kBand + in % rows;
    *tn = in / rows;
  }
}

// Accumulator layout.  The matrix instruction is given B as its row operand,
// so a lane holds 4 consecutive columns n of one row m of the result.
//
// Schedule.  Tiles are TS x TS x 64, 4 waves.  A wave keeps the fragments of
// two 32-value steps in registers: while the matrix cores work on one step,
// the next step's fragments are read from LDS.  LDS holds 2 d + 1 half tiles
// (A_t or B_t) in a ring, d tiles ahead: d = 2 for 256 x 256 (all of the 160 KB)
// and 128 x 128 (two workgroups on a compute unit), 4 for 64 x 64 (two):
//   step 0 of tile t: read step 1 of tile t; below 256, load A of t + d
//   wait for A and B of t + 1, barrier: the halves of t are free
//   step 1 of tile t: read step 0 of tile t + 1, load B of t + d; at 256, also
//     A of t + d + 1
// One barrier a tile, and no wait between a read or load and the next matrix
// instruction.  Loads are spread out between the matrix instructions: a load
// holds the address path for 16 clocks and a wave that meets it busy stops
// issuing matrix instructions too.
//
// With GROUPS of 4 waves, each takes a part of the contraction in a ring of its
// own, and the first adds the others' sums up in order: small results, whose
// tiles are fewer than the compute units, keep the matrix cores busier so than
// with the parts in other workgroups and a second kernel to join them.
template <int FMT, int TS, int GROUPS, bool A_MC, bool B_MC, int EPI>
__global__ __launch_bounds__(256 * GROUPS) void k_gemm(GemmArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)  // the body is device builtins throughout
  constexpr int NW = 4, WN = 2, WS = TS / 2, MT = WS / 16, NT = WS / 16;
  constexpr bool DUAL = EPI == kEpiGated;
  using LA = Loader<TS, A_MC, NW, false>;
  using LB = Loader<TS, B_MC, NW, DUAL>;
  constexpr int kHalf = LA::kBytes, kRing = TS == 64 && GROUPS == 1 ? 9 : 5, kAhead = kRing / 2;
  __shared__ __align__(1024) char all_smem[GROUPS * kRing * kHalf];

  // Ask for the arguments together, so that their latency is paid once.
  asm volatile("" ::"s"(g.M), "s"(g.N), "s"(g.K), "s"(g.ka), "s"(g.kb), "s"(g.lda), "s"(g.ldb),
               "s"(g.tiles_m), "s"(g.tiles_n), "s"(g.lower), "s"(g.steps), "s"(g.steps_more),
               "s"(g.batch_a), "s"(g.batch_b), "s"(g.band.m), "s"(g.band.l), "s"(g.a[0]), "s"(g.b[0]));

  const int lane = threadIdx.x & 63;
  const int every = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = every & (NW - 1), group = every / NW;
  char *const smem = all_smem + group * kRing * kHalf;
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  pick_tile(g, blockIdx.x, &tm, &tn);
  const int split = blockIdx.y, batch = blockIdx.z;
  const int row0 = tm * TS, col0 = tn * (DUAL ? TS / 2 : TS);
  // this group's contraction tiles; all groups go through as many turns (and
  // barriers), those without a tile with zeros
  int kt = split * g.steps + (split < g.steps_more ? split : g.steps_more);
  int mine_tiles = g.steps + (split < g.steps_more ? 1 : 0), tiles = mine_tiles;
  if constexpr (GROUPS > 1) {
    const int each = tiles / GROUPS, extra = tiles % GROUPS;
    tiles = each + (extra ? 1 : 0);
    mine_tiles = each + (group < extra ? 1 : 0);
    kt += group * each + (group < extra ? group : extra);
  }

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (tiles > 0) {
    LA la;
    LB lb;
    la.segs = g.a;
    lb.segs = g.b;
    la.off = batch * g.batch_a * 2;
    lb.off = batch * g.batch_b * 2 + (DUAL && (wave & 1) ? g.up_at * 2 : 0);
    la.ld = g.lda;
    lb.ld = g.ldb;
    la.row0 = row0;
    lb.row0 = col0;
    la.rows = g.M;
    lb.rows = g.N;
    la.K = lb.K = g.K;
    la.have = g.ka;
    lb.have = g.kb;
    la.more = lb.more = mine_tiles;
    la.seg = la.kin = 0;
    if (kt > 0) {
      const int per = (g.K + kBK - 1) / kBK;
      la.seg = kt / per;
      la.kin = kt - la.seg * per;
    }
    lb.seg = la.seg;
    lb.kin = la.kin;
    la.place_lanes(wave, lane);
    lb.place_lanes(wave, lane);
    if (GROUPS == 1 || mine_tiles > 0) {
      la.seek(wave, lane);
      lb.seek(wave, lane);
    } else {
      la.none();
      lb.none();
    }
    auto load_a = [&](char *s) {
#pragma unroll
      for (int i = 0; i < LA::kIssues; ++i) la.load(i, s, wave);
    };
    auto load_b = [&](char *s) {
#pragma unroll
      for (int i = 0; i < LB::kIssues; ++i) lb.load(i, s, wave);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      load_a(smem + 2 * i * kHalf);
      load_b(smem + (2 * i + 1) * kHalf);
      la.next(wave, lane);
      lb.next(wave, lane);
    }
    constexpr int kMfma = MT * NT, kReads = MT + NT, kLoads = LA::kIssues + LB::kIssues;
    constexpr int kPer = kMfma / 2 > kReads ? kMfma / 2 / kReads : 1;  // matrix instructions between reads
    constexpr int kGap = kMfma > 4 ? 4 : 2;                            // and between loads:
    // all in step 1, or those of A in step 0
    constexpr bool kLate = kLoads > kMfma / kGap;
    static_assert(kReads * kPer <= kMfma && LB::kIssues <= kMfma / kGap && LA::kIssues <= kMfma / kGap,
                  "reads and loads fit");
    if constexpr (!kLate) {
      load_a(smem + 2 * kAhead * kHalf);
      la.next(wave, lane);
    }

    s16x8 fa[2][MT], fb[2][NT];
    Reader<TS, A_MC> ra;
    Reader<TS, B_MC> rb;
    ra.init(lane, wm * WS);
    rb.init(lane, wn * WS);
    landed<(kLate ? kAhead - 1 : kAhead) * LA::kIssues + (kAhead - 1) * LB::kIssues>();
#pragma unroll
    for (int j = 0; j < NT; ++j) fb[0][j] = rb.get(smem + kHalf, j, 0);
#pragma unroll
    for (int i = 0; i < MT; ++i) fa[0][i] = ra.get(smem, i, 0);

    int slot = 0;                // of A_t; B_t in the next one
    char *sa = smem, *sb = smem + kHalf;
    char *to = smem + 2 * kAhead * kHalf, *free_b = smem;  // where the next A and B go
    settle();
    for (int t = 0; t < tiles; ++t) {
#pragma unroll
      for (int x = 0; x < kMfma; ++x) {
        if (x % kPer == 0 && x / kPer < kReads) {
          const int r = x / kPer;
          if (r < NT)
            fb[1][r] = rb.get(sb, r, 1);
          else
            fa[1][r - NT] = ra.get(sa, r - NT, 1);
        }
        if (kLate && x % kGap == kGap / 2 && x / kGap < LA::kIssues) la.load(x / kGap, to, wave);
        if (x == kMfma - 1) {
          slot = slot >= kRing - 2 ? slot - (kRing - 2) : slot + 2;
          free_b = sa;  // the next B goes where A of t was, the next A where B was
          to = sb;
          sa = smem + slot * kHalf;
          sb = smem + (slot == kRing - 1 ? 0 : slot + 1) * kHalf;
          if (kLate) la.next(wave, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
        mfma<FMT>(acc[x / NT][x % NT], fb[0][x % NT], fa[0][x / NT]);
        __builtin_amdgcn_sched_barrier(0);
      }
      // what was loaded after B of t + 1 may be in flight
      landed<(kAhead - 1) * LA::kIssues + (kAhead - 2) * LB::kIssues>();
#pragma unroll
      for (int x = 0; x < kMfma; ++x) {
        if (x % kPer == 0 && x / kPer < kReads) {
          const int r = x / kPer;
          if (r < NT)
            fb[0][r] = rb.get(sb, r, 0);
          else
            fa[0][r - NT] = ra.get(sa, r - NT, 0);
        }
        if (x % kGap == kGap / 2) {
          if (x / kGap < LB::kIssues)
            lb.load(x / kGap, free_b, wave);
          else if (!kLate && x / kGap < kLoads)
            la.load(x / kGap - LB::kIssues, to, wave);
        }
        if (x == kMfma - 1) {
          lb.next(wave, lane);
          if (!kLate) la.next(wave, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
        mfma<FMT>(acc[x / NT][x % NT], fb[1][x % NT], fa[1][x / NT]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  settle();
  landed<0>();

  // Sums go through LDS, up to 64 rows of a wave at a time, so that what follows
  // reads and writes whole rows, and its code is small: it runs once, and
  // instructions that run once are paid for in fetches.
  if constexpr (GROUPS > 1) {
    // the other groups' sums through LDS, lane by lane
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          *(f32x4 *)(smem + ((wave * MT + i) * NT + j) * 1024 + lane * 16) = acc[i][j];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll 1
    for (int o = 1; o < GROUPS; ++o)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] += *(const f32x4 *)(smem + o * kRing * kHalf + ((wave * MT + i) * NT + j) * 1024 +
                                        lane * 16);
  }
  constexpr int kStaged = WS < 64 ? WS : 64, kTiles = kStaged / 16;
  char *const mine = smem + wave * kStaged * (WS * 4);
  const int first = row0 + wm * WS, n0 = col0 + wn * (DUAL ? WS / 2 : WS);
#pragma unroll 1
  for (int h = 0; h < MT / kTiles; ++h) {
    const int m_in = lane & 15, q = lane >> 4;
#pragma unroll
    for (int hh = 0; hh < MT / kTiles; ++hh)
      if (h == hh) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            *(f32x4 *)const_cast<char *>(staged<WS>(mine, i * 16 + m_in, j * 16 + q * 4)) =
                acc[hh * kTiles + i][j];
      }
    const int m0 = first + h * kStaged, rows = g.M - m0 < kStaged ? g.M - m0 : kStaged;
    float *const part =
        g.splits > 1 ? g.partial + ((long long)split * g.batches + batch) * g.M * g.N : nullptr;
    if (!part)
      finish_staged<EPI, WS>(g.epi, mine, lane, batch, m0, rows, n0, g.N);
    else if constexpr (!DUAL)
      store_staged<WS, 0>(mine, lane, part, m0, rows, n0, g.N);
    if constexpr (EPI == kEpiPoly) {
      if (g.lower && tm != tn) {
        const int cols = g.N - n0 < WS ? g.N - n0 : WS;
        if (!part)
          finish_staged<EPI, WS, kStaged>(g.epi, mine, lane, batch, n0, cols, m0, g.M);
        else
          store_staged<WS, kStaged>(mine, lane, part, n0, cols, m0, g.M);
      }
    }
  }
#endif
}

}  // namespace dense
}  // namespace pdr
