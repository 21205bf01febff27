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
// halves of a gated block's input gradient, and the three products
// hi*hi + hi*lo + lo*hi of fp32 operands split into two fp16 planes.
//
// LDS tiles are written by buffer loads straight to LDS (no registers), whose
// range check supplies the zeros beyond the operands' ends: no access leaves
// the operands whatever the sizes.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense_epilogue.hpp"

namespace pdr {
namespace dense {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) const char lds_char;

constexpr int kBK = 64;  // contraction values per LDS tile (128 bytes of a kc row)
constexpr int kMaxSegs = 6;
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
  int tiles_m, tiles_n, splits, batches;
  float *partial;                      // splits > 1: [split][batch][M][N] fp32
  Epi epi;
};

template <int FMT>
struct Mfma;
template <>
struct Mfma<kBf16> {
  static __device__ __forceinline__ f32x4 go(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Mfma<kF16> {
  static __device__ __forceinline__ f32x4 go(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};

// LDS swizzles: 16-byte chunk c of tile row r is stored at chunk c ^ s(r), so
// that the lanes of one read phase fall on different banks.
//  kc, A: a read takes rows t = 0..15 of one chunk: s = t & 7.
//  kc, B: a read takes rows 16 (t / 4) + t % 4 + const (see the accumulator
//         layout below): s = t % 4 + 4 ((t / 4) & 1).
//  mc, A: a read phase takes 4 rows k of 32 bytes: s moves pairs of chunks.
//  mc, B: a read phase takes 4 rows k of 4 half chunks, 32 bytes apart.
template <bool MC, bool SIDE_B>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (!MC)
    return SIDE_B ? (r & 3) | (((r >> 4) & 1) << 2) : r & 7;
  else
    return SIDE_B ? (r & 1) | (((r >> 1) & 1) << 3) : ((r & 3) << 1) | (((r >> 3) & 1) << 3);
}

// One operand's global-to-LDS copy: ROWS output rows by kBK contraction values
// per tile, NW waves.
template <int ROWS, bool MC, bool SIDE_B, int NW, bool DUAL>
struct Loader {
  static constexpr int kBytes = ROWS * kBK * 2;
  static constexpr int kIssues = kBytes / (NW * 1024);
  uint32_t voff[kIssues];
  const char *base;  // this tile's first byte in the segment
  long long left;    // bytes from base to the operand's end
  int chunk_k;       // kc: first contraction value of this lane's chunk

  __device__ __forceinline__ void init(int wave, int lane, long long ld, int row0, int rows) {
#pragma unroll
    for (int i = 0; i < kIssues; ++i) {
      const int blk = i * NW + wave;
      if constexpr (!MC) {
        const int r = blk * 8 + (lane >> 3);
        const int c = (lane & 7) ^ swizzle<false, SIDE_B>(r);
        chunk_k = c * 8;  // the same for every issue: s depends on r % 8 and bit 4 of r only
        if constexpr (DUAL) {
          // LDS rows 16 q + 4 j + i of a wave's 64: gate column 8 q + 4 (j & 1) + i
          // for j < 2, the up column of the same number for j >= 2
          const int col = (r >> 6) * 32 + ((r >> 4) & 3) * 8 + (r & 7);
          voff[i] = row0 + col < rows ? (uint32_t)((long long)col * ld * 2 + c * 16) : kOutside;
        } else {
          voff[i] = (uint32_t)((long long)r * ld * 2 + c * 16);
        }
      } else {
        constexpr int kLanesPerRow = ROWS / 8;
        const int k = blk * (64 / kLanesPerRow) + lane / kLanesPerRow;
        const int c = (lane % kLanesPerRow) ^ swizzle<true, SIDE_B>(k);
        voff[i] = (uint32_t)((long long)k * ld * 2 + c * 16);
      }
    }
  }

  // Point at contraction value k0 of rows row0.. of an operand.
  __device__ __forceinline__ void seek(const void *p, long long ld, int row0, int rows, int K,
                                       int k0) {
    if constexpr (!MC) {
      const long long at = ((long long)row0 * ld + k0) * 2;
      base = (const char *)p + at;
      left = ((long long)(rows - 1) * ld + K) * 2 - at;
    } else {
      const long long at = ((long long)k0 * ld + row0) * 2;
      base = (const char *)p + at;
      left = ((long long)(K - 1) * ld + rows) * 2 - at;
    }
  }
  __device__ __forceinline__ void advance(long long ld) {
    const long long step = MC ? (long long)kBK * ld * 2 : kBK * 2;
    base += step;
    left -= step;
  }
  __device__ __forceinline__ void load(char *lds, int wave, int k_left) const {
    // The range check turns away whole 4-byte words.  An operand that ends in
    // the middle of one (an odd mc length) is bounded by the word's end: the
    // value beyond is in the same aligned word, so reading it cannot fault, and
    // it belongs to a column that does not exist.
    const uint32_t n = left <= 0                       ? 0u
                       : left >= (long long)kOutside ? kOutside
                                                       : ((uint32_t)left + 3u) & ~3u;
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)n, 0x00020000);
    // a kc row goes on beyond K in memory: chunks past it are turned away here
    const bool off = !MC && chunk_k >= k_left;
#pragma unroll
    for (int i = 0; i < kIssues; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(lds + (i * NW + wave) * 1024), 16,
                                               off ? kOutside : voff[i], 0, 0, 0);
  }
};

// Register fragments of one operand from its LDS tile.
template <int ROWS, bool MC, bool SIDE_B>
struct Reader {
  static constexpr int kVar = MC ? (SIDE_B ? 2 : 8) : 2;
  uint32_t at[kVar];
  // row0: this wave's first output row in the tile
  __device__ __forceinline__ void init(int lane, int row0) {
    const int g = lane >> 4, t = lane & 15;
    if constexpr (!MC) {
      const int r = row0 + (SIDE_B ? 16 * (t >> 2) + (t & 3) : t);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        at[ks] = r * 128 + (((ks * 4 + g) ^ swizzle<false, SIDE_B>(r)) << 4);
    } else {
      const int k = 8 * g + (t >> 2), q = t & 3;
      const int s = swizzle<true, SIDE_B>(k);
#pragma unroll
      for (int v = 0; v < kVar; ++v) {
        const int c = SIDE_B ? row0 / 8 + 2 * q + v : row0 / 8 + 2 * v + (q >> 1);
        at[v] = k * (ROWS * 2) + ((c ^ s) << 4) + (SIDE_B ? 0 : (q & 1) * 8);
      }
    }
  }
  // Tile i of 16 output rows, contraction values 32 ks .. 32 ks + 31.
  __device__ __forceinline__ s16x8 get(const char *lds, int i, int ks) const {
    lds_char *p = (lds_char *)lds;
    if constexpr (!MC) {
      return *(const __attribute__((address_space(3))) s16x8 *)(p + at[ks] + (SIDE_B ? i * 512 : i * 2048));
    } else {
      lds_char *b = p + (SIDE_B ? at[i >> 1] + (i & 1) * 8 : at[i]) + ks * 32 * (ROWS * 2);
      s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)b);
      s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4 *)(b + 4 * ROWS * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Which tile a workgroup takes.  Consecutive workgroups go to different XCDs,
// each with its own L2: every XCD is given a contiguous run of tiles, and runs
// walk bands of kBand tile rows, so that the tiles in flight on one XCD share
// operand rows.
constexpr int kBand = 4;
__device__ __forceinline__ void pick_tile(int id, int tiles_m, int tiles_n, int *tm, int *tn) {
  const int total = tiles_m * tiles_n;
  const int xcd = id & 7, at = id >> 3, each = total >> 3, extra = total & 7;
  const int t = xcd * each + (xcd < extra ? xcd : extra) + at;
  const int band = t / (kBand * tiles_n), in = t - band * kBand * tiles_n;
  const int rows = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
  *tm = band * kBand + in % rows;
  *tn = in / rows;
}

// Accumulator layout.  The matrix instruction is given B as its row operand,
// so a lane holds 4 consecutive rows n of one column m per instruction; B's
// rows are dealt to the 4 instructions of a wave's 64 columns as
// n = 16 q + 4 j + i (q: lane / 16, j: instruction, i: register), which makes
// a lane's 16 values of one m consecutive in memory: 16-byte stores, 128
// contiguous bytes per row and wave.
template <int FMT, int BM, int BN, int WM, int WN, bool A_MC, bool B_MC, int EPI>
__global__ __launch_bounds__(WM *WN * 64) void k_gemm(GemmArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)  // the body is device builtins throughout
  constexpr int NW = WM * WN;
  constexpr int MT = BM / WM / 16;
  constexpr bool DUAL = EPI == kEpiGated;
  static_assert(BN / WN == 64, "a wave owns 64 columns");
  using LA = Loader<BM, A_MC, false, NW, false>;
  using LB = Loader<BN, B_MC, true, NW, DUAL>;
  constexpr int kStage = LA::kBytes + LB::kBytes;
  __shared__ __align__(1024) char smem[2 * kStage];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  pick_tile(blockIdx.x, g.tiles_m, g.tiles_n, &tm, &tn);
  const int split = blockIdx.y, batch = blockIdx.z;
  const int row0 = tm * BM, col0 = tn * (DUAL ? BN / 2 : BN);

  LA la;
  LB lb;
  la.init(wave, lane, g.lda, row0, g.M);
  lb.init(wave, lane, g.ldb, col0, g.N);
  Reader<BM, A_MC, false> ra;
  Reader<BN, B_MC, true> rb;
  ra.init(lane, wm * (BM / WM));
  rb.init(lane, wn * 64);

  const int kt_seg = (g.K + kBK - 1) / kBK, kt_all = kt_seg * g.segs;
  const int each = kt_all / g.splits, extra = kt_all % g.splits;
  int kt = split * each + (split < extra ? split : extra);
  const int kt_end = kt + each + (split < extra ? 1 : 0);
  int seg = kt / kt_seg, kin = kt - seg * kt_seg;
  const long long oa = batch * g.batch_a * 2, ob = batch * g.batch_b * 2;
  auto seek = [&]() {
    la.seek((const char *)g.a[seg] + oa, g.lda, row0, g.M, A_MC ? g.ka : g.K, kin * kBK);
    lb.seek((const char *)g.b[seg] + ob + (DUAL && (wave & 1) ? g.up_at * 2 : 0), g.ldb, col0, g.N,
            B_MC ? g.kb : g.K, kin * kBK);
  };
  auto issue = [&](int buf) {
    char *s = smem + buf * kStage;
    la.load(s, wave, g.K - kin * kBK);
    lb.load(s + LA::kBytes, wave, g.K - kin * kBK);
    if (++kin == kt_seg) {
      kin = 0;
      if (++seg < g.segs) seek();
    } else {
      la.advance(g.lda);
      lb.advance(g.ldb);
    }
  };

  f32x4 acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (kt < kt_end) {
    seek();
    issue(0);
  }
  int buf = 0;
  for (; kt < kt_end; ++kt) {
    __syncthreads();  // tile kt has arrived, and every wave is done with the other buffer
    if (kt + 1 < kt_end) issue(buf ^ 1);
    const char *s = smem + buf * kStage;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      s16x8 fb[4], fa[MT];
#pragma unroll
      for (int j = 0; j < 4; ++j) fb[j] = rb.get(s + LA::kBytes, j, ks);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[i] = ra.get(s, i, ks);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = Mfma<FMT>::go(fb[j], fa[i], acc[i][j]);
    }
    buf ^= 1;
  }

  const int q = lane >> 4;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = row0 + wm * (BM / WM) + i * 16 + (lane & 15);
    if (m >= g.M) continue;
    float v[16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j * 4 + e] = acc[i][j][e];
    if constexpr (DUAL) {
      epi_gated(g.epi, m, col0 + wn * 32 + q * 8, v, v + 8);
    } else {
      const int n = col0 + wn * 64 + q * 16;
      if (g.splits > 1) {
        float *p = g.partial + ((long long)split * g.batches + batch) * g.M * g.N;
        store_partial(p, m, n, g.N, v);
        store_partial(p, m, n + 8, g.N, v + 8);
      } else {
        epi_apply<EPI>(g.epi, batch, m, n, g.N, v);
        epi_apply<EPI>(g.epi, batch, m, n + 8, g.N, v + 8);
      }
    }
  }
#endif
}

}  // namespace dense
}  // namespace pdr
