// dense_skinny.hip -- products with few rows: y = x w^T for one to 64 rows of
// x, as a predictor that answers frame by frame asks for them.
//
// Such a product is a read of w (N K values, each used once per 16 rows), so
// everything serves that read: a workgroup owns 16 rows of w (of the gate and
// of the up weight in a gated product) and its 8 waves take interleaved
// pieces of the contraction, 16 bytes a lane straight from memory into the
// matrix instruction's registers, several loads in flight.  x is small and
// comes from the caches.  The waves' sums meet in LDS in one fixed order and
// go through the same epilogues as the large products'.  Nothing is laid out
// first: rows that do not begin on 16 bytes are read value by value, and fp32
// operands use the fp32 matrix instruction.
//
// Measured: one bf16 row times 4096 x 1024 (8.4 MB) 4.0 us, 2.1 TB/s, of which a
// launch with nothing to do takes about 2; four rows through a gated block of
// 1024 x 2816: 5.0 us for the gate and up products (11.5 MB), 6.2 for the
// other (5.8 MB; 64 workgroups, bound by latency).
#include "dense_internal.hpp"

namespace pdr {
namespace dense {

namespace {

constexpr int kWaves = 8;

template <int FMT>
struct Frag {  // what a lane holds of a row for one matrix step, 16 bytes
  static constexpr int kValues = 8;
  typedef s16x8 T;
  static __device__ __forceinline__ f32x4 go(T a, T b, f32x4 c) {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    if constexpr (FMT == kBf16)
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                     __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                    __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Frag<kF32> {
  static constexpr int kValues = 4;
  typedef f32x4 T;
  static __device__ __forceinline__ f32x4 go(T a, T b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

// Values [k, k + kValues) of a row of K; zeros past its end.
template <int FMT, bool ALIGNED>
__device__ __forceinline__ typename Frag<FMT>::T load_frag(const void *row, int k, int K) {
  typedef typename Frag<FMT>::T T;
  constexpr int V = Frag<FMT>::kValues;
  T v = {};
  if constexpr (ALIGNED) {
    if (k < K) v = *(const T *)((const char *)row + (long long)k * (16 / V));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (k + i < K) {
        if constexpr (FMT == kF32)
          v[i] = ((const float *)row)[k + i];
        else
          v[i] = ((const short *)row)[k + i];
      }
  }
  return v;
}

template <int FMT, int MT, bool ALIGNED, int EPI>
__global__ __launch_bounds__(kWaves * 64) void k_skinny(SkinnyArgs a) {
  typedef Frag<FMT> F;
  constexpr int V = F::kValues, kStep = 4 * V;  // values a wave takes at a time
  constexpr int KINDS = EPI == kEpiGated ? 2 : 1;
  constexpr int kAtOnce = MT == 1 ? 4 : 2;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16;
  // rows past the end repeat the last one and are not stored
  const long long size = fmt_bytes(FMT);
  const int n = n0 + t < a.N ? n0 + t : a.N - 1;
  const char *w[KINDS], *x[MT];
#pragma unroll
  for (int d = 0; d < KINDS; ++d)
    w[d] = (const char *)a.w + ((long long)n * a.ldw + d * a.up_at) * size;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = i * 16 + t < a.M ? i * 16 + t : a.M - 1;
    x[i] = (const char *)a.x + (long long)m * a.ldx * size;
  }
  f32x4 acc[KINDS][MT];
#pragma unroll
  for (int d = 0; d < KINDS; ++d)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[d][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int k0 = wave * kStep; k0 < a.K; k0 += kWaves * kStep * kAtOnce) {
    typename F::T fw[kAtOnce][KINDS], fx[kAtOnce][MT];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int k = k0 + u * kWaves * kStep + q * V;
#pragma unroll
      for (int d = 0; d < KINDS; ++d) fw[u][d] = load_frag<FMT, ALIGNED>(w[d], k, a.K);
#pragma unroll
      for (int i = 0; i < MT; ++i) fx[u][i] = load_frag<FMT, ALIGNED>(x[i], k, a.K);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int d = 0; d < KINDS; ++d)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[d][i] = F::go(fw[u][d], fx[u][i], acc[d][i]);
  }

  // a lane holds columns n = 4 q .. 4 q + 3 of row m = t
  __shared__ f32x4 red[kWaves][KINDS][MT][64];
#pragma unroll
  for (int d = 0; d < KINDS; ++d)
#pragma unroll
    for (int i = 0; i < MT; ++i) red[wave][d][i][lane] = acc[d][i];
  __syncthreads();
  for (int o = threadIdx.x; o < MT * 256; o += kWaves * 64) {
    const int c = o & 15, m = o >> 4;
    if (m >= a.M || n0 + c >= a.epi.store_n) continue;
    float v[KINDS];
#pragma unroll
    for (int d = 0; d < KINDS; ++d) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) s += red[i][d][m >> 4][(c >> 2) * 16 + (m & 15)][c & 3];
      v[d] = n0 + c < a.N ? s : 0.f;
    }
    const Columns<EPI, 1, kAsked> cols(a.epi, 0, n0 + c, a.N);
    typename Columns<EPI, 1, kAsked>::Row row;
    cols.fetch(a.epi, m, row);
    cols.finish(a.epi, m, v, row);
  }
}

template <int FMT, int MT, bool ALIGNED>
void go(const SkinnyArgs &a, bool gated, dim3 grid, hipStream_t st) {
  if (gated)
    hipLaunchKernelGGL((k_skinny<FMT, MT, ALIGNED, kEpiGated>), grid, dim3(kWaves * 64), 0, st, a);
  else
    hipLaunchKernelGGL((k_skinny<FMT, MT, ALIGNED, kEpiLinear>), grid, dim3(kWaves * 64), 0, st, a);
}
template <int FMT, bool ALIGNED>
void go_rows(const SkinnyArgs &a, bool gated, dim3 grid, hipStream_t st) {
  if (a.M <= 16)
    go<FMT, 1, ALIGNED>(a, gated, grid, st);
  else if (a.M <= 32)
    go<FMT, 2, ALIGNED>(a, gated, grid, st);
  else
    go<FMT, 4, ALIGNED>(a, gated, grid, st);
}

}  // namespace

hipError_t launch_skinny(const SkinnyArgs &a, int fmt, bool gated, hipStream_t st) {
  if (a.M <= 0 || a.epi.store_n <= 0) return hipSuccess;
  const dim3 grid((unsigned)((a.epi.store_n + 15) / 16));
  const int v = fmt == kF32 ? 4 : 8;
  const bool aligned = (((uintptr_t)a.x | (uintptr_t)a.w) & 15u) == 0 &&
                       ((a.ldx | a.ldw | a.up_at | a.K) & (v - 1)) == 0;
  if (fmt == kBf16)
    aligned ? go_rows<kBf16, true>(a, gated, grid, st) : go_rows<kBf16, false>(a, gated, grid, st);
  else if (fmt == kF16)
    aligned ? go_rows<kF16, true>(a, gated, grid, st) : go_rows<kF16, false>(a, gated, grid, st);
  else
    aligned ? go_rows<kF32, true>(a, gated, grid, st) : go_rows<kF32, false>(a, gated, grid, st);
  return hipGetLastError();
}

}  // namespace dense
}  // namespace pdr
