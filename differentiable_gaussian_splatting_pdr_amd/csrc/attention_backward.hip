// attention_backward.hip -- the gradients of attention.
//
// Two kernels instead of one: the queries' gradients sum over keys, the keys'
// over queries, and with a workgroup for each result nothing is added by
// atomics, so a result does not depend on the run.  That costs seven products
// where five would do.
#include "attention.hpp"

namespace pdr {
namespace attend {

namespace {

// Weights and score gradients.  With sums that start from
//   start_s = -lse / scale2,  start_dp = -(dy . o)
// the products leave s - lse and dp - delta, and
//   p = exp2(scale2 s),  ds = p dp
// are an exponential and two products a pair.  fp32 scores start from 0, and take
// lse in the exponent: what rounding at lse's magnitude costs them shows (2e-6
// instead of 8e-7 of a gradient).  In fp16 p is taken times 2^15, which keeps
// long rows' weights in the type's range.
constexpr int kShift = 15;

template <int FMT>
__device__ __forceinline__ float start_of(float lse, float scale2) {
  return FMT == kF32 ? -lse : ((FMT == kF16 ? kShift : 0) - lse) / scale2;
}

// s + x . y of 16 bytes each.
template <int FMT>
__device__ __forceinline__ float dot(i32x4 x, i32x4 y, float s) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (FMT == kF32) {
      s = fmaf(__int_as_float(x[j]), __int_as_float(y[j]), s);
    } else {
      s = fmaf(dense::to_f<FMT>((uint16_t)x[j]), dense::to_f<FMT>((uint16_t)y[j]), s);
      s = fmaf(dense::to_f<FMT>((uint16_t)((uint32_t)x[j] >> 16)),
               dense::to_f<FMT>((uint16_t)((uint32_t)y[j] >> 16)), s);
    }
  }
  return s;
}

// A row whose scores are all -infinity (its lse is +infinity) has no gradient, where
// ds of zero would make NaN of a key's infinity.
template <class C>
__device__ __forceinline__ void clear_empty(f32x16 (&sums)[C::kBlocks], float start_s) {
  if (start_s != -INFINITY) return;
#pragma unroll
  for (int b = 0; b < C::kBlocks; ++b) clear(sums[b]);
}

// A tile's weights from its scores, and their gradients, in place.  `start`: of the
// scores in fp32.
template <int FMT>
__device__ __forceinline__ void weigh(float &s, float &dp, float start, float scale2) {
  s = exp2_(FMT == kF32 ? fmaf(s, scale2, start) : s * scale2);
  dp *= s;
}

// ds enters the products in the operands' type.  In fp16 it would leave its range:
// it is taken times a power of two for each column of the result, found from the
// largest value that the column has met.
template <class C, int FMT>
struct Scaled {
  int e;  // ds is taken times 2^e
  __device__ __forceinline__ void init() { e = 100; }
  __device__ __forceinline__ void hold(f32x16 &ds, f32x16 (&sums)[C::kBlocks]) {
    if constexpr (FMT == kF16) {
      float m = 0.f;
#pragma unroll
      for (int r = 0; r < 16; ++r) m = fmaxf(m, fabsf(ds[r]));
      m = fmaxf(m, other_half(m));
      // m 2^e < 2^15 is held
      const int most = m > 0.f ? 15 - __builtin_amdgcn_frexp_expf(m) : 100;
      if (__any(most < e)) {
        // leave room for four times as much
        int to = most - 2 < -120 ? -120 : most - 2;
        if (most >= e) to = e;
        const float by = __builtin_amdgcn_ldexpf(1.f, to - e);
#pragma unroll
        for (int b = 0; b < C::kBlocks; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r) sums[b][r] *= by;
        e = to;
      }
      const float by = __builtin_amdgcn_ldexpf(1.f, e);
#pragma unroll
      for (int r = 0; r < 16; ++r) ds[r] *= by;
    }
  }
  // What the sums are to be multiplied by.
  __device__ __forceinline__ float out() const { return FMT == kF16 ? ldexpf(1.f, -e - kShift) : 1.f; }
};

template <class C>
__device__ __forceinline__ void across32(f32x16 (&c)[C::kBlocks], const lds_char *tile, int u,
                                         const f32x16 &w, const typename C::Lane &at) {
#pragma unroll
  for (int x = 0; x < 2; ++x) C::across(c, tile, 2 * u + x, C::pack(w, 8 * x), at);
}

// A row's starts, from what its lanes hold of dy; `writes`: also for dk and dv.
template <int FMT, int DP>
__device__ __forceinline__ void starts_of_row(const Args &a, const Place &at, int head, int row, bool there, int token,
                                              int in_group, int half, const i32x4 (&dy)[Core<FMT, DP>::kSteps],
                                              bool writes, float *start_s, float *start_dp) {
  using C = Core<FMT, DP>;
  const int group = (int)a.group.d;
  i32x4 o[C::kSteps];
  C::fetch_row(o, a.o.p + (first_of(a.o, at, at.q0 + token, head * group) + in_group * a.o.head) * C::kSize, a.dim,
               half, there);
  float d = 0.f;
#pragma unroll
  for (int i = 0; i < C::kSteps; ++i) d = dot<FMT>(o[i], dy[i], d);
  *start_dp = -(d + other_half(d));
  *start_s = 0.f;
  if (!there) return;
  const long long tokens = a.q_offsets ? a.q_rows : (long long)a.batch * a.q_rows;
  const long long i = (head * tokens + (a.q_offsets ? 0 : (long long)at.seq * a.q_rows) + at.q0) * group + row;
  *start_s = start_of<FMT>(a.lse[i], a.scale2);
  if (half == 0 && writes) *(float2 *)(a.starts + 2 * i) = make_float2(*start_s, *start_dp);
}

// delta = dy . o takes over the rounding of o and, in it, of the forward's weights.
// Since p sums to 1, what ds adds up to with such a delta is by how much it is off:
//   sum p (dp - delta') = delta - delta'.
// A row of n keys loses to that about 1 / n of what rounding its ds costs, so that it
// shows where n is small: queries that see up to kExact keys find the sum in a pass over them
// first.  16 bits, causal, 777 queries: errors of dq 1.60 times those of rounding
// the result, and 1.45 with this; 1.41 is the rounding of ds.
constexpr int kExact = 256;

// The row's start with the sum of ds added, there and for dk and dv.
template <int FMT>
__device__ __forceinline__ void mend_start(const Args &a, const Place &at, int head, int row, int rows, float off,
                                           bool writes, float *start_dp) {
  *start_dp -= FMT == kF16 ? ldexpf(off, -kShift) : off;
  if (!writes || row >= rows) return;
  const long long tokens = a.q_offsets ? a.q_rows : (long long)a.batch * a.q_rows;
  const long long first = (head * tokens + (a.q_offsets ? 0 : (long long)at.seq * a.q_rows) + at.q0) * a.group.d;
  a.starts[2 * (first + row) + 1] = *start_dp;
}

// dq: 128 rows to a workgroup, 32 to a wave, as in the forward; and the rows'
// starts, which is all there is to do where dq is not wanted.  Three products to an
// exponential; bound as the forward is: bf16, packed sequences of up to 4096, 32 heads of
// 128, 539 us, 0.99 PFLOP/s; 8 x 1024 with 12 heads of 64, 50 us.
template <int FMT, int DP>
__global__ __launch_bounds__(256, FMT == kF32 ? 1 : 2) void k_backward_q(Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Core<FMT, DP>;
  constexpr int kKeys = 64;
  using L = Loader<C, kKeys, 4>;
  __shared__ __align__(1024) char shared[4 * L::kBytes];
  lds_char *const smem = (lds_char *)shared;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = (int)fdiv(blockIdx.x, a.heads), head = blockIdx.x - unit * a.kv_heads;
  const Place at = place<kLogWide, false>(a, a.causal ? a.q_tiles - 1 - unit : unit);
  const int group = (int)a.group.d, rows = at.nq * group;
  const int row0 = at.tile << kLogWide;
  if (at.tile < 0 || row0 >= rows) return;
  const int row = row0 + wave * 32 + (lane & 31);
  const bool there = row < rows;
  const int token = (int)fdiv((uint32_t)(there ? row : rows - 1), a.group);
  const int in_group = there ? row - token * group : 0;
  const int ahead = at.nk - at.nq;
  int keys = at.nk;
  if (a.causal) {
    const int last = row0 + 127 < rows ? row0 + 127 : rows - 1;
    const int k = (int)fdiv((uint32_t)last, a.group) + ahead + 1;
    keys = k < 0 ? 0 : k;
  }
  const int first_row = row0 + wave * 32 < rows ? row0 + wave * 32 : rows - 1;
  const int plain = !a.causal ? at.nk : (int)fdiv((uint32_t)first_row, a.group) + ahead + 1;

  i32x4 q[C::kSteps], dy[C::kSteps];
  C::fetch_row(dy, a.dy.p + (first_of(a.dy, at, at.q0 + token, head * group) + in_group * a.dy.head) * C::kSize,
               a.dim, half, there);
  float start_s, start_dp;
  starts_of_row<FMT, DP>(a, at, head, row, there, token, in_group, half, dy, true, &start_s, &start_dp);
  C::fetch_row(q, a.q.p + (first_of(a.q, at, at.q0 + token, head * group) + in_group * a.q.head) * C::kSize,
               a.dim, half, there);
  f32x16 sums[C::kBlocks];
#pragma unroll
  for (int b = 0; b < C::kBlocks; ++b) clear(sums[b]);
  typename C::Lane lanes;
  lanes.init(lane);
  Scaled<C, FMT> scaled;
  scaled.init();
  const Source k(a.k, first_of(a.k, at, at.k0, head), C::kSize), v(a.v, first_of(a.v, at, at.k0, head), C::kSize);
  // a lane's place in the loads is worked out each time, as in k_backward_kv
  auto load = [&](int t, lds_char *to) {
    L loader;
    loader.init(a.dim, wave, lane_again());
    loader.tokens(k, v, t * kKeys, at.nk, to);
  };
  // ds of 32 keys, in s
  auto gradients = [&](f32x16 &s, const lds_char *sk, const lds_char *sv, int t, int u) {
    f32x16 dp;
    fill(s, FMT == kF32 ? 0.f : start_s);
    fill(dp, start_dp);
    C::along(s, sk, u, q, lanes);
    C::along(dp, sv, u, dy, lanes);
    C::template pace_along<2>();
    const int key0 = t * kKeys + u * 32;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float p = s[r], ds = dp[r];
      weigh<FMT>(p, ds, start_s, a.scale2);
      s[r] = ds;
    }
    if (key0 + 32 > plain) {
      const int lane = lane_again(), r = row0 + wave * 32 + (lane & 31);
      const int token = (int)fdiv((uint32_t)(r < rows ? r : rows - 1), a.group);
      const int seen = !a.causal ? at.nk : token + ahead + 1 < at.nk ? token + ahead + 1 : at.nk;
      const int last = here(seen - key0 - 4 * (lane >> 5));
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (row_in(r, 0) >= last) s[r] = 0.f;
    }
  };
  const int tiles = (keys + kKeys - 1) / kKeys;
  // Tile t has come, and the next is on its way.
  auto turn = [&](int t) {
    all_landed<0>();
    if (t + 1 < tiles) load(t + 1, smem + ((t + 1) & 1) * (2 * L::kBytes));
    return smem + (t & 1) * (2 * L::kBytes);
  };
  const bool exact = FMT != kF32 && tiles > 0 && keys <= kExact;
  if (!exact && !a.dq.p) return;
  if (tiles > 0) load(0, smem);
  if (exact) {
    float off = 0.f;
    for (int t = 0; t < tiles; ++t) {
      const lds_char *const sk = turn(t), *const sv = sk + L::kBytes;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f32x16 s;
        gradients(s, sk, sv, t, u);
#pragma unroll
        for (int r = 0; r < 16; ++r) off += s[r];
      }
    }
    const int lane = lane_again();
    mend_start<FMT>(a, at, head, row0 + wave * 32 + (lane & 31), rows, off + other_half(off), lane < 32, &start_dp);
    if (!a.dq.p) return;
    __syncthreads();
    load(0, smem);
  }
  for (int t = 0; t < tiles; ++t) {
    const lds_char *const sk = turn(t), *const sv = sk + L::kBytes;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x16 s;
      gradients(s, sk, sv, t, u);
      scaled.hold(s, sums);
      across32<C>(sums, sk, u, s, lanes);
      C::template pace_across<1>();
    }
  }
  const int lane_now = lane_again(), row_now = row0 + wave * 32 + (lane_now & 31);
  if (row_now >= rows) return;
  const int n = (int)fdiv((uint32_t)row_now, a.group), g = row_now - n * group;
  clear_empty<C>(sums, start_s);
  store_columns<C, FMT>(sums, a.dq.p + (first_of(a.dq, at, at.q0 + n, head * group) + g * a.dq.head) * C::kSize, a.dim,
                        lane_now >> 5, a.scale * scaled.out());
#endif
}

// Sums of a key to dk (which = 0) or dv, or to the parts' sums:
// [part][dk, dv][key head][key][dim].
template <class C, int FMT>
__device__ __forceinline__ void store_keys(const Args &a, const Place &at, const Mat &to, int which, int head,
                                           int key, const f32x16 (&c)[C::kBlocks], int half, float by) {
  const long long where = at.k0 + key;
  if (a.splits > 1) {
    const long long all = (a.q_offsets ? 1LL : a.batch) * a.k_rows;
    const long long mine = (a.q_offsets ? 0 : (long long)at.seq * a.k_rows) + where;
    using P = Core<kF32, C::kBlocks * 32>;
    store_columns<P, kF32>(
        c, (char *)(a.part_k + (((2LL * blockIdx.y + which) * a.kv_heads + head) * all + mine) * a.dim), a.dim, half,
        by);
    return;
  }
  store_columns<C, FMT>(c, to.p + (at.seq * to.batch + where * to.row + head * to.head) * C::kSize, a.dim, half, by);
}

// dq where 128 rows to a workgroup would leave compute units without one: 32 rows,
// whose waves take parts of the keys each, in LDS of their own (fp32 4 x 1024, 8 heads
// of 64, causal: 82 us, about 120 with the larger ones).
template <int FMT, int DP, int NW>
__global__ __launch_bounds__(64 * NW) void k_backward_q_few(Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Core<FMT, DP>;
  constexpr int kKeys = 32;
  using L = Loader<C, kKeys, 1>;
  constexpr int kRing = 4 * L::kBytes;  // two tiles of keys and values
  __shared__ __align__(1024) char shared[NW * kRing];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = (int)fdiv(blockIdx.x, a.heads), head = blockIdx.x - unit * a.kv_heads;
  const Place at = place<kLogFew, false>(a, a.causal ? a.q_tiles - 1 - unit : unit);
  const int group = (int)a.group.d, rows = at.nq * group;
  const int row0 = at.tile << kLogFew;
  if (at.tile < 0 || row0 >= rows) return;
  const int row = row0 + (lane & 31);
  const bool there = row < rows;
  const int token = (int)fdiv((uint32_t)(there ? row : rows - 1), a.group);
  const int in_group = there ? row - token * group : 0;
  const int ahead = at.nk - at.nq;
  const int seen = !a.causal ? at.nk : token + ahead + 1 < at.nk ? token + ahead + 1 : at.nk;
  int keys = at.nk, plain = at.nk;
  if (a.causal) {
    const int last = row0 + 31 < rows ? row0 + 31 : rows - 1;
    keys = (int)fdiv((uint32_t)last, a.group) + ahead + 1;
    plain = (int)fdiv((uint32_t)row0, a.group) + ahead + 1;
    if (keys < 0) keys = 0;
  }

  i32x4 q[C::kSteps], dy[C::kSteps];
  C::fetch_row(dy, a.dy.p + (first_of(a.dy, at, at.q0 + token, head * group) + in_group * a.dy.head) * C::kSize,
               a.dim, half, there);
  float start_s, start_dp;
  starts_of_row<FMT, DP>(a, at, head, row, there, token, in_group, half, dy, wave == 0, &start_s, &start_dp);
  C::fetch_row(q, a.q.p + (first_of(a.q, at, at.q0 + token, head * group) + in_group * a.q.head) * C::kSize,
               a.dim, half, there);
  f32x16 sums[C::kBlocks];
#pragma unroll
  for (int b = 0; b < C::kBlocks; ++b) clear(sums[b]);
  typename C::Lane lanes;
  lanes.init(lane);
  Scaled<C, FMT> scaled;
  scaled.init();
  const Source k(a.k, first_of(a.k, at, at.k0, head), C::kSize), v(a.v, first_of(a.v, at, at.k0, head), C::kSize);
  L load;
  load.init(a.dim, 0, lane);
  lds_char *const ring = (lds_char *)shared + wave * kRing;
  const int all = (keys + kKeys - 1) / kKeys, each = (all + NW - 1) / NW;
  const int begin = wave * each < all ? wave * each : all;
  const int end = begin + each < all ? begin + each : all;
  // ds of tile t, in s
  auto gradients = [&](f32x16 &s, const lds_char *sk, int t) {
    f32x16 dp;
    fill(s, FMT == kF32 ? 0.f : start_s);
    fill(dp, start_dp);
    C::along(s, sk, 0, q, lanes);
    C::along(dp, sk + L::kBytes, 0, dy, lanes);
    C::template pace_along<2>();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float p = s[r], ds = dp[r];
      weigh<FMT>(p, ds, start_s, a.scale2);
      s[r] = ds;
    }
    if ((t + 1) * kKeys > plain) {
      const int last = here(seen - t * kKeys - 4 * half);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (row_in(r, 0) >= last) s[r] = 0.f;
    }
  };
  // Tile t has come, the last one's reads are done, and the next is on its way.
  auto turn = [&](int t) {
    landed<0>();
    if (t + 1 < end) load.tokens(k, v, (t + 1) * kKeys, at.nk, ring + ((t + 1 - begin) & 1) * (2 * L::kBytes));
    return ring + ((t - begin) & 1) * (2 * L::kBytes);
  };
  const bool exact = FMT != kF32 && keys <= kExact;
  if (!exact && !a.dq.p) return;
  if (begin < end) load.tokens(k, v, begin * kKeys, at.nk, ring);
  if (exact) {
    float off = 0.f;
    for (int t = begin; t < end; ++t) {
      f32x16 s;
      gradients(s, turn(t), t);
#pragma unroll
      for (int r = 0; r < 16; ++r) off += s[r];
    }
    off += other_half(off);
    float *const offs = (float *)shared;
    __syncthreads();
    if (half == 0) offs[wave * 32 + lane] = off;
    __syncthreads();
    off = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) off += offs[w * 32 + (lane & 31)];
    mend_start<FMT>(a, at, head, row, rows, off, wave == 0 && half == 0, &start_dp);
    if (!a.dq.p) return;
    __syncthreads();
    if (begin < end) load.tokens(k, v, begin * kKeys, at.nk, ring);
  }
  for (int t = begin; t < end; ++t) {
    const lds_char *const sk = turn(t);
    f32x16 s;
    gradients(s, sk, t);
    scaled.hold(s, sums);
    across32<C>(sums, sk, 0, s, lanes);
    C::template pace_across<1>();
  }
  clear_empty<C>(sums, start_s);
  // the waves' sums, where their keys were
  __syncthreads();
  const float by = a.scale * scaled.out();
#pragma unroll
  for (int b = 0; b < C::kBlocks; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *(float4 *)(shared + wave * kRing + (lane & 31) * (DP * 4) + (((b * 32 + row_in(r, half)) / 4 ^ (lane & 7)) * 16)) =
          make_float4(sums[b][r] * by, sums[b][r + 1] * by, sums[b][r + 2] * by, sums[b][r + 3] * by);
  __syncthreads();
  for (int x = threadIdx.x; x < 32 * (DP / 4); x += 64 * NW) {
    const int i = x / (DP / 4), d = x % (DP / 4) * 4;
    if (row0 + i >= rows || d >= a.dim) continue;
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 o = *(const float4 *)(shared + w * kRing + i * (DP * 4) + ((d / 4 ^ (i & 7)) * 16));
      c[0] += o.x;
      c[1] += o.y;
      c[2] += o.z;
      c[3] += o.w;
    }
    const int n = (int)fdiv((uint32_t)(row0 + i), a.group), g = row0 + i - n * group;
    store4<FMT>(a.dq.p + (first_of(a.dq, at, at.q0 + n, head * group) + g * a.dq.head + d) * C::kSize, c);
  }
#endif
}

// dk and dv: 128 keys to a workgroup, 32 to a wave; the waves share tiles of
// rows (of all heads that read these keys), and of their starts.  Four products to an
// exponential, and the sums of two of them in registers: with keys and values that is all
// that two waves a SIMD leave, so that fragments are read as they are needed and the
// other wave covers the wait.  bf16, packed sequences of up to 4096: 850 us, 0.83
// PFLOP/s, against 1182 with one wave that reads ahead and 1026 with the products shared by a
// pair of waves; 8 x 1024 with 12 heads of 64, 63 us (66 with fragments read ahead: two
// waves instead of three).
template <int FMT, int DP>
__global__ __launch_bounds__(256, FMT == kF32 ? 1 : 2) void k_backward_kv(Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Core<FMT, DP>;
  constexpr int kRows = 64;
  using L = Loader<C, kRows, 4>;
  constexpr int kStage = 2 * L::kBytes + 2 * kRows * 4;
  __shared__ __align__(1024) char shared[2 * kStage];
  lds_char *const smem = (lds_char *)shared;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = (int)fdiv(blockIdx.x, a.heads), head = blockIdx.x - unit * a.kv_heads;
  const Place at = place<kLogWide, true>(a, unit);
  const int group = (int)a.group.d, rows = at.nq * group;
  const int key0 = at.tile << kLogWide;
  if (at.tile < 0 || key0 >= at.stored) return;
  const int key = key0 + wave * 32 + (lane & 31);
  const bool there = key < at.nk;
  const int ahead = at.nk - at.nq;
  // the first row that sees a key; none sees what is no key
  auto first_row = [&](int k) {
    if (k >= at.nk) return rows;
    const long long r = a.causal ? (long long)(k - ahead) * group : 0;
    return r < 0 ? 0 : r > rows ? rows : (int)r;
  };
  const int plain = first_row(key0 + wave * 32 + 31);  // from here on the wave needs no mask
  // this part's tiles of rows
  int begin = first_row(key0) / kRows;
  const int last = key0 < at.nk ? (rows + kRows - 1) / kRows : begin;
  const int each = (last - begin + a.splits - 1) / a.splits;
  begin += blockIdx.y * each;
  const int end = begin + each < last ? begin + each : last;

  i32x4 k[C::kSteps], v[C::kSteps];
  C::fetch_row(k, a.k.p + first_of(a.k, at, at.k0 + (there ? key : 0), head) * C::kSize, a.dim, half, there);
  C::fetch_row(v, a.v.p + first_of(a.v, at, at.k0 + (there ? key : 0), head) * C::kSize, a.dim, half, there);
  f32x16 dk[C::kBlocks], dv[C::kBlocks];
#pragma unroll
  for (int b = 0; b < C::kBlocks; ++b) {
    clear(dk[b]);
    clear(dv[b]);
  }
  typename C::Lane lanes;
  lanes.init(lane);
  Scaled<C, FMT> scaled;
  scaled.init();
  const Source from_q(a.q, first_of(a.q, at, at.q0, head * group), C::kSize);
  const Source from_dy(a.dy, first_of(a.dy, at, at.q0, head * group), C::kSize);
  const long long tokens = a.q_offsets ? a.q_rows : (long long)a.batch * a.q_rows;
  const long long first =
      (head * tokens + (a.q_offsets ? 0 : (long long)at.seq * a.q_rows) + at.q0) * group;
  // What only this and the ends need of a lane's number is worked out each time: with
  // two waves on a SIMD there is no register to hold it, and what is fetched back
  // from scratch memory waits for all loads in flight.
  auto load = [&](int t, lds_char *stage) {
    const int lane = lane_again();
    L loader;
    loader.init(a.dim, wave, lane);
    loader.grouped(from_q, from_dy, t * kRows, rows, a.group, stage);
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)(a.starts + 2 * (first + t * kRows)), 0, kRows * 8, 0x00020000);
    // one wave each
    if (wave < 2)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (lds_void *)(stage + 2 * L::kBytes + wave * (kRows * 4)), 4,
          (lane * 8 + wave * 4) | (int)L::outside(t * kRows + lane >= rows), 0, 0, 0);
  };
  if (begin < end) load(begin, smem);
  for (int t = begin; t < end; ++t) {
    const lds_char *const sq = smem + ((t - begin) & 1) * kStage, *const sy = sq + L::kBytes;
    const auto *const stats = (const __attribute__((address_space(3))) float *)(sq + 2 * L::kBytes);
    all_landed<0>();
    if (t + 1 < end) load(t + 1, smem + ((t + 1 - begin) & 1) * kStage);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x16 s, dp;
      float start[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        start[r] = stats[u * 32 + row_in(r, half)];
        s[r] = FMT == kF32 ? 0.f : start[r];
        dp[r] = stats[kRows + u * 32 + row_in(r, half)];
      }
      C::along(s, sq, u, k, lanes);
      C::along(dp, sy, u, v, lanes);
      if constexpr (FMT == kF32) C::template pace_along<2, 8>();
      const int r0 = t * kRows + u * 32;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float p = s[r], ds = dp[r];
        weigh<FMT>(p, ds, start[r], a.scale2);
        s[r] = p;
        dp[r] = ds;
      }
      if (r0 < plain || r0 + 32 > rows) {
        const int lane = lane_again(), half = lane >> 5, key = key0 + wave * 32 + (lane & 31);
        const int first = here(first_row(key) - r0 - 4 * half), last = here(rows - r0 - 4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (row_in(r, 0) < first || row_in(r, 0) >= last) s[r] = dp[r] = 0.f;
      }
      across32<C>(dv, sy, u, s, lanes);
      scaled.hold(dp, dk);
      across32<C>(dk, sq, u, dp, lanes);
      if constexpr (FMT == kF32) C::template pace_across<2>();
    }
  }
  const int lane_now = lane_again(), half_now = lane_now >> 5, key_now = key0 + wave * 32 + (lane_now & 31);
  if (key_now >= at.stored) return;
  if (key_now >= at.nk) {
    // no key: zeros, where a row's infinity or NaN has made NaN of weights of zero
#pragma unroll
    for (int b = 0; b < C::kBlocks; ++b) {
      clear(dk[b]);
      clear(dv[b]);
    }
  }
  store_keys<C, FMT>(a, at, a.dk, 0, head, key_now, dk, half_now, a.scale * scaled.out());
  store_keys<C, FMT>(a, at, a.dv, 1, head, key_now, dv, half_now, FMT == kF16 ? ldexpf(1.f, -kShift) : 1.f);
#endif
}

// dk (y = 0) and dv: the sums of the parts.  One thread per 4 values.
template <int FMT>
__global__ __launch_bounds__(256) void k_join_keys(Args a, FastDiv quads, FastDiv keys, long long rows) {
  constexpr int kSize = FMT == kF32 ? 4 : 2;
  const uint32_t x = blockIdx.x * 256u + threadIdx.x, i = fdiv(x, quads);
  if (i >= rows) return;
  const int d = (int)(x - i * quads.d) * 4;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float4 p = *(const float4 *)(a.part_k + ((2LL * s + blockIdx.y) * rows + i) * a.dim + d);
    v[0] += p.x;
    v[1] += p.y;
    v[2] += p.z;
    v[3] += p.w;
  }
  // row i is key n of a head, of all sequences' keys
  const uint32_t head = fdiv(i, keys), n = i - head * keys.d;
  long long seq = 0, token = n;
  if (!a.q_offsets) {
    seq = n / (uint32_t)a.k_rows;
    token = n - seq * a.k_rows;
  }
  const Mat &to = blockIdx.y ? a.dv : a.dk;
  store4<FMT>(to.p + (seq * to.batch + token * to.row + head * to.head + d) * kSize, v);
}

template <int FMT>
void go_q(const Args &a, hipStream_t st) {
  const dim3 grid((unsigned)a.q_tiles * a.kv_heads);
  if (a.dim <= 64)
    hipLaunchKernelGGL((k_backward_q<FMT, 64>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_backward_q<FMT, 128>), grid, dim3(256), 0, st, a);
}
template <int FMT>
void go_q_few(const Args &a, hipStream_t st) {
  const dim3 grid((unsigned)a.q_tiles * a.kv_heads);
  constexpr int kWaves = FMT == kF32 ? 2 : 4;  // what leaves LDS for two workgroups, or one at 128
  if (a.dim <= 64)
    hipLaunchKernelGGL((k_backward_q_few<FMT, 64, kWaves>), grid, dim3(64 * kWaves), 0, st, a);
  else
    hipLaunchKernelGGL((k_backward_q_few<FMT, 128, kWaves>), grid, dim3(64 * kWaves), 0, st, a);
}
template <int FMT>
void go_kv(const Args &a, hipStream_t st) {
  const dim3 grid((unsigned)a.k_tiles * a.kv_heads, (unsigned)a.splits);
  if (a.dim <= 64)
    hipLaunchKernelGGL((k_backward_kv<FMT, 64>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_backward_kv<FMT, 128>), grid, dim3(256), 0, st, a);
  if (a.splits > 1) {
    const long long keys = (a.q_offsets ? 1LL : a.batch) * a.k_rows, rows = keys * a.kv_heads;
    hipLaunchKernelGGL(k_join_keys<FMT>, dim3((unsigned)((rows * (a.dim / 4) + 255) / 256), 2), dim3(256), 0, st, a,
                       make_fastdiv((uint32_t)a.dim / 4), make_fastdiv((uint32_t)keys), rows);
  }
}

}  // namespace

hipError_t launch_backward_q(const Args &a, int fmt, hipStream_t st) {
  if (!a.q_tiles || !a.kv_heads) return hipSuccess;
  if (fmt == kBf16)
    go_q<kBf16>(a, st);
  else if (fmt == kF16)
    go_q<kF16>(a, st);
  else
    go_q<kF32>(a, st);
  return hipGetLastError();
}

hipError_t launch_backward_q_few(const Args &a, int fmt, hipStream_t st) {
  if (!a.q_tiles || !a.kv_heads) return hipSuccess;
  if (fmt == kBf16)
    go_q_few<kBf16>(a, st);
  else if (fmt == kF16)
    go_q_few<kF16>(a, st);
  else
    go_q_few<kF32>(a, st);
  return hipGetLastError();
}

hipError_t launch_backward_kv(const Args &a, int fmt, hipStream_t st) {
  if (!a.k_tiles || !a.kv_heads) return hipSuccess;
  if (fmt == kBf16)
    go_kv<kBf16>(a, st);
  else if (fmt == kF16)
    go_kv<kF16>(a, st);
  else
    go_kv<kF32>(a, st);
  return hipGetLastError();
}

}  // namespace attend
}  // namespace pdr
