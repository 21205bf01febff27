// attention_forward.hip -- softmax(scale q k^T) v, in one pass over the keys.
//
// A lane (with its other half) owns one query: scores come out of the matrix
// cores with keys in registers, so a running maximum and sum need one exchange
// between halves a tile, and the weights go back in as they are.
#include <type_traits>

#include "attention.hpp"

namespace pdr {
namespace attend {

namespace {

// The running softmax of a lane's query, in units of log2, and the sums of
// values under it.  `most` follows the maximum only when that has grown by more
// than kSlack: weights of up to 2^8 are as good as those up to 1, in sums of fp32
// and in the operands' range, and nearly all tiles are spared a pass over the sums.
// fp16 weights enter the products times 2^12, so that the smallest are kept to 2^-37 of
// the largest and not to 2^-25, which many keys' sum would show (65536 keys, all but
// one of them 2^-24.5 of it: 0.0027 came out as 0.0039); what is left of the range, to
// 2^16, is for a slack of 3 (with 2^14 and 1 there are more passes over the sums: 8 x 4096,
// 16 heads of 128, 640 us instead of 614).
template <int FMT>
constexpr float kUp = FMT == kF16 ? 12.f : 0.f;  // log2 of that
template <int FMT>
constexpr float kSlack = FMT == kF16 ? 3.f : 8.f;
template <class C>
struct Query {
  f32x16 out[C::kBlocks];
  float most, sum;  // sum: of this half's keys

  __device__ __forceinline__ void init() {
    most = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int b = 0; b < C::kBlocks; ++b) clear(out[b]);
  }
  // Scores of 32 N keys to weights, in place.
  template <int N>
  __device__ __forceinline__ void weigh(f32x16 (&s)[N], float scale2) {
    float m = s[0][0];
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) m = fmaxf(m, s[u][r]);
    m = fmaxf(m, other_half(m)) * scale2;
    const bool grows = m > most + kSlack<C::kFmt>;
    if (__any(grows)) {
      // another query's maximum changes nothing here; a lane that has seen nothing yet has no sums
      const float up = grows ? m : most, down = up == -INFINITY ? 1.f : exp2_(most - up);
      most = up;
      sum *= down;
#pragma unroll
      for (int b = 0; b < C::kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) out[b][r] *= down;
    }
    const float from = most == -INFINITY ? 0.f : most - kUp<C::kFmt>;  // nothing seen yet
    // a tile's sum first: beside a key that takes most of the weight each of many small
    // ones would be rounded at its magnitude (65536 keys: 1.4e-3 of the sum)
    float tile = 0.f;
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[u][r] = exp2_(fmaf(s[u][r], scale2, -from));
        tile += s[u][r];
      }
    sum += tile;
  }
  // The same where masks may hide what is not finite; `seen` as of mask().
  template <int N>
  __device__ __forceinline__ void take_carefully(const lds_char *values, const f32x16 (&s)[N],
                                                 const typename C::Lane &at, int half, int seen) {
#pragma unroll
    for (int u = 0; u < N; ++u) C::across_careful(out, values, u, s[u], at, half, seen - 32 * u);
  }
  // 32 N keys' values under these weights.
  template <int N>
  __device__ __forceinline__ void take(const lds_char *values, const f32x16 (&s)[N], const typename C::Lane &at) {
#pragma unroll
    for (int x = 0; x < 2 * N; ++x) C::across(out, values, x, C::pack(s[x >> 1], (x & 1) * 8), at);
  }
};

// What a query's sums are to be multiplied by, and its lse.  A query without
// keys has neither maximum nor sum; with NaN scores it has a sum.
__device__ __forceinline__ float weight_of(float most, float sum) {
  return most == -INFINITY && sum == 0.f ? 0.f : 1.f / sum;
}
template <int FMT>
__device__ __forceinline__ float lse_of(float most, float sum) {
  return most == -INFINITY && sum == 0.f ? INFINITY : most + (__log2f(sum) - kUp<FMT>);
}

// Scores of keys that the lane's query does not see; `seen` counts from the tile's
// first key of this half.
__device__ __forceinline__ void mask(f32x16 &s, int key0, int seen) {
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (key0 + row_in(r, 0) >= seen) s[r] = -INFINITY;
}

// What a lane needs to know of its row.
struct Row {
  bool there;
  int token, in_group;
  int seen;   // keys that it sees: those below
  __device__ __forceinline__ Row(const Args &a, const Place &at, int row, int rows) {
    there = row < rows;
    const int r = there ? row : rows - 1;
    token = (int)fdiv((uint32_t)r, a.group);
    in_group = r - token * (int)a.group.d;
    seen = at.nk;
    if (a.causal && token + at.nk - at.nq + 1 < seen) seen = token + at.nk - at.nq + 1;
  }
};
// Keys that a row of the tile sees.
__device__ __forceinline__ int keys_of(const Args &a, const Place &at, int last_row, int rows) {
  if (!a.causal) return at.nk;
  const int k = (int)fdiv((uint32_t)(last_row < rows ? last_row : rows - 1), a.group) + at.nk - at.nq + 1;
  return k < 0 ? 0 : k;
}
__device__ __forceinline__ char *row_at(const Mat &m, const Place &at, const Row &r, int head, int group,
                                        int size) {
  return m.p + (first_of(m, at, at.q0 + r.token, head * group) + r.in_group * m.head) * size;
}
// A row's place among all queries' rows.
__device__ __forceinline__ long long rows_before(const Args &a, const Place &at, int head) {
  const long long all = a.q_offsets ? a.q_rows : (long long)a.batch * a.q_rows;
  return (head * all + (a.q_offsets ? 0 : (long long)at.seq * a.q_rows) + at.q0) * a.group.d;
}

// 128 rows to a workgroup, 32 to a wave; the waves share tiles of 64 keys, the next of
// which is on its way.  A tile costs two products and an exponential a pair, which the
// other wave of the SIMD works on meanwhile (256 registers a lane leave room for two).
// Bound by the matrix cores at the clock that the card's power allows, 2.0 of 2.4 GHz:
// bf16, a prompt of 16384 tokens with 16 heads of 128, 1040 us, 1.06 PFLOP/s; packed
// sequences of up to 4096, 410 us, 0.86; 8 x 1024 with 12 heads of 64, where there are
// twice as many exponentials to a product, 41 us.
template <int FMT, int DP>
__global__ __launch_bounds__(256, FMT == kF32 ? 1 : 2) void k_forward(Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Core<FMT, DP>;
  constexpr int kKeys = 64;
  using L = Loader<C, kKeys, 4>;
  __shared__ __align__(1024) char shared[4 * L::kBytes];
  lds_char *const smem = (lds_char *)shared;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // heads change fastest, so that an XCD's workgroups share few heads' keys;
  // where queries see what is before them, the longest tiles go first
  const int unit = (int)fdiv(blockIdx.x, a.heads), head = blockIdx.x - unit * a.kv_heads;
  const Place at = place<kLogWide, false>(a, a.causal ? a.q_tiles - 1 - unit : unit);
  const int group = (int)a.group.d, rows = at.nq * group;
  const int row0 = at.tile << kLogWide, mine = row0 + wave * 32;
  if (at.tile < 0 || row0 >= rows) return;
  const Row row(a, at, mine + (lane & 31), rows);
  const int keys = keys_of(a, at, row0 + 127, rows), plain = keys_of(a, at, row0, rows);

  i32x4 q[C::kSteps];
  C::fetch_row(q, row_at(a.q, at, row, head, group, C::kSize), a.dim, half, row.there);
  typename C::Lane lanes;
  lanes.init(lane);
  Query<C> query;
  query.init();
  const Source k(a.k, first_of(a.k, at, at.k0, head), C::kSize), v(a.v, first_of(a.v, at, at.k0, head), C::kSize);
  L load;
  load.init(a.dim, wave, lane);
  const int tiles = (keys + kKeys - 1) / kKeys;
  if (tiles > 0) {
    load.tokens(k, v, 0, at.nk, smem);
  }
  // Tile t: scores, weights, sums of values.
  auto turn = [&](int t, auto masked) {
    const lds_char *const sk = smem + (t & 1) * (2 * L::kBytes), *const sv = sk + L::kBytes;
    all_landed<0>();
    if (t + 1 < tiles) {
      lds_char *const next = smem + ((t + 1) & 1) * (2 * L::kBytes);
      load.tokens(k, v, (t + 1) * kKeys, at.nk, next);
    }
    f32x16 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      clear(s[u]);
      C::along(s[u], sk, u, q, lanes);
    }
    C::template pace_along<2>();
    if constexpr (decltype(masked)::value) {
      const int seen = row.seen - t * kKeys;
#pragma unroll
      for (int u = 0; u < 2; ++u) mask(s[u], u * 32, seen - 4 * half);
      query.template weigh<2>(s, a.scale2);
      if (C::any_not_finite(sv, 0, lane) || C::any_not_finite(sv, 1, lane))
        query.template take_carefully<2>(sv, s, lanes, half, seen);
      else
        query.template take<2>(sv, s, lanes);
    } else {
      query.template weigh<2>(s, a.scale2);
      query.template take<2>(sv, s, lanes);
      C::template pace_across<2>();
    }
  };
  // tiles that all rows of the workgroup see, and the others
  const int whole = plain / kKeys < tiles ? plain / kKeys : tiles;
  int t = 0;
  for (; t < whole; ++t) turn(t, std::false_type());
  for (; t < tiles; ++t) turn(t, std::true_type());
  const float sum = query.sum + other_half(query.sum);
  if (!row.there) return;
  if (a.lse && half == 0)
    a.lse[rows_before(a, at, head) + mine + (lane & 31)] = lse_of<FMT>(query.most, sum);
  store_columns<C, FMT>(query.out, row_at(a.o, at, row, head, group, C::kSize), a.dim, half,
                        weight_of(query.most, sum));
#endif
}

// Few queries: 32 rows to a workgroup, whose waves take parts of the keys each,
// in LDS of their own; workgroups along y take further parts, joined below.  Keys
// go straight to registers (a lane's chunks of one row are what along() wants),
// so that only values take up LDS and two workgroups' loads are in flight on a
// compute unit.  Bound by memory where the cache is long (bf16, 16 sequences of up to
// 32768 keys, 8 key heads of 128: 268 us, 4.8 TB/s, and 7 to join 16 parts), by latency
// where it is short (one sequence of 1024 keys: 9.4 us, of which about 5 are a launch and
// the first loads).
template <int FMT, int DP, int NW>
__global__ __launch_bounds__(64 * NW, FMT == kF32 && DP > 64 ? 1 : 2) void k_forward_few(Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Core<FMT, DP>;
  constexpr int kKeys = 32;
  using L = Loader<C, kKeys, 1>;
  constexpr int kRing = 2 * L::kBytes;
  static_assert(kRing >= 32 * DP * 4, "a wave's sums fit where its values were");
  __shared__ __align__(1024) char shared[NW * kRing];
  lds_char *const smem = (lds_char *)shared;
  __shared__ float stats[NW][32][2];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = (int)fdiv(blockIdx.x, a.heads), head = blockIdx.x - unit * a.kv_heads;
  const Place at = place<kLogFew, false>(a, a.causal ? a.q_tiles - 1 - unit : unit);
  const int group = (int)a.group.d, rows = at.nq * group;
  const int row0 = at.tile << kLogFew;
  if (at.tile < 0 || row0 >= rows) return;
  const Row row(a, at, row0 + (lane & 31), rows);
  const int keys = keys_of(a, at, row0 + 31, rows), plain = keys_of(a, at, row0, rows);

  typename C::Lane lanes;
  lanes.init(lane);
  Query<C> query;
  query.init();
  const Source k(a.k, first_of(a.k, at, at.k0, head), C::kSize), v(a.v, first_of(a.v, at, at.k0, head), C::kSize);
  L load;
  load.init(a.dim, 0, lane);
  lds_char *const ring = smem + wave * kRing;
  // this wave's tiles
  const int all = (keys + kKeys - 1) / kKeys, parts = a.splits * NW;
  const int each = (all + parts - 1) / parts, part = blockIdx.y * NW + wave;
  const int begin = part * each < all ? part * each : all;
  const int end = begin + each < all ? begin + each : all;
  i32x4 keys_now[C::kSteps], keys_next[C::kSteps], q[C::kSteps];
  C::fetch_row(q, row_at(a.q, at, row, head, group, C::kSize), a.dim, half, row.there);
  if (begin < end) {
    C::fetch_rows(keys_now, k, begin * kKeys, at.nk, a.dim, lane);
    load.tokens(v, begin * kKeys, at.nk, ring);
  }
  // The compiler waits for these here; left to the loop, it would wait in each turn for
  // all that is in flight, the next tile included.
#pragma unroll
  for (int i = 0; i < C::kSteps; ++i) asm volatile("" : "+v"(q[i]), "+v"(keys_now[i]));
  for (int t = begin; t < end; ++t) {
    const lds_char *const sv = ring + ((t - begin) & 1) * L::kBytes;
    if (t + 1 < end) {
      landed<C::kSteps + L::kIssues>();  // the last tile's reads of LDS are done
      C::fetch_rows(keys_next, k, (t + 1) * kKeys, at.nk, a.dim, lane);
      load.tokens(v, (t + 1) * kKeys, at.nk, ring + ((t + 1 - begin) & 1) * L::kBytes);
      landed<C::kSteps + L::kIssues>();
    } else {
      landed<0>();
    }
    f32x16 s[1];
    clear(s[0]);
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) s[0] = C::go(keys_now[i], q[i], s[0]);
    bool careful = false;
    if ((t + 1) * kKeys > plain) {
      mask(s[0], 0, here(row.seen - t * kKeys - 4 * half));
      careful = C::any_not_finite(sv, 0, lane);
    }
    query.template weigh<1>(s, a.scale2);
    if (careful) {
      query.template take_carefully<1>(sv, s, lanes, half, row.seen - t * kKeys);
    } else {
      query.template take<1>(sv, s, lanes);
      C::template pace_across<1>();
    }
#pragma unroll
    for (int i = 0; i < C::kSteps; ++i) keys_now[i] = keys_next[i];
  }
  const float sum = query.sum + other_half(query.sum);
  __syncthreads();
  if (half == 0) {
    stats[wave][lane][0] = query.most;
    stats[wave][lane][1] = sum;
  }
#pragma unroll
  for (int b = 0; b < C::kBlocks; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *(float4 *)(shared + wave * kRing + (lane & 31) * (DP * 4) + (((b * 32 + row_in(r, half)) / 4 ^ (lane & 7)) * 16)) =
          make_float4(query.out[b][r], query.out[b][r + 1], query.out[b][r + 2], query.out[b][r + 3]);
  __syncthreads();
  constexpr int kQuads = DP / 4;
  const long long before = rows_before(a, at, head) + row0;
  for (int x = threadIdx.x; x < 32 * kQuads; x += 64 * NW) {
    const int i = x / kQuads, d = x % kQuads * 4;
    if (row0 + i >= rows || d >= a.dim) continue;
    float most = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) most = fmaxf(most, stats[w][i][0]);
    const float from = most == -INFINITY ? 0.f : most;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, total = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float by = exp2_(stats[w][i][0] - from);
      const float4 o = *(const float4 *)(shared + w * kRing + i * (DP * 4) + ((d / 4 ^ (i & 7)) * 16));
      total = fmaf(stats[w][i][1], by, total);
      v[0] = fmaf(o.x, by, v[0]);
      v[1] = fmaf(o.y, by, v[1]);
      v[2] = fmaf(o.z, by, v[2]);
      v[3] = fmaf(o.w, by, v[3]);
    }
    if (a.splits > 1) {
      const long long all_rows =
          (long long)a.kv_heads * group * (a.q_offsets ? a.q_rows : (long long)a.batch * a.q_rows);
      const long long to = blockIdx.y * all_rows + before + i;
      *(float4 *)(a.part_o + to * a.dim + d) = make_float4(v[0], v[1], v[2], v[3]);
      if (d == 0) *(float2 *)(a.part_ml + to * 2) = make_float2(most, total);
    } else {
      const float by = weight_of(most, total);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= by;
      const Row r(a, at, row0 + i, rows);
      store4<FMT>(row_at(a.o, at, r, head, group, C::kSize) + d * C::kSize, v);
      if (a.lse && d == 0) a.lse[before + i] = lse_of<FMT>(most, total);
    }
  }
#endif
}

// Sums of the parts.  One thread per 4 values of a row.
template <int FMT>
__global__ __launch_bounds__(256) void k_join(Args a, FastDiv quads, FastDiv rows_each, uint32_t rows) {
  constexpr int kSize = FMT == kF32 ? 4 : 2;
  const uint32_t x = blockIdx.x * 256u + threadIdx.x;
  const uint32_t i = fdiv(x, quads);
  if (i >= rows) return;
  const int d = (int)(x - i * quads.d) * 4;
  float most = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) most = fmaxf(most, a.part_ml[(s * (long long)rows + i) * 2]);
  const float from = most == -INFINITY ? 0.f : most;
  float v[4] = {0.f, 0.f, 0.f, 0.f}, total = 0.f;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const long long at = s * (long long)rows + i;
    const float2 ml = *(const float2 *)(a.part_ml + at * 2);
    const float4 o = *(const float4 *)(a.part_o + at * a.dim + d);
    const float by = exp2_(ml.x - from);
    total = fmaf(ml.y, by, total);
    v[0] = fmaf(o.x, by, v[0]);
    v[1] = fmaf(o.y, by, v[1]);
    v[2] = fmaf(o.z, by, v[2]);
    v[3] = fmaf(o.w, by, v[3]);
  }
  const float by = weight_of(most, total);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= by;
  if (a.lse && d == 0) a.lse[i] = lse_of<FMT>(most, total);
  // row i is head g of token n, for a key head
  const uint32_t head = fdiv(i, rows_each), in = i - head * rows_each.d;
  const uint32_t token = fdiv(in, a.group), g = in - token * a.group.d;
  long long seq = 0, n = token;
  if (!a.q_offsets) {
    seq = token / (uint32_t)a.q_rows;
    n = token - seq * a.q_rows;
  }
  store4<FMT>(a.o.p + (seq * a.o.batch + n * a.o.row + (head * a.group.d + g) * a.o.head + d) * kSize, v);
}

template <int FMT>
void go(const Args &a, hipStream_t st) {
  const dim3 grid((unsigned)a.q_tiles * a.kv_heads);
  if (a.dim <= 64)
    hipLaunchKernelGGL((k_forward<FMT, 64>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_forward<FMT, 128>), grid, dim3(256), 0, st, a);
}
template <int FMT, int DP>
void go_few(const Args &a, hipStream_t st) {
  const dim3 grid((unsigned)a.q_tiles * a.kv_heads, (unsigned)a.splits);
  if constexpr (FMT != kF32 || DP == 64) {  // fp32 rows of 128: LDS for four waves
    if (a.waves == 8) {
      hipLaunchKernelGGL((k_forward_few<FMT, DP, 8>), grid, dim3(512), 0, st, a);
      return;
    }
  }
  hipLaunchKernelGGL((k_forward_few<FMT, DP, 4>), grid, dim3(256), 0, st, a);
}
template <int FMT>
void go_few(const Args &a, long long rows, hipStream_t st) {
  if (a.dim <= 64)
    go_few<FMT, 64>(a, st);
  else
    go_few<FMT, 128>(a, st);
  if (a.splits > 1)
    hipLaunchKernelGGL(k_join<FMT>, dim3((unsigned)((rows * (a.dim / 4) + 255) / 256)), dim3(256), 0, st, a,
                       make_fastdiv((uint32_t)a.dim / 4), make_fastdiv((uint32_t)(rows / a.kv_heads)),
                       (uint32_t)rows);
}

}  // namespace

hipError_t launch_forward(const Args &a, int fmt, hipStream_t st) {
  if (!a.q_tiles || !a.kv_heads) return hipSuccess;
  if (fmt == kBf16)
    go<kBf16>(a, st);
  else if (fmt == kF16)
    go<kF16>(a, st);
  else
    go<kF32>(a, st);
  return hipGetLastError();
}

hipError_t launch_forward_few(const Args &a, int fmt, hipStream_t st) {
  const long long rows =
      (a.q_offsets ? 1LL : a.batch) * a.q_rows * a.kv_heads * (long long)a.group.d;
  if (!rows) return hipSuccess;
  if (fmt == kBf16)
    go_few<kBf16>(a, rows, st);
  else if (fmt == kF16)
    go_few<kF16>(a, rows, st);
  else
    go_few<kF32>(a, rows, st);
  return hipGetLastError();
}

}  // namespace attend
}  // namespace pdr
