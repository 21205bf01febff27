// blocks.hip -- the operators of include/pdr_blocks.h: argument checks,
// workspaces and the order of launches.
#include <math.h>
#include <stdint.h>

#include "attention.hpp"
#include "attention_plan.hpp"
#include "norm.hpp"
#include "pdr_blocks.h"

using namespace pdr;

namespace {

using dense::fmt_bytes;
using dense::kF32;

bool good_fmt(int f) { return f == dense::kF32 || f == dense::kF16 || f == dense::kBf16; }
bool good_len(long long n) { return n >= 0 && n <= 0x7fffffffLL - 256; }
bool good_ptr(const void *p, int fmt) { return ((uintptr_t)p & (uintptr_t)(fmt_bytes(fmt) - 1)) == 0; }
bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

int in_workspace(long long need, void *workspace, size_t bytes) {
  return need > 0 && (!workspace || !aligned(workspace, 256) || bytes < (size_t)need) ? PDR_ERR_WORKSPACE : PDR_OK;
}
int status(hipError_t e) { return e == hipSuccess ? PDR_OK : PDR_ERR_HIP; }

// ---------------------------------------------------------------- attention

using attend::Args;
using attend::Mat;
using attend::Sizes;
using attend::takes_few;

// A tensor of the call: `heads` heads over `rows` tokens (of each sequence).
bool good_tensor(const pdr_attention &p, const void *t, long long row, long long head, long long batch,
                 long long rows, long long heads) {
  if (!rows || (!p.q_offsets && !p.batch)) return true;
  const long long per = 16 / fmt_bytes(p.fmt);
  if (!t || !aligned(t, 16)) return false;
  if (row < 0 || head < 0 || batch < 0 || row % per || head % per || batch % per) return false;
  return row <= attend::kMaxRow && head <= attend::kMaxHead && head * (heads - 1) <= attend::kMaxHeads &&
         batch < 1LL << 40;
}

int check_attention(const pdr_attention *p, bool backward) {
  if (!p || !good_fmt(p->fmt)) return PDR_ERR_INVALID_ARG;
  if (!good_len(p->batch) || !good_len(p->q_rows) || !good_len(p->k_rows)) return PDR_ERR_INVALID_ARG;
  if (p->kv_heads < 1 || p->kv_heads > 65536 || p->heads < 1 || p->heads > 65536 || p->heads % p->kv_heads)
    return PDR_ERR_INVALID_ARG;
  if (p->dim < 1 || p->dim > 128 || p->dim % (16 / fmt_bytes(p->fmt))) return PDR_ERR_INVALID_ARG;
  // the backward's sums start from lse / scale, which has to be finite
  if (!(p->scale >= 0x1p-64f) || !(p->scale <= 0x1p64f)) return PDR_ERR_INVALID_ARG;
  const bool packed = p->q_offsets != nullptr;
  if (packed != (p->k_offsets != nullptr) || (packed && p->key_lengths)) return PDR_ERR_INVALID_ARG;
  if (!aligned(p->q_offsets, 4) || !aligned(p->k_offsets, 4) || !aligned(p->key_lengths, 4) || !aligned(p->lse, 4))
    return PDR_ERR_INVALID_ARG;
  const __int128 seqs = packed ? 1 : p->batch;
  if (seqs * p->q_rows * p->heads >= 1 << 29 || (__int128)p->batch * p->kv_heads >= 1 << 23)
    return PDR_ERR_INVALID_ARG;
  const auto &a = *p;
  if (!good_tensor(a, a.q, a.q_row, a.q_head, a.q_batch, a.q_rows, a.heads) ||
      !good_tensor(a, a.k, a.k_row, a.k_head, a.k_batch, a.k_rows, a.kv_heads) ||
      !good_tensor(a, a.v, a.v_row, a.v_head, a.v_batch, a.k_rows, a.kv_heads) ||
      !good_tensor(a, a.o, a.o_row, a.o_head, a.o_batch, a.q_rows, a.heads))
    return PDR_ERR_INVALID_ARG;
  if (!backward) return PDR_OK;
  const bool queries = seqs && p->q_rows;
  if (queries && !p->lse) return PDR_ERR_INVALID_ARG;
  if (!p->dk != !p->dv || seqs * p->k_rows * p->kv_heads >= 1 << 29) return PDR_ERR_INVALID_ARG;
  if (!good_tensor(a, a.dy, a.dy_row, a.dy_head, a.dy_batch, a.q_rows, a.heads)) return PDR_ERR_INVALID_ARG;
  if (a.dq && !good_tensor(a, a.dq, a.dq_row, a.dq_head, a.dq_batch, a.q_rows, a.heads)) return PDR_ERR_INVALID_ARG;
  if (a.dk && (!good_tensor(a, a.dk, a.dk_row, a.dk_head, a.dk_batch, a.k_rows, a.kv_heads) ||
               !good_tensor(a, a.dv, a.dv_row, a.dv_head, a.dv_batch, a.k_rows, a.kv_heads)))
    return PDR_ERR_INVALID_ARG;
  return PDR_OK;
}

Mat mat(const void *p, long long row, long long head, long long batch) {
  return {(char *)const_cast<void *>(p), row, head, batch};
}

Args args_of(const pdr_attention &p) {
  Args a = {};
  a.q = mat(p.q, p.q_row, p.q_head, p.q_batch);
  a.k = mat(p.k, p.k_row, p.k_head, p.k_batch);
  a.v = mat(p.v, p.v_row, p.v_head, p.v_batch);
  a.o = mat(p.o, p.o_row, p.o_head, p.o_batch);
  a.dy = mat(p.dy, p.dy_row, p.dy_head, p.dy_batch);
  a.dq = mat(p.dq, p.dq_row, p.dq_head, p.dq_batch);
  a.dk = mat(p.dk, p.dk_row, p.dk_head, p.dk_batch);
  a.dv = mat(p.dv, p.dv_row, p.dv_head, p.dv_batch);
  a.q_offsets = p.q_offsets;
  a.k_offsets = p.k_offsets;
  a.key_lengths = p.key_lengths;
  a.lse = p.lse;
  a.scale = p.scale;
  a.scale2 = (float)(p.scale * 1.4426950408889634);
  a.causal = p.causal != 0;
  a.batch = (int)p.batch;
  a.kv_heads = (int)p.kv_heads;
  a.dim = (int)p.dim;
  a.q_rows = (int)p.q_rows;
  a.k_rows = (int)p.k_rows;
  a.splits = 1;
  a.per_tile = make_fastdiv((uint32_t)(p.batch > 0 ? p.batch : 1));
  a.group = make_fastdiv((uint32_t)(p.heads / p.kv_heads));
  a.heads = make_fastdiv((uint32_t)p.kv_heads);
  return a;
}

// Tiles of 2^log rows, `each` to a token, of all sequences (attention.hpp).
int tiles_of(const pdr_attention &p, long long tokens, long long each, int log) {
  if (p.q_offsets) return (int)((tokens * each >> log) + p.batch + 2);
  return (int)(((tokens * each + (1 << log) - 1) >> log) * p.batch);
}

constexpr long long kFewUnits = 512;       // workgroups of 32 rows to aim for: two to a compute unit,
constexpr long long kUnequalUnits = 2048;  // and of sequences of different lengths (a cache of 16 sequences up
                                           // to 32768 keys: 4 parts 298 us, 16 parts 272)
constexpr long long kFewKeys = 256;        // keys of a workgroup, at least
constexpr long long kAlone = 1024;         // keys that one workgroup takes without a join

struct Plan {
  bool few;
  int waves, splits;
  size_t part_o, part_ml;  // bytes
};

// Few queries: several workgroups over the keys until the card has work.
Plan plan_of(const pdr_attention &p) {
  const Sizes n(p);
  const long long units = (n.rows + 31) / 32 * n.seqs * p.kv_heads;
  Plan plan = {takes_few(p), 4, 1, 0, 0};
  if (!plan.few || !n.rows) return plan;
  if (n.keys <= kAlone) {
    // eight waves where that leaves one workgroup to a compute unit; their LDS holds no fp32 rows of 128
    if (units < 512 && !(p.fmt == kF32 && p.dim > 64)) plan.waves = 8;
    return plan;
  }
  const long long aim = p.q_offsets || p.key_lengths ? kUnequalUnits : kFewUnits;
  long long splits = (aim + units - 1) / units;
  const long long most = (n.keys + kFewKeys - 1) / kFewKeys;
  if (splits > most) splits = most;
  plan.splits = (int)(splits < 1 ? 1 : splits);
  if (plan.splits > 1) {
    const size_t all = (size_t)(p.q_offsets ? 1 : p.batch) * p.q_rows * p.heads * plan.splits;
    plan.part_o = round256(all * p.dim * 4);
    plan.part_ml = round256(all * 8);
  }
  return plan;
}

// Parts that the rows are cut into for dk and dv, until the card has work; the
// bytes of their sums.  All gradients, us, with parts of at least 64, 128 and 256 rows, and
// of 128 with 1024 workgroups to aim for:
//   fp16 7 packed, up to 777, 6 heads of 72, 2 of keys    48   59   80   58
//   bf16 2 x 512, 8 heads of 128                          47   40   43   40
//   bf16 2048, 4 heads of 64                              46   46   46   55
//   fp16 4 x 300, 4 heads of 64                           24   23   23   23
//   fp32 4 x 1024, 8 heads of 64                         179  179  179  204
//   fp32 2 x 700, 6 heads of 128, 3 of keys, not causal  256  251  257  250
//   bf16 8 x 1024, 12 heads of 64, not causal            109  109  110  134
//   bf16 16384, 2 heads of 128, 1 of keys                765  765  765  738
constexpr long long kKeyUnits = 512;  // workgroups of 128 keys to aim for
constexpr long long kKeyRows = 128;   // rows of a part, at least
int key_splits(const pdr_attention &p, size_t *bytes) {
  *bytes = 0;
  const Sizes n(p);
  const long long units = (n.keys + 127) / 128 * n.seqs * p.kv_heads;
  if (!p.dk || !units) return 1;
  long long splits = (kKeyUnits + units - 1) / units;
  if (splits > n.rows / kKeyRows) splits = n.rows / kKeyRows;
  if (splits <= 1) return 1;
  *bytes = round256((size_t)(p.q_offsets ? 1 : p.batch) * p.k_rows * p.kv_heads * p.dim * splits * 8);
  return (int)splits;
}

long long tokens_of(const pdr_attention &p) { return (p.q_offsets ? 1 : p.batch) * p.q_rows; }
// Bytes of a value for each query and head.
size_t row_values(const pdr_attention &p) { return round256((size_t)tokens_of(p) * p.heads * 4); }

// ------------------------------------------------------- layer norm, dropout

bool good_rows(const void *p, long long ld, long long rows, long long cols, int fmt) {
  if (!rows || !cols) return true;
  return p && good_ptr(p, fmt) && ld >= (rows > 1 ? cols : 0) && ld < 1LL << 40;
}

int check_norm(const pdr_layer_norm *p, bool backward) {
  if (!p || !good_fmt(p->fmt) || !good_len(p->rows) || p->cols < 0 || p->cols > norm::kMaxCols)
    return PDR_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !(p->eps < INFINITY)) return PDR_ERR_INVALID_ARG;
  if (!good_rows(p->x, p->ldx, p->rows, p->cols, p->fmt) || !good_ptr(p->weight, p->fmt) ||
      !good_ptr(p->bias, p->fmt) || !aligned(p->stats, 8))
    return PDR_ERR_INVALID_ARG;
  if (!backward) return good_rows(p->y, p->ldy, p->rows, p->cols, p->fmt) ? PDR_OK : PDR_ERR_INVALID_ARG;
  if (!good_rows(p->dy, p->lddy, p->rows, p->cols, p->fmt) || (p->rows && p->cols && !p->stats))
    return PDR_ERR_INVALID_ARG;
  if (p->dx && !good_rows(p->dx, p->lddx, p->rows, p->cols, p->fmt)) return PDR_ERR_INVALID_ARG;
  return good_ptr(p->dweight, p->fmt) && good_ptr(p->dbias, p->fmt) ? PDR_OK : PDR_ERR_INVALID_ARG;
}

norm::Norm norm_of(const pdr_layer_norm &p, bool backward) {
  norm::Norm a = {};
  a.x = p.x;
  a.weight = p.weight;
  a.bias = backward ? nullptr : p.bias;
  a.rows = p.rows;
  a.cols = (int)p.cols;
  a.fmt = p.fmt;
  a.eps = p.eps;
  a.by_cols = p.cols ? (float)(1.0 / (double)p.cols) : 0.f;
  a.stats = p.stats;
  a.ldx = p.ldx;
  uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.weight | (uintptr_t)a.bias;
  long long lens = p.cols | p.ldx;
  if (backward) {
    a.dy = p.dy;
    a.dx = p.dx;
    a.dweight = p.dweight;
    a.dbias = p.dbias;
    a.lddy = p.lddy;
    a.lddx = p.lddx;
    bits |= (uintptr_t)a.dy | (uintptr_t)a.dx;
    lens |= p.lddy | (p.dx ? p.lddx : 0);
  } else {
    a.y = p.y;
    a.ldy = p.ldy;
    bits |= (uintptr_t)a.y;
    lens |= p.ldy;
  }
  a.vec = (bits & 15) == 0 && (lens & 7) == 0;
  return a;
}

// Bytes of the blocks' sums, and of what there is of each row for dweight.
size_t norm_parts(const pdr_layer_norm &p) {
  if ((!p.dweight && !p.dbias) || !p.rows || !p.cols) return 0;
  return 2 * (size_t)norm::norm_blocks(p.rows, p.cols) * p.cols * 4;
}
size_t norm_offsets(const pdr_layer_norm &p) {
  return p.dweight && p.cols ? 4 * (size_t)norm::norm_offsets(p.rows, p.cols) : 0;
}

int check_dropout(const pdr_dropout_args *p) {
  if (!p || !good_fmt(p->fmt) || p->rows < 0 || p->cols < 0 || (__int128)p->rows * p->cols >= 1LL << 40)
    return PDR_ERR_INVALID_ARG;
  if (!(p->p >= 0.0 && p->p <= 1.0) || !aligned(p->seed_at, 8)) return PDR_ERR_INVALID_ARG;
  if (!good_rows(p->x, p->ldx, p->rows, p->cols, p->fmt) || !good_rows(p->y, p->ldy, p->rows, p->cols, p->fmt) ||
      (p->res && !good_rows(p->res, p->ldr, p->rows, p->cols, p->fmt)))
    return PDR_ERR_INVALID_ARG;
  return PDR_OK;
}

}  // namespace

extern "C" {

long long pdr_attention_forward_workspace_bytes(const pdr_attention *p) {
  const int rc = check_attention(p, false);
  if (rc != PDR_OK) return rc;
  const Plan plan = plan_of(*p);
  return (long long)(plan.part_o + plan.part_ml);
}
int pdr_attention_forward(const pdr_attention *p, void *workspace, size_t workspace_bytes, void *stream) {
  int rc = check_attention(p, false);
  if (rc != PDR_OK) return rc;
  const Plan plan = plan_of(*p);
  rc = in_workspace((long long)(plan.part_o + plan.part_ml), workspace, workspace_bytes);
  if (rc != PDR_OK) return rc;
  if (!tokens_of(*p)) return PDR_OK;
  Args a = args_of(*p);
  a.q_tiles = tiles_of(*p, p->q_rows, p->heads / p->kv_heads, plan.few ? attend::kLogFew : attend::kLogWide);
  if (!plan.few) return status(attend::launch_forward(a, p->fmt, (hipStream_t)stream));
  a.splits = plan.splits;
  a.waves = plan.waves;
  a.part_o = (float *)workspace;
  a.part_ml = (float *)((char *)workspace + plan.part_o);
  return status(attend::launch_forward_few(a, p->fmt, (hipStream_t)stream));
}

long long pdr_attention_backward_workspace_bytes(const pdr_attention *p) {
  const int rc = check_attention(p, true);
  if (rc != PDR_OK) return rc;
  size_t parts;
  key_splits(*p, &parts);
  return (long long)(2 * row_values(*p) + parts);
}
int pdr_attention_backward(const pdr_attention *p, void *workspace, size_t workspace_bytes, void *stream) {
  const long long need = pdr_attention_backward_workspace_bytes(p);
  if (need < 0) return (int)need;
  const int rc = in_workspace(need, workspace, workspace_bytes);
  if (rc != PDR_OK) return rc;
  const hipStream_t st = (hipStream_t)stream;
  Args a = args_of(*p);
  a.starts = (float *)workspace;
  a.part_k = (float *)((char *)workspace + 2 * row_values(*p));
  hipError_t e = hipSuccess;
  if (tokens_of(*p)) {
    const bool few = takes_few(*p);
    a.q_tiles = tiles_of(*p, p->q_rows, p->heads / p->kv_heads, few ? attend::kLogFew : attend::kLogWide);
    e = few ? attend::launch_backward_q_few(a, p->fmt, st) : attend::launch_backward_q(a, p->fmt, st);
  }
  if (e == hipSuccess && p->dk) {
    size_t parts;
    a.splits = key_splits(*p, &parts);
    a.k_tiles = tiles_of(*p, p->k_rows, 1, attend::kLogWide);
    e = attend::launch_backward_kv(a, p->fmt, st);
  }
  return status(e);
}

long long pdr_layer_norm_forward_workspace_bytes(const pdr_layer_norm *p) { return check_norm(p, false); }
int pdr_layer_norm_forward(const pdr_layer_norm *p, void *, size_t, void *stream) {
  const int rc = check_norm(p, false);
  return rc != PDR_OK ? rc : status(norm::launch_norm(norm_of(*p, false), (hipStream_t)stream));
}
long long pdr_layer_norm_backward_workspace_bytes(const pdr_layer_norm *p) {
  const int rc = check_norm(p, true);
  return rc != PDR_OK ? rc : (long long)(norm_parts(*p) + norm_offsets(*p));
}
int pdr_layer_norm_backward(const pdr_layer_norm *p, void *workspace, size_t workspace_bytes, void *stream) {
  const long long need = pdr_layer_norm_backward_workspace_bytes(p);
  if (need < 0) return (int)need;
  const int rc = in_workspace(need, workspace, workspace_bytes);
  if (rc != PDR_OK) return rc;
  norm::Norm a = norm_of(*p, true);
  a.part = need ? (float *)workspace : nullptr;
  a.offs = norm_offsets(*p) ? (float *)((char *)workspace + norm_parts(*p)) : nullptr;
  return status(norm::launch_norm_backward(a, (hipStream_t)stream));
}

long long pdr_dropout_workspace_bytes(const pdr_dropout_args *p) { return check_dropout(p); }
int pdr_dropout(const pdr_dropout_args *p, void *, size_t, void *stream) {
  const int rc = check_dropout(p);
  if (rc != PDR_OK) return rc;
  norm::Drop a = {};
  a.x = p->x;
  a.res = p->res;
  a.y = p->y;
  a.seed_at = p->seed_at;
  a.seed = p->seed;
  a.offset = p->offset;
  a.count = p->rows * p->cols;
  a.cols = p->cols;
  a.ldx = p->ldx;
  a.ldr = p->ldr;
  a.ldy = p->ldy;
  a.fmt = p->fmt;
  a.t = (uint32_t)rint(p->p * 65536.0);
  a.scale = a.t < 65536 ? (float)(65536.0 / (65536.0 - a.t)) : 0.f;
  const bool run = p->rows <= 1 || (p->ldx == p->cols && p->ldy == p->cols && (!p->res || p->ldr == p->cols));
  a.vec = run && aligned(p->x, 16) && aligned(p->y, 16) && aligned(p->res, 16);
  return status(norm::launch_dropout(a, (hipStream_t)stream));
}

}  // extern "C"
