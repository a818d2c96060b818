// Host side of rotary positions and of the int8 cache's C ABI: frequencies,
// argument checks, workspace layout.  Nothing here allocates or synchronises.
#include <math.h>
#include <string.h>

#include "tq_int8_cache.cuh"

namespace tq {
namespace i8 {

static bool al(const void *p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static bool status_ok(const int32_t *p) { return !p || al(p, 4); }
static bool type_ok(int type) { return type == TQ_F32 || type == TQ_F16 || type == TQ_BF16; }

static tq_status mapped(cudaError_t e) {
  if (e == cudaSuccess) return TQ_OK;
  cudaGetLastError();                 // the status reports it; leave no stale error behind
  return TQ_ERR_CUDA;
}

// -- rotary positions

static bool rope_ok(const tq_rope *r, int head_dim) {
  return r && r->rot_dim >= 2 && r->rot_dim % 2 == 0 && r->rot_dim <= head_dim &&
         (r->layout == TQ_ROPE_HALF || r->layout == TQ_ROPE_INTERLEAVED) && isfinite(r->magnitude);
}

static bool stride_ok(int64_t stride, int heads, int head_dim) {
  return stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * head_dim;
}

// shapes and strides of one tensor (its pointers: pointers_ok)
static bool heads_ok(const tq_head_rows *t, int head_dim, bool out) {
  if (t->n_heads <= 0 || t->n_heads > 65536 || !stride_ok(t->src_stride, t->n_heads, head_dim)) return false;
  if (!out) return true;
  return stride_ok(t->dst_stride, t->n_heads, head_dim) && (t->dst != t->src || t->dst_stride == t->src_stride);
}

static bool pointers_ok(const tq_head_rows *t, bool out) {
  return al(t->src, 16) && (out ? al(t->dst, 16) : !t->dst) && (!t->norm_weight || al(t->norm_weight, 16));
}

static Part part_of(const tq_head_rows *t, int head_dim) {
  Part p;
  memset(&p, 0, sizeof(p));
  p.src = t->src;
  p.dst = t->dst;
  p.norm = t->norm_weight;
  p.src_stride = t->src_stride;
  p.dst_stride = t->dst_stride;
  p.n_heads = t->n_heads;
  p.head_dim = head_dim;
  p.turns = 1;
  return p;
}

static void set_rope(StepArgs &a, const tq_rope *r, int inverse, float eps, const int32_t *positions) {
  a.turns = r->turns;
  a.rot = r->rot_dim;
  a.layout = r->layout;
  a.gain = r->magnitude;
  a.sign = inverse ? -1.f : 1.f;
  a.eps = eps;
  a.eps_root = eps > 0.f ? sqrtf(eps) : 0.f;
  a.positions = positions;
}

// -- the cache

static bool shape_ok(const tq_int8 *c) {
  return c && c->n_kv_heads > 0 && c->n_kv_heads <= 65536 && c->head_dim > 0 && c->head_dim <= 256 &&
         c->head_dim % 16 == 0 && c->n_cells > 0 && c->n_cells <= 0xffffffffLL / c->n_kv_heads &&
         al(c->rows, 16) && al(c->scales, 16);
}

static bool pair_ok(const tq_int8 *k, const tq_int8 *v) { return shape_ok(k) && shape_ok(v) && k->n_cells == v->n_cells; }

static Part stored(const tq_int8 *c, const void *src, int64_t stride) {
  Part p;
  memset(&p, 0, sizeof(p));
  p.src = src;
  p.src_stride = stride;
  p.cells = static_cast<int8_t *>(c->rows);
  p.scales = static_cast<uint16_t *>(c->scales);
  p.n_heads = c->n_kv_heads;
  p.head_dim = c->head_dim;
  return p;
}

constexpr int64_t kMaxRows = 0x7fffffffLL;

}  // namespace i8
}  // namespace tq

using namespace tq;
using namespace tq::i8;

extern "C" {

tq_status tq_rope_frequencies(int rot_dim, double base, const tq_rope_scaling *scaling, double *freqs,
                              float *magnitude) {
  if (rot_dim < 2 || rot_dim > 256 || rot_dim % 2 || !(base > 0.0) || !isfinite(base) || !freqs || !magnitude)
    return TQ_ERR_INVALID_ARG;
  const int kind = scaling ? scaling->kind : TQ_ROPE_PLAIN, n = rot_dim / 2;
  if (kind < TQ_ROPE_PLAIN || kind > TQ_ROPE_PAIRS) return TQ_ERR_INVALID_ARG;
  double factor = 1.0;
  if (kind != TQ_ROPE_PLAIN) {
    factor = scaling->factor;
    if (!(factor > 0.0) || !isfinite(factor)) return TQ_ERR_INVALID_ARG;
  }
  if (kind == TQ_ROPE_BASE) {
    if (rot_dim == 2) return TQ_ERR_INVALID_ARG;
    base *= pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    if (!(base > 0.0) || !isfinite(base)) return TQ_ERR_INVALID_ARG;
  }
  const double two_pi = 6.283185307179586476925;
  double lo = 0.0, hi = 0.0;
  if (kind == TQ_ROPE_ROTATIONS || kind == TQ_ROPE_PAIRS) {
    const tq_rope_scaling &s = *scaling;
    if (!(s.original_len > 0.0) || !isfinite(s.original_len) || !(s.beta_slow > 0.0) || !(s.beta_fast > s.beta_slow) ||
        !isfinite(s.beta_fast))
      return TQ_ERR_INVALID_ARG;
    if (kind == TQ_ROPE_PAIRS) {
      if (!(base > 1.0)) return TQ_ERR_INVALID_ARG;
      auto pair_of = [&](double beta) { return rot_dim * log(s.original_len / (two_pi * beta)) / (2.0 * log(base)); };
      lo = fmax(floor(pair_of(s.beta_fast)), 0.0);
      hi = fmax(fmin(ceil(pair_of(s.beta_slow)), rot_dim - 1.0), lo);
      if (hi == lo) hi += 0.001;
    }
  }
  for (int j = 0; j < n; ++j) {
    const double f = pow(base, -2.0 * j / rot_dim);
    double keep = 1.0;                           // share of f as it is
    if (kind == TQ_ROPE_LINEAR) keep = 0.0;
    if (kind == TQ_ROPE_ROTATIONS)
      keep = fmin(fmax((scaling->original_len * f / two_pi - scaling->beta_slow) / (scaling->beta_fast - scaling->beta_slow), 0.0), 1.0);
    if (kind == TQ_ROPE_PAIRS) keep = 1.0 - fmin(fmax((j - lo) / (hi - lo), 0.0), 1.0);
    freqs[j] = kind == TQ_ROPE_BASE || kind == TQ_ROPE_PLAIN ? f : keep * f + (1.0 - keep) * f / factor;
  }
  *magnitude = kind == TQ_ROPE_PAIRS && factor > 1.0 ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
  return TQ_OK;
}

tq_status tq_rope_turns(const double *freqs, int n, uint64_t *turns) {
  if (!freqs || !turns || n < 0) return TQ_ERR_INVALID_ARG;
  for (int j = 0; j < n; ++j)
    if (!isfinite(freqs[j])) return TQ_ERR_INVALID_ARG;
  for (int j = 0; j < n; ++j) {
    double t = fabs(freqs[j]) / 6.283185307179586476925;
    t = (t - floor(t)) * 4294967296.0;
    const double whole = floor(t);
    const uint64_t x = (static_cast<uint64_t>(whole) << 32) + static_cast<uint64_t>((t - whole) * 4294967296.0);
    turns[j] = freqs[j] < 0.0 ? 0 - x : x;       // (a turn is 2^64)
  }
  return TQ_OK;
}

tq_status tq_rope_rows(const tq_rope *rope, const tq_head_rows *q, const tq_head_rows *k, int head_dim, int type,
                       float eps, int inverse, const int32_t *positions, int64_t n_rows, int32_t *dev_status,
                       tq_stream stream) {
  if (head_dim < 8 || head_dim > 256 || head_dim % 8 || !type_ok(type) || !rope_ok(rope, head_dim) || (!q && !k) ||
      n_rows < 0 || n_rows > kMaxRows)
    return TQ_ERR_INVALID_ARG;
  const tq_head_rows *t[2] = {q, k};
  for (const tq_head_rows *x : t) {
    if (!x) continue;
    if (!heads_ok(x, head_dim, true)) return TQ_ERR_INVALID_ARG;
    if (x->norm_weight && (inverse || !isfinite(eps) || eps < 0.f)) return TQ_ERR_INVALID_ARG;
  }
  if (n_rows == 0) return TQ_OK;
  if (!al(rope->turns, 16) || !al(positions, 4) || !status_ok(dev_status)) return TQ_ERR_INVALID_ARG;
  StepArgs a;
  memset(&a, 0, sizeof(a));
  for (int i = 0; i < 2; ++i) {
    if (!t[i]) continue;
    if (!pointers_ok(t[i], true)) return TQ_ERR_INVALID_ARG;
    a.part[i] = part_of(t[i], head_dim);
  }
  set_rope(a, rope, inverse, eps, positions);
  a.status = dev_status;
  a.n_rows = n_rows;
  return mapped(launch_step_rows(type, a, static_cast<cudaStream_t>(stream)));
}

static tq_status rows_shape(const tq_int8 *k, const tq_int8 *v, int64_t k_stride, int64_t v_stride, int type,
                            int64_t n_rows) {
  if (!pair_ok(k, v) || !type_ok(type) || n_rows < 0 || n_rows > kMaxRows ||
      !stride_ok(k_stride, k->n_kv_heads, k->head_dim) || !stride_ok(v_stride, v->n_kv_heads, v->head_dim))
    return TQ_ERR_INVALID_ARG;
  return TQ_OK;
}

tq_status tq_int8_set_rows(const tq_int8 *k, const tq_int8 *v, const void *k_src, int64_t k_stride,
                           const void *v_src, int64_t v_stride, int src_type, const int64_t *slots, int64_t n_rows,
                           int32_t *dev_status, tq_stream stream) {
  const tq_status st = rows_shape(k, v, k_stride, v_stride, src_type, n_rows);
  if (st != TQ_OK || n_rows == 0) return st;
  if (!al(k_src, 16) || !al(v_src, 16) || !al(slots, 8) || !status_ok(dev_status)) return TQ_ERR_INVALID_ARG;
  StepArgs a;
  memset(&a, 0, sizeof(a));
  a.part[K] = stored(k, k_src, k_stride);
  a.part[V] = stored(v, v_src, v_stride);
  a.slots = slots;
  a.status = dev_status;
  a.n_rows = n_rows;
  a.n_cells = k->n_cells;
  return mapped(launch_step_rows(src_type, a, static_cast<cudaStream_t>(stream)));
}

tq_status tq_int8_rope_set_rows(const tq_int8 *k, const tq_int8 *v, const tq_rope *rope, const tq_head_rows *q,
                                const tq_head_rows *k_rows, const void *v_src, int64_t v_stride, int type, float eps,
                                const int32_t *positions, const int64_t *slots, int64_t n_rows, int32_t *dev_status,
                                tq_stream stream) {
  if (!k_rows) return TQ_ERR_INVALID_ARG;
  const tq_status st = rows_shape(k, v, k_rows->src_stride, v_stride, type, n_rows);
  if (st != TQ_OK) return st;
  if (!rope_ok(rope, k->head_dim) || k_rows->n_heads != k->n_kv_heads || (q && !heads_ok(q, k->head_dim, true)))
    return TQ_ERR_INVALID_ARG;
  if ((k_rows->norm_weight || (q && q->norm_weight)) && (!isfinite(eps) || eps < 0.f)) return TQ_ERR_INVALID_ARG;
  if (n_rows == 0) return TQ_OK;
  if (!al(rope->turns, 16) || !pointers_ok(k_rows, false) || (q && !pointers_ok(q, true)) || !al(v_src, 16) ||
      !al(positions, 4) || !al(slots, 8) || !status_ok(dev_status))
    return TQ_ERR_INVALID_ARG;
  StepArgs a;
  memset(&a, 0, sizeof(a));
  if (q) a.part[Q] = part_of(q, k->head_dim);
  a.part[K] = stored(k, k_rows->src, k_rows->src_stride);
  a.part[K].norm = k_rows->norm_weight;
  a.part[K].turns = 1;
  a.part[V] = stored(v, v_src, v_stride);
  set_rope(a, rope, 0, eps, positions);
  a.slots = slots;
  a.status = dev_status;
  a.n_rows = n_rows;
  a.n_cells = k->n_cells;
  return mapped(launch_step_rows(type, a, static_cast<cudaStream_t>(stream)));
}

tq_status tq_int8_get_rows(const tq_int8 *k, const tq_int8 *v, void *k_dst, int64_t k_stride, void *v_dst,
                           int64_t v_stride, int dst_type, const int64_t *slots, int64_t n_rows,
                           int32_t *dev_status, tq_stream stream) {
  const tq_status st = rows_shape(k, v, k_stride, v_stride, dst_type, n_rows);
  if (st != TQ_OK || n_rows == 0) return st;
  if (!al(k_dst, 16) || !al(v_dst, 16) || !al(slots, 8) || !status_ok(dev_status)) return TQ_ERR_INVALID_ARG;
  p4::RowsArgs a;
  memset(&a, 0, sizeof(a));
  const tq_int8 *c[2] = {k, v};
  void *dst[2] = {k_dst, v_dst};
  const int64_t stride[2] = {k_stride, v_stride};
  for (int i = 0; i < 2; ++i) {
    a.dst[i] = dst[i];
    a.codes[i] = static_cast<uint8_t *>(c[i]->rows);
    a.scales[i] = static_cast<uint16_t *>(c[i]->scales);
    a.stride[i] = stride[i];
    a.n_heads[i] = c[i]->n_kv_heads;
    a.head_dim[i] = c[i]->head_dim;
    a.width[i] = p4::row_width(c[i]->head_dim);
  }
  a.slots = slots;
  a.status = dev_status;
  a.n_rows = n_rows;
  a.n_cells = k->n_cells;
  return mapped(i8::launch_get_rows(dst_type, a, static_cast<cudaStream_t>(stream)));
}

// -- attention

static tq_status decode_shape(const tq_int8 *k, const tq_int8 *v, int n_q_heads, int n_seq) {
  if (!pair_ok(k, v) || k->n_kv_heads != v->n_kv_heads || n_q_heads <= 0 || n_q_heads > 65536 ||
      n_q_heads % k->n_kv_heads || n_seq < 0 || n_seq > (1 << 24))
    return TQ_ERR_INVALID_ARG;
  const int wk = p4::row_width(k->head_dim), wv = p4::row_width(v->head_dim);
  return wk == wv || (wk == 256 && wv == 128) ? TQ_OK : TQ_ERR_UNSUPPORTED;
}

// Workspace: laid out as the paged calls' (status word, arrival counters, partial results), so that one serves both.
// Two partial results per CTA, each of at most 4096 values and (maximum, sum) of 8 columns a head (tq_int8_decode.cuh).
constexpr size_t kCountersOff = 256;
static size_t decode_bytes() {
  return TQ_PAGED4_WORKSPACE_HEAD + sizeof(float) * 2 * static_cast<size_t>(p4::max_ctas(2)) * (4096 + 128);
}

size_t tq_int8_decode_workspace(const tq_int8 *k, const tq_int8 *v, int n_q_heads, int n_seq) {
  return decode_shape(k, v, n_q_heads, n_seq) == TQ_OK ? decode_bytes() : 0;
}

tq_status tq_int8_decode(const tq_int8 *k, const tq_int8 *v, int page_size, const int32_t *block_table, int max_pages,
                         const int32_t *seq_len, int n_seq, const void *q, int q_type, int64_t q_stride,
                         int n_q_heads, float scale, void *out, void *workspace, size_t workspace_bytes,
                         tq_stream stream) {
  const tq_status st = decode_shape(k, v, n_q_heads, n_seq);
  if (st != TQ_OK) return st;
  if (q_type == TQ_F32) return TQ_ERR_UNSUPPORTED;
  if (q_type != TQ_F16 && q_type != TQ_BF16) return TQ_ERR_INVALID_ARG;
  if (page_size < 1 || page_size > 65536 || (page_size & (page_size - 1)) || !isfinite(scale) || max_pages <= 0 ||
      !stride_ok(q_stride, n_q_heads, k->head_dim))
    return TQ_ERR_INVALID_ARG;
  // (the kernel counts cells in 32 bits, up to the end of the last key tile)
  if (static_cast<int64_t>(max_pages) * page_size > 0x7fff0000LL || n_seq > 0x7fffffff / n_q_heads)
    return TQ_ERR_INVALID_ARG;
  if (n_seq == 0) return TQ_OK;
  if (!al(block_table, 4) || !al(seq_len, 4) || !al(q, 16) || !al(out, 16)) return TQ_ERR_INVALID_ARG;
  const int wk = p4::row_width(k->head_dim), wv = p4::row_width(v->head_dim);
  if (!al(workspace, 256) || workspace_bytes < decode_bytes()) return TQ_ERR_WORKSPACE;
  p4::AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.k_codes = static_cast<const uint8_t *>(k->rows);
  a.k_scales = static_cast<const uint16_t *>(k->scales);
  a.v_codes = static_cast<const uint8_t *>(v->rows);
  a.v_scales = static_cast<const uint16_t *>(v->scales);
  a.block_table = block_table;
  a.seq_len = seq_len;
  a.q = q;
  a.out = out;
  a.status = static_cast<int32_t *>(workspace);
  a.counters = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + kCountersOff);
  a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + TQ_PAGED4_WORKSPACE_HEAD);
  a.q_stride = q_stride;
  a.n_rows = n_seq;
  a.n_seq = n_seq;
  a.max_pages = max_pages;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  // whole pages of the cache; ids are 32-bit numbers
  const int64_t pages = k->n_cells >> a.page_shift;
  a.n_pages = static_cast<int32_t>(pages < 0x7fffffffLL ? pages : 0x7fffffffLL);
  a.n_heads = n_q_heads;
  a.n_kv_heads = k->n_kv_heads;
  a.group = n_q_heads / k->n_kv_heads;
  a.dk = k->head_dim;
  a.dv = v->head_dim;
  a.wk = wk;
  a.wv = wv;
  a.bf16 = q_type == TQ_BF16;
  a.causal = 1;
  a.n_rows_cache = k->n_cells * k->n_kv_heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  return mapped(i8::launch_decode(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
