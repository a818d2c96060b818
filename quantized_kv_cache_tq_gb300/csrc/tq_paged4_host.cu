// Host side of the paged 4-bit cache's C ABI: argument checks, workspace layout
// and the choice of kernel.  Nothing here allocates or synchronises.
#include <math.h>
#include <string.h>

#include "tq_paged4.cuh"
#include "tq_paged4_few.cuh"
#include "tq_testing.h"

namespace tq {
namespace p4 {

cudaError_t launch_few_plain(const AttnArgs &a, int columns, cudaStream_t s);
cudaError_t launch_few_wide(const AttnArgs &a, int columns, cudaStream_t s);
cudaError_t launch_few_diff(const AttnArgs &a, cudaStream_t s);

cudaError_t launch_few(const AttnArgs &a, int columns, cudaStream_t s) {
  if (a.diff) return launch_few_diff(a, s);
  return a.wk == 256 ? launch_few_wide(a, columns, s) : launch_few_plain(a, columns, s);
}

static bool al(const void *p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static size_t up(size_t x, size_t n) { return (x + n - 1) / n * n; }

static int shift_of(int page_size, int lo, int hi) {
  if (page_size < lo || page_size > hi || (page_size & (page_size - 1))) return -1;
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

static bool shape_ok(int n_kv_heads, int head_dim, int page_size, int n_pages) {
  return n_kv_heads > 0 && n_kv_heads <= 65536 && head_dim % 8 == 0 && row_width(head_dim) > 0 &&
         shift_of(page_size, 16, 1024) >= 0 && n_pages > 0 &&
         static_cast<int64_t>(n_pages) * page_size < 0x100000000LL / n_kv_heads;     // 32-bit row numbers
}

static bool cache_ok(const tq_paged4 *c) {
  return c && shape_ok(c->n_kv_heads, c->head_dim, c->page_size, c->n_pages) && al(c->codes, 16) &&
         al(c->scales, 16);
}

static bool pair_ok(const tq_paged4 *k, const tq_paged4 *v) {
  return cache_ok(k) && cache_ok(v) && k->page_size == v->page_size && k->n_pages == v->n_pages;
}

static tq_status mapped(cudaError_t e) {
  if (e == cudaSuccess) return TQ_OK;
  cudaGetLastError();                 // the status reports it; leave no stale error behind
  return TQ_ERR_CUDA;
}

// Shape checks common to the attention calls; `diff` from the caller.
static tq_status heads_ok(const tq_paged4 *k, const tq_paged4 *v, int n_heads, int n_seq, bool diff) {
  if (!pair_ok(k, v) || n_seq < 0 || n_seq > (1 << 24)) return TQ_ERR_INVALID_ARG;
  if (k->n_kv_heads != (diff ? 2 : 1) * v->n_kv_heads) return TQ_ERR_INVALID_ARG;
  if (n_heads <= 0 || n_heads > 65536 || n_heads % v->n_kv_heads) return TQ_ERR_INVALID_ARG;
  return few_supported(row_width(k->head_dim), row_width(v->head_dim), diff) ? TQ_OK : TQ_ERR_UNSUPPORTED;
}

bool few_supported(int wk, int wv, bool diff) {
  if (diff) return (wk == 64 && wv <= 128) || (wk == 128 && (wv == 128 || wv == 256));
  return (wk == wv) || (wk == 256 && wv == 128);
}

// Workspace: status word, arrival counters (one per CTA of either kernel, in a place that does not depend on the shape,
// so that calls of different shapes can share it), partials of either kernel.  Partials are written before they are read:
// only the head in front of them has to be zero before the first use.
constexpr size_t kCountersOff = 256, kHead = TQ_PAGED4_WORKSPACE_HEAD;
static_assert(kCountersOff + sizeof(int32_t) * kMaxCtas <= kHead, "counters");
struct Layout {
  size_t part_off, total;
};

static Layout few_layout(int wv) {
  Layout L;
  const size_t ctas = static_cast<size_t>(max_ctas(2));            // at most two per SM
  const size_t columns = 16, tiles = 2;                            // the larger of the two column widths
  L.part_off = kHead;
  L.total = L.part_off + sizeof(float) * 2 * ctas * (4 * columns + tiles * (wv / 16) * 128);
  return L;
}

// How the prompt kernel shares its work out: one line over the SMs, or n_split CTAs per item (256-row tile, K
// head), whichever is estimated to end first.  In key tiles of one CTA (2 us): a CTA costs its key tiles + 4 for
// set-up and epilogue, + 4 where rows' partial results are written and merged; a line costs its share, and 14 for
// finding it and for the items cut at its ends.  Measured, line against split: 2048 rows over 32768 cells 818 /
// 926 us, over 4096 cells 114 / 104 us, three differential chunks of up to 700 rows 90 / 104 us, 20 chunks of up to
// 300 rows 90 / 83 us.
// Of the splits only those are taken whose rows' partial results fit in the room of a line's (row_room; no shape is
// known where the estimate would choose another): a workspace for some rows then serves every call of fewer.
constexpr int kMaxSplit = 16;
static int64_t row_room() { return 2 * 256 * static_cast<int64_t>(max_ctas(1)); }     // (two partials of 256 rows per CTA)
struct Share {
  bool line;
  int n_split;
};
static Share prefill_share(int64_t n_rows, int n_seq, int group, int k_heads, int maps, int64_t max_len) {
  const int64_t sms = sm_count(), tiles = (max_len + 127) / 128;
  // (row tiles: the full ones and about half a tile per sequence)
  int64_t items = (n_rows * group + 128 * (n_seq < n_rows ? n_seq : n_rows)) / 256 * k_heads;
  if (items < k_heads) items = k_heads;
  Share best = {true, 1};
  int64_t least = (items * (tiles + 4) + sms - 1) / sms + 14;
  for (int c = 1; c <= kMaxSplit && (c == 1 || (tiles / c >= 4 && n_rows * group * k_heads * c <= row_room())); ++c) {
    const int64_t cost = (items * c + sms - 1) / sms * ((tiles + c - 1) / c + 4 + (c > 1 || maps > 1 ? 4 : 0));
    if (cost < least) {
      best = {false, c};
      least = cost;
    }
  }
  return best;
}

// Whether a ragged call goes to the prompt kernel.  Up to 16 query columns per KV head (two tiles of the few-row
// kernel) the 256-row tiles of the prompt kernel would stand nearly empty.
static bool takes_prefill(const tq_paged4 *k, const tq_paged4 *v, int64_t rows_per_seq, int group) {
  return prefill_supported(row_width(k->head_dim), row_width(v->head_dim)) && rows_per_seq * group > 16;
}

// row_off: where the rows' partial results begin.  The size only grows with n_rows, and depends neither on how the work
// is shared out nor on sequences and lengths, so that a workspace serves every smaller call: it has room for a line's
// shared items or for a split's rows, and behind it for the rows of two maps.
static Layout prefill_layout(const tq_paged4 *k, const tq_paged4 *v, int n_heads, int64_t n_rows, int n_split,
                             size_t *row_off) {
  const int wv = row_width(v->head_dim), maps = k->n_kv_heads / v->n_kv_heads;
  Layout L = few_layout(wv);
  *row_off = L.part_off;
  if (!takes_prefill(k, v, n_rows, n_heads / v->n_kv_heads)) return L;
  const size_t row = sizeof(float) * (wv + 4), room = static_cast<size_t>(row_room()) * row;
  size_t end = L.part_off + room;
  if (maps > 1) {
    if (n_split == 1) *row_off = end;         // (differential rows leave partial results in the line form too)
    end += static_cast<size_t>(n_rows) * n_heads * maps * row;
  }
  if (end > L.total) L.total = end;
  return L;
}

struct Call {
  const tq_paged4 *k, *v;
  const int32_t *block_table, *seq_len, *q_start;
  const void *q;
  const float *lam, *norm_weight;
  void *out, *workspace;
  size_t workspace_bytes;
  int64_t q_stride, n_rows, max_rows, max_len;
  int max_pages, n_seq, q_type, n_heads, causal;
  float scale, eps, out_scale;
  bool diff, ragged;
  tq_stream stream;
};

static tq_status attend(const Call &c) {
  tq_status st = heads_ok(c.k, c.v, c.n_heads, c.n_seq, c.diff);
  if (st != TQ_OK) return st;
  if (c.q_type == TQ_F32) return TQ_ERR_UNSUPPORTED;
  if (c.q_type != TQ_F16 && c.q_type != TQ_BF16) return TQ_ERR_INVALID_ARG;
  if (!isfinite(c.scale) || c.max_pages <= 0 || c.n_rows < 0 || c.max_rows < 0 || c.max_len < 0)
    return TQ_ERR_INVALID_ARG;
  if (c.diff && (!al(c.lam, 4) || (c.norm_weight && !al(c.norm_weight, 4)) || !isfinite(c.eps) || c.eps < 0.f ||
                 !isfinite(c.out_scale)))
    return TQ_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(c.diff ? 2 : 1) * c.n_heads * c.k->head_dim;
  if (c.q_stride < row || c.q_stride % 8) return TQ_ERR_INVALID_ARG;
  if (c.n_rows > 0x7fffffffLL / c.n_heads) return TQ_ERR_INVALID_ARG;
  // (the kernels count cells in 32 bits, up to the end of the last key tile)
  if (static_cast<int64_t>(c.max_pages) * c.k->page_size > 0x7fff0000LL) return TQ_ERR_INVALID_ARG;
  if (c.n_seq == 0 || c.n_rows == 0) return TQ_OK;
  if (!al(c.block_table, 4) || !al(c.seq_len, 4) || (c.ragged && !al(c.q_start, 4)) || !al(c.q, 16) || !al(c.out, 16))
    return TQ_ERR_INVALID_ARG;
  const int wk = row_width(c.k->head_dim), wv = row_width(c.v->head_dim);
  const int group = c.n_heads / c.v->n_kv_heads;
  const int64_t rows = !c.ragged ? 1 : c.max_rows && c.max_rows < c.n_rows ? c.max_rows : c.n_rows;
  const bool prompt = c.ragged && takes_prefill(c.k, c.v, rows, group);
  Share share = {false, 1};
  if (prompt)
    share = prefill_share(c.n_rows, c.n_seq, group, c.k->n_kv_heads, c.diff ? 2 : 1,
                          c.max_len ? c.max_len : static_cast<int64_t>(c.max_pages) * c.k->page_size);
  const bool line = share.line;
  const int n_split = share.n_split;
  size_t row_off = 0;
  const Layout L = prompt ? prefill_layout(c.k, c.v, c.n_heads, c.n_rows, n_split, &row_off) : few_layout(wv);
  if (!al(c.workspace, 256) || c.workspace_bytes < L.total) return TQ_ERR_WORKSPACE;
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.k_codes = static_cast<const uint8_t *>(c.k->codes);
  a.k_scales = static_cast<const uint16_t *>(c.k->scales);
  a.v_codes = static_cast<const uint8_t *>(c.v->codes);
  a.v_scales = static_cast<const uint16_t *>(c.v->scales);
  a.block_table = c.block_table;
  a.seq_len = c.seq_len;
  a.q_start = c.ragged ? c.q_start : nullptr;
  a.q = c.q;
  a.out = c.out;
  a.lam = c.lam;
  a.norm_weight = c.norm_weight;
  a.status = static_cast<int32_t *>(c.workspace);
  a.counters = reinterpret_cast<int32_t *>(static_cast<char *>(c.workspace) + kCountersOff);
  a.part = reinterpret_cast<float *>(static_cast<char *>(c.workspace) + L.part_off);
  a.q_stride = c.q_stride;
  a.n_rows = c.n_rows;
  a.n_seq = c.n_seq;
  a.max_pages = c.max_pages;
  a.n_pages = c.k->n_pages;
  a.page_shift = shift_of(c.k->page_size, 16, 1024);
  a.n_heads = c.n_heads;
  a.n_kv_heads = c.v->n_kv_heads;
  a.group = group;
  a.inv_group = 1.f / static_cast<float>(group);
  a.dk = c.k->head_dim;
  a.dv = c.v->head_dim;
  a.wk = wk;
  a.wv = wv;
  a.bf16 = c.q_type == TQ_BF16;
  a.causal = c.causal ? 1 : 0;
  a.diff = c.diff;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  a.eps = c.eps;
  a.out_scale = c.out_scale;
  a.n_split = n_split;
  a.line = line;
  a.row_part = reinterpret_cast<float *>(static_cast<char *>(c.workspace) + row_off);
  if (prompt) {
    const int64_t tiles = c.n_rows * group / 256 + c.n_seq;        // upper bound over ragged sequences
    if (tiles * n_split * c.k->n_kv_heads > 0x7fffffffLL || (c.n_rows * c.n_heads + 7) / 8 > 0x7fffffffLL)
      return TQ_ERR_UNSUPPORTED;
    a.n_tiles = static_cast<int32_t>(tiles);
    return mapped(launch_prefill(a, static_cast<cudaStream_t>(c.stream)));
  }
  const int columns = rows * group > 8 ? 16 : 8;
  return mapped(launch_few(a, columns, static_cast<cudaStream_t>(c.stream)));
}

static bool is_diff(const tq_paged4 *k, const tq_paged4 *v) { return k && v && k->n_kv_heads != v->n_kv_heads; }

}  // namespace p4
}  // namespace tq

using namespace tq;
using namespace tq::p4;

extern "C" {

tq_status tq_paged4_plane_bytes(int n_kv_heads, int head_dim, int page_size, int n_pages, size_t *codes_bytes,
                                size_t *scales_bytes) {
  if (!shape_ok(n_kv_heads, head_dim, page_size, n_pages) || !codes_bytes || !scales_bytes) return TQ_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(n_pages) * n_kv_heads * page_size;
  *codes_bytes = rows * (row_width(head_dim) / 2);
  *scales_bytes = rows * 4;
  return TQ_OK;
}

tq_status tq_page_plan(const int32_t *seq_len, const int32_t *n_new, int n_seq, int page_size, int32_t *block_table,
                       int max_pages, int32_t *free_pages, int64_t free_capacity, const int32_t *free_count,
                       int32_t *new_len, int32_t *new_free_count, int32_t *q_start, int32_t *page_start,
                       int64_t *slots, int32_t *positions, int64_t n_rows, int32_t *dev_status, tq_stream stream) {
  PlanArgs a;
  a.page_shift = shift_of(page_size, 1, 65536);
  if (a.page_shift < 0 || n_seq < 0 || max_pages <= 0 || free_capacity < 0 || free_capacity > 0x7fffffffLL ||
      n_rows < 0 || n_rows > 0x7fffffffLL - 1)
    return TQ_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) * page_size > 0x7fffffffLL) return TQ_ERR_INVALID_ARG;
  if (!al(free_count, 4) || !al(new_free_count, 4) || !al(q_start, 4) || !al(page_start, 4)) return TQ_ERR_INVALID_ARG;
  if (n_seq > 0 && (!al(seq_len, 4) || !al(n_new, 4) || !al(block_table, 4) || !al(new_len, 4)))
    return TQ_ERR_INVALID_ARG;
  if (free_capacity > 0 && !al(free_pages, 4)) return TQ_ERR_INVALID_ARG;
  if (n_rows > 0 && (!al(slots, 8) || !al(positions, 4))) return TQ_ERR_INVALID_ARG;
  if (dev_status && !al(dev_status, 4)) return TQ_ERR_INVALID_ARG;
  a.seq_len = seq_len;
  a.n_new = n_new;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.new_len = new_len;
  a.new_free_count = new_free_count;
  a.q_start = q_start;
  a.page_start = page_start;
  a.slots = slots;
  a.positions = positions;
  a.status = dev_status;
  a.n_rows = n_rows;
  a.free_capacity = free_capacity;
  a.n_seq = n_seq;
  a.max_pages = max_pages;
  return mapped(launch_page_plan(a, static_cast<cudaStream_t>(stream)));
}

static tq_status rows_call(bool set, const tq_paged4 *k, const tq_paged4 *v, const void *kp, int64_t k_stride,
                           const void *vp, int64_t v_stride, int type, const int64_t *slots, int64_t n_rows,
                           int32_t *dev_status, tq_stream stream) {
  if (!pair_ok(k, v)) return TQ_ERR_INVALID_ARG;
  if (type != TQ_F32 && type != TQ_F16 && type != TQ_BF16) return TQ_ERR_INVALID_ARG;
  if (n_rows < 0 || k_stride % 8 || v_stride % 8 || k_stride < static_cast<int64_t>(k->n_kv_heads) * k->head_dim ||
      v_stride < static_cast<int64_t>(v->n_kv_heads) * v->head_dim)
    return TQ_ERR_INVALID_ARG;
  if (n_rows == 0) return TQ_OK;
  if (!al(kp, 16) || !al(vp, 16) || !al(slots, 8) || (dev_status && !al(dev_status, 4))) return TQ_ERR_INVALID_ARG;
  // (at most 16 lanes a row and head, 256 to a CTA, 2^31 - 1 CTAs)
  if (n_rows > 0x7fffffffLL || n_rows * (k->n_kv_heads + v->n_kv_heads) > 0x7fffffe00LL) return TQ_ERR_INVALID_ARG;
  RowsArgs a;
  const tq_paged4 *c[2] = {k, v};
  const void *p[2] = {kp, vp};
  const int64_t stride[2] = {k_stride, v_stride};
  for (int i = 0; i < 2; ++i) {
    a.src[i] = p[i];
    a.dst[i] = const_cast<void *>(p[i]);
    a.codes[i] = static_cast<uint8_t *>(c[i]->codes);
    a.scales[i] = static_cast<uint16_t *>(c[i]->scales);
    a.stride[i] = stride[i];
    a.n_heads[i] = c[i]->n_kv_heads;
    a.head_dim[i] = c[i]->head_dim;
    a.width[i] = row_width(c[i]->head_dim);
  }
  a.slots = slots;
  a.status = dev_status;
  a.n_rows = n_rows;
  a.k_blocks = 0;
  a.page_shift = shift_of(k->page_size, 16, 1024);
  a.n_cells = static_cast<int64_t>(k->n_pages) << a.page_shift;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return mapped(set ? launch_set_rows(type, a, s) : launch_get_rows(type, a, s));
}

tq_status tq_paged4_set_rows(const tq_paged4 *k, const tq_paged4 *v, const void *k_src, int64_t k_stride,
                             const void *v_src, int64_t v_stride, int src_type, const int64_t *slots, int64_t n_rows,
                             int32_t *dev_status, tq_stream stream) {
  return rows_call(true, k, v, k_src, k_stride, v_src, v_stride, src_type, slots, n_rows, dev_status, stream);
}

tq_status tq_paged4_get_rows(const tq_paged4 *k, const tq_paged4 *v, void *k_dst, int64_t k_stride, void *v_dst,
                             int64_t v_stride, int dst_type, const int64_t *slots, int64_t n_rows,
                             int32_t *dev_status, tq_stream stream) {
  return rows_call(false, k, v, k_dst, k_stride, v_dst, v_stride, dst_type, slots, n_rows, dev_status, stream);
}

size_t tq_paged4_decode_workspace(const tq_paged4 *k, const tq_paged4 *v, int n_heads, int n_seq) {
  if (heads_ok(k, v, n_heads, n_seq, is_diff(k, v)) != TQ_OK) return 0;
  return few_layout(row_width(v->head_dim)).total;
}

size_t tq_paged4_prefill_workspace(const tq_paged4 *k, const tq_paged4 *v, int n_heads, int n_seq, int64_t n_rows,
                                   int64_t max_len) {
  if (heads_ok(k, v, n_heads, n_seq, is_diff(k, v)) != TQ_OK || n_rows < 0 || max_len < 0) return 0;
  if (n_rows > 0x7fffffffLL / n_heads) return 0;
  size_t row_off = 0;
  return prefill_layout(k, v, n_heads, n_rows, 1, &row_off).total;
}

tq_status tq_paged4_decode(const tq_paged4 *k, const tq_paged4 *v, const int32_t *block_table, int max_pages,
                           const int32_t *seq_len, int n_seq, const void *q, int q_type, int64_t q_stride,
                           int n_q_heads, float scale, void *out, void *workspace, size_t workspace_bytes,
                           tq_stream stream) {
  Call c = {k, v, block_table, seq_len, nullptr, q, nullptr, nullptr, out, workspace, workspace_bytes, q_stride,
            n_seq, 1, 0, max_pages, n_seq, q_type, n_q_heads, 1, scale, 0.f, 1.f, false, false, stream};
  return attend(c);
}

tq_status tq_paged4_prefill(const tq_paged4 *k, const tq_paged4 *v, const int32_t *block_table, int max_pages,
                            const int32_t *seq_len, const int32_t *q_start, int n_seq, const void *q, int q_type,
                            int64_t q_stride, int64_t n_rows, int n_q_heads, int64_t max_rows, int64_t max_len,
                            float scale, int causal, void *out, void *workspace, size_t workspace_bytes,
                            tq_stream stream) {
  Call c = {k, v, block_table, seq_len, q_start, q, nullptr, nullptr, out, workspace, workspace_bytes, q_stride,
            n_rows, max_rows, max_len, max_pages, n_seq, q_type, n_q_heads, causal, scale, 0.f, 1.f, false, true,
            stream};
  return attend(c);
}

tq_status tq_paged4_diff_decode(const tq_paged4 *k, const tq_paged4 *v, const int32_t *block_table, int max_pages,
                                const int32_t *seq_len, int n_seq, const void *q, int q_type, int64_t q_stride,
                                int n_heads, const float *lambda, const float *norm_weight, float eps,
                                float out_scale, float scale, void *out, void *workspace, size_t workspace_bytes,
                                tq_stream stream) {
  Call c = {k, v, block_table, seq_len, nullptr, q, lambda, norm_weight, out, workspace, workspace_bytes, q_stride,
            n_seq, 1, 0, max_pages, n_seq, q_type, n_heads, 1, scale, eps, out_scale, true, false, stream};
  return attend(c);
}

tq_status tq_paged4_diff_prefill(const tq_paged4 *k, const tq_paged4 *v, const int32_t *block_table, int max_pages,
                                 const int32_t *seq_len, const int32_t *q_start, int n_seq, const void *q,
                                 int q_type, int64_t q_stride, int64_t n_rows, int n_heads, int64_t max_rows,
                                 int64_t max_len, const float *lambda, const float *norm_weight, float eps,
                                 float out_scale, float scale, int causal, void *out, void *workspace,
                                 size_t workspace_bytes, tq_stream stream) {
  Call c = {k, v, block_table, seq_len, q_start, q, lambda, norm_weight, out, workspace, workspace_bytes, q_stride,
            n_rows, max_rows, max_len, max_pages, n_seq, q_type, n_heads, causal, scale, eps, out_scale, true, true,
            stream};
  return attend(c);
}

int tq_testing_paged4_few_grid(int k_width, int v_width, int columns, int diff, int sms, int *merge_bytes, int *smem) {
  auto of = [&](auto cfg) {
    using C = decltype(cfg);
    *merge_bytes = C::merge_bytes(C::grid(sms));
    *smem = C::SMEM;
    return C::grid(sms);
  };
  if (sms <= 0 || !merge_bytes || !smem || !few_supported(k_width, v_width, diff != 0)) return 0;
  if (diff) {
    if (k_width == 64) return v_width == 64 ? of(FewCfg<64, 64, 1, 2>()) : of(FewCfg<64, 128, 1, 2>());
    return v_width == 128 ? of(FewCfg<128, 128, 1, 2>()) : of(FewCfg<128, 256, 1, 2>());
  }
  const bool one = columns <= 8;
  if (k_width == 64) return one ? of(FewCfg<64, 64, 1, 1>()) : of(FewCfg<64, 64, 2, 1>());
  if (k_width == 128) return one ? of(FewCfg<128, 128, 1, 1>()) : of(FewCfg<128, 128, 2, 1>());
  if (v_width == 128) return one ? of(FewCfg<256, 128, 1, 1>()) : of(FewCfg<256, 128, 2, 1>());
  return one ? of(FewCfg<256, 256, 1, 1>()) : of(FewCfg<256, 256, 2, 1>());
}

}  // extern "C"
