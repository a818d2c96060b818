// Internal declarations of the paged 4-bit cache: launch arguments shared by its
// host calls (tq_paged4_host.cu) and kernels.
//
// A row is stored as D / 2 bytes of 4-bit codes (D: the head dim rounded up to 64,
// 128 or 256; element i in the low (i even) or high nibble of byte i / 2) and a
// binary16 pair (scale, offset): value = scale * code + offset.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tq_internal.h"

namespace tq {
namespace p4 {

// stored row width in elements of a head dim (0: not supported)
constexpr int row_width(int head_dim) {
  return head_dim <= 0 || head_dim > 256 ? 0 : head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
}

struct PlanArgs {
  const int32_t *seq_len;
  const int32_t *n_new;
  int32_t *block_table;
  int32_t *free_pages;
  const int32_t *free_count;
  int32_t *new_len;
  int32_t *new_free_count;
  int32_t *q_start;
  int32_t *page_start;
  int64_t *slots;
  int32_t *positions;
  int32_t *status;
  int64_t n_rows;
  int64_t free_capacity;
  int32_t n_seq;
  int32_t max_pages;
  int32_t page_shift;
};
cudaError_t launch_page_plan(const PlanArgs &a, cudaStream_t s);

struct RowsArgs {
  // one entry for K (0) and V (1); src / dst rows of `stride` elements
  const void *src[2];
  void *dst[2];
  uint8_t *codes[2];
  uint16_t *scales[2];
  int64_t stride[2];
  int32_t n_heads[2];
  int32_t head_dim[2];
  int32_t width[2];
  const int64_t *slots;
  int32_t *status;
  int64_t n_rows;
  int64_t n_cells;
  int32_t page_shift;
  uint32_t k_blocks;       // CTAs of the K rows (set at the launch)
};
cudaError_t launch_set_rows(int type, const RowsArgs &a, cudaStream_t s);
cudaError_t launch_get_rows(int type, const RowsArgs &a, cudaStream_t s);

struct AttnArgs {
  const uint8_t *k_codes;
  const uint16_t *k_scales;
  const uint8_t *v_codes;
  const uint16_t *v_scales;
  const int32_t *block_table;
  const int32_t *seq_len;
  const int32_t *q_start;    // null: one query row per sequence
  const void *q;
  void *out;
  const float *lam;          // differential: weight of the second map per output head
  const float *norm_weight;  // differential: RMS norm over each output row, or null
  int32_t *status;
  int32_t *counters;         // arrivals per work-sharing group, self-resetting
  float *part;               // partial results of items that CTAs share
  float *row_part;           // prompt kernel: of rows [row][head][map][split][4 + width]: (R, l, 0, 0), values
  int64_t q_stride;          // elements between query rows
  int64_t n_rows;            // query rows in q / out
  int32_t n_seq;
  int32_t max_pages;         // block table width
  int32_t n_pages;
  int32_t page_shift;
  int32_t n_heads;           // output heads
  int32_t n_kv_heads;        // V heads
  float inv_group;                 // 1 / group
  int32_t group;             // output heads per V head
  int32_t dk, dv;            // logical head dims
  int32_t wk, wv;            // stored widths
  int32_t bf16;              // element type of q and out: bfloat16 (1) or binary16 (0)
  int32_t causal;
  int32_t diff;
  float scale_log2;
  float eps;
  float out_scale;
  int32_t line;              // prompt kernel: one line of work over the SMs (else n_split CTAs per item)
  int32_t n_split;           // prompt kernel: key-range splits per tile
  int32_t n_tiles;           // prompt kernel: upper bound of row tiles over all sequences
};

// CTAs of a launch whose CTAs share items, `per_sm` on each SM: each has an arrival counter in the workspace's head.
constexpr int kMaxCtas = 960;
inline int max_ctas(int per_sm) { return sm_count() * per_sm < kMaxCtas ? sm_count() * per_sm : kMaxCtas; }

// Few-row kernel: 8 or 16 query columns at a time, keys split evenly over the grid.
bool few_supported(int wk, int wv, bool diff);
cudaError_t launch_few(const AttnArgs &a, int columns, cudaStream_t s);

// Prompt kernel: 256-row tiles on the tcgen05 tensor cores.
bool prefill_supported(int wk, int wv);
cudaError_t launch_prefill(const AttnArgs &a, cudaStream_t s);

// out_scale / sqrt(mean(o^2) + eps) of a differential row with the sum of squares `ss`, out_scale without a norm.  A row of
// zeros (no cell, or values that are 0) stays one where eps is 0.
__device__ __forceinline__ float diff_factor(const AttnArgs &a, float ss) {
  if (!a.norm_weight) return a.out_scale;
  const float mean = ss / static_cast<float>(a.dv) + a.eps;
  return mean != 0.f ? rsqrtf(mean) * a.out_scale : 0.f;
}

// A launch that may begin while the one before it on the stream is still running (programmatic dependent launch); the
// kernel waits itself before it reads what that writes.
template <typename Args>
cudaError_t launch_beside(void (*kern)(Args), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                          const Args &a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace p4
}  // namespace tq
