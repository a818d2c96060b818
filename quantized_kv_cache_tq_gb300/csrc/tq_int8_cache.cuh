// Internal declarations of rotary positions and of the int8 cache's rows and
// single-token attention: launch arguments shared by their host calls
// (tq_int8_host.cu) and kernels.
//
// A row is stored as head_dim codes of 8 bits and a binary16 scale: value = scale * code.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tq_paged4.cuh"

namespace tq {
namespace i8 {

// What happens to a tensor's rows.
struct Part {
  const void *src;
  void *dst;               // rows out, or null
  int8_t *cells;           // quantised into a cache, or null
  uint16_t *scales;
  const float *norm;       // RMS norm per head, or null
  int64_t src_stride, dst_stride;
  int32_t n_heads;         // 0: no such tensor
  int32_t head_dim;
  int32_t turns;           // whether the rows are rotated
};

constexpr int Q = 0, K = 1, V = 2;

// Work as a line of units (a head of a tile of rows), tensor after tensor, `per` for each CTA and one more for the first
// `more` of them.
struct Units {
  int64_t part[3];
  int64_t per;
  int32_t more;
};

struct StepArgs {
  Part part[3];
  const uint64_t *turns;      // [rot / 2], 2^-64 of a turn per position
  const int32_t *positions;   // null: no part turns
  const int64_t *slots;       // null: no part is quantised
  int32_t *status;
  int64_t n_rows;
  int64_t n_cells;
  int32_t rot;
  int32_t layout;
  float gain;                 // factor on what turns
  float sign;                 // -1: the other way round
  float eps, eps_root;        // and its square root
  Units units;                // (set at the launch)
};
cudaError_t launch_step_rows(int type, const StepArgs &a, cudaStream_t s);
cudaError_t launch_get_rows(int type, const p4::RowsArgs &a, cudaStream_t s);

// Attention: AttnArgs with the planes' int8 rows as k_codes and v_codes.
cudaError_t launch_decode(const p4::AttnArgs &a, cudaStream_t s);

}  // namespace i8
}  // namespace tq
