// Rows on their way to the attention: RMS norm per head, rotary positions, and
// int8 rows into and out of the cache.
//
//   y_i = norm_i x_i / sqrt(mean(x^2) + eps)
//   angle of pair j at position p: 2 pi frac(p turns_j / 2^64), exact modulo a turn
//   scale = binary16(max |y| / 127), code_i = clamp(rint(y_i / scale), -127, 127)
//
// One warp per row and head, a row's elements spread over the lanes; a rotated
// element finds its partner in shared memory.
#include <math.h>

#include "tq_common.cuh"
#include "tq_int8_cache.cuh"

namespace tq {
namespace i8 {
namespace {

constexpr int RT = 256;             // threads of a CTA
constexpr int PER = 8;              // elements of a row per lane

template <int TYPE>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  if (TYPE == TQ_F32) return static_cast<const float *>(p)[i];
  if (TYPE == TQ_F16) return __half2float(static_cast<const __half *>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
template <int TYPE>
__device__ __forceinline__ void store1(void *p, int64_t i, float x) {
  if (TYPE == TQ_F32) static_cast<float *>(p)[i] = x;
  else if (TYPE == TQ_F16) static_cast<__half *>(p)[i] = __float2half_rn(x);
  else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

template <int TYPE>
__global__ void __launch_bounds__(RT) step_rows_kernel(const StepArgs a) {
  __shared__ float rows[RT / 32][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = a.part[Q].n_heads + a.part[K].n_heads + a.part[V].n_heads;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (RT / 32) + warp;
  const int64_t row = unit / heads;
  if (row >= a.n_rows) return;
  int head = static_cast<int>(unit - row * heads), w = Q;
  while (head >= a.part[w].n_heads) head -= a.part[w++].n_heads;
  const Part &p = a.part[w];
  const int pos = a.positions ? a.positions[row] : 0;
  const int64_t slot = a.slots ? a.slots[row] : 0;
  const bool cell_ok = static_cast<uint64_t>(slot) < static_cast<uint64_t>(a.n_cells);
  if (lane == 0 && (pos < -1 || (p.cells && !cell_ok && slot != -1))) set_status(a.status, TQ_ERR_DEVICE_CHECK);
  if (pos < 0 || (p.cells && !cell_ok)) return;

  const int d = p.head_dim;
  const int64_t at = row * p.src_stride + static_cast<int64_t>(head) * d;
  float x[PER], ss = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    x[i] = e < d ? load1<TYPE>(p.src, at + e) : 0.f;
    ss = fmaf(x[i], x[i], ss);
  }
  if (p.norm) {
    const float mean = warp_sum(ss) / static_cast<float>(d) + a.eps, r = mean != 0.f ? rsqrtf(mean) : 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 32 * i < d) x[i] *= r * p.norm[lane + 32 * i];
  }
  if (p.turns) {
#pragma unroll
    for (int i = 0; i < PER; ++i) rows[warp][lane + 32 * i] = x[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      if (e >= a.rot) continue;
      const bool half = a.layout == TQ_ROPE_HALF;
      const int h = a.rot / 2, j = half ? (e < h ? e : e - h) : e >> 1;
      const bool second = half ? e >= h : e & 1;
      const float other = rows[warp][half ? (second ? e - h : e + h) : e ^ 1];
      const uint64_t t = a.turns[j];
      const uint32_t turn = static_cast<uint32_t>(pos) * static_cast<uint32_t>(t >> 32) +
                            __umulhi(static_cast<uint32_t>(pos), static_cast<uint32_t>(t));
      float s, c;
      sincospif(static_cast<float>(static_cast<int32_t>(turn)) * 0x1p-31f, &s, &c);
      s *= a.sign;
      x[i] = a.gain * (second ? fmaf(other, s, x[i] * c) : fmaf(-other, s, x[i] * c));
    }
  }
  if (!p.cells) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 32 * i < d) store1<TYPE>(p.dst, row * p.dst_stride + static_cast<int64_t>(head) * d + lane + 32 * i, x[i]);
    return;
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -127.f * 65504.f), 127.f * 65504.f) : 0.f;
    top = fmaxf(top, fabsf(x[i]));
  }
  const __half hs = __float2half_rn(__fdiv_rn(warp_max(top), 127.f));
  const float s = __half2float(hs);
  const int64_t cell_row = slot * p.n_heads + head;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (lane + 32 * i < d)
      p.cells[cell_row * d + lane + 32 * i] =
          s > 0.f ? static_cast<int8_t>(rintf(fminf(fmaxf(__fdiv_rn(x[i], s), -127.f), 127.f))) : 0;
  if (lane == 0) p.scales[cell_row] = __half_as_ushort(hs);
}

template <int TYPE>
__global__ void __launch_bounds__(RT) get_rows_kernel(const p4::RowsArgs a) {
  const int lane = threadIdx.x & 31;
  const int heads = a.n_heads[0] + a.n_heads[1];
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (RT / 32) + (threadIdx.x >> 5);
  const int64_t row = unit / heads;
  if (row >= a.n_rows) return;
  int head = static_cast<int>(unit - row * heads);
  const int w = head >= a.n_heads[0];
  if (w) head -= a.n_heads[0];
  const int64_t slot = a.slots[row];
  if (static_cast<uint64_t>(slot) >= static_cast<uint64_t>(a.n_cells)) {
    if (slot != -1 && lane == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);
    return;
  }
  const int d = a.head_dim[w];
  const int64_t cell_row = slot * a.n_heads[w] + head;
  const float s = __half2float(__ushort_as_half(a.scales[w][cell_row]));
  for (int e = lane; e < d; e += 32)
    store1<TYPE>(a.dst[w], row * a.stride[w] + static_cast<int64_t>(head) * d + e,
                 s * static_cast<float>(reinterpret_cast<const int8_t *>(a.codes[w])[cell_row * d + e]));
}

unsigned grid_of(int64_t n_rows, int64_t heads) { return static_cast<unsigned>((n_rows * heads + RT / 32 - 1) / (RT / 32)); }

}  // namespace

cudaError_t launch_step_rows(int type, const StepArgs &a, cudaStream_t s) {
  const unsigned grid = grid_of(a.n_rows, a.part[Q].n_heads + a.part[K].n_heads + a.part[V].n_heads);
  switch (type) {
    case TQ_F32: step_rows_kernel<TQ_F32><<<grid, RT, 0, s>>>(a); break;
    case TQ_F16: step_rows_kernel<TQ_F16><<<grid, RT, 0, s>>>(a); break;
    default: step_rows_kernel<TQ_BF16><<<grid, RT, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_get_rows(int type, const p4::RowsArgs &a, cudaStream_t s) {
  const unsigned grid = grid_of(a.n_rows, a.n_heads[0] + a.n_heads[1]);
  switch (type) {
    case TQ_F32: get_rows_kernel<TQ_F32><<<grid, RT, 0, s>>>(a); break;
    case TQ_F16: get_rows_kernel<TQ_F16><<<grid, RT, 0, s>>>(a); break;
    default: get_rows_kernel<TQ_BF16><<<grid, RT, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace i8
}  // namespace tq
