// Single-token attention over int8 cells.
//
//   out = sum_t p_t s^V_t c^V_t / sum_t p_t,   p_t = 2^(x_t - R),  x_t = scale log2(e) s^K_t (q . c^K_t)
//
// One CTA per sequence and query head, a warp per key in turn; every warp keeps a
// running maximum, sum and values, which the CTA puts together at the end.
#include <math.h>

#include "tq_common.cuh"
#include "tq_int8_cache.cuh"

namespace tq {
namespace i8 {
namespace {

constexpr int NW = 8;
constexpr int PER = 8;              // elements of a row per lane

__device__ __forceinline__ float load16(const void *p, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : __half2float(static_cast<const __half *>(p)[i]);
}

__global__ void __launch_bounds__(NW * 32) decode_kernel(const p4::AttnArgs a) {
  __shared__ float vals[NW][256];
  __shared__ float stat[NW][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seq = blockIdx.x / a.n_heads, head = blockIdx.x - seq * a.n_heads, hv = head / a.group;
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  int len = a.seq_len[seq];
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);
    len = len < 0 ? 0 : static_cast<int>(cap);
  }
  float q[PER], o[PER], R = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    q[i] = e < a.dk ? load16(a.q, seq * a.q_stride + static_cast<int64_t>(head) * a.dk + e, a.bf16) : 0.f;
    o[i] = 0.f;
  }
  for (int t = warp; t < len; t += NW) {
    const int page = a.block_table[static_cast<int64_t>(seq) * a.max_pages + (t >> a.page_shift)];
    const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages);
    if (!ok && lane == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);
    const int64_t cell = (static_cast<int64_t>(page) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
    const int64_t r = cell * a.n_kv_heads + hv;
    const float ks = ok ? __half2float(__ushort_as_half(a.k_scales[r])) : 0.f;
    const float vs = ok ? __half2float(__ushort_as_half(a.v_scales[r])) : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (ok && lane + 32 * i < a.dk)
        dot = fmaf(q[i], static_cast<float>(reinterpret_cast<const int8_t *>(a.k_codes)[r * a.dk + lane + 32 * i]), dot);
    const float x = warp_sum(dot) * ks * a.scale_log2;
    if (x > R) {
      const float f = exp2f(R - x);
      R = x;
      l *= f;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] *= f;
    }
    const float p = exp2f(x - R);
    l += p;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (ok && lane + 32 * i < a.dv)
        o[i] = fmaf(p * vs, static_cast<float>(reinterpret_cast<const int8_t *>(a.v_codes)[r * a.dv + lane + 32 * i]), o[i]);
  }
  if (lane == 0) {
    stat[warp][0] = R;
    stat[warp][1] = l;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) vals[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float M = -INFINITY, sum = 0.f, y = 0.f;
  for (int w = 0; w < NW; ++w) M = fmaxf(M, stat[w][0]);
  const int e = threadIdx.x;
  for (int w = 0; w < NW; ++w) {
    const float f = stat[w][0] == -INFINITY ? 0.f : exp2f(stat[w][0] - M);
    sum += f * stat[w][1];
    y += f * vals[w][e];
  }
  y = sum != 0.f ? y / sum : 0.f;
  if (e < a.dv) {
    const int64_t at = (static_cast<int64_t>(seq) * a.n_heads + head) * a.dv + e;
    if (a.bf16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
    else static_cast<__half *>(a.out)[at] = __float2half_rn(y);
  }
}

}  // namespace

cudaError_t launch_decode(const p4::AttnArgs &a, cudaStream_t s) {
  decode_kernel<<<static_cast<unsigned>(a.n_seq) * a.n_heads, NW * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace i8
}  // namespace tq
