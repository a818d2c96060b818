// Rows into and out of the paged 4-bit cache.
//
// Quantise-on-write of a row x (one token, one KV head): with a = min x, b = max x,
//   offset m = binary16(a), scale s = binary16((b - a) / 15),
//   code_i = clamp(rint((x_i - m) / s), 0, 15)      (0 where s = 0)
// in fp32 with IEEE division, so the codes are those of the plain formula.  The
// binary16 roundings of m and s are part of the format: the codes are chosen
// against the rounded pair that a reader multiplies with.
//
// Both directions are bound by memory (2 or 4 bytes in, 0.53 bytes out per
// element) as long as the arithmetic stays small.  A lane holds 16 consecutive
// elements of a row -- two 16-byte loads of 16-bit input, one 8-byte store of
// codes -- and 4, 8 or 16 lanes share a row (widths 64, 128, 256), so minimum and
// maximum take 2 to 4 shuffles.  K and V go in one launch.
// - Quotients: with r the correctly rounded reciprocal of s (one per row),
//   q0 = d r and q = q0 + r (d - q0 s) is the correctly rounded d / s (Markstein,
//   "Computation of elementary functions on the IBM RISC System/6000 processor",
//   1990): the remainder is exact, and a quotient by an 11-bit s never lies nearer
//   than 2^-36 of itself to the middle of two floats.  Three operations instead of
//   a division; rows whose s is below 2^-14, where something could underflow, divide.
// - A code is rounded by adding and subtracting 1.5 2^23, and four codes are packed
//   by fused multiply-adds as one number below 2^16.
// - Rows with NaN or magnitudes beyond 65504 are found by one check of the row's
//   smallest and largest magnitudes (NaN-propagating) and cleaned on a path of
//   their own.
#include "tq_common.cuh"
#include "tq_paged4.cuh"

namespace tq {
namespace p4 {
namespace {

constexpr int RT = 256;

// 8 consecutive elements as floats
template <int TYPE>
__device__ __forceinline__ void load8(const void *src, int64_t at, float *x) {
  if (TYPE == TQ_F32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(src) + at);
    const float4 u = __ldcs(p), w = __ldcs(p + 1);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + at));
    const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if (TYPE == TQ_F16) f = __half22float2(*reinterpret_cast<const __half2 *>(&r[i]));
      else f = make_float2(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// fminf / fmaxf that hand NaN on
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int TYPE>
__device__ __forceinline__ void store8(void *dst, int64_t at, const float *x) {
  if (TYPE == TQ_F32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(dst) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == TQ_F16) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + at) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// What a thread works on: 16 elements from `e0` on of head `head` of row `row`.
struct Place {
  int which;               // 0: K, 1: V
  int64_t row, cell_row;   // source row; row of the cache planes (page, head, cell in page)
  int head, e0, lanes;
  bool active, ok;         // a row of this launch; its slot is a cell
};

__device__ __forceinline__ Place place_of(const RowsArgs &a) {
  Place p;
  uint32_t blk = blockIdx.x;
  p.which = blk >= a.k_blocks;
  if (p.which) blk -= a.k_blocks;
  const int sh = a.width[p.which] == 64 ? 2 : a.width[p.which] == 128 ? 3 : 4;     // log2 of the lanes of a row
  p.lanes = 1 << sh;
  p.e0 = (threadIdx.x & (p.lanes - 1)) * 16;
  const uint32_t heads = a.n_heads[p.which];
  const uint64_t rh = (static_cast<uint64_t>(blk) * RT + threadIdx.x) >> sh;
  const uint64_t row = rh <= 0xffffffffu ? static_cast<uint32_t>(rh) / heads : rh / heads;
  p.row = static_cast<int64_t>(row);
  p.head = static_cast<int>(rh - row * heads);
  p.active = p.row < a.n_rows;
  p.ok = false;
  p.cell_row = 0;
  if (p.active) {
    const int64_t slot = __ldg(a.slots + p.row);
    p.ok = slot >= 0 && slot < a.n_cells;
    if (!p.ok && slot != -1 && p.e0 == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);
    if (p.ok) {
      const int64_t page = slot >> a.page_shift;
      p.cell_row = ((page * heads + p.head) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
    }
  }
  return p;
}

template <int TYPE>
__global__ void __launch_bounds__(RT) set_rows_kernel(const RowsArgs a) {
  const Place p = place_of(a);
  const int d = a.head_dim[p.which];
  float x[16];
  const int n = p.ok ? min(16, max(0, d - p.e0)) : 0;      // 0, 8 or 16 elements of the row here
  const int64_t at = p.row * a.stride[p.which] + static_cast<int64_t>(p.head) * d + p.e0;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  if (n >= 8) load8<TYPE>(a.src[p.which], at, x);
  if (n >= 16) load8<TYPE>(a.src[p.which], at + 8, x + 8);
  float lo = INFINITY, hi = -INFINITY;
  auto range = [&]() {
    lo = INFINITY;
    hi = -INFINITY;
    if (n >= 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo = min_nan(lo, x[i]);
        hi = max_nan(hi, x[i]);
      }
    }
    if (n >= 16) {
#pragma unroll
      for (int i = 8; i < 16; ++i) {
        lo = min_nan(lo, x[i]);
        hi = max_nan(hi, x[i]);
      }
    }
  };
  range();
  if (n > 0 && !(lo >= -65504.f && hi <= 65504.f)) {
    // a stored value is finite: NaN counts as 0, larger magnitudes as binary16's largest
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -65504.f), 65504.f) : 0.f;
    range();
  }
  for (int o = 1; o < p.lanes; o <<= 1) {                  // the lanes of a row are neighbours in one warp
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!p.ok) return;
  const __half hm = __float2half_rn(lo), hs = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
  const float m = __half2float(hm), s = __half2float(hs);
  constexpr float kRound = 12582912.f;                     // 1.5 2^23
  float pack[4] = {0.f, 0.f, 0.f, 0.f};                    // four codes each
  if (s >= 0x1p-14f && n > 0) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 15; i >= 0; --i) {
      const float t = x[i] - m, q0 = t * r, q = fmaf(fmaf(-q0, s, t), r, q0);
      const float c = (fminf(fmaxf(q, 0.f), 15.f) + kRound) - kRound;
      pack[i >> 2] = fmaf(pack[i >> 2], 16.f, c);
    }
  } else if (s > 0.f) {
#pragma unroll
    for (int i = 15; i >= 0; --i)
      pack[i >> 2] = fmaf(pack[i >> 2], 16.f, rintf(fminf(fmaxf(__fdiv_rn(x[i] - m, s), 0.f), 15.f)));
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = static_cast<uint32_t>(pack[2 * i]) | static_cast<uint32_t>(pack[2 * i + 1]) << 16;
  if (n < 16) w[1] = 0;                                    // zero codes beyond the row
  if (n < 8) w[0] = 0;
  uint8_t *codes = a.codes[p.which] + p.cell_row * (a.width[p.which] / 2) + p.e0 / 2;
  *reinterpret_cast<uint2 *>(codes) = make_uint2(w[0], w[1]);
  if (p.e0 == 0)
    reinterpret_cast<uint32_t *>(a.scales[p.which])[p.cell_row] =
        __half_as_ushort(hs) | static_cast<uint32_t>(__half_as_ushort(hm)) << 16;
}

template <int TYPE>
__global__ void __launch_bounds__(RT) get_rows_kernel(const RowsArgs a) {
  const Place p = place_of(a);
  const int d = a.head_dim[p.which];
  if (!p.ok || p.e0 >= d) return;
  const uint32_t sm = reinterpret_cast<const uint32_t *>(a.scales[p.which])[p.cell_row];
  const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(sm)));
  const float m = __half2float(__ushort_as_half(static_cast<uint16_t>(sm >> 16)));
  const uint2 w = *reinterpret_cast<const uint2 *>(a.codes[p.which] + p.cell_row * (a.width[p.which] / 2) + p.e0 / 2);
  const int64_t at = p.row * a.stride[p.which] + static_cast<int64_t>(p.head) * d + p.e0;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t c = ((i < 8 ? w.x : w.y) >> (4 * (i & 7))) & 15u;
    x[i] = fmaf(s, static_cast<float>(c), m);
  }
  store8<TYPE>(a.dst[p.which], at, x);
  if (d - p.e0 >= 16) store8<TYPE>(a.dst[p.which], at + 8, x + 8);
}

unsigned grid_of(RowsArgs &a) {
  unsigned b[2];
  for (int i = 0; i < 2; ++i) b[i] = static_cast<unsigned>((a.n_rows * a.n_heads[i] * (a.width[i] / 16) + RT - 1) / RT);
  a.k_blocks = b[0];
  return b[0] + b[1];
}

}  // namespace

cudaError_t launch_set_rows(int type, const RowsArgs &args, cudaStream_t s) {
  RowsArgs a = args;
  const unsigned grid = grid_of(a);
  switch (type) {
    case TQ_F32: set_rows_kernel<TQ_F32><<<grid, RT, 0, s>>>(a); break;
    case TQ_F16: set_rows_kernel<TQ_F16><<<grid, RT, 0, s>>>(a); break;
    default: set_rows_kernel<TQ_BF16><<<grid, RT, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_get_rows(int type, const RowsArgs &args, cudaStream_t s) {
  RowsArgs a = args;
  const unsigned grid = grid_of(a);
  switch (type) {
    case TQ_F32: get_rows_kernel<TQ_F32><<<grid, RT, 0, s>>>(a); break;
    case TQ_F16: get_rows_kernel<TQ_F16><<<grid, RT, 0, s>>>(a); break;
    default: get_rows_kernel<TQ_BF16><<<grid, RT, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace p4
}  // namespace tq
