// Rows into and out of the paged 4-bit cache.
//
// Quantise-on-write of a row x (one token, one KV head): with a = min x, b = max x,
//   offset m = binary16(a), scale s = binary16((b - a) / 15),
//   code_i = clamp(rint((x_i - m) / s), 0, 15)      (0 where s = 0)
// in fp32 with IEEE division, so the codes are those of the plain formula.  The
// binary16 roundings of m and s are part of the format: the codes are chosen
// against the rounded pair that a reader multiplies with.
//
// Both directions read or write 2 or 4 bytes and 0.53 bytes per element.  A lane
// holds twice 8 elements of a row, a row's lanes side by side, so that every load
// and store of 16-bit elements is of whole sectors (16 elements in a line per lane:
// rows out 26.2 instead of 21.2 us); 4, 8 or 16 lanes share a row (widths 64, 128,
// 256), and minimum and maximum take 2 to 4 shuffles.  K and V go in one launch.
// - Quotients: with r the correctly rounded reciprocal of s (one per row),
//   q0 = d r and q = q0 + r (d - q0 s) is the correctly rounded d / s (Markstein,
//   "Computation of elementary functions on the IBM RISC System/6000 processor",
//   1990): the remainder is exact, and a quotient by an 11-bit s never lies nearer
//   than 2^-36 of itself to the middle of two floats.  Three operations instead of
//   a division; rows whose s is below 2^-14, where something could underflow, divide.
// - The steps run on pairs of elements (f32x2).  A code is rounded by adding
//   1.5 2^23 and read off the sum's low bits: eight sums, each 16 times the one
//   before, make eight codes and one constant.  Clamping is left out where the row's
//   smallest and largest element show that no code leaves 0 .. 15 (nearly every row).
// - Minimum and maximum of 16-bit inputs are taken on their pairs.  Rows with NaN or
//   magnitudes beyond 65504 show in them (NaN-propagating) and are cleaned on a path
//   of their own.
// Measured, 20001 rows of 8 heads of 128, K and V, in turn over sets larger than L2:
//   rows in   fp16 28.7 us (3.6 TB/s), bf16 29.4 us, fp32 31.6 us (5.9 TB/s)
//   rows out  fp16 21.2 us (4.9 TB/s), bf16 21.6 us, fp32 41.0 us (4.5 TB/s)
// Rows in are bound by instructions: 16-bit rows take nearly as long as 32-bit ones.
// 40 registers and 6 CTAs per SM hide their latencies best (4 CTAs 33.2 us, 5 CTAs
// 30.1 us; two rows per thread 31.0 us, four 33.0 us).  Of 32 rows, the launch and
// the chain slot - row - store are all there is.
#include "tq_common.cuh"
#include "tq_paged4.cuh"

namespace tq {
namespace p4 {
namespace {

constexpr int RT = 256;             // threads of a CTA

// 8 consecutive elements as they are in memory (32-bit ones: two fours)
template <int TYPE>
struct Raw {
  uint4 u[TYPE == TQ_F32 ? 2 : 1];
};
template <int TYPE>
__device__ __forceinline__ void load8(const void *src, int64_t at, Raw<TYPE> &r) {
  if (TYPE == TQ_F32) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(src) + at);
    r.u[0] = __ldcs(p);
    r.u[TYPE == TQ_F32 ? 1 : 0] = __ldcs(p + 1);
  } else {
    r.u[0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + at));
  }
}
template <int TYPE>
__device__ __forceinline__ void unpack8(const Raw<TYPE> &w, float *x) {
  if (TYPE == TQ_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = w.u[TYPE == TQ_F32 ? i : 0];
      x[4 * i] = __uint_as_float(u.x);
      x[4 * i + 1] = __uint_as_float(u.y);
      x[4 * i + 2] = __uint_as_float(u.z);
      x[4 * i + 3] = __uint_as_float(u.w);
    }
  } else {
    const uint32_t r[4] = {w.u[0].x, w.u[0].y, w.u[0].z, w.u[0].w};
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

// smallest and largest of 8 elements, NaN if there is one
template <int TYPE>
__device__ __forceinline__ void range8(const Raw<TYPE> &w, float &lo, float &hi) {
  if (TYPE == TQ_F32) {
    float x[8];
    unpack8<TYPE>(w, x);
    lo = hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = min_nan(lo, x[i]);
      hi = max_nan(hi, x[i]);
    }
  } else if (TYPE == TQ_F16) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&w.u[0]);
    const __half2 a = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
    const __half2 b = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    lo = __half2float(__hmin_nan(__low2half(a), __high2half(a)));
    hi = __half2float(__hmax_nan(__low2half(b), __high2half(b)));
  } else {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w.u[0]);
    const __nv_bfloat162 a = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
    const __nv_bfloat162 b = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    lo = __bfloat162float(__hmin_nan(__low2bfloat16(a), __high2bfloat16(a)));
    hi = __bfloat162float(__hmax_nan(__low2bfloat16(b), __high2bfloat16(b)));
  }
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

// Which elements a thread holds: 8 from `e0` and 8 from `e0 + 8 lanes` on of head
// `head` of row `row`, and where their cell is.
struct Place {
  int which;               // 0: K, 1: V
  int head, e0, lanes;
  int n;                   // eights of the row that this thread has: 0, 1 or 2
  bool ok;                 // a row of this launch whose slot is a cell
  uint32_t cell_row;       // row of the cache planes (page, head, cell in page); below 2^32 by the caches' limits
  int64_t at;              // element of the input or output
};
__device__ __forceinline__ Place place_of(const RowsArgs &a) {
  Place p;
  uint32_t blk = blockIdx.x;
  p.which = blk >= a.k_blocks;
  if (p.which) blk -= a.k_blocks;
  const int sh = a.width[p.which] == 64 ? 2 : a.width[p.which] == 128 ? 3 : 4;     // log2 of the lanes of a row
  p.lanes = 1 << sh;
  p.e0 = (threadIdx.x & (p.lanes - 1)) * 8;
  const uint32_t heads = a.n_heads[p.which];
  const uint64_t rh = (static_cast<uint64_t>(blk) * RT + threadIdx.x) >> sh;
  const uint64_t row = rh <= 0xffffffffu ? static_cast<uint32_t>(rh) / heads : rh / heads;
  p.head = static_cast<int>(rh - row * heads);
  const int d = a.head_dim[p.which];
  p.n = (p.e0 < d) + (p.e0 + 8 * p.lanes < d);
  p.at = static_cast<int64_t>(row) * a.stride[p.which] + static_cast<int64_t>(p.head) * d + p.e0;
  p.ok = false;
  p.cell_row = 0;
  if (row < static_cast<uint64_t>(a.n_rows)) {
    const int64_t slot = __ldg(a.slots + row);
    p.ok = static_cast<uint64_t>(slot) < static_cast<uint64_t>(a.n_cells);
    if (p.ok) {
      const uint32_t cell = static_cast<uint32_t>(slot), page = cell >> a.page_shift;
      p.cell_row = ((page * heads + p.head) << a.page_shift) + (cell & ((1u << a.page_shift) - 1));
    } else if (slot != -1 && p.e0 == 0) {
      set_status(a.status, TQ_ERR_DEVICE_CHECK);
    }
  }
  return p;
}

// the first of the thread's words of codes (the other is `lanes` further on)
__device__ __forceinline__ int64_t codes_at(const Place &p) {
  return static_cast<int64_t>(p.cell_row) * (2 * p.lanes) + p.e0 / 8;
}

template <int TYPE>
__global__ void __launch_bounds__(RT, 6) set_rows_kernel(const RowsArgs a) {
  const Place p = place_of(a);
  const int n = p.ok ? p.n : 0;
  Raw<TYPE> raw[2];
  raw[0] = raw[1] = Raw<TYPE>{};
  if (n >= 1) load8<TYPE>(a.src[p.which], p.at, raw[0]);
  if (n >= 2) load8<TYPE>(a.src[p.which], p.at + 8 * p.lanes, raw[1]);
  float lo = INFINITY, hi = -INFINITY;
  if (n >= 1) range8<TYPE>(raw[0], lo, hi);
  if (n >= 2) {
    float l1, h1;
    range8<TYPE>(raw[1], l1, h1);
    lo = min_nan(lo, l1);
    hi = max_nan(hi, h1);
  }
  float x[16];
  unpack8<TYPE>(raw[0], x);
  unpack8<TYPE>(raw[1], x + 8);
  if (n > 0 && !(lo >= -65504.f && hi <= 65504.f)) {
    // a stored value is finite: NaN counts as 0, larger magnitudes as binary16's largest
    lo = INFINITY;
    hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -65504.f), 65504.f) : 0.f;
      if (i < 8 * n) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
      }
    }
  }
  for (int o = 1; o < p.lanes; o <<= 1) {                  // the lanes of a row are neighbours in one warp
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!p.ok) return;
  const __half hm = __float2half_rn(lo), hs = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
  const float m = __half2float(hm), s = __half2float(hs);
  constexpr float kRound = 12582912.f;                     // 1.5 2^23: a code added to it is its low bits
  uint32_t w[2] = {0, 0};
  if (s >= 0x1p-14f) {
    const float r = __frcp_rn(s);
    const float2 m2 = make_float2(m, m), r2 = make_float2(r, r), s2 = make_float2(-s, -s), up = make_float2(kRound, kRound);
    float2 c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = sub2(make_float2(x[2 * i], x[2 * i + 1]), m2), q0 = mul2(t, r2);
      c[i] = fma2(fma2(q0, s2, t), r2, q0);
    }
    // (x - m) / s lies in [-0.5, 15.5) for every element if it does for the smallest and the largest
    if (!(lo - m >= -0.499f * s && hi - m <= 15.499f * s)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = make_float2(fminf(fmaxf(c[i].x, 0.f), 15.f), fminf(fmaxf(c[i].y, 0.f), 15.f));
    }
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      c[i] = add2(c[i], up);
      w[i >> 2] = w[i >> 2] * 256 + __float_as_uint(c[i].x) + __float_as_uint(c[i].y) * 16;
    }
    constexpr uint32_t base = 0x11111111u * 0x4b400000u;   // what 1.5 2^23 left in each of the eight, modulo 2^32
    w[0] -= base;
    w[1] -= base;
  } else if (s > 0.f) {
#pragma unroll
    for (int i = 15; i >= 0; --i)
      w[i >> 3] = w[i >> 3] * 16 + static_cast<uint32_t>(rintf(fminf(fmaxf(__fdiv_rn(x[i] - m, s), 0.f), 15.f)));
  }
  if (n < 2) w[1] = 0;                                     // zero codes beyond the row
  if (n < 1) w[0] = 0;
  uint32_t *codes = reinterpret_cast<uint32_t *>(a.codes[p.which]) + codes_at(p);
  codes[0] = w[0];
  codes[p.lanes] = w[1];
  if (p.e0 == 0)
    reinterpret_cast<uint32_t *>(a.scales[p.which])[p.cell_row] =
        __half_as_ushort(hs) | static_cast<uint32_t>(__half_as_ushort(hm)) << 16;
}

template <int TYPE>
__global__ void __launch_bounds__(RT) get_rows_kernel(const RowsArgs a) {
  const Place p = place_of(a);
  if (!p.ok || p.n == 0) return;
  const uint32_t *codes = reinterpret_cast<const uint32_t *>(a.codes[p.which]) + codes_at(p);
  const uint32_t sm = __ldcs(reinterpret_cast<const uint32_t *>(a.scales[p.which]) + p.cell_row);
  const uint32_t w[2] = {__ldcs(codes), __ldcs(codes + p.lanes)};
  const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(sm)));
  const float m = __half2float(__ushort_as_half(static_cast<uint16_t>(sm >> 16)));
  const float2 s2 = make_float2(s, s), m2 = make_float2(m, m), big = make_float2(-8388608.f, -8388608.f);
  float x[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {                            // a nibble in the low bits of 2^23 is the float 2^23 + code
    const uint32_t u = w[k / 4] >> (8 * (k & 3));
    const float2 c = add2(make_float2(__uint_as_float((u & 15u) | 0x4b000000u),
                                      __uint_as_float(((u >> 4) & 15u) | 0x4b000000u)), big);
    const float2 y = fma2(s2, c, m2);
    x[2 * k] = y.x;
    x[2 * k + 1] = y.y;
  }
  store8<TYPE>(a.dst[p.which], p.at, x);
  if (p.n >= 2) store8<TYPE>(a.dst[p.which], p.at + 8 * p.lanes, x + 8);
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
