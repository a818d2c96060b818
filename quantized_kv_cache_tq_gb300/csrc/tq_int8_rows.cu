// Rows on their way to the attention: RMS norm per head, rotary positions, and
// int8 rows into and out of the cache.
//
//   y_i = norm_i x_i / sqrt(mean(x^2) + eps)
//   angle of pair j at position p: 2 pi frac(p turns_j / 2^64), exact modulo a turn
//   scale = binary16(max |y| / 127), code_i = clamp(rint(y_i / scale), -127, 127)
//
// 2 to 8 bytes an element are read or written and some 10 operations done: memory is
// what bounds long calls, latency short ones.
// - A lane holds twice 8 elements of a row, 4, 8 or 16 lanes a row (widths 64, 128,
//   256), so that every access is of 8 or 16 bytes and neighbouring lanes share
//   sectors.  Which two eights: in the half layout those that turn together, so that
//   no element looks for its partner in another lane (half_any, where half of rot_dim
//   is no multiple of 8: the partners are read a second time, element by element).
// - The angle is an integer product: the position times the pair's 64-bit fraction of
//   a turn, of which the upper 32 bits below the whole turns are kept.  Sine and cosine
//   are then polynomials on an eighth of a turn either way (turn_sincos), eight per
//   thread, used for all heads that the thread goes through.
// - A thread goes through 1 to 8 heads of its row, the next one's elements on their way
//   while it works; which, the launch chooses by how many CTAs there are (heads_per).
#include <math.h>

#include "tq_common.cuh"
#include "tq_int8_cache.cuh"

namespace tq {
namespace i8 {
namespace {

constexpr int RT = 256;             // threads of a CTA
#ifndef NB0
#define NB0 4
#endif
#ifndef NB1
#define NB1 4
#endif
#ifndef MAXH
#define MAXH 8
#endif
#ifndef ENOUGH
#define ENOUGH 8
#endif
constexpr int kEnough = ENOUGH;
constexpr float kTop = 127.f * 65504.f;

enum Rot { kNone = 0, kHalf = 1, kInterleaved = 2, kHalfAny = 3 };

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
__device__ __forceinline__ void unpack8(const Raw<TYPE> &w, float2 *x) {
  if (TYPE == TQ_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = w.u[TYPE == TQ_F32 ? i : 0];
      x[2 * i] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      x[2 * i + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  } else {
    const uint32_t r[4] = {w.u[0].x, w.u[0].y, w.u[0].z, w.u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == TQ_F16) x[i] = __half22float2(*reinterpret_cast<const __half2 *>(&r[i]));
      else x[i] = make_float2(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u));
    }
  }
}
template <int TYPE>
__device__ __forceinline__ void store8(void *dst, int64_t at, const float2 *x) {
  if (TYPE == TQ_F32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(dst) + at);
    p[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    p[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
  } else {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == TQ_F16) {
        const __half2 h = __floats2half2_rn(x[i].x, x[i].y);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + at) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}
template <int TYPE>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  if (TYPE == TQ_F32) return __ldcs(static_cast<const float *>(p) + i);
  const uint16_t u = __ldcs(static_cast<const uint16_t *>(p) + i);
  return TYPE == TQ_F16 ? __half2float(__ushort_as_half(u)) : __uint_as_float(static_cast<uint32_t>(u) << 16);
}

// sin and cos of a 32-bit fraction of a turn: the nearest quarter turn taken off exactly, then polynomials in the
// angle t on [-pi/4, pi/4], fitted for the least largest error (sine 3.6e-9 relative, cosine 1e-10; what counts is the
// rounding of t and of the sums, some 1e-7).
__device__ __forceinline__ void turn_sincos(uint32_t turn, float &s, float &c) {
  const uint32_t q = (turn + 0x20000000u) >> 30;
  const float t = static_cast<float>(static_cast<int32_t>(turn - (q << 30))) * 1.46291807926715968e-9f;   // 2 pi / 2^32
  const float u = t * t;
  const float ps = fmaf(t * u, fmaf(u, fmaf(u, -1.9517e-4f, 8.33218e-3f), -1.6666655e-1f), t);
  const float pc = fmaf(u, fmaf(u, fmaf(u, fmaf(u, 2.44384510e-5f, -1.38873675e-3f), 4.16666469e-2f), -0.5f), 1.f);
  s = __uint_as_float(__float_as_uint(q & 1 ? pc : ps) ^ (q << 30 & 0x80000000u));
  c = __uint_as_float(__float_as_uint(q & 1 ? ps : pc) ^ ((q + 1) << 30 & 0x80000000u));
}

// largest magnitude of three numbers, NaN if there is one
__device__ __forceinline__ float top3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Codes of 16 numbers x by scale s > 0, in four words.
__device__ __forceinline__ void codes16(const float2 *x, float s, uint32_t *w) {
  float2 c[8];
  if (s >= 0x1p-14f) {
    // the correctly rounded quotient from the correctly rounded reciprocal: q0 = x r, q = q0 + r (x - q0 s) (Markstein,
    // "Computation of elementary functions on the IBM RISC System/6000 processor", 1990); at most 127 (1 + 2^-11)
    const float r = __frcp_rn(s);
    const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 q0 = mul2(x[i], r2);
      c[i] = fma2(fma2(q0, s2, x[i]), r2, q0);
    }
  } else {                            // scales below binary16's normal numbers: rounded by up to half of themselves
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = make_float2(fminf(fmaxf(__fdiv_rn(x[i].x, s), -127.f), 127.f), fminf(fmaxf(__fdiv_rn(x[i].y, s), -127.f), 127.f));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = add2(c[i], make_float2(12582912.f, 12582912.f));   // 1.5 2^23: the code in the low byte
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = prmt_b32(prmt_b32(__float_as_uint(c[2 * i].x), __float_as_uint(c[2 * i].y), 0x0040u),
                    prmt_b32(__float_as_uint(c[2 * i + 1].x), __float_as_uint(c[2 * i + 1].y), 0x0040u), 0x5410u);
}

template <int TYPE, int ROT>
__global__ void __launch_bounds__(RT, ROT == kNone ? NB0 : ROT == kHalfAny ? 2 : NB1) step_rows_kernel(const StepArgs a) {
  // ---- which tensor, which heads, which row
  int w = Q, group = blockIdx.y;
  while (group >= a.groups[w]) group -= a.groups[w++];
  const Part &p = a.part[w];
  const int d = p.head_dim, sh = d <= 64 ? 2 : d <= 128 ? 3 : 4, lanes = 1 << sh;      // lanes of a row
  const int l = threadIdx.x & (lanes - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (RT >> sh) + (threadIdx.x >> sh);
  int pos = -1;
  bool ok = row < a.n_rows;
  int64_t slot = 0;
  if (ok) {
    pos = ROT == kNone ? 0 : __ldg(a.positions + row);
    if (p.cells) slot = __ldg(a.slots + row);
    const bool cell_ok = !p.cells || static_cast<uint64_t>(slot) < static_cast<uint64_t>(a.n_cells);
    if (l == 0 && (pos < -1 || (!cell_ok && slot != -1))) set_status(a.status, TQ_ERR_DEVICE_CHECK);
    ok = pos >= 0 && cell_ok;
  }
  const bool turns = ROT != kNone && p.turns;

  // ---- the lane's two eights
  const int h = a.rot / 2;
  int c0 = l, c1 = l + lanes;
  if (ROT == kHalf && turns) {        // eights j and j + h / 8 turn together, the ones that pass are paired as they come
    const int n = h / 8;
    c0 = l < n ? l : n + l;
    c1 = l < n ? n + l : lanes + l;
  }
  const int n_in = ok ? (8 * c0 < d) + (8 * c1 < d) : 0;                               // (c0 < c1)

  // ---- angles: half, of pairs 8 c0 ..; interleaved, of pairs 4 c0 .. and 4 c1 ..; half_any, of each element
  constexpr int NA = ROT == kNone ? 1 : ROT == kHalfAny ? 16 : 8;
  float ca[NA], sa[NA];
  bool turned[2] = {false, false};                                                     // whether an eight turns at all
  if (turns && ok) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int e = 8 * (NA == 16 && i >= 8 ? c1 : c0) + (i & 7);                      // (half_any: the element)
      const int j = ROT == kHalf ? 8 * c0 + i : ROT == kInterleaved ? 4 * (i < 4 ? c0 : c1) + (i & 3) : e < h ? e : e - h;
      if (ROT == kInterleaved || ROT == kHalfAny) turned[NA == 16 ? i / 8 : i / 4] |= ROT == kHalfAny ? e < a.rot : j < h;
      else turned[0] = turned[1] = 8 * c0 < h;
      ca[i] = 1.f;
      sa[i] = 0.f;
      if (j < h) {
        const uint64_t t = __ldg(a.turns + j);
        const uint32_t u = static_cast<uint32_t>(pos);
        turn_sincos(u * static_cast<uint32_t>(t >> 32) + __umulhi(u, static_cast<uint32_t>(t)), sa[i], ca[i]);
        sa[i] *= a.sign * a.gain;
        ca[i] *= a.gain;
      }
    }
  }

  // ---- head after head
  int head = group * a.heads_per;
  const int heads = min(p.n_heads, head + a.heads_per);
  int64_t at = row * p.src_stride + static_cast<int64_t>(head) * d;
  Raw<TYPE> next[2];
  next[0] = next[1] = Raw<TYPE>{};
  auto fetch = [&]() {
    if (n_in >= 1) load8<TYPE>(p.src, at + 8 * c0, next[0]);
    if (n_in >= 2) load8<TYPE>(p.src, at + 8 * c1, next[1]);
  };
  fetch();
  for (; head < heads; ++head) {
    float2 x[8];                      // elements 8 c0 .. and 8 c1 ..
    unpack8<TYPE>(next[0], x);
    unpack8<TYPE>(next[1], x + 4);
    float y[ROT == kHalfAny ? 16 : 1];        // half_any: the partners
    if (ROT == kHalfAny && turns) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = 8 * (i < 8 ? c0 : c1) + (i & 7);
        y[ROT == kHalfAny ? i : 0] = ok && e < a.rot ? load1<TYPE>(p.src, at + (e < h ? e + h : e - h)) : 0.f;
      }
      __syncwarp();                   // rows that turn in place: everything is read before something is written
    }
    at += d;
    if (head + 1 < heads) fetch();
    if (p.norm) {
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) s2 = fma2(x[i], x[i], s2);
      float ss = s2.x + s2.y;
      for (int o = 1; o < lanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float mean = ss / static_cast<float>(d) + a.eps, r = mean != 0.f ? rsqrtf(mean) : 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (k < n_in) {
          const float4 *n4 = reinterpret_cast<const float4 *>(p.norm + 8 * (k ? c1 : c0));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 n = __ldg(n4 + i);
            x[4 * k + 2 * i] = mul2(x[4 * k + 2 * i], make_float2(n.x * r, n.y * r));
            x[4 * k + 2 * i + 1] = mul2(x[4 * k + 2 * i + 1], make_float2(n.z * r, n.w * r));
          }
        }
      if (ROT == kHalfAny && turns) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = 8 * (i < 8 ? c0 : c1) + (i & 7);
          if (ok && e < a.rot) y[ROT == kHalfAny ? i : 0] *= r * __ldg(p.norm + (e < h ? e + h : e - h));
        }
      }
    }
    if (ROT == kHalf && turned[0]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = make_float2(ca[2 * i], ca[2 * i + 1]), s = make_float2(sa[2 * i], sa[2 * i + 1]);
        const float2 u = x[i], v = x[4 + i];
        x[i] = sub2(mul2(u, c), mul2(v, s));
        x[4 + i] = fma2(u, s, mul2(v, c));
      }
    }
    if (ROT == kInterleaved) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (turned[k]) {
          const int n = h - 4 * (k ? c1 : c0);             // its pairs that turn
#pragma unroll
          for (int i = 4 * k; i < 4 * k + 4; ++i) {
            const float2 u = x[i], v = make_float2(fmaf(-u.y, sa[i % NA], u.x * ca[i % NA]), fmaf(u.x, sa[i % NA], u.y * ca[i % NA]));
            if (n >= 4 || (i & 3) < n) x[i] = v;
          }
        }
    }
    if (ROT == kHalfAny && turns) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = 8 * (i < 8 ? c0 : c1) + (i & 7), k = ROT == kHalfAny ? i : 0;
        float &v = i & 1 ? x[i / 2].y : x[i / 2].x;
        if (e < a.rot) v = e < h ? fmaf(-y[k], sa[k % NA], v * ca[k % NA]) : fmaf(y[k], sa[k % NA], v * ca[k % NA]);
      }
    }
    if (!p.cells) {
      const int64_t to = row * p.dst_stride + static_cast<int64_t>(head) * d;
      if (n_in >= 1) store8<TYPE>(p.dst, to + 8 * c0, x);
      if (n_in >= 2) store8<TYPE>(p.dst, to + 8 * c1, x + 4);
      continue;
    }
    // ---- int8 (elements beyond the row are zeros)
    float top = top3(x[0].x, x[0].y, x[1].x);
    top = top3(top, x[1].y, x[2].x);
    top = top3(top, x[2].y, x[3].x);
    top = top3(top, x[3].y, x[4].x);
    top = top3(top, x[4].y, x[5].x);
    top = top3(top, x[5].y, x[6].x);
    top = top3(top, x[6].y, x[7].x);
    top = top3(top, x[7].y, x[7].y);
    if (!(top <= kTop)) {             // a stored value is finite: NaN counts as 0, larger magnitudes as the largest
      top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i].x = x[i].x == x[i].x ? fminf(fmaxf(x[i].x, -kTop), kTop) : 0.f;
        x[i].y = x[i].y == x[i].y ? fminf(fmaxf(x[i].y, -kTop), kTop) : 0.f;
        top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
      }
    }
    for (int o = 1; o < lanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (n_in == 0) continue;
    const __half hs = __float2half_rn(__fdiv_rn(top, 127.f));
    const float s = __half2float(hs);
    uint32_t cw[4] = {0, 0, 0, 0};
    if (s > 0.f) codes16(x, s, cw);
    const int64_t cell_row = slot * p.n_heads + head;
    int8_t *to = p.cells + cell_row * d;
    *reinterpret_cast<uint2 *>(to + 8 * c0) = make_uint2(cw[0], cw[1]);
    if (n_in >= 2) *reinterpret_cast<uint2 *>(to + 8 * c1) = make_uint2(cw[2], cw[3]);
    if (l == 0) p.scales[cell_row] = __half_as_ushort(hs);
  }
}

template <int TYPE>
__global__ void __launch_bounds__(RT, 4) get_rows_kernel(const p4::RowsArgs a, const int heads_per, const int k_groups) {
  const int w = static_cast<int>(blockIdx.y) >= k_groups, group = blockIdx.y - (w ? k_groups : 0);
  const int d = a.head_dim[w], sh = d <= 64 ? 2 : d <= 128 ? 3 : 4, lanes = 1 << sh, l = threadIdx.x & (lanes - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (RT >> sh) + (threadIdx.x >> sh);
  if (row >= a.n_rows) return;
  const int64_t slot = __ldg(a.slots + row);
  if (static_cast<uint64_t>(slot) >= static_cast<uint64_t>(a.n_cells)) {
    if (slot != -1 && l == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);
    return;
  }
  const int n_in = (8 * l < d) + (8 * (l + lanes) < d);
  if (n_in == 0) return;
  int head = group * heads_per;
  const int heads = min(a.n_heads[w], head + heads_per);
  int64_t cell_row = slot * a.n_heads[w] + head, to = row * a.stride[w] + static_cast<int64_t>(head) * d + 8 * l;
  uint2 c[2], next[2];
  uint16_t s_next = 0;
  next[1] = make_uint2(0, 0);
  auto fetch = [&]() {
    const uint8_t *p = a.codes[w] + cell_row * d + 8 * l;
    s_next = __ldcs(a.scales[w] + cell_row);
    next[0] = __ldcs(reinterpret_cast<const uint2 *>(p));
    if (n_in >= 2) next[1] = __ldcs(reinterpret_cast<const uint2 *>(p + 8 * lanes));
  };
  fetch();
  for (; head < heads; ++head, to += d) {
    c[0] = next[0];
    c[1] = next[1];
    const __half hs = __ushort_as_half(s_next);
    ++cell_row;
    if (head + 1 < heads) fetch();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k >= n_in) break;
      const uint32_t u[2] = {c[k].x ^ 0x80808080u, c[k].y ^ 0x80808080u};              // code + 128
      if (TYPE == TQ_F16) {
        // 1024 + 128 + code as binary16, 1152 taken off; the product, rounded once, is that of fp32 rounded once
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = prmt_b32(u[i / 2], 0x64646464u, i & 1 ? 0x4342u : 0x4140u);
          const __half2 y = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&v), __float2half2_rn(1152.f)), __half2half2(hs));
          r[i] = *reinterpret_cast<const uint32_t *>(&y);
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dst[w]) + to + 8 * lanes * k) = make_uint4(r[0], r[1], r[2], r[3]);
      } else {
        const float s = __half2float(hs);
        float2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {                      // a byte in the low bits of 2^23 is the float 2^23 + code + 128
          const uint32_t v0 = prmt_b32(u[i / 2], 0x4b000000u, i & 1 ? 0x7442u : 0x7440u);
          const uint32_t v1 = prmt_b32(u[i / 2], 0x4b000000u, i & 1 ? 0x7443u : 0x7441u);
          y[i] = mul2(make_float2(s, s), add2(make_float2(__uint_as_float(v0), __uint_as_float(v1)),
                                              make_float2(-8388736.f, -8388736.f)));
        }
        store8<TYPE>(a.dst[w], to + 8 * lanes * k, y);
      }
    }
  }
}

// Heads that a thread goes through: as many as leave enough CTAs for the SMs (and no more than 65535 in a grid's y).
int heads_of(int64_t row_ctas, const int *n_heads, int parts, int *groups, int *total) {
  for (int per = MAXH;; per /= 2) {
    *total = 0;
    for (int i = 0; i < parts; ++i) *total += groups[i] = (n_heads[i] + per - 1) / per;
    if (per == 1 || row_ctas * *total >= kEnough * sm_count()) {
      while (*total > 65535) {
        per *= 2;
        *total = 0;
        for (int i = 0; i < parts; ++i) *total += groups[i] = (n_heads[i] + per - 1) / per;
      }
      return per;
    }
  }
}

int64_t row_ctas_of(int64_t n_rows, int head_dim) {
  const int rows = RT / (p4::row_width(head_dim) / 16);
  return (n_rows + rows - 1) / rows;
}

template <int TYPE>
void launch_step(const StepArgs &a, dim3 grid, cudaStream_t s) {
  if (!a.positions) step_rows_kernel<TYPE, kNone><<<grid, RT, 0, s>>>(a);
  else if (a.layout == TQ_ROPE_INTERLEAVED) step_rows_kernel<TYPE, kInterleaved><<<grid, RT, 0, s>>>(a);
  else if (a.rot % 16 == 0) step_rows_kernel<TYPE, kHalf><<<grid, RT, 0, s>>>(a);
  else step_rows_kernel<TYPE, kHalfAny><<<grid, RT, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_step_rows(int type, const StepArgs &args, cudaStream_t s) {
  StepArgs a = args;
  int n_heads[3], total = 0;
  int64_t x = 0;
  for (int i = 0; i < 3; ++i) {
    n_heads[i] = a.part[i].n_heads;
    const int64_t r = n_heads[i] ? row_ctas_of(a.n_rows, a.part[i].head_dim) : 0;
    if (r > x) x = r;
  }
  a.heads_per = heads_of(x, n_heads, 3, a.groups, &total);
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(total));
  switch (type) {
    case TQ_F32: launch_step<TQ_F32>(a, grid, s); break;
    case TQ_F16: launch_step<TQ_F16>(a, grid, s); break;
    default: launch_step<TQ_BF16>(a, grid, s); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_get_rows(int type, const p4::RowsArgs &a, cudaStream_t s) {
  int groups[2], total = 0;
  const int64_t k = row_ctas_of(a.n_rows, a.head_dim[0]), v = row_ctas_of(a.n_rows, a.head_dim[1]), x = k > v ? k : v;
  const int per = heads_of(x, a.n_heads, 2, groups, &total);
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(total));
  switch (type) {
    case TQ_F32: get_rows_kernel<TQ_F32><<<grid, RT, 0, s>>>(a, per, groups[0]); break;
    case TQ_F16: get_rows_kernel<TQ_F16><<<grid, RT, 0, s>>>(a, per, groups[0]); break;
    default: get_rows_kernel<TQ_BF16><<<grid, RT, 0, s>>>(a, per, groups[0]); break;
  }
  return cudaGetLastError();
}

}  // namespace i8
}  // namespace tq
