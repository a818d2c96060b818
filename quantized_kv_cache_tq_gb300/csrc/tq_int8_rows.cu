// Rows on their way to the attention: RMS norm per head, rotary positions, and
// int8 rows into and out of the cache.
//
//   y_i = norm_i x_i / sqrt(mean(x^2) + eps)
//   angle of pair j at position p: 2 pi frac(p turns_j / 2^64), exact modulo a turn
//   scale = binary16(max |y| / 127), code_i = clamp(rint(y_i / scale), -127, 127)
//
// 2 to 8 bytes an element are read or written and some 10 operations done: memory is what bounds long calls, latency
// short ones.  20001 rows of 32 + 8 heads of 128, 16-bit, rotated: 65 us, 6.3 TB/s (92% of a copy's rate), normed first
// 71; 16001 rows of which K and V go into the cache 64 us (83%; normed 84, held by its instructions: 58% of the issue
// slots are busy without the norm); 20001 rows of 8 heads into the cache 22.5 and out of it 22.8 (80%).  48 rows 2.4 us.
// - A lane holds twice 8 elements of a row, 4, 8 or 16 lanes a row (widths 64, 128, 256), so that every access is of 8
//   or 16 bytes and neighbouring lanes share sectors.  Which two eights: in the half layout those that turn together, so
//   that no element looks for its partner in another lane (half_any, where half of rot_dim is no multiple of 8: by way of
//   shared memory, 80-wide heads, 20 of them turned, 182 -> 73 us).  32-bit rows that nothing turns: four fours, since an
//   eight is two halves of a sector there (20001 rows in 47 -> 37.5 us, out 50 -> 39.8, now 36.7).
// - The angle is an integer product: the position times the pair's 64-bit fraction of
//   a turn, of which the upper 32 bits below the whole turns are kept.  Sine and cosine
//   are then polynomials on an eighth of a turn either way (turn_sincos), eight per
//   thread, used for all heads that the thread goes through.
// - A unit of work is one head of the 8 to 32 rows that a CTA takes side by side.  All units of a tensor, tile after
//   tile, and of one tensor after the other form a line, of which each CTA takes an equal share (one unit, in short
//   calls): no CTA is left over for a last wave, and what a row needs -- position, slot, angles -- is worked out once
//   for the heads that follow.  Each thread copies its elements of the next units to a ring of its own in shared memory
//   (cp.async) while it works: registers hold one unit, and nobody waits for anybody else.
#include <math.h>

#include "tq_common.cuh"
#include "tq_int8_cache.cuh"

namespace tq {
namespace i8 {
namespace {

constexpr int RT = 128;             // threads of a CTA
constexpr int kStages = 3;          // units of a thread's ring
// CTAs per SM: what the registers allow.  Rotations run best with 95 of them: six CTAs instead of five (rope of 20001
// rows 71 instead of 65 us) leave the loads of positions and angles one after the other, four (67 us) too few of them
// on their way.  More stages than three read no faster and hinder the writes (71 us with four).
constexpr int ctas_of(int rot) { return rot == 0 ? 8 : rot == 3 ? 4 : 5; }
// Rows out: 16 CTAs of 32 registers a thread; of fp32 rows ten, which spill nothing (20001 rows 36.7 us; sixteen spilled
// and took 39.8, twelve 39.0).
constexpr int get_ctas(int type) { return type == TQ_F32 ? 10 : 16; }
constexpr float kTop = 127.f * 65504.f;

enum Rot { kNone = 0, kHalf = 1, kInterleaved = 2, kHalfAny = 3 };

// 8 consecutive elements as they are in memory (32-bit ones: two fours)
template <int TYPE>
struct Raw {
  uint4 u[TYPE == TQ_F32 ? 2 : 1];
};

// 16 bytes, or (n = 0) zeros.  Eights of 32-bit elements are copied in two halves of a sector, which meet in L1.
template <int TYPE>
__device__ __forceinline__ void cp16(uint32_t to, const void *from, uint32_t n) {
  if (TYPE == TQ_F32)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
  return u;
}
__device__ __forceinline__ uint32_t lds4b(uint32_t at) {
  uint32_t u;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(at) : "memory");
  return u;
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
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
// g sin and g cos of a 32-bit fraction of a turn: the nearest quarter turn taken off exactly, then polynomials in the
// angle on [-pi/4, pi/4], fitted for the least largest error (with these coefficients: sine 4.6e-9 relative, cosine
// 5.2e-10); the results are rounded once.  FINE: the angle is t + low, t an fp32 number, low what its rounding, that of
// 2 pi / 2^32 (whose rest is kLow) and the integer's last 6 bits leave.  fp32 rows have it, whose error it makes less by
// a twelfth (rms 4.25e-8 -> 3.9e-8, 10000 rows 71.3 us with and without); 16-bit rows round 2^12 times as coarsely (and
// 300 of them took 3.6 us with it, 3.3 without).
template <bool FINE>
__device__ __forceinline__ void turn_sincos(uint32_t turn, float g, float &s, float &c) {
  constexpr float kTurn = 1.46291807926715968e-9f, kLow = static_cast<float>(1.46291807926715968e-9 - static_cast<double>(kTurn));
  const uint32_t q = (turn + 0x20000000u) >> 30;
  const int32_t n = static_cast<int32_t>(turn - (q << 30));
  const float high = static_cast<float>(FINE ? n & ~63 : n), t = high * kTurn;
  const float low = FINE ? fmaf(high, kLow, fmaf(static_cast<float>(n & 63), kTurn, fmaf(high, kTurn, -t))) : 0.f;
  const float u = t * t;
  const float ps = fmaf(u, fmaf(u, -1.9517e-4f, 8.33218e-3f), -1.6666655e-1f);
  const float pc = fmaf(u, fmaf(u, fmaf(u, 2.44384510e-5f, -1.38873675e-3f), 4.16666469e-2f), -0.5f);
  const float gs = fmaf(t, g, g * (FINE ? fmaf(t * u, ps, low) : t * u * ps));
  const float gc = fmaf(g, FINE ? fmaf(u, pc, -t * low) : u * pc, g);
  s = __uint_as_float(__float_as_uint(q & 1 ? gc : gs) ^ (q << 30 & 0x80000000u));
  c = __uint_as_float(__float_as_uint(q & 1 ? gs : gc) ^ ((q + 1) << 30 & 0x80000000u));
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
    // The correctly rounded quotient from the correctly rounded reciprocal: q0 = x r, q = q0 + r (x - q0 s) (Markstein,
    // "Computation of elementary functions on the IBM RISC System/6000 processor", 1990); it is at most 127 (1 + 2^-11).
    // One Newton step rounds the reciprocal of an 11-bit number correctly: none lies nearer than 2^-36 of itself to the
    // middle of two floats.
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = fmaf(fmaf(-s, r, 1.f), r, r);
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

// The mean of a row's squares, `lanes` lanes a row.
__device__ __forceinline__ float mean_square(const float2 *x, int lanes, int d) {
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) s2 = fma2(x[i], x[i], s2);
  float ss = s2.x + s2.y;
  for (int o = 1; o < lanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return ss / static_cast<float>(d);
}
// A row's elements in shared memory times a power of two, which is returned: the row's largest number or `root` comes to
// lie in [1, 4), one of them at least.  Rows that do not ask for it stay as they are.  `at`: the thread's first word of
// `words` that lie `step` bytes apart.
template <int TYPE>
__device__ __forceinline__ float rescale(uint32_t at, int words, uint32_t step, int lanes, float root, bool asked) {
  constexpr int E = TYPE == TQ_F32 ? 1 : 2;       // elements of 32 bits (16-bit ones: bfloat16)
  float top = root;
#pragma unroll 1
  for (int i = 0; i < 4 * words; ++i) {
    const uint32_t u = lds4b(at + (i >> 2) * step + (i & 3) * 4);
    top = fmaxf(top, fabsf(__uint_as_float(E == 1 ? u : u & 0xffff0000u)));
    if (E == 2) top = fmaxf(top, fabsf(__uint_as_float(u << 16)));
  }
  for (int o = 1; o < lanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float by = asked ? __uint_as_float((254 - min(__float_as_uint(top) >> 23, 253u)) << 23) : 1.f;
#pragma unroll 1
  for (int i = 0; i < 4 * words; ++i) {
    const uint32_t to = at + (i >> 2) * step + (i & 3) * 4, u = lds4b(to);
    uint32_t v;
    if (E == 1) {
      v = __float_as_uint(__uint_as_float(u) * by);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(u << 16) * by, __uint_as_float(u & 0xffff0000u) * by);
      v = *reinterpret_cast<const uint32_t *>(&h);
    }
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
  }
  return by;
}

// a / b of numbers below 2^32, as nearly all are, in 32 bits
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return static_cast<uint64_t>(a) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// log2 of the lanes of a row
__host__ __device__ constexpr int lane_shift(int head_dim) { return head_dim <= 64 ? 2 : head_dim <= 128 ? 3 : 4; }

// The launch may begin beside the one before it (p4::launch_beside); nothing is read or written before that has ended.
__device__ __forceinline__ void after_earlier_launches() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A CTA's share of `n` units, `more` of which are left over for the first CTAs.
struct Share {
  int64_t at, end;
};
__device__ __forceinline__ Share share_of(const Units &u) {
  const int64_t b = blockIdx.x, at = b * u.per + min(b, static_cast<int64_t>(u.more));
  return {at, at + u.per + (b < u.more)};
}

template <int TYPE, int ROT>
__global__ void __launch_bounds__(RT, ctas_of(ROT)) step_rows_kernel(const StepArgs a) {
  constexpr int S = kStages, W = TYPE == TQ_F32 ? 2 : 1;        // stages; 16-byte words of an eight
  constexpr bool kFours = TYPE == TQ_F32 && ROT == kNone;
  __shared__ uint4 ring[S][2 * W][RT];            // each thread's own
  __shared__ float line[ROT == kHalfAny ? RT * 16 + 32 * 4 : 1];      // half_any: rows, where the partners are found
  after_earlier_launches();
  for (Share u = share_of(a.units); u.at < u.end;) {
    // ---- units of one tensor: from head `head` of the rows of tile `tile` on
    int w = Q;
    int64_t unit = u.at;
    while (unit >= a.units.part[w]) unit -= a.units.part[w++];
    int left = static_cast<int>(min(min(u.end - u.at, a.units.part[w] - unit), int64_t{1 << 30}));
    u.at += left;
    const Part &p = a.part[w];
    const int d = p.head_dim, sh = lane_shift(d), lanes = 1 << sh;
    const int l = threadIdx.x & (lanes - 1);
    const int64_t tile = quotient(unit, p.n_heads);
    uint32_t row = static_cast<uint32_t>(tile) * (RT >> sh) + (threadIdx.x >> sh);      // (there are less than 2^31)
    const uint32_t n_rows = static_cast<uint32_t>(a.n_rows);
    int head = static_cast<int>(unit - tile * p.n_heads);
    const bool turns = ROT != kNone && p.turns, stored = p.cells != nullptr;

    // ---- the lane's two eights
    const int h = a.rot / 2;
    int c0 = l, c1 = l + lanes;
    if (ROT == kHalf && turns) {      // eights j and j + h / 8 turn together, the ones that pass are paired as they come
      const int n = h / 8;
      c0 = l < n ? l : n + l;
      c1 = l < n ? n + l : lanes + l;
    }
    // (c0 < c1.  32-bit rows that nothing turns: four fours, l + k lanes, so that every access is of whole sectors.)
    const int n_row = kFours ? max(0, (d - 4 * l + 4 * lanes - 1) >> (sh + 2)) : (8 * c0 < d) + (8 * c1 < d);

    int pos_next = -1;
    int64_t slot_next = -1;
    auto look_up = [&](uint32_t r) {   // a row's position and cell, asked for ahead of time
      if (r < n_rows) {
        pos_next = ROT == kNone ? 0 : __ldg(a.positions + r);
        slot_next = stored ? __ldg(a.slots + r) : 0;
      } else {
        pos_next = -1;
        slot_next = -1;
      }
    };
    look_up(row);

    // ---- copies of the next units' elements, on their way while this one is worked on
    // (rows behind the last one read that one again; eights behind the head dim are zeros)
    constexpr int size = TYPE == TQ_F32 ? 4 : 2;
    auto row_at = [&](uint32_t r, int hd) {
      return static_cast<const char *>(p.src) +
             (min(r, n_rows - 1) * p.src_stride + static_cast<int64_t>(hd) * d + (n_row >= 1 ? (kFours ? 4 * l : 8 * c0) : 0)) * size;
    };
    const char *from = row_at(row, head);
    const int to_c1 = n_row >= 2 ? 8 * (c1 - c0) * size : 0, n_heads = p.n_heads;
    const uint32_t size0 = n_row >= 1 ? 16 : 0, size1 = n_row >= 2 ? 16 : 0;
    uint32_t from_row = row;
    int from_left = left, from_head = head;
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(&ring[0][0][threadIdx.x]));
    constexpr uint32_t kStage = sizeof(ring[0]), kWord = sizeof(ring[0][0]);
    uint32_t fill = ring_at;
    auto fetch = [&]() {
      if (--from_left >= 0) {
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
          if (kFours) cp16<TQ_F16>(fill + i * kWord, i < n_row ? from + 16 * i * lanes : from, i < n_row ? 16 : 0);
          else cp16<TYPE>(fill + i * kWord, from + (i < W ? 0 : to_c1) + 16 * (i % W), i < W ? size0 : size1);
        }
        from += d * size;
        if (++from_head == n_heads) {
          from_head = 0;
          from_row += RT >> sh;
          from = row_at(from_row, 0);
        }
        fill = fill == ring_at + (S - 1) * kStage ? ring_at : fill + kStage;
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch();

    constexpr int NA = ROT == kNone ? 1 : ROT == kHalfAny ? 16 : 8;
    float ca[NA], sa[NA];
    bool turned[2], ok = false;                                                        // whether an eight turns at all
    char *to = nullptr;               // where the unit's first eight goes, and the row's scale
    uint16_t *to_scale = nullptr;
    const int to_next = stored ? d : d * size, to_second = (c1 - c0) * (stored ? 8 : 8 * size);
    int n_in = 0;
    uint32_t stage = ring_at;
    auto take_up = [&]() {            // the row: its position, its cell, its angles
      // half: of pairs 8 c0 ..; interleaved: of pairs 4 c0 .. and 4 c1 ..; half_any: of each element
      auto pair_of = [&](int i) {
        const int e = 8 * (NA == 16 && i >= 8 ? c1 : c0) + (i & 7);                    // (half_any: the element)
        return ROT == kHalf ? 8 * c0 + i : ROT == kInterleaved ? 4 * (i < 4 ? c0 : c1) + (i & 3) : e < h ? e : e - h;
      };
      uint64_t t[NA];
      if (turns)
#pragma unroll
        for (int i = 0; i < NA; ++i) t[i] = pair_of(i) < h ? __ldg(a.turns + pair_of(i)) : 0;
      const int pos = pos_next;
      const int64_t slot = slot_next;
      look_up(row + (RT >> sh));
      const bool cell_ok = !stored || static_cast<uint64_t>(slot) < static_cast<uint64_t>(a.n_cells);
      if (l == 0 && (pos < -1 || (!cell_ok && slot != -1))) set_status(a.status, TQ_ERR_DEVICE_CHECK);
      ok = pos >= 0 && cell_ok;
      if (stored) {                   // (rows of a plane are less than 2^32)
        const uint32_t cell_row = static_cast<uint32_t>(slot) * n_heads + head;
        to = reinterpret_cast<char *>(p.cells) + static_cast<uint64_t>(cell_row) * d + (kFours ? 4 * l : 8 * c0);
        to_scale = p.scales + cell_row;
      } else {
        to = static_cast<char *>(p.dst) + (row * p.dst_stride + static_cast<int64_t>(head) * d + 8 * c0) * size;
      }
      n_in = ok ? n_row : 0;
      turned[0] = turned[1] = false;
      if (turns && ok) {
#pragma unroll
        for (int i = 0; i < NA; ++i) {
          // (a pair beyond the last one: frequency 0, no element asks for it)
          const uint32_t q = static_cast<uint32_t>(pos);
          turn_sincos<TYPE == TQ_F32>(q * static_cast<uint32_t>(t[i] >> 32) + __umulhi(q, static_cast<uint32_t>(t[i])), a.gain, sa[i], ca[i]);
          sa[i] *= ROT == kHalfAny && 8 * (i < 8 ? c0 : c1) + (i & 7) < h ? -a.sign : a.sign;
        }
        turned[0] = ROT == kHalfAny ? 8 * c0 < a.rot : pair_of(0) < h;
        turned[1] = ROT == kHalf ? turned[0] : ROT == kHalfAny ? 8 * c1 < a.rot : pair_of(4 % NA) < h;
      }
    };

    // ---- unit after unit
    for (bool fresh = true; left > 0; --left) {
      if (head == n_heads) {
        head = 0;
        row += RT >> sh;
        fresh = true;
      }
      if (fresh) take_up();
      fresh = false;
      ++head;
      cp_wait<S - 2>();
      float2 x[8];                      // elements 8 c0 .. and 8 c1 ..
      auto read = [&](uint32_t at) {
        Raw<TYPE> r0, r1;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          r0.u[i] = lds16(at + i * kWord);
          r1.u[i] = lds16(at + (W + i) * kWord);
        }
        unpack8<TYPE>(r0, x);
        unpack8<TYPE>(r1, x + 4);
      };
      read(stage);
      stage = stage == ring_at + (S - 1) * kStage ? ring_at : stage + kStage;
      fetch();                          // (not to where this unit's elements are)
      if (p.norm) {
        float mean = mean_square(x, lanes, d) + a.eps;
        if (TYPE != TQ_F16) {           // (its squares lie in [2^-48, 2^32])
          // Rows whose squares may leave fp32's range, once more as multiples of a power of two: the norm is the same.
          const bool far = !(mean >= 0x1p-80f && mean <= 0x1p80f);
          if (__any_sync(0xffffffffu, far)) {
            const uint32_t here_at = stage == ring_at ? ring_at + (S - 1) * kStage : stage - kStage;
            const float root = a.eps_root * rescale<TYPE>(here_at, 2 * W, kWord, lanes, a.eps_root, far);
            read(here_at);
            mean = mean_square(x, lanes, d) + (far ? root * root : a.eps);
          }
        }
        const float r = mean != 0.f ? rsqrtf(mean) : 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (k < n_in) {
            const float4 *n4 = reinterpret_cast<const float4 *>(p.norm + 8 * (k ? c1 : c0));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 n = __ldg(n4 + i);
              x[4 * k + 2 * i] = mul2(mul2(x[4 * k + 2 * i], make_float2(r, r)), make_float2(n.x, n.y));
              x[4 * k + 2 * i + 1] = mul2(mul2(x[4 * k + 2 * i + 1], make_float2(r, r)), make_float2(n.z, n.w));
            }
          }
      }
      if (ROT == kHalf && turned[0]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = make_float2(ca[2 * i], ca[2 * i + 1]), s = make_float2(sa[2 * i], sa[2 * i + 1]);
          const float2 u = x[i], v = x[4 + i];
          x[i] = fma2(make_float2(-v.x, -v.y), s, mul2(u, c));
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
        float *mine = line + (threadIdx.x >> sh) * (16 * lanes + 4);
        __syncwarp();                 // the unit before has been read
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<float2 *>(mine + 8 * (i < 4 ? c0 : c1) + 2 * (i & 3)) = x[i];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (turned[k]) {
#pragma unroll
            for (int i = 8 * k; i < 8 * k + 8; ++i) {
              const int e = 8 * (k ? c1 : c0) + (i & 7), m = i % NA;
              float &v = i & 1 ? x[i / 2].y : x[i / 2].x;
              const float r = fmaf(mine[e < h ? e + h : e - h], sa[m], v * ca[m]);     // (sa: -sin in the first half)
              v = e < a.rot ? r : v;
            }
          }
      }
      char *const here = to;
      to += to_next;
      if (!stored) {
        if (n_in >= 1) store8<TYPE>(here, 0, x);
        if (n_in >= 2) store8<TYPE>(here + to_second, 0, x + 4);
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
      // (top / 127, rounded correctly, as the codes' quotients are)
      const float q0 = top * (1.f / 127.f);
      const __half hs = __float2half_rn(fmaf(fmaf(q0, -127.f, top), 1.f / 127.f, q0));
      const float s = __half2float(hs);
      uint32_t cw[4] = {0, 0, 0, 0};
      if (s > 0.f) codes16(x, s, cw);
      if (kFours) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < n_in) *reinterpret_cast<uint32_t *>(here + k * 4 * lanes) = cw[k];
      } else {
        *reinterpret_cast<uint2 *>(here) = make_uint2(cw[0], cw[1]);
        if (n_in >= 2) *reinterpret_cast<uint2 *>(here + to_second) = make_uint2(cw[2], cw[3]);
      }
      if (l == 0) *to_scale++ = __half_as_ushort(hs);
    }
    cp_wait<0>();                     // (the ring is filled anew)
  }
}

struct GetArgs {
  p4::RowsArgs rows;
  Units units;
};

template <int TYPE>
__global__ void __launch_bounds__(RT, get_ctas(TYPE)) get_rows_kernel(const GetArgs args) {
  const p4::RowsArgs &a = args.rows;
  after_earlier_launches();
  for (Share u = share_of(args.units); u.at < u.end;) {
    const int w = u.at >= args.units.part[0];
    const int64_t unit = w ? u.at - args.units.part[0] : u.at;
    const int d = a.head_dim[w], sh = lane_shift(d), lanes = 1 << sh, l = threadIdx.x & (lanes - 1);
    const int64_t tile = quotient(unit, a.n_heads[w]), row = tile * (RT >> sh) + (threadIdx.x >> sh);
    int head = static_cast<int>(unit - tile * a.n_heads[w]);
    const int heads = static_cast<int>(min(static_cast<int64_t>(a.n_heads[w]), head + (u.end - u.at)));
    u.at += heads - head;
    if (row >= a.n_rows) continue;
    const int64_t slot = __ldg(a.slots + row);
    if (static_cast<uint64_t>(slot) >= static_cast<uint64_t>(a.n_cells)) {
      if (slot != -1 && l == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);
      continue;
    }
    // A lane's codes: two eights, l and l + lanes; of 32-bit rows four fours, so that every access is of whole sectors.
    constexpr int N = TYPE == TQ_F32 ? 4 : 2, E = 16 / N;
    const int n_in = (d - E * l + E * lanes - 1) >> (sh + (N == 4 ? 2 : 3));
    if (E * l >= d) continue;
    int64_t cell_row = slot * a.n_heads[w] + head, to = row * a.stride[w] + static_cast<int64_t>(head) * d + E * l;
    uint32_t next[4] = {0, 0, 0, 0};
    uint16_t s_next = 0;
    auto fetch = [&]() {
      const uint8_t *p = a.codes[w] + cell_row * d + E * l;
      s_next = __ldcs(a.scales[w] + cell_row);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < n_in) {
          if (N == 4) {
            next[k] = __ldcs(reinterpret_cast<const uint32_t *>(p + E * lanes * k));
          } else {
            const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p + E * lanes * k));
            next[2 * k % 4] = v.x;
            next[(2 * k + 1) % 4] = v.y;
          }
        }
    };
    fetch();
    for (; head < heads; ++head, to += d) {
      uint32_t u[4];                                         // code + 128
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = next[i] ^ 0x80808080u;
      const __half hs = __ushort_as_half(s_next);
      ++cell_row;
      if (head + 1 < heads) fetch();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (k >= n_in) break;
        if (TYPE == TQ_F16) {
          // 1024 + 128 + code as binary16, 1152 taken off; the product, rounded once, is that of fp32 rounded once
          uint32_t r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = prmt_b32(u[(2 * k + i / 2) % 4], 0x64646464u, i & 1 ? 0x4342u : 0x4140u);
            const __half2 y = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&v), __float2half2_rn(1152.f)), __half2half2(hs));
            r[i] = *reinterpret_cast<const uint32_t *>(&y);
          }
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dst[w]) + to + E * lanes * k) = make_uint4(r[0], r[1], r[2], r[3]);
        } else {
          const float s = __half2float(hs);
          float2 y[4];
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {                  // a byte in the low bits of 2^23 is the float 2^23 + code + 128
            const uint32_t v = u[N == 4 ? k : (2 * k + i / 2) % 4];
            y[i] = mul2(make_float2(s, s), add2(make_float2(__uint_as_float(prmt_b32(v, 0x4b000000u, i & 1 ? 0x7442u : 0x7440u)),
                                                            __uint_as_float(prmt_b32(v, 0x4b000000u, i & 1 ? 0x7443u : 0x7441u))),
                                                make_float2(-8388736.f, -8388736.f)));
          }
          if (TYPE == TQ_F32) *reinterpret_cast<float4 *>(static_cast<float *>(a.dst[w]) + to + E * lanes * k) = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
          else store8<TYPE>(a.dst[w], to + E * lanes * k, y);
        }
      }
    }
  }
}

// The line of work of up to three tensors, cut for at most `ctas` CTAs; the CTAs that it takes.
unsigned cut(Units &u, const int *n_heads, const int *head_dim, int parts, int64_t n_rows, int ctas) {
  int64_t n = 0;
  for (int i = 0; i < 3; ++i) {
    const int rows = i < parts ? RT >> lane_shift(head_dim[i]) : 1;
    u.part[i] = i < parts ? (n_rows + rows - 1) / rows * n_heads[i] : 0;
    n += u.part[i];
  }
  const int64_t grid = n < ctas ? n : ctas;
  u.per = n / grid;
  u.more = static_cast<int32_t>(n % grid);
  return static_cast<unsigned>(grid);
}

template <int TYPE, int ROT>
cudaError_t launch_step_t(StepArgs &a, cudaStream_t s) {
  int n_heads[3], head_dim[3];
  for (int i = 0; i < 3; ++i) {
    n_heads[i] = a.part[i].n_heads;
    head_dim[i] = a.part[i].head_dim;
  }
  const unsigned grid = cut(a.units, n_heads, head_dim, 3, a.n_rows, ctas_of(ROT) * sm_count());
  return p4::launch_beside(step_rows_kernel<TYPE, ROT>, grid, RT, 0, s, a);
}

template <int TYPE>
cudaError_t launch_step(StepArgs &a, cudaStream_t s) {
  if (!a.positions) return launch_step_t<TYPE, kNone>(a, s);
  if (a.layout == TQ_ROPE_INTERLEAVED) return launch_step_t<TYPE, kInterleaved>(a, s);
  return a.rot % 16 == 0 ? launch_step_t<TYPE, kHalf>(a, s) : launch_step_t<TYPE, kHalfAny>(a, s);
}

}  // namespace

cudaError_t launch_step_rows(int type, const StepArgs &args, cudaStream_t s) {
  StepArgs a = args;
  return type == TQ_F32 ? launch_step<TQ_F32>(a, s) : type == TQ_F16 ? launch_step<TQ_F16>(a, s) : launch_step<TQ_BF16>(a, s);
}

cudaError_t launch_get_rows(int type, const p4::RowsArgs &a, cudaStream_t s) {
  GetArgs g;
  g.rows = a;
  const unsigned grid = cut(g.units, a.n_heads, a.head_dim, 2, a.n_rows, get_ctas(type) * sm_count());
  return type == TQ_F32   ? p4::launch_beside(get_rows_kernel<TQ_F32>, grid, RT, 0, s, g)
         : type == TQ_F16 ? p4::launch_beside(get_rows_kernel<TQ_F16>, grid, RT, 0, s, g)
                          : p4::launch_beside(get_rows_kernel<TQ_BF16>, grid, RT, 0, s, g);
}

}  // namespace i8
}  // namespace tq
