// Prompt attention over the paged 4-bit cache on the tcgen05 tensor cores.
//
//   out[row] = sum_t p_t v_t / sum_t p_t,   p_t = 2^(x_t - R),
//   x_t = scale log2(e) (s_t (q . code_t) + m_t sum(q)),   v_t = s'_t code'_t + m'_t
//
// A CTA takes two tiles A, B of 128 rows -- a row is a (query, head) pair of one
// sequence and KV head -- over key tiles of 128, which both tiles share, so that a
// key tile is unpacked once for 256 rows.  24 warps:
//   0-7, 8-15  softmax of tile A, B: two threads per row (TMEM lane), 64 keys each;
//   16-19      unpack: one key per thread, its packed rows held in registers one
//              tile ahead, written as operand tiles (double buffered);
//   20         issues the products: S = Q K^T and O += P V.
// Tensor memory holds O of both tiles (256 columns), their P as 16-bit pairs (128)
// and ONE score buffer (128) that the tiles use in turn: it is free again as soon as
// the softmax threads have read it into registers, so the next product of scores
// runs beside the rest of the softmax and does not wait for P V.  (With a buffer per
// tile and P written over it, a tile's scores had to wait for its P V: 1200 us at
// 2048 rows over 32768 cells, 8 KV heads, against NEW_FIG.)
// The code of all roles has to stay small: with the products' loops unrolled for one
// thread and a whole row's 128 keys per softmax thread, the product warp waited for
// instructions (1390 us in that form).
//
// Numbers, so that 16-bit operands cost no accuracy beyond the output's own:
// - Scores: K's operand is the code itself (a nibble masked in place reads as the
//   binary16 subnormal code 2^-24 or 2^-20, exact), q is scaled by a power of two
//   per row (exact for 16-bit inputs down to 2^-23 of the row's largest entry).  The
//   offset's term rides along as one more k step: with a_t = m_t / s_t in two
//   binary16 parts and sum(q) in three, the product is s_t-free, so the softmax
//   multiplies a score by one number per key, s_t, in fp32.  (A row with
//   |a_t| >= 2^19 is constant to 3e-5 and takes its offset alone.)
// - Values: v_t 2^-tau rounded to binary16 (relative 2^-12 on average half), tau the
//   largest exponent among 32 neighbouring keys; the weights p_t 2^tau are rounded
//   to binary16 too.  Both roundings meet the values themselves.  R is a running
//   maximum of x_t + tau, raised only when it would grow by more than 2^12 (which binary16 weights leave room
//   for; with 2^8 the rescaling of O cost a tenth of the time).  Sums of
//   weights stay in fp32.
//
// With few row tiles a tile's keys are split over several CTAs; the partial results
// (R, sum, values) of each row are merged by a second kernel, which also forms the
// difference and the norm of differential attention (whose two maps run as separate
// heads here: their products share nothing but V).
#pragma once

#include <math.h>

#include "tq_common.cuh"
#include "tq_paged4.cuh"
#include "tq_paged4_few.cuh"
#include "tq_tc.cuh"

namespace tq {
namespace p4 {
namespace pre {

constexpr int BM = 128, BN = 128;             // rows of a tile, keys of a key tile
constexpr int HK = BN / 2;                    // keys of a softmax thread
constexpr int NT = 768;
constexpr int W_UNPACK = 16, W_MMA = 20;      // first warps of the roles after the softmax
constexpr int REG_SOFTMAX = 88, REG_UNPACK = 96, REG_MMA = 32;    // of 80 at the launch: 4 x 88 + 96 + 32 = 6 x 80

template <int DK, int DV>
struct Cfg {
  static constexpr int KC = DK / 8 + 2;       // 8-element chunks of a Q / K row: dims, then the offset's k step
  static constexpr int VC = DV / 8;
  // operand tiles without swizzle: core matrices of 8 rows x 16 bytes
  static constexpr uint32_t Q_BYTES = KC * 2048;               // [chunk][row / 8]
  static constexpr uint32_t K_BYTES = 16 * KC * 128;           // [key / 8][chunk]
  static constexpr uint32_t V_BYTES = 16 * VC * 128;           // [key / 8][chunk]
  static constexpr uint32_t SQ = 0;
  static constexpr uint32_t SKV = 2 * Q_BYTES;                 // two buffers of (K, V)
  static constexpr uint32_t KV_BYTES = K_BYTES + V_BYTES;
  // (K of a tile may be written as soon as its buffer's scores are done, their softmax still running: four of these)
  static constexpr uint32_t SSC = SKV + 2 * KV_BYTES;          // [j & 3][key] scale of a score
  static constexpr uint32_t STAU = SSC + 4 * BN * 4;           // [j & 3][32 keys] (tau, 2^-tau)
  static constexpr uint32_t SROW = STAU + 4 * 4 * 8;           // [tile][half][row] exchange between a row's threads
  static constexpr uint32_t TOTAL = SROW + 2 * 2 * BM * 8;
  static constexpr int SKS = KC / 2, PKS = BN / 16;            // k steps of S and of PV
};

struct Bars {
  uint64_t k[2], v[2];    // K, V of key tile j (buffer j & 1) written    phase j >> 1
  uint64_t kf[2];         // S_j of every row tile computed: K is free    phase j >> 1
  uint64_t s[2];          // S_j of tile X computed                       phase j
  uint64_t rd[2];         // S_j of tile X read                           phase j
  uint64_t p[2];          // P_j of tile X written                        phase j
  uint64_t pv[2][2];      // PV_j of tile X (buffer j & 1) computed       phase j >> 1
};

// tcgen05.mma with the A operand in tensor memory
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)));
}

__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Bounded wait for phase `parity` of `bar` by a whole warp.  Without a suspend-time hint: with one, a warp that
// found the phase open slept on past its end, on every step of the chain score - softmax - product (WAIT_FIG).
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity) {
  const uint32_t at = tc::smem_u32(bar);
  for (int it = 0; it < (1 << 22); ++it) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(at), "r"(parity)
                 : "memory");
    if (__all_sync(0xffffffffu, ok != 0)) return true;
  }
  return false;
}

// one lane of the warp, the same every time
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }

}  // namespace pre

template <int DK, int DV>
__global__ void __launch_bounds__(pre::NT, 1) prefill_kernel(const AttnArgs a) {
  using namespace pre;
  using C = Cfg<DK, DV>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_fail, s_seq, s_tile, s_sum[NT / 32];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int maps = a.diff ? 2 : 1, k_heads = maps * a.n_kv_heads;
  // heads fastest, row tiles slowest and from the last one down (under a causal mask the longest first)
  const int kh = blockIdx.x % k_heads, rest = blockIdx.x / k_heads;
  const int split = rest % a.n_split, n_split = a.n_split;
  const int want = a.n_tiles - 1 - rest / n_split;
  const int hv = kh / maps, map = kh - hv * maps, G = a.group;

  // ---- the tile's sequence
  if (tid == 0) {
    s_fail = 0;
    s_seq = -1;
  }
  int base = 0;
  for (int s0 = 0; s0 < a.n_seq; s0 += NT) {
    int v = 0;
    if (s0 + tid < a.n_seq) {
      const few::SeqWork w = few::seq_work<1>(a, s0 + tid, blockIdx.x == 0);
      v = static_cast<int>((static_cast<long long>(w.rows) * G + 2 * BM - 1) / (2 * BM));
    }
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w == warp) x += all;
      all += s_sum[w];
    }
    x += base;
    if (v > 0 && x - v <= want && want < x) {
      s_seq = s0 + tid;
      s_tile = want - (x - v);
    }
    base += all;
  }
  __syncthreads();
  if (s_seq < 0) return;                      // fewer tiles than the host's upper bound
  const few::SeqWork sw = few::seq_work<1>(a, s_seq, false);
  const int rows_all = sw.rows * G;           // rows of the sequence for this KV head
  const int r0 = s_tile * 2 * BM;
  const int n_q = rows_all - r0 > BM ? 2 : 1; // row tiles in use
  auto limit_of = [&](int r) { return a.causal ? max(0, sw.len - sw.rows + r / G + 1) : sw.len; };
  const int kv_hi = limit_of(min(rows_all, r0 + 2 * BM) - 1);
  const int tiles_all = (kv_hi + BN - 1) / BN;
  const int t_lo = static_cast<int>(static_cast<long long>(tiles_all) * split / n_split);
  const int n_t = static_cast<int>(static_cast<long long>(tiles_all) * (split + 1) / n_split) - t_lo;

  if (warp == W_MMA) tc::tmem_alloc<512>(&tmem_slot);
  if (tid == NT - 1) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.k[i], 4);
      tc::mbar_init(&bars.v[i], 4);
      tc::mbar_init(&bars.kf[i], n_q);
      tc::mbar_init(&bars.s[i], 1);
      tc::mbar_init(&bars.rd[i], 8);
      tc::mbar_init(&bars.p[i], 8);
      tc::mbar_init(&bars.pv[i][0], 1);
      tc::mbar_init(&bars.pv[i][1], 1);
    }
    tc::mbar_init_fence();
  }

  // ---- Q: the softmax threads bring their rows, half of the dims each
  const int X = warp >> 3, half = (warp >> 2) & 1;                     // X 0, 1: softmax of tile A, B
  const int row = tid & (BM - 1);
  const int r = r0 + X * BM + row;            // row of the sequence
  const bool row_ok = X < n_q && r < rows_all;
  float fx = 1.f;                             // x = fx s_t (score), fx > 0
  {
    constexpr int NC = DK / 16;               // 8-element chunks of a thread
    const bool here = X < n_q;
    const int qi = row_ok ? r / G : 0, head = hv * G + (row_ok ? r - qi * G : 0);
    const uint16_t *src = static_cast<const uint16_t *>(a.q) + (static_cast<int64_t>(sw.row0) + qi) * a.q_stride +
                          static_cast<int64_t>(maps * head + map) * a.dk;
    float2 *ex = reinterpret_cast<float2 *>(smem + C::SROW) + (X & 1) * 2 * BM;     // [half][row]: (max, sum)
    uint4 raw[NC];
    float mx = 0.f, sum = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = 8 * (half * NC + c);
      raw[c] = make_uint4(0, 0, 0, 0);
      if (row_ok && d < a.dk) raw[c] = __ldg(reinterpret_cast<const uint4 *>(src + d));
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v[8];
      few::unpack8(raw[c], a.bf16, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mx = fmaxf(mx, fabsf(v[e]));
        sum += v[e];
      }
    }
    if (here) ex[half * BM + row] = make_float2(mx, sum);
    __syncthreads();
    if (here) {
      const float2 e0 = ex[row], e1 = ex[BM + row];
      mx = fmaxf(e0.x, e1.x);
      sum = e0.y + e1.y;
      // largest entry in [2^e, 2^(e + 1)) -> [2^12, 2^13); the scale's sign goes into q, a scale of 0 makes it 0
      const int e = mx > 0.f ? static_cast<int>(__float_as_uint(mx) >> 23) - 127 : 0;
      const float s1 = __uint_as_float(static_cast<uint32_t>((12 - e) / 2 + 127) << 23);
      const float s2 = __uint_as_float(static_cast<uint32_t>((12 - e) - (12 - e) / 2 + 127) << 23) *
                       (a.scale_log2 > 0.f ? 1.f : a.scale_log2 < 0.f ? -1.f : 0.f);
      if (a.scale_log2 != 0.f) fx = fmaxf(fabsf(a.scale_log2) * exp2f(static_cast<float>(12 + e)), 1e-37f);
      unsigned char *dst = smem + C::SQ + X * C::Q_BYTES + (row >> 3) * 128 + (row & 7) * 16;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float v[8];
        few::unpack8(raw[c], a.bf16, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * s1 * s2 * ((i & 1) ? 0.0625f : 1.f);
        // the order in which a code word unpacks: (0, 4), (1, 5), (2, 6), (3, 7)
        *reinterpret_cast<uint4 *>(dst + (half * NC + c) * 2048) =
            make_uint4(few::half2_bits(v[0], v[4]), few::half2_bits(v[1], v[5]), few::half2_bits(v[2], v[6]),
                       few::half2_bits(v[3], v[7]));
      }
      if (half == 0) {
        const float qs = sum * s1 * s2 * 0x1p-20f;
        const __half h0 = __float2half_rn(qs);
        const __half h1 = __float2half_rn(qs - __half2float(h0));
        const __half h2 = __float2half_rn(qs - __half2float(h0) - __half2float(h1));
        const __half z = __float2half_rn(0.f);
        *reinterpret_cast<uint4 *>(dst + (DK / 8) * 2048) =
            make_uint4(bits(__halves2half2(h0, h1)), bits(__halves2half2(h2, h0)), bits(__halves2half2(h1, z)), 0);
      } else {
        *reinterpret_cast<uint4 *>(dst + (DK / 8 + 1) * 2048) = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if (warp >= W_UNPACK && warp < W_MMA) {
    // the unused half of the offset's k step
    const int key = tid - 32 * W_UNPACK;
#pragma unroll
    for (int b = 0; b < 2; ++b)
      *reinterpret_cast<uint4 *>(smem + C::SKV + b * C::KV_BYTES + (key >> 3) * (C::KC * 128) + (DK / 8 + 1) * 128 +
                                 (key & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
  tc::fence_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const uint32_t sbase = tc::smem_u32(smem);
  constexpr uint32_t TS = 0, TP = 128, TO = 256;        // TMEM columns: S, P of tile X at 128 + 64 X, O at 256 + 128 X

  float R = -INFINITY, l = 0.f;
  if (warp >= W_MMA) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_MMA));
    if (warp == W_MMA) {
      // ===================== products =====================
      // The whole warp goes through the loop, so that descriptors stay in uniform registers; one lane issues.
      constexpr uint32_t ID_S = tc::idesc_f16(BM, BN, false, false);
      constexpr uint32_t ID_PV = tc::idesc_f16(BM, DV, false, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const bool one = elect();
      const uint64_t q0 = tc::sdesc(sbase + C::SQ, 2048, 128);
      const uint64_t k0 = tc::sdesc(sbase + C::SKV, 128, C::KC * 128);
      const uint64_t v0 = tc::sdesc(sbase + C::SKV + C::K_BYTES, C::VC * 128, 128);
      bool ok = true;
      auto product = [&](int x, int j) {      // O += P V of row tile x, key tile j
        if (x == 0) ok = wait_warp(&bars.v[j & 1], (j >> 1) & 1);
        if (ok) ok = wait_warp(&bars.p[x], j & 1);
        if (!ok) return;
        tc::fence_after_sync();
        const uint64_t v = v0 + static_cast<uint64_t>((j & 1) * (C::KV_BYTES >> 4));
        if (one) {
#pragma unroll
          for (int ks = 0; ks < C::PKS; ++ks)
            mma_ta(tm + TO + 128 * x, tm + TP + 64 * x + 8 * ks, v + ((ks * 2 * C::VC * 128) >> 4), ID_PV, j > 0 || ks > 0);
          tc::mma_commit(&bars.pv[x][j & 1]);
        }
        __syncwarp();
      };
      // steps (j, x): scores once the step before has read its own, then the product of this row tile's step
      // before.  (Its P is ready by the time that the scores are read: the same threads do both, in this order.)
      for (int j = 0; j <= n_t && ok && n_t > 0; ++j) {
        const uint64_t k = k0 + static_cast<uint64_t>((j & 1) * (C::KV_BYTES >> 4));
#pragma unroll 1
        for (int x = 0; x < n_q && ok; ++x) {
          if (j < n_t) {
            if (x == 0) ok = wait_warp(&bars.k[j & 1], (j >> 1) & 1);
            const int xl = x == 0 ? n_q - 1 : 0, jl = x == 0 ? j - 1 : j;              // the step before
            if (ok && jl >= 0) ok = wait_warp(&bars.rd[xl], jl & 1);
            if (!ok) break;
            tc::fence_after_sync();
            if (one) {
#pragma unroll
              for (int ks = 0; ks < C::SKS; ++ks)
                tc::mma_f16(tm + TS, q0 + x * (C::Q_BYTES >> 4) + ((ks * 4096) >> 4), k + ((ks * 256) >> 4), ID_S, ks > 0);
              tc::mma_commit(&bars.s[x]);
              tc::mma_commit(&bars.kf[j & 1]);
            }
            __syncwarp();
          }
          if (j > 0) product(x, j - 1);
        }
      }
      if (!ok) s_fail = 1;
    }
  } else if (warp >= W_UNPACK) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_UNPACK));
    // ===================== unpack: one key of the tile per thread =====================
    const int key = tid - 32 * W_UNPACK;
    const int32_t *table = a.block_table + static_cast<int64_t>(s_seq) * a.max_pages;
    const int mask = (1 << a.page_shift) - 1;
    auto page_of = [&](int j) {
      const int t = (t_lo + j) * BN + key;
      return j < n_t && t < kv_hi ? __ldg(table + (t >> a.page_shift)) : -2;       // -2: no such key
    };
    uint4 kraw[DK / 32], vraw[DV / 32];
    uint32_t ksm = 0, vsm = 0;                // (scale, offset) pairs
    // row of the planes of this thread's key in tile j, or -1
    auto row_of = [&](int j, int page) -> int64_t {
      if (page < 0 || page >= a.n_pages) {
        if (page != -2) set_status(a.status, TQ_ERR_DEVICE_CHECK);                 // a zero row
        return -1;
      }
      const int t = (t_lo + j) * BN + key;
      return static_cast<int64_t>(page) * a.n_kv_heads * (mask + 1) + (t & mask);  // of V head 0
    };
    auto load_k = [&](int64_t rw) {
      ksm = 0;
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) kraw[i] = make_uint4(0, 0, 0, 0);
      if (rw >= 0) {
        // (row of K head kh: K planes have `maps` heads per V head)
        const int64_t in = rw & mask, k = (rw - in) * maps + static_cast<int64_t>(kh) * (mask + 1) + in;
        const uint4 *p = reinterpret_cast<const uint4 *>(a.k_codes + k * (DK / 2));
        ksm = __ldg(reinterpret_cast<const uint32_t *>(a.k_scales) + k);
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) kraw[i] = __ldg(p + i);
      }
    };
    auto load_v = [&](int64_t rw) {
      vsm = 0;
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) vraw[i] = make_uint4(0, 0, 0, 0);
      if (rw >= 0) {
        const int64_t v = rw + static_cast<int64_t>(hv) * (mask + 1);
        const uint4 *p = reinterpret_cast<const uint4 *>(a.v_codes + v * (DV / 2));
        vsm = __ldg(reinterpret_cast<const uint32_t *>(a.v_scales) + v);
#pragma unroll
        for (int i = 0; i < DV / 32; ++i) vraw[i] = __ldg(p + i);
      }
    };
    int64_t rw = row_of(0, page_of(0));
    load_k(rw);
    load_v(rw);
    int page = page_of(1);
    bool ok = true;
    for (int j = 0; j < n_t; ++j) {
      const int b = j & 1;
      if (j >= 2) ok = wait_warp(&bars.kf[b], ((j - 2) >> 1) & 1);      // the K buffer's last users
      if (!ok) { s_fail = 1; break; }
      unsigned char *kd = smem + C::SKV + b * C::KV_BYTES + (key >> 3) * (C::KC * 128) + (key & 7) * 16;
      unsigned char *vd = smem + C::SKV + b * C::KV_BYTES + C::K_BYTES + (key >> 3) * (C::VC * 128) + (key & 7) * 16;
      // exponent of the 32 keys' values (with K: the softmax needs it)
      const float2 vsc = __half22float2(as_half2(vsm));
      const float top = fmaxf(fabsf(vsc.y), fabsf(fmaf(15.f, vsc.x, vsc.y)));
      int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      e = min(30, max(-30, __reduce_max_sync(0xffffffffu, e)));
      const float dn = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);            // 2^-tau
      if (lane == 0) 
        reinterpret_cast<float2 *>(smem + C::STAU)[(j & 3) * 4 + (warp - W_UNPACK)] = make_float2(static_cast<float>(e), dn);
      {
        float2 sm = __half22float2(as_half2(ksm));
        float off = __fdividef(sm.y, sm.x);
        uint32_t keep = 0xffffffffu;
        if (!(fabsf(off) < 0x1p19f)) {        // (a scale of 0 too) constant row: its offset alone
          keep = 0;
          off = sm.y > 0.f ? 0x1p16f : sm.y < 0.f ? -0x1p16f : 0.f;
          sm.x = sm.y != 0.f ? fabsf(sm.y) * 0x1p-16f : 1.f;
        }
        const __half hi = __float2half_rn(off * 0.0625f);
        const __half lo = __float2half_rn(off * 0.0625f - __half2float(hi));
        *reinterpret_cast<uint4 *>(kd + (DK / 8) * 128) =
            make_uint4(bits(__halves2half2(hi, hi)), bits(__halves2half2(hi, lo)),
                       bits(__halves2half2(lo, __float2half_rn(0.f))), 0);
        reinterpret_cast<float *>(smem + C::SSC)[(j & 3) * BN + key] = sm.x;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
          const uint32_t w[4] = {kraw[i].x & keep, kraw[i].y & keep, kraw[i].z & keep, kraw[i].w & keep};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t u = w[c] >> 8;
            *reinterpret_cast<uint4 *>(kd + (4 * i + c) * 128) =
                make_uint4(w[c] & 0x000f000fu, w[c] & 0x00f000f0u, u & 0x000f000fu, u & 0x00f000f0u);
          }
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.k[b]);
      rw = row_of(j + 1, page);
      load_k(rw);                             // on its way while the values are unpacked
      if (j >= 2)                             // the V buffer's last users
        for (int x = 0; x < n_q && ok; ++x) ok = wait_warp(&bars.pv[x][b], ((j - 2) >> 1) & 1);
      if (!ok) { s_fail = 1; break; }
      {
        const __half2 vs = __float2half2_rn(vsc.x * dn), vm = __float2half2_rn(vsc.y * dn);
        const __half2 k1024 = as_half2(0x64006400u), k16 = as_half2(0x2c002c00u), k64 = as_half2(0xd400d400u);
#pragma unroll
        for (int i = 0; i < DV / 32; ++i) {
          const uint32_t w[4] = {vraw[i].x, vraw[i].y, vraw[i].z, vraw[i].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t u = w[c] >> 8;
            // 1024 + code, and 1024 + 16 code
            const __half2 c0 = __hsub2(as_half2((w[c] & 0x000f000fu) | 0x64006400u), k1024);
            const __half2 c1 = __hfma2(as_half2((w[c] & 0x00f000f0u) | 0x64006400u), k16, k64);
            const __half2 c2 = __hsub2(as_half2((u & 0x000f000fu) | 0x64006400u), k1024);
            const __half2 c3 = __hfma2(as_half2((u & 0x00f000f0u) | 0x64006400u), k16, k64);
            *reinterpret_cast<uint4 *>(vd + (4 * i + c) * 128) =
                make_uint4(bits(__hfma2(c0, vs, vm)), bits(__hfma2(c1, vs, vm)), bits(__hfma2(c2, vs, vm)),
                           bits(__hfma2(c3, vs, vm)));
          }
        }
      }
      load_v(rw);
      page = page_of(j + 2);
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.v[b]);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFTMAX));
    // ===================== softmax: 64 keys of a row per thread =====================
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lane_off + TS + HK * half, tp = tmem + lane_off + TP + 64 * X + (HK / 2) * half;
    const uint32_t to = tmem + lane_off + TO + 128 * X;
    const int pair = 1 + 4 * X + (warp & 3);                            // named barrier of the rows' two warps
    float *ex = reinterpret_cast<float *>(smem + C::SROW) + X * 4 * BM; // [j & 1][half][row]
    const int lim = row_ok ? limit_of(r) : 0;
    const float2 fx2 = make_float2(fx, fx);
    bool ok = true;
    for (int j = 0; j < (X < n_q ? n_t : 0); ++j) {
      const int b = j & 1;
      if (ok) {
        ok = wait_warp(&bars.s[X], j & 1);
        if (ok) ok = wait_warp(&bars.k[b], (j >> 1) & 1);               // the tile's scales
      }
      if (!ok) {                              // a wait ran out: the row's other warp still meets this one
        tc::named_sync(pair, 64);
        continue;
      }
      tc::fence_after_sync();
      float y[HK];
      {
        uint32_t *u = reinterpret_cast<uint32_t *>(y);
        tc::tmem_ld32(ts, u);
        tc::tmem_ld32(ts + 32, u + 32);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.rd[X]);
      }
      const float4 *sc = reinterpret_cast<const float4 *>(smem + C::SSC + ((j & 3) * BN + HK * half) * 4);
#pragma unroll
      for (int i = 0; i < HK / 4; ++i) {
        const float4 s4 = sc[i];
        const float2 u = mul2(make_float2(y[4 * i], y[4 * i + 1]), make_float2(s4.x, s4.y));
        const float2 w = mul2(make_float2(y[4 * i + 2], y[4 * i + 3]), make_float2(s4.z, s4.w));
        y[4 * i] = u.x;
        y[4 * i + 1] = u.y;
        y[4 * i + 2] = w.x;
        y[4 * i + 3] = w.y;
      }
      const int nvis = lim - (t_lo + j) * BN - HK * half;               // of the thread's keys, those that the row sees
      if (__any_sync(0xffffffffu, nvis < HK)) {
#pragma unroll
        for (int i = 0; i < HK; ++i)
          if (i >= nvis) y[i] = -INFINITY;
      }
      const float2 *tau = reinterpret_cast<const float2 *>(smem + C::STAU) + 4 * (j & 3) + 2 * half;
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          m0 = max3(m0, y[32 * c + i], y[32 * c + i + 1]);
          m1 = max3(m1, y[32 * c + i + 2], y[32 * c + i + 3]);
        }
        top = fmaxf(top, fmaf(fmaxf(m0, m1), fx, tau[c].x));
      }
      // (two places in turn: the other thread may still be reading the last tile's)
      ex[(2 * (j & 1) + half) * BM + row] = top;
      tc::named_sync(pair, 64);
      top = fmaxf(top, ex[(2 * (j & 1) + (half ^ 1)) * BM + row]);
      if (j > 0) {                            // P and O stand still
        ok = wait_warp(&bars.pv[X][(j - 1) & 1], ((j - 1) >> 1) & 1);
        if (!ok) continue;
        tc::fence_after_sync();
      }
      const bool raise = top > R + RAISE;
      if (__any_sync(0xffffffffu, raise)) {
        const float f = raise ? exp2f(R - top) : 1.f;                   // 0 at the first raise
        if (raise) R = top;
        l *= f;
        if (j > 0) {
#pragma unroll 1
          for (int c = half * (DV / 2); c < (half + 1) * (DV / 2); c += 8) {
            uint32_t o[8];
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7])
                         : "r"(to + c));
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            st8(to + c, o);
          }
        }
      }
      const float Rs = R == -INFINITY ? 0.f : R;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float2 t2 = tau[c];
        const float2 off = make_float2(t2.x - Rs, t2.x - Rs);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = 32 * c + 16 * h + 2 * i;
            const float2 e = fma2(make_float2(y[k], y[k + 1]), fx2, off);
            const float2 w = make_float2(tc::ex2(e.x), tc::ex2(e.y));   // masked: 0
            sum = add2(sum, w);
            p[i] = few::half2_bits(w.x, w.y);
          }
          st8(tp + 16 * c + 8 * h, p);
        }
        l = fmaf(sum.x + sum.y, t2.y, l);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars.p[X]);
    }
    // the last product has to be done before O is read
    if (ok && X < n_q && n_t > 0) {
      ok = wait_warp(&bars.pv[X][(n_t - 1) & 1], ((n_t - 1) >> 1) & 1);
      tc::fence_after_sync();
    }
    if (!ok) s_fail = 1;
    // ===================== epilogue: columns in the order of the code words, half of them per thread =====================
    if (X < n_q) {
      tc::named_sync(pair, 64);                                         // the last exchange was read
      ex[half * BM + row] = l;
      tc::named_sync(pair, 64);
      l += ex[(half ^ 1) * BM + row];
    }
    if (ok && X < n_q) {
      const int qi = row_ok ? r / G : 0, head = hv * G + (row_ok ? r - qi * G : 0);
      const int64_t out_row = static_cast<int64_t>(sw.row0) + qi;
      const bool partial = n_split > 1 || a.diff;
      const float inv = l != 0.f ? 1.f / l : 0.f;                       // nothing visible: zeros (NaN stays NaN)
      float *part = a.part + (((out_row * a.n_heads + head) * maps + map) * n_split + split) * (DV + 4);
      if (partial && row_ok && half == 0) *reinterpret_cast<float4 *>(part) = make_float4(R, l, 0.f, 0.f);
#pragma unroll 1
      for (int c = half * (DV / 2); c < (half + 1) * (DV / 2); c += 32) {
        uint32_t o[32];
        if (n_t > 0) {
          tc::tmem_ld32(to + c, o);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float v[8];                                                    // dims c + 8 g ..
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = __uint_as_float(o[8 * g + 2 * e]);
            v[e + 4] = __uint_as_float(o[8 * g + 2 * e + 1]);
          }
          const int d = c + 8 * g;
          if (!row_ok || d >= a.dv) continue;
          if (partial) {
            *reinterpret_cast<float4 *>(part + 4 + d) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(part + 8 + d) = make_float4(v[4], v[5], v[6], v[7]);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (a.bf16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e] * inv, v[2 * e + 1] * inv);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
              } else {
                w[e] = few::half2_bits(v[2 * e] * inv, v[2 * e + 1] * inv);
              }
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (out_row * a.n_heads + head) * a.dv + d) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (s_fail && tid == 0) set_status(a.status, TQ_ERR_TIMEOUT);
  if (warp == W_MMA) tc::tmem_dealloc<512>(tmem);
}

// One warp per (row, output head): the key splits of each map together, then the difference and the norm.
template <int DV>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t row = id / a.n_heads;
  const int head = static_cast<int>(id - row * a.n_heads);
  if (row >= a.n_rows) return;
  // the row's sequence; rows of none stay as they are
  int lo = 0, hi = a.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.q_start[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  const few::SeqWork sw = few::seq_work<1>(a, lo, false);
  if (row < sw.row0 || row >= sw.row0 + sw.rows) return;
  const int maps = a.diff ? 2 : 1;
  constexpr int N = DV / 32;                  // values per lane: dims N lane ..
  float y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = 0.f;
  for (int m = 0; m < maps; ++m) {
    const float *part = a.part + ((row * a.n_heads + head) * maps + m) * static_cast<int64_t>(a.n_split) * (DV + 4);
    float M = -INFINITY;
    for (int s = 0; s < a.n_split; ++s) M = fmaxf(M, __ldg(part + static_cast<int64_t>(s) * (DV + 4)));
    float l = 0.f, o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.n_split; ++s) {
      const float *p = part + static_cast<int64_t>(s) * (DV + 4);
      const float2 rl = __ldg(reinterpret_cast<const float2 *>(p));
      const float w = rl.x == -INFINITY ? 0.f : exp2f(rl.x - M);
      l = fmaf(w, rl.y, l);
      if (N * lane < a.dv) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float2 v = __ldg(reinterpret_cast<const float2 *>(p + 4 + N * lane + i));
          o[i] = fmaf(w, v.x, o[i]);
          o[i + 1] = fmaf(w, v.y, o[i + 1]);
        }
      }
    }
    const float f = (l != 0.f ? 1.f / l : 0.f) * (m == 0 ? 1.f : -a.lam[head]);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = fmaf(f, o[i], y[i]);
  }
  if (a.diff) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(y[i], y[i], ss);
    ss = warp_sum(ss);
    const float r = a.norm_weight ? rsqrtf(ss / static_cast<float>(a.dv) + a.eps) * a.out_scale : a.out_scale;
#pragma unroll
    for (int i = 0; i < N; ++i)
      y[i] *= r * (a.norm_weight && N * lane + i < a.dv ? a.norm_weight[N * lane + i] : 1.f);
  }
  if (N * lane < a.dv)
#pragma unroll
    for (int i = 0; i < N; i += 2)
      few::store2(a.out, (row * a.n_heads + head) * a.dv + N * lane + i, y[i], y[i + 1], a.bf16);
}

template <int DK, int DV>
cudaError_t launch_prefill_t(const AttnArgs &a, cudaStream_t s) {
  using C = pre::Cfg<DK, DV>;
  static_assert(C::TOTAL <= 227 * 1024, "shared memory");
  static_assert(4 * pre::REG_SOFTMAX + pre::REG_UNPACK + pre::REG_MMA <= 6 * 80, "registers");
  auto kern = prefill_kernel<DK, DV>;
  cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kern), C::TOTAL);
  if (e != cudaSuccess) return e;
  const int k_heads = (a.diff ? 2 : 1) * a.n_kv_heads;
  kern<<<static_cast<unsigned>(a.n_tiles) * a.n_split * k_heads, pre::NT, C::TOTAL, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || (a.n_split == 1 && !a.diff)) return e;
  prefill_merge_kernel<DV><<<static_cast<unsigned>((a.n_rows * a.n_heads + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace p4
}  // namespace tq
