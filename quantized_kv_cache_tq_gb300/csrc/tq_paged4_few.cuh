// Attention of a few query columns over the paged 4-bit cache (decode steps,
// short verify batches, and any head dim the prompt kernel does not take).
//
//   out[c] = sum_t p_t (s_t code_t + m_t) / sum_t p_t,   p_t = 2^(x_t - R),
//   x_t = scale log2(e) (s^K_t (q . code^K_t) + m^K_t sum(q))
//
// Columns are (query row, head) pairs of one sequence and V head, eight per
// tensor-core tile.  With so few columns the work is reading the cache once, so
// everything is arranged around the loads:
//
// - A warp streams its own 32-key tiles through a private ring of cp.async
//   stages.  Every lane copies exactly the code words that it will feed to the
//   tensor core as a fragment (lane (g, t) of mma.m16n8k16 needs key g for the
//   scores and dims 16 g .. for the values), so a lane waits for its own copies
//   only, shared memory is read without bank conflicts, and no barrier stands in
//   the loop.
// - Codes become operands with one AND: (w & 0x000f000f) read as two binary16
//   values is the subnormal pair code 2^-24, (w & 0x00f000f0) is code 2^-20; the
//   powers of two are exact and go into q (2^-4 on the second kind) and into the
//   output (2^24, 2^20).  Eight codes cost four ANDs and one shift; the values
//   take two byte permutes more per 16 codes to pair up neighbouring keys.
// - q is scaled by a power of two per column, so that its binary16 form is exact
//   for binary16 and bfloat16 inputs down to 2^-23 of the column's largest entry
//   (smaller ones lose low bits below that).  Scores are thus exact up to fp32
//   accumulation.
// - The value weights p_t s_t are rounded to binary16 (relative 2^-11, an eighth
//   of bfloat16's rounding of the output): R is a running maximum of
//   x_t + exponent(s_t), so the largest weight lies in [1, 2^9] whatever the
//   scales, and sums of p_t and p_t m_t stay in fp32.  R is raised only when it
//   would grow by more than 2^8 (the sums are rescaled then).
// - Codes count from a row's smallest value, so with w the rounded weight, sum w c
//   + sum p m would carry the rounding of w times the whole range of the row.  The
//   sum taken is sum w (c - c0) + sum p (m + s c0) with c0 = clamp(-m / s, 0, 15)
//   per row, the code that stands for 0: the rounding then meets the values
//   themselves (binary16 output error over 32768 keys: 7.2e-4 without, 2.2e-4 with;
//   the plain fp32 form has 2.1e-4, the output's own rounding).
//
// Split of the work: the keys of all (sequence, V head, column chunk) items, in
// units of 64, form one line that is cut into equal shares, one per CTA.  Shares
// do not depend on how ragged the batch is, nothing about lengths is needed on
// the host (a captured graph follows the device's lengths), and a CTA's first
// and last item are the only ones that other CTAs share.  Of those the partial
// (R, sums, values) goes to the workspace and the last CTA to arrive merges.
#pragma once

#include <math.h>

#include "tq_common.cuh"
#include "tq_paged4.cuh"
#include "tq_tc.cuh"

namespace tq {
namespace p4 {

constexpr int UNIT = 64;              // keys per unit of work
constexpr int TILE = 32;              // keys per warp tile
constexpr int MIN_SHARE = 4;          // units per CTA at least: one tile for each of eight warps

// MAPS = 2: differential attention; tile n of the columns belongs to map n and
// reads K head 2 hv + n.  MAPS = 1: NT tiles of eight columns read K head hv.
template <int DK, int DV, int NT, int MAPS>
struct FewCfg {
  static constexpr int NW = 8;                            // warps
  static constexpr int THREADS = NW * 32;
  static constexpr int KW = DK / 32;                      // words of a K row per lane
  static constexpr int VW = DV / 64;                      // words of a V row per lane
  static constexpr int KS = DK / 16;                      // k steps of the scores
  static constexpr int MT = DV / 16;                      // m tiles of the values
  static constexpr int COLS = 8 * (MAPS == 2 ? 1 : NT);   // (row, head) columns per item
  static constexpr int NC = 8 * NT;                       // columns incl. maps
  // per SM: two where value accumulators and query fragments leave room in 128 registers a thread
  static constexpr int CTAS = NT * (4 * MT + 2 * KS) <= 80 ? 2 : 1;
  // one stage: K words [map][key row 4][lane], V words [key 8][lane], scales [map + 1][32]
  static constexpr int K_BYTES = TILE * DK / 2;
  static constexpr int V_BYTES = TILE * DV / 2;
  static constexpr int STAGE = MAPS * K_BYTES + V_BYTES + (MAPS + 1) * TILE * 4;
  static constexpr int MERGE = NW * NT * MT * 512 + NW * NC * 12 + NC * 16;  // CTA merge, in the same place
  static constexpr int BUDGET = (CTAS == 2 ? 108 : 216) * 1024;
  static constexpr int FIT = BUDGET / (NW * STAGE);
  static constexpr int STAGES = FIT < 2 ? 2 : (FIT > 4 ? 4 : FIT);
  static constexpr int SMEM = NW * STAGES * STAGE > MERGE ? NW * STAGES * STAGE : MERGE;
  // a partial result: (R, l, z) of every column, then the value fragments
  static constexpr int PART = 4 * NC + NT * MT * 128;
};

namespace few {

__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// W words (1, 2, 4) of one lane; n = 0 writes zeros
template <int W>
__device__ __forceinline__ void cpw(uint32_t dst, const void *src, bool there) {
  if (W == 1) cp4(dst, src, there ? 4 : 0);
  else if (W == 2) cp8(dst, src, there ? 8 : 0);
  else cp16(dst, src, there ? 16 : 0);
}
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <int W>
__device__ __forceinline__ void lds(uint32_t *r, uint32_t at) {
  if (W == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(at));
  else if (W == 2) asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
  else
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}

// 8 consecutive query elements (16-byte aligned) as floats; zeros where there are none
__device__ __forceinline__ void load8(const void *q, int64_t i, bool there, int bf16, float *x) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (there) u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(q) + i));
  const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = bf16 ? make_float2(__uint_as_float(r[k] << 16), __uint_as_float(r[k] & 0xffff0000u))
                          : __half22float2(*reinterpret_cast<const __half2 *>(&r[k]));
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}

__device__ __forceinline__ void store2(void *out, int64_t i, float a, float b, int bf16) {
  uint32_t r;
  if (bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    r = *reinterpret_cast<const uint32_t *>(&h);
  } else {
    r = half2_bits(a, b);
  }
  *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(out) + i) = r;
}

// A sequence as the work line sees it.
struct SeqWork {
  int len;            // cells attended
  int row0, rows;     // its query rows
  int chunks;         // column chunks per V head
  long long units;    // per item
  long long items;
};

template <int COLS>
__device__ __forceinline__ SeqWork seq_work(const AttnArgs &a, int s, bool report) {
  SeqWork w;
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  int len = a.seq_len[s];
  if (len < 0 || len > cap) {                   // longer than its block table: what the table holds
    if (report) set_status(a.status, TQ_ERR_DEVICE_CHECK);
    len = len < 0 ? 0 : static_cast<int>(cap);
  }
  w.len = len;
  w.row0 = s;
  w.rows = 1;
  if (a.q_start) {
    int r0 = a.q_start[s], r1 = a.q_start[s + 1];
    if (r0 < 0 || r1 < r0 || r1 > a.n_rows) {   // rows outside q: none
      if (report) set_status(a.status, TQ_ERR_DEVICE_CHECK);
      r0 = r1 = 0;
    }
    w.row0 = r0;
    w.rows = r1 - r0;
  }
  w.chunks = static_cast<int>((static_cast<long long>(w.rows) * a.group + COLS - 1) / COLS);
  w.units = (len + UNIT - 1) / UNIT;
  w.items = static_cast<long long>(w.chunks) * a.n_kv_heads;
  return w;
}

// Units of the sequences s0 .. s0 + threads - 1: this thread's sequence spans [lo, hi) of the
// line that stands at `base` before them; returns their sum (to every thread).
template <int COLS, int NW>
__device__ __forceinline__ long long scan_chunk(const AttnArgs &a, int s0, long long base, long long *sums, bool report,
                                                long long &lo, long long &hi) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long v = 0;
  if (s0 + tid < a.n_seq) {
    const SeqWork w = seq_work<COLS>(a, s0 + tid, report);
    v = w.units * w.items;
  }
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w == warp) x += all;
    all += sums[w];
  }
  lo = base + x - v;
  hi = base + x;
  return all;
}

}  // namespace few

template <int DK, int DV, int NT, int MAPS>
__global__ void __launch_bounds__(FewCfg<DK, DV, NT, MAPS>::THREADS, FewCfg<DK, DV, NT, MAPS>::CTAS)
    few_kernel(const AttnArgs a) {
  using C = FewCfg<DK, DV, NT, MAPS>;
  using namespace few;
  constexpr int NW = C::NW, KW = C::KW, VW = C::VW, MT = C::MT, NC = C::NC, COLS = C::COLS;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[NW];
  __shared__ long long s_pre;
  __shared__ int s_seq, s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

  // ---- this CTA's share of the work line: units [cur, end) of `total`
  long long total = 0, pre = 0, mine_lo = 0, mine_hi = 0;
  for (int s0 = 0; s0 < a.n_seq; s0 += C::THREADS)
    total += scan_chunk<COLS, NW>(a, s0, total, s_scan, blockIdx.x == 0, mine_lo, mine_hi);
  const long long n_work = min(static_cast<long long>(gridDim.x), (total + MIN_SHARE - 1) / MIN_SHARE);
  const bool works = blockIdx.x < n_work;
  long long cur = 0, end = 0;
  int seq = 0;
  if (works) {
    cur = blockIdx.x * total / n_work;
    end = (blockIdx.x + 1) * total / n_work;
    long long at = 0;
    for (int s0 = 0; s0 < a.n_seq; s0 += C::THREADS) {
      // (a batch of one chunk still has its sums in registers)
      if (a.n_seq > C::THREADS) at += scan_chunk<COLS, NW>(a, s0, at, s_scan, false, mine_lo, mine_hi);
      if (mine_lo <= cur && cur < mine_hi) {
        s_seq = s0 + tid;
        s_pre = mine_lo;
      }
    }
    __syncthreads();
    seq = s_seq;
    pre = s_pre;
  }
  const long long share0 = cur;

  while (cur < end) {
    // ---- one segment: units u0 .. u1 - 1 of an item
    SeqWork w = seq_work<COLS>(a, seq, false);
    if (cur - pre >= w.units * w.items) {
      pre += w.units * w.items;
      ++seq;
      continue;
    }
    const long long item = (cur - pre) / w.units;
    const int u0 = static_cast<int>((cur - pre) - item * w.units);
    const int u1 = static_cast<int>(min(static_cast<long long>(w.units), u0 + (end - cur)));
    const int hv = static_cast<int>(item / w.chunks), chunk = static_cast<int>(item - static_cast<long long>(hv) * w.chunks);
    const int cols_all = w.rows * a.group;
    const int c_base = chunk * COLS;
    // position of a column's row among the keys: it sees keys < its limit
    const int last_row = min(cols_all - 1, c_base + COLS - 1) / a.group;
    auto limit_of = [&](int row) { return a.causal ? max(0, w.len - w.rows + row + 1) : w.len; };
    const int k_begin = u0 * UNIT;
    const int k_end = min(limit_of(last_row), u1 * UNIT);
    const int n_tiles = k_end > k_begin ? (k_end - k_begin + TILE - 1) / TILE : 0;
    const int32_t *table = a.block_table + static_cast<int64_t>(seq) * a.max_pages;

    // ---- the warp's tile copies
    const uint32_t ring = tc::smem_u32(smem) + warp * C::STAGES * C::STAGE;
    auto page_at = [&](int key) { return key < k_end ? __ldg(table + (key >> a.page_shift)) : -1; };
    auto issue = [&](int tile, int p0, int p1) {
      const int slot = (tile / NW) % C::STAGES;
      const uint32_t st = ring + slot * C::STAGE;
      const int key0 = k_begin + tile * TILE;
      const int mask = (1 << a.page_shift) - 1;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int page = hf ? p1 : p0;
        const bool okp = page >= 0 && page < a.n_pages;
        const int kb = key0 + 16 * hf;
        if (!okp && kb < k_end && lane == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);   // zero rows
        const int64_t pg = okp ? page : 0;
#pragma unroll
        for (int m = 0; m < MAPS; ++m) {
          const int64_t r0 = (pg * (MAPS * a.n_kv_heads) + MAPS * hv + m) << a.page_shift;
          const uint8_t *base = a.k_codes + (r0 + (kb & mask)) * (DK / 2);
          const uint32_t kst = st + m * C::K_BYTES;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const bool there = okp && kb + g + 8 * r < k_end;
#pragma unroll
            for (int c = 0; c < (KW + 3) / 4; ++c) {
              constexpr int W = KW < 4 ? KW : 4;
              cpw<W>(kst + (((2 * hf + r) * ((KW + 3) / 4) + c) * 32 + lane) * (4 * W),
                     base + (there ? (g + 8 * r) * (DK / 2) + c * 64 + 4 * W * t : 0), there);
            }
          }
          if ((lane >> 4) == hf) {
            const bool there = okp && kb + (lane & 15) < k_end;
            cp4(st + MAPS * C::K_BYTES + C::V_BYTES + (m * 32 + lane) * 4,
                a.k_scales + 2 * (there ? r0 + (kb & mask) + (lane & 15) : 0), there ? 4 : 0);
          }
        }
        const int64_t r0 = (pg * a.n_kv_heads + hv) << a.page_shift;
        const uint8_t *base = a.v_codes + (r0 + (kb & mask)) * (DV / 2);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int kk = 2 * t + (r & 1) + 8 * (r >> 1);
          const bool there = okp && kb + kk < k_end;
          cpw<VW>(st + MAPS * C::K_BYTES + ((4 * hf + r) * 32 + lane) * (4 * VW),
                  base + (there ? kk * (DV / 2) + 4 * VW * g : 0), there);
        }
        if ((lane >> 4) == hf) {
          const bool there = okp && kb + (lane & 15) < k_end;
          cp4(st + MAPS * C::K_BYTES + C::V_BYTES + (MAPS * 32 + lane) * 4,
              a.v_scales + 2 * (there ? r0 + (kb & mask) + (lane & 15) : 0), there ? 4 : 0);
        }
      }
    };
    auto pages_of = [&](int tile, int &p0, int &p1) {
      p0 = p1 = -1;
      if (tile < n_tiles) {
        const int key0 = k_begin + tile * TILE;
        p0 = page_at(key0);
        p1 = page_at(key0 + 16);
      }
    };
    int pg0[C::STAGES], pg1[C::STAGES];
#pragma unroll
    for (int i = 0; i < C::STAGES; ++i) pages_of(warp + i * NW, pg0[i], pg1[i]);
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
      if (warp + i * NW < n_tiles) issue(warp + i * NW, pg0[i], pg1[i]);
      tc::cp_async_commit();
    }
    int pn0 = pg0[C::STAGES - 1], pn1 = pg1[C::STAGES - 1];

    // ---- query fragments: column g of tile n, the dims of this lane's K words
    uint32_t qf[NT][C::KS][2];
    float qx[NT][2], fx[NT][2];     // of columns 2t, 2t + 1: scale * log2(e) * sum(q), and the score factor
    int lim[NT][2];                 // their limits
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = c_base + (MAPS == 2 ? 0 : 8 * n) + g;
      const bool okc = c < cols_all;
      const int row = okc ? c / a.group : 0, head = hv * a.group + (okc ? c - row * a.group : 0);
      const int64_t qb = (w.row0 + row) * a.q_stride + static_cast<int64_t>(MAPS == 2 ? 2 * head + n : head) * a.dk;
      float v[KW][8], mx = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const int d0 = (i / 4) * 128 + (KW < 4 ? KW : 4) * 8 * t + 8 * (i % 4);
        load8(a.q, qb + d0, okc && d0 < a.dk, a.bf16, v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          mx = fmaxf(mx, fabsf(v[i][e]));
          sum += v[i][e];
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      // max in [2^ex, 2^(ex+1)) -> scaled to [2^12, 2^13)
      const int ex = mx > 0.f ? static_cast<int>(__float_as_uint(mx) >> 23) - 127 : 0;
      // the factor 2^(12 - ex) as two, so that each is a normal number
      const float s1 = __uint_as_float(static_cast<uint32_t>((12 - ex) / 2 + 127) << 23);
      const float s2 = __uint_as_float(static_cast<uint32_t>((12 - ex) - (12 - ex) / 2 + 127) << 23);
#pragma unroll
      for (int i = 0; i < KW; ++i)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          qf[n][2 * i + hf][0] = half2_bits(v[i][2 * hf] * s1 * s2, v[i][2 * hf + 4] * s1 * s2);
          qf[n][2 * i + hf][1] =
              half2_bits(v[i][2 * hf + 1] * s1 * s2 * 0.0625f, v[i][2 * hf + 5] * s1 * s2 * 0.0625f);
        }
      // this lane's softmax columns are 2t and 2t + 1: their values sit in lanes g = 2t, 2t + 1
      const float f = a.scale_log2 * exp2f(12.f + static_cast<float>(ex));          // 2^24 2^(ex - 12)
      const float qs = a.scale_log2 * sum;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fx[n][i] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + i));
        qx[n][i] = __shfl_sync(0xffffffffu, qs, 4 * (2 * t + i));
        const int cc = c_base + (MAPS == 2 ? 0 : 8 * n) + 2 * t + i;
        lim[n][i] = cc < cols_all ? limit_of(cc / a.group) : 0;
      }
    }
    const int lim_min = limit_of(c_base / a.group);       // every column of the chunk sees the keys below

    float acc[NT][MT][4];
    float R[NT][2], Rs[NT][2], l[NT][2], z[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[n][i][c] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        R[n][i] = -INFINITY;
        Rs[n][i] = 0.f;
        l[n][i] = 0.f;
        z[n][i] = 0.f;
      }
    }

    for (int tile = warp; tile < n_tiles; tile += NW) {
      cp_wait<C::STAGES - 2>();
      __syncwarp();               // everybody's copies of this tile are there, and the slot refilled next was read
      {
        const int nt = tile + (C::STAGES - 1) * NW;
        if (nt < n_tiles) issue(nt, pn0, pn1);
        tc::cp_async_commit();
        pages_of(nt + NW, pn0, pn1);
      }
      const uint32_t st = ring + ((tile / NW) % C::STAGES) * C::STAGE;
      const uint32_t sc = st + MAPS * C::K_BYTES + C::V_BYTES;
      const int key0 = k_begin + tile * TILE;
      const bool masked = key0 + TILE > lim_min || key0 + TILE > k_end;

      // value scales and offsets of the lane's score rows (keys g + 8 j), exponents of the scales
      float vs[4], vm[4], ve[4], vc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t u;
        lds<1>(&u, sc + (MAPS * 32 + 8 * j + g) * 4);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
        const float c0 = fminf(fmaxf(__fdividef(-f.y, f.x), 0.f), 15.f);     // (0 / 0 and NaN: 0)
        vs[j] = f.x;
        vc[j] = -c0;
        vm[j] = fmaf(f.x, c0, f.y);
        ve[j] = f.x > 0.f ? static_cast<float>(static_cast<int>(__float_as_uint(f.x) >> 23) - 127) : -24.f;
      }
      uint32_t pb[NT][2][2];                // weights as B fragments [half][keys 0-7, 8-15]
#pragma unroll
      for (int m = 0; m < MAPS; ++m) {
        constexpr int N1 = MAPS == 2 ? 1 : NT;
        float s[N1][2][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t kw[2][KW];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < (KW + 3) / 4; ++c) {
              constexpr int W = KW < 4 ? KW : 4;
              lds<W>(&kw[r][4 * c], st + m * C::K_BYTES + (((2 * hf + r) * ((KW + 3) / 4) + c) * 32 + lane) * (4 * W));
            }
#pragma unroll
          for (int n = 0; n < N1; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[n][hf][c] = 0.f;
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            const uint32_t a0 = kw[0][i], a1 = kw[1][i], b0 = a0 >> 8, b1 = a1 >> 8;
#pragma unroll
            for (int n = 0; n < N1; ++n) {
              const int nn = MAPS == 2 ? m : n;
              mma16816(s[n][hf], a0 & 0x000f000fu, a1 & 0x000f000fu, a0 & 0x00f000f0u, a1 & 0x00f000f0u,
                       qf[nn][2 * i][0], qf[nn][2 * i][1]);
              mma16816(s[n][hf], b0 & 0x000f000fu, b1 & 0x000f000fu, b0 & 0x00f000f0u, b1 & 0x00f000f0u,
                       qf[nn][2 * i + 1][0], qf[nn][2 * i + 1][1]);
            }
          }
        }
        float ks[4], km[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t u;
          lds<1>(&u, sc + (m * 32 + 8 * j + g) * 4);
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
          ks[j] = f.x;
          km[j] = f.y;
        }
#pragma unroll
        for (int n = 0; n < N1; ++n) {
          const int nn = MAPS == 2 ? m : n;
          float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int j = 2 * hf + (c >> 1), i = c & 1;
              float x = fmaf(ks[j] * s[n][hf][c], fx[nn][i], km[j] * qx[nn][i]);
              if (masked && key0 + 8 * j + g >= min(lim[nn][i], k_end)) x = -INFINITY;
              s[n][hf][c] = x;
              mt[i] = fmaxf(mt[i], x + ve[j]);
            }
          const bool raise = mt[0] > R[nn][0] + 8.f || mt[1] > R[nn][1] + 8.f;
          if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = mt[i];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              if (x > R[nn][i] + 8.f) {
                const float f = exp2f(R[nn][i] - x);      // 0 at the first raise
                R[nn][i] = Rs[nn][i] = x;
                l[nn][i] *= f;
                z[nn][i] *= f;
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                  acc[nn][k][i] *= f;
                  acc[nn][k][i + 2] *= f;
                }
              }
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float wt[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int j = 2 * hf + (c >> 1), i = c & 1;
              const float p = tc::ex2(s[n][hf][c] - Rs[nn][i]);
              l[nn][i] += p;
              z[nn][i] = fmaf(p, vm[j], z[nn][i]);
              wt[c] = p * vs[j];
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const __half2 h = __floats2half2_rn(wt[2 * r], wt[2 * r + 1]);
              const float2 f = __half22float2(h);
              z[nn][0] = fmaf(f.x, vc[2 * hf + r], z[nn][0]);
              z[nn][1] = fmaf(f.y, vc[2 * hf + r], z[nn][1]);
              pb[nn][hf][r] = transpose8(*reinterpret_cast<const uint32_t *>(&h));
            }
          }
        }
      }
      // values: m tile 4 o + q holds dims 16 g + 8 o + 2 q (rows g) and + 1 (rows g + 8) of the lane's words
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t vw[4][VW];
#pragma unroll
        for (int r = 0; r < 4; ++r) lds<VW>(vw[r], st + MAPS * C::K_BYTES + ((4 * hf + r) * 32 + lane) * (4 * VW));
#pragma unroll
        for (int o = 0; o < VW; ++o)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7632u : 0x5410u;
            const uint32_t xa = prmt_b32(vw[0][o], vw[1][o], sel), xb = prmt_b32(vw[2][o], vw[3][o], sel);
            const uint32_t ya = xa >> 8, yb = xb >> 8;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(acc[n][4 * o + 2 * half], xa & 0x000f000fu, xa & 0x00f000f0u, xb & 0x000f000fu,
                       xb & 0x00f000f0u, pb[n][hf][0], pb[n][hf][1]);
              mma16816(acc[n][4 * o + 2 * half + 1], ya & 0x000f000fu, ya & 0x00f000f0u, yb & 0x000f000fu,
                       yb & 0x00f000f0u, pb[n][hf][0], pb[n][hf][1]);
            }
          }
      }
    }
    cp_wait<0>();

    // ---- the CTA's warps together: fragments [warp][n][mt][lane] and (R, l, z) [warp][column]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], o);
          z[n][i] += __shfl_xor_sync(0xffffffffu, z[n][i], o);
        }
    __syncthreads();                        // the ring is no longer read
    float4 *frag = reinterpret_cast<float4 *>(smem);
    float *stat = reinterpret_cast<float *>(smem + NW * NT * MT * 512);      // [warp][column][3]
    float *wts = stat + NW * NC * 3;                                         // [column][4]: R, l, z of the CTA
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < MT; ++k)
        frag[((warp * NT + n) * MT + k) * 32 + lane] =
            make_float4(acc[n][k][0], acc[n][k][1], acc[n][k][2], acc[n][k][3]);
      if (g == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float *p = stat + (warp * NC + 8 * n + 2 * t + i) * 3;
          p[0] = R[n][i];
          p[1] = l[n][i];
          p[2] = z[n][i];
        }
    }
    __syncthreads();
    if (tid < NC) {
      float M = -INFINITY;
      for (int x = 0; x < NW; ++x) M = fmaxf(M, stat[(x * NC + tid) * 3]);
      float ls = 0.f, zs = 0.f;
      for (int x = 0; x < NW; ++x) {
        float *p = stat + (x * NC + tid) * 3;
        const float f = p[0] == -INFINITY ? 0.f : exp2f(p[0] - M);
        ls += f * p[1];
        zs += f * p[2];
        p[0] = f;                           // the warp's weight
      }
      wts[4 * tid] = M;
      wts[4 * tid + 1] = ls;
      wts[4 * tid + 2] = zs;
    }
    __syncthreads();

    // this item's share holders: CTAs c0 .. c1
    const long long ia = pre + item * w.units, ib = ia + w.units;
    const int c0 = static_cast<int>(((ia + 1) * n_work - 1) / total), c1 = static_cast<int>((ib * n_work - 1) / total);
    const bool whole = c0 == c1;
    float *mine = a.part + static_cast<int64_t>(2 * blockIdx.x + (cur == share0 ? 0 : 1)) * C::PART;
    constexpr int NF = NT * MT * 32;        // float4 fragments per partial
    constexpr int PER = (NF + C::THREADS - 1) / C::THREADS;
    float4 o4[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int f = tid + k * C::THREADS;
      o4[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (f < NF) {
        const int col = 8 * (f / (MT * 32)) + 2 * (f & 3);
        for (int x = 0; x < NW; ++x) {
          const float4 v = frag[x * NF + f];
          const float w0 = stat[(x * NC + col) * 3], w1 = stat[(x * NC + col + 1) * 3];
          o4[k].x = fmaf(w0, v.x, o4[k].x);
          o4[k].y = fmaf(w1, v.y, o4[k].y);
          o4[k].z = fmaf(w0, v.z, o4[k].z);
          o4[k].w = fmaf(w1, v.w, o4[k].w);
        }
        if (!whole) reinterpret_cast<float4 *>(mine + 4 * NC)[f] = o4[k];
      }
    }
    bool finish = whole;
    if (!whole) {
      if (tid < NC) reinterpret_cast<float4 *>(mine)[tid] = *reinterpret_cast<float4 *>(wts + 4 * tid);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(a.counters + c0, 1) == c1 - c0;
      __syncthreads();
      finish = s_last != 0;
      if (finish) {
        __threadfence();
        if (tid == 0) a.counters[c0] = 0;
        // CTA c0's partial is in its slot 0 when the item's part begins its share, else in slot 1; the
        // others' parts begin their shares
        auto part_of = [&](int c) {
          return a.part + static_cast<int64_t>(2 * (c0 + c) + (c == 0 && c0 * total / n_work < ia ? 1 : 0)) * C::PART;
        };
        const int n_con = c1 - c0 + 1;
        float *cw = reinterpret_cast<float *>(smem);             // [CTA][column]: weight of its partial
        for (int col = warp; col < NC; col += NW) {
          float M = -INFINITY, ls = 0.f, zs = 0.f;
          for (int c = lane; c < n_con; c += 32) {
            const float r = __ldcg(part_of(c) + 4 * col);
            cw[c * NC + col] = r;
            M = fmaxf(M, r);
          }
          M = warp_max(M);
          for (int c = lane; c < n_con; c += 32) {
            const float4 p = __ldcg(reinterpret_cast<const float4 *>(part_of(c)) + col);
            const float f = p.x == -INFINITY ? 0.f : exp2f(p.x - M);
            cw[c * NC + col] = f;
            ls = fmaf(f, p.y, ls);
            zs = fmaf(f, p.z, zs);
          }
          ls = warp_sum(ls);
          zs = warp_sum(zs);
          if (lane == 0) {
            wts[4 * col + 1] = ls;
            wts[4 * col + 2] = zs;
          }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int f = tid + k * C::THREADS;
          o4[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (f < NF) {
            const int col = 8 * (f / (MT * 32)) + 2 * (f & 3);
            auto add = [&](int c, const float4 &v) {
              const float2 w2 = *reinterpret_cast<const float2 *>(cw + c * NC + col);
              o4[k].x = fmaf(w2.x, v.x, o4[k].x);
              o4[k].y = fmaf(w2.y, v.y, o4[k].y);
              o4[k].z = fmaf(w2.x, v.z, o4[k].z);
              o4[k].w = fmaf(w2.y, v.w, o4[k].w);
            };
            add(0, __ldcg(reinterpret_cast<const float4 *>(part_of(0) + 4 * NC) + f));
            const float4 *p = reinterpret_cast<const float4 *>(part_of(1) + 4 * NC) + f;
#pragma unroll 8
            for (int c = 1; c < n_con; ++c, p += 2 * C::PART / 4) add(c, __ldcg(p));
          }
        }
      }
    }
    if (finish) {
      // fragment f = (n, mt, lane): dims d, d + 1 of columns col, col + 1
      __syncthreads();                      // `frag` is free for the differential exchange
      float *ex = reinterpret_cast<float *>(smem);               // [column 8][DV] of map 0, then of the difference
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int f = tid + k * C::THREADS;
        if (f < NF) {
          const int n = f / (MT * 32), mt = (f / 32) % MT, fl = f & 31;
          const int d = (fl >> 2) * (DV / 8) + 8 * (mt >> 2) + 2 * (mt & 3);
          const int col = 8 * n + 2 * (fl & 3);
          float v[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float ls = wts[4 * (col + i) + 1], zs = wts[4 * (col + i) + 2];
            const float inv = ls != 0.f ? 1.f / ls : 0.f;        // nothing visible: zeros (NaN stays NaN)
            v[i][0] = ((i ? o4[k].y : o4[k].x) * 16777216.f + zs) * inv;
            v[i][1] = ((i ? o4[k].w : o4[k].z) * 1048576.f + zs) * inv;
            if (MAPS == 2) {
              ex[(col + i) * DV + d] = v[i][0];
              ex[(col + i) * DV + d + 1] = v[i][1];
            } else {
              const int c = c_base + col + i;
              if (c < cols_all && d < a.dv) {
                const int row = c / a.group, head = hv * a.group + c - row * a.group;
                store2(a.out, ((w.row0 + row) * static_cast<int64_t>(a.n_heads) + head) * a.dv + d, v[i][0], v[i][1],
                       a.bf16);
              }
            }
          }
        }
      }
      if (MAPS == 2) {
        // warp c: column c; o = map 0 - lambda map 1, RMS norm over the row, store
        __syncthreads();
        const int c = c_base + warp;
        if (c < cols_all) {
          const int row = c / a.group, head = hv * a.group + c - row * a.group;
          const float lam = a.lam[head];
          float y[DV / 32], ss = 0.f;
#pragma unroll
          for (int i = 0; i < DV / 64; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = 64 * i + 2 * lane + e;
              const float x = d < a.dv ? ex[warp * DV + d] - lam * ex[(8 + warp) * DV + d] : 0.f;
              y[2 * i + e] = x;
              ss = fmaf(x, x, ss);
            }
          ss = warp_sum(ss);
          const float r = a.norm_weight ? rsqrtf(ss / static_cast<float>(a.dv) + a.eps) * a.out_scale : a.out_scale;
#pragma unroll
          for (int i = 0; i < DV / 64; ++i) {
            const int d = 64 * i + 2 * lane;
            if (d < a.dv) {
              const float g0 = a.norm_weight ? a.norm_weight[d] : 1.f, g1 = a.norm_weight ? a.norm_weight[d + 1] : 1.f;
              store2(a.out, ((w.row0 + row) * static_cast<int64_t>(a.n_heads) + head) * a.dv + d, y[2 * i] * r * g0,
                     y[2 * i + 1] * r * g1, a.bf16);
            }
          }
        }
      }
    }
    __syncthreads();                        // shared memory is reused by the next segment
    cur += u1 - u0;
  }

  // sequences without cells: their rows are zeros
  for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x) {
    const few::SeqWork w = few::seq_work<COLS>(a, s, false);
    if (w.len == 0) {
      const int64_t n = static_cast<int64_t>(w.rows) * a.n_heads * a.dv / 2, at = static_cast<int64_t>(w.row0) * a.n_heads * a.dv;
      for (int64_t i = tid; i < n; i += C::THREADS) few::store2(a.out, at + 2 * i, 0.f, 0.f, a.bf16);
    }
  }
}

template <int DK, int DV, int NT, int MAPS>
cudaError_t launch_few_t(const AttnArgs &a, cudaStream_t s) {
  using C = FewCfg<DK, DV, NT, MAPS>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  static_assert(MAPS == 1 || NT == 2, "differential: one tile of columns per map");
  auto kern = few_kernel<DK, DV, NT, MAPS>;
  cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<sm_count() * C::CTAS, C::THREADS, C::SMEM, s>>>(a);
  return cudaGetLastError();
}

}  // namespace p4
}  // namespace tq
