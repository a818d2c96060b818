// Single-token attention over int8 cells.
//
//   out[c] = sum_t p_t s^V_t v_t / sum_t p_t,   p_t = 2^(x_t - R),  x_t = scale log2(e) s^K_t (q . k_t)
//
// Columns are the query heads of a KV head, eight per tensor-core tile.  The work is reading the cache once, so
// everything is arranged around the loads:
//
// - A warp streams its own 16-key tiles through a private ring of cp.async stages: it waits for its own copies only,
//   and no CTA barrier stands in the loop.  Each lane looks up one key's cell, so that pages of any size, single cells
//   among them, cost the same; the copying lanes get the row numbers by shuffles.  Rows are swizzled by 16-byte chunks
//   so that copies and both kinds of reads spread over the banks.
// - Codes become binary16 operands exactly: (w & 0x00ff00ff) ^ 0x64806480 is the pair 1024 + (code + 128), and 1152 is
//   taken off (three instructions for two codes).  Scores want pairs within a row: the words of a K row serve as they
//   are, the head dim's order being free as long as q has the same.  The value operand wants pairs of neighbouring
//   keys: two PRMT lay two rows' words side by side.
// - Scores: q is scaled by a power of two per column, so that its binary16 form is exact for binary16 and bfloat16
//   inputs down to 2^-23 of the column's largest entry.
// - The value weights p_t s^V_t are rounded to binary16: R is a running maximum of x_t + exponent(s^V_t), so the
//   largest weight lies in [1, 2^13] whatever the scales, and the sum of p_t stays in fp32.  R is raised only when it
//   would grow by more than 2^12.  Binary16 outputs (FINE) take what that rounding left in a second product, since it
//   would cost them nearly as much again as their own rounding.
//
// Split of the work as in the paged 4-bit kernel (tq_paged4_few.cuh): an item is a (sequence, KV head, column chunk),
// its keys come in units of 64; few items of like length are cut into even pieces, else all units form one line that is
// cut into equal shares.  CTAs that share an item leave partial results, the last to arrive merges them in the order of
// the CTAs.
#pragma once

#include <math.h>

#include "tq_common.cuh"
#include "tq_int8_cache.cuh"
#include "tq_paged4_few.cuh"
#include "tq_tc.cuh"

namespace tq {
namespace i8 {

using p4::AttnArgs;
using p4::RAISE;
using p4::UNIT;

constexpr int TILE = 16;              // keys per warp tile
constexpr int MIN_PIECE = 2;          // units of a piece at least: one tile for each of eight warps
constexpr int SET = p4::SETUP;         // units of work that an item costs besides its keys

template <int WK, int WV, int NT, bool FINE>
struct Cfg {
  static constexpr int KS = WK / 16, MT = WV / 16;        // k steps of the scores, m tiles of the values
  static constexpr int KCH = WK / 16, VCH = WV / 16;      // 16-byte chunks of a row
  static constexpr int NW = 8;
  static constexpr int THREADS = NW * 32;
  static constexpr int NC = 8 * NT;                       // columns
  static constexpr int CTAS = NT * (4 * MT + 2 * KS) <= 48 ? 2 : 1;     // per SM, by the registers
  // one stage: K rows, V rows, per key (K scale's word, V scale's word, selector of the half, -)
  static constexpr int K_BYTES = TILE * WK, V_BYTES = TILE * WV;
  static constexpr int SC = K_BYTES + V_BYTES;
  static constexpr int STAGE = SC + TILE * 16;
  static constexpr int MERGE = NW * NT * MT * 512 + NW * NC * 8 + NC * 8;       // CTA merge, in the same place
  static constexpr int BUDGET = (CTAS == 2 ? 111 : 222) * 1024;
  static constexpr int FIT = BUDGET / (NW * STAGE);
  static constexpr int STAGES = FIT > 4 ? 4 : FIT;
  static constexpr int RING = NW * STAGES * STAGE;
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  static constexpr int PART = 2 * NC + NT * MT * 128;     // a partial result: (R, l) of every column, then fragments
  // the grid: all CTAs that the SMs hold, as far as the merge of an item that every one of them shares finds room
  static constexpr int merge_bytes(int ctas) { return ctas * NC * 8 + THREADS * 16; }
  static constexpr int grid(int sms) {
    const int room = (SMEM - THREADS * 16) / (NC * 8), fit = room < p4::kMaxCtas ? room : p4::kMaxCtas;
    return sms < (fit + CTAS - 1) / CTAS ? sms * CTAS : fit;
  }
  static_assert(STAGES >= 2 && STAGE % 128 == 0, "stages");
};

// Byte offset of 16-byte chunk c of row r.  K: one lane quad reads four chunks of a row, eight lanes those of rows r and
// r + 1, which the turn of odd rows by four chunks puts on eight different places.  V: eight lanes read two neighbouring
// chunks of rows 0, 2, 4 and 6 (rows of 64 bytes: half chunks, two rows a line).
template <int W>
__device__ __forceinline__ uint32_t k_chunk(int r, int c) {
  return W == 64 ? r * 64 + c * 16 : r * W + ((c ^ ((r & 1) << 2)) * 16);
}
template <int W>
__device__ __forceinline__ uint32_t v_chunk(int r, int c) {
  return W == 64 ? (r >> 1) * 128 + (((((r & 1) << 2) + c) ^ (r & 6)) * 16) : r * W + ((c ^ (r & 6)) * 16);
}

// Codes in bytes 0 and 2 (even) or 1 and 3 (odd) of a word as a pair of binary16 numbers.
__device__ __forceinline__ uint32_t codes_at(uint32_t w) {
  const uint32_t x = (w & 0x00ff00ffu) ^ 0x64806480u;                     // 1024 + 128 + code
  const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), __float2half2_rn(1152.f));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t even_codes(uint32_t w) { return codes_at(w); }
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return codes_at(w >> 8); }

__device__ __forceinline__ float scale_of(uint32_t word, uint32_t sel) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(prmt_b32(word, 0u, sel))));
}

template <int WK, int WV, int NT, bool FINE>
__global__ void __launch_bounds__(Cfg<WK, WV, NT, FINE>::THREADS, Cfg<WK, WV, NT, FINE>::CTAS)
    decode_kernel(const AttnArgs a) {
  using C = Cfg<WK, WV, NT, FINE>;
  using namespace p4::few;
  constexpr int NW = C::NW, MT = C::MT, NC = C::NC;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Scan s_scan[NW];
  __shared__ int s_longest[NW];
  __shared__ float s_l[NC];
  __shared__ long long s_pre;
  __shared__ int s_seq, s_last;

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");     // nothing that earlier launches write is read before this

  // ---- this CTA's share of the work: a piece of an item, or the line's units [cur, end)
  Scan sum = {0, 0};
  long long lo = 0, hi = 0, first = 0;
  int longest = 0;
  for (int s0 = 0; s0 < a.n_seq; s0 += C::THREADS)
    scan_chunk<NC, NW>(a, s0, s_scan, blockIdx.x == 0, sum, lo, hi, first, longest);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) s_longest[warp] = longest;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) longest = max(longest, s_longest[w]);
  const long long total = sum.line;
  const int pieces = sum.item > 0 && sum.item <= gridDim.x ? gridDim.x / static_cast<int>(sum.item) : 0;   // per item
  // (a line costs a CTA the taking up of a second item, which the even pieces may then take longer)
  const bool even = pieces > 0 && static_cast<long long>(max(MIN_PIECE, (longest + pieces - 1) / pieces) - SET) *
                                          static_cast<long long>(gridDim.x) <= total;
  const long long n_work = even ? pieces * sum.item : min(static_cast<long long>(gridDim.x), total);
  const bool works = blockIdx.x < n_work;
  long long cur = 0, end = 0, pre = 0;
  int seq = 0;
  if (works) {
    cur = even ? blockIdx.x / pieces : blockIdx.x * total / n_work;        // (even: an item)
    end = even ? cur + 1 : (blockIdx.x + 1) * total / n_work;
    Scan at = {0, 0};
    for (int s0 = 0; s0 < a.n_seq; s0 += C::THREADS) {
      // (a batch of one chunk still has its sums in registers)
      if (a.n_seq > C::THREADS) scan_chunk<NC, NW>(a, s0, s_scan, false, at, lo, hi, first, longest);
      const int s = s0 + tid;
      if (s < a.n_seq && hi > lo) {
        const SeqWork w = seq_work<NC>(a, s, false);
        if (even ? first <= cur && cur < first + w.items : lo <= cur && cur < hi) {
          s_seq = s;
          s_pre = even ? first : lo;
        }
      }
    }
    __syncthreads();
    seq = s_seq;
    pre = s_pre;
  }
  const long long share0 = cur;

  // ---- the warp's ring, and the lane's places in its rows
  const uint32_t ring = tc::smem_u32(smem) + warp * (C::STAGES * C::STAGE);
  const uint32_t kc_at = k_chunk<WK>(lane / C::KCH, lane % C::KCH), vc_at = C::K_BYTES + v_chunk<WV>(lane / C::VCH, lane % C::VCH);
  const uint32_t k_size = (lane % C::KCH) * 16 < a.dk ? 16 : 0, v_size = (lane % C::VCH) * 16 < a.dv ? 16 : 0;
  uint32_t k_at[C::KS / 4];                     // reads: K row g, chunks t + 4 j
#pragma unroll
  for (int j = 0; j < C::KS / 4; ++j) k_at[j] = k_chunk<WK>(g, t + 4 * j);
  const uint32_t v_at = C::K_BYTES + (WV == 64 ? v_chunk<WV>(2 * t, g >> 1) + 8 * (g & 1) : v_chunk<WV>(2 * t, g));
  const int page_mask = (1 << a.page_shift) - 1;
  const uint8_t *k_base = a.k_codes + (k_size ? 16 * (lane % C::KCH) : 0), *v_base = a.v_codes + (v_size ? 16 * (lane % C::VCH) : 0);
  const uint16_t *scales = lane < TILE ? a.k_scales : a.v_scales;
  // (the last scale of a plane with an odd number of them is half a word)
  const uint32_t last_row = static_cast<uint32_t>(a.n_rows_cache - 1);

  while (cur < end) {
    // ---- one segment: units u0 .. u1 - 1 of an item, which CTAs c0 .. c0 + n_con - 1 share
    const SeqWork w = seq_work<NC>(a, seq, false);
    long long item, ia = 0;               // ia: the line's unit that is the item's first one
    int u0, u1, c0, n_con;
    if (even) {
      item = cur - pre;
      const int n = max(1, min(pieces, static_cast<int>(w.units) / MIN_PIECE)), i = blockIdx.x % pieces;
      if (i >= n) break;
      u0 = static_cast<int>(i * w.units / n);
      u1 = static_cast<int>((i + 1) * w.units / n);
      c0 = blockIdx.x - i;
      n_con = n;
      cur = end;
    } else {
      const long long per = w.units + SET;
      if (w.units == 0 || cur - pre >= per * w.items) {
        if (w.units > 0) pre += per * w.items;
        ++seq;
        continue;
      }
      item = (cur - pre) / per;
      const int r = static_cast<int>((cur - pre) - item * per), stop = static_cast<int>(min(per, r + (end - cur)));
      cur += stop - r;
      u0 = max(0, r - SET);
      u1 = max(0, stop - SET);
      if (u1 <= u0) continue;
      ia = pre + item * per + SET;
      auto owner = [&](long long x) { return static_cast<int>(((x + 1) * n_work - 1) / total); };
      c0 = owner(ia);
      n_con = owner(ia + w.units - 1) - c0 + 1;
    }
    const int hv = static_cast<int>(item) / w.chunks, chunk = static_cast<int>(item) - hv * w.chunks;
    const int c_base = chunk * NC, n_cols = min(NC, a.group - c_base);
    const int k_begin = u0 * UNIT, k_end = min(w.len, u1 * UNIT);
    const int n_tiles = k_end > k_begin ? (k_end - k_begin + TILE - 1) / TILE : 0;
    const int32_t *table = a.block_table + static_cast<int64_t>(seq) * a.max_pages;

    // ---- query rows: column g of tile n, the dims of this lane's K chunks (converted further down, while the
    // first copies are on their way)
    uint4 qraw[NT][C::KS / 4][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = 8 * n + g;
      const int64_t qb = seq * a.q_stride + static_cast<int64_t>(hv * a.group + c_base + c) * a.dk;
#pragma unroll
      for (int j = 0; j < C::KS / 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int d0 = 16 * (t + 4 * j) + 8 * i;
          qraw[n][j][i] = make_uint4(0, 0, 0, 0);
          if (c < n_cols && d0 < a.dk)
            qraw[n][j][i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + qb + d0));
        }
    }

    // ---- the warp's tile copies
    auto page_of = [&](int tile) {                              // of the lane's key (both halves of a warp look up the same)
      const int key = k_begin + tile * TILE + (lane & 15);
      return key < k_end ? __ldg(table + (key >> a.page_shift)) : -1;
    };
    auto issue = [&](int tile, int page, uint32_t st) {
      const int key = k_begin + tile * TILE + (lane & 15);
      const bool in = key < k_end, ok = in && static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages);
      if (in && !ok) set_status(a.status, TQ_ERR_DEVICE_CHECK);
      // (numbers of rows fit 32 bits, checked on the host; all ones: no row, zeros)
      const uint32_t row = ok ? ((static_cast<uint32_t>(page) << a.page_shift) + (key & page_mask)) *
                                        static_cast<uint32_t>(a.n_kv_heads) + hv
                              : 0xffffffffu;
      cp4(st + C::SC + (lane & 15) * 16 + (lane < TILE ? 0 : 4), scales + (ok ? row & ~1u : 0u),
          !ok ? 0 : row == last_row && !(row & 1) ? 2 : 4);
      if (lane < TILE)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + C::SC + lane * 16 + 8), "r"(row & 1 ? 0x4432u : 0x4410u) : "memory");
#pragma unroll
      for (int i = 0; i < C::KCH / 2; ++i) {
        const uint32_t r = __shfl_sync(0xffffffffu, row, i * (32 / C::KCH) + lane / C::KCH);
        cp16(st + kc_at + i * 512, k_base + (r == 0xffffffffu ? 0 : static_cast<uint64_t>(r) * a.dk),
             r == 0xffffffffu ? 0 : k_size);
      }
#pragma unroll
      for (int i = 0; i < C::VCH / 2; ++i) {
        const uint32_t r = __shfl_sync(0xffffffffu, row, i * (32 / C::VCH) + lane / C::VCH);
        // (the turn's share of i: rows of a copy lie 32 / VCH apart)
        const uint32_t turn = WV == 64 ? 0u : ((i * (32 / C::VCH)) & 6) * 16u;
        cp16(st + ((vc_at + i * 512) ^ turn), v_base + (r == 0xffffffffu ? 0 : static_cast<uint64_t>(r) * a.dv),
             r == 0xffffffffu ? 0 : v_size);
      }
    };
    uint32_t st = ring, st_fill = ring;           // the stage read, and the one filled, next
    auto next_stage = [&](uint32_t x) { return x == ring + (C::STAGES - 1) * C::STAGE ? ring : x + C::STAGE; };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
      const int tile = warp + i * NW;
      if (tile < n_tiles) issue(tile, page_of(tile), st_fill);
      st_fill = next_stage(st_fill);
      tc::cp_async_commit();
    }
    int page_next = page_of(warp + (C::STAGES - 1) * NW);

    // ---- query fragments
    uint32_t qf[NT][C::KS][2];
    float2 fx[NT];                  // of columns 2t, 2t + 1: the score factor
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float v[C::KS / 4][16], mx = 0.f;
#pragma unroll
      for (int j = 0; j < C::KS / 4; ++j) {
        unpack8(qraw[n][j][0], a.bf16, v[j]);
        unpack8(qraw[n][j][1], a.bf16, v[j] + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(v[j][e]));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // max in [2^ex, 2^(ex+1)) -> scaled to [2^12, 2^13), by two factors, so that each is a normal number
      const int ex = mx > 0.f ? static_cast<int>(__float_as_uint(mx) >> 23) - 127 : 0;
      const float s1 = __uint_as_float(static_cast<uint32_t>((12 - ex) / 2 + 127) << 23);
      const float s2 = __uint_as_float(static_cast<uint32_t>((12 - ex) - (12 - ex) / 2 + 127) << 23);
#pragma unroll
      for (int j = 0; j < C::KS / 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float *x = v[j] + 4 * i;
          qf[n][4 * j + i][0] = half2_bits(x[0] * s1 * s2, x[2] * s1 * s2);
          qf[n][4 * j + i][1] = half2_bits(x[1] * s1 * s2, x[3] * s1 * s2);
        }
      // this lane's softmax columns are 2t and 2t + 1: their factors sit in lanes g = 2t, 2t + 1
      const float f = a.scale_log2 * 0x1p-12f * __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
      fx[n] = make_float2(__shfl_sync(0xffffffffu, f, 8 * t), __shfl_sync(0xffffffffu, f, 8 * t + 4));
    }

    float acc[NT][MT][4];
    float2 R[NT], Rs[NT], l[NT];              // of columns 2t, 2t + 1; Rs: R, or 0 as long as there is none
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[n][i][c] = 0.f;
      R[n] = make_float2(-INFINITY, -INFINITY);
      Rs[n] = l[n] = make_float2(0.f, 0.f);
    }

    for (int tile = warp; tile < n_tiles; tile += NW, st = next_stage(st)) {
      const int key0 = k_begin + tile * TILE;
      cp_wait<C::STAGES - 2>();
      __syncwarp();               // everybody's copies of this tile are there; the slot filled next was read
      {
        const int nt = tile + (C::STAGES - 1) * NW;
        if (nt < n_tiles) issue(nt, page_next, st_fill);
        st_fill = next_stage(st_fill);
        tc::cp_async_commit();
        page_next = page_of(nt + NW);
      }

      // scores of keys g and g + 8, columns 2t and 2t + 1
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[n][c] = 0.f;
#pragma unroll
      for (int j = 0; j < C::KS / 4; ++j) {
        uint32_t w0[4], w1[4];
        lds<4>(w0, st + k_at[j]);
        lds<4>(w1, st + k_at[j] + 8 * WK);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x0 = even_codes(w0[i]), x1 = even_codes(w1[i]), x2 = odd_codes(w0[i]), x3 = odd_codes(w1[i]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(s[n], x0, x1, x2, x3, qf[n][4 * j + i][0], qf[n][4 * j + i][1]);
        }
      }
      float ks[2], vs[2], ve[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t u[4];
        lds<4>(u, st + C::SC + (g + 8 * r) * 16);
        ks[r] = scale_of(u[0], u[2]);
        vs[r] = scale_of(u[1], u[2]);
        ve[r] = vs[r] != 0.f ? static_cast<float>(static_cast<int>(__float_as_uint(fabsf(vs[r])) >> 23) - 127) : -24.f;
      }
      uint32_t pb[NT][2], pl[NT][2];        // weights as B fragments [keys 0-7, 8-15], and what their rounding left
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float2 x[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          x[r] = mul2(mul2(make_float2(ks[r], ks[r]), make_float2(s[n][2 * r], s[n][2 * r + 1])), fx[n]);
          if (key0 + 8 * r + g >= k_end) x[r] = make_float2(-INFINITY, -INFINITY);
        }
        const float mt[2] = {fmaxf(x[0].x + ve[0], x[1].x + ve[1]), fmaxf(x[0].y + ve[0], x[1].y + ve[1])};
        const bool raise = mt[0] > R[n].x + RAISE || mt[1] > R[n].y + RAISE;
        if (__any_sync(0xffffffffu, raise)) {
          auto lift = [&](float m, float &r, float &rs, float &lo, int i) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (m > r + RAISE) {
              const float f = exp2f(r - m);             // 0 at the first raise
              r = rs = m;
              lo *= f;
#pragma unroll
              for (int k = 0; k < MT; ++k) {
                acc[n][k][i] *= f;
                acc[n][k][i + 2] *= f;
              }
            }
          };
          lift(mt[0], R[n].x, Rs[n].x, l[n].x, 0);
          lift(mt[1], R[n].y, Rs[n].y, l[n].y, 1);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 d = sub2(x[r], Rs[n]);
          const float2 p = make_float2(tc::ex2(d.x), tc::ex2(d.y));
          l[n] = add2(l[n], p);
          const float2 wv = mul2(p, make_float2(vs[r], vs[r]));
          const __half2 h = __floats2half2_rn(wv.x, wv.y);
          pb[n][r] = transpose8(*reinterpret_cast<const uint32_t *>(&h));
          if (FINE) {
            const float2 left = sub2(wv, __half22float2(h));
            pl[n][r] = transpose8(half2_bits(left.x, left.y));
          }
        }
      }
      // values: m tile 2 i + e of a lane's word i holds dims 4 i + 2 e of its piece (rows g) and + 1 (rows g + 8)
      constexpr int VW = WV == 64 ? 2 : 4, VJ = WV == 256 ? 2 : 1;         // words of a piece, pieces
#pragma unroll
      for (int j = 0; j < VJ; ++j) {
        uint32_t w0[4], w1[4], w2[4], w3[4];      // keys 2t, 2t + 1, 2t + 8, 2t + 9
        const uint32_t at = st + v_at + j * 128;
        const uint32_t at1 = WV == 64 ? st + (v_at ^ 64u) : at + WV;
        lds<VW>(w0, at);
        lds<VW>(w1, at1);
        lds<VW>(w2, at + 8 * WV);
        lds<VW>(w3, at1 + 8 * WV);
#pragma unroll
        for (int i = 0; i < VW; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t sel = e ? 0x7632u : 0x5410u;
            const uint32_t ya = prmt_b32(w0[i], w1[i], sel), yb = prmt_b32(w2[i], w3[i], sel);
            const uint32_t x0 = even_codes(ya), x1 = odd_codes(ya), x2 = even_codes(yb), x3 = odd_codes(yb);
            const int m = (j * VW + i) * 2 + e;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(acc[n][m], x0, x1, x2, x3, pb[n][0], pb[n][1]);
              if (FINE) mma16816(acc[n][m], x0, x1, x2, x3, pl[n][0], pl[n][1]);
            }
          }
      }
    }
    cp_wait<0>();

    // ---- the CTA's warps together: fragments [warp][n][mt][lane] and (R, l) [warp][column]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, o);
        l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, o);
      }
    __syncthreads();                        // the ring is no longer read
    float4 *frag = reinterpret_cast<float4 *>(smem);
    float2 *stat = reinterpret_cast<float2 *>(smem + NW * NT * MT * 512);      // [warp][column]: (R, l), then a weight
    float2 *own = stat + NW * NC;                                              // [column]: the CTA's
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < MT; ++k)
        frag[((warp * NT + n) * MT + k) * 32 + lane] =
            make_float4(acc[n][k][0], acc[n][k][1], acc[n][k][2], acc[n][k][3]);
      if (g == 0) {
        stat[warp * NC + 8 * n + 2 * t] = make_float2(R[n].x, l[n].x);
        stat[warp * NC + 8 * n + 2 * t + 1] = make_float2(R[n].y, l[n].y);
      }
    }
    __syncthreads();
    if (tid < NC) {
      float M = -INFINITY, ls = 0.f;
      for (int x = 0; x < NW; ++x) M = fmaxf(M, stat[x * NC + tid].x);
      for (int x = 0; x < NW; ++x) {
        float2 *p = stat + x * NC + tid;
        const float f = p->x == -INFINITY ? 0.f : exp2f(p->x - M);
        ls += f * p->y;
        p->x = f;                           // the warp's weight
      }
      own[tid] = make_float2(M, ls);
      s_l[tid] = ls;
    }
    __syncthreads();

    // Fragments with columns that exist: of each (tile, m tile), lanes (g, t) with 1, 2 or 4 of the t.  A thread takes
    // PER of them, or several threads one.
    const int tsh = n_cols > 4 ? 2 : n_cols > 2 ? 1 : 0;
    const int n_frag = NT * MT * (8 << tsh);
    auto frag_at = [&](int v) { return (v >> (3 + tsh)) * 32 + ((v >> tsh) & 7) * 4 + (v & ((1 << tsh) - 1)); };
    auto col_of = [&](int f) { return 8 * (f / (MT * 32)) + 2 * (f & 3); };
    constexpr int PER = (NT * MT * 32 + C::THREADS - 1) / C::THREADS;
    auto add = [](float4 &o, float w0, float w1, const float4 &p) {
      o.x = fmaf(w0, p.x, o.x);
      o.y = fmaf(w1, p.y, o.y);
      o.z = fmaf(w0, p.z, o.z);
      o.w = fmaf(w1, p.w, o.w);
    };
    const bool whole = n_con == 1;
    float *mine = a.part + static_cast<int64_t>(2 * blockIdx.x + (even || share0 >= ia ? 0 : 1)) * C::PART;
    float4 o4[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int v = tid + k * C::THREADS;
      o4[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (v < n_frag) {
        const int f = frag_at(v), col = col_of(f);
#pragma unroll
        for (int x = 0; x < NW; ++x)
          add(o4[k], stat[x * NC + col].x, stat[x * NC + col + 1].x, frag[x * (NT * MT * 32) + f]);
        if (!whole) reinterpret_cast<float4 *>(mine + 2 * NC)[v] = o4[k];
      }
    }
    bool finish = whole;
    if (!whole) {
      if (tid < NC) reinterpret_cast<float2 *>(mine)[tid] = own[tid];
      __syncthreads();
      if (tid == 0) s_last = arrive_one(a.counters + c0) == n_con - 1;
      __syncthreads();
      finish = s_last != 0;
      if (finish) {
        if (tid == 0) a.counters[c0] = 0;
        // CTA c0's partial is in its slot 0 when the item's part begins its share, else in slot 1; the others' parts
        // begin their shares
        const int slot0 = even || c0 * total / n_work >= ia ? 0 : 1;
        auto part_of = [&](int c) { return a.part + static_cast<int64_t>(2 * (c0 + c) + (c == 0 ? slot0 : 0)) * C::PART; };
        // with few fragments, `teams` threads share one, each taking every teams-th partial
        const int teams = n_frag < C::THREADS ? C::THREADS / n_frag : 1, team = n_frag < C::THREADS ? tid / n_frag : 0;
        const int v0 = n_frag < C::THREADS ? tid - team * n_frag : tid;
        constexpr int B = C::CTAS == 2 ? 16 : 24;                // loads in flight per thread
        float4 p[B];
        auto fetch = [&](int c, int v) {
#pragma unroll
          for (int i = 0; i < B; ++i) {
            p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + i * teams < n_con && v < n_frag)
              p[i] = __ldcg(reinterpret_cast<const float4 *>(part_of(c + i * teams) + 2 * NC) + v);
          }
        };
        fetch(team, v0);                                         // on its way while the weights are worked out
        float *cw = reinterpret_cast<float *>(smem);             // [CTA][column]: weight of its partial
        float *cl = cw + n_con * NC;
        for (int col = warp; col < NC; col += NW) {
          float M = -INFINITY, ls = 0.f;
#pragma unroll 2
          for (int c = lane; c < n_con; c += 32) {
            const float2 r = __ldcg(reinterpret_cast<const float2 *>(part_of(c)) + col);
            cw[c * NC + col] = r.x;
            cl[c * NC + col] = r.y;
            M = fmaxf(M, r.x);
          }
          M = warp_max(M);
          for (int c = lane; c < n_con; c += 32) {
            const float r = cw[c * NC + col];
            const float f = r == -INFINITY ? 0.f : exp2f(r - M);
            cw[c * NC + col] = f;
            ls = fmaf(f, cl[c * NC + col], ls);
          }
          ls = warp_sum(ls);
          if (lane == 0) s_l[col] = ls;
        }
        __syncthreads();
        float4 *red = reinterpret_cast<float4 *>(cl + n_con * NC);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int v = v0 + k * C::THREADS, col = col_of(frag_at(v < n_frag ? v : 0));
          if (k > 0) fetch(team, v);
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c = team; c < n_con; c += B * teams) {
            if (c > team) fetch(c, v);
#pragma unroll
            for (int i = 0; i < B; ++i)
              if (c + i * teams < n_con) {
                const float2 w2 = *reinterpret_cast<const float2 *>(cw + (c + i * teams) * NC + col);
                add(o, w2.x, w2.y, p[i]);
              }
          }
          o4[k] = o;
        }
        if (teams > 1) {
          if (team > 0 && team < teams) red[(team - 1) * n_frag + v0] = o4[0];
          __syncthreads();
          if (team == 0)
            for (int x = 1; x < teams; ++x) add(o4[0], 1.f, 1.f, red[(x - 1) * n_frag + v0]);
        }
      }
    }
    if (finish) {
      // fragment f = (n, mt, lane): dims d, d + 1 of columns col, col + 1
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int v = tid + k * C::THREADS;
        if (v < n_frag) {
          const int f = frag_at(v), mt = (f / 32) % MT, fl = f & 31, col = col_of(f);
          constexpr int VW = WV == 64 ? 2 : 4;
          const int d = 128 * (mt / (2 * VW)) + 4 * VW * (fl >> 2) + 2 * (mt % (2 * VW));
          if (d < a.dv) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (col + i >= n_cols) continue;
              const float ls = s_l[col + i], inv = ls != 0.f ? 1.f / ls : 0.f;
              const int64_t at = (static_cast<int64_t>(seq) * a.n_heads + hv * a.group + c_base + col + i) * a.dv + d;
              store2(a.out, at, (i ? o4[k].y : o4[k].x) * inv, (i ? o4[k].w : o4[k].z) * inv, a.bf16);
            }
          }
        }
      }
    }
    __syncthreads();                        // shared memory is reused by the next segment's copies
  }

  // sequences without cells: their rows are zeros
  for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x) {
    if (seq_work<NC>(a, s, false).len == 0) {
      const int64_t n = static_cast<int64_t>(a.n_heads) * a.dv / 2, at = s * 2 * n;
      for (int64_t i = tid; i < n; i += C::THREADS) store2(a.out, at + 2 * i, 0.f, 0.f, a.bf16);
    }
  }
}

template <int WK, int WV, int NT, bool FINE>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t s) {
  using C = Cfg<WK, WV, NT, FINE>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  static_assert(C::merge_bytes(C::grid(1 << 20)) <= C::SMEM && C::grid(152) == 152 * C::CTAS, "merge");
  auto kern = decode_kernel<WK, WV, NT, FINE>;
  cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  return p4::launch_beside(kern, C::grid(sm_count()), C::THREADS, C::SMEM, s, a);
}

// up to eight columns in one tile, else two tiles at a time; binary16 outputs keep the weights to 22 bits
template <int WK, int WV>
cudaError_t launch_w(const AttnArgs &a, cudaStream_t s) {
  if (a.group <= 8) return a.bf16 ? launch_t<WK, WV, 1, false>(a, s) : launch_t<WK, WV, 1, true>(a, s);
  return a.bf16 ? launch_t<WK, WV, 2, false>(a, s) : launch_t<WK, WV, 2, true>(a, s);
}

}  // namespace i8
}  // namespace tq
