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
// tile and P written over it, a tile's scores had to wait for its P V: 1200 us at 2048
// rows over 32768 cells, 8 KV heads, against 1016 us in that step.)  A softmax thread
// has its weights in registers before it waits for the tile's last P V, so only their
// store stands between two products (807 -> 786 us).
// The code of all roles has to stay small: with the products' loops unrolled for one
// thread and a whole row's 128 keys per softmax thread, the product warp waited for
// instructions (1390 us in that form).
//
// Numbers:
// - Scores: K's operand is the code itself (a nibble masked in place reads as the
//   binary16 subnormal code 2^-24 or 2^-20, exact), q is scaled by a power of two
//   per row (exact for 16-bit inputs down to 2^-23 of the row's largest entry).  The
//   offset's term rides along as one more k step: with a_t = m_t / s_t in two
//   binary16 parts and sum(q) in three for the first of them and two for the second,
//   the product is s_t-free, so the softmax multiplies a score by one number per key,
//   s_t, in fp32.  Parts and powers of two leave errors of 2^-22 of a_t and of some
//   2^-21 of q's largest entry.  (A row with |a_t| >= 2^23 is constant to 2e-6 and
//   takes its offset alone.)
// - Values: v_t 2^-tau rounded to binary16 (relative 2^-12 on average half), tau the
//   largest exponent among 32 neighbouring keys; the weights p_t 2^tau are rounded
//   to binary16 too.  Both roundings meet the values themselves.  To bfloat16 outputs
//   they are nothing; binary16 outputs have 2.9e-4 relative error at 2048 rows over
//   32768 cells, against 2.1e-4 of rounding alone, and at worst (few thousand keys of
//   like weight, values around 0) 3.5e-4 against 2.0e-4.  (Centred codes as the value
//   operand, scales in the weights and offsets in an fp32 sum come to 2.5e-4, in 1012 us
//   instead of 787 at that step: two more numbers per key and row from shared memory.)  R is a
//   running maximum of x_t + tau, raised only when it would grow by more than 2^12
//   (which binary16 weights leave room for; with 2^8 the rescaling of O cost a tenth of
//   the time).  Sums of weights stay in fp32.
// - Where the largest values of the 32 keys are more than 2^SPREAD apart, each key has
//   its own tau instead.  (A shared one rounds a key's values in steps set by another
//   key, which a row may give no weight or, as a later row's, not see at all: by 0.5%
//   at 2^-14 of the largest, and to nothing at 2^-24.  Up to 2^SPREAD it costs 2^-15 of
//   the key's largest value: 15 times the rounding of a subnormal scale.)  The softmax
//   threads then add a key's tau to its score and sum the weights by 2^-tau each: 776 us
//   without such rows, 794 with one in every fiftieth page of 64 cells, 1231 with some
//   among every 32 keys.
//
// What bounds it (2048 rows over 32768 cells: 775 us, 1.38 PFLOP/s of 1.92): a pair of
// row tiles takes 3640 clocks per key tile, set-up of items included, of which the tensor
// pipe is busy 2400 (the k step for the offset included), the schedulers issue in 2500
// and the exponentials take 1050; the rest is the chain scores - softmax - P V of the two
// tiles.  Part of the exponentials by a polynomial was slower in every share (an eighth
// 794 us, a quarter 831, against 787 then): the instructions weigh more.  Short calls are
// bound by the way to the first product, 13000 clocks of 22000 for one key tile, mostly
// instructions fetched for the first time: Q, lengths and output are read and written by
// whole lines and without divisions for that (5 prompts of up to 300 rows 38.2 -> 31.8 us;
// 31.4 now).
//
// Split of the work, two ways:
// - LINE, where there are many (row tile, KV head) items: their key tiles, with
//   ITEM_COST empty ones before each item, form one line that is cut into equal shares,
//   one per SM, from the device's lengths.  A CTA's first and last item may be shared with
//   others: partial results go to the workspace and the last CTA to arrive merges them,
//   in the order of the CTAs.
// - else (a short chunk behind a long context) each item's keys are cut into n_split
//   parts, a CTA each, whose partial results a second kernel merges with all SMs: one
//   CTA would read up to 16 parts of 135 KB alone.
// Differential attention's two maps run as separate heads (their products share
// nothing but V), and the second kernel forms the difference and the norm.
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
constexpr int ITEM_COST = 4;                  // key tiles' worth of time that an item costs besides its keys
constexpr int NT = 768;
constexpr int W_UNPACK = 16, W_MMA = 20, W_NEXT = 21;      // first warps of the roles after the softmax
constexpr int SPREAD = 6;                     // exponents that 32 keys' values may be apart and still share one
constexpr int REG_SOFTMAX = 96, REG_UNPACK = 64, REG_MMA = 32;    // of 80 at the launch: 4 x 96 + 64 + 32 = 6 x 80

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
  static constexpr uint32_t STAU = SSC + 4 * BN * 4;           // [j & 3][32 keys] (tau, 2^-tau), or (-, 0): one per key
  static constexpr uint32_t SROW = STAU + 4 * 4 * 8;           // [tile][half][row] exchange between a row's threads
  static constexpr uint32_t SFX = SROW + 2 * 2 * BM * 8;       // [row] factor of a row's scores
  static constexpr uint32_t SKTAU = SFX + 2 * BM * 4;          // [j & 3][key] (tau, 2^-tau) of each key
  static constexpr uint32_t TOTAL = SKTAU + 4 * BN * 8;
  static constexpr int SKS = KC / 2, PKS = BN / 16;            // k steps of S and of PV
};

struct Bars {
  uint64_t k[2], v[2];    // K, V of key tile j (buffer j & 1) written    phase j >> 1
  uint64_t sc[4];         // scales of key tile j (j & 3) written         phase j >> 2
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
// found the phase open slept on past its end, on every step of the chain score - softmax - product (1282 us with it,
// 1233 without, at 2048 rows over 32768 cells).
// SLEEP: with a pause between two tries, for the unpack warps, which have time and leave the others their issue slots
// (811 -> 804 us).
template <bool SLEEP = false>
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity) {
  const uint32_t at = tc::smem_u32(bar);
  for (int it = 0; it < (1 << 19); ++it) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(at), "r"(parity)
                 : "memory");
    if (__all_sync(0xffffffffu, ok != 0)) return true;
    if (SLEEP) __nanosleep(64);
  }
  return false;
}

// one lane of the warp, the same every time
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void sts1(uint32_t at, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}
__device__ __forceinline__ void sts4(uint32_t at, const uint32_t *x) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
}
__device__ __forceinline__ float lds1(uint32_t at) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }

// A piece of an item: key tiles t_lo .. t_lo + n_t - 1 of 256 rows of one sequence and K head kh, with what every
// role needs to know of the rows.
struct Piece {
  int seq, kh;
  int t_lo, n_t;            // n_t < 0: no more pieces
  int c0, n_con, slot;      // LINE: the CTAs that share the item, c0 .. c0 + n_con - 1; where this partial goes
  int slot0;                // ... and where that of c0 is
  int row0, rem;            // row of the input and head of the group of the tile's first row
  int left;                 // rows of the sequence from the tile's first one on
  int lim0;                 // keys that the tile's first row's query sees (below 0: none)
  int kv_hi;                // ... and its last row's
};

// 256-row tile `i` of a sequence of w.rows queries: its first row is head `rem` of query `q`.  Walked in order, so
// that one division per sequence does.
struct Tile {
  int i, q, rem;
  int rows_all, dq, dr;     // rows of the sequence; 256 rows are dq queries and dr heads
};
__device__ __forceinline__ Tile first_tile(const AttnArgs &a, const few::SeqWork &w, int i) {
  Tile t;
  t.i = i;
  t.rows_all = w.rows * a.group;
  t.dq = 2 * BM / a.group;
  t.dr = 2 * BM - t.dq * a.group;
  t.q = i * 2 * BM / a.group;
  t.rem = i * 2 * BM - t.q * a.group;
  return t;
}
__device__ __forceinline__ void next_tile(const AttnArgs &a, Tile &t) {
  ++t.i;
  t.q += t.dq;
  t.rem += t.dr;
  if (t.rem >= a.group) {
    t.rem -= a.group;
    ++t.q;
  }
}
__device__ __forceinline__ int kv_hi_of(const AttnArgs &a, const few::SeqWork &w, const Tile &t) {
  // (the query of row 255 is the one before the next tile's first row's, or its own)
  int last = w.rows - 1;
  if (t.rows_all - t.i * 2 * BM > 2 * BM) last = t.q + t.dq - (t.rem + t.dr == 0 ? 1 : 0) + (t.rem + t.dr > a.group ? 1 : 0);
  return a.causal ? max(0, w.len - w.rows + last + 1) : w.len;
}
__device__ __forceinline__ int key_tiles(int kv_hi) { return (static_cast<uint32_t>(kv_hi) + BN - 1) / BN; }
__device__ __forceinline__ int tiles_of(const AttnArgs &a, const few::SeqWork &w) {
  return (static_cast<uint32_t>(w.rows * a.group) + 2 * BM - 1) / (2 * BM);
}
__device__ __forceinline__ void rows_of_piece(const AttnArgs &a, const few::SeqWork &w, const Tile &t, Piece &p) {
  p.row0 = w.row0 + t.q;
  p.rem = t.rem;
  p.left = t.rows_all - t.i * 2 * BM;
  p.lim0 = a.causal ? w.len - w.rows + t.q + 1 : w.len;
  p.kv_hi = kv_hi_of(a, w, t);
}

// A piece, read anew (what only begin and end of its work need is not kept in registers through the loop).
__device__ __forceinline__ Piece read_piece(const Piece *p) {
  const volatile int *q = reinterpret_cast<const volatile int *>(p);
  return {q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7], q[8], q[9], q[10], q[11], q[12]};
}

// Row `r` (of 256) of a piece: its query's row of the input, its head within the group.
__device__ __forceinline__ void query_of(const AttnArgs &a, int rem, int r, int &qi, int &head) {
  // floor((x + 1/2) / G) in fp32 is exact: x < 2^22, and (x + 1/2) / G is at least 1 / 2G away from an integer
  const int x = rem + r;
  qi = static_cast<int>((static_cast<float>(x) + 0.5f) * a.inv_group);
  head = x - qi * a.group;
}

// One CTA's walk along the line (one thread).
struct Walk {
  long long cur, end, pre;  // units of the line; pre: where the current item begins
  long long share0, total, n_work;
  int seq, tile, kh;
};
__device__ inline Piece next_piece(const AttnArgs &a, Walk &w) {
  Piece p = {0, 0, 0, -1, 0, 1, 0, 0, 0, 0, 0, 0, 0};
  const int k_heads = (a.diff ? 2 : 1) * a.n_kv_heads;
  while (w.cur < w.end) {
    const few::SeqWork sw = few::seq_work<1>(a, w.seq, false);
    if (w.tile >= tiles_of(a, sw)) {
      ++w.seq;
      w.tile = w.kh = 0;
      continue;
    }
    const Tile t = first_tile(a, sw, w.tile);
    const int tiles = key_tiles(kv_hi_of(a, sw, t)), per = tiles + ITEM_COST;
    const int r = static_cast<int>(w.cur - w.pre);
    if (r >= per) {                           // the next item: heads first, then tiles
      w.pre += per;
      if (++w.kh == k_heads) {
        w.kh = 0;
        ++w.tile;
      }
      continue;
    }
    const int stop = static_cast<int>(min(static_cast<long long>(per), r + (w.end - w.cur)));
    w.cur += stop - r;
    const int u0 = max(0, r - ITEM_COST), u1 = max(0, stop - ITEM_COST);
    // (an item without keys is its last empty unit's: its rows are zeros)
    if (u1 <= u0 && !(tiles == 0 && stop == per)) continue;
    p.seq = w.seq;
    rows_of_piece(a, sw, t, p);
    p.kh = w.kh;
    p.t_lo = u0;
    p.n_t = u1 - u0;
    if (tiles > 0) {
      const long long ia = w.pre + ITEM_COST;
      auto owner = [&](long long x) { return static_cast<int>(((x + 1) * w.n_work - 1) / w.total); };
      p.c0 = owner(ia);
      p.n_con = owner(ia + tiles - 1) - p.c0 + 1;
      p.slot = w.share0 >= ia ? 0 : 1;
      p.slot0 = p.c0 * w.total / w.n_work >= ia ? 0 : 1;
    }
    return p;
  }
  return p;
}

}  // namespace pre

template <int DK, int DV, bool LINE>
__global__ void __launch_bounds__(pre::NT, 1) prefill_kernel(const AttnArgs a) {
  using namespace pre;
  using C = Cfg<DK, DV>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) Bars bars;
  __shared__ Piece s_piece[2];
  __shared__ Walk s_walk;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_fail, s_last;
  __shared__ long long s_sum[32];            // of warps (fewer than 32), or of 32 sequences

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int maps = a.diff ? 2 : 1, k_heads = maps * a.n_kv_heads, G = a.group;

  if (warp == W_MMA) tc::tmem_alloc<512>(&tmem_slot);
  if (tid == NT - 1) {
    for (int i = 0; i < 4; ++i) tc::mbar_init(&bars.sc[i], 4);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.k[i], 4);
      tc::mbar_init(&bars.v[i], 4);
      tc::mbar_init(&bars.kf[i], 2);
      tc::mbar_init(&bars.s[i], 1);
      tc::mbar_init(&bars.rd[i], 8);
      tc::mbar_init(&bars.p[i], 8);
      tc::mbar_init(&bars.pv[i][0], 1);
      tc::mbar_init(&bars.pv[i][1], 1);
    }
    tc::mbar_init_fence();
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
  // The launch may have begun beside the one before it (programmatic dependent launch).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // ---- the first piece.  Up to 32 sequences each warp finds it alone, else the CTA together.
  if (tid == 0) {
    s_fail = 0;
    s_piece[0].n_t = s_piece[1].n_t = -1;
  }
  __syncwarp();
  {
    // in the split form heads fastest, row tiles slowest and from the last one down (under a causal mask the
    // longest first)
    const int want = LINE ? 0 : a.n_tiles - 1 - static_cast<int>(blockIdx.x) / k_heads / a.n_split;
    const bool alone = a.n_seq <= 32;
    auto scan = [&](long long v) {            // over the warp, inclusive
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      return v;
    };
    // the same over the CTA, behind `at`; moves `at` past all of it
    auto scan_all = [&](long long v, long long &at) {
      long long x = scan(v), all = 0;
      __syncthreads();
      if (lane == 31) s_sum[warp] = x;
      __syncthreads();
      for (int k = 0; k < NT / 32; ++k) {
        if (k == warp) x += all;
        all += s_sum[k];
      }
      x += at;
      at += all;
      return x;
    };
    if (!LINE) {
      long long at = 0;
      for (int s0 = 0; s0 < a.n_seq; s0 += NT) {
        const int s = s0 + (alone ? lane : tid);
        few::SeqWork w;
        long long v = 0;
        if (s < a.n_seq) {
          w = few::seq_work<1>(a, s, blockIdx.x == 0);
          v = tiles_of(a, w);
        }
        const long long x = alone ? scan(v) : scan_all(v, at);
        if (v > 0 && x - v <= want && want < x && (warp == 0 || !alone)) {
          Piece p = {s, static_cast<int>(blockIdx.x) % k_heads, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0, 0};
          rows_of_piece(a, w, first_tile(a, w, static_cast<int>(want - (x - v))), p);
          const int tiles = key_tiles(p.kv_hi), split = static_cast<int>(blockIdx.x) / k_heads % a.n_split;
          p.t_lo = tiles * split / a.n_split;                // (below 2^24 tiles, 16 splits)
          p.n_t = tiles * (split + 1) / a.n_split - p.t_lo;
          s_piece[0] = p;
        }
      }
    } else {
      auto cost = [&](const few::SeqWork &w, const Tile &t) {
        return static_cast<long long>(key_tiles(kv_hi_of(a, w, t)) + ITEM_COST) * k_heads;
      };
      long long begin = 0, end = 0, n_work = 0, total = 0;
      auto share = [&]() {
        n_work = min(static_cast<long long>(gridDim.x), total);
        if (blockIdx.x >= n_work) return false;
        begin = blockIdx.x * total / n_work;
        end = (blockIdx.x + 1) * total / n_work;
        return true;
      };
      if (alone) {                            // a warp per sequence, a lane per tile
        for (int s = warp; s < a.n_seq; s += NT / 32) {
          const few::SeqWork w = few::seq_work<1>(a, s, blockIdx.x == 0);
          const int n = tiles_of(a, w);
          long long v = 0;
          for (int i = lane; i < n; i += 32) v += cost(w, first_tile(a, w, i));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane == 0) s_sum[s] = v;
        }
        __syncthreads();
        const long long v = lane < a.n_seq ? s_sum[lane] : 0, x = scan(v);
        total = __shfl_sync(0xffffffffu, x, 31);
        if (share() && x - v <= begin && begin < x && warp == 0) {
          s_walk.seq = lane;
          s_walk.pre = x - v;
        }
      } else {                                // a thread per sequence; a second pass finds the share's begin
        for (int pass = 0; pass < 2; ++pass) {
          if (pass == 1 && !share()) break;
          long long at = 0;
          for (int s0 = 0; s0 < a.n_seq; s0 += NT) {
            const int s = s0 + tid;
            long long v = 0;
            if (s < a.n_seq) {
              const few::SeqWork w = few::seq_work<1>(a, s, pass == 0 && blockIdx.x == 0);
              const int n = tiles_of(a, w);
              for (Tile t = first_tile(a, w, 0); t.i < n; next_tile(a, t)) v += cost(w, t);
            }
            const long long x = scan_all(v, at);
            if (pass == 1 && x - v <= begin && begin < x) {
              s_walk.seq = s;
              s_walk.pre = x - v;
            }
          }
          total = at;
        }
        __syncthreads();
      }
      if (warp == 0 && blockIdx.x < n_work) {                // the tile and head where the share begins
        __syncwarp();
        Walk k = {begin, end, s_walk.pre, begin, total, n_work, s_walk.seq, 0, 0};
        const few::SeqWork w = few::seq_work<1>(a, k.seq, false);
        const int n = tiles_of(a, w);
        for (int i0 = 0; i0 < n; i0 += 32) {
          const long long c = i0 + lane < n ? cost(w, first_tile(a, w, i0 + lane)) : 0, x = scan(c) + k.pre;
          const uint32_t hit = __ballot_sync(0xffffffffu, begin < x);
          const int l = hit ? __ffs(hit) - 1 : 31;
          k.pre = __shfl_sync(0xffffffffu, hit ? x - c : x, l);
          if (hit) {
            k.tile = i0 + l;
            const long long per = __shfl_sync(0xffffffffu, c, l) / k_heads;
            k.kh = static_cast<int>((begin - k.pre) / per);
            k.pre += k.kh * per;
            break;
          }
        }
        __syncwarp();
        if (lane == 0) {
          s_piece[0] = next_piece(a, k);
          s_walk = k;
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  if (s_piece[0].n_t < 0) {                   // no work for this CTA
    if (warp == W_MMA) tc::tmem_dealloc<512>(tmem);
    return;
  }
  const uint32_t sbase = tc::smem_u32(smem);
  constexpr uint32_t TS = 0, TP = 128, TO = 256;        // TMEM columns: S, P of tile X at 128 + 64 X, O at 256 + 128 X
  // Barriers of the CTA: 0 all warps between two pieces; 1 .. 8 the two warps of 32 rows; 9 Q written (softmax
  // and product warps); 10 the softmax warps.  Phases of the mbarriers count the CTA's key tiles over all pieces
  // (J below); a tile B without rows takes part in them without work.
  constexpr int BAR_Q = 9, BAR_SOFT = 10;

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
      int base = 0;
      for (int i = 0;; ++i) {
        const int n_t = s_piece[i & 1].n_t;
        if (n_t < 0) break;
        const bool two = s_piece[i & 1].left > BM;
        auto product = [&](int x, int j) {    // O += P V of row tile x, key tile j of the piece
          const int J = base + j;
          if (x == 0) ok = wait_warp(&bars.v[J & 1], (J >> 1) & 1);
          if (ok) ok = wait_warp(&bars.p[x], J & 1);
          if (!ok) return;
          tc::fence_after_sync();
          const uint64_t v = v0 + static_cast<uint64_t>((J & 1) * (C::KV_BYTES >> 4));
          if (one) {
            if (x == 0 || two) {
#pragma unroll
              for (int ks = 0; ks < C::PKS; ++ks)
                mma_ta(tm + TO + 128 * x, tm + TP + 64 * x + 8 * ks, v + ((ks * 2 * C::VC * 128) >> 4), ID_PV,
                       j > 0 || ks > 0);
            }
            tc::mma_commit(&bars.pv[x][J & 1]);
          }
          __syncwarp();
        };
        tc::named_sync(BAR_Q, 32 * (W_UNPACK + 1));
        // steps (j, x): scores once the step before has read its own, then the product of this row tile's step
        // before.  (Its P is ready by the time that the scores are read: the same threads do both, in this order.)
        for (int j = 0; j <= n_t && ok && n_t > 0; ++j) {
          const int J = base + j;
          const uint64_t k = k0 + static_cast<uint64_t>((J & 1) * (C::KV_BYTES >> 4));
#pragma unroll 1
          for (int x = 0; x < 2 && ok; ++x) {
            if (j < n_t) {
              if (x == 0) ok = wait_warp(&bars.k[J & 1], (J >> 1) & 1);
              const int Jl = x == 0 ? J - 1 : J;                        // the step before: (Jl, 1 - x)
              if (ok && Jl >= 0) ok = wait_warp(&bars.rd[1 - x], Jl & 1);
              if (!ok) break;
              tc::fence_after_sync();
              if (one) {
                if (x == 0 || two) {
#pragma unroll
                  for (int ks = 0; ks < C::SKS; ++ks)
                    tc::mma_f16(tm + TS, q0 + x * (C::Q_BYTES >> 4) + ((ks * 4096) >> 4), k + ((ks * 256) >> 4), ID_S,
                                ks > 0);
                }
                tc::mma_commit(&bars.s[x]);
                tc::mma_commit(&bars.kf[J & 1]);
              }
              __syncwarp();
            }
            if (j > 0) product(x, j - 1);
          }
        }
        if (!ok) s_fail = 1;
        base += n_t;
        __syncthreads();
      }
    } else {
      // the piece after the current one; the other warps only meet the CTA
      for (int i = 0;; ++i) {
        if (s_piece[i & 1].n_t < 0) break;
        if (warp == W_NEXT && lane == 0) {
          if (LINE) {
            Walk k = s_walk;
            s_piece[(i + 1) & 1] = next_piece(a, k);
            s_walk = k;
          } else {
            s_piece[(i + 1) & 1].n_t = -1;
          }
        }
        __syncwarp();
        __syncthreads();
      }
    }
  } else if (warp >= W_UNPACK) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_UNPACK));
    // ===================== unpack: one key of the tile per thread =====================
    const int key = tid - 32 * W_UNPACK;
    const int mask = (1 << a.page_shift) - 1;
    bool ok = true;
    int base = 0;
    for (int i = 0;; ++i) {
      const Piece pc = s_piece[i & 1];
      if (pc.n_t < 0) break;
      const int n_t = pc.n_t, t_lo = pc.t_lo, kh = pc.kh, hv = kh / maps;
      const int kv_hi = pc.kv_hi;
      const int32_t *table = a.block_table + static_cast<int64_t>(pc.seq) * a.max_pages;
      auto page_of = [&](int j) {
        const uint32_t t = static_cast<uint32_t>(t_lo + j) * BN + key;               // (up to 2^31 + 127)
        return j < n_t && t < static_cast<uint32_t>(kv_hi) ? __ldg(table + (t >> a.page_shift)) : -2;   // no such key
      };
      constexpr int CK = DK / 32, CV = DV / 32;
      constexpr uint32_t NONE = 0xffffffffu;
      uint4 kraw[CK], vraw[CV];
      uint32_t ksm = 0, vsm = 0;              // (scale, offset) pairs
      uint32_t kr, vr;                        // rows of the planes (below 2^32 by the caches' limits)
      auto rows_of = [&](int j, int page) {
        kr = vr = NONE;
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.n_pages)) {
          if (page != -2) set_status(a.status, TQ_ERR_DEVICE_CHECK);                 // a zero row
          return;
        }
        const uint32_t in = (static_cast<uint32_t>(t_lo + j) * BN + key) & mask;
        const uint32_t pg = static_cast<uint32_t>(page) * a.n_kv_heads;
        kr = ((pg * maps + kh) << a.page_shift) + in;
        vr = ((pg + hv) << a.page_shift) + in;
      };
      auto load_k = [&]() {
        ksm = kr != NONE ? __ldg(reinterpret_cast<const uint32_t *>(a.k_scales) + kr) : 0;
#pragma unroll
        for (int c = 0; c < CK; ++c) {
          kraw[c] = make_uint4(0, 0, 0, 0);
          if (kr != NONE)
            kraw[c] = __ldg(reinterpret_cast<const uint4 *>(a.k_codes + static_cast<uint64_t>(kr) * (DK / 2)) + c);
        }
      };
      auto load_v = [&]() {
        vsm = vr != NONE ? __ldg(reinterpret_cast<const uint32_t *>(a.v_scales) + vr) : 0;
#pragma unroll
        for (int c = 0; c < CV; ++c) {
          vraw[c] = make_uint4(0, 0, 0, 0);
          if (vr != NONE)
            vraw[c] = __ldg(reinterpret_cast<const uint4 *>(a.v_codes + static_cast<uint64_t>(vr) * (DV / 2)) + c);
        }
      };
      rows_of(0, page_of(0));
      load_k();
      load_v();
      int page = page_of(1);
      for (int j = 0; j < n_t; ++j) {
        const int J = base + j, b = J & 1;
        if (J >= 2) ok = wait_warp<true>(&bars.kf[b], ((J - 2) >> 1) & 1);    // the K buffer's last users
        if (!ok) { s_fail = 1; break; }
        unsigned char *kd = smem + C::SKV + b * C::KV_BYTES + (key >> 3) * (C::KC * 128) + (key & 7) * 16;
        unsigned char *vd = smem + C::SKV + b * C::KV_BYTES + C::K_BYTES + (key >> 3) * (C::VC * 128) + (key & 7) * 16;
        // exponent of the 32 keys' values (with K: the softmax needs it), or of the key's own where they are far apart
        const float2 vsc = __half22float2(as_half2(vsm));
        const float top = fmaxf(fabsf(vsc.y), fabsf(fmaf(15.f, vsc.x, vsc.y)));
        const int own = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        const int most = __reduce_max_sync(0xffffffffu, own);
        const bool apart = __any_sync(0xffffffffu, top > 0.f && most - own > SPREAD);
        const int e = min(30, max(-30, apart ? own : most));
        const float dn = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);            // 2^-tau
        reinterpret_cast<float2 *>(smem + C::SKTAU)[(J & 3) * BN + key] = make_float2(static_cast<float>(e), dn);
        if (lane == 0)
          reinterpret_cast<float2 *>(smem + C::STAU)[(J & 3) * 4 + (warp - W_UNPACK)] =
              make_float2(static_cast<float>(e), apart ? 0.f : dn);
        {
          float2 sm = __half22float2(as_half2(ksm));
          float off = __fdividef(sm.y, sm.x);
          uint32_t keep = 0xffffffffu;
          if (!(fabsf(off) < 0x1p23f)) {      // (a scale of 0 too) constant row: its offset alone
            keep = 0;
            off = sm.y > 0.f ? 0x1p16f : sm.y < 0.f ? -0x1p16f : 0.f;
            sm.x = sm.y != 0.f ? fabsf(sm.y) * 0x1p-16f : 1.f;
          }
          // off 2^-8 = hi + lo 2^-8: times sum(q) 2^-16 and, for lo, 2^-24, of which each has its own parts
          const __half hi = __float2half_rn(off * 0x1p-8f);
          const __half lo = __float2half_rn(off - __half2float(hi) * 0x1p8f);
          *reinterpret_cast<uint4 *>(kd + (DK / 8) * 128) =
              make_uint4(bits(__halves2half2(hi, hi)), bits(__halves2half2(hi, lo)),
                         bits(__halves2half2(lo, __float2half_rn(0.f))), 0);
          reinterpret_cast<float *>(smem + C::SSC)[(J & 3) * BN + key] = sm.x;
#pragma unroll
          for (int i = 0; i < CK; ++i) {
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
        if (lane == 0) {
          tc::mbar_arrive(&bars.sc[J & 3]);
          tc::mbar_arrive(&bars.k[b]);
        }
        rows_of(j + 1, page);
        load_k();                             // on its way while the values are unpacked
        if (J >= 2)                           // the V buffer's last users
          for (int x = 0; x < 2 && ok; ++x) ok = wait_warp<true>(&bars.pv[x][b], ((J - 2) >> 1) & 1);
        if (!ok) { s_fail = 1; break; }
        {
          const __half2 vs = __float2half2_rn(vsc.x * dn), vm = __float2half2_rn(vsc.y * dn);
          const __half2 k1024 = as_half2(0x64006400u), k16 = as_half2(0x2c002c00u), k64 = as_half2(0xd400d400u);
#pragma unroll
          for (int i = 0; i < CV; ++i) {
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
        load_v();
        page = page_of(j + 2);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.v[b]);
      }
      base += n_t;
      __syncthreads();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFTMAX));
    // ===================== softmax: 64 keys of a row per thread =====================
    const int X = warp >> 3, half = (warp >> 2) & 1;                    // tile A, B; keys 0-63, 64-127
    const int row = tid & (BM - 1);
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lane_off + TS + HK * half, tp = ts + TP - TS + 64 * X - (HK / 2) * half;
    const uint32_t to = ts + TO - TS + 128 * X - HK * half;
    const int pair = 1 + 4 * X + (warp & 3);                            // named barrier of the rows' two warps
    bool ok = true;
    int base = 0;
    for (int i = 0;; ++i) {
      const int n_t = s_piece[i & 1].n_t;
      if (n_t < 0) break;
      bool here, row_ok;
      int lim;                                // keys that the row sees, from the piece's first one on
      {
        const Piece pc = read_piece(&s_piece[i & 1]);
        const int hv = pc.kh / maps, map = pc.kh - hv * maps;
        here = X == 0 || pc.left > BM;
        row_ok = X * BM + row < pc.left;
        int qi, head;
        query_of(a, pc.rem, row_ok ? X * BM + row : 0, qi, head);
        lim = (!row_ok ? 0 : a.causal ? max(0, pc.lim0 + qi) : pc.lim0) - pc.t_lo * BN;
        // ---- Q: a warp takes 16 rows, 8 beside each other, of which 4 lanes share one: a load touches 8 lines (with a
        // row per lane 32; the first product then waited 6000 clocks for Q) and a store of 8 lanes 128 bytes
        if (here) {
          constexpr int NC = DK / 32;         // 8-element chunks of a lane and row
          const int sub = lane >> 3, r0 = X * BM + 16 * (warp & 7) + (lane & 7);
          uint4 raw[2][NC];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const bool there = r0 + 8 * t < pc.left;
            query_of(a, pc.rem, there ? r0 + 8 * t : 0, qi, head);
            const uint16_t *src = static_cast<const uint16_t *>(a.q) + static_cast<int64_t>(pc.row0 + qi) * a.q_stride +
                                  static_cast<int64_t>(maps * (head + hv * G) + map) * a.dk;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const int d = 8 * (sub + 4 * c);
              raw[t][c] = there && d < a.dk ? __ldg(reinterpret_cast<const uint4 *>(src + d)) : make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            float mx = 0.f;
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              float v[8];
              few::unpack8(raw[t][c], a.bf16, v);
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                mx = max3(mx, fabsf(v[e]), fabsf(v[e + 1]));
                s2 = add2(s2, make_float2(v[e], v[e + 1]));
              }
            }
            float sum = s2.x + s2.y;
#pragma unroll
            for (int o = 8; o < 32; o <<= 1) {
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            // largest entry in [2^e, 2^(e + 1)) -> [2^12, 2^13); the scale's sign goes into q, a scale of 0 makes it 0.
            // (A row whose entries all lie below 2^-114 keeps fewer bits.)
            const int e = mx > 0.f ? max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -114) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(12 - e + 127) << 23) *
                             (a.scale_log2 > 0.f ? 1.f : a.scale_log2 < 0.f ? -1.f : 0.f);
            unsigned char *dst = smem + C::SQ + X * C::Q_BYTES + (2 * (warp & 7) + t) * 128 + (lane & 7) * 16;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              float v[8];
              few::unpack8(raw[t][c], a.bf16, v);
#pragma unroll
              for (int k = 0; k < 8; k += 2) {
                const float2 u = mul2(make_float2(v[k], v[k + 1]), make_float2(up, up * 0.0625f));
                v[k] = u.x;
                v[k + 1] = u.y;
              }
              // the order in which a code word unpacks: (0, 4), (1, 5), (2, 6), (3, 7)
              *reinterpret_cast<uint4 *>(dst + (sub + 4 * c) * 2048) =
                  make_uint4(few::half2_bits(v[0], v[4]), few::half2_bits(v[1], v[5]), few::half2_bits(v[2], v[6]),
                             few::half2_bits(v[3], v[7]));
            }
            if (sub == 0) {
              const float qs = sum * up * 0x1p-16f, ql = qs * 0x1p-8f;
              const __half h0 = __float2half_rn(qs);
              const __half h1 = __float2half_rn(qs - __half2float(h0));
              const __half h2 = __float2half_rn(qs - __half2float(h0) - __half2float(h1));
              const __half l0 = __float2half_rn(ql);
              const __half l1 = __float2half_rn(ql - __half2float(l0));
              const __half z = __float2half_rn(0.f);
              *reinterpret_cast<uint4 *>(dst + (DK / 8) * 2048) =
                  make_uint4(bits(__halves2half2(h0, h1)), bits(__halves2half2(h2, l0)), bits(__halves2half2(l1, z)), 0);
            } else if (sub == 1) {
              *reinterpret_cast<uint4 *>(dst + (DK / 8 + 1) * 2048) = make_uint4(0, 0, 0, 0);
            } else if (sub == 2) {
              reinterpret_cast<float *>(smem + C::SFX)[r0 + 8 * t] =
                  a.scale_log2 != 0.f
                      ? fmaxf(fabsf(a.scale_log2) * 4096.f * __uint_as_float(static_cast<uint32_t>(e + 127) << 23), 1e-37f)
                      : 1.f;
            }
          }
        }
      }
      tc::fence_async_smem();
      tc::named_sync(BAR_Q, 32 * (W_UNPACK + 1));

      const float fx = reinterpret_cast<const float *>(smem + C::SFX)[X * BM + row];    // x = fx s_t (score), fx > 0
      float R = -INFINITY, l = 0.f;
      const uint32_t ex = sbase + C::SROW + (X * 4 * BM + row) * 4;                     // [J & 1][half][row]
      const float2 fx2 = make_float2(fx, fx);
      int nvis = lim - HK * half;             // of the thread's keys of the tile, those that the row sees
      const int J0 = base;
      base += n_t;
      for (int J = J0; J < base; ++J, nvis -= BN) {
        if (ok) {
          ok = wait_warp(&bars.s[X], J & 1);
          // the tile's scales.  (Not K's own barrier: K of tile J + 2 may be there already, and a slow warp would
          // miss the phase.  Scales of J + 4 wait for scores that wait for this warp.)
          if (ok && here) ok = wait_warp(&bars.sc[J & 3], (J >> 2) & 1);
        }
        if (!here) {                          // no rows: the phases go on, no faster than with rows
          if (ok && J > J0) ok = wait_warp(&bars.pv[X][(J - 1) & 1], ((J - 1) >> 1) & 1);
          if (lane == 0) {
            tc::mbar_arrive(&bars.rd[X]);
            tc::mbar_arrive(&bars.p[X]);
          }
          continue;
        }
        if (!ok) {                            // a wait ran out: the row's other warp still meets this one
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
        const uint32_t sc = sbase + C::SSC + ((J & 3) * BN + HK * half) * 4;
#pragma unroll
        for (int k = 0; k < HK / 4; ++k) {
          const float4 s4 = few::lds4(sc + 16 * k);
          const float2 u = mul2(make_float2(y[4 * k], y[4 * k + 1]), make_float2(s4.x, s4.y));
          const float2 w = mul2(make_float2(y[4 * k + 2], y[4 * k + 3]), make_float2(s4.z, s4.w));
          y[4 * k] = u.x;
          y[4 * k + 1] = u.y;
          y[4 * k + 2] = w.x;
          y[4 * k + 3] = w.y;
        }
        if (__any_sync(0xffffffffu, nvis < HK)) {
#pragma unroll
          for (int k = 0; k < HK; ++k)
            if (k >= nvis) y[k] = -INFINITY;
        }
        float4 tau = few::lds4(sbase + C::STAU + (4 * (J & 3) + 2 * half) * 8);   // (tau, 2^-tau) of both 32 keys
        const uint32_t key_tau = sbase + C::SKTAU + ((J & 3) * BN + HK * half) * 8;
        const bool apart = tau.y == 0.f || tau.w == 0.f;
        if (apart) {                          // each key's tau goes into its score, whose factor it has to stand
          float un;
          asm("rcp.approx.f32 %0, %1;" : "=f"(un) : "f"(fx));
#pragma unroll
          for (int k = 0; k < HK; k += 2) {
            const float4 t4 = few::lds4(key_tau + 8 * k);
            y[k] = fmaf(t4.x, un, y[k]);
            y[k + 1] = fmaf(t4.z, un, y[k + 1]);
          }
          tau = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            m0 = max3(m0, y[32 * c + k], y[32 * c + k + 1]);
            m1 = max3(m1, y[32 * c + k + 2], y[32 * c + k + 3]);
          }
          top = fmaxf(top, fmaf(fmaxf(m0, m1), fx, c ? tau.z : tau.x));
        }
        // (two places in turn: the other thread may still be reading the last tile's)
        sts1(ex + (2 * (J & 1) + half) * BM * 4, top);
        tc::named_sync(pair, 64);
        top = fmaxf(top, lds1(ex + (2 * (J & 1) + (half ^ 1)) * BM * 4));
        const bool raise = top > R + RAISE, any = __any_sync(0xffffffffu, raise);
        const float f = raise ? exp2f(R - top) : 1.f;                   // 0 at the first raise
        if (raise) R = top;
        l *= f;
        const float Rs = R == -INFINITY ? 0.f : R;
        if (apart) {                          // the sum of weights key by key (tau's factor of 0 leaves them out below)
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < HK; k += 2) {
            const float4 t4 = few::lds4(key_tau + 8 * k);
            sum = fmaf(tc::ex2(fmaf(y[k], fx, -Rs)), t4.y, sum);
            sum = fmaf(tc::ex2(fmaf(y[k + 1], fx, -Rs)), t4.w, sum);
          }
          l += sum;
        }
        uint32_t p[HK / 2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float2 t2 = c ? make_float2(tau.z, tau.w) : make_float2(tau.x, tau.y);
          const float2 off = make_float2(t2.x - Rs, t2.x - Rs);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 16 * c; q < 16 * c + 16; ++q) {
            const float2 e = fma2(make_float2(y[2 * q], y[2 * q + 1]), fx2, off);
            const float2 w = make_float2(tc::ex2(e.x), tc::ex2(e.y));                   // masked: 0
            sum = add2(sum, w);
            p[q] = few::half2_bits(w.x, w.y);
          }
          l = fmaf(sum.x + sum.y, t2.y, l);
        }
        if (J > J0) {                         // only now must P and O stand still
          ok = wait_warp(&bars.pv[X][(J - 1) & 1], ((J - 1) >> 1) & 1);
          if (!ok) continue;
          tc::fence_after_sync();
          if (any) {
#pragma unroll 1
            for (int c = half * (DV / 2); c < (half + 1) * (DV / 2); c += 8) {
              uint32_t o[8];
              asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                           : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7])
                           : "r"(to + c));
              tc::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              st8(to + c, o);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) st8(tp + 8 * c, p + 8 * c);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars.p[X]);
      }
      // the last product has to be done before O is read
      if (ok && base > J0) {
        ok = wait_warp(&bars.pv[X][(base - 1) & 1], ((base - 1) >> 1) & 1);
        tc::fence_after_sync();
      }
      if (!ok) s_fail = 1;
      // ===================== epilogue: columns in the order of the code words, half of them per thread =====================
      if (here) {
        tc::named_sync(pair, 64);                                       // the last exchange was read
        sts1(ex + half * BM * 4, l);
        tc::named_sync(pair, 64);
        l += lds1(ex + (half ^ 1) * BM * 4);
      }
      const Piece pc = read_piece(&s_piece[i & 1]);
      const int hv = pc.kh / maps, map = pc.kh - hv * maps;
      const bool rows_part = a.diff || a.n_split > 1;
      // where row r (of 256) puts its values: the output, or its partial results (R, l, -, -, values)
      auto out_of = [&](int r) {
        int qi, head;
        query_of(a, pc.rem, r, qi, head);
        return static_cast<int64_t>(pc.row0 + qi) * a.n_heads + hv * G + head;
      };
      auto part_at = [&](int64_t at) {
        const int split = LINE ? 0 : static_cast<int>(blockIdx.x) / k_heads % a.n_split;
        return a.row_part + ((at * maps + map) * a.n_split + split) * (DV + 4);
      };
      // 64 bytes of each of the warp's rows (lane: row), values from dim d on, by way of shared memory (where Q was), so
      // that a store touches 8 lines: 4 lanes share a row.  Swizzled, so that neither side has bank conflicts.
      const uint32_t stage = sbase + C::SQ + X * C::Q_BYTES + (warp & 7) * 2048;
      auto put64 = [&](const uint32_t *w, int d) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) sts4(stage + lane * 64 + ((c ^ (lane >> 1)) & 3) * 16, w + 4 * c);
        __syncwarp();
        const int c = lane & 3, dim = d + c * (rows_part ? 4 : 8);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int rl = 8 * t + (lane >> 2), r = X * BM + 32 * (warp & 3) + rl;
          const float4 u = few::lds4(stage + rl * 64 + ((c ^ (rl >> 1)) & 3) * 16);
          if (r >= pc.left || dim >= a.dv) continue;
          const int64_t to_row = out_of(r);
          if (rows_part) *reinterpret_cast<float4 *>(part_at(to_row) + 4 + dim) = u;
          else *reinterpret_cast<float4 *>(static_cast<uint16_t *>(a.out) + to_row * a.dv + dim) = u;
        }
      };
      // 32 values of each row: times `inv` to the output, or as they are to the partial results
      auto put32 = [&](int d, const float *v, float inv) {
        uint32_t w[16];
        if (rows_part) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[16 * h + e]);
            put64(w, d + 16 * h);
          }
          return;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e] * inv, v[2 * e + 1] * inv);
          w[e] = a.bf16 ? *reinterpret_cast<const uint32_t *>(&h) : few::half2_bits(v[2 * e] * inv, v[2 * e + 1] * inv);
        }
        put64(w, d);
      };
      // (R, l) of the row to its partial results; 1 / l for the output (nothing visible: zeros; NaN stays NaN)
      auto put_sums = [&](float m, float sum) {
        if (rows_part && row_ok && half == 0)
          *reinterpret_cast<float4 *>(part_at(out_of(X * BM + row))) = make_float4(m, sum, 0.f, 0.f);
        return sum != 0.f ? 1.f / sum : 0.f;
      };
      const bool shared = LINE && pc.n_con > 1;
      // a shared item's partial: (R, l) [row], then the dims in fours [four][row]
      constexpr int SLOT = 2 * BM * (DV + 2);
      float *mine = a.part + static_cast<int64_t>(2 * blockIdx.x + pc.slot) * SLOT;
      const int at = X * BM + row;
      float inv = 0.f;
      if (here) {
        if (!shared) inv = put_sums(R, l);
        else if (half == 0) reinterpret_cast<float2 *>(mine)[at] = make_float2(R, l);
      }
      if (ok && here) {
#pragma unroll 1
        for (int c = half * (DV / 2); c < (half + 1) * (DV / 2); c += 32) {
          uint32_t o[32];
          if (base > J0) {
            tc::tmem_ld32(to + c, o);
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          }
          float v[32];                        // dims c ..: the columns are in the order of the code words
#pragma unroll
          for (int k = 0; k < 32; k += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[k + e] = __uint_as_float(o[k + 2 * e]);
              v[k + e + 4] = __uint_as_float(o[k + 2 * e + 1]);
            }
          if (shared) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              reinterpret_cast<float4 *>(mine + 4 * BM)[((c + k) / 4) * 2 * BM + at] =
                  make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          } else {
            put32(c, v, inv);
          }
        }
        tc::fence_before_sync();
      }
      if (shared) {
        tc::named_sync(BAR_SOFT, 32 * W_UNPACK);
        if (tid == 0) {
          s_last = few::arrive_one(a.counters + pc.c0) == pc.n_con - 1;
          if (s_last) a.counters[pc.c0] = 0;
        }
        tc::named_sync(BAR_SOFT, 32 * W_UNPACK);
        if (s_last && here) {
          auto part_of = [&](int c) {
            return a.part + static_cast<int64_t>(2 * (pc.c0 + c) + (c == 0 ? pc.slot0 : 0)) * SLOT;
          };
          float M = -INFINITY, sum = 0.f;
          for (int c = 0; c < pc.n_con; ++c) M = fmaxf(M, __ldcg(reinterpret_cast<const float2 *>(part_of(c)) + at).x);
          for (int c = 0; c < pc.n_con; ++c) {
            const float2 q = __ldcg(reinterpret_cast<const float2 *>(part_of(c)) + at);
            sum = fmaf(q.x == -INFINITY ? 0.f : exp2f(q.x - M), q.y, sum);
          }
          inv = put_sums(M, sum);
#pragma unroll 1
          for (int d = half * (DV / 2); d < (half + 1) * (DV / 2); d += 32) {
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0.f;
            for (int c = 0; c < pc.n_con; ++c) {
              const float *q = part_of(c);
              const float rc = __ldcg(reinterpret_cast<const float2 *>(q) + at).x;
              const float w = rc == -INFINITY ? 0.f : exp2f(rc - M);
#pragma unroll
              for (int f = 0; f < 8; ++f) {
                const float4 u = __ldcg(reinterpret_cast<const float4 *>(q + 4 * BM) + (d / 4 + f) * 2 * BM + at);
                v[4 * f] = fmaf(w, u.x, v[4 * f]);
                v[4 * f + 1] = fmaf(w, u.y, v[4 * f + 1]);
                v[4 * f + 2] = fmaf(w, u.z, v[4 * f + 2]);
                v[4 * f + 3] = fmaf(w, u.w, v[4 * f + 3]);
              }
            }
            put32(d, v, inv);
          }
        }
      }
      __syncthreads();
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (row >= a.n_rows) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int maps = a.diff ? 2 : 1;
  constexpr int N = DV / 32;                  // values per lane: dims N lane ..
  const bool in = N * lane < a.dv;
  auto part_of = [&](int m, int k) {
    return a.row_part + (((row * a.n_heads + head) * maps + m) * static_cast<int64_t>(a.n_split) + k) * (DV + 4);
  };
  auto load = [&](const float *p, float2 &rl, float2 *v) {
    rl = __ldcg(reinterpret_cast<const float2 *>(p));
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      v[i] = in ? __ldcg(reinterpret_cast<const float2 *>(p + 4 + N * lane) + i) : make_float2(0.f, 0.f);
  };
  // first parts of both maps, on their way beside the search (a row of no sequence reads what is there, unused)
  float2 rl[2], v[2][N / 2];
  load(part_of(0, 0), rl[0], v[0]);
  if (maps == 2) load(part_of(1, 0), rl[1], v[1]);
  // the row's sequence; rows of none stay as they are
  int lo = 0, hi = a.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.q_start[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  const int row_lo = a.q_start[lo], row_hi = a.q_start[lo + 1];
  if (row_lo < 0 || row_hi > a.n_rows || row < row_lo || row >= row_hi) return;
  float y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = 0.f;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    if (m == maps) break;
    float M = rl[m].x;
    for (int k = 1; k < a.n_split; ++k) M = fmaxf(M, __ldcg(part_of(m, k)));
    float l = 0.f, o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.f;
    auto add = [&](const float2 &q, const float2 *u) {
      const float w = q.x == -INFINITY ? 0.f : exp2f(q.x - M);
      l = fmaf(w, q.y, l);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        o[i] = fmaf(w, u[i / 2].x, o[i]);
        o[i + 1] = fmaf(w, u[i / 2].y, o[i + 1]);
      }
    };
    add(rl[m], v[m]);
#pragma unroll 4
    for (int k = 1; k < a.n_split; ++k) {
      float2 q, u[N / 2];
      load(part_of(m, k), q, u);
      add(q, u);
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
    const float r = diff_factor(a, ss);
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
  const int k_heads = (a.diff ? 2 : 1) * a.n_kv_heads;
  auto kern = a.line ? prefill_kernel<DK, DV, true> : prefill_kernel<DK, DV, false>;
  cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kern), C::TOTAL);
  if (e != cudaSuccess) return e;
  const unsigned grid = a.line ? static_cast<unsigned>(max_ctas(1)) : static_cast<unsigned>(a.n_tiles) * a.n_split * k_heads;
  e = launch_beside(kern, grid, pre::NT, C::TOTAL, s, a);
  if (e != cudaSuccess || (a.n_split == 1 && !a.diff)) return e;
  return launch_beside(prefill_merge_kernel<DV>, static_cast<unsigned>((a.n_rows * a.n_heads + 7) / 8), 256, 0, s, a);
}

}  // namespace p4
}  // namespace tq
