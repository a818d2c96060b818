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
// Split of the work, two ways:
// - LINE, where there are many (row tile, KV head) items: their key tiles, with ITEM_COST
//   empty ones before each item, form one line that is cut into equal shares, one per
//   SM, from the device's lengths.  A CTA's first and last item may be shared with
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
constexpr int ITEM_COST = 4;                      // key tiles' worth of time that an item costs besides its keys (8 us)
constexpr int NT = 768;
constexpr int W_UNPACK = 16, W_MMA = 20, W_NEXT = 21;      // first warps of the roles after the softmax
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
  static constexpr uint32_t STAU = SSC + 4 * BN * 4;           // [j & 3][32 keys] (tau, 2^-tau)
  static constexpr uint32_t SROW = STAU + 4 * 4 * 8;           // [tile][half][row] exchange between a row's threads
  static constexpr uint32_t TOTAL = SROW + 2 * 2 * BM * 8;
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
// found the phase open slept on past its end, on every step of the chain score - softmax - product (WAIT_FIG).
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity) {
  const uint32_t at = tc::smem_u32(bar);
  for (int it = 0; it < (1 << 19); ++it) {
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

__device__ __forceinline__ void sts1(uint32_t at, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}
__device__ __forceinline__ float lds1(uint32_t at) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
  return x;
}

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }

// A piece of an item: key tiles t_lo .. t_lo + n_t - 1 of 256 rows of one sequence and K head.
struct Piece {
  int seq, tile, kh;        // tile: which 256 rows of the sequence
  int t_lo, n_t;            // n_t < 0: no more pieces
  int c0, n_con, slot;      // LINE: the CTAs that share the item, c0 .. c0 + n_con - 1; where this partial goes
  int slot0;                // ... and where that of c0 is
};

// Rows and key tiles of one 256-row tile.
struct Tile {
  int r0, rows_all, kv_hi, tiles;
};
__device__ __forceinline__ Tile tile_of(const AttnArgs &a, const few::SeqWork &w, int tile) {
  Tile t;
  t.rows_all = w.rows * a.group;
  t.r0 = tile * 2 * BM;
  const int last = min(t.rows_all, t.r0 + 2 * BM) - 1;
  t.kv_hi = a.causal ? max(0, w.len - w.rows + last / a.group + 1) : w.len;
  t.tiles = (t.kv_hi + BN - 1) / BN;
  return t;
}
__device__ __forceinline__ int tiles_of(const AttnArgs &a, const few::SeqWork &w) {
  return static_cast<int>((static_cast<long long>(w.rows) * a.group + 2 * BM - 1) / (2 * BM));
}

// A piece, read anew (what only begin and end of its work need is not kept in registers through the loop).
__device__ __forceinline__ Piece read_piece(const Piece *p) {
  const volatile int *q = reinterpret_cast<const volatile int *>(p);
  return {q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7], q[8]};
}

// Row tiles of a piece that have rows.
__device__ __forceinline__ int row_tiles(const AttnArgs &a, const Piece &p) {
  const few::SeqWork w = few::seq_work<1>(a, p.seq, false);
  return w.rows * a.group - p.tile * 2 * BM > BM ? 2 : 1;
}

// One CTA's walk along the line (one thread).
struct Walk {
  long long cur, end, pre;  // units of the line; pre: where the current item begins
  long long share0, total, n_work;
  int seq, tile, kh;
};
__device__ inline Piece next_piece(const AttnArgs &a, Walk &w) {
  Piece p = {0, 0, 0, 0, -1, 0, 1, 0, 0};
  const int k_heads = (a.diff ? 2 : 1) * a.n_kv_heads;
  while (w.cur < w.end) {
    const few::SeqWork sw = few::seq_work<1>(a, w.seq, false);
    if (w.tile >= tiles_of(a, sw)) {
      ++w.seq;
      w.tile = w.kh = 0;
      continue;
    }
    const Tile t = tile_of(a, sw, w.tile);
    const int per = t.tiles + ITEM_COST;
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
    if (u1 <= u0 && !(t.tiles == 0 && stop == per)) continue;
    p.seq = w.seq;
    p.tile = w.tile;
    p.kh = w.kh;
    p.t_lo = u0;
    p.n_t = u1 - u0;
    if (t.tiles > 0) {
      const long long ia = w.pre + ITEM_COST;
      auto owner = [&](long long x) { return static_cast<int>(((x + 1) * w.n_work - 1) / w.total); };
      p.c0 = owner(ia);
      p.n_con = owner(ia + t.tiles - 1) - p.c0 + 1;
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
  __shared__ long long s_sum[NT / 32];

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int maps = a.diff ? 2 : 1, k_heads = maps * a.n_kv_heads, G = a.group;

  // ---- the first piece
  {
    // in the split form heads fastest, row tiles slowest and from the last one down (under a causal mask the
    // longest first)
    const int want = LINE ? 0 : a.n_tiles - 1 - static_cast<int>(blockIdx.x) / k_heads / a.n_split;
    if (tid == 0) {
      s_fail = 0;
      s_piece[0].n_t = s_piece[1].n_t = -1;
      s_piece[0].seq = -1;
    }
    // Line (or row tiles) of the sequences s0 .. before `at`; a second pass finds the share's begin.
    long long total = 0, begin = 0, end = 0, n_work = 0;
    for (int pass = 0; pass < (LINE ? 2 : 1); ++pass) {
      long long at = 0;
      if (pass == 1) {
        n_work = min(static_cast<long long>(gridDim.x), total);
        if (blockIdx.x >= n_work) break;
        begin = blockIdx.x * total / n_work;
        end = (blockIdx.x + 1) * total / n_work;
      }
      for (int s0 = 0; s0 < a.n_seq; s0 += NT) {
        const int s = s0 + tid;
        long long v = 0;
        if (s < a.n_seq) {
          const few::SeqWork w = few::seq_work<1>(a, s, pass == 0 && blockIdx.x == 0);
          const int n = tiles_of(a, w);
          if (!LINE) v = n;
          else
            for (int i = 0; i < n; ++i) v += tile_of(a, w, i).tiles + ITEM_COST;
          if (LINE) v *= k_heads;
        }
        long long x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) s_sum[warp] = x;
        __syncthreads();
        long long all = 0;
        for (int w = 0; w < NT / 32; ++w) {
          if (w == warp) x += all;
          all += s_sum[w];
        }
        x += at;
        at += all;
        if (!LINE && v > 0 && x - v <= want && want < x) {
          const few::SeqWork w = few::seq_work<1>(a, s, false);
          Piece p = {s, static_cast<int>(want - (x - v)), static_cast<int>(blockIdx.x) % k_heads, 0, 0, 0, 1, 0, 0};
          const int tiles = tile_of(a, w, p.tile).tiles, split = static_cast<int>(blockIdx.x) / k_heads % a.n_split;
          p.t_lo = static_cast<int>(static_cast<long long>(tiles) * split / a.n_split);
          p.n_t = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / a.n_split) - p.t_lo;
          s_piece[0] = p;
        }
        if (LINE && pass == 1 && v > 0 && x - v <= begin && begin < x) {
          const few::SeqWork w = few::seq_work<1>(a, s, false);
          Walk k = {begin, end, x - v, begin, total, n_work, s, 0, 0};
          for (;;) {                          // (begin < x: the loop ends at one of the sequence's tiles)
            const long long t = static_cast<long long>(tile_of(a, w, k.tile).tiles + ITEM_COST) * k_heads;
            if (begin < k.pre + t) break;
            k.pre += t;
            ++k.tile;
          }
          const int per = tile_of(a, w, k.tile).tiles + ITEM_COST;
          k.kh = static_cast<int>((begin - k.pre) / per);
          k.pre += static_cast<long long>(k.kh) * per;
          s_piece[0] = next_piece(a, k);
          s_walk = k;
        }
      }
      if (pass == 0) total = at;
    }
    __syncthreads();
  }
  if (s_piece[0].n_t < 0) return;             // no work for this CTA

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
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
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
        const bool two = row_tiles(a, s_piece[i & 1]) == 2;
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
                mma_ta(tm + TO + 128 * x, tm + TP + 64 * x + 8 * ks, v + ((ks * 2 * C::VC * 128) >> 4), ID_PV, j > 0 || ks > 0);
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
                    tc::mma_f16(tm + TS, q0 + x * (C::Q_BYTES >> 4) + ((ks * 4096) >> 4), k + ((ks * 256) >> 4), ID_S, ks > 0);
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
      const int kv_hi = tile_of(a, few::seq_work<1>(a, pc.seq, false), pc.tile).kv_hi;
      const int32_t *table = a.block_table + static_cast<int64_t>(pc.seq) * a.max_pages;
      auto page_of = [&](int j) {
        const int t = (t_lo + j) * BN + key;
        return j < n_t && t < kv_hi ? __ldg(table + (t >> a.page_shift)) : -2;       // -2: no such key
      };
      uint4 kraw[DK / 32], vraw[DV / 32];
      uint32_t ksm = 0, vsm = 0;              // (scale, offset) pairs
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
        for (int c = 0; c < DK / 32; ++c) kraw[c] = make_uint4(0, 0, 0, 0);
        if (rw >= 0) {
          // (row of K head kh: K planes have `maps` heads per V head)
          const int64_t in = rw & mask, k = (rw - in) * maps + static_cast<int64_t>(kh) * (mask + 1) + in;
          const uint4 *p = reinterpret_cast<const uint4 *>(a.k_codes + k * (DK / 2));
          ksm = __ldg(reinterpret_cast<const uint32_t *>(a.k_scales) + k);
#pragma unroll
          for (int c = 0; c < DK / 32; ++c) kraw[c] = __ldg(p + c);
        }
      };
      auto load_v = [&](int64_t rw) {
        vsm = 0;
#pragma unroll
        for (int c = 0; c < DV / 32; ++c) vraw[c] = make_uint4(0, 0, 0, 0);
        if (rw >= 0) {
          const int64_t v = rw + static_cast<int64_t>(hv) * (mask + 1);
          const uint4 *p = reinterpret_cast<const uint4 *>(a.v_codes + v * (DV / 2));
          vsm = __ldg(reinterpret_cast<const uint32_t *>(a.v_scales) + v);
#pragma unroll
          for (int c = 0; c < DV / 32; ++c) vraw[c] = __ldg(p + c);
        }
      };
      int64_t rw = row_of(0, page_of(0));
      load_k(rw);
      load_v(rw);
      int page = page_of(1);
      for (int j = 0; j < n_t; ++j) {
        const int J = base + j, b = J & 1;
        if (J >= 2) ok = wait_warp(&bars.kf[b], ((J - 2) >> 1) & 1);    // the K buffer's last users
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
          reinterpret_cast<float2 *>(smem + C::STAU)[(J & 3) * 4 + (warp - W_UNPACK)] = make_float2(static_cast<float>(e), dn);
        {
          float2 sm = __half22float2(as_half2(ksm));
          float off = __fdividef(sm.y, sm.x);
          uint32_t keep = 0xffffffffu;
          if (!(fabsf(off) < 0x1p19f)) {      // (a scale of 0 too) constant row: its offset alone
            keep = 0;
            off = sm.y > 0.f ? 0x1p16f : sm.y < 0.f ? -0x1p16f : 0.f;
            sm.x = sm.y != 0.f ? fabsf(sm.y) * 0x1p-16f : 1.f;
          }
          const __half hi = __float2half_rn(off * 0.0625f);
          const __half lo = __float2half_rn(off * 0.0625f - __half2float(hi));
          *reinterpret_cast<uint4 *>(kd + (DK / 8) * 128) =
              make_uint4(bits(__halves2half2(hi, hi)), bits(__halves2half2(hi, lo)),
                         bits(__halves2half2(lo, __float2half_rn(0.f))), 0);
          reinterpret_cast<float *>(smem + C::SSC)[(J & 3) * BN + key] = sm.x;
#pragma unroll
          for (int c4 = 0; c4 < DK / 32; ++c4) {
            const uint32_t w[4] = {kraw[c4].x & keep, kraw[c4].y & keep, kraw[c4].z & keep, kraw[c4].w & keep};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t u = w[c] >> 8;
              *reinterpret_cast<uint4 *>(kd + (4 * c4 + c) * 128) =
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
        rw = row_of(j + 1, page);
        load_k(rw);                           // on its way while the values are unpacked
        if (J >= 2)                           // the V buffer's last users
          for (int x = 0; x < 2 && ok; ++x) ok = wait_warp(&bars.pv[x][b], ((J - 2) >> 1) & 1);
        if (!ok) { s_fail = 1; break; }
        {
          const __half2 vs = __float2half2_rn(vsc.x * dn), vm = __float2half2_rn(vsc.y * dn);
          const __half2 k1024 = as_half2(0x64006400u), k16 = as_half2(0x2c002c00u), k64 = as_half2(0xd400d400u);
#pragma unroll
          for (int c4 = 0; c4 < DV / 32; ++c4) {
            const uint32_t w[4] = {vraw[c4].x, vraw[c4].y, vraw[c4].z, vraw[c4].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t u = w[c] >> 8;
              // 1024 + code, and 1024 + 16 code
              const __half2 c0 = __hsub2(as_half2((w[c] & 0x000f000fu) | 0x64006400u), k1024);
              const __half2 c1 = __hfma2(as_half2((w[c] & 0x00f000f0u) | 0x64006400u), k16, k64);
              const __half2 c2 = __hsub2(as_half2((u & 0x000f000fu) | 0x64006400u), k1024);
              const __half2 c3 = __hfma2(as_half2((u & 0x00f000f0u) | 0x64006400u), k16, k64);
              *reinterpret_cast<uint4 *>(vd + (4 * c4 + c) * 128) =
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
      float fx = 1.f;                         // x = fx s_t (score), fx > 0
      {
      const Piece pc = read_piece(&s_piece[i & 1]);
      const few::SeqWork sw = few::seq_work<1>(a, pc.seq, false);
      const Tile tl = tile_of(a, sw, pc.tile);
      const int hv = pc.kh / maps, map = pc.kh - hv * maps;
      const int r = tl.r0 + X * BM + row;     // row of the sequence
      here = X == 0 || tl.rows_all - tl.r0 > BM;
      row_ok = r < tl.rows_all;
      const int qi = row_ok ? r / G : 0, head = hv * G + (row_ok ? r - qi * G : 0);
      const int64_t out_row = static_cast<int64_t>(sw.row0) + qi;
      lim = (!row_ok ? 0 : a.causal ? max(0, sw.len - sw.rows + qi + 1) : sw.len) - pc.t_lo * BN;
      // ---- Q: half of the row's dims per thread
      if (here) {
        constexpr int NC = DK / 16;           // 8-element chunks of a thread
        const uint16_t *src = static_cast<const uint16_t *>(a.q) + out_row * a.q_stride +
                              static_cast<int64_t>(maps * head + map) * a.dk;
        float2 *ex = reinterpret_cast<float2 *>(smem + C::SROW) + X * 2 * BM;           // [half][row]: (max, sum)
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
        ex[half * BM + row] = make_float2(mx, sum);
        tc::named_sync(pair, 64);
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
          for (int k = 0; k < 8; ++k) v[k] = v[k] * s1 * s2 * ((k & 1) ? 0.0625f : 1.f);
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
        tc::named_sync(pair, 64);             // the exchange is free for the maxima
      }
      }
      tc::fence_async_smem();
      tc::named_sync(BAR_Q, 32 * (W_UNPACK + 1));

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
        const float4 tau = few::lds4(sbase + C::STAU + (4 * (J & 3) + 2 * half) * 8);   // (tau, 2^-tau) of both 32 keys
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
        if (J > J0) {                         // P and O stand still
          ok = wait_warp(&bars.pv[X][(J - 1) & 1], ((J - 1) >> 1) & 1);
          if (!ok) continue;
          tc::fence_after_sync();
        }
        const bool raise = top > R + RAISE;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? exp2f(R - top) : 1.f;                 // 0 at the first raise
          if (raise) R = top;
          l *= f;
          if (J > J0) {
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
        const float Rs = R == -INFINITY ? 0.f : R;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float2 t2 = c ? make_float2(tau.z, tau.w) : make_float2(tau.x, tau.y);
          const float2 off = make_float2(t2.x - Rs, t2.x - Rs);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const int k = 32 * c + 16 * h + 2 * q;
              const float2 e = fma2(make_float2(y[k], y[k + 1]), fx2, off);
              const float2 w = make_float2(tc::ex2(e.x), tc::ex2(e.y));                 // masked: 0
              sum = add2(sum, w);
              p[q] = few::half2_bits(w.x, w.y);
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
      const few::SeqWork sw = few::seq_work<1>(a, pc.seq, false);
      const int hv = pc.kh / maps, map = pc.kh - hv * maps, r = pc.tile * 2 * BM + X * BM + row;
      const int qi = row_ok ? r / G : 0, head = hv * G + (row_ok ? r - qi * G : 0);
      const int64_t out_row = static_cast<int64_t>(sw.row0) + qi;
      // 8 dims of the row: values times `inv` to the output, or as they are to the rows' partial results
      const bool rows_part = a.diff || a.n_split > 1;
      float *part = a.row_part + (((out_row * a.n_heads + head) * maps + map) * a.n_split +
                                  (LINE ? 0 : static_cast<int>(blockIdx.x) / k_heads % a.n_split)) * (DV + 4);
      auto put = [&](int d, const float *v, float inv) {
        if (!row_ok || d >= a.dv) return;
        if (rows_part) {
          *reinterpret_cast<float4 *>(part + 4 + d) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4 *>(part + 8 + d) = make_float4(v[4], v[5], v[6], v[7]);
          return;
        }
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
      };
      // (R, l) of the row to its partial results; 1 / l for the output (nothing visible: zeros; NaN stays NaN)
      auto put_sums = [&](float m, float sum) {
        if (rows_part && row_ok && half == 0) *reinterpret_cast<float4 *>(part) = make_float4(m, sum, 0.f, 0.f);
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
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float v[8];                                                  // dims c + 8 g ..
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[e] = __uint_as_float(o[8 * g + 2 * e]);
              v[e + 4] = __uint_as_float(o[8 * g + 2 * e + 1]);
            }
            const int d = c + 8 * g;
            if (shared) {
              float4 *q = reinterpret_cast<float4 *>(mine + 4 * BM) + (d / 4) * 2 * BM + at;
              q[0] = make_float4(v[0], v[1], v[2], v[3]);
              q[2 * BM] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
              put(d, v, inv);
            }
          }
        }
        tc::fence_before_sync();
      }
      if (shared) {
        __threadfence();
        tc::named_sync(BAR_SOFT, 32 * W_UNPACK);
        if (tid == 0) {
          s_last = atomicAdd(a.counters + pc.c0, 1) == pc.n_con - 1;
          if (s_last) a.counters[pc.c0] = 0;
        }
        tc::named_sync(BAR_SOFT, 32 * W_UNPACK);
        if (s_last && here) {
          __threadfence();
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
          for (int d = half * (DV / 2); d < (half + 1) * (DV / 2); d += 16) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = 0.f;
            for (int c = 0; c < pc.n_con; ++c) {
              const float *q = part_of(c);
              const float rc = __ldcg(reinterpret_cast<const float2 *>(q) + at).x;
              const float w = rc == -INFINITY ? 0.f : exp2f(rc - M);
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const float4 u = __ldcg(reinterpret_cast<const float4 *>(q + 4 * BM) + (d / 4 + f) * 2 * BM + at);
                v[4 * f] = fmaf(w, u.x, v[4 * f]);
                v[4 * f + 1] = fmaf(w, u.y, v[4 * f + 1]);
                v[4 * f + 2] = fmaf(w, u.z, v[4 * f + 2]);
                v[4 * f + 3] = fmaf(w, u.w, v[4 * f + 3]);
              }
            }
            put(d, v, inv);
            put(d + 8, v + 8, inv);
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
    const float *part = a.row_part + ((row * a.n_heads + head) * maps + m) * static_cast<int64_t>(a.n_split) * (DV + 4);
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
  const int k_heads = (a.diff ? 2 : 1) * a.n_kv_heads;
  auto kern = a.line ? prefill_kernel<DK, DV, true> : prefill_kernel<DK, DV, false>;
  cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kern), C::TOTAL);
  if (e != cudaSuccess) return e;
  const unsigned grid = a.line ? static_cast<unsigned>(sm_count()) : static_cast<unsigned>(a.n_tiles) * a.n_split * k_heads;
  kern<<<grid, pre::NT, C::TOTAL, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || (a.n_split == 1 && !a.diff)) return e;
  prefill_merge_kernel<DV><<<static_cast<unsigned>((a.n_rows * a.n_heads + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace p4
}  // namespace tq
