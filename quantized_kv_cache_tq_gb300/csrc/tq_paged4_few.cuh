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
//   stages: it waits for its own copies only, and no CTA barrier stands in the
//   loop.  (Bulk copies were measured too: issuing four of them per tile from one
//   lane takes more instructions than ten cp.async of the whole warp.)  Rows are
//   swizzled by 16-byte chunks (chunk_at), so that the copies, the 16-byte reads of K
//   rows and the transposing matrix reads of V rows all spread over the banks.
// - Codes become operands with one AND: (w & 0x000f000f) read as two binary16
//   values is the subnormal pair code 2^-24, (w & 0x00f000f0) is code 2^-20; the
//   powers of two are exact and go into q (2^-4 on the second kind) and into the
//   output (2^24, 2^20).  Eight codes cost four ANDs and one shift.  The value
//   operand wants neighbouring keys in one register: a transposing ldmatrix over
//   16-bit units (four codes) delivers them so.
// - q is scaled by a power of two per column, so that its binary16 form is exact
//   for binary16 and bfloat16 inputs down to 2^-23 of the column's largest entry
//   (smaller ones lose low bits below that).  Scores are thus exact up to fp32
//   accumulation.
// - The value weights p_t s_t are rounded to binary16 (relative 2^-11, an eighth
//   of bfloat16's rounding of the output): R is a running maximum of
//   x_t + exponent(s_t), so the largest weight lies in [1, 2^13] whatever the
//   scales, and sums of p_t and p_t m_t stay in fp32.  R is raised only when it
//   would grow by more than 2^12 (the sums are rescaled then).
// - Codes count from a row's smallest value, so with w the rounded weight, sum w c
//   + sum p m would carry the rounding of w times the whole range of the row.  The
//   sum taken is sum w (c - c0) + sum p (m + s c0) with c0 = clamp(-m / s, 0, 15)
//   per row, the code that stands for 0: the rounding then meets the values
//   themselves.
// - Binary16 outputs (FINE) take two steps more, since the above would cost them half
//   as much again as their own rounding: what a weight's rounding leaves goes into a
//   second product, and the value operand is code - 8 (see low_code).  Output error
//   over 48000 keys, relative: 1.99e-4, that of the output's own rounding, against
//   2.25e-4 with the second product alone and about 2.9e-4 with neither.  Time of 40
//   ragged sequences 165 us, against 148 with the second product alone and 136 in
//   bfloat16; of one sequence of 32768 keys 19.1, 18.1 and 17.3 us.
// Measured (8 KV heads of 128, 4 query heads each): 40 ragged sequences of up to 32768
// keys 135.5 us in bfloat16, 5.48 TB/s.  With all CTAs reading, two per SM, the memory
// is what bounds it, and the pair of a CTA's SM ends up to 20 us later than the other.
// One sequence of 900 keys 10.1 us, of one key 6.1: the launch, the lengths, the page,
// the row, the merge are a chain of some eight trips to L2 or memory.
//
// Split of the work.  An item is a (sequence, V head, column chunk), its keys come
// in units of 64.  Nothing about lengths is needed on the host: every CTA works its
// share out from the device's lengths, so a captured graph follows them.
// - Few items of like length: each is cut into as many pieces as there are CTAs per
//   item, and a CTA has one piece.
// - Else the items' units form one line that is cut into equal shares, one per CTA,
//   however ragged the batch is.  Taking up an item costs a CTA about what SETUP
//   units do (measured: 4 to 5 us, against 0.5 us per unit with all CTAs reading), so
//   every item begins with that many empty units: short sequences then do not pile
//   up on one CTA (40 ragged sequences: the CTAs ended between 106 and 171 us
//   without them).
// An item that several CTAs share leaves partial results (R, sums, values) in the
// workspace, a CTA's first and last item at most, and the last CTA to arrive merges
// them: in the order of the CTAs, so that a repeated call gives the same bits.
#pragma once

#include <math.h>

#include "tq_common.cuh"
#include "tq_paged4.cuh"
#include "tq_tc.cuh"

namespace tq {
namespace p4 {

constexpr float RAISE = 12.f;         // growth of the maximum (log2) that rescales
constexpr int UNIT = 64;              // keys per unit of work
constexpr int TILE = 32;              // keys per warp tile
constexpr int MIN_PIECE = 4;          // units of a piece at least: one tile for each of eight warps
constexpr int SETUP = 8;              // units' worth of work that an item costs besides its keys

// MAPS = 1: NT tiles of eight columns read K head hv.  MAPS = 2, differential
// attention: one tile, columns 0 .. 3 of map 0 and 4 .. 7 of map 1 for the same four
// (row, head) pairs.  Its scores add up both maps' products, each map's query
// fragments holding zeros in the other's columns, so that everything after them --
// softmax, weights, and the V rows, read once for both maps -- is that of one tile.
template <int DK, int DV, int NT, int MAPS>
struct FewCfg {
  static constexpr int KS = DK / 16;                      // k steps of the scores
  static constexpr int MT = DV / 16;                      // m tiles of the values
  static constexpr int NW = 8;                            // warps
  static constexpr int THREADS = NW * 32;
  static constexpr int KW = DK / 32;                      // words of a K row per lane
  static constexpr int COLS = MAPS == 2 ? 4 : 8 * NT;     // (row, head) columns per item
  static constexpr int NC = 8 * NT;                       // columns incl. maps
  // per SM: two where value accumulators and query fragments leave room in 128 registers a thread
  static constexpr int CTAS = NT * (4 * MT + 2 * KS * MAPS) <= (DK == 128 && MAPS == 2 ? 64 : 48) ? 2 : 1;
  // one stage: K rows [map][key], V rows [key], scale pairs [K maps, V][key]
  static constexpr int K_BYTES = TILE * DK / 2;
  static constexpr int V_BYTES = TILE * DV / 2;
  static constexpr int SC = MAPS * K_BYTES + V_BYTES;
  static constexpr int STAGE = SC + (MAPS + 1) * TILE * 4;
  static constexpr int PREP = TILE * (24 + 8 * MAPS);     // a warp's unpacked scales of one tile
  static constexpr int MERGE = NW * NT * MT * 512 + NW * NC * 12 + NC * 16;  // CTA merge, in the same place
  static constexpr int BUDGET = (CTAS == 2 ? 111 : 222) * 1024;
  static constexpr int FIT = (BUDGET - NW * PREP) / (NW * STAGE);
  static constexpr int STAGES = FIT < 2 ? 2 : (FIT > 4 ? 4 : FIT);
  static constexpr int RING = NW * (STAGES * STAGE + PREP);
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  // a partial result: (R, l, z) of every column, then the value fragments
  static constexpr int PART = 4 * NC + NT * MT * 128;
  // The grid: all CTAs that the SMs hold, as far as the merge of an item that every one of them shares finds room in
  // shared memory (a weight and two sums per CTA and column, and the teams' sums).  At 152 SMs every shape has room.
  static constexpr int merge_bytes(int ctas) { return ctas * NC * 12 + THREADS * 16; }
  static constexpr int grid(int sms) {
    const int room = (SMEM - THREADS * 16) / (NC * 12), fit = room < kMaxCtas ? room : kMaxCtas;
    return sms < (fit + CTAS - 1) / CTAS ? sms * CTAS : fit;
  }
};

namespace few {

template <int N>
struct Int {
  static constexpr int value = N;
};

__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// without a size: all 4 / 16 bytes
__device__ __forceinline__ void cp4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Byte offset of 16-byte chunk c of row r in a tile of rows of D codes: lines of 128 bytes hold 8 / CH rows
// of CH chunks, and a line's chunks are turned by its number, so that one chunk of 8 neighbouring rows
// falls on 8 different places.
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
  constexpr int CH = D / 32, RL = 8 / CH;
  return (r / RL) * 128 + ((((r % RL) * CH + c) ^ ((r / RL) % CH)) * 16);
}

// Two 8 x 8 matrices of 16-bit units per pair of registers, transposed: lane (g, t) gets column g of rows 2t, 2t + 1.
__device__ __forceinline__ void ldsm4t(uint32_t *r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes in bits 0 .. 3 (low) or 4 .. 7 (high) of both 16-bit halves as binary16 pairs: code 2^-24, code 2^-20, or (FINE)
// code - 8.  The tensor cores cut their sums off below 2^-24 of the largest term, always downwards, so a sum of codes
// whose mean is later taken off again is short by some 10^-6 of that mean.
template <bool FINE>
__device__ __forceinline__ uint32_t low_code(uint32_t x) {
  x &= 0x000f000fu;
  if (!FINE) return x;
  x |= 0x64006400u;                           // 1024 + code
  const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), __float2half2_rn(1032.f));
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool FINE>
__device__ __forceinline__ uint32_t high_code(uint32_t x) {
  x &= 0x00f000f0u;
  if (!FINE) return x;
  x |= 0x64006400u;                           // 1024 + 16 code
  const __half2 h = __hfma2(*reinterpret_cast<const __half2 *>(&x), __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
  return *reinterpret_cast<const uint32_t *>(&h);
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

// 8 elements of 16 bits as floats
__device__ __forceinline__ void unpack8(const uint4 &u, int bf16, float *x) {
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

__device__ __forceinline__ void sts4(uint32_t at, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
__device__ __forceinline__ void sts2(uint32_t at, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(at), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ float2 lds2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ float4 lds4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

// A sequence as the work line sees it.
struct SeqWork {
  int len;            // cells attended
  int row0, rows;     // its query rows
  int chunks;         // column chunks per V head
  long long units;    // per item
  long long items;    // (below 2^31, checked on the host)
};

// Arrival of a CTA whose threads have met at a barrier: what they wrote is visible to the CTAs that arrive later,
// and what earlier ones wrote to this CTA behind its next barrier.  (Fences of all threads around a plain atomic
// take 0.4 to 0.6 us more per call.)
__device__ __forceinline__ int arrive_one(int32_t *counter) {
  int r;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(r) : "l"(counter) : "memory");
  return r;
}

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

// Place of this thread's sequence on the line, which stands at `line` and `item` before sequence s0 (one
// sequence per thread): units [lo, hi) with SETUP ones per item, first item `first`.  Moves `line` and `item`
// past all of them.
struct Scan {
  long long line, item;
};
template <int COLS, int NW>
__device__ __forceinline__ void scan_chunk(const AttnArgs &a, int s0, Scan *sums, bool report, Scan &at, long long &lo,
                                           long long &hi, long long &first, int &units) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Scan v = {0, 0};
  if (s0 + tid < a.n_seq) {
    const SeqWork w = seq_work<COLS>(a, s0 + tid, report);
    if (w.units > 0) v = {(w.units + SETUP) * w.items, w.items};
    if (w.items > 0) units = max(units, static_cast<int>(w.units));
  }
  Scan x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y0 = __shfl_up_sync(0xffffffffu, x.line, o), y1 = __shfl_up_sync(0xffffffffu, x.item, o);
    if (lane >= o) {
      x.line += y0;
      x.item += y1;
    }
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  Scan all = {0, 0};
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w == warp) {
      x.line += all.line;
      x.item += all.item;
    }
    all.line += sums[w].line;
    all.item += sums[w].item;
  }
  lo = at.line + x.line - v.line;
  hi = at.line + x.line;
  first = at.item + x.item - v.item;
  at.line += all.line;
  at.item += all.item;
}

}  // namespace few

template <int DK, int DV, int NT, int MAPS, bool FINE>
__global__ void __launch_bounds__(FewCfg<DK, DV, NT, MAPS>::THREADS, FewCfg<DK, DV, NT, MAPS>::CTAS)
    few_kernel(const AttnArgs a) {
  using C = FewCfg<DK, DV, NT, MAPS>;
  using namespace few;
  constexpr int NW = C::NW, KW = C::KW, MT = C::MT, NC = C::NC, COLS = C::COLS;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Scan s_scan[NW];
  __shared__ int s_longest[NW];
  __shared__ float s_lz[NC][2];               // sums of the item's columns
  __shared__ long long s_pre;
  __shared__ int s_seq, s_last;

  // (the warp number through a shuffle: the compiler then knows that it is the same for the warp)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");     // nothing that earlier launches write is read before this

  // ---- this CTA's share of the work: a piece of an item, or the line's units [cur, end)
  Scan sum = {0, 0};
  long long lo = 0, hi = 0, first = 0;
  int longest = 0;
  for (int s0 = 0; s0 < a.n_seq; s0 += C::THREADS)
    scan_chunk<COLS, NW>(a, s0, s_scan, blockIdx.x == 0, sum, lo, hi, first, longest);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) s_longest[warp] = longest;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) longest = max(longest, s_longest[w]);
  const long long total = sum.line;
  const int pieces = sum.item > 0 && sum.item <= gridDim.x ? gridDim.x / static_cast<int>(sum.item) : 0;   // per item
  // (a line costs a CTA the taking up of a second item, which the even pieces may then take longer)
  const bool even = pieces > 0 && static_cast<long long>(max(MIN_PIECE, (longest + pieces - 1) / pieces) - SETUP) *
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
      if (a.n_seq > C::THREADS) scan_chunk<COLS, NW>(a, s0, s_scan, false, at, lo, hi, first, longest);
      const int s = s0 + tid;
      if (s < a.n_seq && hi > lo) {
        const SeqWork w = seq_work<COLS>(a, s, false);
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
  const uint32_t ring = tc::smem_u32(smem) + warp * (C::STAGES * C::STAGE + C::PREP);
  const uint32_t prep = ring + C::STAGES * C::STAGE;
  constexpr int KCH = DK / 32, VCH = DV / 32;   // 16-byte chunks of a row
  constexpr int KW4 = KW < 4 ? KW : 4;          // words of a lane's piece of a K row (of each 64 bytes)
  const uint32_t kc_at = chunk_at<DK>(lane / KCH, lane % KCH), vc_at = chunk_at<DV>(lane / VCH, lane % VCH);   // copies
  uint32_t k_at[(KW + 3) / 4], v_at[VCH / 2];   // reads: K row g; V matrices of rows 0-7 / 8-15 and two chunks
#pragma unroll
  for (int c = 0; c < (KW + 3) / 4; ++c) k_at[c] = chunk_at<DK>(g, (4 * KW4 * t + 64 * c) / 16) + (4 * KW4 * t) % 16;
#pragma unroll
  for (int c = 0; c < VCH / 2; ++c) v_at[c] = chunk_at<DV>(lane & 15, 2 * c + (lane >> 4));
  const int page_mask = (1 << a.page_shift) - 1;

  while (cur < end) {
    // ---- one segment: units u0 .. u1 - 1 of an item, which CTAs c0 .. c0 + n_con - 1 share
    const SeqWork w = seq_work<COLS>(a, seq, false);
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
      const long long per = w.units + SETUP;
      if (w.units == 0 || cur - pre >= per * w.items) {
        if (w.units > 0) pre += per * w.items;
        ++seq;
        continue;
      }
      item = (cur - pre) / per;
      const int r = static_cast<int>((cur - pre) - item * per), stop = static_cast<int>(min(per, r + (end - cur)));
      cur += stop - r;
      u0 = max(0, r - SETUP);
      u1 = max(0, stop - SETUP);
      if (u1 <= u0) continue;
      ia = pre + item * per + SETUP;
      auto owner = [&](long long x) { return static_cast<int>(((x + 1) * n_work - 1) / total); };
      c0 = owner(ia);
      n_con = owner(ia + w.units - 1) - c0 + 1;
    }
    const int hv = static_cast<int>(item) / w.chunks, chunk = static_cast<int>(item) - hv * w.chunks;
    const int cols_all = w.rows * a.group;
    const int c_base = chunk * COLS;
    // position of a column's row among the keys: it sees keys < its limit
    const int last_row = min(cols_all - 1, c_base + COLS - 1) / a.group;
    auto limit_of = [&](int row) { return a.causal ? max(0, w.len - w.rows + row + 1) : w.len; };
    const int k_begin = u0 * UNIT;
    const int k_end = min(limit_of(last_row), u1 * UNIT);
    const int n_tiles = k_end > k_begin ? (k_end - k_begin + TILE - 1) / TILE : 0;
    const int32_t *table = a.block_table + static_cast<int64_t>(seq) * a.max_pages;

    // ---- query rows: column g of tile n, the dims of this lane's K words (converted further down, while the
    // first copies are on their way)
    uint4 qraw[NT][KW];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = c_base + (MAPS == 2 ? g & 3 : 8 * n + g);
      const int row = c / a.group, head = hv * a.group + (c - row * a.group);
      const int64_t qb = (w.row0 + row) * a.q_stride + static_cast<int64_t>(MAPS == 2 ? 2 * head + (g >> 2) : head) * a.dk;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const int d0 = (i / 4) * 128 + KW4 * 8 * t + 8 * (i % 4);
        qraw[n][i] = make_uint4(0, 0, 0, 0);
        if (c < cols_all && d0 < a.dk)
          qraw[n][i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + qb + d0));
      }
    }

    // ---- the warp's tile copies.  Row numbers of a plane fit 32 bits (checked on the host); their bytes do not.
    const bool small_pages = a.page_shift < 5;                 // a tile's halves lie in two pages
    const uint32_t v_page_rows = static_cast<uint32_t>(a.n_kv_heads) << a.page_shift;
    const uint32_t v_row = static_cast<uint32_t>(hv) << a.page_shift;
    const uint8_t *k_base = a.k_codes + 16 * lane, *v_base = a.v_codes + 16 * lane;
    const uint8_t *ks_base = reinterpret_cast<const uint8_t *>(a.k_scales) + 4 * lane;
    const uint8_t *vs_base = reinterpret_cast<const uint8_t *>(a.v_scales) + 4 * lane;
    auto pages_of = [&](int tile, int &p0, int &p1) {          // of the tile's 16-key halves
      const int key = k_begin + tile * TILE;
      p0 = p1 = -1;
      if (tile < n_tiles) {
        p0 = p1 = __ldg(table + (key >> a.page_shift));
        if (small_pages) p1 = key + 16 < k_end ? __ldg(table + ((key + 16) >> a.page_shift)) : -1;
      }
    };
    auto issue = [&](int tile, int p0, int p1, uint32_t st) {
      const int key = k_begin + tile * TILE, left = k_end - key;
      const bool ok0 = static_cast<unsigned>(p0) < static_cast<unsigned>(a.n_pages);
      const bool ok1 = static_cast<unsigned>(p1) < static_cast<unsigned>(a.n_pages);
      const uint32_t in = key & page_mask;
      auto plane = [&](auto dim, const uint8_t *base, uint32_t row0, uint32_t row1, uint32_t dst, bool full) {
        constexpr int D = decltype(dim)::value, ROWS = 32 / (D / 32), N = TILE / ROWS;     // rows a copy, copies
        const uint8_t *s0 = base + static_cast<uint64_t>(row0) * (D / 2);
        const uint8_t *s1 = small_pages ? base + static_cast<uint64_t>(row1) * (D / 2) : s0 + 16 * (D / 2);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint8_t *src = (i < N / 2 ? s0 : s1) + (i % (N / 2)) * 512;
          // (a row of 256 codes is a line of its own, whose turn repeats after 8 rows, two copies)
          const uint32_t to = (st + dst + i * 512) ^ (D == 256 && (i & 1) ? 64u : 0u);
          if (full) {
            cp16(to, src);
          } else {
            const bool there = (i < N / 2 ? ok0 : ok1) && i * ROWS + lane / (D / 32) < left;
            cp16(to, there ? src : base, there ? 16 : 0);
          }
        }
      };
      auto scales = [&](const uint8_t *base, uint32_t row0, uint32_t row1, int p, bool full) {
        const uint32_t to = st + C::SC + (p * TILE + lane) * 4;
        const bool second = small_pages && lane >= 16;       // (lane 16 copies the first row of its half)
        const uint8_t *src = base + static_cast<uint64_t>(second ? row1 : row0) * 4 - (second ? 64 : 0);
        if (full) {
          cp4(to, src);
        } else {
          const bool there = (lane < 16 ? ok0 : ok1) && lane < left;
          cp4(to, there ? src : base, there ? 4 : 0);
        }
      };
      auto all = [&](bool full) {
        const uint32_t b0 = p0 * v_page_rows, b1 = p1 * v_page_rows;
#pragma unroll
        for (int m = 0; m < MAPS; ++m) {
          const uint32_t r = (static_cast<uint32_t>(MAPS * hv + m) << a.page_shift) + in;
          // (the second half of a small page's tile begins its page)
          const uint32_t r1 = r - in;
          plane(Int<DK>{}, k_base, MAPS * b0 + r, MAPS * b1 + r1, m * C::K_BYTES + kc_at, full);
          scales(ks_base, MAPS * b0 + r, MAPS * b1 + r1, m, full);
        }
        plane(Int<DV>{}, v_base, b0 + v_row + in, b1 + v_row, MAPS * C::K_BYTES + vc_at, full);
        scales(vs_base, b0 + v_row + in, b1 + v_row, MAPS, full);
      };
      if (ok0 && ok1 && left >= TILE) {
        all(true);
      } else {                        // the last tile, or a page outside the cache: zeros for what is not there
        if (lane == 0 && (!ok0 || (!ok1 && left > 16))) set_status(a.status, TQ_ERR_DEVICE_CHECK);
        all(false);
      }
    };
    uint32_t st = ring, st_fill = ring;           // the stage read, and the one filled, next
    auto next_stage = [&](uint32_t x) { return x == ring + (C::STAGES - 1) * C::STAGE ? ring : x + C::STAGE; };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
      int p0, p1;
      pages_of(warp + i * NW, p0, p1);
      if (warp + i * NW < n_tiles) issue(warp + i * NW, p0, p1, st_fill);
      st_fill = next_stage(st_fill);
      tc::cp_async_commit();
    }
    int pn0, pn1;
    pages_of(warp + (C::STAGES - 1) * NW, pn0, pn1);

    // ---- query fragments
    uint32_t qf[MAPS][NT][C::KS][2];
    float2 qx[NT], fx[NT];          // of columns 2t, 2t + 1: scale * log2(e) * sum(q), and the score factor
    int lim[NT][2];                 // their limits
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float v[KW][8], mx = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        unpack8(qraw[n][i], a.bf16, v[i]);
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
          const uint32_t even = half2_bits(v[i][2 * hf] * s1 * s2, v[i][2 * hf + 4] * s1 * s2);
          const uint32_t odd = half2_bits(v[i][2 * hf + 1] * s1 * s2 * 0.0625f, v[i][2 * hf + 5] * s1 * s2 * 0.0625f);
#pragma unroll
          for (int m = 0; m < MAPS; ++m) {
            const bool here = MAPS == 1 || (g >> 2) == m;
            qf[m][n][2 * i + hf][0] = here ? even : 0;
            qf[m][n][2 * i + hf][1] = here ? odd : 0;
          }
        }
      // this lane's softmax columns are 2t and 2t + 1: their values sit in lanes g = 2t, 2t + 1
      // (2^24 2^(ex - 12), as two factors: a small scale may come with queries near the end of their range)
      const float f = a.scale_log2 * 4096.f * __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
      const float qs = a.scale_log2 * sum;
      fx[n] = make_float2(__shfl_sync(0xffffffffu, f, 8 * t), __shfl_sync(0xffffffffu, f, 8 * t + 4));
      qx[n] = make_float2(__shfl_sync(0xffffffffu, qs, 8 * t), __shfl_sync(0xffffffffu, qs, 8 * t + 4));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int cc = c_base + (MAPS == 2 ? (2 * t + i) & 3 : 8 * n + 2 * t + i);
        lim[n][i] = cc < cols_all ? limit_of(cc / a.group) : 0;
      }
    }
    const int lim_min = limit_of(c_base / a.group);       // every column of the chunk sees the keys below

    float acc[NT][MT][4];
    float2 R[NT], Rs[NT], l[NT], z[NT];       // of columns 2t, 2t + 1; Rs: R, or 0 as long as there is none
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[n][i][c] = 0.f;
      R[n] = make_float2(-INFINITY, -INFINITY);
      Rs[n] = l[n] = z[n] = make_float2(0.f, 0.f);
    }

    for (int tile = warp; tile < n_tiles; tile += NW, st = next_stage(st)) {
      const int key0 = k_begin + tile * TILE;
      cp_wait<C::STAGES - 2>();
      __syncwarp();               // everybody's copies of this tile are there; the slot filled next was read
      {
        const int nt = tile + (C::STAGES - 1) * NW;
        if (nt < n_tiles) issue(nt, pn0, pn1, st_fill);
        st_fill = next_stage(st_fill);
        tc::cp_async_commit();
        pages_of(nt + NW, pn0, pn1);
      }
      // the lane's key: its scales ready for use
      {
        auto pair = [&](int p) {
          uint32_t u;
          lds<1>(&u, st + C::SC + (p * TILE + lane) * 4);
          return __half22float2(*reinterpret_cast<const __half2 *>(&u));
        };
        const float2 v = pair(MAPS), k = pair(0);
        const float c0 = fminf(fmaxf(__fdividef(-v.y, v.x), 0.f), 15.f), vm = fmaf(v.x, c0, v.y);   // (0 / 0, NaN: 0)
        const float e = v.x != 0.f ? static_cast<float>(static_cast<int>(__float_as_uint(fabsf(v.x)) >> 23) - 127) : -24.f;
        sts4(prep + lane * 16, v.x, v.x, vm, vm);
        sts2(prep + TILE * 16 + lane * 8, (FINE ? 8.f : 0.f) - c0, e);
        sts2(prep + TILE * 24 + lane * 8, k.x, k.y);
        if (MAPS == 2) {
          const float2 k1 = pair(MAPS - 1);
          sts2(prep + TILE * 32 + lane * 8, k1.x, k1.y);
        }
        __syncwarp();
      }
      const bool masked = key0 + TILE > lim_min || key0 + TILE > k_end;

      float4 vsc[4];              // of keys g + 8 j: V's (scale, scale, centred offset, the same)
      float2 vce[4], ksc[4];      // V's -c0 and exponent; K's scale and offset, of the map of the lane's columns
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        vsc[j] = lds4(prep + (8 * j + g) * 16);
        vce[j] = lds2(prep + TILE * 16 + (8 * j + g) * 8);
        ksc[j] = lds2(prep + TILE * (MAPS == 2 ? 24 + 8 * (t >> 1) : 24) + (8 * j + g) * 8);
      }
      uint32_t pb[NT][2][2];                // weights as B fragments [half][keys 0-7, 8-15]
      uint32_t pl[NT][2][2];                // and what their rounding left (FINE)
      float s[NT][2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[n][hf][c] = 0.f;
#pragma unroll
        for (int m = 0; m < MAPS; ++m) {
          uint32_t kw[2][KW];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < (KW + 3) / 4; ++c) {
              constexpr int W = KW < 4 ? KW : 4;
              lds<W>(&kw[r][4 * c], st + m * C::K_BYTES + (16 * hf + 8 * r) * (DK / 2) + k_at[c]);
            }
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            const uint32_t a0 = kw[0][i], a1 = kw[1][i], b0 = a0 >> 8, b1 = a1 >> 8;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(s[n][hf], a0 & 0x000f000fu, a1 & 0x000f000fu, a0 & 0x00f000f0u, a1 & 0x00f000f0u,
                       qf[m][n][2 * i][0], qf[m][n][2 * i][1]);
              mma16816(s[n][hf], b0 & 0x000f000fu, b1 & 0x000f000fu, b0 & 0x00f000f0u, b1 & 0x00f000f0u,
                       qf[m][n][2 * i + 1][0], qf[m][n][2 * i + 1][1]);
            }
          }
        }
      }
      {
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
          float2 x[4];                      // scores of keys g + 8 j, columns 2t and 2t + 1
          float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 sj = make_float2(s[nn][j >> 1][2 * (j & 1)], s[nn][j >> 1][2 * (j & 1) + 1]);
            x[j] = fma2(mul2(make_float2(ksc[j].x, ksc[j].x), sj), fx[nn], mul2(make_float2(ksc[j].y, ksc[j].y), qx[nn]));
          }
          if (masked) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = key0 + 8 * j + g;
              if (key >= min(lim[nn][0], k_end)) x[j].x = -INFINITY;
              if (key >= min(lim[nn][1], k_end)) x[j].y = -INFINITY;
            }
          }
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const float2 u = add2(x[j], make_float2(vce[j].y, vce[j].y));
            const float2 w = add2(x[j + 1], make_float2(vce[j + 1].y, vce[j + 1].y));
            mt[0] = max3(mt[0], u.x, w.x);
            mt[1] = max3(mt[1], u.y, w.y);
          }
          const bool raise = mt[0] > R[nn].x + RAISE || mt[1] > R[nn].y + RAISE;
          if (__any_sync(0xffffffffu, raise)) {
            auto lift = [&](float x, float &r, float &rs, float &lo, float &zo, int i) {
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              if (x > r + RAISE) {
                const float f = exp2f(r - x);             // 0 at the first raise
                r = rs = x;
                lo *= f;
                zo *= f;
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                  acc[nn][k][i] *= f;
                  acc[nn][k][i + 2] *= f;
                }
              }
            };
            lift(mt[0], R[nn].x, Rs[nn].x, l[nn].x, z[nn].x, 0);
            lift(mt[1], R[nn].y, Rs[nn].y, l[nn].y, z[nn].y, 1);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 d = sub2(x[j], Rs[nn]);
            const float2 p = make_float2(tc::ex2(d.x), tc::ex2(d.y));
            l[nn] = add2(l[nn], p);
            z[nn] = fma2(p, make_float2(vsc[j].z, vsc[j].w), z[nn]);
            const float2 w = mul2(p, make_float2(vsc[j].x, vsc[j].y));
            const __half2 h = __floats2half2_rn(w.x, w.y);
            float2 r = __half22float2(h);
            pb[nn][j >> 1][j & 1] = transpose8(*reinterpret_cast<const uint32_t *>(&h));
            if (FINE) {
              const float2 left = sub2(w, r);
              const __half2 lo = __floats2half2_rn(left.x, left.y);
              r = add2(r, __half22float2(lo));
              pl[nn][j >> 1][j & 1] = transpose8(*reinterpret_cast<const uint32_t *>(&lo));
            }
            z[nn] = fma2(r, make_float2(vce[j].x, vce[j].x), z[nn]);
          }
        }
      }
      // values: m tile 2 c + e holds dims 32 c + 4 g + 2 e (rows g) and + 1 (rows g + 8)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int c2 = 0; c2 < VCH / 2; ++c2) {
          uint32_t vw[4];                   // (chunk 2 c2: keys 0-7, 8-15), (chunk 2 c2 + 1: the same)
          ldsm4t(vw, st + MAPS * C::K_BYTES + (16 * hf) * (DV / 2) + v_at[c2]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t xa = vw[2 * e], xb = vw[2 * e + 1], ya = xa >> 8, yb = xb >> 8;
            const int mt = 2 * (2 * c2 + e);
            const uint32_t x[8] = {low_code<FINE>(xa), high_code<FINE>(xa), low_code<FINE>(xb), high_code<FINE>(xb),
                                   low_code<FINE>(ya), high_code<FINE>(ya), low_code<FINE>(yb), high_code<FINE>(yb)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(acc[n][mt], x[0], x[1], x[2], x[3], pb[n][hf][0], pb[n][hf][1]);
              mma16816(acc[n][mt + 1], x[4], x[5], x[6], x[7], pb[n][hf][0], pb[n][hf][1]);
              if (FINE) {
                mma16816(acc[n][mt], x[0], x[1], x[2], x[3], pl[n][hf][0], pl[n][hf][1]);
                mma16816(acc[n][mt + 1], x[4], x[5], x[6], x[7], pl[n][hf][0], pl[n][hf][1]);
              }
            }
          }
        }
    }
    cp_wait<0>();

    // ---- the CTA's warps together: fragments [warp][n][mt][lane] and (R, l, z) [warp][column]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, o);
        l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, o);
        z[n].x += __shfl_xor_sync(0xffffffffu, z[n].x, o);
        z[n].y += __shfl_xor_sync(0xffffffffu, z[n].y, o);
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
          p[0] = i ? R[n].y : R[n].x;
          p[1] = i ? l[n].y : l[n].x;
          p[2] = i ? z[n].y : z[n].x;
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
      s_lz[tid][0] = wts[4 * tid + 1] = ls;
      s_lz[tid][1] = wts[4 * tid + 2] = zs;
    }
    __syncthreads();

    // Fragments with columns that exist: of each (tile, m tile), lanes (g, t) with 1, 2 or 4 of the t.  A thread
    // takes PER of them, or several threads one.
    const int n_cols = min(COLS, cols_all - c_base);
    const int tsh = MAPS == 2 ? (n_cols > 2 ? 2 : 1) : n_cols > 4 ? 2 : n_cols > 2 ? 1 : 0;
    const int n_frag = NT * MT * (8 << tsh);
    auto frag_at = [&](int v) {
      const int low = v & ((1 << tsh) - 1);               // (two maps: t = 0 and 2)
      return (v >> (3 + tsh)) * 32 + ((v >> tsh) & 7) * 4 + (MAPS == 2 && tsh == 1 ? 2 * low : low);
    };
    constexpr int PER = (NT * MT * 32 + C::THREADS - 1) / C::THREADS;
    const bool whole = n_con == 1;
    float *mine = a.part + static_cast<int64_t>(2 * blockIdx.x + (even || share0 >= ia ? 0 : 1)) * C::PART;
    float4 o4[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int v = tid + k * C::THREADS;
      o4[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (v < n_frag) {
        const int f = frag_at(v), col = 8 * (f / (MT * 32)) + 2 * (f & 3);
#pragma unroll
        for (int x = 0; x < NW; ++x) {
          const float4 p = frag[x * (NT * MT * 32) + f];
          const float w0 = stat[(x * NC + col) * 3], w1 = stat[(x * NC + col + 1) * 3];
          o4[k].x = fmaf(w0, p.x, o4[k].x);
          o4[k].y = fmaf(w1, p.y, o4[k].y);
          o4[k].z = fmaf(w0, p.z, o4[k].z);
          o4[k].w = fmaf(w1, p.w, o4[k].w);
        }
        if (!whole) reinterpret_cast<float4 *>(mine + 4 * NC)[v] = o4[k];
      }
    }
    bool finish = whole;
    if (!whole) {
      if (tid < NC) reinterpret_cast<float4 *>(mine)[tid] = *reinterpret_cast<float4 *>(wts + 4 * tid);
      __syncthreads();
      if (tid == 0) s_last = arrive_one(a.counters + c0) == n_con - 1;
      __syncthreads();
      finish = s_last != 0;
      if (finish) {
        if (tid == 0) a.counters[c0] = 0;
        // CTA c0's partial is in its slot 0 when the item's part begins its share, else in slot 1; the
        // others' parts begin their shares
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
              p[i] = __ldcg(reinterpret_cast<const float4 *>(part_of(c + i * teams) + 4 * NC) + v);
          }
        };
        fetch(team, v0);                                         // on its way while the weights are worked out
        float *cw = reinterpret_cast<float *>(smem);             // [CTA][column]: weight of its partial
        float2 *clz = reinterpret_cast<float2 *>(cw + n_con * NC);
        for (int col = warp; col < NC; col += NW) {
          float M = -INFINITY, ls = 0.f, zs = 0.f;
#pragma unroll 2
          for (int c = lane; c < n_con; c += 32) {
            const float4 r = __ldcg(reinterpret_cast<const float4 *>(part_of(c)) + col);
            cw[c * NC + col] = r.x;
            clz[c * NC + col] = make_float2(r.y, r.z);
            M = fmaxf(M, r.x);
          }
          M = warp_max(M);
          for (int c = lane; c < n_con; c += 32) {
            const float r = cw[c * NC + col];
            const float2 lz = clz[c * NC + col];
            const float f = r == -INFINITY ? 0.f : exp2f(r - M);
            cw[c * NC + col] = f;
            ls = fmaf(f, lz.x, ls);
            zs = fmaf(f, lz.y, zs);
          }
          ls = warp_sum(ls);
          zs = warp_sum(zs);
          if (lane == 0) {
            s_lz[col][0] = ls;
            s_lz[col][1] = zs;
          }
        }
        __syncthreads();
        float4 *red = reinterpret_cast<float4 *>(clz + n_con * NC);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int v = v0 + k * C::THREADS;
          const int f = frag_at(v < n_frag ? v : 0), col = 8 * (f / (MT * 32)) + 2 * (f & 3);
          if (k > 0) fetch(team, v);
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c = team; c < n_con; c += B * teams) {
            if (c > team) fetch(c, v);
#pragma unroll
            for (int i = 0; i < B; ++i) {
              if (c + i * teams < n_con) {
                const float2 w2 = *reinterpret_cast<const float2 *>(cw + (c + i * teams) * NC + col);
                o.x = fmaf(w2.x, p[i].x, o.x);
                o.y = fmaf(w2.y, p[i].y, o.y);
                o.z = fmaf(w2.x, p[i].z, o.z);
                o.w = fmaf(w2.y, p[i].w, o.w);
              }
            }
          }
          o4[k] = o;
        }
        if (teams > 1) {
          if (team > 0 && team < teams) red[(team - 1) * n_frag + v0] = o4[0];
          __syncthreads();
          if (team == 0)
            for (int x = 1; x < teams; ++x) {
              const float4 q = red[(x - 1) * n_frag + v0];
              o4[0].x += q.x;
              o4[0].y += q.y;
              o4[0].z += q.z;
              o4[0].w += q.w;
            }
        }
      }
    }
    if (finish) {
      // fragment f = (n, mt, lane): dims d, d + 1 of columns col, col + 1
      __syncthreads();                      // shared memory is free for the differential exchange
      float *ex = reinterpret_cast<float *>(smem);               // [column][DV]
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int v = tid + k * C::THREADS;
        if (v < n_frag) {
          const int f = frag_at(v), n = f / (MT * 32), mt = (f / 32) % MT, fl = f & 31;
          const int d = 32 * (mt >> 1) + 4 * (fl >> 2) + 2 * (mt & 1);
          const int col = 8 * n + 2 * (fl & 3);
          float y[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float ls = s_lz[col + i][0], zs = s_lz[col + i][1];
            const float inv = ls != 0.f ? 1.f / ls : 0.f;        // nothing visible: zeros (NaN stays NaN)
            y[i][0] = ((i ? o4[k].y : o4[k].x) * (FINE ? 1.f : 16777216.f) + zs) * inv;
            y[i][1] = ((i ? o4[k].w : o4[k].z) * (FINE ? 1.f : 1048576.f) + zs) * inv;
            if (MAPS == 2) {
              ex[(col + i) * DV + d] = y[i][0];
              ex[(col + i) * DV + d + 1] = y[i][1];
            } else {
              const int c = c_base + col + i;
              if (c < cols_all && d < a.dv) {
                const int row = c / a.group, head = hv * a.group + c - row * a.group;
                store2(a.out, ((w.row0 + row) * static_cast<int64_t>(a.n_heads) + head) * a.dv + d, y[i][0], y[i][1],
                       a.bf16);
              }
            }
          }
        }
      }
      if (MAPS == 2) {
        // warp c < 4: columns c and 4 + c; o = map 0 - lambda map 1, RMS norm over the row, store
        __syncthreads();
        const int c = c_base + warp;
        if (warp < COLS && c < cols_all) {
          const int row = c / a.group, head = hv * a.group + c - row * a.group;
          const float lam = a.lam[head];
          float y[DV / 32], ss = 0.f;
#pragma unroll
          for (int i = 0; i < DV / 64; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = 64 * i + 2 * lane + e;
              const float x = d < a.dv ? ex[warp * DV + d] - lam * ex[(4 + warp) * DV + d] : 0.f;
              y[2 * i + e] = x;
              ss = fmaf(x, x, ss);
            }
          ss = warp_sum(ss);
          const float r = diff_factor(a, ss);
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
    __syncthreads();                        // shared memory is reused by the next segment's copies
  }

  // sequences without cells: their rows are zeros
  for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x) {
    const few::SeqWork w = few::seq_work<COLS>(a, s, false);
    if (w.len == 0) {
      const int64_t n = static_cast<int64_t>(w.rows) * a.n_heads * a.dv / 2;
      const int64_t at = static_cast<int64_t>(w.row0) * a.n_heads * a.dv;
      for (int64_t i = tid; i < n; i += C::THREADS) few::store2(a.out, at + 2 * i, 0.f, 0.f, a.bf16);
    }
  }
}

template <int DK, int DV, int NT, int MAPS, bool FINE>
cudaError_t launch_few_t(const AttnArgs &a, cudaStream_t s) {
  using C = FewCfg<DK, DV, NT, MAPS>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  static_assert(C::merge_bytes(C::grid(1 << 20)) <= C::SMEM && C::grid(152) == 152 * C::CTAS, "merge");
  static_assert(MAPS == 1 || NT == 1, "differential: one tile of columns for both maps");
  auto kern = few_kernel<DK, DV, NT, MAPS, FINE>;
  cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_beside(kern, C::grid(sm_count()), C::THREADS, C::SMEM, s, a);
}

// (binary16 outputs keep the weights to 22 bits)
template <int DK, int DV, int NT, int MAPS>
cudaError_t launch_few_t(const AttnArgs &a, cudaStream_t s) {
  return a.bf16 ? launch_few_t<DK, DV, NT, MAPS, false>(a, s) : launch_few_t<DK, DV, NT, MAPS, true>(a, s);
}

}  // namespace p4
}  // namespace tq
