// Single-token attention over int8 cells.
//
//   out[c] = sum_t p_t s^V_t v_t / sum_t p_t,   p_t = 2^(x_t - R),  x_t = scale log2(e) s^K_t (q . k_t)
//
// Columns are the query heads of a KV head, eight per tensor-core tile.  The work is reading the cache once, so
// everything is arranged around the loads.  Batches of long sequences are bound by HBM (40 ragged sequences of up to
// 32768 cells, 8 KV heads of 128: 188 to 197 us, 6.3 to 6.5 TB/s, 92 to 97% of a copy's rate; heads of 256 357 to 371
// us, 97% and more; single scattered cells 6 x 140000 260 us, 86%), short calls by the chain from the lengths to the
// merge (700 cells 8.1 us, 300 cells 6.6 us).
//
// - A warp streams its own tiles of 32 keys (16 where rows are wide) through a private ring of cp.async stages: it waits
//   for its own copies only, and no CTA barrier stands in the loop.  Each lane looks up one key's cell, so that pages of
//   any size, single cells among them, serve; where half a tile lies in one page its rows lie at even distances, else the
//   copying lanes get the row numbers by shuffles (40 ragged sequences over 16-cell pages: 203 us by shuffles, 195
//   without).  Rows lie in such places that copies and both kinds of reads spread over the banks.
// - The pages of the tile that is copied next are copied ahead as well, one ring turn before they are needed.
// - Codes become binary16 operands exactly: (w & 0x00ff00ff) ^ 0x64806480 is the pair 1024 + (code + 128), and 1152 is
//   taken off (two instructions for two codes, one more for the odd bytes).  Scores want pairs within a row: the words
//   of a K row serve as they are, the head dim's order being free as long as q has the same.  The value operand wants
//   pairs of neighbouring keys: a transposing ldmatrix over 16-bit units (two codes) delivers them so.
//   (Codes + 128 as binary16 subnormals, 128 sum(q) and 128 sum(p) taken off at the end, save the subtractions and no
//   time: they run on a pipe that is free.  They cost precision where a heavy key's values are near 0.)
// - One CTA of eight warps per SM (two where rows have 64 codes), with registers for two score tiles at a time in four
//   chains of products: with two CTAs of 16-key tiles an SM the per-tile work (455 against 315 instructions per 16 keys)
//   and the wait for products kept memory idle, and the CTAs of a pair ended up to 50 us apart (40 ragged sequences: 218
//   against 190 us).
// - Widths are those of the powers of two, and 80, 96 and 192 (K), since copies and products of zeros cost as much as
//   those of codes (40 ragged sequences, heads of 80 as 128 wide: 190 us, as 80 wide 158; 192 / 128 as 256 / 128: 284,
//   192 / 128 wide 263).
// - Scores: q is scaled by a power of two per column, so that its binary16 form is exact for binary16 and bfloat16
//   inputs down to 2^-23 of the column's largest entry.
// - The value weights p_t s^V_t are rounded to binary16: R + TOP follows the maximum of x_t + exponent(s^V_t), so the
//   largest weight lies in [2^12, 2^15] whatever the scales, and the sum of p_t stays in fp32.  R is raised only when it
//   would grow by more than 2^RAISE.  Weights end at 2^-25, that is 2^-37 of the largest: were the largest 1, those of
//   100000 keys 16 nats below it, one percent of the sum, would lose a third of themselves, and one nat further all.
//   The small step of R costs nothing up to 8 columns, and 4% at 16 (40 ragged sequences of 128 query heads: 221 us, with
//   steps of 2^12 213, of 2^4 218, both before the second product).
//   What that rounding left is a second product, so that a weight has 22 bits: 11 would cost binary16 results as much
//   again as their own rounding, and make every twentieth bfloat16 result another number than the exact one rounded
//   (now a few in a thousand).  That takes nothing where memory is the bound, and 2 to 13% of short and 16-column calls
//   (one sequence of 700 cells 7.9 -> 8.1 us, 64 of 1024 28.1 -> 29.4, 40 ragged ones of 128 query heads 221 -> 241).
// - Sums are fp32, but the matrix pipe cuts its own instead of rounding them: a warp that adds up 50000 keys one way gets
//   3e-4 too little, next to a heavy key 6e-4.  Its share of a long sequence is mostly a few thousand.
//
// Split of the work.  A CTA's warps take one, two or four KV heads (1 << hs) of the same cells side by side, so that what
// it reads of a cell lies together (40 ragged sequences 241 us with one head at a time, 196 so; single scattered cells 362
// and 262); the warps left take every so many-th tile.  An item is a (sequence, group of heads, column chunk), its
// keys come in units of 64.  Nothing about lengths is needed on the host: every CTA works its share out from the device's
// lengths.
// - Few items of like length: each is cut into as many pieces as there are CTAs per item, and a CTA has one piece.
// - Else the items' units form one line that is cut into equal shares, one per CTA, however ragged the batch is; taking
//   up an item counts as SET units.
// An item that several CTAs share leaves partial results (R, sum, values) in the workspace, a CTA's first and last item
// at most, and the last CTA to arrive merges them in the order of the CTAs, so that a repeated call gives the same bits.
// An item costs some 5 us besides its keys, mostly instructions one after the other; sending off the next item's first
// copies before the merge does not shorten that (256 sequences of 512 cells, then 60 us: 64).
#pragma once

#include <math.h>

#include "tq_common.cuh"
#include "tq_int8_cache.cuh"
#include "tq_paged4_few.cuh"
#include "tq_tc.cuh"

namespace tq {
namespace i8 {

using p4::AttnArgs;

// Log2 of the weight of a key that sets the running maximum (its value scale's mantissa makes it up to twice as much),
// and of the growth that raises the maximum.  Even numbers, so that both are exact next to scores of 2^24 as well, and
// their sum 14: the largest weight is then 2^14 (2 - 2^-10), and twice that, the maximum being rounded, still finite.
constexpr float TOP = 12.f, RAISE = 2.f;
constexpr int UNIT = 64;              // keys per unit of work
// Units of a piece at least.  Two are one tile of wide rows for each of eight warps, and of 32-key tiles only four: half of
// the warps have none then.  Four units leave none without, and are slower up to 1500 cells (one sequence of 570 cells 8.0
// us with two, 8.7 with four; of 700 8.2 and 8.9; of 1500 8.2 and 8.3; of 4096 9.1 and 8.8; 256-wide of 700 9.8 and 11.8):
// a warp's tiles come one after the other, and half as many CTAs ask for them.
constexpr int MIN_PIECE = 2;
// Units that one CTA has sooner done alone than shared and merged, two tiles for each of eight warps (one sequence of 300
// cells 6.6 against 7.8 us, of 440 7.1 against 7.9; of more units, shared: of 570 8.1)
constexpr int ALONE = 8;
// Units' worth of work that an item costs besides its keys (256 sequences of 512 cells, and 40 ragged ones with heads of
// 80 and 16 columns: 60.4 and 221 us with 4, 61.1 and 209 with 6, 62.3 and 206 with 8)
constexpr int SET = 6;
// Heads side by side, two choices.  A share of few units has little to gain, and more heads a CTA means fewer CTAs per
// head's keys (a sequence of 700 cells over 16-cell pages 8.5 us with one head at a time, 9.2 with two).  And the CTA
// that merges an item reads all its partial results (a sequence of 32768 cells 21.2 us with 19 of one head, 24.4 with 40
// of two).
constexpr int LONG = 8;               // units of a share at least (100 short sequences: 4 26.5, 8 21.9, 16 24.5 us)
constexpr int MERGED = 72;            // partial results of a head, times heads, at most

// Heads side by side whose partial results a CTA has room for in the workspace: 4 Ki values of fragments.
constexpr int part_heads(int wv, int nt) { return 512 / (wv * nt) < 4 ? 512 / (wv * nt) : 4; }

// Widths of rows: 64, 80, 96, 128, 192 (K), 256.  Those of 80 and 96 codes lie at odd numbers of 16-byte chunks.
constexpr bool pow2(int w) { return (w & (w - 1)) == 0; }
constexpr int pitch_of(int w) { return w == 96 ? 112 : w; }

template <int WK, int WV, int NT>
struct Cfg {
  static constexpr int KS = WK / 16, MT = WV / 16;        // k steps of the scores, m tiles of the values
  static constexpr int KJ = WK / 64, KR = KS - 4 * KJ;    // fours of K chunks, and the chunks left, a word a lane
  static constexpr int MP = MT <= 4 ? 4 : MT <= 8 ? 8 : 16;       // places of m tiles in merges
  static constexpr int KCH = WK / 16, VCH = WV / 16;      // 16-byte chunks of a row
  static constexpr int NW = 8;                            // (3 bits)
  static constexpr int THREADS = NW * 32;
  static constexpr int NC = 8 * NT;                       // columns
  // CTAs per SM: two where registers and rings leave room (decode of 40 ragged sequences, heads of 64: 116 -> 108 us)
  static constexpr int CTAS = WK == 64 && NT == 1 ? 2 : 1;
  static constexpr int TILE = WK + WV <= 256 ? 32 : 16;   // keys per warp tile
  static constexpr int HALVES = TILE / 16;
  // one stage: K rows, V rows, the words of the K and V scales, the halves of these that count, and the pages of the
  // tile that is to be copied when this one is read
  static constexpr int K_PITCH = pitch_of(WK), V_PITCH = pitch_of(WV);
  static constexpr int K_BYTES = TILE * K_PITCH, V_BYTES = TILE * V_PITCH;
  static constexpr int SC = K_BYTES + V_BYTES;
  static constexpr int STAGE = (SC + TILE * 16 + 127) / 128 * 128;
  static constexpr int PREP = TILE * 16;                  // a warp's unpacked scales of one tile
  static constexpr int MERGE = NW * NT * MP * 512 + NW * NC * 8 + NC * 8;       // CTA merge, in the same place
  static constexpr int FIT = (222 * 1024 / CTAS / NW - PREP) / STAGE;
  static constexpr int STAGES = FIT > 4 ? 4 : FIT;
  static constexpr int RING = NW * (STAGES * STAGE + PREP);
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  static constexpr int PART = 2 * NC + NT * MP * 128;     // a head's partial result: (R, l) by column, then fragments
  static constexpr int HEADS = part_heads(16 * MP, NT);       // heads side by side at most
  // A merge: (weight, sum) of every CTA and column, and the fragments of one CTA at least.  The grid: one CTA per SM, as
  // far as the merge of an item that every one of them shares finds room.
  static constexpr int merge_bytes(int ctas) { return ctas * NC * 8 + NT * MP * 512; }
  static constexpr int grid(int sms) {
    const int room = (SMEM - NT * MP * 512) / (NC * 8), fit = room < p4::kMaxCtas ? room : p4::kMaxCtas;
    return sms < (fit + CTAS - 1) / CTAS ? sms * CTAS : fit;
  }
  static_assert(STAGES >= 2 && STAGE % 128 == 0, "stages");
  static_assert(HEADS * PART <= 4096 + 128, "partial results");
  static_assert(2 * MERGED * NC * 8 + HEADS * NT * MP * 512 <= SMEM, "merge of heads side by side");
};

// Byte offset of 16-byte chunk c of row r.  K: one lane quad reads four chunks of a row, eight lanes those of rows r and
// r + 1, which lie on eight different places: odd rows are turned by four chunks, or (rows at odd numbers of chunks, P)
// even ones by P - 4, or they are four chunks apart as they are (192).  V: a matrix read takes one chunk of eight rows.
template <int W>
__device__ __forceinline__ uint32_t k_chunk(int r, int c) {
  constexpr int P = pitch_of(W) / 16;
  if (W == 64 || W == 192) return r * W + c * 16;
  if (P & 1) return (r * P + (r & 1 ? c : c + P - 4 < P ? c + P - 4 : c - 4)) * 16;
  return r * W + ((c ^ ((r & 1) << 2)) * 16);
}
template <int W>
__device__ __forceinline__ uint32_t v_chunk(int r, int c) {
  constexpr int P = pitch_of(W) / 16;
  if (P & 1) return (r * P + c) * 16;
  return W == 64 ? (r >> 1) * 128 + (((((r & 1) << 2) + c) ^ ((r >> 1) & 3)) * 16) : r * W + ((c ^ (r & 7)) * 16);
}
// The turn's share of copy i in a V chunk's place: its rows are 32 / (W / 16) i and on.
template <int W>
__device__ __forceinline__ constexpr uint32_t v_turn(int i) { return W == 64 ? 0u : ((i * (512 / W)) & 7) * 16u; }

// Codes in bytes 0 and 2 of a word as a pair of binary16 numbers (of w >> 8: those in bytes 1 and 3).
__device__ __forceinline__ uint32_t codes_of(uint32_t w) {
  const uint32_t x = (w & 0x00ff00ffu) ^ 0x64806480u;                     // 1024 + 128 + code
  const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), __float2half2_rn(1152.f));
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ const uint8_t *ahead(const uint8_t *p, uint32_t step, int i) {
  uint64_t r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(step), "r"(i), "l"(reinterpret_cast<uint64_t>(p)));
  return reinterpret_cast<const uint8_t *>(r);
}

__device__ __forceinline__ float scale_of(uint32_t word, uint32_t sel) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(prmt_b32(word, 0u, sel))));
}

// a / b (b > 0, a >= 0): of numbers below 2^32, as nearly all are, in 32 bits
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if ((static_cast<uint64_t>(a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A sequence's length as the call takes it.
__device__ __forceinline__ int length_of(const AttnArgs &a, int s, bool report) {
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  const int len = a.seq_len[s];
  if (len >= 0 && len <= cap) return len;
  if (report) set_status(a.status, TQ_ERR_DEVICE_CHECK);
  return len < 0 ? 0 : static_cast<int>(cap);
}

// What lies before a sequence on a line where every sequence with cells takes its units and SET more: `units` of them,
// and `seqs` such sequences.
struct Line {
  long long units;
  int seqs, longest;
};
// Sequence s0 + tid (few: s0 + lane, every warp for itself): its units, and what lies before it.  Moves `at` past all
// sequences of the block (few: of the warp).
template <int NW>
__device__ __forceinline__ void scan_lengths(const AttnArgs &a, int s0, bool few, Line *sums, bool report, Line &at,
                                             Line &before, int &own) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, s = s0 + (few ? lane : tid);
  own = s < a.n_seq ? (length_of(a, s, report) + UNIT - 1) / UNIT : 0;
  Line x = {own > 0 ? own + SET : 0, own > 0 ? 1 : 0, own};
  const Line v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x.units, o);
    const int n = __shfl_up_sync(0xffffffffu, x.seqs, o);
    if (lane >= o) {
      x.units += u;
      x.seqs += n;
    }
  }
  x.longest = __reduce_max_sync(0xffffffffu, own);
  Line all = {0, 0, 0};
  if (few) {
    all = {__shfl_sync(0xffffffffu, x.units, 31), __shfl_sync(0xffffffffu, x.seqs, 31), x.longest};
  } else {
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w == warp) {
        x.units += all.units;
        x.seqs += all.seqs;
      }
      all.units += sums[w].units;
      all.seqs += sums[w].seqs;
      all.longest = max(all.longest, sums[w].longest);
    }
  }
  before = {at.units + x.units - v.units, at.seqs + x.seqs - v.seqs, 0};
  at = {at.units + all.units, at.seqs + all.seqs, max(at.longest, all.longest)};
}

template <int WK, int WV, int NT>
__global__ void __launch_bounds__(Cfg<WK, WV, NT>::THREADS, Cfg<WK, WV, NT>::CTAS)
    decode_kernel(const AttnArgs a) {
  using C = Cfg<WK, WV, NT>;
  using namespace p4::few;
  constexpr int NW = C::NW, MT = C::MT, NC = C::NC, TILE = C::TILE;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Line s_scan[NW];
  __shared__ float s_inv[NW * NC];
  __shared__ long long s_pre;
  __shared__ int s_seq, s_last;

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");     // nothing that earlier launches write is read before this

  // ---- the work, as a line of units
  Line sum = {0, 0, 0}, before = {0, 0, 0};
  int own = 0;
  const bool few = a.n_seq <= 32;         // every warp looks at all sequences: no barriers
  for (int s0 = 0; s0 < a.n_seq; s0 += C::THREADS)
    scan_lengths<NW>(a, s0, few, s_scan, blockIdx.x == 0, sum, before, own);
  const int chunks = (a.group + NC - 1) / NC, grid = gridDim.x;
  const long long line1 = sum.units * chunks;             // (of one KV head)
  // Heads side by side: as many as the KV heads divide into, while the CTAs' shares stay LONG and whoever merges the
  // longest sequence's item has at most MERGED partial results to read (one from each CTA's share, and one more at
  // either end).
  int hs = 0;
  while ((2 << hs) <= C::HEADS && a.n_kv_heads % (2 << hs) == 0) {
    const long long n = a.n_kv_heads >> (hs + 1), line = n * line1;
    if (line < static_cast<long long>(LONG) * grid ||
        static_cast<long long>(sum.longest) * grid > ((MERGED >> (hs + 1)) - 2) * line)
      break;
    ++hs;
  }
  const int per_seq = (a.n_kv_heads >> hs) * chunks;      // items of a sequence
  const long long total = sum.units * per_seq, items = static_cast<long long>(sum.seqs) * per_seq;
  const int pieces = items > 0 && items <= grid ? grid / static_cast<int>(items) : 0;   // per item
  // (a line costs a CTA the taking up of a second item, which the even pieces may then take longer)
  const int least = max(1, MIN_PIECE >> hs);              // units of a piece
  const bool even = pieces > 0 &&
                    static_cast<long long>(max(least, (sum.longest + pieces - 1) / pieces) - SET) * grid <= total;
  const int n_work = static_cast<int>(even ? pieces * items : min(static_cast<long long>(grid), total));     // shares
  // piece o of the line: where it begins, and which one unit x belongs to
  auto start_of = [&](int o) { return quotient(o * total, n_work); };
  auto piece_of = [&](long long x) { return static_cast<int>(quotient((x + 1) * n_work - 1, total)); };

  // ---- the warp's ring, and the lane's places in its rows
  const int head_of = warp & ((1 << hs) - 1), tile0 = warp >> hs, tiles_by = NW >> hs;
  const uint32_t ring = tc::smem_u32(smem) + warp * (C::STAGES * C::STAGE + C::PREP), prep = ring + C::STAGES * C::STAGE;
  const uint32_t kc_at = k_chunk<WK>(lane / C::KCH, lane % C::KCH);
  const uint32_t vc_at = C::K_BYTES + v_chunk<WV>(lane / C::VCH, lane % C::VCH);
  const uint32_t k_size = (lane % C::KCH) * 16 < a.dk ? 16 : 0, v_size = (lane % C::VCH) * 16 < a.dv ? 16 : 0;
  uint32_t k_at[C::KJ], k_word[C::KR + 1];      // reads: K row g, chunks t + 4 j; words t of the chunks left
#pragma unroll
  for (int j = 0; j < C::KJ; ++j) k_at[j] = k_chunk<WK>(g, t + 4 * j);
#pragma unroll
  for (int y = 0; y < C::KR; ++y) k_word[y] = k_chunk<WK>(g, 4 * C::KJ + y) + 4 * t;
  uint32_t v_at[(MT + 1) / 2];                  // matrices of keys 0-7 / 8-15, chunks 2 j, 2 j + 1 (a last one twice)
#pragma unroll
  for (int j = 0; j < (MT + 1) / 2; ++j) v_at[j] = C::K_BYTES + v_chunk<WV>(lane & 15, min(2 * j + (lane >> 4), MT - 1));
  constexpr bool EVEN = pow2(WK) && pow2(WV);   // a copy's lanes take whole rows, the same chunks each time
  const int page_mask = (1 << a.page_shift) - 1;
  const bool apart = TILE / 2 >> a.page_shift > 1;        // half a tile lies in several pages
  const uint8_t *k_base = a.k_codes + (k_size ? 16 * (lane % C::KCH) : 0);
  const uint8_t *v_base = a.v_codes + (v_size ? 16 * (lane % C::VCH) : 0);
  // (the last scale of a plane with an odd number of them is half a word)
  const uint32_t last_row = static_cast<uint32_t>(a.n_rows_cache - 1);

  // ---- this CTA's piece: of an item (even), or the line's units [cur, end)
  const int piece = blockIdx.x;
  long long cur = 0, end = 0, pre = 0;
  int seq = 0;
  if (piece < n_work) {
    cur = even ? piece / pieces : start_of(piece);
    end = even ? cur + 1 : start_of(piece + 1);
    auto has = [&](const Line &b, int n, long long &first) {   // whether the share begins in the n units after b
      first = even ? static_cast<long long>(b.seqs) * per_seq : b.units * per_seq;
      return n > 0 && first <= cur && cur < first + (even ? per_seq : static_cast<long long>(n + SET) * per_seq);
    };
    long long first;
    if (few) {
      const int from = __ffs(__ballot_sync(0xffffffffu, has(before, own, first))) - 1;
      seq = from;
      pre = __shfl_sync(0xffffffffu, first, from);
    } else {
      Line at = {0, 0, 0};
      for (int s0 = 0; s0 < a.n_seq; s0 += C::THREADS) {
        // (a batch of one block still has its sums in registers)
        if (a.n_seq > C::THREADS) scan_lengths<NW>(a, s0, false, s_scan, false, at, before, own);
        if (has(before, own, first)) {
          s_seq = s0 + tid;
          s_pre = first;
        }
      }
      __syncthreads();
      seq = s_seq;
      pre = s_pre;
    }
  }
  const long long share0 = cur;

  while (cur < end) {
    // ---- one segment: units u0 .. u1 - 1 of an item, which CTAs c0 .. c0 + n_con - 1 share
    const int len = length_of(a, seq, false), units = (len + UNIT - 1) / UNIT;
    long long ia = 0;                     // the line's unit that is the item's first one
    int item, u0, u1, c0, n_con;
    if (even) {
      item = static_cast<int>(cur - pre);
      const int n = units <= ALONE >> hs ? 1 : max(1, min(pieces, units / least)), i = piece % pieces;
      if (i >= n) break;
      const int each = units / n, rest = units - each * n;    // (the first pieces take one unit of the rest each)
      u0 = i * each + min(i, rest);
      u1 = u0 + each + (i < rest ? 1 : 0);
      c0 = piece - i;
      n_con = n;
      cur = end;
    } else {
      const int per = units + SET;
      if (units == 0 || cur - pre >= static_cast<long long>(per) * per_seq) {
        if (units > 0) pre += static_cast<long long>(per) * per_seq;
        ++seq;
        continue;
      }
      item = static_cast<int>(quotient(cur - pre, per));
      const int r = static_cast<int>((cur - pre) - static_cast<long long>(item) * per);
      const int stop = static_cast<int>(min(static_cast<long long>(per), r + (end - cur)));
      cur += stop - r;
      u0 = max(0, r - SET);
      u1 = max(0, stop - SET);
      if (u1 <= u0) continue;
      ia = pre + static_cast<long long>(item) * per + SET;
      c0 = piece_of(ia);
      n_con = piece_of(ia + units - 1) - c0 + 1;
    }
    const int hg = chunks == 1 ? item : item / chunks, chunk = item - hg * chunks, h0 = hg << hs, hv = h0 + head_of;
    const int c_base = chunk * NC, n_cols = min(NC, a.group - c_base);
    const int k_begin = u0 * UNIT, k_end = min(len, u1 * UNIT);
    const int n_tiles = k_end > k_begin ? (k_end - k_begin + TILE - 1) / TILE : 0;
    const int32_t *table = a.block_table + static_cast<int64_t>(seq) * a.max_pages;

    // ---- query rows: column g of tile n, the dims of this lane's K chunks (converted further down, while the
    // first copies are on their way)
    uint4 qraw[NT][C::KJ][2];
    uint2 qword[NT][C::KR + 1];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = 8 * n + g;
      const int64_t qb = seq * a.q_stride + static_cast<int64_t>(hv * a.group + c_base + c) * a.dk;
#pragma unroll
      for (int j = 0; j < C::KJ; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int d0 = 16 * (t + 4 * j) + 8 * i;
          qraw[n][j][i] = make_uint4(0, 0, 0, 0);
          if (c < n_cols && d0 < a.dk)
            qraw[n][j][i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + qb + d0));
        }
#pragma unroll
      for (int y = 0; y < C::KR; ++y) {
        const int d0 = 16 * (4 * C::KJ + y) + 4 * t;
        qword[n][y] = make_uint2(0, 0);
        if (c < n_cols && d0 < a.dk)
          qword[n][y] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + qb + d0));
      }
    }

    // ---- the warp's tile copies.  Numbers of rows fit 32 bits (checked on the host); all ones: no row, zeros.
    const uint32_t kv_heads = a.n_kv_heads;
    // Which half of its word a key's scale is: all the same for an even number of KV heads, else by the cell, whose
    // number is even where the key's is, but for pages of one cell (odd_cells: noted with the copy).
    const uint32_t half_sel = (hv ^ (kv_heads & lane)) & 1 ? 0x4432u : 0x4410u;
    const bool odd_cells = (kv_heads & 1) && a.page_shift == 0;
    auto page_of = [&](int tile) {                              // of the lane's key
      const int key = k_begin + tile * TILE + (lane & (TILE - 1));
      return key < k_end ? __ldg(table + (key >> a.page_shift)) : -1;
    };
    auto scales_in = [&](uint32_t row, bool ok, uint32_t st) {
      if (TILE < 32 && lane >= TILE) return;
      const uint32_t n = !ok ? 0 : row == last_row && !(row & 1) ? 2 : 4;
      cp4(st + C::SC + lane * 4, a.k_scales + (row & ~1u), n);
      cp4(st + C::SC + (TILE + lane) * 4, a.v_scales + (row & ~1u), n);
      if (odd_cells)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + C::SC + (2 * TILE + lane) * 4), "r"(row & 1 ? 0x4432u : 0x4410u)
                     : "memory");
    };
    auto issue = [&](int tile, int page, uint32_t st) {
      const int key = k_begin + tile * TILE + (lane & (TILE - 1));
      const int ahead_key = key + (C::STAGES - 1) * tiles_by * TILE;
      if (TILE == 32 || lane < TILE)
        cp4(st + C::SC + (3 * TILE + lane) * 4, table + (ahead_key < k_end ? ahead_key >> a.page_shift : 0),
            ahead_key < k_end ? 4 : 0);
      const bool in = key < k_end, ok = in && static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages);
      const uint32_t row = ((static_cast<uint32_t>(page) << a.page_shift) + (key & page_mask)) * kv_heads + hv;
      const uint32_t there = __ballot_sync(0xffffffffu, ok);
      scales_in(ok ? row : 0, ok, st);
      if (EVEN && there == 0xffffffffu && !apart) {             // half a tile in one page: its rows at even distances
        const uint32_t k_step = (32 / C::KCH) * kv_heads * a.dk, v_step = (32 / C::VCH) * kv_heads * a.dv;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          constexpr int NK = TILE * C::KCH / 64, NV = TILE * C::VCH / 64;        // copies of half a tile
          const uint32_t row0 = __shfl_sync(0xffffffffu, row, h * (TILE / 2));
          const uint8_t *ks = k_base + static_cast<uint64_t>(row0 + (lane / C::KCH) * kv_heads) * a.dk;
          const uint8_t *vs = v_base + static_cast<uint64_t>(row0 + (lane / C::VCH) * kv_heads) * a.dv;
#pragma unroll
          for (int i = 0; i < NK; ++i) cp16(st + kc_at + (h * NK + i) * 512, ahead(ks, k_step, i), k_size);
#pragma unroll
          for (int i = 0; i < NV; ++i)
            cp16(st + (vc_at ^ v_turn<WV>(h * NV + i)) + (h * NV + i) * 512, ahead(vs, v_step, i), v_size);
        }
      } else {                            // rows apart, the last tile, a page outside the cache: zeros for the missing
        if (in && !ok) set_status(a.status, TQ_ERR_DEVICE_CHECK);
        const uint32_t mine = ok ? row : 0;
#pragma unroll
        for (int i = 0; i < TILE * C::KCH / 32; ++i) {
          const int k = (32 * i + lane) / C::KCH, c = (32 * i + lane) % C::KCH;
          const uint32_t size = EVEN ? k_size : 16 * c < a.dk ? 16 : 0, to = EVEN ? kc_at + i * 512 : k_chunk<WK>(k, c);
          const uint8_t *from = (EVEN ? k_base : a.k_codes + (size ? 16 * c : 0));
          from += static_cast<uint64_t>(__shfl_sync(0xffffffffu, mine, k)) * a.dk;
          cp16(st + to, from, there >> k & 1 ? size : 0);
        }
#pragma unroll
        for (int i = 0; i < TILE * C::VCH / 32; ++i) {
          const int k = (32 * i + lane) / C::VCH, c = (32 * i + lane) % C::VCH;
          const uint32_t size = EVEN ? v_size : 16 * c < a.dv ? 16 : 0;
          const uint32_t to = EVEN ? (vc_at ^ v_turn<WV>(i)) + i * 512 : C::K_BYTES + v_chunk<WV>(k, c);
          const uint8_t *from = (EVEN ? v_base : a.v_codes + (size ? 16 * c : 0));
          from += static_cast<uint64_t>(__shfl_sync(0xffffffffu, mine, k)) * a.dv;
          cp16(st + to, from, there >> k & 1 ? size : 0);
        }
      }
    };
    uint32_t st = ring, st_fill = ring;           // the stage read next, and the one filled: the one read last
    auto next_stage = [&](uint32_t x) { return x == ring + (C::STAGES - 1) * C::STAGE ? ring : x + C::STAGE; };
    int page[C::STAGES - 1];                      // of the first tiles, looked up at once
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) page[i] = page_of(tile0 + i * tiles_by);
#pragma unroll 1
    for (int i = 0; i < C::STAGES - 1; ++i) {     // (not unrolled: instructions are fetched anew for every segment)
      if (tile0 + i * tiles_by < n_tiles) issue(tile0 + i * tiles_by, page[0], st_fill);
#pragma unroll
      for (int j = 1; j < C::STAGES - 1; ++j) page[j - 1] = page[j];
      st_fill = next_stage(st_fill);
      tc::cp_async_commit();
    }

    // ---- query fragments
    uint32_t qf[NT][C::KS][2];
    float2 fx[NT];                  // of columns 2t, 2t + 1: the score factor
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float v[4 * C::KS], mx = 0.f;         // four of each k step
#pragma unroll
      for (int j = 0; j < 2 * C::KJ; ++j) unpack8(qraw[n][j / 2][j & 1], a.bf16, v + 8 * j);
#pragma unroll
      for (int y = 0; y < C::KR; ++y) {
        float w[8];
        unpack8(make_uint4(qword[n][y].x, qword[n][y].y, 0, 0), a.bf16, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[16 * C::KJ + 4 * y + e] = w[e];
      }
#pragma unroll
      for (int e = 0; e < 4 * C::KS; ++e) mx = fmaxf(mx, fabsf(v[e]));
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // max in [2^ex, 2^(ex+1)) -> scaled to [2^12, 2^13) (below 2^-114 to less, exactly as well)
      const int ex = mx > 0x1p-114f ? static_cast<int>(__float_as_uint(mx) >> 23) - 127 : -114;
      const float up = __uint_as_float(static_cast<uint32_t>(12 - ex + 127) << 23);
#pragma unroll
      for (int i = 0; i < C::KS; ++i) {
        const float *x = v + 4 * i;
        const float2 lo = mul2(make_float2(x[0], x[2]), make_float2(up, up));
        const float2 hi = mul2(make_float2(x[1], x[3]), make_float2(up, up));
        qf[n][i][0] = half2_bits(lo.x, lo.y);
        qf[n][i][1] = half2_bits(hi.x, hi.y);
      }
      // this lane's softmax columns are 2t and 2t + 1: their factors sit in lanes g = 2t, 2t + 1
      const float f = a.scale_log2 * 0x1p-12f * __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
      fx[n] = make_float2(__shfl_sync(0xffffffffu, f, 8 * t), __shfl_sync(0xffffffffu, f, 8 * t + 4));
    }

    float acc[NT][MT][4];
    // of columns 2t, 2t + 1; Ru: R + TOP + RAISE; Rs: R, or 0 as long as there is none
    float2 R[NT], Ru[NT], Rs[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[n][i][c] = 0.f;
      R[n] = Ru[n] = make_float2(-INFINITY, -INFINITY);
      Rs[n] = l[n] = make_float2(0.f, 0.f);
    }

    for (int tile = tile0; tile < n_tiles; tile += tiles_by, st = next_stage(st)) {
      const int key0 = k_begin + tile * TILE;
      cp_wait<C::STAGES - 2>();
      __syncwarp();               // everybody's copies of this tile are there; the slot filled next was read
      {
        const int nt = tile + (C::STAGES - 1) * tiles_by;
        // Where a tile's rows lie apart, the warps of a cell's heads keep together, so that what they read of a cell is
        // asked for at once (6 x 140000 single cells 321 -> 265 us; in larger pages the wait costs more than it gives).
        if (hs > 0 && apart) asm volatile("bar.sync %0, %1;" ::"r"(1 + tile0), "r"(32 << hs) : "memory");
        if (nt < n_tiles) {
          uint32_t p;
          lds<1>(&p, st + C::SC + (3 * TILE + (lane & (TILE - 1))) * 4);
          issue(nt, static_cast<int>(p), st_fill);
        }
        st_fill = st;
        tc::cp_async_commit();
      }

      // the lane's key: its scales ready for use (V's exponent is an integer in the low bits of 2^23; 0's counts as -24)
      if (TILE == 32 || lane < TILE) {
        uint32_t u[2], sel = half_sel;
        lds<1>(u, st + C::SC + lane * 4);
        lds<1>(u + 1, st + C::SC + (TILE + lane) * 4);
        if (odd_cells) lds<1>(&sel, st + C::SC + (2 * TILE + lane) * 4);
        const float x = scale_of(u[1], sel);
        sts4(prep + lane * 16, scale_of(u[0], sel), x,
             fmaxf(__uint_as_float((__float_as_uint(fabsf(x)) >> 23) | 0x4b000000u) - 8388735.f, -24.f), 0.f);
      }
      __syncwarp();
      // scores of keys g + 8 j, columns 2t and 2t + 1
      constexpr int H = C::HALVES;
      float s[NT][H][4];
      {
        float s2[NT][H][4];                 // (of every other step, so that no product waits for the one before)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int hf = 0; hf < H; ++hf)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[n][hf][c] = s2[n][hf][c] = 0.f;
#pragma unroll
        for (int j = 0; j < C::KJ; ++j) {
          uint32_t w0[H][4], w1[H][4];
#pragma unroll
          for (int hf = 0; hf < H; ++hf) {
            lds<4>(w0[hf], st + k_at[j] + hf * 16 * C::K_PITCH);
            lds<4>(w1[hf], st + k_at[j] + (hf * 16 + 8) * C::K_PITCH);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int hf = 0; hf < H; ++hf) {
              const uint32_t x0 = codes_of(w0[hf][i]), x1 = codes_of(w1[hf][i]);
              const uint32_t x2 = codes_of(w0[hf][i] >> 8), x3 = codes_of(w1[hf][i] >> 8);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816((i & 1 ? s2 : s)[n][hf], x0, x1, x2, x3, qf[n][4 * j + i][0], qf[n][4 * j + i][1]);
            }
        }
#pragma unroll
        for (int y = 0; y < C::KR; ++y)
#pragma unroll
          for (int hf = 0; hf < H; ++hf) {
            uint32_t w0, w1;
            lds<1>(&w0, st + k_word[y] + hf * 16 * C::K_PITCH);
            lds<1>(&w1, st + k_word[y] + (hf * 16 + 8) * C::K_PITCH);
            const uint32_t x0 = codes_of(w0), x1 = codes_of(w1), x2 = codes_of(w0 >> 8), x3 = codes_of(w1 >> 8);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816((y & 1 ? s2 : s)[n][hf], x0, x1, x2, x3, qf[n][4 * C::KJ + y][0], qf[n][4 * C::KJ + y][1]);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int hf = 0; hf < H; ++hf)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[n][hf][c] += s2[n][hf][c];
      }
      float4 sc[2 * H];                     // of keys g + 8 j: the scales, V's exponent
#pragma unroll
      for (int j = 0; j < 2 * H; ++j) sc[j] = lds4(prep + (g + 8 * j) * 16);
      uint32_t pb[NT][2 * H], pl[NT][2 * H];      // weights as B fragments [keys 8 j ..], and what their rounding left
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float2 x[2 * H];
        float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 2 * H; ++j) {
          const float2 sj = make_float2(s[n][j >> 1][2 * (j & 1)], s[n][j >> 1][2 * (j & 1) + 1]);
          x[j] = mul2(mul2(make_float2(sc[j].x, sc[j].x), sj), fx[n]);
        }
        if (key0 + TILE > k_end) {
#pragma unroll
          for (int j = 0; j < 2 * H; ++j)
            if (key0 + 8 * j + g >= k_end) x[j] = make_float2(-INFINITY, -INFINITY);
        }
#pragma unroll
        for (int j = 0; j < 2 * H; j += 2) {
          const float2 u = add2(x[j], make_float2(sc[j].z, sc[j].z));
          const float2 w = add2(x[j + 1], make_float2(sc[j + 1].z, sc[j + 1].z));
          mt[0] = max3(mt[0], u.x, w.x);
          mt[1] = max3(mt[1], u.y, w.y);
        }
        const bool raise = mt[0] > Ru[n].x || mt[1] > Ru[n].y;
        if (__any_sync(0xffffffffu, raise)) {
          auto lift = [&](float m, float &r, float &ru, float &rs, float &lo, int i) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (m > ru) {
              const float low = m - TOP, f = exp2f(r - low);    // 0 at the first raise
              r = rs = low;
              ru = m + RAISE;
              lo *= f;
#pragma unroll
              for (int k = 0; k < MT; ++k) {
                acc[n][k][i] *= f;
                acc[n][k][i + 2] *= f;
              }
            }
          };
          lift(mt[0], R[n].x, Ru[n].x, Rs[n].x, l[n].x, 0);
          lift(mt[1], R[n].y, Ru[n].y, Rs[n].y, l[n].y, 1);
        }
        float2 lt;                // the tile's own sum: next to a heavy key's p, l rounds 1 addend of 4
#pragma unroll
        for (int j = 0; j < 2 * H; ++j) {
          const float2 d = sub2(x[j], Rs[n]);
          const float2 p = make_float2(tc::ex2(d.x), tc::ex2(d.y));
          lt = j == 0 ? p : add2(lt, p);
          const float2 wv = mul2(p, make_float2(sc[j].y, sc[j].y));
          const __half2 h = __floats2half2_rn(wv.x, wv.y);
          pb[n][j] = transpose8(*reinterpret_cast<const uint32_t *>(&h));
          const float2 left = sub2(wv, __half22float2(h));
          pl[n][j] = transpose8(half2_bits(left.x, left.y));
        }
        l[n] = add2(l[n], lt);
      }
      // values: m tile c holds dims 16 c + 2 g (rows g) and + 1 (rows g + 8)
#pragma unroll
      for (int hf = 0; hf < H; ++hf)
#pragma unroll
        for (int c = 0; c < MT; c += 2) {
          uint32_t vw[4];                   // (chunk c: keys 0-7, 8-15), (chunk c + 1: the same)
          ldsm4t(vw, st + v_at[c / 2] + hf * 16 * C::V_PITCH);
#pragma unroll
          for (int e = 0; e < (c + 1 < MT ? 2 : 1); ++e) {
            const uint32_t x0 = codes_of(vw[2 * e]), x1 = codes_of(vw[2 * e] >> 8);
            const uint32_t x2 = codes_of(vw[2 * e + 1]), x3 = codes_of(vw[2 * e + 1] >> 8);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(acc[n][c + e], x0, x1, x2, x3, pb[n][2 * hf], pb[n][2 * hf + 1]);
              mma16816(acc[n][c + e], x0, x1, x2, x3, pl[n][2 * hf], pl[n][2 * hf + 1]);
            }
          }
        }
    }
    cp_wait<0>();

    // ---- a head's warps together: fragments [warp][n][mt][lane] and (R, l) [warp][column]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, o);
        l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, o);
      }
    __syncthreads();                        // the ring is no longer read
    float4 *frag = reinterpret_cast<float4 *>(smem);
    // [warp][column]: (R, l), then (weight, l)
    float2 *stat = reinterpret_cast<float2 *>(smem + NW * NT * C::MP * 512);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < MT; ++k)
        frag[((warp * NT + n) * C::MP + k) * 32 + lane] =
            make_float4(acc[n][k][0], acc[n][k][1], acc[n][k][2], acc[n][k][3]);
      if (g == 0) {
        stat[warp * NC + 8 * n + 2 * t] = make_float2(R[n].x, l[n].x);
        stat[warp * NC + 8 * n + 2 * t + 1] = make_float2(R[n].y, l[n].y);
      }
    }
    __syncthreads();

    // Fragments with columns that exist: of each (head, tile, m tile), lanes (g, t) with 1, 2 or 4 of the t.
    const int heads = 1 << hs;
    const int tsh = n_cols > 4 ? 2 : n_cols > 2 ? 1 : 0;
    constexpr int FSH = NT * C::MP == 4 ? 5 : NT * C::MP == 8 ? 6 : NT * C::MP == 16 ? 7 : 8;
    const int fsh = FSH + tsh, n_frag = 1 << fsh, ash = fsh + hs, all_frag = 1 << ash;
    static_assert(NT * C::MP * 8 == 1 << FSH, "fragments");
    auto frag_at = [&](int v) { return (v >> (3 + tsh)) * 32 + ((v >> tsh) & 7) * 4 + (v & ((1 << tsh) - 1)); };
    auto col_of = [&](int f) { return 8 * (f / (C::MP * 32)) + 2 * (f & 3); };
    auto is_there = [&](int f) { return MT == C::MP || (f / 32) % C::MP < MT; };
    auto add = [](float4 &o, float w0, float w1, const float4 &p) {
      o.x = fmaf(w0, p.x, o.x);
      o.y = fmaf(w1, p.y, o.y);
      o.z = fmaf(w0, p.z, o.z);
      o.w = fmaf(w1, p.w, o.w);
    };
    // fragment f of head h0 + h: dims d, d + 1 of columns col, col + 1
    const int64_t out0 = (static_cast<int64_t>(seq) * a.n_heads + h0 * a.group + c_base) * a.dv;
    auto put = [&](int h, int f, const float4 &o) {
      const int mt = (f / 32) % C::MP, fl = f & 31, col = col_of(f);
      const int d = 16 * mt + 2 * (fl >> 2);
      if (d >= a.dv) return;
      const int64_t at = out0 + ((h * a.group + col) * a.dv + d);
      const float i0 = s_inv[h * NC + col], i1 = s_inv[h * NC + col + 1];
      if (col < n_cols) store2(a.out, at, o.x * i0, o.z * i0, a.bf16);
      if (col + 1 < n_cols) store2(a.out, at + a.dv, o.y * i1, o.w * i1, a.bf16);
    };
    auto inverse = [](float ls) { return ls != 0.f ? 1.f / ls : 0.f; };
    const bool whole = n_con == 1;
    float *mine = a.part + static_cast<int64_t>(2 * piece + (even || share0 >= ia ? 0 : 1)) * C::HEADS * C::PART;
    if (tid < NW * NC) {                    // (head, column, warp of the head): the warp's weight, and the sums
      const int x = tid & (tiles_by - 1), hcol = tid >> (3 - hs), h = hcol / NC, col = hcol - h * NC;
      float2 *at = stat + (h + (x << hs)) * NC + col;
      const float2 rl = *at;
      float M = rl.x;
#pragma unroll
      for (int o = 1; o < NW; o <<= 1)
        if (o < tiles_by) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float f = rl.x == -INFINITY ? 0.f : exp2f(rl.x - M);
      float ls = f * rl.y;
#pragma unroll
      for (int o = 1; o < NW; o <<= 1)
        if (o < tiles_by) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      at->x = f;
      if (x == 0) {
        s_inv[hcol] = inverse(ls);
        if (!whole) reinterpret_cast<float2 *>(mine + h * C::PART)[col] = make_float2(M, ls);
      }
    }
    __syncthreads();
    for (int v = tid; v < all_frag; v += C::THREADS) {
      const int h = v >> fsh, u = v & (n_frag - 1), f = frag_at(u), col = col_of(f);
      if (!is_there(f)) continue;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NW; ++k)
        if (k < tiles_by) {
          const int x = h + (k << hs);
          add(o, stat[x * NC + col].x, stat[x * NC + col + 1].x, frag[x * (NT * C::MP * 32) + f]);
        }
      if (whole) put(h, f, o);
      else reinterpret_cast<float4 *>(mine + h * C::PART + 2 * NC)[u] = o;
    }
    if (!whole) {
      __syncthreads();
      if (tid == 0) s_last = arrive_one(a.counters + c0) == n_con - 1;
      __syncthreads();
      if (s_last) {
        if (tid == 0) a.counters[c0] = 0;
        // CTA c0's partial is in its slot 0 when the item's part begins its share, else in slot 1; the others' parts
        // begin their shares
        const int slot0 = even || start_of(c0) >= ia ? 0 : 1;
        auto part_of = [&](int c, int h) {
          return a.part + (static_cast<int64_t>(2 * (c0 + c) + (c == 0 ? slot0 : 0)) * C::HEADS + h) * C::PART;
        };
        // shared memory: [CTA][head, column] weights and sums, then the fragments of as many CTAs as there is room for
        constexpr int CSH = NT == 1 ? 3 : 4;
        const int hsh = CSH + hs, hc = 1 << hsh;
        static_assert(NC == 1 << CSH, "columns");
        float *cw = reinterpret_cast<float *>(smem), *cl = cw + n_con * hc;
        float4 *buf = reinterpret_cast<float4 *>(cl + n_con * hc);
        const int room = (C::SMEM - n_con * hc * 8) >> (ash + 4);
        auto fetch = [&](int c1) {                               // of CTAs c1 and on
          const int n = min(room, n_con - c1) * all_frag;
          for (int i = tid; i < n; i += C::THREADS) {
            const int c = i >> ash, v = i & (all_frag - 1);
            if (!is_there(frag_at(v & (n_frag - 1)))) continue;
            cp16(tc::smem_u32(buf + i), part_of(c1 + c, v >> fsh) + 2 * NC + 4 * (v & (n_frag - 1)));
          }
          tc::cp_async_commit();
        };
        fetch(0);                                                // on its way while the weights are worked out
        for (int i = tid; i < n_con * hc; i += C::THREADS) {
          const int c = i >> hsh, col = i & (hc - 1);
          const float2 r = __ldcg(reinterpret_cast<const float2 *>(part_of(c, col / NC)) + col % NC);
          cw[i] = r.x;
          cl[i] = r.y;
        }
        __syncthreads();
        for (int col = tid >> 3; col < hc; col += C::THREADS / 8) {      // eight threads a column
          float M = -INFINITY, ls = 0.f;
          for (int c = tid & 7; c < n_con; c += 8) M = fmaxf(M, cw[c * hc + col]);
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
          for (int c = tid & 7; c < n_con; c += 8) {
            const float r = cw[c * hc + col];
            const float f = r == -INFINITY ? 0.f : exp2f(r - M);
            cw[c * hc + col] = f;
            ls = fmaf(f, cl[c * hc + col], ls);
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
          if ((tid & 7) == 0) s_inv[col] = inverse(ls);
        }
        constexpr int MOST = (C::HEADS * NT * C::MP * 32 + C::THREADS - 1) / C::THREADS;     // fragments of a thread
        float4 o[MOST];
#pragma unroll
        for (int k = 0; k < MOST; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c1 = 0; c1 < n_con; c1 += room) {
          cp_wait<0>();
          __syncthreads();
#pragma unroll
          for (int k = 0; k < MOST; ++k) {
            const int v = tid + k * C::THREADS;
            if (v >= all_frag) break;
            if (!is_there(frag_at(v & (n_frag - 1)))) continue;
            const int col = (v >> fsh) * NC + col_of(frag_at(v & (n_frag - 1)));
#pragma unroll 8
            for (int c = c1; c < min(n_con, c1 + room); ++c) {
              const float2 w2 = *reinterpret_cast<const float2 *>(cw + c * hc + col);
              add(o[k], w2.x, w2.y, buf[(c - c1) * all_frag + v]);
            }
          }
          if (c1 + room < n_con) {
            __syncthreads();
            fetch(c1 + room);
          }
        }
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
          const int v = tid + k * C::THREADS;
          if (v < all_frag) put(v >> fsh, frag_at(v & (n_frag - 1)), o[k]);
        }
      }
    }
    __syncthreads();                        // shared memory is reused by the next segment's copies
  }

  // sequences without cells: their rows are zeros
  for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x) {
    if (length_of(a, s, false) == 0) {
      const int64_t n = static_cast<int64_t>(a.n_heads) * a.dv / 2, at = s * 2 * n;
      for (int64_t i = tid; i < n; i += C::THREADS) store2(a.out, at + 2 * i, 0.f, 0.f, a.bf16);
    }
  }
}

template <int WK, int WV, int NT>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t s) {
  using C = Cfg<WK, WV, NT>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  static_assert(C::merge_bytes(C::grid(1 << 20)) <= C::SMEM && C::grid(152) == 152 * C::CTAS, "merge");
  auto kern = decode_kernel<WK, WV, NT>;
  cudaError_t e = set_dynamic_smem(reinterpret_cast<const void *>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  return p4::launch_beside(kern, C::grid(sm_count()), C::THREADS, C::SMEM, s, a);
}

// up to eight columns in one tile, else two tiles at a time
template <int WK, int WV>
cudaError_t launch_w(const AttnArgs &a, cudaStream_t s) {
  return a.group <= 8 ? launch_t<WK, WV, 1>(a, s) : launch_t<WK, WV, 2>(a, s);
}

}  // namespace i8
}  // namespace tq
