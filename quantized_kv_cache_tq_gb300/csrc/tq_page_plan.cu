// Block tables and slot maps of a batch, built from request lengths on the GPU.
//
// With old_s = seq_len[s], d_s = n_new[s], new_s = old_s + d_s and pages(n) =
// ceil(n / page_size): a sequence that shrinks returns pages(old) - pages(new)
// page ids to the free list's end, one that grows takes pages(new) - pages(old)
// from it.  Both are exclusive prefix sums over the sequences, so every page's
// place on the list is known without any atomic and the result does not depend
// on timing.
//
// The first kernel is one CTA: it checks everything, then writes lengths, prefix
// sums and the returned pages (one thread per page, which finds its sequence by
// bisection of the prefix sums in shared memory).  The second gives one thread to
// each new row: the row finds its sequence in q_start, and its page either in the
// block table (held before) or straight on the free list (new), so it does not
// wait for other rows; the row at a new page's first cell also writes the table
// entry (a new page always starts with a new row).  A step of up to SMALL_ROWS
// rows and one chunk of sequences is done by the first kernel alone.
//
// Neither has bytes to speak of (12 per row): what counts is the length of the
// chain of dependent loads, lengths -> sums -> page -> slot.  Measured: a step of 48
// sequences 4.2 us, of which an empty launch is about half; 700 admissions with 1.0 M
// rows 10.1 us (12 MB written in 1.8 us at the memory's rate), 10.5 with the second
// launch waiting for the first one's end.
#include "tq_common.cuh"
#include "tq_paged4.cuh"

namespace tq {
namespace p4 {
namespace {

constexpr int PT = 1024;          // threads of the planning CTA, sequences of a chunk
constexpr int SMALL_ROWS = 4096;

struct Sums {                     // rows, pages returned, pages taken
  long long r, b, m;
};

__device__ __forceinline__ Sums add(const Sums &x, const Sums &y) { return {x.r + y.r, x.b + y.b, x.m + y.m}; }

// Exclusive prefix sums over the CTA; `total` gets the sums over all threads.
__device__ Sums scan(Sums v, Sums *warp_sums, Sums &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto inclusive = [&](Sums x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      Sums y;
      y.r = __shfl_up_sync(0xffffffffu, x.r, o);
      y.b = __shfl_up_sync(0xffffffffu, x.b, o);
      y.m = __shfl_up_sync(0xffffffffu, x.m, o);
      if (lane >= o) x = add(x, y);
    }
    return x;
  };
  const Sums x = inclusive(v);
  __syncthreads();                // the previous call's sums are no longer read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const Sums w = inclusive(warp_sums[lane]);               // every warp: sums of warps 0 .. lane
  Sums before = {0, 0, 0};
  total.r = __shfl_sync(0xffffffffu, w.r, 31);
  total.b = __shfl_sync(0xffffffffu, w.b, 31);
  total.m = __shfl_sync(0xffffffffu, w.m, 31);
  const long long br = __shfl_sync(0xffffffffu, w.r, max(warp - 1, 0));
  const long long bb = __shfl_sync(0xffffffffu, w.b, max(warp - 1, 0));
  const long long bm = __shfl_sync(0xffffffffu, w.m, max(warp - 1, 0));
  if (warp > 0) before = {br, bb, bm};
  return {before.r + x.r - v.r, before.b + x.b - v.b, before.m + x.m - v.m};
}

struct Seq {
  long long old_len, new_len;
  int have, need;                 // pages before and after
  bool ok;
};

__device__ __forceinline__ Seq read_seq(const PlanArgs &a, int s) {
  Seq q;
  q.old_len = a.seq_len[s];
  q.new_len = q.old_len + a.n_new[s];
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  q.ok = q.old_len >= 0 && q.old_len <= cap && q.new_len >= 0 && q.new_len <= cap;
  const long long up = (1ll << a.page_shift) - 1;
  q.have = q.ok ? static_cast<int>((q.old_len + up) >> a.page_shift) : 0;
  q.need = q.ok ? static_cast<int>((q.new_len + up) >> a.page_shift) : 0;
  return q;
}

__device__ __forceinline__ Sums sums_of(const Seq &q) {
  const long long d = q.ok ? q.new_len - q.old_len : 0;
  return {d > 0 ? d : 0, q.have > q.need ? q.have - q.need : 0, q.need > q.have ? q.need - q.have : 0};
}

// The last i in [lo, hi] with at(i) <= r (at ascending, at(lo) <= r).
template <typename F>
__device__ __forceinline__ int bisect(int lo, int hi, int r, F at) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at(mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Slot and position of row r, the i-th new cell of a sequence that held `old_len` cells and takes
// its new pages from place `page_start` below `top` on.
__device__ __forceinline__ void fill_row(const PlanArgs &a, int r, int i, int seq, int old_len, int page_start, int top) {
  const int pos = old_len + i;
  const int j = pos >> a.page_shift, in = pos & ((1 << a.page_shift) - 1);
  const int have = static_cast<int>((static_cast<long long>(old_len) + (1 << a.page_shift) - 1) >> a.page_shift);
  int32_t *entry = a.block_table + static_cast<int64_t>(seq) * a.max_pages + j;
  int page;
  if (j < have) {
    page = *entry;
  } else {
    page = a.free_pages[top - 1 - (page_start + j - have)];
    if (in == 0) *entry = page;
  }
  a.slots[r] = (static_cast<int64_t>(page) << a.page_shift) + in;
  a.positions[r] = pos;
}

// ROWS: the rows too, in the same launch (one chunk of sequences).
template <bool ROWS>
__global__ void __launch_bounds__(PT) plan_kernel(const PlanArgs a) {
  __shared__ Sums warp_sums[PT / 32];
  __shared__ int s_rows[PT], s_back[PT], s_more[PT], s_need[PT], s_old[PT];
  const int tid = threadIdx.x;
  if (!ROWS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the rows' launch may begin beside this one
  const long long count = *a.free_count;
  const bool one = a.n_seq <= PT;           // the only chunk: its sums are computed once
  Sums all = {0, 0, 0}, at = {0, 0, 0}, v = {0, 0, 0};
  Seq q = {0, 0, 0, 0, false};
  bool ok = true;
  for (int s0 = 0; s0 < a.n_seq; s0 += PT) {
    v = {0, 0, 0};
    if (s0 + tid < a.n_seq) {
      q = read_seq(a, s0 + tid);
      ok = ok && q.ok;
      v = sums_of(q);
    }
    Sums t;
    at = scan(v, warp_sums, t);
    all = add(all, t);
  }
  ok = ok && count >= 0 && count + all.b <= a.free_capacity && count + all.b - all.m >= 0 && all.r <= a.n_rows;
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (tid == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);
    all = at = {0, 0, 0};
  }
  Sums carry = {0, 0, 0};
  for (int s0 = 0; s0 < a.n_seq; s0 += PT) {
    const int s = s0 + tid, n = min(PT, a.n_seq - s0);
    Sums t = all;
    if (!one) {
      v = {0, 0, 0};
      if (s < a.n_seq) {
        q = read_seq(a, s);
        if (ok) v = sums_of(q);
      }
      at = add(carry, scan(v, warp_sums, t));
    }
    if (s < a.n_seq) {
      a.q_start[s] = static_cast<int>(at.r);
      a.page_start[s] = static_cast<int>(at.m);
      a.new_len[s] = static_cast<int>(ok ? q.new_len : q.old_len);
      s_back[tid] = static_cast<int>(at.b - carry.b);
      s_need[tid] = q.need;
      if (ROWS) {
        s_rows[tid] = static_cast<int>(at.r);
        s_more[tid] = static_cast<int>(at.m);
        s_old[tid] = static_cast<int>(q.old_len);
      }
    }
    __syncthreads();
    for (int i = tid; i < t.b; i += PT) {   // returned pages of the chunk, one thread each
      const int c = bisect(0, n - 1, i, [&](int x) { return s_back[x]; });
      a.free_pages[count + carry.b + i] =
          a.block_table[static_cast<int64_t>(s0 + c) * a.max_pages + s_need[c] + i - s_back[c]];
    }
    carry = add(carry, t);
  }
  if (tid == 0) {
    a.q_start[a.n_seq] = static_cast<int>(carry.r);
    a.page_start[a.n_seq] = static_cast<int>(carry.m);
    *a.new_free_count = static_cast<int>(count + carry.b - carry.m);
  }
  if (ROWS) {
    __syncthreads();                        // the returned pages are on the free list
    for (int r = tid; r < a.n_rows; r += PT) {
      if (r < carry.r) {
        const int c = bisect(0, a.n_seq - 1, r, [&](int x) { return s_rows[x]; });
        fill_row(a, r, r - s_rows[c], c, s_old[c], s_more[c], static_cast<int>(count + carry.b));
      } else {
        a.slots[r] = -1;
        a.positions[r] = -1;
      }
    }
  }
}

// ROWS_PER rows of a CTA lie in few sequences: the CTA looks its first and last one up, its threads between them.
constexpr int ROWS_PER = 1024;

__global__ void __launch_bounds__(256) rows_kernel(const PlanArgs a) {
  __shared__ int s_seq[2];
  const int r0 = static_cast<int>(static_cast<long long>(blockIdx.x) * ROWS_PER);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = a.q_start[a.n_seq];
  const int top = *a.new_free_count + a.page_start[a.n_seq];
  const int r1 = static_cast<int>(min(static_cast<long long>(r0) + ROWS_PER, static_cast<long long>(a.n_rows)));
  auto start = [&](int x) { return a.q_start[x]; };
  if (threadIdx.x < 2 && r0 < total)
    s_seq[threadIdx.x] = bisect(0, a.n_seq - 1, threadIdx.x ? min(r1, total) - 1 : r0, start);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ROWS_PER / 256; ++i) {
    const int r = r0 + i * 256 + threadIdx.x;
    if (r < min(r1, total)) {
      const int s = bisect(s_seq[0], s_seq[1], r, start);
      const int first = a.q_start[s];
      fill_row(a, r, r - first, s, a.new_len[s] - (a.q_start[s + 1] - first), a.page_start[s], top);
    } else if (r < r1) {
      a.slots[r] = -1;
      a.positions[r] = -1;
    }
  }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs &a, cudaStream_t s) {
  // one launch for steps of few rows; beyond, one CTA would write them slower than a second launch takes
  if (a.n_rows <= SMALL_ROWS && a.n_seq <= PT) {
    plan_kernel<true><<<1, PT, 0, s>>>(a);
    return cudaGetLastError();
  }
  plan_kernel<false><<<1, PT, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.n_rows == 0) return e;        // a step in which sequences only shrink has no rows to fill
  return launch_beside(rows_kernel, static_cast<unsigned>((a.n_rows + ROWS_PER - 1) / ROWS_PER), 256, 0, s, a);
}

}  // namespace p4
}  // namespace tq
