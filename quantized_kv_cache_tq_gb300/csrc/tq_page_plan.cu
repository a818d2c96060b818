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
// sums and the returned pages.  The second gives one thread to each new row: the
// row finds its sequence by bisection of q_start, and its page either in the
// block table (held before) or straight on the free list (new), so it does not
// wait for other rows; the row at a new page's first cell also writes the table
// entry (a new page always starts with a new row).
#include "tq_common.cuh"
#include "tq_paged4.cuh"

namespace tq {
namespace p4 {
namespace {

constexpr int PT = 1024;          // threads of the planning CTA

struct Sums {                     // rows, pages returned, pages taken
  long long r, b, m;
};

__device__ __forceinline__ Sums add(const Sums &x, const Sums &y) { return {x.r + y.r, x.b + y.b, x.m + y.m}; }

// Exclusive prefix sums over the CTA; `total` gets the sums over all threads.
__device__ Sums scan(Sums v, Sums *warp_sums, Sums &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sums y;
    y.r = __shfl_up_sync(0xffffffffu, x.r, o);
    y.b = __shfl_up_sync(0xffffffffu, x.b, o);
    y.m = __shfl_up_sync(0xffffffffu, x.m, o);
    if (lane >= o) x = add(x, y);
  }
  __syncthreads();                // the previous call's sums are no longer read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  Sums before = {0, 0, 0};
  total = {0, 0, 0};
  for (int w = 0; w < PT / 32; ++w) {
    if (w == warp) before = total;
    total = add(total, warp_sums[w]);
  }
  x = add(before, x);
  return {x.r - v.r, x.b - v.b, x.m - v.m};
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

// Slot and position of new row r (see the head of the file); -1 behind the last one.
__device__ __forceinline__ void fill_row(const PlanArgs &a, long long r, int total, int top) {
  if (r >= total) {
    a.slots[r] = -1;
    a.positions[r] = -1;
    return;
  }
  int lo = 0, hi = a.n_seq - 1;             // the last sequence whose first row is <= r and that has rows
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.q_start[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  const int first = a.q_start[lo];
  const int old_len = a.new_len[lo] - (a.q_start[lo + 1] - first);
  const int pos = old_len + static_cast<int>(r - first);
  const int j = pos >> a.page_shift, in = pos & ((1 << a.page_shift) - 1);
  const int have = (old_len + (1 << a.page_shift) - 1) >> a.page_shift;
  int32_t *entry = a.block_table + static_cast<int64_t>(lo) * a.max_pages + j;
  int page;
  if (j < have) {
    page = *entry;
  } else {
    page = a.free_pages[top - 1 - (a.page_start[lo] + j - have)];
    if (in == 0) *entry = page;
  }
  a.slots[r] = (static_cast<int64_t>(page) << a.page_shift) + in;
  a.positions[r] = pos;
}

// ROWS: the rows too (short batches), in the same launch.
template <bool ROWS>
__global__ void __launch_bounds__(PT) plan_kernel(const PlanArgs a) {
  __shared__ Sums warp_sums[PT / 32];
  const int tid = threadIdx.x;
  const long long count = *a.free_count;
  Sums all = {0, 0, 0};
  bool ok = true;
  for (int s0 = 0; s0 < a.n_seq; s0 += PT) {
    Sums v = {0, 0, 0};
    if (s0 + tid < a.n_seq) {
      const Seq q = read_seq(a, s0 + tid);
      ok = ok && q.ok;
      v = sums_of(q);
    }
    Sums t;
    scan(v, warp_sums, t);
    all = add(all, t);
  }
  ok = ok && count >= 0 && count + all.b <= a.free_capacity && count + all.b - all.m >= 0 && all.r <= a.n_rows;
  ok = __syncthreads_and(ok);
  if (!ok && tid == 0) set_status(a.status, TQ_ERR_DEVICE_CHECK);
  Sums carry = {0, 0, 0};
  for (int s0 = 0; s0 < a.n_seq; s0 += PT) {
    const int s = s0 + tid;
    Seq q = {0, 0, 0, 0, false};
    Sums v = {0, 0, 0};
    if (s < a.n_seq) {
      q = read_seq(a, s);
      if (ok) v = sums_of(q);
    }
    Sums t;
    const Sums at = add(carry, scan(v, warp_sums, t));
    if (s < a.n_seq) {
      a.q_start[s] = static_cast<int>(at.r);
      a.page_start[s] = static_cast<int>(at.m);
      const int32_t *row = a.block_table + static_cast<int64_t>(s) * a.max_pages;
      if (ok)
        for (int j = q.need; j < q.have; ++j) a.free_pages[count + at.b + j - q.need] = row[j];
      a.new_len[s] = static_cast<int>(ok ? q.new_len : q.old_len);
    }
    carry = add(carry, t);
  }
  if (tid == 0) {
    a.q_start[a.n_seq] = static_cast<int>(carry.r);
    a.page_start[a.n_seq] = static_cast<int>(carry.m);
    *a.new_free_count = static_cast<int>(count + carry.b - carry.m);
  }
  if (ROWS) {
    __syncthreads();              // the CTA's own writes to global memory are visible to it
    for (long long r = tid; r < a.n_rows; r += PT)
      fill_row(a, r, static_cast<int>(carry.r), static_cast<int>(count + carry.b));
  }
}

__global__ void __launch_bounds__(256) rows_kernel(const PlanArgs a) {
  const long long r = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (r < a.n_rows) fill_row(a, r, a.q_start[a.n_seq], *a.new_free_count + a.page_start[a.n_seq]);
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs &a, cudaStream_t s) {
  if (a.n_rows <= 2 * PT) {
    plan_kernel<true><<<1, PT, 0, s>>>(a);
    return cudaGetLastError();
  }
  plan_kernel<false><<<1, PT, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  rows_kernel<<<static_cast<unsigned>((a.n_rows + 255) / 256), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace p4
}  // namespace tq
