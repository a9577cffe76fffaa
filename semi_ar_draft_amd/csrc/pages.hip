// Page bookkeeping of a paged key-value cache: the pages a step's rows need,
// the rows' places, and the return of the pages a verification leaves unused.
//
// [summary] section 5 (the variable-length verify batch: rows laid end to
// end, an offset and a marker per row).  Integer work on a few numbers per
// request, bound by latency: one launch each, in which every workgroup scans
// the requests for itself (12 bytes a request, from the caches) and then
// writes its own share of the rows or pages, one a thread, so that no workgroup
// waits for another and a row costs one search in LDS and one load behind it.
// Arrays that may be updated in place (held, n_free, len) are written by the
// last workgroup to finish, after every other has read them.  Measured, of
// which a launch of nothing takes 2 to 3: reserve 3.3 us for one request, 5.9
// for 512 requests and 3300 rows; commit 3.0 for 9 requests, 5.7 for 512.
#include "common.hpp"
#include "internal.hpp"

namespace dspark {
namespace {

// Exclusive scan over the requests of N counts at once, each below 2^31 in
// total or the result is not used: every thread sums its run of consecutive
// requests, the workgroup scans the sums.  x holds the counts on entry and
// their exclusive prefixes on return, entry B the totals.  Returns false (to
// every thread) if a total passes 2^31 - 1.
template <int N>
__device__ __forceinline__ bool scan_requests(int B, int32_t* const (&x)[N], int64_t (*red)[N]) {
  const int per = (B + kPagesThreads - 1) / kPagesThreads;
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int64_t sum[N], incl[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    sum[k] = 0;
    for (int b = b0; b < b1; ++b) sum[k] += x[k][b];
    incl[k] = sum[k];
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t u = __shfl_up(incl[k], o, 64);
      if (lane >= o) incl[k] += u;
    }
  if (lane == 63)
#pragma unroll
    for (int k = 0; k < N; ++k) red[w][k] = incl[k];
  __syncthreads();
  bool ok = true;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    int64_t at = incl[k] - sum[k], total = 0;
#pragma unroll
    for (int i = 0; i < kPagesThreads / 64; ++i) {
      if (i < w) at += red[i][k];
      total += red[i][k];
    }
    for (int b = b0; b < b1; ++b) {
      const int32_t c = x[k][b];
      x[k][b] = (int32_t)at;
      at += c;
    }
    const bool fits = total <= INT32_MAX;
    ok = ok && fits;
    if (threadIdx.x == 0) x[k][B] = fits ? (int32_t)total : 0;
  }
  __syncthreads();
  return ok;
}

// The last index b of [0, B) with first[b] <= i (first non-decreasing,
// first[0] = 0): the request that entry i belongs to, empty ones skipped.
__device__ __forceinline__ int owner(const int32_t* first, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// True in every thread of the last workgroup of the launch to come here.  The
// others' loads have returned (their values are used before), and nothing they
// stored is read, so that the count needs no fence.  *bad (LDS) counts in its
// upper half: nonzero in the last workgroup if it was in any.
__device__ __forceinline__ bool last_workgroup(unsigned int* done, int* flag, int* bad) {
  __syncthreads();
  if (gridDim.x == 1) return true;
  if (threadIdx.x == 0) {
    const unsigned int mine = 1u + (*bad ? 0x10000u : 0u);   // fewer than 2^16 workgroups
    const unsigned int n = __hip_atomic_fetch_add(done, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + mine;
    *flag = (n & 0xFFFFu) == gridDim.x;
    *bad = n >> 16;
    if (*flag) __hip_atomic_store(done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *flag != 0;
}

// Pages popped from the stack's top in request order: the j-th new page of
// request b is free_list[n_free - 1 - (new pages of earlier requests) - j].
// A row's slot needs no table entry of this launch: a page past held[b] is
// looked up in the free list.
__global__ __launch_bounds__(kPagesThreads) void pages_reserve_impl(const PagesArgs a) {
  __shared__ int32_t n[kPagesMaxB + 1], x[kPagesMaxB + 1], lens[kPagesMaxB], helds[kPagesMaxB];
  __shared__ int64_t red[kPagesThreads / 64][2];
  __shared__ int bad, flag;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  const int64_t page = (int64_t)1 << a.page_shift;
  for (int b = threadIdx.x; b < a.B; b += kPagesThreads) {
    const int32_t k = a.K[b], len = a.len[b], held = a.held[b];
    const int64_t need = ((int64_t)len + k + page) >> a.page_shift;
    // (pages taken now for tokens that are cached already would hold none of them)
    const bool ok = k >= -1 && len >= 0 && held >= 0 && held <= a.cols && need <= a.cols &&
                    len <= (int64_t)held << a.page_shift;
    if (!ok) bad = 1;
    lens[b] = len;
    helds[b] = held;
    n[b] = ok ? k + 1 : 0;
    x[b] = ok && need > held ? (int32_t)(need - held) : 0;
  }
  const int32_t n_free = *a.n_free;
  __syncthreads();
  const bool fits = scan_requests<2>(a.B, {n, x}, red);
  const int32_t total = n[a.B], extra = x[a.B];
  const bool in_pool = n_free >= 0 && n_free <= a.n_pages && extra <= n_free;
  const bool refused = bad || !fits || total > a.n_rows || !in_pool;
  if (refused && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(a.err, (bad || !fits || total > a.n_rows ? kErrCache : 0) | (in_pool ? 0 : kErrPool));

  // the packed rows (unsigned: the step behind the last row may pass 2^31)
  const unsigned stride = gridDim.x * kPagesThreads;
  for (unsigned u = blockIdx.x * kPagesThreads + threadIdx.x; u < (unsigned)a.n_rows; u += stride) {
    const int i = (int)u;
    int req = -1, pos = -1, slot = -1;
    if (!refused && i < total) {
      req = owner(n, a.B, i);
      const int32_t held = helds[req];
      pos = lens[req] + i - n[req];
      const int p = pos >> a.page_shift;
      const int32_t id =
          p < held ? a.table[req * a.tstride + p] : a.free_list[n_free - 1 - x[req] - (p - held)];
      if ((unsigned)id < (unsigned)a.n_pages)
        slot = (int)((int64_t)id << a.page_shift) + (pos & ((int)page - 1));
      else
        atomicOr(a.err, kErrPage);
    }
    a.row_req[i] = req;
    a.row_pos[i] = pos;
    a.row_slot[i] = slot;
  }
  // the new table entries (none if refused), and the offsets
  if (!refused)
    for (int i = blockIdx.x * kPagesThreads + threadIdx.x; i < extra; i += (int)stride) {
      const int b = owner(x, a.B, i);
      a.table[b * a.tstride + helds[b] + (i - x[b])] = a.free_list[n_free - 1 - i];
    }
  for (int b = blockIdx.x * kPagesThreads + threadIdx.x; b <= a.B; b += (int)stride) a.offs[b] = refused ? 0 : n[b];
  if (!last_workgroup(a.done, &flag, &bad)) return;
  for (int b = threadIdx.x; b < a.B; b += kPagesThreads)
    a.held_out[b] = helds[b] + (refused ? 0 : x[b + 1] - x[b]);
  if (threadIdx.x == 0) *a.n_free_out = refused ? n_free : n_free - extra;
}

// Pages keep .. held - 1 of every request, pushed in request order and by
// ascending place.  What a workgroup pushes stands behind the stack's top until
// the last one raises it, which it does if every id is a page's.
__global__ __launch_bounds__(kPagesThreads) void pages_commit_impl(const PagesArgs a) {
  __shared__ int32_t x[kPagesMaxB + 1], helds[kPagesMaxB];
  __shared__ int64_t red[kPagesThreads / 64][1];
  __shared__ int bad, bad_id, flag;
  if (threadIdx.x == 0) bad = bad_id = 0;
  __syncthreads();
  const int64_t page = (int64_t)1 << a.page_shift;
  auto new_len = [&](int b) -> int64_t {
    return a.finished && a.finished[b] ? 0 : (int64_t)a.len[b] + a.accept[b] + 1;
  };
  for (int b = threadIdx.x; b < a.B; b += kPagesThreads) {
    const int32_t acc = a.accept[b], len = a.len[b], held = a.held[b];
    const int64_t k = (new_len(b) + page - 1) >> a.page_shift;
    const bool ok = acc >= -1 && len >= 0 && held >= 0 && held <= a.cols && k <= held;
    if (!ok) bad = 1;
    helds[b] = held;
    x[b] = ok ? held - (int32_t)k : 0;
  }
  const int32_t n_free = *a.n_free;
  __syncthreads();
  const bool fits = scan_requests<1>(a.B, {x}, red);
  const int32_t given = x[a.B];
  const bool in_pool = n_free >= 0 && n_free <= a.n_pages && given <= a.n_pages - n_free;
  bool refused = bad || !fits || !in_pool;
  if (refused && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(a.err, (bad || !fits ? kErrCache : 0) | (in_pool ? 0 : kErrPool));
  if (!refused)
    for (int i = blockIdx.x * kPagesThreads + threadIdx.x; i < given; i += gridDim.x * kPagesThreads) {
      const int b = owner(x, a.B, i);
      const int32_t id = a.table[b * a.tstride + helds[b] - (x[b + 1] - i)];
      if ((unsigned)id >= (unsigned)a.n_pages) {
        atomicOr(a.err, kErrPage);
        bad_id = 1;
      }
      a.free_list[n_free + i] = id;
    }
  if (!last_workgroup(a.done, &flag, &bad_id)) return;
  refused = refused || bad_id != 0;
  for (int b = threadIdx.x; b < a.B; b += kPagesThreads) {
    const int32_t len = a.len[b], held = helds[b];
    a.len_out[b] = refused ? len : (int32_t)new_len(b);
    a.held_out[b] = refused ? held : held - (x[b + 1] - x[b]);
  }
  if (threadIdx.x == 0) *a.n_free_out = refused ? n_free : n_free + given;
}

}  // namespace

const void* pages_reserve_kernel() { return (const void*)&pages_reserve_impl; }
const void* pages_commit_kernel() { return (const void*)&pages_commit_impl; }

}  // namespace dspark
