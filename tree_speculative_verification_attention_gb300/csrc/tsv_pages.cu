// tsv_pages.cu — page lists against a pool of reference counts: resize, fork,
// compact; and the contents of pages.
//
// The pool is the counts alone: a free page is one whose count is 0, and pages
// are handed out by rising id, so a call's result is a function of its
// arguments.  Finding the k-th free page is a prefix sum over the counts.  One
// cluster does it: its CTAs split the pool (a warp takes a contiguous range, 256
// counts at a time), exchange their totals through distributed shared memory,
// and each then hands out, or moves, what lies in its own range.  Cluster
// barriers stand between the phases, so there is no workspace.  The lists are the
// other half of the work.  Where they, or the pool, are large, what needs no
// common order is done by launches of its own, on all SMs; where they are small,
// one launch does everything, since a call then takes as long as its chain of
// loads and barriers (about 5 us of it the launch and the first two loads).
//
// Measured on the stream (a call alone, in a captured graph):
//   resize  32 requests that take 1 to 4 entries and give them back, 8192 pages:
//           11.5 us for the two calls; 128 requests that take up to 2048 entries
//           each and give them back, 2^20 pages: 37 us for the two
//   fork    8 lists of one of 69 entries 13 us; 128 lists of up to 2048 entries,
//           2^17 pages: 19 us
//   compact 4096 pages 8.8 us; 2^20 pages and 128 lists of up to 8192 entries 26 us
//   copy    8 pages of 32 KB 2.9 us; 4096 of 128 KB 156 us, 6.9 TB/s (what a plain
//           copy reaches)
#include <cuda_runtime.h>

#include "tsv_device.cuh"
#include "tsv_internal.h"

namespace tsv {

namespace {

constexpr int kPoolThreads = 1024, kPoolWarps = 32;
static_assert(kPoolWarps == 32, "scan_counts takes a warp's sum per lane");
static_assert(TSV_MAX_BATCH <= kPoolThreads, "a thread per request");
constexpr int kPoolCtas = 16;  // of a cluster, at most (8 where the device holds no 16)

__device__ __forceinline__ int ld_dsmem_i32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// The counterpart of `p` in CTA `rank` of the cluster.
__device__ __forceinline__ int remote_i32(const int* p, int rank) { return ld_dsmem_i32(mapa_shared(smem_u32(p), (uint32_t)rank)); }

// Four counts from page `at` on (a multiple of 4); pages past the end count as `none`.
__device__ __forceinline__ int4 load_counts(const int32_t* refs, int at, int pages, int none) {
  if (at + 4 <= pages) return __ldcg(reinterpret_cast<const int4*>(refs + at));
  int4 v = make_int4(none, none, none, none);
  if (at < pages) v.x = __ldcg(refs + at);
  if (at + 1 < pages) v.y = __ldcg(refs + at + 1);
  if (at + 2 < pages) v.z = __ldcg(refs + at + 2);
  return v;
}

// Eight counts in a row, from page `at` on (a multiple of 8).
struct EightCounts {
  int c[8];
  __device__ __forceinline__ EightCounts(const int32_t* refs, int at, int pages, int none) {
    const int4 a = load_counts(refs, at, pages, none), b = load_counts(refs, at + 4, pages, none);
    c[0] = a.x;
    c[1] = a.y;
    c[2] = a.z;
    c[3] = a.w;
    c[4] = b.x;
    c[5] = b.y;
    c[6] = b.z;
    c[7] = b.w;
  }
};

// The range of pages of a warp: whole chunks of 256.
struct PoolShare {
  int first, end;
  __device__ __forceinline__ PoolShare(int pages, int warp) : PoolShare(pages, blockIdx.x * kPoolWarps + warp, gridDim.x * kPoolWarps) {}
  __device__ __forceinline__ PoolShare(int pages, int w, int warps) {
    const int chunks = (pages + 255) >> 8;
    first = (int)((int64_t)chunks * w / warps) << 8;
    end = min(pages, (int)((int64_t)chunks * (w + 1) / warps) << 8);
  }
};

// Pages with count 0 (LIVE: above 0) from `first` up to `end`.
template <bool LIVE>
__device__ __forceinline__ int count_pages(const int32_t* refs, int first, int end, int lane) {
  int n = 0;
#pragma unroll 8
  for (int at = first + 4 * lane; at < end; at += 128) {
    const int4 v = load_counts(refs, at, end, LIVE ? 0 : 1);
    n += LIVE ? (v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0) : (v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0);
  }
  return (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
}

// Every warp's count -> what lies before its range, and the whole pool's: the
// warps' sums in shared memory, the CTAs' through the cluster.
struct PoolScan {
  int warp_sum[kPoolWarps];
  int total;
};
__device__ __forceinline__ int scan_counts(PoolScan& s, int mine, int warp, int lane, int* all) {
  if (lane == 0) s.warp_sum[warp] = mine;
  __syncthreads();
  int v = s.warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  const int inside = __shfl_sync(0xffffffffu, v, warp) - mine;
  if (warp == 0 && lane == 31) s.total = v;
  cluster_sync_all();
  int t = lane < gridDim.x ? remote_i32(&s.total, lane) : 0;
  int before = lane < blockIdx.x ? t : 0;
  *all = (int)__reduce_add_sync(0xffffffffu, (unsigned)t);
  before = (int)__reduce_add_sync(0xffffffffu, (unsigned)before);
  return before + inside;
}

// What the requests of a call want, the same in every CTA.
struct PoolRequests {
  int32_t held[TSV_MAX_BATCH], want[TSV_MAX_BATCH], need[TSV_MAX_BATCH], upto[TSV_MAX_BATCH];
  int32_t bad[TSV_MAX_BATCH];  // (of the CTA's own requests)
  PoolScan scan;
  int32_t needed;              // by all requests
  int32_t granted;
};

// upto[b]: pages needed up to and with request b (one warp).
__device__ __forceinline__ void sum_needs(PoolRequests& r, int B, int lane) {
  int64_t before = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    int64_t v = b0 + lane < B ? r.need[b0 + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (b0 + lane < B) r.upto[b0 + lane] = (int32_t)min(before + v, (int64_t)INT32_MAX);  // (more than any pool holds)
    before += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) r.needed = (int32_t)min(before, (int64_t)INT32_MAX);
}

// Whether request b gets what it needs out of `free` pages.
__device__ __forceinline__ bool is_served(const PoolRequests& r, int b, int free) { return r.need[b] == 0 || r.upto[b] <= free; }

// Hands out the free pages of the warp's range, the first of which is the pool's
// `rank`-th: give(b, k, id) for page k of request b's need.
template <typename Give>
__device__ __forceinline__ void hand_out(PoolRequests& r, const tsv_page_pool& pool, const PoolShare& share, int rank, int granted, int B,
                                         int lane, Give give) {
  EightCounts now(pool.refs_d, share.first + 8 * lane, share.end, 1);
#pragma unroll 1
  for (int at = share.first; at < share.end && rank < granted; at += 256) {
    const int page = at + 8 * lane;
    const EightCounts next(pool.refs_d, page + 256, share.end, 1);  // on its way meanwhile
    uint32_t f = 0u;  // free pages of the lane
#pragma unroll
    for (int e = 0; e < 8; ++e) f |= (now.c[e] == 0 ? 1u : 0u) << e;
    const int n = __popc(f);
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    int k = rank + upto - n;
    if (n > 0 && k < granted) {
      int lo = 0, hi = B - 1;  // the first request with upto > k
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (r.upto[mid] > k) hi = mid;
        else lo = mid + 1;
      }
      for (; f && k < granted; f &= f - 1, ++k) {
        while (r.upto[lo] <= k) ++lo;
        const int id = page + __ffs(f) - 1;
        pool.refs_d[id] = 1;
        give(lo, k - (r.upto[lo] - r.need[lo]), id);
      }
    }
    rank += __shfl_sync(0xffffffffu, upto, 31);
    now = next;
  }
}

// Entries from `first` up to `end` of a list by `threads` threads, U of a thread
// in flight: for_entries hands f the ids (-1: none) and their places.
constexpr int kFlight = 8;
template <typename F>
__device__ __forceinline__ void for_entries(const int32_t* ids, int first, int end, int t, int threads, F f) {
#pragma unroll 1
  for (int i = first + t; i < end; i += kFlight * threads) {
    int32_t id[kFlight];
    bool on[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      on[q] = i + q * threads < end;
      id[q] = on[q] ? __ldcg(ids + i + q * threads) : -1;
    }
    f(id, on, i);
  }
}
// Whether all are pages that some list holds.
__device__ __forceinline__ bool entries_held(const tsv_page_pool& p, const int32_t* ids, int first, int end, int t, int threads) {
  bool fine = true;
  for_entries(ids, first, end, t, threads, [&](const int32_t (&id)[kFlight], const bool (&on)[kFlight], int) {
    int32_t count[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) count[q] = (uint32_t)id[q] < (uint32_t)p.num_pages ? __ldcg(p.refs_d + id[q]) : 0;
#pragma unroll
    for (int q = 0; q < kFlight; ++q) fine &= !on[q] || count[q] > 0;
  });
  return fine;
}
// One reference less of each (valid ids); false when one was not held, whose count
// then stays what it was.
__device__ __forceinline__ bool drop_entries(const tsv_page_pool& p, const int32_t* ids, int first, int end, int t, int threads) {
  bool fine = true;
  for_entries(ids, first, end, t, threads, [&](const int32_t (&id)[kFlight], const bool (&on)[kFlight], int) {
    int32_t before[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) before[q] = on[q] ? atomicSub(p.refs_d + id[q], 1) : 1;
#pragma unroll
    for (int q = 0; q < kFlight; ++q)
      if (before[q] <= 0) {
        atomicAdd(p.refs_d + id[q], 1);
        fine = false;
      }
  });
  return fine;
}

// Entries `first` up to `end` of list b become those of its source, shared.
__device__ __forceinline__ void share_entries(const PagesForkArgs& a, int b, int source, int first, int end, int t, int threads) {
  int32_t* list = const_cast<int32_t*>(a.to.ids_d) + (int64_t)b * a.to.stride;
  for_entries(a.from.ids_d + (int64_t)source * a.from.stride, first, end, t, threads,
              [&](const int32_t (&id)[kFlight], const bool (&on)[kFlight], int i) {
#pragma unroll
                for (int q = 0; q < kFlight; ++q) {
                  if (!on[q]) continue;
                  list[i + q * threads] = id[q];
                  atomicAdd(a.pool.refs_d + id[q], 1);
                }
              });
}

// The cluster's requests are shared out: request b belongs to CTA b % CTAs, and
// there to a group of warps.  for_own(b, t, threads) runs on each of them.
template <typename F>
__device__ __forceinline__ void for_own(int B, int warp, int lane, F f) {
  const int own = (B - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // requests of this CTA
  if (own <= 0) return;
  const int group = max(1, kPoolWarps / own);  // warps of a request
  for (int i = warp / group; i < own; i += kPoolWarps / group)
    f((int)blockIdx.x + i * (int)gridDim.x, (warp % group) * 32 + lane, group * 32);
}

__global__ void __launch_bounds__(kPoolThreads, 1) pages_resize_kernel(const PagesResizeArgs a) {
  __shared__ PoolRequests r;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  bool shrinks = false;
  if (tid < a.B) {
    const int held = __ldcg(a.pages + tid), rows = __ldg(a.rows + tid);
    const int want = rows / a.page_size + (rows % a.page_size > 0 ? 1 : 0);
    const bool bad = held < 0 || held > a.table.pages || rows < 0 || want > a.table.pages;
    r.held[tid] = held;
    r.want[tid] = want;
    r.need[tid] = bad ? 0 : max(0, want - held);
    r.bad[tid] = bad;
    shrinks = !bad && want < held;
  }
  shrinks = __syncthreads_or(shrinks);  // the same in every CTA
  if (warp == 0) sum_needs(r, a.B, lane);
  if (shrinks) {
    for_own(a.B, warp, lane, [&](int b, int t, int threads) {
      if (r.bad[b] || r.want[b] >= r.held[b]) return;
      const int32_t* ids = a.table.ids_d + (int64_t)b * a.table.stride;
      bool bad = false;
      bad |= !entries_held(a.pool, ids, r.want[b], r.held[b], t, threads);
      if (t == 0 && __ldg(a.rows + b) % a.page_size > 0) {  // new rows would go to the last page
        const int32_t id = __ldcg(ids + r.want[b] - 1);
        bad |= (uint32_t)id >= (uint32_t)a.pool.num_pages || __ldcg(a.pool.refs_d + id) != 1;
      }
      if (bad) atomicOr(&r.bad[b], 2);
    });
    cluster_sync_all();  // every look at the counts comes before the first change
    for_own(a.B, warp, lane, [&](int b, int t, int threads) {
      if (r.bad[b] & 3 || r.want[b] >= r.held[b]) return;
      const int32_t* ids = a.table.ids_d + (int64_t)b * a.table.stride;
      if (!drop_entries(a.pool, ids, r.want[b], r.held[b], t, threads)) atomicOr(&r.bad[b], 4);  // (listed more often than counted)
    });
    cluster_sync_all();  // (its release and acquire cover global memory among the cluster's threads)
  } else {
    __syncthreads();
  }
  int free = 0;
  if (r.needed > 0) {
    const PoolShare share(a.pool.num_pages, warp);
    const int mine = count_pages<false>(a.pool.refs_d, share.first, share.end, lane);
    const int rank = scan_counts(r.scan, mine, warp, lane, &free);
    if (tid == 0) r.granted = 0;
    __syncthreads();
    if (tid < a.B && is_served(r, tid, free)) atomicMax(&r.granted, r.need[tid] ? r.upto[tid] : 0);
    __syncthreads();
    hand_out(r, a.pool, share, rank, r.granted, a.B, lane, [&](int b, int k, int id) {
      const_cast<int32_t*>(a.table.ids_d)[(int64_t)b * a.table.stride + r.held[b] + k] = id;
    });
  }
  if (tid < a.B && tid % gridDim.x == blockIdx.x) {
    const bool bad = r.bad[tid] & 3, served = is_served(r, tid, free);
    if (!bad && served) a.pages[tid] = r.want[tid];
    a.status[tid] = r.bad[tid] ? TSV_ERR_INVALID_ARG : served ? TSV_OK : TSV_ERR_NO_PAGES;
  }
  cluster_sync_all();  // the others have read this CTA's total
}

// A fork of many entries is three launches, so that the lists' part of it runs on as
// many SMs as there are lists: give back (kForkBack), the pages of the lists' own
// (kForkTake), share (pages_share_kernel).  With few entries one cluster does it all.
// (What a list gives back may be looked at while others are looked over: a page that
// a list holds has a count above 0 whatever the others do.)
enum { kForkAll = 0, kForkTake = 1 };

// List b of a fork: what it wants; whether the numbers fit.
struct ForkList {
  int held, full, part, source;  // source -1: stays as it is
  bool bad;
  __device__ __forceinline__ ForkList(const PagesForkArgs& a, int b) {
    const int rows = __ldg(a.rows + b);
    held = __ldcg(a.to_pages + b);
    source = __ldg(a.source + b);
    full = rows / a.page_size;
    part = rows % a.page_size > 0 ? 1 : 0;
    bad = source < -1 || source >= a.F || (source >= 0 && (rows < 0 || held < 0 || held > a.to.pages));
    if (source >= 0 && !bad) {
      const int has = __ldg(a.from_pages + source);
      bad = has < 0 || has > a.from.pages || full + part > has || full + part > a.to.pages;
    }
  }
};

__global__ void __launch_bounds__(kPoolThreads, 1) pages_give_back_kernel(const PagesForkArgs a) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  const int b = blockIdx.x, t = threadIdx.x;
  const ForkList l(a, b);
  bool bad = l.bad;
  if (!bad && l.source >= 0) {
    const int32_t* old = a.to.ids_d + (int64_t)b * a.to.stride;
    const int32_t* ids = a.from.ids_d + (int64_t)l.source * a.from.stride;
    bool fine = entries_held(a.pool, old, 0, l.held, t, kPoolThreads) & entries_held(a.pool, ids, 0, l.full + l.part, t, kPoolThreads);
    bad = __syncthreads_or(!fine);
    if (!bad && !drop_entries(a.pool, old, 0, l.held, t, kPoolThreads)) bad = true;
    // (2: listed more often than counted.  Its other pages went back: the list is empty.)
    const bool over = __syncthreads_or(bad) && !__syncthreads_or(!fine);
    if (t == 0) a.status[b] = over ? 2 : bad ? 1 : 0;
    return;
  }
  if (t == 0) a.status[b] = bad ? 1 : 0;
}

template <int KIND>
__global__ void __launch_bounds__(kPoolThreads, 1) pages_fork_kernel(const PagesForkArgs a) {
  __shared__ PoolRequests r;
  __shared__ int32_t source[TSV_MAX_BATCH], full[TSV_MAX_BATCH];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  if (tid < a.B) {
    const ForkList l(a, tid);
    int bad = l.bad ? 1 : 0;
    if (KIND == kForkTake) {
      const int found = __ldcg(a.status + tid);
      bad = found == 2 ? 4 : found;
    }
    r.held[tid] = l.held;
    r.want[tid] = l.full + l.part;
    full[tid] = l.full;
    source[tid] = bad & 3 ? -1 : l.source;
    r.need[tid] = bad || l.source < 0 ? 0 : l.part;
    r.bad[tid] = bad;
  }
  __syncthreads();
  if (KIND == kForkAll) {
    for_own(a.B, warp, lane, [&](int b, int t, int threads) {
      if (source[b] < 0) return;
      const int32_t* old = a.to.ids_d + (int64_t)b * a.to.stride;
      const int32_t* ids = a.from.ids_d + (int64_t)source[b] * a.from.stride;
      const bool fine = entries_held(a.pool, old, 0, r.held[b], t, threads) & entries_held(a.pool, ids, 0, r.want[b], t, threads);
      if (!fine) atomicOr(&r.bad[b], 2);
    });
    __syncthreads();
    for_own(a.B, warp, lane, [&](int b, int t, int threads) {
      if (source[b] < 0 || (r.bad[b] & 3)) return;
      const int32_t* old = a.to.ids_d + (int64_t)b * a.to.stride;
      if (!drop_entries(a.pool, old, 0, r.held[b], t, threads)) atomicOr(&r.bad[b], 4);  // (listed more often than counted)
    });
    cluster_sync_all();  // (its release and acquire cover global memory among the cluster's threads)
    // What the owners found: the needs are the same in every CTA.
    if (tid < a.B) {
      const int bad = remote_i32(&r.bad[tid], tid % gridDim.x);
      if (bad & 3) source[tid] = -1;
      if (bad) r.need[tid] = 0;
    }
    __syncthreads();
  }
  if (warp == 0) sum_needs(r, a.B, lane);
  __syncthreads();
  int free = 0;
  const PoolShare share(a.pool.num_pages, warp);
  if (r.needed > 0) {
    const int mine = count_pages<false>(a.pool.refs_d, share.first, share.end, lane);
    const int rank = scan_counts(r.scan, mine, warp, lane, &free);  // (a barrier of the cluster: counts are read before pages are shared)
    if (tid == 0) r.granted = 0;
    __syncthreads();
    if (tid < a.B && is_served(r, tid, free)) atomicMax(&r.granted, r.need[tid] ? r.upto[tid] : 0);
    __syncthreads();
    // (A page that becomes shared below has another holder: its count is never 0.)
    hand_out(r, a.pool, share, rank, r.granted, a.B, lane, [&](int b, int, int id) {
      const_cast<int32_t*>(a.to.ids_d)[(int64_t)b * a.to.stride + full[b]] = id;
      a.copy_src[b] = __ldg(a.from.ids_d + (int64_t)source[b] * a.from.stride + full[b]);
      a.copy_dst[b] = id;
    });
  }
  if (KIND == kForkTake && r.needed == 0) cluster_sync_all();  // every CTA has read the status words that are written below
  if (KIND == kForkAll) {
    for_own(a.B, warp, lane, [&](int b, int t, int threads) {
      if (source[b] < 0 || r.bad[b] || !is_served(r, b, free)) return;
      share_entries(a, b, source[b], 0, full[b], t, threads);
    });
  }
  if (tid < a.B && tid % gridDim.x == blockIdx.x) {
    const int bad = r.bad[tid];
    const bool served = is_served(r, tid, free);
    if (source[tid] >= 0) a.to_pages[tid] = served && !bad ? r.want[tid] : 0;
    if (source[tid] < 0 || !served || r.need[tid] == 0) {
      a.copy_src[tid] = -1;
      a.copy_dst[tid] = -1;
    }
    a.status[tid] = bad ? TSV_ERR_INVALID_ARG : served ? TSV_OK : TSV_ERR_NO_PAGES;
  }
  cluster_sync_all();  // the others have read this CTA's flags and total
}

// The whole pages of the lists that the launch before served, 8192 entries a CTA.
constexpr int kShareEntries = kPoolThreads * kFlight;
__global__ void __launch_bounds__(kPoolThreads, 1) pages_share_kernel(const PagesForkArgs a, int chunks) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  const int b = blockIdx.x / chunks, first = (blockIdx.x - b * chunks) * kShareEntries;
  if (__ldcg(a.status + b) != TSV_OK) return;
  const ForkList l(a, b);
  if (l.source >= 0) share_entries(a, b, l.source, first, min(l.full, first + kShareEntries), threadIdx.x, kPoolThreads);
}

// Counts and new ids of the pages that move, thread t of `threads`.
constexpr int kMoveThreads = 256;
__device__ __forceinline__ void move_counts(const PagesCompactArgs& a, int moved, int t, int threads) {
  constexpr int U = 4;
#pragma unroll 1
  for (int i = t; i < moved; i += U * threads) {
    int src[U], dst[U], count[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const bool on = i + q * threads < moved;
      src[q] = on ? __ldcg(a.move_src + i + q * threads) : -1;
      dst[q] = on ? __ldcg(a.move_dst + i + q * threads) : -1;
    }
#pragma unroll
    for (int q = 0; q < U; ++q) count[q] = src[q] >= 0 ? __ldcg(a.pool.refs_d + src[q]) : 0;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (src[q] < 0) continue;
      a.new_id[src[q]] = dst[q];
      a.refs_out[src[q]] = 0;
      a.refs_out[dst[q]] = count[q];
    }
  }
}

// The holes below L and the pages in use from L on, by rising id, and what does not
// move, of a warp's share; `before` pages in use lie in front of it, `kept` below L.
__device__ __forceinline__ void place_pages(const PagesCompactArgs& a, const PoolShare& share, int before, int L, int kept, int lane) {
  int live = before;  // pages in use before the current one
  const bool aligned = ((reinterpret_cast<uintptr_t>(a.new_id) | reinterpret_cast<uintptr_t>(a.refs_out)) & 15) == 0;
  EightCounts now(a.pool.refs_d, share.first + 8 * lane, share.end, 0);
#pragma unroll 1
  for (int at = share.first; at < share.end; at += 256) {
    const int page = at + 8 * lane;
    const EightCounts next(a.pool.refs_d, page + 256, share.end, 0);  // on its way meanwhile
    int n = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) n += now.c[e] > 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    int k = live + upto - n;
    // New ids and counts that are known already; a hole's count and a moved page's id
    // come below.
    int id_out[8], count_out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int id = page + e;
      const bool used = now.c[e] > 0, low = id < L;
      id_out[e] = used && low ? id : -1;
      count_out[e] = low || !used ? now.c[e] : 0;
      if (id < share.end) {
        if (low && !used) a.move_dst[id - k] = id;
        if (!low && used) a.move_src[k - kept] = id;
      }
      k += used;
    }
    // (A moved page's count is still to be read when the counts are written in place.)
    const bool in_place = a.refs_out == a.pool.refs_d;
    if (page + 8 <= share.end) {
      int4* to_id = reinterpret_cast<int4*>(a.new_id + page);
      if (aligned) {
        to_id[0] = make_int4(id_out[0], id_out[1], id_out[2], id_out[3]);
        to_id[1] = make_int4(id_out[4], id_out[5], id_out[6], id_out[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a.new_id[page + e] = id_out[e];
      }
      if (!in_place) {
        int4* to_count = reinterpret_cast<int4*>(a.refs_out + page);
        if (aligned) {
          to_count[0] = make_int4(count_out[0], count_out[1], count_out[2], count_out[3]);
          to_count[1] = make_int4(count_out[4], count_out[5], count_out[6], count_out[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) a.refs_out[page + e] = count_out[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (page + e >= share.end) break;
        a.new_id[page + e] = id_out[e];
        if (!in_place) a.refs_out[page + e] = count_out[e];
      }
    }
    live += __shfl_sync(0xffffffffu, upto, 31);
    now = next;
  }
}

// The same by as many CTAs as hold four warps each, of `warps` that shared the counts.
constexpr int kPlaceWarps = 4;
__global__ void __launch_bounds__(32 * kPlaceWarps) pages_place_kernel(const PagesCompactArgs a, int warps) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const PoolShare share(a.pool.num_pages, blockIdx.x * kPlaceWarps + (threadIdx.x >> 5), warps);
  if (share.first >= share.end) return;
  const int before = __ldcg(a.new_id + share.first), L = __ldcg(a.new_id + share.first + 1), kept = L - __ldcg(a.moved);
  __syncwarp();  // (read by every lane before they are written)
  place_pages(a, share, before, L, kept, lane);
}

// SPLIT: counting alone; placing and moving are launches of their own.
template <bool SPLIT>
__global__ void __launch_bounds__(kPoolThreads, 1) pages_compact_kernel(const PagesCompactArgs a) {
  __shared__ PoolScan scan;
  __shared__ int below;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  const int pages = a.pool.num_pages;
  const PoolShare share(pages, warp);
  int L = 0;
  const int before = scan_counts(scan, count_pages<true>(a.pool.refs_d, share.first, share.end, lane), warp, lane, &L);
  // Pages in use below L: the warp whose range holds page L knows (the last one
  // when every page is in use), and tells every CTA.
  const bool last = blockIdx.x == gridDim.x - 1 && warp == kPoolWarps - 1;
  if ((share.first <= L && L < share.end) || (last && L == pages)) {
    const int n = before + count_pages<true>(a.pool.refs_d, share.first, min(L, share.end), lane);
    if (lane < gridDim.x)
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&below), (uint32_t)lane)), "r"(n) : "memory");
  }
  cluster_sync_all();
  const int kept = below, moved = L - kept;
  if (blockIdx.x == 0 && tid == 0) *a.moved = moved;
  if (blockIdx.x == 0 && tid < a.n) a.status[tid] = TSV_OK;
  if (SPLIT) {  // on to pages_place_kernel, in the words that it writes
    if (lane == 0 && share.first < share.end) {
      a.new_id[share.first] = before;
      a.new_id[share.first + 1] = L;  // (a share has 256 pages at least, but for a last one of two chunks at least)
    }
    return;
  }
  place_pages(a, share, before, L, kept, lane);
  cluster_sync_all();  // (its release and acquire cover global memory among the cluster's threads)
  move_counts(a, moved, blockIdx.x * kPoolThreads + tid, gridDim.x * kPoolThreads);
}

__global__ void __launch_bounds__(kMoveThreads) pages_move_kernel(const PagesCompactArgs a) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  move_counts(a, __ldg(a.moved), blockIdx.x * kMoveThreads + threadIdx.x, gridDim.x * kMoveThreads);
}

// Entries of the lists under their new ids: a CTA per row and 4096 entries.
constexpr int kRemapThreads = 512, kRemapEntries = 4096;
__global__ void __launch_bounds__(kRemapThreads) pages_remap_kernel(const PagesCompactArgs a, int chunks) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  int row = blockIdx.x / chunks, t = 0;
  const int first = (blockIdx.x - row * chunks) * kRemapEntries;
  while (row >= a.lists[t].B) row -= a.lists[t++].B;
  const tsv_page_lists& l = a.lists[t];
  const int held = __ldg(l.pages_d + row);
  bool bad = held < 0 || held > l.table.pages;
  if (!bad) {
    const int32_t* from = l.table.ids_d + (int64_t)row * l.table.stride;
    int32_t* to = l.out_d + (int64_t)row * l.out_stride;
    const int end = min(held, first + kRemapEntries);
#pragma unroll 4
    for (int i = first + threadIdx.x; i < end; i += kRemapThreads) {
      const int32_t id = from[i];
      const int32_t now = (uint32_t)id < (uint32_t)a.pool.num_pages ? __ldg(a.new_id + id) : -1;
      bad |= now < 0;
      to[i] = now;
    }
  }
  if (bad) a.status[t] = TSV_ERR_INVALID_ARG;
}

// CTAs of a call's cluster: one per two steps of 32 warps x 256 counts, or per
// 8192 entries that the lists have room for.
int pool_ctas(int32_t num_pages, int64_t entries, int most) {
  int n = 1;
  while (n < most && (num_pages > n * 16384 || entries > n * (int64_t)8192)) n *= 2;
  return n;
}

// From where on a call is several launches.  128 lists with room for 2048 entries each
// (262144): 40 us as one launch, 19 as three; 8 lists of 69: 12.9 us and 12.1, but 9.6
// and 12.6 of the host's time.  A compaction of 2^20 pages: 52 us as one launch, 26 as
// three; of 4096: 8.8 and 8.6, and 11.8 and 15.4 of the host's.
constexpr int64_t kForkSplit = 32768;  // entries that the lists have room for
constexpr int kCompactSplit = 131072;  // pages

}  // namespace

int pages_cluster_limit() {
  // Clusters of 16 have to be asked for, kernel by kernel.
  int most = kPoolCtas;
  const void* kernels[5] = {reinterpret_cast<const void*>(pages_resize_kernel), reinterpret_cast<const void*>(pages_fork_kernel<kForkAll>),
                            reinterpret_cast<const void*>(pages_fork_kernel<kForkTake>),
                            reinterpret_cast<const void*>(pages_compact_kernel<false>),
                            reinterpret_cast<const void*>(pages_compact_kernel<true>)};
  for (const void* k : kernels) {
    int fit = 0;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(kPoolCtas);
      cfg.blockDim = dim3(kPoolThreads);
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = kPoolCtas;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&fit, k, &cfg) != cudaSuccess) fit = 0;
    }
    if (fit < 1) {
      cudaGetLastError();
      most = 8;
    }
  }
  return most;
}

cudaError_t launch_pages_resize(const PagesResizeArgs& a, int most, cudaStream_t st) {
  const int n = pool_ctas(a.pool.num_pages, (int64_t)a.B * a.table.pages, most);
  return launch_pdl(pages_resize_kernel, dim3(n), dim3(kPoolThreads), 0, st, (unsigned)n, a);
}

cudaError_t launch_pages_fork(const PagesForkArgs& a, int most, cudaStream_t st) {
  const int64_t entries = (int64_t)a.B * a.to.pages;
  if (entries <= kForkSplit) {
    const int n = pool_ctas(a.pool.num_pages, entries, most);
    return launch_pdl(pages_fork_kernel<kForkAll>, dim3(n), dim3(kPoolThreads), 0, st, (unsigned)n, a);
  }
  cudaError_t e = launch_pdl(pages_give_back_kernel, dim3(a.B), dim3(kPoolThreads), 0, st, 0u, a);
  if (e != cudaSuccess) return e;
  const int n = pool_ctas(a.pool.num_pages, 0, most);
  e = launch_pdl(pages_fork_kernel<kForkTake>, dim3(n), dim3(kPoolThreads), 0, st, (unsigned)n, a);
  if (e != cudaSuccess) return e;
  const int chunks = (a.to.pages + kShareEntries - 1) / kShareEntries;
  return launch_pdl(pages_share_kernel, dim3(a.B * chunks), dim3(kPoolThreads), 0, st, 0u, a, chunks);
}

cudaError_t launch_pages_compact(const PagesCompactArgs& a, int most, int num_sms, cudaStream_t st) {
  const int n = pool_ctas(a.pool.num_pages, 0, most);
  const bool split = a.pool.num_pages > kCompactSplit;
  cudaError_t e = split ? launch_pdl(pages_compact_kernel<true>, dim3(n), dim3(kPoolThreads), 0, st, (unsigned)n, a)
                        : launch_pdl(pages_compact_kernel<false>, dim3(n), dim3(kPoolThreads), 0, st, (unsigned)n, a);
  if (e == cudaSuccess && split)
    e = launch_pdl(pages_place_kernel, dim3(n * kPoolWarps / kPlaceWarps), dim3(32 * kPlaceWarps), 0, st, 0u, a, n * kPoolWarps);
  if (e == cudaSuccess && split) e = launch_pdl(pages_move_kernel, dim3(2 * num_sms), dim3(kMoveThreads), 0, st, 0u, a);
  if (e != cudaSuccess || a.n == 0) return e;
  int64_t rows = 0;
  int32_t width = 1;
  for (int t = 0; t < a.n; ++t) {
    rows += a.lists[t].B;
    width = width > a.lists[t].table.pages ? width : a.lists[t].table.pages;
  }
  const int64_t chunks = ((int64_t)width + kRemapEntries - 1) / kRemapEntries;
  if (rows * chunks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(pages_remap_kernel, dim3((unsigned)(rows * chunks)), dim3(kRemapThreads), 0, st, 0u, a, (int)chunks);
}

// ---------------------------------------------------------------- contents

namespace {

// Address of 16-byte vector v of a page: runs of run16 vectors, n1 of them s1
// apart, and those s0 apart.
struct PageShape {
  int32_t run16, n1;
  int64_t s1, s0;
  int32_t vectors;
};

constexpr int kCopyThreads = 256, kCopyBatch = 8;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PagesCopyArgs a, const PageShape shape) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  const tsv_paged_cache& c = a.cache;
  const int tid = threadIdx.x;
  int n = a.n;
  if (a.count) n = max(0, min(n, __ldg(a.count)));
  if (blockIdx.x == gridDim.x - 1) {  // the ids are checked once
    bool bad = false;
#pragma unroll 8
    for (int i = tid; i < n; i += kCopyThreads) {
      const int32_t s = __ldg(a.src + i), d = __ldg(a.dst + i);
      bad |= (s != -1 && (uint32_t)s >= (uint32_t)c.num_pages) || (d != -1 && (uint32_t)d >= (uint32_t)c.num_pages);
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) *a.status = bad ? TSV_ERR_INVALID_ARG : TSV_OK;
  }
  constexpr int kPart = kCopyThreads * kCopyBatch;  // vectors of a part
  const int parts = (shape.vectors + kPart - 1) / kPart;
  const int64_t units = 2ll * n * parts;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t pk = u / parts;
    const int part = (int)(u - pk * parts), pair = (int)(pk >> 1);
    const bool is_v = pk & 1;
    const int32_t s = __ldg(a.src + pair), d = __ldg(a.dst + pair);
    if ((uint32_t)s >= (uint32_t)c.num_pages || (uint32_t)d >= (uint32_t)c.num_pages) continue;
    const uint8_t* base = static_cast<const uint8_t*>(is_v ? c.v_d : c.k_d);
    const uint8_t* from = base + (int64_t)s * c.stride_page;
    uint8_t* to = const_cast<uint8_t*>(base) + (int64_t)d * c.stride_page;
    uint4 x[kCopyBatch];
    int64_t at[kCopyBatch];
#pragma unroll
    for (int q = 0; q < kCopyBatch; ++q) {
      const int v = part * kPart + q * kCopyThreads + tid;
      at[q] = -1;
      if (v >= shape.vectors) continue;
      const int run = v / shape.run16, row = run / shape.n1;
      at[q] = 16ll * (v - run * shape.run16) + (run - row * shape.n1) * shape.s1 + row * shape.s0;
      x[q] = __ldcs(reinterpret_cast<const uint4*>(from + at[q]));
    }
#pragma unroll
    for (int q = 0; q < kCopyBatch; ++q)
      if (at[q] >= 0) __stcs(reinterpret_cast<uint4*>(to + at[q]), x[q]);
    if (part == 0) {
      float* scale = is_v ? c.v_scale_d : c.k_scale_d;
      for (int g = tid; g < c.Hkv; g += kCopyThreads) scale[(int64_t)d * c.Hkv + g] = scale[(int64_t)s * c.Hkv + g];
    }
  }
}

}  // namespace

cudaError_t launch_pages_copy(const PagesCopyArgs& a, int num_sms, cudaStream_t st) {
  const tsv_paged_cache& c = a.cache;
  // Rows and heads by rising stride; neighbours that lie next to each other are one run.
  PageShape s{};
  const bool heads_inside = c.stride_head <= c.stride_row;
  int64_t run = c.D, n1 = heads_inside ? c.Hkv : c.page_size, n0 = heads_inside ? c.page_size : c.Hkv;
  s.s1 = heads_inside ? c.stride_head : c.stride_row;
  s.s0 = heads_inside ? c.stride_row : c.stride_head;
  if (s.s1 == run || n1 == 1) {
    run *= n1;
    n1 = n0;
    s.s1 = s.s0;
    s.s0 = 0;
    n0 = 1;
    if (s.s1 == run || n1 == 1) {
      run *= n1;
      n1 = 1;
    }
  }
  s.run16 = (int32_t)(run / 16);
  s.n1 = (int32_t)n1;
  s.vectors = (int32_t)((int64_t)c.page_size * c.Hkv * c.D / 16);
  const int64_t parts = (s.vectors + kCopyThreads * kCopyBatch - 1) / (kCopyThreads * kCopyBatch);
  // Few units a CTA, so that CTAs that start keep loads going while others store: 4096
  // pages of 128 KB take 183 us with 8 CTAs an SM in the grid, 156 with 64.  (Not one a
  // unit: a.n may be far above the count on the device.)
  const int64_t units = 2ll * a.n * parts, most = (int64_t)num_sms * 64;
  const int grid = (int)(units < 1 ? 1 : units < most ? units : most);
  return launch_pdl(pages_copy_kernel, dim3(grid), dim3(kCopyThreads), 0, st, 0u, a, s);
}

}  // namespace tsv
