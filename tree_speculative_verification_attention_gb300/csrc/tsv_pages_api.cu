// tsv_pages_api.cu — the C ABI declared in include/tsv_pages.h: argument checks
// and launches.  Nothing is allocated here.
#include <cuda_runtime.h>

#include "tsv_internal.h"

using namespace tsv;

namespace {

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
tsv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TSV_OK : TSV_ERR_CUDA; }

tsv_status check_pool(const tsv_page_pool* p) {
  if (!p || !p->refs_d || addr(p->refs_d) % 16 || p->num_pages < 1) return TSV_ERR_INVALID_ARG;
  return p->num_pages > (1 << 27) ? TSV_ERR_UNSUPPORTED : TSV_OK;
}

tsv_status check_lists(const tsv_page_table* t, int64_t rows) {
  if (!t || !t->ids_d || addr(t->ids_d) % 4 || t->pages < 1) return TSV_ERR_INVALID_ARG;
  if (rows > 1 && t->stride < t->pages) return TSV_ERR_INVALID_ARG;
  return t->pages > TSV_PAGED_MAX_ROWS ? TSV_ERR_UNSUPPORTED : TSV_OK;
}

// n / d of d > 0, rounded down.
__int128 floor_div(__int128 n, int64_t d) { return n / d - (n % d < 0 ? 1 : 0); }

// Whether two sets of lists have an entry in common (rows of one table may take turns, or
// its columns be split): for each row of b, whether a row of a begins before its end and
// ends behind its beginning.
bool lists_meet(const tsv_page_table& a, int64_t ra, const tsv_page_table& b, int64_t rb) {
  const int64_t stride = ra > 1 ? a.stride : a.pages;
  const __int128 first = ((__int128)addr(b.ids_d) - (__int128)addr(a.ids_d)) / 4;  // (both are multiples of 4)
  if (first >= (__int128)(ra - 1) * stride + a.pages || (rb > 1 ? (__int128)(rb - 1) * b.stride : 0) + b.pages <= -first)
    return false;  // one set ends before the other: as a rule
  for (int64_t j = 0; j < rb; ++j) {
    const __int128 at = first + (__int128)j * b.stride;
    const __int128 lo = floor_div(at - a.pages, stride) + 1, hi = floor_div(at + b.pages - 1, stride);
    if ((lo > 0 ? lo : 0) <= (hi < ra - 1 ? hi : ra - 1)) return true;
  }
  return false;
}

int cluster_of(tsv_handle h) {  // (the handle's device is current)
  if (h->pages_cluster == 0) h->pages_cluster = pages_cluster_limit();
  return h->pages_cluster;
}

}  // namespace

extern "C" {

tsv_status tsv_pages_resize(tsv_handle h, const tsv_page_pool* pool, const tsv_page_table* table, int32_t* pages_d,
                            const int32_t* rows_d, int32_t B, int32_t page_size, int32_t* status_d, void* stream) {
  if (!h || B < 1 || B > TSV_MAX_BATCH || page_size < 1 || !pages_d || !rows_d || !status_d) return TSV_ERR_INVALID_ARG;
  tsv_status st = check_pool(pool);
  if (st == TSV_OK) st = check_lists(table, B);
  if (st != TSV_OK) return st;
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  PagesResizeArgs a{};
  a.pool = *pool;
  a.table = *table;
  a.pages = pages_d;
  a.rows = rows_d;
  a.B = B;
  a.page_size = page_size;
  a.status = status_d;
  return cuda_status(launch_pages_resize(a, cluster_of(h), static_cast<cudaStream_t>(stream)));
}

tsv_status tsv_pages_fork(tsv_handle h, const tsv_page_pool* pool, const tsv_page_table* from, const int32_t* from_pages_d,
                          int32_t F, const int32_t* source_d, const int32_t* rows_d, const tsv_page_table* to,
                          int32_t* to_pages_d, int32_t B, int32_t page_size, int32_t* copy_src_d, int32_t* copy_dst_d,
                          int32_t* status_d, void* stream) {
  if (!h || B < 1 || B > TSV_MAX_BATCH || F < 1 || F > 65536 || page_size < 1) return TSV_ERR_INVALID_ARG;
  if (!from_pages_d || !source_d || !rows_d || !to_pages_d || !copy_src_d || !copy_dst_d || !status_d) return TSV_ERR_INVALID_ARG;
  tsv_status st = check_pool(pool);
  if (st == TSV_OK) st = check_lists(from, F);
  if (st == TSV_OK) st = check_lists(to, B);
  if (st != TSV_OK) return st;
  if (lists_meet(*from, F, *to, B) || copy_src_d == copy_dst_d) return TSV_ERR_INVALID_ARG;
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  PagesForkArgs a{};
  a.pool = *pool;
  a.from = *from;
  a.to = *to;
  a.from_pages = from_pages_d;
  a.to_pages = to_pages_d;
  a.source = source_d;
  a.rows = rows_d;
  a.F = F;
  a.B = B;
  a.page_size = page_size;
  a.copy_src = copy_src_d;
  a.copy_dst = copy_dst_d;
  a.status = status_d;
  return cuda_status(launch_pages_fork(a, cluster_of(h), static_cast<cudaStream_t>(stream)));
}

tsv_status tsv_pages_compact(tsv_handle h, const tsv_page_pool* pool, int32_t* refs_out_d, const tsv_page_lists* lists,
                             int32_t n, int32_t* new_id_d, int32_t* move_src_d, int32_t* move_dst_d, int32_t* moved_d,
                             int32_t* status_d, void* stream) {
  if (!h || n < 0 || n > TSV_PAGES_MAX_LISTS || (n > 0 && (!lists || !status_d))) return TSV_ERR_INVALID_ARG;
  if (!refs_out_d || !new_id_d || !move_src_d || !move_dst_d || !moved_d) return TSV_ERR_INVALID_ARG;
  tsv_status st = check_pool(pool);
  if (st != TSV_OK) return st;
  if (new_id_d == refs_out_d || new_id_d == pool->refs_d || move_src_d == move_dst_d) return TSV_ERR_INVALID_ARG;
  PagesCompactArgs a{};
  int64_t rows = 0, width = 1;
  for (int t = 0; t < n; ++t) {
    const tsv_page_lists& l = lists[t];
    if (l.B < 1 || !l.pages_d || !l.out_d || addr(l.out_d) % 4) return TSV_ERR_INVALID_ARG;
    st = check_lists(&l.table, l.B);
    if (st != TSV_OK) return st;
    if (l.B > 1 && l.out_stride < l.table.pages) return TSV_ERR_INVALID_ARG;
    if (l.out_d == l.table.ids_d && l.B > 1 && l.out_stride != l.table.stride) return TSV_ERR_INVALID_ARG;
    a.lists[t] = l;
    rows += l.B;
    if (l.table.pages > width) width = l.table.pages;
  }
  if (rows * ((width + 1023) / 1024) > INT32_MAX) return TSV_ERR_UNSUPPORTED;
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  a.pool = *pool;
  a.refs_out = refs_out_d;
  a.n = n;
  a.new_id = new_id_d;
  a.move_src = move_src_d;
  a.move_dst = move_dst_d;
  a.moved = moved_d;
  a.status = status_d;
  return cuda_status(launch_pages_compact(a, cluster_of(h), h->num_sms, static_cast<cudaStream_t>(stream)));
}

tsv_status tsv_pages_copy(tsv_handle h, const tsv_paged_cache* cache, const int32_t* src_d, const int32_t* dst_d, int32_t n,
                          const int32_t* count_d, int32_t* status_d, void* stream) {
  if (!h || n < 0 || !status_d || (n > 0 && (!src_d || !dst_d))) return TSV_ERR_INVALID_ARG;
  PagesCopyArgs a{};
  const tsv_status st = check_paged_cache(cache, &a.cache);
  if (st != TSV_OK) return st;
  if ((int64_t)a.cache.page_size * a.cache.Hkv * a.cache.D > ((int64_t)1 << 33)) return TSV_ERR_UNSUPPORTED;
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  a.src = src_d;
  a.dst = dst_d;
  a.n = n;
  a.count = count_d;
  a.status = status_d;
  return cuda_status(launch_pages_copy(a, h->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
