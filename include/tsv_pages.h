/*
 * tsv_pages.h — C ABI of libtsv's page management (sm_103a): which request
 * holds which page of a paged cache (tsv_paged.h), decided on the device.
 *
 *   tsv_pages_resize   lists of pages grow and shrink
 *   tsv_pages_fork     lists that share the pages of others
 *   tsv_pages_compact  pages in use move to the low ids
 *   tsv_pages_copy     the contents of pages, inside one layer's cache
 *
 * The conventions of tsv.h hold for every call here (handles, streams,
 * ownership, status arrays), and a call may be made while another device than
 * the handle's is current.  No call needs a workspace, and results depend on
 * the arguments alone: pages are handed out by rising id, never by a race.
 *
 * A pool counts, for each page, the lists that hold it: refs_d[p] >= 0, and 0
 * is a free page.  The caller zero-fills the counts once; it may add to one
 * itself to keep a page (a prefix held for later requests, say) out of reach.
 * Page ids are the same in every layer's cache, so one pool and one set of
 * tables serve all layers, and what moves contents (tsv_pages_copy) is called
 * for each.
 *
 * Counts that do not add up (a page on more lists than it counts) never reach a
 * page outside the pool, but some list that gives such a page back is reported
 * with TSV_ERR_INVALID_ARG after the fact: a resize has shortened it, a fork has
 * left it empty (unchanged, if the page was free before the list was looked at).
 *
 * A list is a row of a page table with a count beside it: pages_d[b] entries of
 * row b are held.  Entries behind them are never read, and keep what they hold
 * unless a call says that it writes them.
 */
#ifndef TSV_PAGES_H_
#define TSV_PAGES_H_

#include "tsv_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* At most 2^27 pages (TSV_PAGED_MAX_ROWS rows hold fewer of any size). */
typedef struct {
  int32_t* refs_d; /* [num_pages], 16-byte aligned */
  int32_t num_pages;
} tsv_page_pool;

/*
 * tsv_pages_resize — request b's list gets rows[b] / page_size pages, rounded
 * up.  First the lists that shrink give back what lies behind (their entries
 * stay as they are), then the others take the free pages of lowest id, request
 * by request in order, entry by entry.  rows[b] = 0 frees a list.
 *   table, pages_d  lists and their counts (both in / out), B of them
 *   rows_d          int32 [B]
 *   page_size       >= 1
 *   status_d (out)  int32 [B]: TSV_OK; TSV_ERR_NO_PAGES for the first request
 *                   in order whose pages are not there, and for every one
 *                   behind it that needs any: their lists stay as they were;
 *                   TSV_ERR_INVALID_ARG (list unchanged, and it takes none) when
 *                   pages[b] or the pages wanted do not fit the table, an id to
 *                   be given back is out of range or not held, or the rows end
 *                   inside a page, kept by a list that shrinks, that other
 *                   lists hold too (new rows would be written there: fork the
 *                   list instead)
 */
tsv_status tsv_pages_resize(tsv_handle h, const tsv_page_pool* pool, const tsv_page_table* table, int32_t* pages_d,
                            const int32_t* rows_d, int32_t B, int32_t page_size, int32_t* status_d, void* stream);

/*
 * tsv_pages_fork — list b of `to` becomes the first rows[b] rows of list
 * source[b] of `from`: whole pages are shared, and a last page that the rows
 * fill in part is one of its own, into which the caller copies the source's
 * (tsv_pages_copy of copy_src, copy_dst in each layer's cache).  What list b
 * held before is given back first, of all lists before any takes a page.
 *   from, from_pages_d, F  source lists (read only), 1 .. 65536 of them
 *   source_d        int32 [B]; -1 leaves list b as it is
 *   rows_d          int32 [B]
 *   to, to_pages_d  lists and their counts (both in / out), B of them; must not
 *                   overlap the source lists (of one table, rows or columns
 *                   apart from each other will do, also in turn)
 *   copy_src_d, copy_dst_d (out) int32 [B]: the page that list b's last page is
 *                   to be copied from, and that page; -1 when there is none
 *   status_d (out)  int32 [B]: TSV_OK; TSV_ERR_NO_PAGES, as in tsv_pages_resize,
 *                   for lists that need a page of their own: the list is then
 *                   empty; TSV_ERR_INVALID_ARG (list unchanged) when source[b],
 *                   rows[b] or a count does not fit, or an id on either list is
 *                   out of range or not held
 */
tsv_status tsv_pages_fork(tsv_handle h, const tsv_page_pool* pool, const tsv_page_table* from, const int32_t* from_pages_d,
                          int32_t F, const int32_t* source_d, const int32_t* rows_d, const tsv_page_table* to,
                          int32_t* to_pages_d, int32_t B, int32_t page_size, int32_t* copy_src_d, int32_t* copy_dst_d,
                          int32_t* status_d, void* stream);

/* Lists whose entries a compaction rewrites: B >= 1 rows (not limited to
 * TSV_MAX_BATCH) of `table`, pages_d [B] of them held each; the new ids go to
 * out_d[b * out_stride + i], which may be the table itself (equal strides). */
typedef struct {
  tsv_page_table table;
  const int32_t* pages_d;
  int32_t* out_d;
  int64_t out_stride;
  int32_t B;
} tsv_page_lists;
#define TSV_PAGES_MAX_LISTS 8

/*
 * tsv_pages_compact — the L pages in use get the ids 0 .. L - 1: those below L
 * keep theirs, and the others, by rising id, take the free ones below L, by
 * rising id.  The contents are the caller's to move: tsv_pages_copy of
 * move_src, move_dst and moved in each layer's cache.
 *   refs_out_d (out) int32 [num_pages]: the counts under the new ids; may be the
 *                   pool's own
 *   lists, n        every list of the pool (n of them, 0 .. TSV_PAGES_MAX_LISTS
 *                   tables), on the host
 *   new_id_d (out)  int32 [num_pages]: new id of every page, -1 for a free one
 *   move_src_d, move_dst_d (out) int32 [num_pages / 2] at least: the moved
 *                   pages' old and new ids; entries behind the moved ones are
 *                   not written
 *   moved_d  (out)  int32 [1]: how many
 *   status_d (out)  int32 [n]: TSV_OK, or TSV_ERR_INVALID_ARG when a count
 *                   does not fit its table or an entry is out of range or free
 *                   (such an entry becomes -1; such a count's row is left out).
 *                   NULL when n is 0
 */
tsv_status tsv_pages_compact(tsv_handle h, const tsv_page_pool* pool, int32_t* refs_out_d, const tsv_page_lists* lists,
                             int32_t n, int32_t* new_id_d, int32_t* move_src_d, int32_t* move_dst_d, int32_t* moved_d,
                             int32_t* status_d, void* stream);

/*
 * tsv_pages_copy — page dst[i] of the cache takes the codes and the scales of
 * page src[i], K and V.  Pairs with an id of -1 are left out.  No page may be
 * the destination of two pairs, or of one and the source of another (its
 * contents would be either's).  A page has 2^33 bytes of codes at most.
 *   src_d, dst_d    int32 [n], n >= 0
 *   count_d         int32 [1], NULL: n.  Only the first count pairs are copied
 *                   (none when it is negative, n when it is more)
 *   status_d (out)  int32 [1]: TSV_OK, or TSV_ERR_INVALID_ARG when an id is out
 *                   of range (that pair is left out, others are copied)
 */
tsv_status tsv_pages_copy(tsv_handle h, const tsv_paged_cache* cache, const int32_t* src_d, const int32_t* dst_d, int32_t n,
                          const int32_t* count_d, int32_t* status_d, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TSV_PAGES_H_ */
