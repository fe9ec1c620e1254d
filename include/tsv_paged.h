/*
 * tsv_paged.h — C ABI of libtsv's paged 8-bit KV cache (sm_103a): rotary
 * positions, writing rows into the cache, token-tree attention over it, and
 * the commit of an accepted path.
 *
 *   tsv_rope_frequencies      frequencies of a rotary position encoding (host)
 *   tsv_rope                  rotates the heads of queries or keys by position
 *   tsv_paged_append          rotates, quantises and writes new K/V rows
 *   tsv_paged_tree_attention  tsv_tree_attention over prefix and tree pages
 *   tsv_paged_commit          the accepted path's rows, moved behind the prefix
 *
 * The conventions of tsv.h hold for every call here (handles, streams,
 * ownership, status arrays, the zero-filled workspace).  In addition a call may
 * be made while another device than the handle's is current.
 *
 * The cache.  Pages of page_size rows; a row of one KV head is D codes of 8
 * bits (e4m3: sign, 4 exponent bits, 3 fraction bits, largest value 448), and a
 * page holds one fp32 scale per KV head for K and one for V: value = code x
 * scale.  The library writes scales that are powers of two, so a change of
 * scale moves a code's exponent and loses nothing until values fall below
 * 2^-6 x scale; it reads any finite scale >= 0.  (A page of zeros has 2^-126.)
 *
 * A request has two lists of pages, each a row of a page table: its verified
 * rows 0 .. prefix_len - 1 lie in its prefix pages (row r in page r /
 * page_size), and the nodes of its speculated tree in its tree pages (node i in
 * page i / page_size).  Rejected nodes thus never touch the scale of a page
 * that holds verified rows, and a commit never reads what it writes.  Prefix
 * pages may be shared between requests as long as nobody writes to them: every
 * page that a call writes must belong to one request (and once in its list).
 */
#ifndef TSV_PAGED_H_
#define TSV_PAGED_H_

#include "tsv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Pages of the cache.  Code d of (page p, row r, head g) is the byte at
 * p * stride_page + r * stride_row + g * stride_head + d, in K and in V.
 * Pointers k_d and v_d are 16-byte aligned, the strides multiples of 16 (any
 * order of rows and heads inside a page); page_size is 16, 32, 64 or 128, D is
 * 64 or 128.  Strides of dimensions of size 1 are not used. */
typedef struct {
  void* k_d;
  void* v_d;
  float* k_scale_d; /* [num_pages, Hkv] contiguous */
  float* v_scale_d; /* [num_pages, Hkv] contiguous */
  int64_t stride_page, stride_row, stride_head;
  int32_t num_pages, page_size, Hkv, D;
} tsv_paged_cache;

/* Page lists of B requests: entry i of request b is ids_d[b * stride + i],
 * i < pages; pages x page_size is TSV_PAGED_MAX_ROWS at most.  Entries that a
 * call does not need are not read. */
#define TSV_PAGED_MAX_ROWS (1 << 30)
typedef struct {
  const int32_t* ids_d;
  int64_t stride;
  int32_t pages;
} tsv_page_table;

/* Layout and direction of a rotation. */
#define TSV_ROPE_INTERLEAVED 1u /* pairs (2i, 2i + 1); else (i, i + rotary_dim / 2) */
#define TSV_ROPE_INVERSE 2u     /* by the negative angle: the gradient of the rotation */

/* Scaling of the frequencies for contexts longer than the trained one. */
typedef enum {
  TSV_ROPE_SCALE_NONE = 0,   /* w_i = base^(-2i / rotary_dim) */
  TSV_ROPE_SCALE_LINEAR = 1, /* w_i / factor */
  TSV_ROPE_SCALE_NTK = 2,    /* base grows to base * factor^(rotary_dim / (rotary_dim - 2)) */
  TSV_ROPE_SCALE_BANDS = 3,  /* w_i / factor below `low` turns in the trained context, w_i above `high`, between
                                them a linear mixture in the number of turns */
  TSV_ROPE_SCALE_YARN = 4    /* the mixture linear in i, between the (whole) indices with `high` and `low` turns;
                                amplitude 0.1 ln(factor) + 1 */
} tsv_rope_scaling;

/*
 * tsv_rope_frequencies — the rotary_dim / 2 angular frequencies (radians per
 * position) and the amplitude that tsv_rope and tsv_paged_append take, on the
 * host in 64 bits; copy them to the device once.
 *   rotary_dim  even, >= 2;  base > 0;  scaling a tsv_rope_scaling
 *   factor      > 0 (LINEAR, NTK, BANDS, YARN);  trained  trained context
 *               length > 0 and 0 < low < high (BANDS, YARN)
 *   inv_freq_host (out) double [rotary_dim / 2];  amplitude_host (out) float
 */
tsv_status tsv_rope_frequencies(int32_t rotary_dim, double base, int scaling, double factor,
                                double trained, double low, double high, double* inv_freq_host,
                                float* amplitude_host);

/*
 * tsv_rope — y = amplitude * R(position * w) x on the first rotary_dim elements
 * of each head, pair by pair ((a, b) -> (a cos - b sin, b cos + a sin)); the
 * others are copied.
 *   dtype         TSV_BF16 or TSV_F32 (x and y; the arithmetic is fp32, one
 *                 rounding at the end)
 *   x_d           element (n, h, d) at n * x_stride_n + h * x_stride_h + d
 *   y_d     (out) the same with its own strides; may be x_d itself with equal
 *                 strides (in place), must not overlap it otherwise
 *   N, H, D       N >= 0 rows, H >= 1 heads, 2 <= D <= 1024
 *   positions_d   int32 [N], any sign
 *   inv_freq_d    double [rotary_dim / 2]; rotary_dim even, 2 .. D.  The angle
 *                 is reduced to one turn in 64-bit fixed point, so far
 *                 positions lose nothing
 *   flags         TSV_ROPE_INTERLEAVED, TSV_ROPE_INVERSE
 * Pointers and strides of any alignment (16-byte ones run faster).
 */
tsv_status tsv_rope(tsv_handle h, tsv_dtype dtype, const void* x_d, int64_t x_stride_n, int64_t x_stride_h,
                    void* y_d, int64_t y_stride_n, int64_t y_stride_h, int32_t N, int32_t H, int32_t D,
                    const int32_t* positions_d, const double* inv_freq_d, int32_t rotary_dim,
                    float amplitude, uint32_t flags, void* stream);

/*
 * tsv_paged_append — writes K and V rows row_offsets[b] .. row_offsets[b+1]-1
 * (request b's new tokens) as rows start[b], start[b] + 1, ... of the pages
 * that `table` lists for b: K rotated by its position, both quantised.
 *   need(x) = the smallest power of two s >= 2^-126 with |x| <= 448 s for all
 *             finite x among the page's new values of that head
 *   a page whose first row is new:   scale = need
 *   a page with rows before start[b]: scale = max(its scale, need); its rows
 *             before start[b] are requantised when the scale grows
 * Codes are rounded to nearest even; infinities become +-448 x scale, NaN stays
 * NaN.  Rows behind the new ones keep their codes.
 *   dtype         TSV_BF16 or TSV_F32: type of k_d and v_d
 *   k_d, v_d      element (n, g, d) at n * stride_n + g * stride_h + d; 16-byte
 *                 aligned pointers and strides (for heads and rows, in bytes)
 *   N, B          all rows; requests, 1 .. TSV_MAX_BATCH
 *   max_rows      no request has more new rows than this
 *   start_d       int32 [B], NULL: 0 (tree pages are written from their start)
 *   positions_d   int32 [N]; may be NULL when inv_freq_d is NULL
 *   inv_freq_d, rotary_dim, amplitude, flags   as in tsv_rope (no
 *                 TSV_ROPE_INVERSE); inv_freq_d NULL: K is written as given
 *   status_d (out) int32 [B]: TSV_OK, or TSV_ERR_INVALID_ARG when the request's
 *                 rows do not fit max_rows or its page list, or a page id is out
 *                 of range: none of that request's rows are written
 * Needs no workspace.
 */
tsv_status tsv_paged_append(tsv_handle h, tsv_dtype dtype, const tsv_paged_cache* cache,
                            const tsv_page_table* table, const int32_t* start_d, const void* k_d,
                            int64_t k_stride_n, int64_t k_stride_h, const void* v_d, int64_t v_stride_n,
                            int64_t v_stride_h, const int32_t* row_offsets_d, int32_t B, int32_t N,
                            int32_t max_rows, const int32_t* positions_d, const double* inv_freq_d,
                            int32_t rotary_dim, float amplitude, uint32_t flags, int32_t* status_d,
                            void* stream);

/* Workspace bytes of tsv_paged_tree_attention (zero-fill once, as in tsv.h). */
tsv_status tsv_paged_tree_attention_workspace_size(tsv_handle h, tsv_dtype dtype,
                                                   const tsv_paged_cache* cache, int32_t B,
                                                   int32_t max_nodes, int32_t Hq, uint32_t flags,
                                                   size_t* bytes);

/*
 * tsv_paged_tree_attention — tsv_tree_attention over the paged cache: node i of
 * request b, query head h, KV head g = h / (Hq / Hkv),
 *   out[i,h] = sum_j softmax_j(scale * <q[i,h], k_j>) v_j
 * over the request's prefix rows and those of its tree's rows that node i sees.
 * The lengths are read on the device, so a captured call follows them.
 *   dtype         TSV_BF16 (tensor cores) or TSV_F32 (CUDA cores): q and out
 *   q_d           element (n, h, d) at n * q_stride_n + h * q_stride_h + d;
 *                 16-byte aligned pointer and strides (in bytes)
 *   prefix_len_d  int32 [B] rows in the prefix pages
 *   tree_table    the tree pages; NULL: there are no tree keys, every node sees
 *                 the prefix alone (a single new token whose row was appended
 *                 to the prefix pages, prefix_len counting it)
 *   node_offsets_d int32 [B+1]: rows of q and out of each request
 *   anc_d         uint32 [N][TSV_ANC_WORDS] from tsv_tree_prepare (16-byte
 *                 aligned): node i sees tree row j iff bit j is set; NULL:
 *                 node i sees tree rows 0 .. i (a chain of new tokens)
 *   out_d   (out) [N, Hq, D] contiguous, 16-byte aligned; 0 for a node that
 *                 sees nothing
 *   max_nodes     1 .. TSV_MAX_NODES; no request has more nodes
 *   scale         softmax scale; 0 means 1/sqrt(D)
 *   status_d (out) int32 [B]: TSV_OK; TSV_ERR_INVALID_ARG when the request's
 *                 lengths do not fit N, max_nodes or its page lists, or a page id
 *                 is out of range (its outputs are undefined, nothing out of
 *                 range is read); TSV_ERR_TIMEOUT on a device-side timeout, and
 *                 from later calls until the workspace is zeroed again
 *   flags         TSV_ATTN_DEFAULT or TSV_ATTN_SIMT (CUDA cores for bf16 too)
 * Rows past a request's lengths may hold anything.  A NaN in a V row reaches
 * only the nodes that see the row.
 *   Which kernel runs follows from the shapes alone: rows per KV head (max_nodes
 * x Hq / Hkv), requests, KV heads, and the keys that `table` has room for.  The
 * same call gives the same bits again; a wider table can change the last ones.
 *   Accuracy.  Scores and sums are fp32.  On the tensor cores a weight (its
 * softmax term times the V scale of its page) is rounded: with few rows to
 * 2^-8 of itself (two e4m3 terms) or 2^-18 of the largest among 256 keys (2^-14
 * where their V scales lie up to 2^4 apart), with many to 2^-12 of itself
 * (fp16) or 2^-36 of the row's largest; V scales further apart count in what a
 * row's weights are relative to, up to 2^40.  q is held to 2^-17 of its row's
 * largest value with few rows, 2^-31 with many.
 */
tsv_status tsv_paged_tree_attention(tsv_handle h, tsv_dtype dtype, const void* q_d, int64_t q_stride_n,
                                    int64_t q_stride_h, const tsv_paged_cache* cache,
                                    const tsv_page_table* table, const int32_t* prefix_len_d,
                                    const tsv_page_table* tree_table, const int32_t* node_offsets_d,
                                    const uint32_t* anc_d, void* out_d, int32_t B, int32_t N,
                                    int32_t max_nodes, int32_t Hq, float scale, void* workspace_d,
                                    size_t workspace_bytes, int32_t* status_d, uint32_t flags,
                                    void* stream);

/*
 * tsv_paged_commit — appends the accepted path to the prefix: row prefix_len[b]
 * + k of request b's prefix pages takes the value of tree row path[k], k = 0 ..
 * accept_len[b], quantised as tsv_paged_append quantises.  The tree pages are
 * only read.
 *   max_nodes     1 .. TSV_MAX_NODES; no request has more nodes
 *   path_d        int32 [N], accept_len_d int32 [B]: as the verify calls write
 *                 them (path[0] = 0, strictly rising)
 *   new_len_d (out) int32 [B]: prefix_len[b] + 1 + accept_len[b] (-1 when the
 *                 request is rejected); may be NULL, and may be prefix_len's own
 *                 successor buffer but not prefix_len_d itself
 *   status_d (out) int32 [B]: TSV_OK or TSV_ERR_INVALID_ARG (a path that is not
 *                 one, lengths that do not fit N, max_nodes or the page lists, a
 *                 page id out of range): nothing of that request is written
 * Needs no workspace.
 */
tsv_status tsv_paged_commit(tsv_handle h, const tsv_paged_cache* cache, const tsv_page_table* table,
                            const tsv_page_table* tree_table, const int32_t* prefix_len_d,
                            const int32_t* node_offsets_d, const int32_t* path_d,
                            const int32_t* accept_len_d, int32_t B, int32_t N, int32_t max_nodes,
                            int32_t* new_len_d, int32_t* status_d, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TSV_PAGED_H_ */
