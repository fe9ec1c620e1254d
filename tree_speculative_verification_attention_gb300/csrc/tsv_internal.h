// tsv_internal.h — declarations shared by the library's translation units
// (launch wrappers and the attention work plan).  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tsv.h"
#include "../../include/tsv_paged.h"

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMssClusterSizeEntries = 9;  // entries of the resident-cluster table (sizes 0..8)

struct tsv_handle_s {
  int device;
  int num_sms;
  EncodeTiledFn encode;
  bool tc_attr_set[2];    // rows-on-lanes kernel (tile pairs), D = 64, 128
  bool tc1_attr_set[2];   // rows-on-lanes kernel (one tile), D = 64, 128
  bool keys_attr_set[2];  // keys-on-lanes kernel, D = 64, 128
  bool mss_attr_set;      // MSS kernel's shared-memory limit
  size_t mss_staged_limit;
  int mss_max_clusters[kMssClusterSizeEntries];  // resident MSS clusters of each size
  uint32_t verify_overlap;  // tsv_set_verify_overlap: TSV_OVERLAP_* flags
  uint32_t paged_attr_mask;   // paged attention kernels whose attributes are set, one bit per (D, tile rows)
  uint32_t append_attr_mask;  // paged append kernels, one bit per (type, D)
};

namespace tsv {

constexpr int kBM = 128;  // query rows (node x head-in-group) per attention CTA = TMEM lanes
constexpr int kBN = 128;  // keys per pipeline block

// How one tsv_tree_attention call is cut into CTAs.  Passed by value as a
// kernel parameter (no host-to-device copy, so a launch can be captured).
// A unit (CTA) is (request b, KV head g, chunk c, M-tile mt); inside request b
// the unit index is ((g * n_chunks + c) * mtiles + mt), so the M-tiles of one
// KV chunk run next to each other and share its rows through L2.  Requests
// take consecutive unit ranges in slot order: slot s holds request
// slot_req[s], longest key range first, so that the block scheduler starts
// the longest CTAs first (longest-processing-time list scheduling).
struct AttnPlan {
  int32_t B, Hq, Hkv, G, D;
  int32_t n_units;
  int32_t chunk_keys;  // keys per chunk (multiple of kBN), same for every request
  float scale_log2;    // softmax scale * log2(e)
  int32_t unit_start[TSV_MAX_BATCH + 1];  // per slot
  int32_t slot_req[TSV_MAX_BATCH];
  int32_t n_chunks[TSV_MAX_BATCH];
  int32_t mtiles[TSV_MAX_BATCH];
  int32_t prefix[TSV_MAX_BATCH];
  int32_t nodes[TSV_MAX_BATCH];
  int32_t node_off[TSV_MAX_BATCH];
  int64_t part_row[TSV_MAX_BATCH];  // first partial row of request b, -1 when n_chunks == 1
  int32_t ctr_base[TSV_MAX_BATCH];  // first merge counter of request b (one per KV head x M-tile)
  int64_t part_rows_total;
  int32_t n_counters;
  // Keys-on-lanes kernel: every request is cut into n_chunks[b] == cluster
  // chunks of chunk_len[b] keys (a multiple of 128); the chunks of one (KV
  // head, M-tile) group are consecutive units and form one cluster.
  // Tile-pair rows kernel: cluster == n_chunks[b] (2 .. 8, the same for every
  // request) when the chunks of a (KV head, tile pair) merge in a cluster,
  // else 0.
  int32_t chunk_len[TSV_MAX_BATCH];
  int32_t cluster;
  int32_t keys_kernel;  // 1: keys-on-lanes kernel, 0: rows-on-lanes kernel
  // Keys-on-lanes kernel: every unit runs in the first wave (n_units <= SMs),
  // so each CTA pulls its first K/V blocks into L2 before waiting for the
  // previous kernel; with later waves the prefetch would only add traffic.
  int32_t prefetch_l2;
  // Keys-on-lanes kernel with one chunk per request and more units than SMs:
  // a persistent launch of `grid` CTAs (one per SM), each taking a sequence of
  // units, so that its producer streams the next unit's K/V while the key
  // lanes finish the previous unit.
  int32_t persistent;
  int32_t grid;
  // Rows-on-lanes kernel: 1 = two 128-row query tiles per CTA (units are
  // tile pairs), 0 = one tile per CTA (every request has mtiles <= 1).
  int32_t tc_tile_pairs;
};

// Launches a kernel with programmatic stream serialization (it may be
// scheduled while the previous kernel in the stream drains; the kernel waits
// for it with pdl_wait() before touching global memory) and, when cluster > 0,
// thread-block clusters of that many CTAs along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              unsigned cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster > 0) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct Workspace {
  char* base;
  size_t size;
  size_t used;
  void* take(size_t bytes) {
    size_t off = (used + 255) & ~(size_t)255;
    if (off + bytes > size) return nullptr;
    used = off + bytes;
    return base + off;
  }
};

// Launch wrappers (defined next to their kernels); return the launch error.
cudaError_t launch_tree_prepare(const int32_t* parent, const int32_t* node_offsets, int32_t B,
                                uint32_t* anc, int32_t* depth, int32_t* status, cudaStream_t st);

cudaError_t launch_attention_tc(const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                const CUtensorMap& tmap_v, const AttnPlan& plan,
                                const int32_t* parent, const uint32_t* anc, void* out,
                                float* part_o, float* part_lse, int32_t* counters,
                                int32_t* status, cudaStream_t st);
cudaError_t attention_tc_set_attributes(int D);
size_t attention_tc_smem_bytes(int D);
// The same with one query tile per CTA (plans with tc_tile_pairs == 0).
cudaError_t launch_attention_tc1(const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                 const CUtensorMap& tmap_v, const AttnPlan& plan,
                                 const int32_t* parent, const uint32_t* anc, void* out,
                                 float* part_o, float* part_lse, int32_t* counters,
                                 int32_t* status, cudaStream_t st);
cudaError_t attention_tc1_set_attributes(int D);
size_t attention_tc1_smem_bytes(int D);

constexpr int kKeysBlockKeys = 128;  // keys per block of the keys-on-lanes kernel
constexpr int kKeysTileRows = 64;    // query rows per CTA of the keys-on-lanes kernel
constexpr int kKeysMaxUnitsPerCta = 48;  // units one CTA of a persistent keys launch may take
cudaError_t launch_attention_keys(const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                  const CUtensorMap& tmap_v, const AttnPlan& plan,
                                  const int32_t* parent, const uint32_t* anc, void* out,
                                  int32_t* status, cudaStream_t st);
cudaError_t attention_keys_set_attributes(int D);
size_t attention_keys_smem_bytes(int D);

cudaError_t launch_attention_simt(bool bf16, const void* q, const void* k, const void* v,
                                  int64_t sb, int64_t sl, int64_t sh, void* out,
                                  const int32_t* prefix_len, const int32_t* node_offsets,
                                  const uint32_t* anc, int32_t B, int32_t N, int32_t Hq,
                                  int32_t Hkv, int32_t D, float scale, cudaStream_t st);

// Greedy verification: argmax over vocab slices folded into one 64-bit word
// per row, the last CTA of a request walks.
int greedy_splits(int64_t V, int32_t N, int num_sms);
cudaError_t launch_greedy_verify(const float* logits, int64_t V, int32_t N, int splits,
                                 const int32_t* tokens, const int32_t* parent,
                                 const int32_t* node_offsets, int32_t B, unsigned long long* rowbest,
                                 int32_t* counters, int32_t* path, int32_t* accept_len, int32_t* bonus,
                                 int32_t* status, int beside, cudaStream_t st);
cudaError_t launch_greedy_walk(unsigned long long* rowbest, const int32_t* tokens, const int32_t* parent,
                               const int32_t* node_offsets, int32_t B, int32_t* path,
                               int32_t* accept_len, int32_t* bonus, int32_t* status,
                               cudaStream_t st);

// Layout of a greedy verification workspace (the one tsv_tree_verify_greedy
// uses): B int32 completion counters, then N 64-bit row argmax words; both
// start at zero and every call leaves them at zero.
inline size_t greedy_counter_bytes(int32_t B) { return ((size_t)B * 4 + 255) & ~(size_t)255; }
inline size_t greedy_row_word_bytes(int32_t N) { return ((size_t)N * 8 + 255) & ~(size_t)255; }
inline size_t greedy_workspace_bytes(int32_t B, int32_t N) {
  return greedy_counter_bytes(B) + greedy_row_word_bytes(N);
}

// Stochastic verification: one cluster of mss_cluster_size(V, B, ...) CTAs
// per request, each owning a slice of the vocabulary.  `beside`: 0 waits for
// the previous kernel on the stream before reading; kMssBesideCompact and
// kMssBesideFull start beside it (two-warp CTAs that fit next to an attention
// CTA, or the full-size CTAs on SMs it leaves free) and complete after it.
// `room`: the full-size CTAs leave registers for a greedy CTA beside each.
constexpr int kMssClusterSizes = kMssClusterSizeEntries;
constexpr int kMssBesideCompact = 1, kMssBesideFull = 2;
// Largest cluster of the full-size CTAs beside a running kernel: a cluster
// needs that many idle SMs in one GPC, which a running grid seldom leaves
// (measured beside the GQA rows-on-lanes launch: clusters of 8 started only as
// it ended, clusters of 4 or 2 ran beside it).
constexpr int kMssBesideMaxCluster = 4;
int mss_cluster_size(int64_t V, int32_t B, const int* max_clusters, int cap);
cudaError_t launch_mss_verify(const float* llm_logits, const float* ssm_probs, int64_t V,
                              const int32_t* tokens, const int32_t* parent,
                              const int32_t* node_offsets, const float* u_acc, const float* u_smp,
                              float inv_t, int32_t top_k, float top_p, int32_t B, float* resid,
                              int32_t* path, int32_t* accept_len, int32_t* bonus, int32_t* n_tried,
                              int32_t* status, size_t staged_limit, const int* max_clusters,
                              int beside, int room, cudaStream_t st);
// Sets the MSS kernels' dynamic shared-memory limit on `device` to all that is
// left beside their static shared memory, returns the staged kernel's limit
// (the largest staged slice set a launch may use) and fills
// max_clusters[0..kMssClusterSizes-1] with the clusters of each size the
// device holds at once.
cudaError_t mss_set_attributes(int device, size_t* staged_limit, int* max_clusters);
constexpr int kMssMaxTopK = 1024;  // largest top_k of the warped stochastic verification

// Token-tree construction: expansion (top-k children per frontier row) and
// merge of several trees per request.
constexpr int kTreeMergeMaxInput = 1024;  // input nodes of one request's merge
cudaError_t launch_tree_expand(const float* logits, int64_t V, int32_t F, int32_t k, int32_t* tokens,
                               int num_sms, cudaStream_t st);
cudaError_t launch_tree_merge(const int32_t* parent, const int32_t* tokens, const int32_t* tree_offsets,
                              const int32_t* request_trees, int32_t B, int32_t* out_parent,
                              int32_t* out_tokens, int32_t* out_source, int32_t* out_count,
                              int32_t* status, cudaStream_t st);

// KV commit of the accepted path: rows hold row_chunks 16-byte chunks per
// cache row (Hkv x D x element size / 16); strides in bytes.
cudaError_t launch_kv_commit(uint8_t* k, uint8_t* v, int64_t sb, int64_t sl, int64_t sh, int32_t B,
                             int32_t Hkv, int32_t d_chunks, const int32_t* prefix_len,
                             const int32_t* node_offsets, const int32_t* path,
                             const int32_t* accept_len, int32_t* new_len, int32_t* status,
                             cudaStream_t st);

// Rotary positions (tsv_rope).
struct RopeArgs {
  const void* x;
  void* y;
  int64_t xs_n, xs_h, ys_n, ys_h;  // elements
  int32_t N, H, D, rot;
  const int32_t* positions;
  const double* inv_freq;
  float amplitude;
  int32_t interleaved, inverse;
};
cudaError_t launch_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t st);

// New rows of a paged cache (tsv_paged_append and tsv_paged_commit).
struct PagedWriteArgs {
  tsv_paged_cache cache;
  tsv_page_table table;       // pages written
  const int32_t* start;       // [B] rows kept in front of the new ones, NULL: 0
  const int32_t* offsets;     // [B+1] rows of k / v (append) or of path (commit)
  int32_t B, N, max_rows;     // max_rows: new rows of one request at most
  int32_t head_loop;          // head groups that one CTA takes in turn
  int32_t* status;
  // append
  const void* k;
  const void* v;
  int64_t ks_n, ks_h, vs_n, vs_h;
  const int32_t* positions;
  const double* inv_freq;     // NULL: no rotation
  int32_t rot, interleaved;
  float amplitude;
  // commit
  tsv_page_table tree_table;  // pages read
  const int32_t* path;
  const int32_t* accept_len;
  int32_t* new_len;
};
size_t paged_append_smem_bytes(int32_t page_size, int32_t rot);
constexpr int kPagedWriteMaxWarps = 32;
constexpr int paged_write_rows(int32_t D) { return 512 / D; }  // rows of one (page, head) that a warp takes
// Warps of a CTA, a whole page of one head at least, and the heads they hold.
inline int paged_write_warps(int32_t page_size, int32_t D) {
  const int page = page_size / paged_write_rows(D);
  return page > 8 ? page : 8;
}
inline int paged_write_heads(int32_t page_size, int32_t D) {
  return paged_write_warps(page_size, D) * paged_write_rows(D) / page_size;
}
cudaError_t paged_append_set_attributes(bool bf16, int32_t D);
cudaError_t launch_paged_append(const PagedWriteArgs& a, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_paged_commit(const PagedWriteArgs& a, int num_sms, cudaStream_t st);

// Tree attention over a paged cache.
struct PagedAttnArgs {
  const void* q;
  int64_t qs_n, qs_h;
  tsv_paged_cache cache;
  tsv_page_table table;
  tsv_page_table tree_table;  // ids_d NULL: no tree keys
  const int32_t* prefix_len;
  const int32_t* offsets;
  const uint32_t* anc;
  void* out;
  int32_t* status;
  int32_t B, N, max_nodes, Hq, G;
  float scale;
};
// Tensor-core kernel: row tiles of R = 16, 32 or 64 query rows; its workspace
// holds one word per request (set by a CTA that gave up a wait for it), one
// completion counter per CTA, then two partial results per CTA (O [R][D], then
// maxima and sums [2][R]).
constexpr int32_t kPagedWideRows = 256;
constexpr int32_t kPagedWideCtas = 160;  // at most: shared memory holds the weights of so many parts
// Rows of a unit of the tensor-core kernels: 16, 32, 64 (keys on the TMEM lanes)
// or 256 (rows on them), of `rows` query rows in each of `groups` (request, KV
// head) pairs, over up to `keys` keys (what the page tables hold).  More rows
// share a block's cost, but units that are few are cut into many parts, and
// parts cost more the more rows they have.  Measured (us; 8 query heads a KV
// head, D = 128), 32 / 64 / 256 rows a unit:
//   1 request x 16384 keys x 8 KV heads:   64 rows 32 / 46 / 62, 256 rows 67 / 63 / 99, 512 rows 118 / 100 / 93
//   1 request x 32768 keys x 8 KV heads:   1024 rows - / 333 / 199
//   4 requests x 4096 keys x 8 KV heads:   128 rows 50 / 44 / 60, 256 rows 88 / 66 / 70
//   13 requests x 256 keys x 8 KV heads:   256 rows 77 / 55 / 45; 2048 keys 178 / 117 / 84
//   32 requests x 4096 keys x 8 KV heads:  40 rows 169 / 111 / 200, 128 rows 318 / 215 / 203, 256 rows 612 / 399 / 241
// (128 rows over long prefixes of many requests stay with 64 a unit: 6 % there,
// against 36 % the other way with few requests.)
inline int32_t paged_attn_rows(int64_t rows, int64_t groups, int64_t keys) {
  if (rows <= 32) return rows <= 16 ? 16 : 32;
  const int64_t wide = groups * ((rows + kPagedWideRows - 1) / kPagedWideRows);
  if (rows > 128 && wide * (keys / 128 + 1) >= (wide >= 96 ? 1024 : 4096)) return kPagedWideRows;
  return groups * ((rows + 63) / 64) >= 32 ? 64 : 32;
}
struct PagedAttnLayout {
  size_t part_o, part_ml, total;
};
inline PagedAttnLayout paged_attn_layout(int grid, int32_t R, int32_t D) {
  PagedAttnLayout l;
  l.part_o = ((size_t)(TSV_MAX_BATCH + grid) * 4 + 255) & ~(size_t)255;
  l.part_ml = l.part_o + (size_t)grid * 2 * R * D * 4;
  l.total = l.part_ml + (size_t)grid * 2 * 2 * R * 4;
  return l;
}
cudaError_t paged_attention_set_attributes(int32_t D, int32_t R);
cudaError_t launch_paged_attention(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int32_t R, int grid,
                                   void* ws, cudaStream_t st);
cudaError_t paged_attention_wide_set_attributes(int32_t D);
cudaError_t launch_paged_attention_wide(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int num_sms, void* ws,
                                        cudaStream_t st);
cudaError_t launch_paged_attention_simt(const PagedAttnArgs& a, bool bf16, cudaStream_t st);

}  // namespace tsv
