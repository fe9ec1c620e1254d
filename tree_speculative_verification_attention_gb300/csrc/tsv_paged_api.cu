// tsv_paged_api.cu — the C ABI declared in include/tsv_paged.h: argument
// checks, launch planning and launches.  Nothing is allocated here.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "tsv_internal.h"

using namespace tsv;

namespace tsv {

DeviceScope::DeviceScope(int device) {
  int now = -1;
  ok = cudaGetDevice(&now) == cudaSuccess;
  if (ok && now != device) {
    ok = cudaSetDevice(device) == cudaSuccess;
    if (ok) before = now;
  }
}
DeviceScope::~DeviceScope() {
  if (before >= 0) cudaSetDevice(before);
}

static inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

tsv_status check_paged_cache(const tsv_paged_cache* in, tsv_paged_cache* c) {
  if (!in) return TSV_ERR_INVALID_ARG;
  *c = *in;
  if (!c->k_d || !c->v_d || !c->k_scale_d || !c->v_scale_d || !aligned16(c->k_d) || !aligned16(c->v_d))
    return TSV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k_scale_d) | reinterpret_cast<uintptr_t>(c->v_scale_d)) & 3) return TSV_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->Hkv < 1) return TSV_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return TSV_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return TSV_ERR_UNSUPPORTED;
  if ((int64_t)c->num_pages * c->page_size > INT32_MAX) return TSV_ERR_UNSUPPORTED;
  if (c->Hkv == 1) c->stride_head = c->D;
  if (c->num_pages == 1) c->stride_page = (int64_t)c->page_size * c->Hkv * c->D;
  const int64_t s[3] = {c->stride_page, c->stride_row, c->stride_head};
  for (int64_t x : s)
    if (x < c->D || x % 16 || x >= ((int64_t)1 << 40)) return TSV_ERR_INVALID_ARG;
  return TSV_OK;
}

}  // namespace tsv

namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
tsv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TSV_OK : TSV_ERR_CUDA; }

tsv_status check_table(const tsv_page_table* t, int32_t B, const tsv_paged_cache& c) {
  if (!t || !t->ids_d || t->pages < 1) return TSV_ERR_INVALID_ARG;
  if (B > 1 && t->stride < t->pages) return TSV_ERR_INVALID_ARG;
  if ((int64_t)t->pages * c.page_size > TSV_PAGED_MAX_ROWS) return TSV_ERR_UNSUPPORTED;
  return TSV_OK;
}

// Rows of heads in 16-byte vectors: pointer and strides aligned.
bool rows_aligned(const void* p, int64_t sn, int64_t sh, int64_t esz) {
  return aligned16(p) && (sn * esz) % 16 == 0 && (sh * esz) % 16 == 0;
}

tsv_status check_attention(tsv_handle h, tsv_dtype dtype, const tsv_paged_cache* cache, tsv_paged_cache* c, int32_t B,
                           int32_t max_nodes, int32_t most, int32_t Hq, uint32_t flags) {
  if (!h || (dtype != TSV_F32 && dtype != TSV_BF16) || (flags & ~TSV_ATTN_SIMT)) return TSV_ERR_INVALID_ARG;
  if (B < 1 || B > TSV_MAX_BATCH || max_nodes < 1 || max_nodes > most) return TSV_ERR_INVALID_ARG;
  const tsv_status st = check_paged_cache(cache, c);
  if (st != TSV_OK) return st;
  if (Hq < 1 || Hq % c->Hkv) return TSV_ERR_INVALID_ARG;
  if (c->Hkv > 65535) return TSV_ERR_UNSUPPORTED;
  return TSV_OK;
}

// One KV head's rows of a page as a box of a 4-D map (D, Hkv, rows, pages).
tsv_status encode_pages(tsv_handle h, CUtensorMap* map, const void* base, const tsv_paged_cache& c) {
  const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.Hkv, (cuuint64_t)c.page_size, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c.stride_head, (cuuint64_t)c.stride_row, (cuuint64_t)c.stride_page};
  const cuuint32_t box[4] = {(cuuint32_t)c.D, 1, (cuuint32_t)c.page_size, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = h->encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? TSV_OK : TSV_ERR_INVALID_ARG;
}

bool paged_uses_tc(tsv_dtype dtype, uint32_t flags) { return dtype == TSV_BF16 && !(flags & TSV_ATTN_SIMT); }

// The tensor-core kernel of R query rows a unit.
tsv_status launch_tree_kernels(tsv_handle h, const PagedAttnArgs& a, int32_t R, void* workspace_d, cudaStream_t stream) {
  const bool wide = R == kPagedWideRows;
  const uint32_t bit = 1u << ((wide ? 3 : R == 16 ? 0 : R == 32 ? 1 : 2) + (a.cache.D == 128 ? 4 : 0));
  if (!(h->paged_attr_mask & bit)) {
    if ((wide ? paged_attention_wide_set_attributes(a.cache.D) : paged_attention_set_attributes(a.cache.D, R)) != cudaSuccess)
      return TSV_ERR_CUDA;
    h->paged_attr_mask |= bit;
  }
  CUtensorMap tk, tv;
  tsv_status st = encode_pages(h, &tk, a.cache.k_d, a.cache);
  if (st == TSV_OK) st = encode_pages(h, &tv, a.cache.v_d, a.cache);
  if (st != TSV_OK) return st;
  if (wide) return cuda_status(launch_paged_attention_wide(tk, tv, a, h->num_sms, workspace_d, stream));
  return cuda_status(launch_paged_attention(tk, tv, a, R, h->num_sms, workspace_d, stream));
}

// Rows a unit of the tree attention's kernel when each request has one token.
int32_t chunk_token_rows(int32_t G, int32_t B, const tsv_paged_cache& c) {
  return paged_attn_rows(G, (int64_t)B * c.Hkv, TSV_PAGED_MAX_ROWS);
}

// Head groups that one CTA of an append or commit takes in turn, of about
// `pages` pages to write.  What it does once (the angles, or the chain of loads
// from the lengths to the path's pages) costs as much as `once` groups, and the
// next group's rows are loaded under the current one's arithmetic: the grid is
// split over the heads as finely as does not cost another wave of 32 warps per
// SM.
int32_t head_loop(const PagedWriteArgs& a, int64_t pages, int once, int num_sms) {
  const int64_t groups = cdiv(a.cache.Hkv, paged_write_heads(a.cache.page_size, a.cache.D));
  const int64_t slots = num_sms * std::max(1, 32 / paged_write_warps(a.cache.page_size, a.cache.D));
  int64_t loop = groups, least = INT64_MAX;
  for (int64_t z = 1; z <= std::min<int64_t>(groups, 256); ++z) {
    const int64_t cost = cdiv(pages * z, slots) * (once + cdiv(groups, z));
    if (cost > least) continue;
    least = cost;
    loop = cdiv(groups, z);
  }
  return (int32_t)loop;
}

}  // namespace

extern "C" {

tsv_status tsv_rope_frequencies(int32_t rotary_dim, double base, int scaling, double factor, double trained,
                                double low, double high, double* inv_freq_host, float* amplitude_host) {
  if (rotary_dim < 2 || rotary_dim % 2 || !inv_freq_host || !amplitude_host) return TSV_ERR_INVALID_ARG;
  if (!(base > 0.0) || isinf(base) || scaling < TSV_ROPE_SCALE_NONE || scaling > TSV_ROPE_SCALE_YARN)
    return TSV_ERR_INVALID_ARG;
  if (scaling != TSV_ROPE_SCALE_NONE && (!(factor > 0.0) || isinf(factor))) return TSV_ERR_INVALID_ARG;
  const bool mixed = scaling == TSV_ROPE_SCALE_BANDS || scaling == TSV_ROPE_SCALE_YARN;
  if (mixed && (!(trained > 0.0) || isinf(trained) || !(low > 0.0) || !(high > low) || isinf(high)))
    return TSV_ERR_INVALID_ARG;
  if (scaling == TSV_ROPE_SCALE_YARN && base == 1.0) return TSV_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  if (scaling == TSV_ROPE_SCALE_NTK && rotary_dim > 2)
    base *= pow(factor, (double)rotary_dim / (rotary_dim - 2));
  double first = 0.0, last = 0.0;
  if (scaling == TSV_ROPE_SCALE_YARN) {  // indices whose frequencies turn `high` and `low` times in the trained context
    first = std::max(floor(rotary_dim * log(trained / (high * two_pi)) / (2.0 * log(base))), 0.0);
    last = std::min(ceil(rotary_dim * log(trained / (low * two_pi)) / (2.0 * log(base))), rotary_dim - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double w = pow(base, -2.0 * i / rotary_dim);
    if (scaling == TSV_ROPE_SCALE_LINEAR) w /= factor;
    if (mixed) {
      const double t = scaling == TSV_ROPE_SCALE_BANDS ? (trained * w / two_pi - low) / (high - low)
                                                       : 1.0 - (i - first) / std::max(last - first, 1e-3);
      const double keep = std::min(std::max(t, 0.0), 1.0);
      w = w * keep + w / factor * (1.0 - keep);
    }
    inv_freq_host[i] = w;
  }
  *amplitude_host = scaling == TSV_ROPE_SCALE_YARN ? (float)(0.1 * log(std::max(factor, 1.0)) + 1.0) : 1.f;
  return TSV_OK;
}

tsv_status tsv_rope(tsv_handle h, tsv_dtype dtype, const void* x_d, int64_t x_stride_n, int64_t x_stride_h,
                    void* y_d, int64_t y_stride_n, int64_t y_stride_h, int32_t N, int32_t H, int32_t D,
                    const int32_t* positions_d, const double* inv_freq_d, int32_t rotary_dim,
                    float amplitude, uint32_t flags, void* stream) {
  if (!h || (dtype != TSV_F32 && dtype != TSV_BF16)) return TSV_ERR_INVALID_ARG;
  if (flags & ~(TSV_ROPE_INTERLEAVED | TSV_ROPE_INVERSE)) return TSV_ERR_INVALID_ARG;
  if (N < 0 || H < 1 || D < 2 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > D) return TSV_ERR_INVALID_ARG;
  if (D > 1024 || (int64_t)H * D > (1 << 30)) return TSV_ERR_UNSUPPORTED;
  if (N == 0) return TSV_OK;
  if (!x_d || !y_d || !positions_d || !inv_freq_d) return TSV_ERR_INVALID_ARG;
  const uintptr_t esz = dtype == TSV_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(x_d) | reinterpret_cast<uintptr_t>(y_d)) % esz || reinterpret_cast<uintptr_t>(positions_d) % 4 ||
      reinterpret_cast<uintptr_t>(inv_freq_d) % 8)
    return TSV_ERR_INVALID_ARG;
  if (x_d == y_d && ((N > 1 && x_stride_n != y_stride_n) || (H > 1 && x_stride_h != y_stride_h)))
    return TSV_ERR_INVALID_ARG;
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  RopeArgs a{};
  a.x = x_d;
  a.y = y_d;
  a.xs_n = x_stride_n;
  a.xs_h = x_stride_h;
  a.ys_n = y_stride_n;
  a.ys_h = y_stride_h;
  a.N = N;
  a.H = H;
  a.D = D;
  a.rot = rotary_dim;
  a.positions = positions_d;
  a.inv_freq = inv_freq_d;
  a.amplitude = amplitude;
  a.interleaved = (flags & TSV_ROPE_INTERLEAVED) ? 1 : 0;
  a.inverse = (flags & TSV_ROPE_INVERSE) ? 1 : 0;
  return cuda_status(launch_rope(a, dtype == TSV_BF16, h->num_sms, static_cast<cudaStream_t>(stream)));
}

tsv_status tsv_paged_append(tsv_handle h, tsv_dtype dtype, const tsv_paged_cache* cache,
                            const tsv_page_table* table, const int32_t* start_d, const void* k_d,
                            int64_t k_stride_n, int64_t k_stride_h, const void* v_d, int64_t v_stride_n,
                            int64_t v_stride_h, const int32_t* row_offsets_d, int32_t B, int32_t N,
                            int32_t max_rows, const int32_t* positions_d, const double* inv_freq_d,
                            int32_t rotary_dim, float amplitude, uint32_t flags, int32_t* status_d,
                            void* stream) {
  if (!h || (dtype != TSV_F32 && dtype != TSV_BF16) || (flags & ~TSV_ROPE_INTERLEAVED)) return TSV_ERR_INVALID_ARG;
  if (B < 1 || B > TSV_MAX_BATCH || N < 0 || max_rows < 0 || !row_offsets_d || !status_d) return TSV_ERR_INVALID_ARG;
  PagedWriteArgs a{};
  tsv_status st = check_paged_cache(cache, &a.cache);
  if (st == TSV_OK) st = check_table(table, B, a.cache);
  if (st != TSV_OK) return st;
  if (inv_freq_d && (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > a.cache.D)) return TSV_ERR_INVALID_ARG;
  const int64_t esz = dtype == TSV_BF16 ? 2 : 4;
  if (N > 0) {
    if (!k_d || !v_d || (inv_freq_d && !positions_d)) return TSV_ERR_INVALID_ARG;
    if (!rows_aligned(k_d, k_stride_n, k_stride_h, esz) || !rows_aligned(v_d, v_stride_n, v_stride_h, esz))
      return TSV_ERR_INVALID_ARG;
  }
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  a.table = *table;
  a.start = start_d;
  a.offsets = row_offsets_d;
  a.B = B;
  a.N = N;
  a.max_rows = std::min(max_rows, N);
  a.status = status_d;
  a.k = k_d;
  a.v = v_d;
  a.ks_n = k_stride_n;
  a.ks_h = k_stride_h;
  a.vs_n = v_stride_n;
  a.vs_h = v_stride_h;
  a.positions = positions_d;
  a.inv_freq = inv_freq_d;
  a.rot = inv_freq_d ? rotary_dim : 0;
  a.interleaved = (flags & TSV_ROPE_INTERLEAVED) ? 1 : 0;
  a.amplitude = amplitude;
  a.head_loop = head_loop(a, std::max<int64_t>(1, cdiv(N, a.cache.page_size) + B / 2), inv_freq_d ? 2 : 0, h->num_sms);
  const uint32_t bit = 1u << ((dtype == TSV_BF16 ? 2 : 0) + (a.cache.D == 128 ? 1 : 0));
  if (!(h->append_attr_mask & bit)) {
    if (paged_append_set_attributes(dtype == TSV_BF16, a.cache.D) != cudaSuccess) return TSV_ERR_CUDA;
    h->append_attr_mask |= bit;
  }
  return cuda_status(launch_paged_append(a, dtype == TSV_BF16, h->num_sms, static_cast<cudaStream_t>(stream)));
}

tsv_status tsv_paged_tree_attention_workspace_size(tsv_handle h, tsv_dtype dtype, const tsv_paged_cache* cache,
                                                   int32_t B, int32_t max_nodes, int32_t Hq, uint32_t flags,
                                                   size_t* bytes) {
  tsv_paged_cache c;
  if (!bytes) return TSV_ERR_INVALID_ARG;
  const tsv_status st = check_attention(h, dtype, cache, &c, B, max_nodes, TSV_MAX_NODES, Hq, flags);
  if (st != TSV_OK) return st;
  const int32_t R = paged_attn_rows((int64_t)max_nodes * (Hq / c.Hkv), (int64_t)B * c.Hkv, TSV_PAGED_MAX_ROWS);  // for every table
  *bytes = paged_uses_tc(dtype, flags) ? paged_attn_layout(h->num_sms, R, c.D).total : 0;
  return TSV_OK;
}

tsv_status tsv_paged_tree_attention(tsv_handle h, tsv_dtype dtype, const void* q_d, int64_t q_stride_n,
                                    int64_t q_stride_h, const tsv_paged_cache* cache,
                                    const tsv_page_table* table, const int32_t* prefix_len_d,
                                    const tsv_page_table* tree_table, const int32_t* node_offsets_d,
                                    const uint32_t* anc_d, void* out_d, int32_t B, int32_t N,
                                    int32_t max_nodes, int32_t Hq, float scale, void* workspace_d,
                                    size_t workspace_bytes, int32_t* status_d, uint32_t flags,
                                    void* stream) {
  PagedAttnArgs a{};
  tsv_status st = check_attention(h, dtype, cache, &a.cache, B, max_nodes, TSV_MAX_NODES, Hq, flags);
  if (st == TSV_OK) st = check_table(table, B, a.cache);
  if (st == TSV_OK && tree_table) st = check_table(tree_table, B, a.cache);
  if (st != TSV_OK) return st;
  if (!prefix_len_d || !node_offsets_d || !status_d || N < 0) return TSV_ERR_INVALID_ARG;
  if (!(scale >= 0.f) || isinf(scale) || (anc_d && !aligned16(anc_d))) return TSV_ERR_INVALID_ARG;
  const int64_t esz = dtype == TSV_BF16 ? 2 : 4;
  if (N > 0 && (!q_d || !out_d || !aligned16(out_d) || !rows_aligned(q_d, q_stride_n, q_stride_h, esz)))
    return TSV_ERR_INVALID_ARG;
  if ((int64_t)N * Hq > INT32_MAX) return TSV_ERR_UNSUPPORTED;
  const bool use_tc = paged_uses_tc(dtype, flags);
  const int32_t R = paged_attn_rows((int64_t)max_nodes * (Hq / a.cache.Hkv), (int64_t)B * a.cache.Hkv,
                                    (int64_t)table->pages * a.cache.page_size);
  if (use_tc && (!workspace_d || !aligned16(workspace_d) ||
                 workspace_bytes < paged_attn_layout(h->num_sms, R, a.cache.D).total))
    return TSV_ERR_INVALID_ARG;
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  a.q = q_d;
  a.qs_n = q_stride_n;
  a.qs_h = q_stride_h;
  a.table = *table;
  if (tree_table) a.tree_table = *tree_table;
  a.prefix_len = prefix_len_d;
  a.offsets = node_offsets_d;
  a.anc = anc_d;
  a.out = out_d;
  a.status = status_d;
  a.B = B;
  a.N = N;
  a.max_nodes = max_nodes;
  a.Hq = Hq;
  a.G = Hq / a.cache.Hkv;
  a.scale = scale == 0.f ? 1.f / sqrtf((float)a.cache.D) : scale;
  if (use_tc) return launch_tree_kernels(h, a, R, workspace_d, static_cast<cudaStream_t>(stream));
  return cuda_status(launch_paged_attention_simt(a, dtype == TSV_BF16, static_cast<cudaStream_t>(stream)));
}

tsv_status tsv_paged_commit(tsv_handle h, const tsv_paged_cache* cache, const tsv_page_table* table,
                            const tsv_page_table* tree_table, const int32_t* prefix_len_d,
                            const int32_t* node_offsets_d, const int32_t* path_d,
                            const int32_t* accept_len_d, int32_t B, int32_t N, int32_t max_nodes,
                            int32_t* new_len_d, int32_t* status_d, void* stream) {
  if (!h || B < 1 || B > TSV_MAX_BATCH || N < 0 || max_nodes < 1 || max_nodes > TSV_MAX_NODES) return TSV_ERR_INVALID_ARG;
  if (!prefix_len_d || !node_offsets_d || !accept_len_d || !status_d || (N > 0 && !path_d)) return TSV_ERR_INVALID_ARG;
  if (new_len_d == prefix_len_d) return TSV_ERR_INVALID_ARG;
  PagedWriteArgs a{};
  tsv_status st = check_paged_cache(cache, &a.cache);
  if (st == TSV_OK) st = check_table(table, B, a.cache);
  if (st == TSV_OK) st = check_table(tree_table, B, a.cache);
  if (st != TSV_OK) return st;
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  a.table = *table;
  a.tree_table = *tree_table;
  a.start = prefix_len_d;
  a.offsets = node_offsets_d;
  a.B = B;
  a.N = N;
  a.max_rows = max_nodes;
  a.status = status_d;
  a.path = path_d;
  a.accept_len = accept_len_d;
  a.new_len = new_len_d;
  a.head_loop = head_loop(a, B + B / 2, 4, h->num_sms);  // (an accepted path ends in one or two pages)
  return cuda_status(launch_paged_commit(a, h->num_sms, static_cast<cudaStream_t>(stream)));
}

tsv_status tsv_paged_chunk_attention_workspace_size(tsv_handle h, tsv_dtype dtype, const tsv_paged_cache* cache, int32_t B,
                                                    int32_t N, int32_t max_rows, int32_t Hq, uint32_t flags, size_t* bytes) {
  tsv_paged_cache c;
  if (!bytes || N < 0) return TSV_ERR_INVALID_ARG;
  const tsv_status st = check_attention(h, dtype, cache, &c, B, max_rows, INT32_MAX, Hq, flags);
  if (st != TSV_OK) return st;
  *bytes = paged_uses_tc(dtype, flags) ? paged_chunk_layout(h->num_sms, c.D).total : 0;  // (more than single tokens want)
  return TSV_OK;
}

tsv_status tsv_paged_chunk_attention(tsv_handle h, tsv_dtype dtype, const void* q_d, int64_t q_stride_n, int64_t q_stride_h,
                                     const tsv_paged_cache* cache, const tsv_page_table* table, const int32_t* start_d,
                                     const int32_t* row_offsets_d, void* out_d, int32_t B, int32_t N, int32_t max_rows,
                                     int32_t Hq, int32_t window, float scale, void* workspace_d, size_t workspace_bytes,
                                     int32_t* status_d, uint32_t flags, void* stream) {
  PagedAttnArgs a{};
  tsv_status st = check_attention(h, dtype, cache, &a.cache, B, max_rows, INT32_MAX, Hq, flags);
  if (st == TSV_OK) st = check_table(table, B, a.cache);
  if (st != TSV_OK) return st;
  if (!start_d || !row_offsets_d || !status_d || N < 0 || window < 0) return TSV_ERR_INVALID_ARG;
  if (!(scale >= 0.f) || isinf(scale)) return TSV_ERR_INVALID_ARG;
  const int64_t esz = dtype == TSV_BF16 ? 2 : 4;
  if (N > 0 && (!q_d || !out_d || !aligned16(out_d) || !rows_aligned(q_d, q_stride_n, q_stride_h, esz)))
    return TSV_ERR_INVALID_ARG;
  if ((int64_t)N * Hq > INT32_MAX) return TSV_ERR_UNSUPPORTED;
  const bool use_tc = paged_uses_tc(dtype, flags), by_chunks = use_tc && (max_rows > 1 || window > 0);
  const bool by_tokens = use_tc && (!by_chunks || (window == 0 && paged_chunk_apart(B, N, max_rows)));
  const int32_t R = chunk_token_rows(Hq / a.cache.Hkv, B, a.cache);
  if (use_tc && (!workspace_d || !aligned16(workspace_d) ||
                 workspace_bytes < std::max(by_chunks ? paged_chunk_layout(h->num_sms, a.cache.D).total : 0,
                                            by_tokens ? paged_attn_layout(h->num_sms, R, a.cache.D).total : 0)))
    return TSV_ERR_INVALID_ARG;
  const DeviceScope scope(h->device);
  if (!scope.ok) return TSV_ERR_CUDA;
  a.q = q_d;
  a.qs_n = q_stride_n;
  a.qs_h = q_stride_h;
  a.table = *table;
  a.prefix_len = start_d;
  a.offsets = row_offsets_d;
  a.out = out_d;
  a.status = status_d;
  a.B = B;
  a.N = N;
  a.max_nodes = max_rows;
  a.Hq = Hq;
  a.G = Hq / a.cache.Hkv;
  a.scale = scale == 0.f ? 1.f / sqrtf((float)a.cache.D) : scale;
  a.chunk = 1;
  a.window = window;
  a.least = 1;
  if (by_tokens) {
    // Requests of more rows do not fit this launch's most: they are passed over, and
    // their status is the joining launch's.
    PagedAttnArgs tokens = a;
    tokens.max_nodes = 1;
    st = launch_tree_kernels(h, tokens, R, workspace_d, static_cast<cudaStream_t>(stream));
    if (st != TSV_OK || !by_chunks) return st;
    a.least = 2;
  }
  if (by_chunks) {
    const uint32_t bit = a.cache.D == 128 ? 2u : 1u;
    if (!(h->chunk_attr_mask & bit)) {
      if (paged_chunk_set_attributes(a.cache.D) != cudaSuccess) return TSV_ERR_CUDA;
      h->chunk_attr_mask |= bit;
    }
    CUtensorMap tk, tv;
    st = encode_pages(h, &tk, a.cache.k_d, a.cache);
    if (st == TSV_OK) st = encode_pages(h, &tv, a.cache.v_d, a.cache);
    if (st != TSV_OK) return st;
    return cuda_status(launch_paged_chunk(tk, tv, a, h->num_sms, workspace_d, static_cast<cudaStream_t>(stream)));
  }
  if (dtype == TSV_F32 && !(flags & TSV_ATTN_SIMT) && max_rows > 1) {
    const uint32_t bit = a.cache.D == 128 ? 8u : 4u;
    if (!(h->chunk_attr_mask & bit)) {
      if (paged_chunk_f32_set_attributes(a.cache.D) != cudaSuccess) return TSV_ERR_CUDA;
      h->chunk_attr_mask |= bit;
    }
    return cuda_status(launch_paged_chunk_f32(a, h->num_sms, static_cast<cudaStream_t>(stream)));
  }
  return cuda_status(launch_paged_attention_simt(a, dtype == TSV_BF16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
