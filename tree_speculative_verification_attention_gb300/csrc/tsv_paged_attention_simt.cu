// tsv_paged_attention_simt.cu — tree attention over a paged 8-bit cache on CUDA
// cores: fp32 queries, and bf16 ones on request (TSV_ATTN_SIMT).
//
//   out[i,h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale <q[i,h], k_j>)
//
// One CTA per (node, KV head): its 16 warps take 32 keys each in turn, a lane
// per key for the scores (its own K row, the query broadcast from shared
// memory) and a lane per D / 32 elements for the sums over V, with a running
// maximum and sum per query head; the warps' partial results are joined in
// shared memory at the end.  A key that the node does not see is skipped, so
// whatever its V row holds stays out.  The K and V rows of a KV head are read
// once per node (from L2).  With the few CTAs of a small batch the chain of a
// warp's 32 keys bounds it (7 us of loads, products and exchanges), so a CTA has
// all the warps that fit and each keeps its whole K rows and eight V rows in
// flight: 3 ragged requests of up to 40 nodes over up to 1500 keys, 8 heads on 2
// KV heads of 64, 24 us (one V row at a time and 8 warps: 74).
#include <cuda_runtime.h>

#include "tsv_paged_common.cuh"

namespace tsv {

namespace {

constexpr int kSimtWarps = 16;
template <int D>
constexpr int simt_heads() { return D == 64 ? 8 : 4; }  // query heads of one pass: what the joined results leave room for
constexpr int kBatch = 8;      // V rows of a warp in flight

template <typename T>
__device__ __forceinline__ float in_f32(T v);
template <>
__device__ __forceinline__ float in_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float in_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T out_of_f32(float v);
template <>
__device__ __forceinline__ float out_of_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 out_of_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// CHUNK: the nodes are new rows of the prefix pages (a.chunk), of which each sees those up
// to its own, or a window of them.
template <typename T, int D, bool CHUNK>
__global__ void __launch_bounds__(32 * kSimtWarps) paged_attn_simt_kernel(const PagedAttnArgs a) {
  constexpr int kSimtHeads = simt_heads<D>();
  constexpr int E = D / 32;  // elements of V per lane
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  __shared__ float sq[kSimtHeads][D];
  __shared__ float so[kSimtWarps][kSimtHeads][D];
  __shared__ float sm[kSimtWarps][kSimtHeads], sl[kSimtWarps][kSimtHeads];
  __shared__ uint32_t sanc[TSV_ANC_WORDS];

  const int node = (int)blockIdx.x - a.B, g = blockIdx.y;  // the first B CTAs of KV head 0 check the requests
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const tsv_paged_cache& C = a.cache;
  if (node < 0) {
    if (g != 0) return;
    const int b = blockIdx.x;
    PagedRequest r;
    bool bad = !paged_request(a, b, &r, CHUNK);
    if (!bad) bad = paged_bad_page(a, b, r, tid, blockDim.x);
    bad = __syncthreads_or(bad);
    if (tid == 0) a.status[b] = bad ? TSV_ERR_INVALID_ARG : TSV_OK;
    return;
  }
  int b = -1;  // the request that owns the row
  for (int i = tid; i < a.B; i += blockDim.x)
    if (node >= a.offsets[i] && node < a.offsets[i + 1]) b = i;
  b = (int)__reduce_max_sync(0xffffffffu, b);
  if (lane == 0) sm[warp][0] = __int_as_float(b);
  __syncthreads();
  for (int w = 0; w < kSimtWarps; ++w) b = max(b, __float_as_int(sm[w][0]));
  __syncthreads();
  if (b < 0) return;
  PagedRequest r;
  if (!paged_request(a, b, &r, CHUNK)) return;
  const int off = r.off, n = r.n, ps = C.page_size;
  const bool tree = !CHUNK && a.tree_table.ids_d != nullptr;
  const int i = node - off;
  // The prefix rows that the node sees: lo .. P - 1.
  const int P = CHUNK ? r.P - n + i + 1 : r.P;
  const int lo = CHUNK && a.window > 0 ? max(0, P - a.window) : 0;
  if (tid < TSV_ANC_WORDS) {
    const int left = i + 1 - 32 * tid;  // chain: bits 0 .. i
    sanc[tid] = !tree ? 0u
                : a.anc ? a.anc[(int64_t)node * TSV_ANC_WORDS + tid]
                        : (left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u);
  }
  const int keys = P + (tree ? n : 0);
  const int32_t* ids = a.table.ids_d + (int64_t)b * a.table.stride;
  const int32_t* tids = tree ? a.tree_table.ids_d + (int64_t)b * a.tree_table.stride : nullptr;
  const T* q = static_cast<const T*>(a.q) + (int64_t)node * a.qs_n;
  T* out = static_cast<T*>(a.out) + ((int64_t)node * a.Hq + (int64_t)g * a.G) * D;

  for (int h0 = 0; h0 < a.G; h0 += kSimtHeads) {
    const int heads = min(kSimtHeads, a.G - h0);
    __syncthreads();
    for (int x = tid; x < heads * D; x += blockDim.x)
      sq[x / D][x % D] = in_f32<T>(q[(int64_t)(g * a.G + h0 + x / D) * a.qs_h + x % D]) * (a.scale * 1.4426950408889634f);
    __syncthreads();
    float m[kSimtHeads], l[kSimtHeads], o[kSimtHeads][E];
#pragma unroll
    for (int h = 0; h < kSimtHeads; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[h][e] = 0.f;
    }
    for (int k0 = (lo & ~31) + warp * 32; k0 < keys; k0 += kSimtWarps * 32) {
      const int key = k0 + lane;
      bool see = key < P;
      if (CHUNK) see = see && key >= lo;
      else if (!see && key < keys) see = (sanc[(key - P) >> 5] >> ((key - P) & 31)) & 1u;
      int64_t row = 0;   // byte offset of the key's row of this head
      float ks = 0.f, vs = 0.f;
      if (see) {
        const int r = key < P ? key : key - P;
        const int id = (key < P ? ids : tids)[r / ps];
        see = id >= 0 && id < C.num_pages;
        if (see) {
          row = (int64_t)id * C.stride_page + (int64_t)(r % ps) * C.stride_row + (int64_t)g * C.stride_head;
          ks = C.k_scale_d[(int64_t)id * C.Hkv + g];
          vs = C.v_scale_d[(int64_t)id * C.Hkv + g];
        }
      }
      const uint32_t seen = __ballot_sync(0xffffffffu, see);
      if (seen == 0u) continue;
      float s[kSimtHeads];
#pragma unroll
      for (int h = 0; h < kSimtHeads; ++h) s[h] = 0.f;
      if (see) {
        const uint4* kr = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(C.k_d) + row);
        uint4 kw[D / 16];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) kw[c] = kr[c];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 w = kw[c];
          float f[16];
          e4m3x4_to_f32(w.x, 1.f, f);
          e4m3x4_to_f32(w.y, 1.f, f + 4);
          e4m3x4_to_f32(w.z, 1.f, f + 8);
          e4m3x4_to_f32(w.w, 1.f, f + 12);
#pragma unroll
          for (int h = 0; h < kSimtHeads; ++h) {
            if (h >= heads) break;
#pragma unroll
            for (int e = 0; e < 16; ++e) s[h] = fmaf(sq[h][16 * c + e], f[e], s[h]);
          }
        }
      }
      float p[kSimtHeads];
#pragma unroll
      for (int h = 0; h < kSimtHeads; ++h) {
        p[h] = 0.f;
        if (h >= heads) continue;
        const float x = see ? s[h] * ks : -INFINITY;
        float top = x;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float mn = fmaxf(m[h], top);
        const float keep = mn == -INFINITY ? 1.f : exp2f(m[h] - mn);
        // A NaN score is kept (it is the node's own business); only unseen keys are 0.
        p[h] = see ? exp2f(x - (mn == -INFINITY ? 0.f : mn)) : 0.f;
        m[h] = mn;
        l[h] = l[h] * keep + p[h];
        p[h] = see ? p[h] * vs : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[h][e] *= keep;
      }
      // The rows of V, kBatch in flight (a row that is not seen is not read).
#pragma unroll 1
      for (int k1 = 0; k1 < 32; k1 += kBatch) {
        if (((seen >> k1) & ((1u << kBatch) - 1u)) == 0u) continue;
        uint32_t vw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const uint8_t* vp = static_cast<const uint8_t*>(C.v_d) + __shfl_sync(0xffffffffu, row, k1 + u) + lane * E;
          vw[u] = 0u;
          if ((seen >> (k1 + u)) & 1u)
            vw[u] = E == 4 ? *reinterpret_cast<const uint32_t*>(vp) : *reinterpret_cast<const uint16_t*>(vp);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          float f[4];
          if constexpr (E == 4) {
            e4m3x4_to_f32(vw[u], 1.f, f);
          } else {
            const uint32_t two = f16x2_of_e4m3x2(vw[u]);
            f[0] = f16_lo(two);
            f[1] = f16_hi(two);
          }
#pragma unroll
          for (int h = 0; h < kSimtHeads; ++h) {
            if (h >= heads) break;
            const float ph = __shfl_sync(0xffffffffu, p[h], k1 + u);
#pragma unroll
            for (int e = 0; e < E; ++e) o[h][e] = fmaf(ph, f[e], o[h][e]);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kSimtHeads; ++h) {
      if (h >= heads) break;
      float sum = l[h];
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      if (lane == 0) {
        sm[warp][h] = m[h];
        sl[warp][h] = sum;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) so[warp][h][lane * E + e] = o[h][e];
    }
    __syncthreads();
    for (int x = tid; x < heads * D; x += blockDim.x) {
      const int h = x / D, d = x % D;
      float top = -INFINITY, sum = 0.f, acc = 0.f;
      for (int w = 0; w < kSimtWarps; ++w) top = fmaxf(top, sm[w][h]);
      for (int w = 0; w < kSimtWarps; ++w) {
        if (sl[w][h] == 0.f) continue;  // this warp saw nothing
        const float f = exp2f(sm[w][h] - (top == -INFINITY ? 0.f : top));
        sum += f * sl[w][h];
        acc += f * so[w][h][d];
      }
      out[(int64_t)(h0 + h) * D + d] = out_of_f32<T>(sum == 0.f ? 0.f : acc / sum);
    }
  }
}

}  // namespace

template <typename T, int D>
static cudaError_t launch_simt_typed(const PagedAttnArgs& a, cudaStream_t st) {
  const dim3 grid(a.N + a.B, a.cache.Hkv), block(32 * kSimtWarps);
  return a.chunk ? launch_pdl(paged_attn_simt_kernel<T, D, true>, grid, block, 0, st, 0u, a)
                 : launch_pdl(paged_attn_simt_kernel<T, D, false>, grid, block, 0, st, 0u, a);
}

cudaError_t launch_paged_attention_simt(const PagedAttnArgs& a, bool bf16, cudaStream_t st) {
  if (bf16) return a.cache.D == 64 ? launch_simt_typed<__nv_bfloat16, 64>(a, st) : launch_simt_typed<__nv_bfloat16, 128>(a, st);
  return a.cache.D == 64 ? launch_simt_typed<float, 64>(a, st) : launch_simt_typed<float, 128>(a, st);
}

}  // namespace tsv
