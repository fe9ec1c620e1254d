// tsv_paged_chunk_f32.cu — causal attention of chunks of new tokens over a paged
// 8-bit cache, fp32 rows.
//
//   S = (Qh + Ql) K^T,  O += v (Ph + Pl) V    per 16 keys, v their page's V scale
//
// fp32 rows are wanted to fp32's accuracy, which one low-precision product does
// not give; but an e4m3 code is an fp16 value, so only the other operand has to be
// split: a row of q (under a power of two that moves its largest value to
// [2^14, 2^15)) and the p of 16 keys (relative to their largest) are two fp16 terms
// each, off by 2^-22 of themselves.  Products of such terms with codes are exact,
// and sums stay short inside the tensor core (it truncates): S over D, O over the
// 16 keys of a step, which are then added to fp32 registers, where the page's V
// scale is a factor of that addition.
//
// That wants accumulators in registers after every step, so warp-level MMAs fit
// better here than ones whose sums live in TMEM.  A CTA takes 64 rows ((token, head
// of the KV head) pairs) with 4 warps of 16, over 64 keys at a time: codes of the
// next block wait in registers while the current one, widened once for all rows,
// is worked on.  With few tiles a cluster shares a tile's keys and joins through
// distributed shared memory.
//
// What bounds it: issue (four products where one would do, and each step's sums added
// to registers), and with few rows a CTA's chain over its keys.  Measured: 2048
// tokens from the start, 8 query heads on 2: 54 TFLOP/s at D = 64, 64 at D = 128
// (fp32 on CUDA cores could be 80 at the very most).  Five ragged chunks under a
// window of 500: 31 us (135 with a CTA a token on the CUDA cores).
#include <cuda_runtime.h>

#include "tsv_paged_common.cuh"

namespace tsv {

namespace {

constexpr int kFThreads = 128, kFRows = 64, kFKeys = 64;
constexpr int kFNanSlots = 6;  // blocks of a tile with masked keys: 3 at each end

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (a, b) as fp16 terms: the nearest, and the nearest of what is left.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = f16_pair(a, b);
  lo = f16_pair(a - f16_lo(hi), b - f16_hi(hi));
}
// D (16 x 8) = A (16 x 16) B (16 x 8) + C, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool TRANS>
__device__ __forceinline__ void load_matrix4(uint32_t (&r)[4], uint32_t at) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint32_t nan_bytes4(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

template <int D>
struct FCfg {
  static constexpr int kRow = 2 * D + 16;  // bytes of a key's fp16 row: 16 more, so that eight rows meet all banks
  static constexpr int kTile = kFKeys * kRow;
  static constexpr int kPartRow = D + 4;  // floats of a row of partial results
  static constexpr int kOffV = kTile, kOffScale = 2 * kTile;  // f32 [2][4]: K's and V's scales of 16 keys
  static constexpr int kOffNan = kOffScale + 32;              // u32 [kFNanSlots][2]
  static constexpr int kOffMl = kOffNan + 8 * kFNanSlots + 16;  // f32 [2][64]
  static constexpr int kOffQ = kOffMl + 8 * kFRows;  // D = 128: q's two terms (registers hold those of D = 64)
  static constexpr bool kQShared = D == 128;
  static constexpr int kSmem = kOffQ + (kQShared ? 2 * kFRows * kRow : 0);
  static_assert(kFRows * kPartRow * 4 <= 2 * kTile, "a partial's rows fit in the tiles");
  static_assert(kOffMl % 16 == 0, "alignment");
};

template <int D>
__global__ void __launch_bounds__(kFThreads) paged_chunk_f32_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = FCfg<D>;
  constexpr int KS = D / 16, NT = D / 8;  // k-steps of S, column tiles of O
  extern __shared__ __align__(16) uint8_t smem[];
  float* sScale = reinterpret_cast<float*>(smem + C::kOffScale);
  uint32_t* sNan = reinterpret_cast<uint32_t*>(smem + C::kOffNan);
  float* sMl = reinterpret_cast<float*>(smem + C::kOffMl);
  __shared__ int sTile[4];  // request, tile of it
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, pair = lane & 3;
  const int g = blockIdx.y, rank = (int)cluster_ctarank(), parts = gridDim.z;  // (a cluster lies along z)
  const tsv_paged_cache& c = a.cache;
  const int lps = __ffs(c.page_size) - 1;
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();

  if (blockIdx.x < a.B && g == 0 && rank == 0) {  // each request is checked by one CTA
    PagedRequest r;
    bool bad = !paged_request(a, blockIdx.x, &r);
    if (!bad) bad = paged_bad_page(a, blockIdx.x, r, tid, kFThreads);
    bad = __syncthreads_or(bad);
    if (tid == 0) a.status[blockIdx.x] = bad ? TSV_ERR_INVALID_ARG : TSV_OK;
  }
  if (warp == 0) {  // the tile's request
    int before = 0;
    if (lane == 0) sTile[0] = -1;
    __syncwarp();
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      PagedRequest r;
      int tiles = 0;
      if (b0 + lane < a.B && paged_request(a, b0 + lane, &r)) tiles = (int)(((int64_t)r.n * a.G + kFRows - 1) / kFRows);
      int upto = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int x = (int)blockIdx.x - before;
      if (x < upto && x >= upto - tiles) {
        sTile[0] = b0 + lane;
        sTile[1] = x - (upto - tiles);
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  if (tid < 2 * kFNanSlots) sNan[tid] = 0u;
  __syncthreads();
  const int b = sTile[0];
  if (b < 0) return;  // (all of a cluster)
  PagedRequest req;
  paged_request(a, b, &req);
  const int row0 = sTile[1] * kFRows, rows = (int)min((int64_t)kFRows, (int64_t)req.n * a.G - row0), start = req.P - req.n;
  const int p_first = start + row0 / a.G, p_last = start + (row0 + rows - 1) / a.G;
  const int j_first = a.window > 0 ? max(0, p_first - a.window + 1) / kFKeys : 0, j_end = p_last / kFKeys + 1;
  // The CTA's share of the blocks.
  const int j0 = j_first + (int)((int64_t)(j_end - j_first) * rank / parts), j1 = j_first + (int)((int64_t)(j_end - j_first) * (rank + 1) / parts);

  // The thread's two rows, and their fragments of q.
  int64_t out_at[2];
  int pos[2];
  float fr[2];
  constexpr int QR = C::kQShared ? 1 : KS;
  uint32_t qh[QR][4], ql[QR][4];
  const uint32_t q_at = smem_u32(smem) + C::kOffQ;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = warp * 16 + quad + 8 * i, gr = row0 + row, token = gr / a.G, head = g * a.G + (gr - token * a.G);
    const bool on = row < rows;
    pos[i] = start + (on ? token : 0);
    out_at[i] = on ? ((int64_t)(req.off + token) * a.Hq + head) * D : -1;
    const float* q = static_cast<const float*>(a.q) + (int64_t)(req.off + token) * a.qs_n + (int64_t)head * a.qs_h;
    float2 x[KS][2];
    float top = 0.f;
    bool fine = true;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[k][h] = on ? __ldg(reinterpret_cast<const float2*>(q + 16 * k + 8 * h + 2 * pair)) : make_float2(0.f, 0.f);
        const float m = fmaxf(fabsf(x[k][h].x), fabsf(x[k][h].y));
        top = fmaxf(top, m);
        fine &= fabsf(x[k][h].x) < INFINITY && fabsf(x[k][h].y) < INFINITY;
      }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = top < INFINITY ? (int)(__float_as_uint(top) >> 23) : 127;
    const int up = top == 0.f ? 0 : max(-120, min(120, 141 - e));
    const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
    fr[i] = __uint_as_float((uint32_t)(127 - up) << 23) * (a.scale * 1.4426950408889634f);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hi, lo;
        split_pair(x[k][h].x * mul, x[k][h].y * mul, hi, lo);
        // A row with an infinity or a NaN is NaN throughout (its scores are).
        if (!fine) hi = lo = 0x7FFF7FFFu;
        if constexpr (C::kQShared) {
          uint32_t* to = reinterpret_cast<uint32_t*>(smem + C::kOffQ + row * C::kRow + 32 * k + 16 * h + 4 * pair);
          to[0] = hi;
          to[kFRows * C::kRow / 4] = lo;
        } else {
          qh[k][i + 2 * h] = hi;
          ql[k][i + 2 * h] = lo;
        }
      }
  }

  // Codes of a block: a thread takes 16 codes of rows first_row, first_row + kStep, ...
  constexpr int kLanes = D / 16, kStep = kFThreads / kLanes, kPer = kFKeys / kStep;
  const int chunk = tid % kLanes, first_row = tid / kLanes;
  const int32_t* ids = a.table.ids_d + (int64_t)b * a.table.stride;
  const int keys = p_last + 1;
  // Keys in front of the tile's first window, as far as they fill 16: no scale is read of
  // what may be there (0 weights times a scale that is not finite would be NaN).
  const int front = a.window > 0 ? max(0, p_first - a.window + 1) & ~15 : 0;
  uint4 kc[kPer], vc[kPer];
  float scale = 0.f;  // threads 0 .. 7: K's, then V's scales of 16 keys
  auto fetch = [&](int j) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int key = j * kFKeys + first_row + i * kStep;
      kc[i] = vc[i] = make_uint4(0u, 0u, 0u, 0u);
      if (key >= keys) continue;
      const int id = __ldg(ids + (key >> lps));
      if ((uint32_t)id >= (uint32_t)c.num_pages) continue;
      const int64_t at = (int64_t)id * c.stride_page + (int64_t)(key & ((1 << lps) - 1)) * c.stride_row + (int64_t)g * c.stride_head + 16 * chunk;
      kc[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.k_d) + at));
      vc[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.v_d) + at));
    }
    scale = 0.f;
    if (tid < 8) {
      const int key = j * kFKeys + 16 * (tid & 3);
      const int id = key < keys && key >= front ? __ldg(ids + (key >> lps)) : -1;
      if ((uint32_t)id < (uint32_t)c.num_pages) scale = __ldg((tid < 4 ? c.k_scale_d : c.v_scale_d) + (int64_t)id * c.Hkv + g);
    }
  };
  auto widen = [&](uint8_t* tile, int key, const uint4& w) {
    uint4* to = reinterpret_cast<uint4*>(tile + key * C::kRow + 32 * chunk);
    to[0] = make_uint4(f16x2_of_e4m3x2(w.x & 0xFFFFu), f16x2_of_e4m3x2(w.x >> 16), f16x2_of_e4m3x2(w.y & 0xFFFFu), f16x2_of_e4m3x2(w.y >> 16));
    to[1] = make_uint4(f16x2_of_e4m3x2(w.z & 0xFFFFu), f16x2_of_e4m3x2(w.z >> 16), f16x2_of_e4m3x2(w.w & 0xFFFFu), f16x2_of_e4m3x2(w.w >> 16));
  };

  float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  const uint32_t k_at = smem_u32(smem), v_at = k_at + C::kOffV;
  if (j0 < j1) fetch(j0);
#pragma unroll 1
  for (int j = j0; j < j1; ++j) {
    const bool masked = j * kFKeys + kFKeys - 1 > p_first || (a.window > 0 && j * kFKeys <= p_last - a.window);
    __syncthreads();  // everyone is done with the block before
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int key = first_row + i * kStep;
      widen(smem, key, kc[i]);
      if (masked) {  // NaN codes come back into the rows that see them, below
        uint32_t* w = reinterpret_cast<uint32_t*>(&vc[i]);
        uint32_t any = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t bad = nan_bytes4(w[e]);
          any |= bad;
          w[e] &= ~((bad >> 7) * 0xFFu);
        }
        const int slot = j - j_first < 3 ? j - j_first : 3 + j_end - 1 - j;
        if (any && slot < kFNanSlots) atomicOr(&sNan[2 * slot + (key >> 5)], 1u << (key & 31));
      }
      widen(smem + C::kOffV, key, vc[i]);
    }
    if (tid < 8) sScale[tid] = scale;
    __syncthreads();
    if (j + 1 < j1) fetch(j + 1);  // on its way under the products

    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int kq = C::kQShared ? 0 : k;
      if constexpr (C::kQShared) {
        const uint32_t at = q_at + (warp * 16 + (lane & 15)) * C::kRow + 32 * k + 16 * (lane >> 4);
        load_matrix4<false>(qh[0], at);
        load_matrix4<false>(ql[0], at + kFRows * C::kRow);
      }
#pragma unroll
      for (int n = 0; n < 8; n += 2) {  // 16 keys: two column tiles, both halves of the step
        uint32_t w[4];
        const int key = 8 * n + (lane & 7) + 8 * (lane >> 4);
        load_matrix4<false>(w, k_at + key * C::kRow + 32 * k + 16 * ((lane >> 3) & 1));
        mma_16816(s[n], ql[kq], w[0], w[1]);
        mma_16816(s[n + 1], ql[kq], w[2], w[3]);
        mma_16816(s[n], qh[kq], w[0], w[1]);
        mma_16816(s[n + 1], qh[kq], w[2], w[3]);
      }
    }
    // The rows' maxima move, and what was summed up with them.  A step's weights are
    // held relative to its own largest, 2^shift of the row's: V scales may lie far
    // apart, and a row's small weights count where they are large.
    float alpha[2], ref[4][2], shift[4][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top[4], all = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = sScale[k] * fr[i];
        top[k] = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = s[2 * k + h][2 * i + e] * f;
            if (masked) {
              const int back = pos[i] - (j * kFKeys + 16 * k + 8 * h + 2 * pair + e);
              if (back < 0 || (a.window > 0 && back >= a.window)) x = -INFINITY;
            }
            s[2 * k + h][2 * i + e] = x;
            top[k] = fmaxf(top[k], x);
          }
        top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 1));
        top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 2));
        all = fmaxf(all, top[k]);
      }
      const float now = fmaxf(m[i], all);
      alpha[i] = now == -INFINITY ? 1.f : fast_exp2(m[i] - now);
      m[i] = now;
      l[i] *= alpha[i];
      const float base = now == -INFINITY ? 0.f : now;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float d = fmaxf(floorf(top[k] - base), -100.f);  // (a whole number: 2^d is exact)
        ref[k][i] = base + d;
        shift[k][i] = __uint_as_float((uint32_t)(127 + (int)d) << 23);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      o[n][0] *= alpha[0];
      o[n][1] *= alpha[0];
      o[n][2] *= alpha[1];
      o[n][3] *= alpha[1];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // 16 keys a step
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = fast_exp2(s[2 * k + h][2 * i] - ref[k][i]), y = fast_exp2(s[2 * k + h][2 * i + 1] - ref[k][i]);
          l[i] = fmaf(x + y, shift[k][i], l[i]);
          split_pair(x * 8192.f, y * 8192.f, ph[i + 2 * h], pl[i + 2 * h]);
        }
      const float v[2] = {sScale[4 + k] * (shift[k][0] * 0x1p-13f), sScale[4 + k] * (shift[k][1] * 0x1p-13f)};
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t w[4];
        load_matrix4<true>(w, v_at + (16 * k + (lane & 7) + 8 * ((lane >> 3) & 1)) * C::kRow + 16 * (n + (lane >> 4)));
        float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
        mma_16816(d0, pl, w[0], w[1]);
        mma_16816(d1, pl, w[2], w[3]);
        mma_16816(d0, ph, w[0], w[1]);
        mma_16816(d1, ph, w[2], w[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[n][e] = fmaf(d0[e], v[e >> 1], o[n][e]);
          o[n + 1][e] = fmaf(d1[e], v[e >> 1], o[n + 1][e]);
        }
      }
    }
  }
  __syncthreads();  // (NaN words are complete, the tiles idle)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }
  // NaN codes that were kept out of the products, back into the rows that see them.
#pragma unroll 1
  for (int w = 0; w < 2 * kFNanSlots; ++w) {
    const int slot = w >> 1, jb = slot < 3 ? j_first + slot : j_end - 1 - (slot - 3);
#pragma unroll 1
    for (uint32_t seen = sNan[w]; seen; seen &= seen - 1) {
      const int key = jb * kFKeys + 32 * (w & 1) + __ffs(seen) - 1;
      const int id = __ldg(ids + (key >> lps));
      if ((uint32_t)id >= (uint32_t)c.num_pages) continue;
      const uint8_t* v = static_cast<const uint8_t*>(c.v_d) + (int64_t)id * c.stride_page + (int64_t)(key & ((1 << lps) - 1)) * c.stride_row +
                         (int64_t)g * c.stride_head;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int back = pos[e >> 1] - key;
          if (back >= 0 && (a.window == 0 || back < a.window) && (__ldg(v + 8 * n + 2 * pair + (e & 1)) & 0x7F) == 0x7F) o[n][e] = NAN;
        }
    }
  }
  float* out = static_cast<float*>(a.out);
  if (parts == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (out_at[i] < 0) continue;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float2*>(out + out_at[i] + 8 * n + 2 * pair) = make_float2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
    }
    return;
  }
  // The cluster's parts of every row, through shared memory.
  float* sPart = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = warp * 16 + quad + 8 * i;
    if (pair == 0) {
      sMl[row] = m[i];
      sMl[kFRows + row] = l[i];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float2*>(sPart + row * C::kPartRow + 8 * n + 2 * pair) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
  }
  cluster_sync_all();
  constexpr int L4 = D / 4;
  const int mine = kFRows / parts;  // rows that this CTA joins
  for (int i = tid; i < mine * L4; i += kFThreads) {
    const int row = rank * mine + i / L4, d4 = (i % L4) * 4;
    if (row >= rows) break;
    float top = -INFINITY, sum = 0.f;
    for (int r = 0; r < parts; ++r) top = fmaxf(top, ld_dsmem_f32(mapa_shared(smem_u32(sMl + row), (uint32_t)r)));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < parts; ++r) {
      const float pm = ld_dsmem_f32(mapa_shared(smem_u32(sMl + row), (uint32_t)r));
      const float pl = ld_dsmem_f32(mapa_shared(smem_u32(sMl + kFRows + row), (uint32_t)r));
      const float4 v = ld_dsmem_f32x4(mapa_shared(smem_u32(sPart + row * C::kPartRow + d4), (uint32_t)r));
      const float w = pm == -INFINITY ? 1.f : fast_exp2(pm - top);  // (a part without keys is zeros; one of NaN keeps them)
      sum = fmaf(pl, w, sum);
      acc.x = fmaf(v.x, w, acc.x);
      acc.y = fmaf(v.y, w, acc.y);
      acc.z = fmaf(v.z, w, acc.z);
      acc.w = fmaf(v.w, w, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int gr = row0 + row, token = gr / a.G;
    *reinterpret_cast<float4*>(out + ((int64_t)(req.off + token) * a.Hq + g * a.G + (gr - token * a.G)) * D + d4) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
  cluster_sync_all();  // the others have read this CTA's part
}

template <int D>
cudaError_t launch_f32_typed(const PagedAttnArgs& a, int num_sms, cudaStream_t st) {
  const int64_t tiles = (int64_t)a.N * a.G / kFRows + a.B;  // at most
  if (tiles > INT32_MAX || a.cache.Hkv > 65535) return cudaErrorInvalidValue;
  // With fewer tiles than two a SM their keys are shared, four blocks a CTA at least.
  const int64_t blocks = ((int64_t)a.table.pages * a.cache.page_size + kFKeys - 1) / kFKeys;
  int parts = 1;
  while (parts < 8 && tiles * a.cache.Hkv * parts < 2 * num_sms && blocks >= 8 * parts) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, a.cache.Hkv, parts);
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = FCfg<D>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = parts;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, paged_chunk_f32_kernel<D>, a);
}

}  // namespace

cudaError_t paged_chunk_f32_set_attributes(int32_t D) {
  return D == 64 ? cudaFuncSetAttribute(paged_chunk_f32_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, FCfg<64>::kSmem)
                 : cudaFuncSetAttribute(paged_chunk_f32_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, FCfg<128>::kSmem);
}

cudaError_t launch_paged_chunk_f32(const PagedAttnArgs& a, int num_sms, cudaStream_t st) {
  return a.cache.D == 64 ? launch_f32_typed<64>(a, num_sms, st) : launch_f32_typed<128>(a, num_sms, st);
}

}  // namespace tsv
