// tsv_rope.cu — rotary positions on [N, H, D] rows of heads.
//
//   (a, b) -> amplitude * (a cos t - b sin t, b cos t + a sin t),  t = position * w_i
//
// on the first `rot` elements of each head, pairs (i, i + rot/2) or (2i, 2i+1);
// the rest is copied.  Every value is read and written once, so the bound is
// HBM: a CTA takes a few rows, issues the loads of its first vectors, computes
// the rows' rot/2 cosines and sines into shared memory meanwhile (they are the
// same for every head) and then streams the heads in vectors of up to 16 bytes,
// four of them in flight per thread.  A vector of the half layout goes with
// its partner rot/2 elements on, both in one thread's registers; where rot/2 is
// no multiple of 16 bytes the vectors shrink to what divides it.
#include <cuda_runtime.h>

#include "tsv_paged_common.cuh"

namespace tsv {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTableFloats = 2 * 2048;  // cosines and sines of one CTA's rows

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int E>
struct alignas(sizeof(T) * E) Vec {
  T v[E];
};

// n / d of 0 <= n < 2^31 by a multiplication: q = (umulhi(n, m) + n) >> s with
// s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1 (a division each for row,
// head and vector would cost as much issue time as the vector's own work).
struct FastDiv {
  uint32_t d, m;
  int s;
  explicit FastDiv(uint32_t n) : d(n), s(0) {
    while ((1ull << s) < n) ++s;
    m = (uint32_t)((((1ull << s) - n) << 32) / n + 1);
  }
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s); }
};

constexpr int kVectors = 4;  // vectors of a thread in flight

// E elements per access.  Items of one head: rotated ones, then copied ones.  A
// rotated item is a vector of pairs, or (half layout, and single elements) a
// vector and its partner.
template <typename T, int E, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int rows_per_cta, const FastDiv by_row,
                                                            const FastDiv by_head) {
  pdl_trigger();
  pdl_wait();
  __shared__ float table[kRopeTableFloats];
  constexpr bool SPLIT = !INTERLEAVED || E == 1;
  constexpr int PARTS = SPLIT ? 2 : 1, kBatch = kVectors / PARTS;
  constexpr int STEP = INTERLEAVED && SPLIT ? 2 : E;  // from one rotated item to the next
  const int half = a.rot >> 1;
  const int n0 = blockIdx.x * rows_per_cta;
  const int rows = min(rows_per_cta, a.N - n0);
  float* tc = table;
  float* ts = table + rows_per_cta * half;
  const int partner = INTERLEAVED ? 1 : half;
  const int turn_items = (SPLIT ? half : a.rot) / E;
  const T* x = static_cast<const T*>(a.x) + (int64_t)n0 * a.xs_n;
  T* y = static_cast<T*>(a.y) + (int64_t)n0 * a.ys_n;
  const int total = rows * (int)by_row.d;
  Vec<T, E> v[kBatch][PARTS];
  struct Item {
    int r, h, it, d;  // row, head, item, first element
  };
  auto item = [&](int i) {
    Item k;
    k.r = by_row.div(i);
    const int in_row = i - k.r * (int)by_row.d;
    k.h = by_head.div(in_row);
    k.it = in_row - k.h * (int)by_head.d;
    k.d = k.it < turn_items ? k.it * STEP : a.rot + (k.it - turn_items) * E;
    return k;
  };
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kRopeThreads;
      if (i >= total) break;
      const Item k = item(i);
      const T* xr = x + k.r * a.xs_n + k.h * a.xs_h + k.d;
      v[u][0] = *reinterpret_cast<const Vec<T, E>*>(xr);
      if (SPLIT && k.it < turn_items) v[u][PARTS - 1] = *reinterpret_cast<const Vec<T, E>*>(xr + partner);
    }
  };
  load(threadIdx.x);
  for (int i = threadIdx.x; i < rows * half; i += kRopeThreads) {
    const int r = i / half, f = i - r * half;
    float c, s;
    rope_cos_sin(a.positions[n0 + r], rope_turns(a.inv_freq[f]), &c, &s);
    tc[i] = c * a.amplitude;
    ts[i] = (a.inverse ? -s : s) * a.amplitude;
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < total; i0 += kBatch * kRopeThreads) {
    if (i0 != (int)threadIdx.x) load(i0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kRopeThreads;
      if (i >= total) break;
      const Item k = item(i);
      T* yr = y + k.r * a.ys_n + k.h * a.ys_h + k.d;
      if (k.it < turn_items) {
        const float* c = tc + k.r * half;
        const float* s = ts + k.r * half;
        if constexpr (!SPLIT) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            float p = to_f32(v[u][0].v[e]), q = to_f32(v[u][0].v[e + 1]);
            rope_pair(p, q, c[(k.d + e) >> 1], s[(k.d + e) >> 1]);
            v[u][0].v[e] = from_f32<T>(p);
            v[u][0].v[e + 1] = from_f32<T>(q);
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float p = to_f32(v[u][0].v[e]), q = to_f32(v[u][1].v[e]);
            const int f = INTERLEAVED ? k.it : k.d + e;
            rope_pair(p, q, c[f], s[f]);
            v[u][0].v[e] = from_f32<T>(p);
            v[u][1].v[e] = from_f32<T>(q);
          }
          *reinterpret_cast<Vec<T, E>*>(yr + partner) = v[u][1];
        }
      }
      *reinterpret_cast<Vec<T, E>*>(yr) = v[u][0];
    }
  }
}

template <typename T, int E>
cudaError_t launch_rope_vec(const RopeArgs& a, int rows, cudaStream_t st) {
  const int items = (a.interleaved && E > 1 ? a.rot / E : a.rot / 2 / E) + (a.D - a.rot) / E;
  const FastDiv by_head((uint32_t)items), by_row((uint32_t)items * (uint32_t)a.H);
  const dim3 grid((a.N + rows - 1) / rows), block(kRopeThreads);
  if (a.interleaved) return launch_pdl(rope_kernel<T, E, true>, grid, block, 0, st, 0u, a, rows, by_row, by_head);
  return launch_pdl(rope_kernel<T, E, false>, grid, block, 0, st, 0u, a, rows, by_row, by_head);
}

template <typename T>
cudaError_t launch_typed(const RopeArgs& a, int num_sms, cudaStream_t st) {
  // The widest access that every address, the rotated part (half layout: each
  // half of it) and the copied part are whole multiples of.
  const uintptr_t bits = (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) / sizeof(T);
  const int64_t whole = (int64_t)bits | a.xs_n | a.xs_h | a.ys_n | a.ys_h | a.D | (a.interleaved ? a.rot : a.rot / 2);
  int E = 16 / (int)sizeof(T);
  while (E > 1 && whole % E) E >>= 1;
  const int half = a.rot / 2;
  // Rows per CTA: enough for kVectors a thread, as far as the table holds
  // their angles and every SM keeps a CTA.
  const int64_t row_items = (int64_t)a.H * a.D / E;
  int rows = (int)((kVectors * kRopeThreads + row_items - 1) / row_items);
  // A few more where the angles would leave threads idle, as long as 8 CTAs per SM remain.
  rows = max(rows, min((kRopeThreads + half - 1) / half, a.N / (8 * num_sms)));
  rows = min(rows, (kRopeTableFloats / 2) / half);
  rows = max(1, min(rows, a.N / num_sms));
  if constexpr (sizeof(T) == 2)
    if (E == 8) return launch_rope_vec<T, 8>(a, rows, st);
  if (E == 4) return launch_rope_vec<T, 4>(a, rows, st);
  if (E == 2) return launch_rope_vec<T, 2>(a, rows, st);
  return launch_rope_vec<T, 1>(a, rows, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, num_sms, st) : launch_typed<float>(a, num_sms, st);
}

}  // namespace tsv
