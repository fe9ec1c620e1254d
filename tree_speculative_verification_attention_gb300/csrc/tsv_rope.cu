// tsv_rope.cu — rotary positions on [N, H, D] rows of heads.
//
//   (a, b) -> amplitude * (a cos t - b sin t, b cos t + a sin t),  t = position * w_i
//
// on the first `rot` elements of each head, pairs (i, i + rot/2) or (2i, 2i+1);
// the rest is copied.  Every value is read and written once, so the bound is
// HBM: a CTA takes a few rows, computes their rot/2 cosines and sines once
// into shared memory (they are the same for every head) and then streams the
// heads in 16-byte vectors.  A vector of the half layout goes with its partner
// rot/2 elements on, both in one thread's registers.
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

// E elements per access: 16 bytes when everything is aligned, else 1 (half
// layout) or 1 x 2 scalars (interleaved: a pair is two accesses).
template <typename T, int E, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int rows_per_cta) {
  pdl_trigger();
  pdl_wait();
  __shared__ float table[kRopeTableFloats];
  const int half = a.rot >> 1;
  const int n0 = blockIdx.x * rows_per_cta;
  const int rows = min(rows_per_cta, a.N - n0);
  float* tc = table;
  float* ts = table + rows_per_cta * half;
  for (int i = threadIdx.x; i < rows * half; i += kRopeThreads) {
    const int r = i / half, f = i - r * half;
    float c, s;
    rope_cos_sin(a.positions[n0 + r], rope_turns(a.inv_freq[f]), &c, &s);
    tc[i] = c * a.amplitude;
    ts[i] = (a.inverse ? -s : s) * a.amplitude;
  }
  __syncthreads();
  // Work items of one head: rotated vectors, then copied ones.
  constexpr int P = (INTERLEAVED && E == 1) ? 2 : E;  // elements of an item's first access(es)
  const int turn_items = INTERLEAVED ? a.rot / P : half / E;
  const int items = turn_items + (a.D - a.rot + P - 1) / P;
  const int per_row = items * a.H;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  for (int i = threadIdx.x; i < rows * per_row; i += kRopeThreads) {
    const int r = i / per_row, k = i - r * per_row;
    const int h = k / items, it = k - h * items;
    const T* xr = x + (int64_t)(n0 + r) * a.xs_n + (int64_t)h * a.xs_h;
    T* yr = y + (int64_t)(n0 + r) * a.ys_n + (int64_t)h * a.ys_h;
    const float* c = tc + r * half;
    const float* s = ts + r * half;
    if (it >= turn_items) {
      const int d = a.rot + (it - turn_items) * P;
      if constexpr (E > 1) {
        *reinterpret_cast<Vec<T, E>*>(yr + d) = *reinterpret_cast<const Vec<T, E>*>(xr + d);
      } else {
        for (int e = 0; e < P && d + e < a.D; ++e) yr[d + e] = xr[d + e];
      }
    } else if constexpr (INTERLEAVED) {
      const int d = it * P;
      Vec<T, P> v;
      if constexpr (E > 1) {
        v = *reinterpret_cast<const Vec<T, P>*>(xr + d);
      } else {
        v.v[0] = xr[d];
        v.v[1] = xr[d + 1];
      }
#pragma unroll
      for (int e = 0; e < P; e += 2) {
        float p = to_f32(v.v[e]), q = to_f32(v.v[e + 1]);
        rope_pair(p, q, c[(d + e) >> 1], s[(d + e) >> 1]);
        v.v[e] = from_f32<T>(p);
        v.v[e + 1] = from_f32<T>(q);
      }
      if constexpr (E > 1) {
        *reinterpret_cast<Vec<T, P>*>(yr + d) = v;
      } else {
        yr[d] = v.v[0];
        yr[d + 1] = v.v[1];
      }
    } else {
      const int d = it * E;
      Vec<T, E> u = *reinterpret_cast<const Vec<T, E>*>(xr + d);
      Vec<T, E> w = *reinterpret_cast<const Vec<T, E>*>(xr + d + half);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float p = to_f32(u.v[e]), q = to_f32(w.v[e]);
        rope_pair(p, q, c[d + e], s[d + e]);
        u.v[e] = from_f32<T>(p);
        w.v[e] = from_f32<T>(q);
      }
      *reinterpret_cast<Vec<T, E>*>(yr + d) = u;
      *reinterpret_cast<Vec<T, E>*>(yr + d + half) = w;
    }
  }
}

template <typename T>
cudaError_t launch_typed(const RopeArgs& a, int num_sms, cudaStream_t st) {
  constexpr int E = 16 / (int)sizeof(T);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
  const int64_t strides = a.xs_n | a.xs_h | a.ys_n | a.ys_h;
  const int group = a.interleaved ? E : 2 * E;  // rot covers whole vectors (and, half layout, whole partners)
  const bool wide = bits % 16 == 0 && strides % E == 0 && a.D % E == 0 && a.rot % group == 0;
  const int half = a.rot / 2;
  // Rows per CTA: enough for about 4 vectors a thread, as far as the table
  // holds their angles and every SM keeps a CTA.
  const int64_t row_elems = (int64_t)a.H * a.D;
  int rows = (int)((4 * kRopeThreads * (wide ? E : 1) + row_elems - 1) / row_elems);
  rows = min(rows, (kRopeTableFloats / 2) / half);
  rows = max(1, min(rows, a.N / num_sms));
  const dim3 grid((a.N + rows - 1) / rows), block(kRopeThreads);
  if (wide && a.interleaved) return launch_pdl(rope_kernel<T, E, true>, grid, block, 0, st, 0u, a, rows);
  if (wide) return launch_pdl(rope_kernel<T, E, false>, grid, block, 0, st, 0u, a, rows);
  if (a.interleaved) return launch_pdl(rope_kernel<T, 1, true>, grid, block, 0, st, 0u, a, rows);
  return launch_pdl(rope_kernel<T, 1, false>, grid, block, 0, st, 0u, a, rows);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, num_sms, st) : launch_typed<float>(a, num_sms, st);
}

}  // namespace tsv
