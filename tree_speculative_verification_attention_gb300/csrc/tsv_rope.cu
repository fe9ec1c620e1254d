// tsv_rope.cu — rotary positions on [N, H, D] rows of heads.
//
//   (a, b) -> amplitude * (a cos t - b sin t, b cos t + a sin t),  t = position * w_i
//
// on the first `rot` elements of each head, pairs (i, i + rot/2) or (2i, 2i+1);
// the rest is copied.  Every value is read and written once, so the bound is
// HBM: a CTA takes a few rows, issues the loads of its first vectors, computes
// the rows' rot/2 cosines and sines into shared memory meanwhile (they are the
// same for every head) and then streams the heads in vectors of up to 16 bytes.
// A thread keeps its place in the row (head and element, worked out once) and
// goes down the rows, four vectors in flight: what is left per vector is its
// load, its arithmetic and its store, so that issue stays below the copy's
// time.  A vector of the half layout goes with its partner rot/2 elements on,
// both in one thread's registers; where rot/2 is no multiple of 16 bytes the
// vectors shrink to what divides it.
#include <cuda_runtime.h>

#include <type_traits>

#include "tsv_paged_common.cuh"

namespace tsv {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 2048;  // angles of one CTA's rows

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
template <int BYTES>
using Raw = std::conditional_t<BYTES == 16, uint4,
                               std::conditional_t<BYTES == 8, uint2, std::conditional_t<BYTES == 4, uint32_t, unsigned short>>>;

// n / d of 0 <= n < 2^31 by a multiplication (Granlund and Montgomery's division by
// an invariant): (umulhi(n, m) + n) >> s with s = ceil(log2 d), m = floor(2^32
// (2^s - d) / d) + 1.
struct FastDiv {
  uint32_t d, m;
  int s;
  explicit FastDiv(uint32_t n) : d(n), s(0) {
    while ((1ull << s) < n) ++s;
    m = (uint32_t)((((1ull << s) - n) << 32) / n + 1);
  }
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s); }
};

// Each value is read once and written once: streaming accesses leave the L2 to
// others, and keep the written lines from waiting there (16384 rows x 64 heads x
// 128: 82 us with them, 108 us without; a copy of the same bytes takes 82).
template <typename T, int E>
__device__ __forceinline__ Vec<T, E> load_vec(const T* p) {
  union {
    Raw<sizeof(T) * E> raw;
    Vec<T, E> v;
  } w;
  w.raw = __ldcs(reinterpret_cast<const Raw<sizeof(T) * E>*>(p));
  return w.v;
}
template <typename T, int E>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, E>& v) {
  __stcs(reinterpret_cast<Raw<sizeof(T) * E>*>(p), *reinterpret_cast<const Raw<sizeof(T) * E>*>(&v));
}

constexpr int kVectors = 4;  // vectors of a thread in flight

// E elements per access.  Items of one row: per head, rotated ones, then copied
// ones.  A rotated item is a vector of pairs, or (half layout, and single
// elements) a vector and its partner.
template <typename T, int E, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_kernel(const RopeArgs a, int rows_per_cta, const FastDiv by_row,
                                                            const FastDiv by_items, const FastDiv by_half) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  constexpr bool SPLIT = !INTERLEAVED || E == 1;
  constexpr int PARTS = SPLIT ? 2 : 1, BATCH = kVectors / PARTS;
  constexpr int STEP = INTERLEAVED && SPLIT ? 2 : E;  // from one rotated item to the next
  constexpr int PAIRS = SPLIT ? E : E / 2;            // of an item (even, or one)
  __shared__ alignas(16) float2 table[kRopePairs];    // (cosine, sine) [rows][width]
  const int half = a.rot >> 1, width = (half + 1) & ~1;
  const int n0 = blockIdx.x * rows_per_cta;
  const int rows = min(rows_per_cta, a.N - n0);
  const int partner = INTERLEAVED ? 1 : half;
  const int turn_items = half / PAIRS, items = (int)by_items.d, per_row = (int)by_row.d;
  // The thread's items of a row (one, or every blockDim.x-th), and its rows.
  const int tid = threadIdx.x, threads = blockDim.x;
  const int r0 = by_row.div(tid), at_once = max(1, by_row.div(threads));
  const int i0 = at_once > 1 ? tid - r0 * per_row : tid;
  const int first_row = at_once > 1 ? (r0 < at_once ? r0 : rows) : 0;

  Vec<T, E> v[BATCH][PARTS];
  const T* x;
  T* y;
  bool turn;
  int pair;
  auto place = [&](int i) {
    const int h = by_items.div(i), it = i - h * items;
    turn = it < turn_items;
    pair = it * PAIRS;
    const int d = turn ? it * STEP : a.rot + (it - turn_items) * E;
    x = static_cast<const T*>(a.x) + (int64_t)n0 * a.xs_n + (int64_t)h * a.xs_h + d;
    y = static_cast<T*>(a.y) + (int64_t)n0 * a.ys_n + (int64_t)h * a.ys_h + d;
  };
  auto load = [&](int row) {
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int r = row + u * at_once;
      if (r >= rows) break;
      const T* xr = x + r * a.xs_n;
      v[u][0] = load_vec<T, E>(xr);
      if (SPLIT && turn) v[u][PARTS - 1] = load_vec<T, E>(xr + partner);
    }
  };
  if (i0 < per_row) {
    place(i0);
    load(first_row);
  }
  for (int i = tid; i < rows * half; i += threads) {
    const int r = by_half.div(i), f = i - r * half;
    float c, s;
    rope_cos_sin(a.positions[n0 + r], rope_turns(a.inv_freq[f]), &c, &s);
    table[r * width + f] = make_float2(c * a.amplitude, (a.inverse ? -s : s) * a.amplitude);
  }
  __syncthreads();
  for (int i = i0; i < per_row; i += threads) {
    if (i != i0) {
      place(i);
      load(first_row);
    }
    for (int row = first_row; row < rows; row += BATCH * at_once) {
      if (row != first_row) load(row);
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int r = row + u * at_once;
        if (r >= rows) break;
        T* yr = y + r * a.ys_n;
        if (turn) {
          float cs[2 * PAIRS];
          const float2* t = table + r * width + pair;
          if constexpr (PAIRS == 1) {
            *reinterpret_cast<float2*>(cs) = *t;
          } else {
#pragma unroll
            for (int e = 0; e < PAIRS; e += 2)
              *reinterpret_cast<float4*>(cs + 2 * e) = *reinterpret_cast<const float4*>(t + e);
          }
#pragma unroll
          for (int e = 0; e < PAIRS; ++e) {
            T& first = SPLIT ? v[u][0].v[e] : v[u][0].v[2 * e];
            T& second = SPLIT ? v[u][PARTS - 1].v[e] : v[u][0].v[(2 * e + 1) % E];
            float p = to_f32(first), q = to_f32(second);
            rope_pair(p, q, cs[2 * e], cs[2 * e + 1]);
            first = from_f32<T>(p);
            second = from_f32<T>(q);
          }
          if constexpr (SPLIT) store_vec<T, E>(yr + partner, v[u][1]);
        }
        store_vec<T, E>(yr, v[u][0]);
      }
    }
  }
}

template <typename T, int E>
cudaError_t launch_rope_vec(const RopeArgs& a, int num_sms, cudaStream_t st) {
  const int half = a.rot / 2, parts = a.interleaved && E > 1 ? 1 : 2;
  const int items = a.rot / (E * parts) + (a.D - a.rot) / E, per_row = items * a.H;
  // Threads: of 256 at most, those that whole rows or equal shares of one use.
  const int share = per_row > kRopeThreads ? (per_row + kRopeThreads - 1) / kRopeThreads : 1;
  const int used = share > 1 ? (per_row + share - 1) / share : kRopeThreads / per_row * per_row;
  const int threads = (used + 31) / 32 * 32;
  // Rows per CTA: as many as leave one wave of 40 warps per SM (48 registers a
  // thread), up to 8: beyond it more CTAs are better than longer ones (16384
  // rows x 64 heads x 128: 82 us at 8 rows, 90 in one wave of 22, 113 at 1).
  // The table holds their angles.
  const int64_t resident = (int64_t)num_sms * (40 * 32 / threads);
  const int rows = (int)min(min((a.N + resident - 1) / resident, (int64_t)8), (int64_t)(kRopePairs / ((half + 1) & ~1)));
  const dim3 grid((uint32_t)(((int64_t)a.N + rows - 1) / rows)), block(threads);
  const FastDiv by_row((uint32_t)per_row), by_items((uint32_t)items), by_half((uint32_t)half);
  if (a.interleaved) return launch_pdl(rope_kernel<T, E, true>, grid, block, 0, st, 0u, a, rows, by_row, by_items, by_half);
  return launch_pdl(rope_kernel<T, E, false>, grid, block, 0, st, 0u, a, rows, by_row, by_items, by_half);
}

template <typename T>
cudaError_t launch_typed(const RopeArgs& a, int num_sms, cudaStream_t st) {
  // The widest access that every address, the rotated part (half layout: each
  // half of it) and the copied part are whole multiples of.
  const uintptr_t bits = (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) / sizeof(T);
  const int64_t whole = (int64_t)bits | a.xs_n | a.xs_h | a.ys_n | a.ys_h | a.D | (a.interleaved ? a.rot : a.rot / 2);
  int E = 16 / (int)sizeof(T);
  while (E > 1 && whole % E) E >>= 1;
  if constexpr (sizeof(T) == 2)
    if (E == 8) return launch_rope_vec<T, 8>(a, num_sms, st);
  if (E == 4) return launch_rope_vec<T, 4>(a, num_sms, st);
  if (E == 2) return launch_rope_vec<T, 2>(a, num_sms, st);
  return launch_rope_vec<T, 1>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, num_sms, st) : launch_typed<float>(a, num_sms, st);
}

}  // namespace tsv
