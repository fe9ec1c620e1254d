// tsv_paged_common.cuh — device helpers of the paged 8-bit cache: e4m3
// conversion, power-of-two scales, rotary angles, page lookups.
#pragma once

#include "tsv_device.cuh"
#include "tsv_internal.h"

namespace tsv {

// Two fp32 values -> two e4m3 codes (lo in the low byte), nearest even,
// saturating to +-448; NaN -> NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes (low 16 bits of v) -> two fp16 values, exactly.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t v) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(v));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t v) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(v));
  return f;
}

// Four e4m3 codes of a word, times `s`.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float s, float* f) {
  const uint32_t a = f16x2_of_e4m3x2(w & 0xFFFFu), b = f16x2_of_e4m3x2(w >> 16);
  f[0] = f16_lo(a) * s;
  f[1] = f16_hi(a) * s;
  f[2] = f16_lo(b) * s;
  f[3] = f16_hi(b) * s;
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 x 2^8),
// from the bits of a finite amax >= 0.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}
// 1 / s of such a scale, exactly.
__device__ __forceinline__ float pow2_inverse(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// |x| of a finite x, else 0 (infinities and NaN do not take part in a scale).
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Rotary angles.  A frequency is kept as a fraction of a turn per position in
// 64-bit fixed point, rounded to nearest, so that position x frequency modulo one
// turn is an integer product: its error is |position| x 2^-65 turns.
__device__ __forceinline__ uint64_t rope_turns(double w) {
  // w = m 2^(e - 1075) with a 53-bit integer m; 2^64 w / (2 pi) = m C 2^(e - 1077)
  // with C = 2^66 / (2 pi).  Integers throughout: fp64 runs at a small fraction
  // of their rate here.
  constexpr uint64_t C = 0xa2f9836e4e44152aull;
  const uint64_t u = (uint64_t)__double_as_longlong(w);
  const int e = (int)(u >> 52) & 0x7FF;
  const uint64_t m = (u & 0xFFFFFFFFFFFFFull) | (1ull << 52);
  const uint64_t hi = __umul64hi(m, C), lo = m * C;
  const int sh = 1077 - e;
  uint64_t t;  // the product's bits from bit sh on, and the one below them
  if (e == 0 || sh > 128) t = 0;
  else if (sh > 64) t = (sh < 128 ? hi >> (sh - 64) : 0ull) + ((hi >> (sh - 65)) & 1ull);
  else if (sh == 64) t = hi + (lo >> 63);
  else if (sh > 0) t = ((lo >> sh) | (hi << (64 - sh))) + ((lo >> (sh - 1)) & 1ull);
  else t = sh > -64 ? lo << -sh : 0;
  return (u >> 63) ? 0ull - t : t;
}

__device__ __forceinline__ void rope_cos_sin(int32_t position, uint64_t turns, float* c, float* s) {
  const uint64_t t = turns * (uint64_t)(int64_t)position;  // fraction of a turn x 2^64, as a signed number in [-1/2, 1/2)
  // Its upper half rounded to a float; cosine and sine of that are turned on by
  // the rest (64 x 2^-32 turns at most, so that its square, 2^-46, does not count;
  // an upper half that rounds to 2^31 comes back as one less).
  const int32_t hi = (int32_t)(uint32_t)(t >> 32);
  const float f = (float)hi;
  const float rest = fmaf((float)(uint32_t)t, 0x1p-32f, (float)(hi - (int32_t)f - (f == 0x1p31f ? 1 : 0))) * 1.4629180792671596e-9f;  // pi 2^-31
  float s0, c0;
  sincospif(f * 4.656612873077392578125e-10f, &s0, &c0);  // 2^-31: half turns
  *c = fmaf(-s0, rest, c0);
  *s = fmaf(c0, rest, s0);
}

// One rotated pair.  The roundings are spelled out: every kernel and vector
// width gives the same bits.
__device__ __forceinline__ void rope_pair(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fmaf_rn(x, c, -__fmul_rn(y, s));
  b = __fmaf_rn(y, c, __fmul_rn(x, s));
}

// Lengths of request b of an attention call; false when they do not fit the
// call (the request is then skipped by every kernel).  Of a chunk, P counts the
// new rows too.
struct PagedRequest {
  int off, n, P;
};
__device__ __forceinline__ bool paged_request(const PagedAttnArgs& a, int b, PagedRequest* r, bool chunk) {
  const int ps = a.cache.page_size;
  r->off = __ldg(a.offsets + b);
  const int end = __ldg(a.offsets + b + 1);
  r->P = __ldg(a.prefix_len + b);
  r->n = end - r->off;
  if (chunk && r->P >= 0 && r->n >= 0) r->P = (int)min((int64_t)r->P + r->n, (int64_t)INT32_MAX);
  return r->off >= 0 && end >= r->off && end <= a.N && r->n <= a.max_nodes && r->P >= 0 &&
         (int64_t)r->P <= (int64_t)a.table.pages * ps &&
         (a.tree_table.ids_d == nullptr || (int64_t)r->n <= (int64_t)a.tree_table.pages * ps);
}

__device__ __forceinline__ bool paged_request(const PagedAttnArgs& a, int b, PagedRequest* r) { return paged_request(a, b, r, a.chunk != 0); }

// Whether a page id that the request needs is out of range, as far as the
// calling thread's share (index t of `threads`) goes.  A chunk needs the pages
// from the first row's window on, and none without new rows.
__device__ __forceinline__ bool paged_bad_page(const PagedAttnArgs& a, int b, const PagedRequest& r, int t, int threads) {
  const int ps = a.cache.page_size;
  bool bad = false;
  const int32_t* ids = a.table.ids_d + (int64_t)b * a.table.stride;
  const int first = a.window > 0 ? max(0, r.P - r.n + 1 - a.window) / ps : 0;
  const int end = a.chunk && r.n == 0 ? 0 : (r.P + ps - 1) / ps;
  for (int i = first + t; i < end; i += threads) bad |= (uint32_t)ids[i] >= (uint32_t)a.cache.num_pages;
  if (a.tree_table.ids_d) {
    ids = a.tree_table.ids_d + (int64_t)b * a.tree_table.stride;
    for (int i = t; i < (r.n + ps - 1) / ps; i += threads) bad |= (uint32_t)ids[i] >= (uint32_t)a.cache.num_pages;
  }
  return bad;
}

}  // namespace tsv
