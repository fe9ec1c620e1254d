// tsv_paged_tc.cuh — what the two tensor-core kernels of the paged tree
// attention share: the list of blocks and its cut into CTAs, bounded waits, the
// join of partial results, and small wrappers.
#pragma once

#include "tsv_attention_common.cuh"

#include "tsv_paged_common.cuh"

namespace tsv {

constexpr int kPBlock = 128;  // keys of a block

// A descriptor with another low word (its address field; no carry out of it).
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t low) {
  return (base & 0xFFFFFFFF00000000ull) | low;
}
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// tma_load_4d of one KV head's rows of a page, issued by the lane with `lead`
// set (the whole warp calls it, so the operands stay uniform).
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* tmap, uint32_t bar, uint32_t head, uint32_t page,
                                              uint64_t policy, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %7, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %2, %4}], [%5], %6;\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(head), "r"(page), "r"(bar), "l"(policy), "r"((uint32_t)lead)
      : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// One unit of a CTA's range: blocks j .. j1 - 1 of a (request, KV head, row
// tile) group of T blocks, nmain of them over prefix rows.  gx is the place of
// the group in the list of all blocks: it begins with a few places that hold no
// block and stand for what a unit costs beside its blocks, so that a CTA with a
// group's end and another's beginning gets as many blocks fewer.
struct alignas(16) PUnit {
  int b, g, tile, tiles, off, n, P, nmain, T, j, j1, valid;
  int64_t gx;
  __device__ __forceinline__ bool whole() const { return j == 0 && j1 == T; }
};

struct PPad {
  int blocks, least;  // of groups of `least` blocks at least
  __device__ __forceinline__ int of(int T) const { return T >= least ? blocks : 0; }
};

struct PList {
  const int64_t* cum;
  const int4* req;
  int B, G, Hkv, R;
  PPad pad;
  bool tree;
  int64_t x1;  // end of this CTA's range

  __device__ __forceinline__ void request(PUnit& u) const {
    const int4 q = req[u.b];
    u.off = q.x;
    u.n = q.y;
    u.P = q.z;
    u.T = q.w;
    u.nmain = (u.P + kPBlock - 1) / kPBlock;
    u.tiles = (u.n * G + R - 1) / R;
  }
  // The unit at x0 < x1 (called by a whole warp).
  __device__ __forceinline__ PUnit first(int64_t x0) const {
    PUnit u{};
    u.valid = x0 < x1;
    if (!u.valid) return u;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < TSV_MAX_BATCH / 32; ++q) u.b += __popc(__ballot_sync(0xffffffffu, cum[32 * q + lane + 1] <= x0));
    request(u);
    const int64_t rel = x0 - cum[u.b];
    const int none = pad.of(u.T), len = u.T + none;
    const int group = rel <= 0xFFFFFFFFll ? (int)((uint32_t)rel / (uint32_t)len) : (int)(rel / len);
    const int at = (int)(rel - (int64_t)group * len);
    u.j = max(0, at - none);
    u.g = group / u.tiles;
    u.tile = group - u.g * u.tiles;
    u.gx = x0 - at;
    u.j1 = (int)min((int64_t)u.T, x1 - u.gx - none);
    u.valid = u.j < u.j1;  // (else the range ends before the group's first block)
    return u;
  }
  __device__ __forceinline__ void next(PUnit& u) const {
    u.gx += u.T + pad.of(u.T);
    u.valid = u.gx < x1;
    if (!u.valid) return;
    if (++u.tile == u.tiles) {
      u.tile = 0;
      if (++u.g == Hkv) {
        u.g = 0;
        do ++u.b;
        while (cum[u.b + 1] == cum[u.b]);
        request(u);
      }
    }
    u.j = 0;
    u.j1 = (int)min((int64_t)u.T, x1 - u.gx - pad.of(u.T));
    u.valid = u.j1 > 0;
  }
};

// A wait that ran out (or saw another role's) leaves the warp `dead`: it goes
// through the motions without waiting, so that named barriers stay complete.
// The hardware holds a waiting thread for up to 4 us a try (with the hint;
// measured), so that waiting warps do not take the working ones' issue slots;
// 2^18 tries are about a second.  Short on purpose: an SM sub-partition keeps
// about 2000 instructions at hand, and the roles' loops have to share them.
constexpr uint32_t kWaitTries = 1u << 18;
__device__ __forceinline__ bool mbar_try_long(uint32_t at, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 100000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(at), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void pwait(uint64_t* bar, uint32_t parity, volatile int* abort, bool& dead) {
  const uint32_t at = smem_u32(bar);
#pragma unroll 1
  for (uint32_t n = 0; !mbar_try_long(at, parity & 1u); ++n)
    if (dead || *abort || n == kWaitTries) {
      *abort = 1;
      dead = true;
      break;
    }
  __syncwarp();
}
// Arrives for the whole warp, or, once it is dead, not at all: arrivals of a
// warp are added up, and a phase with fewer of them left than a later warp
// brings would be a fault.
__device__ __forceinline__ void parrive(uint64_t* bar, bool dead) {
  if (!__any_sync(0xffffffffu, dead)) mbar_arrive(bar);
}
#define TSV_PWAIT(bar, parity) pwait((bar), (uint32_t)(parity), abort_v, dead)

// The list of blocks: request b holds T_b x Hkv x tiles of them.  A request
// with nothing to see still gets one (empty) block, which writes its zeros.
// One warp works it out, and the CTA's range (sRange: its blocks, its end, all
// places, CTAs) and first unit.
__device__ __forceinline__ void plist_setup(const PagedAttnArgs& a, int R, PPad pad, int64_t* sCum, int4* sReq, PUnit* sFirst,
                                            int64_t* sRange) {
  const int lane = threadIdx.x & 31;
  const bool tree = a.tree_table.ids_d != nullptr;
  int64_t before = 0;
  if (lane == 0) sCum[0] = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < TSV_MAX_BATCH; b0 += 32) {
    const int b = b0 + lane;
    int64_t upto = 0;
    if (b0 < a.B) {
      PagedRequest r;
      if (b < a.B && paged_request(a, b, &r) && r.n > 0) {
        const int T = max(1, (r.P + kPBlock - 1) / kPBlock + (tree ? (r.n + kPBlock - 1) / kPBlock : 0));
        upto = (int64_t)(T + pad.of(T)) * a.cache.Hkv * ((r.n * a.G + R - 1) / R);
        sReq[b] = make_int4(r.off, r.n, r.P, T);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
    }
    sCum[b + 1] = before + upto;
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  __syncwarp();
  const int64_t W = before, ctas = min((int64_t)gridDim.x, W);
  int64_t x0 = W, x1 = W;
  if ((int)blockIdx.x < ctas) {
    if (W < (1 << 22)) {  // 32-bit products and quotients (at most 1024 CTAs)
      x0 = (uint32_t)blockIdx.x * (uint32_t)W / (uint32_t)ctas;
      x1 = ((uint32_t)blockIdx.x + 1u) * (uint32_t)W / (uint32_t)ctas;
    } else {
      x0 = (int64_t)blockIdx.x * W / ctas;
      x1 = ((int64_t)blockIdx.x + 1) * W / ctas;
    }
  }
  const PList mine{sCum, sReq, a.B, a.G, a.cache.Hkv, R, pad, tree, x1};
  const PUnit u = mine.first(x0);
  int64_t blocks = x1 - x0;
  if (pad.blocks > 0) {
    blocks = 0;
    for (PUnit w = u; w.valid; mine.next(w)) blocks += w.j1 - w.j;
  }
  if (lane == 0) {
    *sFirst = u;
    sRange[0] = blocks;
    sRange[1] = x1;
    sRange[2] = W;
    sRange[3] = ctas;
  }
}

// Status of a request.  One CTA checks it, others may give up a wait for it, in any
// order: a word of the workspace makes the timeout win.  Each side writes its own
// word, then looks at (or overwrites) the other's, with a fence between: whichever
// fence comes first, the last store to the status is the timeout's.
__device__ __forceinline__ void report_timeout(const PagedAttnArgs& a, int32_t* timeouts, int b) {
  *static_cast<volatile int32_t*>(timeouts + b) = 1;
  __threadfence();
  *static_cast<volatile int32_t*>(a.status + b) = TSV_ERR_TIMEOUT;
}
__device__ __forceinline__ void report_check(const PagedAttnArgs& a, const int32_t* timeouts, int b, bool bad) {
  *static_cast<volatile int32_t*>(a.status + b) = bad ? TSV_ERR_INVALID_ARG : TSV_OK;
  __threadfence();
  if (*static_cast<const volatile int32_t*>(timeouts + b)) *static_cast<volatile int32_t*>(a.status + b) = TSV_ERR_TIMEOUT;
}

// Joins the partials of CTAs cf .. cl of a group (slots of R rows: part_ml holds
// maxima, then sums; part_o unscaled rows) into `rows` output rows.
template <int D, int R>
__device__ __forceinline__ void join_partials(const float* part_o, const float* part_ml, int cf, int cl, int first_slot, int rows,
                                              const int32_t* row_of, __nv_bfloat16* out, int warp, int warps, int lane) {
  // A warp takes 2 rows at a time, a lane 16 bytes of each; the CTAs'
  // partials are brought to a running maximum in order, five in flight.
  constexpr int RB = 2, CB = 5, L4 = D / 4;  // lanes of a row: D / 4
  const int lane_row = lane / L4, d4 = (lane % L4) * 4;
  constexpr int kRowsPerWarp = 32 / L4;
  for (int r0 = warp * RB * kRowsPerWarp; r0 < rows; r0 += warps * RB * kRowsPerWarp) {
    float top[RB], sum[RB];
    float4 o[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      top[i] = -INFINITY;
      sum[i] = 0.f;
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int c0 = cf; c0 <= cl; c0 += CB) {
      float m[CB][RB], l[CB][RB];
      float4 v[CB][RB];
#pragma unroll
      for (int x = 0; x < CB; ++x) {
        const int c = c0 + x;
        const int64_t s = 2 * c + (c == cf ? first_slot : 0);
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const int r = r0 + i * kRowsPerWarp + lane_row;
          m[x][i] = -INFINITY;
          l[x][i] = 0.f;
          v[x][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c <= cl && r < rows) {
            m[x][i] = __ldcg(part_ml + s * 2 * R + r);
            l[x][i] = __ldcg(part_ml + s * 2 * R + R + r);
            v[x][i] = __ldcg(reinterpret_cast<const float4*>(part_o + (s * R + r) * D + d4));
          }
        }
      }
#pragma unroll
      for (int x = 0; x < CB; ++x)
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const float t2 = fmaxf(top[i], m[x][i]);
          const float f = top[i] == -INFINITY ? 1.f : fast_exp2(top[i] - t2);  // nothing yet: all zero (or NaN)
          const float w = m[x][i] == -INFINITY ? 1.f : fast_exp2(m[x][i] - t2);
          top[i] = t2;
          sum[i] = sum[i] * f + l[x][i] * w;
          o[i].x = o[i].x * f + v[x][i].x * w;
          o[i].y = o[i].y * f + v[x][i].y * w;
          o[i].z = o[i].z * f + v[x][i].z * w;
          o[i].w = o[i].w * f + v[x][i].w * w;
        }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = r0 + i * kRowsPerWarp + lane_row;
      if (r >= rows) continue;
      const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];
      *reinterpret_cast<uint2*>(out + (int64_t)row_of[r] * D + d4) =
          make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv), pack_bf16x2(o[i].z * inv, o[i].w * inv));
    }
  }
}

}  // namespace tsv
