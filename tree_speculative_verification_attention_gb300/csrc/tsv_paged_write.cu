// tsv_paged_write.cu — new rows of a paged 8-bit cache: tsv_paged_append (rows
// of activations, K rotated on the way) and tsv_paged_commit (the accepted
// path's rows of the tree pages).
//
//   scale[page, head] = 2^ceil(log2(amax / 448)) over the page's new rows (and
//                       at least the page's scale while it keeps older rows)
//   code              = e4m3(value / scale), nearest even
//
// A scale needs every new row of its page before the first code can be
// written, so the unit of work is one (page, head): 16 rows per warp, a whole
// page in 1 to 8 warps, its values held in registers between the maximum and
// the rounding - each value is read from HBM once and each code written once,
// which is the bound.  A CTA takes one page for 128 / page_size heads at a
// time and walks `head_loop` such groups: the angles of the page's rows are
// the same for every head and are computed once per CTA.
//
// A lane owns 16 values of a row as two chunks of 8: adjacent chunks, or, for
// the half layout, a chunk and its partner rotary_dim / 2 elements on, so that
// a pair never leaves its thread.
#include <cuda_runtime.h>

#include "tsv_paged_common.cuh"

namespace tsv {

namespace {

constexpr int kWriteThreads = 32 * kPagedWriteWarps;

struct FromCodes {};  // source type of the commit kernel

// 8 consecutive values of a source row, raw.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float* f, float) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* f, float) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};
template <>
struct Chunk<FromCodes> {
  uint2 w;
  __device__ __forceinline__ void clear() { w = make_uint2(0u, 0u); }
  __device__ __forceinline__ void load(const uint8_t* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* f, float s) const {
    e4m3x4_to_f32(w.x, s, f);
    e4m3x4_to_f32(w.y, s, f + 4);
  }
};

__device__ __forceinline__ uint2 pack8(const float* f, float inv) {
  uint2 r;
  r.x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
  r.y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
  return r;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T>
__device__ __forceinline__ float scalar_f32(T v);
template <>
__device__ __forceinline__ float scalar_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float scalar_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T, int D>
__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(const PagedWriteArgs a) {
  constexpr bool kCommit = sizeof(Chunk<T>) == sizeof(uint2);
  constexpr int LPR = D / 16;        // lanes of a row
  constexpr int RPP = 32 / LPR;      // rows of a warp at a time
  constexpr int PASSES = 16 / RPP;   // for its 16 rows
  pdl_trigger();
  pdl_wait();  // the previous kernel's results are visible from here on
  extern __shared__ float angles[];  // cosines [page_size][half], then sines
  __shared__ float amax[2][kPagedWriteWarps];
  __shared__ int32_t spath[TSV_MAX_NODES];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y;
  const tsv_paged_cache& C = a.cache;
  const int ps = C.page_size;
  const int off = a.offsets[b], n_rows = a.offsets[b + 1] - off;
  const int start = a.start ? a.start[b] : 0;
  const int n = kCommit ? a.accept_len[b] + 1 : n_rows;
  // The request's lengths, then every page id (and path entry) that it needs:
  // one that is wrong rejects the whole request.
  bool bad = off < 0 || n_rows < 0 || n_rows > a.max_rows || (int64_t)off + n_rows > a.N || start < 0 ||
             (int64_t)start + n > (int64_t)a.table.pages * ps;
  if (kCommit) bad = bad || n < 1 || n > n_rows || n_rows > TSV_MAX_NODES || (int64_t)n_rows > (int64_t)a.tree_table.pages * ps;
  const int first = bad ? 0 : start / ps;
  const int last = bad || n == 0 ? first - 1 : (start + n - 1) / ps;
  const int32_t* ids = a.table.ids_d + (int64_t)b * a.table.stride;
  if (!bad) {
    for (int i = first + tid; i <= last; i += kWriteThreads) {
      const int id = ids[i];
      if (id < 0 || id >= C.num_pages) bad = true;
    }
    if constexpr (kCommit) {
      const int32_t* tids = a.tree_table.ids_d + (int64_t)b * a.tree_table.stride;
      for (int i = tid; i < n; i += kWriteThreads) {
        const int x = a.path[off + i];
        const int before = i == 0 ? -1 : a.path[off + i - 1];
        int id = -1;
        if (x > before && x < n_rows && (i > 0 || x == 0)) id = tids[x / ps];
        if (id < 0 || id >= C.num_pages) bad = true;
        spath[i] = id * ps + x % ps;  // row of the pool
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) {
    a.status[b] = bad ? TSV_ERR_INVALID_ARG : TSV_OK;
    if (kCommit && a.new_len) a.new_len[b] = bad ? -1 : start + n;
  }
  const int pi = first + blockIdx.x;
  if (bad || pi > last) return;
  const int row0 = pi * ps - start;              // new row held by the page's row 0 (negative: kept rows)
  const int kept = max(-row0, 0), end = min(ps, n - row0);  // new rows: page rows kept .. end - 1
  const int64_t page = ids[pi];

  const bool turn = !kCommit && a.inv_freq != nullptr;
  const int half = a.rot >> 1;
  const float* ct = angles;
  const float* st = angles + ps * half;
  if (turn) {
    const int per = kWriteThreads / half, f = tid % half;
    if (tid < per * half) {
      const uint64_t w = rope_turns(a.inv_freq[f]);
      for (int r = kept + tid / half; r < end; r += per) {
        float c, s;
        rope_cos_sin(a.positions[off + row0 + r], w, &c, &s);
        angles[r * half + f] = c * a.amplitude;
        angles[ps * half + r * half + f] = s * a.amplitude;
      }
    }
    __syncthreads();
  }

  const int wpp = ps >> 4;               // warps of a page
  const int team = warp / wpp, slice = warp - team * wpp;
  const int hp = kPagedWriteWarps / wpp;  // heads at a time
  const int j = lane % LPR, rl = lane / LPR;
  // The lane's chunks: adjacent ones; for K under the half layout with whole
  // chunks on both sides a rotated chunk and its partner.
  const bool pairs = turn && !a.interleaved && a.rot % 16 == 0;
  const int rc = a.rot >> 4;  // chunk pairs of the rotated part
  const int v0 = 16 * j, v1 = v0 + 8;
  const int k0 = !pairs ? v0 : j < rc ? 8 * j : v0;
  const int k1 = !pairs ? v1 : j < rc ? 8 * j + half : v1;

  for (int it = 0; it < a.head_loop; ++it) {
    const int g0 = (blockIdx.z * a.head_loop + it) * hp;
    if (g0 >= C.Hkv) break;  // the same in every thread
    const int g = g0 + team;
    const bool on = g < C.Hkv;
    uint8_t* kp = static_cast<uint8_t*>(C.k_d) + page * C.stride_page + (int64_t)g * C.stride_head;
    uint8_t* vp = static_cast<uint8_t*>(C.v_d) + page * C.stride_page + (int64_t)g * C.stride_head;
    float* ksp = C.k_scale_d + page * C.Hkv + g;
    float* vsp = C.v_scale_d + page * C.Hkv + g;
    Chunk<T> kc[PASSES][2], vc[PASSES][2];
    float kf[PASSES], vf[PASSES];  // source scales (commit)
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = slice * 16 + p * RPP + rl;
      kf[p] = vf[p] = 1.f;
      if (on && r >= kept && r < end) {
        const int i = row0 + r;
        if constexpr (kCommit) {
          const int src = spath[i];
          const int64_t sp = src / ps;
          const int64_t o = sp * C.stride_page + (int64_t)(src - (int)sp * ps) * C.stride_row + (int64_t)g * C.stride_head;
          const uint8_t* ks = static_cast<const uint8_t*>(C.k_d) + o;
          const uint8_t* vs = static_cast<const uint8_t*>(C.v_d) + o;
          kc[p][0].load(ks + k0);
          kc[p][1].load(ks + k1);
          vc[p][0].load(vs + v0);
          vc[p][1].load(vs + v1);
          kf[p] = C.k_scale_d[sp * C.Hkv + g];
          vf[p] = C.v_scale_d[sp * C.Hkv + g];
        } else {
          const T* ks = static_cast<const T*>(a.k) + (int64_t)(off + i) * a.ks_n + (int64_t)g * a.ks_h;
          const T* vs = static_cast<const T*>(a.v) + (int64_t)(off + i) * a.vs_n + (int64_t)g * a.vs_h;
          kc[p][0].load(ks + k0);
          kc[p][1].load(ks + k1);
          vc[p][0].load(vs + v0);
          vc[p][1].load(vs + v1);
        }
      } else {
        kc[p][0].clear();
        kc[p][1].clear();
        vc[p][0].clear();
        vc[p][1].clear();
      }
    }
    const float k_old = on && kept > 0 ? *ksp : 0.f, v_old = on && kept > 0 ? *vsp : 0.f;

    float kx[PASSES][16];
    float km = 0.f, vm = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = slice * 16 + p * RPP + rl;
      kc[p][0].get(kx[p], kf[p]);
      kc[p][1].get(kx[p] + 8, kf[p]);
      if (turn && on && r >= kept && r < end) {
        const float* c = ct + r * half;
        const float* s = st + r * half;
        if (pairs) {
          if (j < rc) {
#pragma unroll
            for (int e = 0; e < 8; ++e) rope_pair(kx[p][e], kx[p][8 + e], c[k0 + e], s[k0 + e]);
          }
        } else if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            if (k0 + e < a.rot) rope_pair(kx[p][e], kx[p][e + 1], c[(k0 + e) >> 1], s[(k0 + e) >> 1]);
        } else if constexpr (!kCommit) {
          // Half layout that cuts a chunk: the partner is read again.
          const T* ks = static_cast<const T*>(a.k) + (int64_t)(off + row0 + r) * a.ks_n + (int64_t)g * a.ks_h;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int d = k0 + e;
            if (d < a.rot) {
              const bool low = d < half;
              const float q = scalar_f32<T>(ks[low ? d + half : d - half]);
              const int f = low ? d : d - half;
              float x = kx[p][e], y = q;
              if (low) {
                rope_pair(x, y, c[f], s[f]);
                kx[p][e] = x;
              } else {
                rope_pair(y, x, c[f], s[f]);
                kx[p][e] = x;
              }
            }
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) km = fmaxf(km, finite_abs(kx[p][e]));
      float vx[16];
      vc[p][0].get(vx, vf[p]);
      vc[p][1].get(vx + 8, vf[p]);
#pragma unroll
      for (int e = 0; e < 16; ++e) vm = fmaxf(vm, finite_abs(vx[e]));
    }
    km = warp_max(km);
    vm = warp_max(vm);
    if (it > 0) __syncthreads();  // the previous group's maxima have been read
    if (lane == 0) {
      amax[0][warp] = km;
      amax[1][warp] = vm;
    }
    __syncthreads();  // also: every thread has read the old scales
    if (!on) continue;
    km = vm = 0.f;
    for (int w = 0; w < wpp; ++w) {
      km = fmaxf(km, amax[0][team * wpp + w]);
      vm = fmaxf(vm, amax[1][team * wpp + w]);
    }
    const float k_scale = fmaxf(k_old, pow2_scale(km)), v_scale = fmaxf(v_old, pow2_scale(vm));
    const float k_inv = 1.f / k_scale, v_inv = 1.f / v_scale;
    if (slice == 0 && lane == 0) {
      *ksp = k_scale;
      *vsp = v_scale;
    }
    const float k_again = k_old * k_inv, v_again = v_old * v_inv;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = slice * 16 + p * RPP + rl;
      uint8_t* kr = kp + (int64_t)r * C.stride_row;
      uint8_t* vr = vp + (int64_t)r * C.stride_row;
      if (r >= kept && r < end) {
        float vx[16];
        vc[p][0].get(vx, vf[p]);
        vc[p][1].get(vx + 8, vf[p]);
        const uint2 va = pack8(vx, v_inv), vb = pack8(vx + 8, v_inv);
        *reinterpret_cast<uint2*>(kr + k0) = pack8(kx[p], k_inv);
        *reinterpret_cast<uint2*>(kr + k1) = pack8(kx[p] + 8, k_inv);
        *reinterpret_cast<uint4*>(vr + v0) = make_uint4(va.x, va.y, vb.x, vb.y);
      } else if (r < kept) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const bool grows = side == 0 ? k_scale > k_old : v_scale > v_old;
          if (!grows) continue;
          uint4* at = reinterpret_cast<uint4*>((side == 0 ? kr : vr) + v0);
          const uint4 w = *at;
          const float m = side == 0 ? k_again : v_again;
          float f[16];
          e4m3x4_to_f32(w.x, m, f);
          e4m3x4_to_f32(w.y, m, f + 4);
          e4m3x4_to_f32(w.z, m, f + 8);
          e4m3x4_to_f32(w.w, m, f + 12);
          const uint2 lo = pack8(f, 1.f), hi = pack8(f + 8, 1.f);
          *at = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  }
}

// Pages that one request's new rows can touch.
int32_t most_pages(const PagedWriteArgs& a) {
  const int64_t ps = a.cache.page_size;
  return (int32_t)((a.max_rows + (a.start ? ps - 1 : 0) + ps - 1) / ps);
}

template <typename T, int D>
cudaError_t launch_typed(const PagedWriteArgs& a, size_t smem, cudaStream_t st) {
  const int hp = kPagedWriteWarps / (a.cache.page_size / 16);
  const int groups = (a.cache.Hkv + hp - 1) / hp;
  const dim3 grid(max(1, most_pages(a)), a.B, (groups + a.head_loop - 1) / a.head_loop);
  return launch_pdl(paged_write_kernel<T, D>, grid, dim3(kWriteThreads), smem, st, 0u, a);
}

}  // namespace

size_t paged_append_smem_bytes(int32_t page_size, int32_t rot) { return (size_t)page_size * rot * sizeof(float); }

cudaError_t paged_append_set_attributes(bool bf16, int32_t D) {
  const int most = (int)paged_append_smem_bytes(128, D);
  const cudaFuncAttribute what = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (bf16)
    return D == 64 ? cudaFuncSetAttribute(paged_write_kernel<__nv_bfloat16, 64>, what, most)
                   : cudaFuncSetAttribute(paged_write_kernel<__nv_bfloat16, 128>, what, most);
  return D == 64 ? cudaFuncSetAttribute(paged_write_kernel<float, 64>, what, most)
                 : cudaFuncSetAttribute(paged_write_kernel<float, 128>, what, most);
}

cudaError_t launch_paged_append(const PagedWriteArgs& a, bool bf16, cudaStream_t st) {
  const size_t smem = a.inv_freq ? paged_append_smem_bytes(a.cache.page_size, a.rot) : 0;
  if (bf16)
    return a.cache.D == 64 ? launch_typed<__nv_bfloat16, 64>(a, smem, st) : launch_typed<__nv_bfloat16, 128>(a, smem, st);
  return a.cache.D == 64 ? launch_typed<float, 64>(a, smem, st) : launch_typed<float, 128>(a, smem, st);
}

cudaError_t launch_paged_commit(const PagedWriteArgs& a, cudaStream_t st) {
  return a.cache.D == 64 ? launch_typed<FromCodes, 64>(a, 0, st) : launch_typed<FromCodes, 128>(a, 0, st);
}

}  // namespace tsv
