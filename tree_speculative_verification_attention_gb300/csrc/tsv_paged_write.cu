// tsv_paged_write.cu — new rows of a paged 8-bit cache: tsv_paged_append (rows
// of activations, K rotated on the way) and tsv_paged_commit (the accepted
// path's rows of the tree pages).
//
//   scale[page, head] = 2^ceil(log2(amax / 448)) over the page's new rows (and
//                       at least the page's scale while it keeps older rows)
//   code              = e4m3(value / scale), nearest even
//
// A scale needs every new row of its page before the first code can be
// written, so the unit of work is one (page, head): 512 values per
// warp (4 or 8 rows), a whole page in 2 to 32 warps, its values held in registers between the maximum and
// the rounding - each value is read from HBM once and each code written once,
// which is the bound.  A CTA takes one page for `hp` heads at a time and walks
// `head_loop` such groups: the angles of the page's rows are the same for every
// head and are computed once per CTA, while its first rows are on their way.
// One row part a lane rather than two or four: 64 registers hold it, so 32
// warps share an SM and one's loads run under another's rounding (18,200 rows of
// 8 requests, 8 heads of 128, bf16, rotated: 33 us, 3.4 TB/s; 16 values of four
// rows a lane: 88 us).  Nothing is saturated there (issue 57 %, DRAM 29 % of their
// peaks): a lane's 32 values take about 250 instructions and the angles, behind two
// barriers a head, and 64 registers, all that the 1024 threads of a 128-row page
// leave, spill 88 to 184 bytes.  Few rows cost a chain
// of loads (lengths, pages, rows, scales): 20 rows x 32 heads 4.4 us, a commit of
// their path 3.9 us, of 128 requests' paths 10 us.
//
// A lane owns 16 values of a row as two chunks of 8: adjacent chunks, or, for
// the half layout, a chunk and its partner rotary_dim / 2 elements on, so that
// a pair never leaves its thread.
#include <cuda_runtime.h>

#include <type_traits>

#include "tsv_paged_common.cuh"

namespace tsv {

namespace {

struct FromCodes {};  // source type of the commit kernel

// 8 consecutive values of a source row, raw.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
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
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
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

// Of values >= 0: their bits order them.
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// The largest finite |x|.  A maximum leaves NaN out by itself; only an infinity
// needs the second look.
__device__ __forceinline__ float finite_amax(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
  if (m == INFINITY) {
    m = 0.f;
    for (int e = 0; e < 16; ++e) m = fmaxf(m, finite_abs(x[e]));
  }
  return m;
}

// The largest finite |value| of two chunks; of bf16 in pairs, as they are.
template <typename T>
__device__ __forceinline__ float source_amax(const Chunk<T> (&c)[2], float s) {
  float x[16];
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const uint32_t w[8] = {c[0].w.x, c[0].w.y, c[0].w.z, c[0].w.w, c[1].w.x, c[1].w.y, c[1].w.z, c[1].w.w};
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7FFF7FFFu));
    const float best = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    if (best < INFINITY) return best;
  }
  c[0].get(x, s);
  c[1].get(x + 8, s);
  return finite_amax(x);
}

// The table of angles: rows of `width` floats, their 16-byte blocks 2i and
// 2i + 1 swapped in the upper half of every 64 floats, so that eight lanes that
// read the first (or second) blocks of eight neighbouring pairs meet 32
// different banks.
__host__ __device__ constexpr int angle_width(int half) { return (half + 7) & ~7; }
__device__ __forceinline__ int angle_at(int f) { return f ^ ((f >> 3) & 4); }

template <typename T>
__device__ __forceinline__ float scalar_f32(T v);
template <>
__device__ __forceinline__ float scalar_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float scalar_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T, int D>
__global__ void __launch_bounds__(32 * kPagedWriteMaxWarps) paged_write_kernel(const PagedWriteArgs a) {
  constexpr bool kCommit = sizeof(Chunk<T>) == sizeof(uint2);
  using S = std::conditional_t<kCommit, uint8_t, T>;  // element of a source row
  constexpr int LPR = D / 16;                      // lanes of a row
  constexpr int ROWS = paged_write_rows(D);        // rows of a warp
  static_assert(LPR * ROWS == 32, "a lane holds a part of one row");
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  extern __shared__ float4 angle_table[];  // cosines [page_size][width], then sines
  __shared__ float amax[2][2][kPagedWriteMaxWarps];
  __shared__ int32_t spath[kCommit ? TSV_MAX_NODES : 1];

  const int tid = threadIdx.x, threads = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y;
  const tsv_paged_cache& C = a.cache;
  const int ps = C.page_size;
  const int off = a.offsets[b], n_rows = a.offsets[b + 1] - off;
  const int start = a.start ? a.start[b] : 0;
  const int n = kCommit ? min(a.accept_len[b], TSV_MAX_NODES) + 1 : n_rows;  // (accept_len may be anything)
  // The request's lengths, then every page id (and path entry) that it needs:
  // one that is wrong rejects the whole request.
  bool bad = off < 0 || n_rows < 0 || n_rows > a.max_rows || (int64_t)off + n_rows > a.N || start < 0 ||
             (int64_t)start + n > (int64_t)a.table.pages * ps;
  if (kCommit) bad = bad || n < 1 || n > n_rows || n_rows > TSV_MAX_NODES || (int64_t)n_rows > (int64_t)a.tree_table.pages * ps;
  const int first = bad ? 0 : start / ps;
  const int last = bad || n == 0 ? first - 1 : (start + n - 1) / ps;
  const int32_t* ids = a.table.ids_d + (int64_t)b * a.table.stride;
  const bool reports = blockIdx.x == 0 && blockIdx.z == 0;
  if (!reports && (int)blockIdx.x > last - first) return;  // no page (or a bad request)
  if (!bad) {
    for (int i = first + tid; i <= last; i += threads) {
      const int id = ids[i];
      if (id < 0 || id >= C.num_pages) bad = true;
    }
    if constexpr (kCommit) {
      const int32_t* tids = a.tree_table.ids_d + (int64_t)b * a.tree_table.stride;
      for (int i = tid; i < n; i += threads) {
        const int x = a.path[off + i];
        const int before = i == 0 ? -1 : a.path[off + i - 1];
        int id = -1;
        if (x > before && x < n_rows && (i > 0 || x == 0)) id = tids[x / ps];
        if (id < 0 || id >= C.num_pages) bad = true;
        spath[i] = id * ps + x % ps;  // row of the pool
      }
    }
  }

  const bool turn = !kCommit && a.inv_freq != nullptr;
  const int half = a.rot >> 1;
  float* ct = reinterpret_cast<float*>(angle_table);
  const int width = angle_width(half);
  float* st = ct + ps * width;
  const int wpp = ps / ROWS;  // warps of a page
  const int team = warp / wpp, slice = warp - team * wpp;
  const int hp = (threads >> 5) / wpp;  // heads at a time
  const int j = lane % LPR, r = slice * ROWS + lane / LPR;  // its lane's row of the page
  // The lane's chunks: adjacent ones; for K under the half layout with whole
  // chunks on both sides a rotated chunk and its partner.
  const bool pairs = turn && !a.interleaved && a.rot % 16 == 0;
  const int rc = a.rot >> 4;  // chunk pairs of the rotated part
  const int v0 = 16 * j, v1 = v0 + 8;
  const int k0 = !pairs ? v0 : j < rc ? 8 * j : v0;
  const int k1 = !pairs ? v1 : j < rc ? 8 * j + half : v1;

  Chunk<T> kc[2], vc[2];
  float kf, vf;  // source scales (commit)
  int parity = 0;
  for (int round = 0;; ++round) {
    const int pi = first + blockIdx.x + round * gridDim.x;
    const bool work = pi <= last;                      // the same in every thread
    const int row0 = pi * ps - start;                  // new row held by the page's row 0 (negative: kept rows)
    const int kept = max(-row0, 0), end = min(ps, n - row0);  // new rows: page rows kept .. end - 1
    const bool row_on = work && r >= kept && r < end;  // the lane's row is a new one
    const int g0 = blockIdx.z * a.head_loop * hp, gn = min(C.Hkv, g0 + a.head_loop * hp);
    // The lane's part of the row at head g0 + team, then hp heads on at each load.
    const S *ks = nullptr, *vs = nullptr;
    int64_t sp = 0;  // page of the source (commit)
    int gk = g0 + team, gv = gk;
    auto source = [&]() {
      if constexpr (kCommit) {
        const int src = row_on ? spath[row0 + r] : 0;
        sp = src / ps;
        const int64_t at = sp * C.stride_page + (int64_t)(src - (int)sp * ps) * C.stride_row + (int64_t)gk * C.stride_head;
        ks = static_cast<const uint8_t*>(C.k_d) + at + k0;
        vs = static_cast<const uint8_t*>(C.v_d) + at + v0;
      } else {
        ks = static_cast<const T*>(a.k) + (int64_t)(off + row0 + r) * a.ks_n + (int64_t)gk * a.ks_h + k0;
        vs = static_cast<const T*>(a.v) + (int64_t)(off + row0 + r) * a.vs_n + (int64_t)gv * a.vs_h + v0;
      }
    };
    auto load_k = [&]() {
      if (row_on && gk < gn) {
        kc[0].load(ks);
        kc[1].load(ks + (k1 - k0));
        if (kCommit) kf = C.k_scale_d[sp * C.Hkv + gk];
      }
      gk += hp;
      ks += hp * (kCommit ? C.stride_head : a.ks_h);
    };
    auto load_v = [&]() {
      if (row_on && gv < gn) {
        vc[0].load(vs);
        vc[1].load(vs + 8);
        if (kCommit) vf = C.v_scale_d[sp * C.Hkv + gv];
      }
      gv += hp;
      vs += hp * (kCommit ? C.stride_head : a.vs_h);
    };
    kf = vf = 1.f;
    kc[0].clear();
    kc[1].clear();
    vc[0].clear();
    vc[1].clear();
    if (round > 0) __syncthreads();  // the previous page's angles have been read
    if (!kCommit) {  // (a commit's rows come from pages that are checked first)
      source();
      load_k();
      load_v();
    }
    if (work && turn) {
      const int per = threads / half, f = tid % half;
      if (tid < per * half) {
        const uint64_t w = rope_turns(a.inv_freq[f]);
        for (int r = kept + tid / half; r < end; r += per) {
          float c, s;
          rope_cos_sin(a.positions[off + row0 + r], w, &c, &s);
          const int at = r * width + angle_at(f);
          ct[at] = c * a.amplitude;
          st[at] = s * a.amplitude;
        }
      }
    }
    if (round == 0) {
      bad = __syncthreads_or(bad);
      if (reports && tid == 0) {
        a.status[b] = bad ? TSV_ERR_INVALID_ARG : TSV_OK;
        if (kCommit && a.new_len) a.new_len[b] = bad ? -1 : start + n;
      }
      if (bad) return;
    } else {
      __syncthreads();
    }
    if (!work) return;
    if (kCommit) {
      source();
      load_k();
      load_v();
    }
    const int64_t page = ids[pi];
    const int64_t to = page * C.stride_page + (int64_t)r * C.stride_row + (int64_t)(g0 + team) * C.stride_head;
    uint8_t* kr = static_cast<uint8_t*>(C.k_d) + to;
    uint8_t* vr = static_cast<uint8_t*>(C.v_d) + to;

    for (int h0 = g0; h0 < gn; h0 += hp) {  // the same in every thread
      const int g = h0 + team;
      const bool on = g < gn;
      float* ksp = C.k_scale_d + page * C.Hkv + g;
      float* vsp = C.v_scale_d + page * C.Hkv + g;
      const float k_old = on && kept > 0 ? *ksp : 0.f, v_old = on && kept > 0 ? *vsp : 0.f;

      float kx[16];
      float km = 0.f, vm = 0.f;
      kc[0].get(kx, kf);
      kc[1].get(kx + 8, kf);
      load_k();  // the next head's K goes while this one is turned and rounded
      if (turn && on && row_on) {
        const float* c = ct + r * width;
        const float* s = st + r * width;
        if (pairs || a.interleaved) {
          // The lane's pairs have the angles 8 j .. 8 j + 7.
          if (pairs ? j < rc : v0 < a.rot) {
            float cs[8], sn[8];
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              *reinterpret_cast<float4*>(cs + e) = *reinterpret_cast<const float4*>(c + angle_at(8 * j + e));
              *reinterpret_cast<float4*>(sn + e) = *reinterpret_cast<const float4*>(s + angle_at(8 * j + e));
            }
            if (pairs) {
#pragma unroll
              for (int e = 0; e < 8; ++e) rope_pair(kx[e], kx[8 + e], cs[e], sn[e]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (v0 + 2 * e < a.rot) rope_pair(kx[2 * e], kx[2 * e + 1], cs[e], sn[e]);
            }
          }
        } else if constexpr (!kCommit) {
          // Half layout that cuts a chunk: the partner is read again.
          const T* row = static_cast<const T*>(a.k) + (int64_t)(off + row0 + r) * a.ks_n + (int64_t)g * a.ks_h;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int d = k0 + e;
            if (d < a.rot) {
              const bool low = d < half;
              const float q = scalar_f32<T>(row[low ? d + half : d - half]);
              const int f = angle_at(low ? d : d - half);
              float x = kx[e], y = q;
              if (low) {
                rope_pair(x, y, c[f], s[f]);
                kx[e] = x;
              } else {
                rope_pair(y, x, c[f], s[f]);
                kx[e] = x;
              }
            }
          }
        }
      }
      km = warp_max(finite_amax(kx));
      vm = warp_max(source_amax(vc, vf));
      // Two sets of maxima in turn: a set is written again behind the next one's barrier.
      float(*most)[kPagedWriteMaxWarps] = amax[parity];
      parity ^= 1;
      if (lane == 0) {
        most[0][warp] = km;
        most[1][warp] = vm;
      }
      __syncthreads();  // also: every thread has read the old scales
      if (!on) continue;  // (no later group of this team is on either)
      km = warp_max(lane < wpp ? most[0][team * wpp + lane] : 0.f);
      vm = warp_max(lane < wpp ? most[1][team * wpp + lane] : 0.f);
      const float k_scale = fmaxf(k_old, pow2_scale(km)), v_scale = fmaxf(v_old, pow2_scale(vm));
      // (A kept scale is the caller's, the others are powers of two.)
      const float k_inv = kept > 0 ? 1.f / k_scale : pow2_inverse(k_scale);
      const float v_inv = kept > 0 ? 1.f / v_scale : pow2_inverse(v_scale);
      if (slice == 0 && lane == 0) {
        *ksp = k_scale;
        *vsp = v_scale;
      }
      const float k_again = k_old * k_inv, v_again = v_old * v_inv;
      if (row_on) {
        float vx[16];
        vc[0].get(vx, vf);
        vc[1].get(vx + 8, vf);
        const uint2 va = pack8(vx, v_inv), vb = pack8(vx + 8, v_inv);
        load_v();
        *reinterpret_cast<uint2*>(kr + k0) = pack8(kx, k_inv);
        *reinterpret_cast<uint2*>(kr + k1) = pack8(kx + 8, k_inv);
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
      kr += hp * C.stride_head;
      vr += hp * C.stride_head;
    }
  }
}

// Pages that one request's new rows can touch.
int32_t most_pages(const PagedWriteArgs& a) {
  const int64_t ps = a.cache.page_size;
  return (int32_t)((a.max_rows + (a.start ? ps - 1 : 0) + ps - 1) / ps);
}

template <typename T, int D>
cudaError_t launch_typed(const PagedWriteArgs& a, size_t smem, int num_sms, cudaStream_t st) {
  const int warps = paged_write_warps(a.cache.page_size, D);
  const int hp = paged_write_heads(a.cache.page_size, D);
  const int groups = (a.cache.Hkv + hp - 1) / hp, gz = (groups + a.head_loop - 1) / a.head_loop;
  // CTAs for every page that a request could touch, up to 8 per SM: lengths are
  // read on the device, most requests touch far fewer pages (a commit one or
  // two), and the rest of a long one is walked.
  const int most = (int)max((int64_t)1, 8 * num_sms / ((int64_t)a.B * gz));
  const dim3 grid(min(max(1, most_pages(a)), most), a.B, gz);
  return launch_pdl(paged_write_kernel<T, D>, grid, dim3(32 * warps), smem, st, 0u, a);
}

}  // namespace

size_t paged_append_smem_bytes(int32_t page_size, int32_t rot) {
  return (size_t)page_size * 2 * angle_width(rot / 2) * sizeof(float);
}

cudaError_t paged_append_set_attributes(bool bf16, int32_t D) {
  const int most = (int)paged_append_smem_bytes(128, D);
  const cudaFuncAttribute what = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (bf16)
    return D == 64 ? cudaFuncSetAttribute(paged_write_kernel<__nv_bfloat16, 64>, what, most)
                   : cudaFuncSetAttribute(paged_write_kernel<__nv_bfloat16, 128>, what, most);
  return D == 64 ? cudaFuncSetAttribute(paged_write_kernel<float, 64>, what, most)
                 : cudaFuncSetAttribute(paged_write_kernel<float, 128>, what, most);
}

cudaError_t launch_paged_append(const PagedWriteArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  const size_t smem = a.inv_freq ? paged_append_smem_bytes(a.cache.page_size, a.rot) : 0;
  if (bf16)
    return a.cache.D == 64 ? launch_typed<__nv_bfloat16, 64>(a, smem, num_sms, st) : launch_typed<__nv_bfloat16, 128>(a, smem, num_sms, st);
  return a.cache.D == 64 ? launch_typed<float, 64>(a, smem, num_sms, st) : launch_typed<float, 128>(a, smem, num_sms, st);
}

cudaError_t launch_paged_commit(const PagedWriteArgs& a, int num_sms, cudaStream_t st) {
  return a.cache.D == 64 ? launch_typed<FromCodes, 64>(a, 0, num_sms, st) : launch_typed<FromCodes, 128>(a, 0, num_sms, st);
}

}  // namespace tsv
