// tsv_paged_attention_wide.cu — tree attention over a paged 8-bit cache for many
// query rows per KV head, query rows on the TMEM lanes.
//
//   S = Q K^T         M = 128 rows, N = 64 keys, K = D       (A = Q, B = K, shared memory)
//   O += P V          M = 128 rows, N = D, K = 64 keys       (A = P, TMEM; B = V, shared memory)
//
// Both products are fp16 with fp32 sums.  An e4m3 code is an fp16 value, so K
// and V are widened without a rounding (one conversion per two codes); a row of
// Q is a bf16 row times a power of two that moves its largest value to
// [2^14, 2^15): exact down to 2^-31 of it.  P is 2^11 p with p <= 2^4, rounded to
// fp16's 11 bits.  The scale of a key's page multiplies S in fp32; the scale of
// its V page, relative to the largest one so far, multiplies P, and its logarithm
// counts in the row's reference maximum: the largest p times scale of a row has
// its 11 bits however small the row's pages are beside others (as far as 2^-40),
// and a weight 2^-25 below that loses bits to fp16's range, 2^-36 below is nothing.
//
// Why another kernel: with rows on N (the kernel for few rows) both products
// take two e4m3 terms of Q and of P, and every 64 rows their own pass over the
// keys.  Here the widening is paid once for 256 rows: a 128-node tree x 64 heads
// on 8 of the cache, 32768 keys: 205 us against 333 (670 TFLOP/s of both
// products).  When it is taken: at paged_attn_rows.
//
// One CTA per SM walks its share of the list of blocks (as the other kernel
// does; a unit is up to 256 rows, two tiles).  Roles (20 warps):
//   0-7    softmax: warps 0-3 tile 0, 4-7 tile 1; a thread owns a row.  The
//          reference maximum moves only when a score passes it by 2^4, and with
//          it the row of O in TMEM; it falls where a larger V scale comes up (O
//          then stays as it is).
//   8-15   widening: a block's codes lie in the upper half of the tile that
//          takes them as fp16 (Q and the two fp16 rings leave no room beside
//          them): every warp reads its part into registers, then all write.
//   16, 17 MMA issuers, one per tile.  S comes in halves of 64 keys, two
//          buffers a tile: PV of one half, then S of the half a block on, which
//          runs under the softmax of the half between them.
//   18, 19 producers of K and of V: a page's rows of the head are one TMA box,
//          asked for a block ahead of their tile's release through L2.
// What bounds it: the chain of a half block through issuer, softmax and issuer
// again, not one unit.  Measured when that case took 219 us: with half of the
// MMAs 195, without widening 204, without exponentials 207, without all three
// 168; without the join of units that were cut (256 rows each) 202.
//
// Masks: the keys of tree blocks by the ancestor words of the row's node, keys
// past the end by their number.  V rows past the last key are zeros, and NaN
// codes of tree rows are kept out of the product and put back only into the
// rows that see them.
#include <type_traits>

#include "tsv_paged_tc.cuh"

namespace tsv {

namespace {

constexpr int kWThreads = 640;
constexpr int kWConvWarp = 8, kWMmaWarp = 16;
// Registers a thread: 640 x 96 at launch = 256 x 128 + 256 x 72 + 128 x 80.
constexpr int kWRegs = 96, kWSoftRegs = 128, kWConvRegs = 72, kWRestRegs = 80;
static_assert(256 * kWSoftRegs + 256 * kWConvRegs + 128 * kWRestRegs <= kWThreads * kWRegs, "register split");
constexpr int kWRows = kPagedWideRows, kWTile = 128;
constexpr float kWThreshold = 4.f;  // log2: how far a score may pass the reference maximum
constexpr float kWScale = 2048.f;   // of P: 2^4 x it is within fp16
constexpr int kWApart = 40;         // log2: V scales that far apart leave a row's weights their bits
constexpr int kHalf = 64;  // keys of a softmax step
// What a unit costs beside its blocks (Q, the pipeline's start and end, its
// results, the join), in blocks.  128 nodes x 64 heads over 32768 keys: 222 us
// at 0, 202 at 8 and 12, 206 at 20; 64 ragged requests of up to 64 nodes over up
// to 700 keys 330, 260, 252, 259.
constexpr PPad kWPad{12, 0};
constexpr int kBarWSoft = 1, kBarWJoin = 2, kBarWConv = 3;

template <int D>
struct WCfg {
  static constexpr int kTileBytes = kPBlock * D * 2;  // fp16 K or V block, or a Q tile
  static constexpr int kStages = 2;
  static constexpr int kOffQ = 0;                                    // [2 tiles]
  static constexpr int kOffK = kOffQ + 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kTiles = kOffV + kStages * kTileBytes, kWeights = kPagedWideCtas * kWRows * 4;
  static constexpr int kOffAnc = kTiles > kWeights ? kTiles : kWeights;       // u32 [256 rows][9]: ancestors (odd stride: no bank conflicts)
  static constexpr int kOffCum = kOffAnc + kWRows * 9 * 4;           // i64 [TSV_MAX_BATCH + 2]
  static constexpr int kOffReq = kOffCum + 8 * (TSV_MAX_BATCH + 2);  // int4 [TSV_MAX_BATCH]
  static constexpr int kOffFr = kOffReq + 16 * TSV_MAX_BATCH;        // f32 [256]: score factor of a row
  static constexpr int kOffRow = kOffFr + 4 * kWRows;                // i32 [256]: output row
  static constexpr int kOffScale = kOffRow + 4 * kWRows;             // f32 [4][28]: K's scales of 8 x 16 keys, V's relative ones, V's largest, [20..] logarithms
  static constexpr int kOffNan = kOffScale + 4 * 112;                // u32 [8]: tree keys whose V row holds a NaN
  static constexpr int kOffUnit = kOffNan + 32;                      // PUnit
  static constexpr int kOffFirst = kOffUnit + 64;                    // PUnit, then i64 [4]
  static constexpr int kOffBar = kOffFirst + 96;
  // k_full[2], k_empty[2], v_full[2], v_empty[2], sc_full[4], s_full[4], p_full[4], pv_done[4], mma_done, kc_full[2], vc_full[2]
  static constexpr int kBars = 29;
  static constexpr int kOffMisc = kOffBar + 8 * kBars + 8;
  static constexpr int kSmem = kOffMisc + 32 + 1024;
  static constexpr uint32_t kColO = 2 * kPBlock;  // S0 | S1 | O0 | O1
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kWRows * (D + 4) * 4 <= kOffAnc, "a partial's rows fit in the tiles");

  static_assert(kOffAnc % 1024 == 0 && kOffCum % 16 == 0 && kOffScale % 16 == 0 && kOffUnit % 16 == 0 && kOffBar % 8 == 0, "alignment");
};

// fp16 A and B, fp32 D; A K-major, B K-major (0) or N-major (1).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Issued by the whole warp, so that the operands stay uniform: the one lane
// with `lead` set issues the MMA.  A from shared memory, then A from TMEM.
__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate,
                                         uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate,
                                            uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}

// 16 bytes of a partial (through L2: another CTA wrote it), or zeros: no branch,
// so that several are in flight.
__device__ __forceinline__ float4 load_part(const float* p, bool on) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}\n"
      : "+f"(v.x), "+f"(v.y), "+f"(v.z), "+f"(v.w)
      : "l"(p), "r"((uint32_t)on)
      : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 codes as 16 fp16 values.
__device__ __forceinline__ void widen(const uint4& w, uint4& a, uint4& b) {
  a = make_uint4(f16x2_of_e4m3x2(w.x & 0xFFFFu), f16x2_of_e4m3x2(w.x >> 16), f16x2_of_e4m3x2(w.y & 0xFFFFu), f16x2_of_e4m3x2(w.y >> 16));
  b = make_uint4(f16x2_of_e4m3x2(w.z & 0xFFFFu), f16x2_of_e4m3x2(w.z >> 16), f16x2_of_e4m3x2(w.w & 0xFFFFu), f16x2_of_e4m3x2(w.w >> 16));
}
// Bytes that are NaN codes, as their top bits.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// What a role keeps of the unit.
struct WUnit {
  int n, P, g, off, row0, j, blocks, nmain, rows, ntiles, ntree;
  // Block j + i: its first key, how many it has.
  __device__ __forceinline__ int base(int i) const { return (j + i < nmain ? j + i : j + i - nmain) * kPBlock; }
  __device__ __forceinline__ int valid(int i) const { return max(0, min(kPBlock, (j + i < nmain ? P : ntree) - base(i))); }
};

template <int D>
__global__ void __launch_bounds__(kWThreads, 1)
    paged_attn_wide_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                           const __grid_constant__ PagedAttnArgs a, int32_t* words, float* __restrict__ part_o,
                           float* __restrict__ part_ml) {
  using C = WCfg<D>;
  int32_t* counters = words + TSV_MAX_BATCH;  // (the first words: requests that a wait was given up for)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  uint32_t* sAnc = reinterpret_cast<uint32_t*>(smem + C::kOffAnc);
  int64_t* sCum = reinterpret_cast<int64_t*>(smem + C::kOffCum);
  int4* sReq = reinterpret_cast<int4*>(smem + C::kOffReq);
  float* sFr = reinterpret_cast<float*>(smem + C::kOffFr);
  int32_t* sRow = reinterpret_cast<int32_t*>(smem + C::kOffRow);
  float* sScale = reinterpret_cast<float*>(smem + C::kOffScale);
  uint32_t* sNan = reinterpret_cast<uint32_t*>(smem + C::kOffNan);
  PUnit* sUnit = reinterpret_cast<PUnit*>(smem + C::kOffUnit);
  PUnit* sFirst = reinterpret_cast<PUnit*>(smem + C::kOffFirst);
  int64_t* sRange = reinterpret_cast<int64_t*>(smem + C::kOffFirst + 64);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* sc_full = v_empty + 2;
  uint64_t* s_full = sc_full + 4;   // [tile][half]
  uint64_t* p_full = s_full + 4;    // [tile][half]
  // A wait must be for the current phase or the one just past, so a barrier
  // whose phases could run two ahead of a waiter is split: here by half.
  uint64_t* pv_done = p_full + 4;   // [tile][half]
  uint64_t* mma_done = pv_done + 4;
  uint64_t* kc_full = mma_done + 1;  // a block's codes are in
  uint64_t* vc_full = kc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  int* abort_flag = reinterpret_cast<int*>(smem + C::kOffMisc + 4);
  int* sJoin = reinterpret_cast<int*>(smem + C::kOffMisc + 8);
  volatile int* abort_v = abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lps = __ffs(a.cache.page_size) - 1;  // pages are powers of two
  const bool tree = a.tree_table.ids_d != nullptr;
  bool dead = false;

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], 8);   // the widening warps
      mbar_init(&k_empty[s], 2);  // both tiles' issuers (the first for both when there is one)
      mbar_init(&v_full[s], 8);
      mbar_init(&v_empty[s], 2);
      mbar_init(&kc_full[s], 1);
      mbar_init(&vc_full[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sc_full[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 128);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kWMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  if (warp == 0) plist_setup(a, kWRows, kWPad, sCum, sReq, sFirst, sRange);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const PList list{sCum, sReq, a.B, a.G, a.cache.Hkv, kWRows, kWPad, tree, sRange[1]};

  // Every role walks the units together: a barrier before each, one when its
  // rows are in, and one behind it.
  if (tid == 0) {
    *sUnit = *sFirst;
    *sJoin = 0;
  }
  int t = 0;            // blocks so far
  int cnt[2] = {0, 0};  // and those of each tile
  auto begin = [&](WUnit& u) {
    __syncthreads();
    if (!sUnit->valid) return false;
    u.n = sUnit->n;
    u.P = sUnit->P;
    u.g = sUnit->g;
    u.off = sUnit->off;
    u.row0 = sUnit->tile * kWRows;
    u.j = sUnit->j;
    u.blocks = sUnit->j1 - u.j;
    u.nmain = sUnit->nmain;
    u.rows = min(kWRows, u.n * a.G - u.row0);
    u.ntiles = u.rows > kWTile ? 2 : 1;
    u.ntree = tree ? u.n : 0;
    return true;
  };
  auto end = [&](const WUnit& u) {
    t += u.blocks;
    cnt[0] += u.blocks;
    if (u.ntiles > 1) cnt[1] += u.blocks;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  WUnit u{};
  // CTAs cf .. cf + parts - 1 share the unit's group; part c is in slot(c).
  struct Group {
    int cf, parts, first;  // first: the group is the first unit of CTA cf, or its last
    __device__ __forceinline__ int64_t slot(int c) const { return 2 * (cf + c) + (c == 0 ? first : 0); }
  };
  auto group = [&]() {
    const int64_t W = sRange[2], ctas = sRange[3], gx = sUnit->gx, g0 = gx + list.pad.of(sUnit->T);  // g0: of its first block
    Group z;
    z.cf = (int)(((g0 + 1) * ctas - 1) / W);
    z.parts = (int)(((g0 + sUnit->T) * ctas - 1) / W) - z.cf + 1;
    z.first = (int64_t)z.cf * W / ctas >= gx ? 0 : 1;
    return z;
  };
  float* weight = reinterpret_cast<float*>(smem);  // [part][row], over the idle tiles
  // The group's rows from its parts (threads 0 .. 511): 16 bytes at a time, two
  // of a thread with four parts each in flight.
  auto join = [&](int i_first) {
    const Group z = group();
    constexpr int kItems = 2, kParts = 4, L4 = D / 4;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
#pragma unroll 1
    for (int i0 = i_first; i0 < u.rows * L4; i0 += kItems * 512) {
      float4 o[kItems];
#pragma unroll
      for (int x = 0; x < kItems; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int c0 = 0; c0 < z.parts; c0 += kParts) {
        float4 v[kParts][kItems];
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
          const float* part = part_o + z.slot(c0 + c) * kWRows * D;
#pragma unroll
          for (int x = 0; x < kItems; ++x) {
            const int i = i0 + x * 512;
            v[c][x] = load_part(part + 4 * i, c0 + c < z.parts && i < u.rows * L4);
          }
        }
#pragma unroll
        for (int c = 0; c < kParts; ++c)
#pragma unroll
          for (int x = 0; x < kItems; ++x) {
            const int i = i0 + x * 512;
            if (c0 + c >= z.parts || i >= u.rows * L4) continue;
            const float w = weight[(c0 + c) * kWRows + i / L4];
            o[x].x += w * v[c][x].x;
            o[x].y += w * v[c][x].y;
            o[x].z += w * v[c][x].z;
            o[x].w += w * v[c][x].w;
          }
      }
#pragma unroll
      for (int x = 0; x < kItems; ++x) {
        const int i = i0 + x * 512;
        if (i < u.rows * L4)
          *reinterpret_cast<uint2*>(out + (int64_t)sRow[i / L4] * D + (i % L4) * 4) =
              make_uint2(pack_bf16x2(o[x].x, o[x].y), pack_bf16x2(o[x].z, o[x].w));
      }
    }
  };

  if (warp >= kWConvWarp && warp < kWMmaWarp) {
    // ---------------------------------------------------------- Q, then K and V, widened
    setmaxnreg_dec<kWConvRegs>();
    while (begin(u)) {
      const int w = warp - kWConvWarp, ct = tid - kWConvWarp * 32;
      const tsv_paged_cache& c = a.cache;
      // A lane's part of a block: 16 codes of rows first_row, first_row + kStep, ...
      constexpr int kLanes = D / 16, kStep = 256 / kLanes, kParts = kPBlock / kStep;  // lanes of a row; 4 or 2 rows of a thread
      // Eight lanes take four 16-code chunks of two rows: their stores meet 32 banks.
      const int chunk = D == 128 ? (ct & 3) | ((ct >> 1) & 4) : ct & 3;
      const int first_row = D == 128 ? ((ct >> 2) & 1) | ((ct >> 4) << 1) : ct >> 2;
      // Warp 0, lanes 0 .. 7: the page of 16 keys each, two blocks ahead, its scales one.
      int sid = -1;
      float sk = 0.f, sv = 0.f, top = 0.f;
      auto look = [&](int i) {
        sid = -1;
        if (w != 0 || lane >= 8 || lane * 16 >= u.valid(i)) return;
        const tsv_page_table& pt = u.j + i < u.nmain ? a.table : a.tree_table;
        sid = __ldg(pt.ids_d + (int64_t)sUnit->b * pt.stride + ((u.base(i) + lane * 16) >> lps));
      };
      auto scales = [&]() {
        sk = sv = 0.f;
        if ((uint32_t)sid < (uint32_t)c.num_pages) {
          sk = __ldg(c.k_scale_d + (int64_t)sid * c.Hkv + u.g);
          sv = __ldg(c.v_scale_d + (int64_t)sid * c.Hkv + u.g);
        }
      };
      // The lane's codes of a block, out of the tile's upper half.
      auto take = [&](const uint8_t* tile, int valid, uint4 (&codes)[kParts]) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          const int key = first_row + q * kStep;
          const int at = D == 128 ? key * 128 + ((chunk ^ (key & 7)) << 4) : key * 64 + ((chunk ^ ((key >> 1) & 3)) << 4);
          codes[q] = make_uint4(0u, 0u, 0u, 0u);
          if (key < valid) codes[q] = *reinterpret_cast<const uint4*>(tile + C::kTileBytes / 2 + at);
        }
      };
      auto put = [&](uint8_t* tile, int key, const uint4& codes) {
        uint4 x, y;
        widen(codes, x, y);
        uint8_t* row = tile + (chunk >> 2) * (kPBlock * 128) + key * 128;
        const int at = (((2 * chunk) & 7) ^ (key & 7)) << 4;  // chunk 2 c of 8 values, and its neighbour
        *reinterpret_cast<uint4*>(row + at) = x;
        *reinterpret_cast<uint4*>(row + (at ^ 16)) = y;
      };
      look(0);
      scales();
      if (u.blocks > 1) look(1);
      {
        constexpr int E = D / 32;
#pragma unroll 1
        for (int r = w * 32; r < w * 32 + 32; ++r) {
          if (r >= u.ntiles * kWTile) break;
          const int gr = u.row0 + r, node = gr / a.G, head = u.g * a.G + (gr - node * a.G);
          uint32_t raw[E / 2];
#pragma unroll
          for (int e = 0; e < E / 2; ++e) raw[e] = 0u;
          if (r < u.rows) {
            const __nv_bfloat16* src =
                static_cast<const __nv_bfloat16*>(a.q) + (int64_t)(u.off + node) * a.qs_n + (int64_t)head * a.qs_h + lane * E;
            if constexpr (E == 4) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
              raw[0] = v.x;
              raw[1] = v.y;
            } else {
              raw[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
            }
          }
          uint32_t top = 0u;
#pragma unroll
          for (int e = 0; e < E / 2; ++e) top = max(top, max((raw[e] << 16) & 0x7FFF0000u, raw[e] & 0x7FFF0000u));
          top = __reduce_max_sync(0xffffffffu, top);
          const bool fine = top < 0x7F800000u;  // a row with an infinity or a NaN is NaN throughout (its scores are)
          const int up = top == 0u ? 0 : max(-120, min(120, 141 - (int)(top >> 23)));
          const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
          if (lane == 0) {
            sFr[r] = __uint_as_float((uint32_t)(127 - up) << 23) * (a.scale * 1.4426950408889634f);
            sRow[r] = r < u.rows ? (u.off + node) * a.Hq + head : -1;
          }
          uint32_t h[E / 2];
#pragma unroll
          for (int e = 0; e < E / 2; ++e)
            h[e] = fine ? pack_f16x2(__uint_as_float(raw[e] << 16) * mul, __uint_as_float(raw[e] & 0xFFFF0000u) * mul) : 0x7FFF7FFFu;
          const int d = lane * E, rt = r & (kWTile - 1);
          uint8_t* at = sQ + (r >> 7) * C::kTileBytes + (d >> 6) * (kWTile * 128) + rt * 128 +
                        ((((d & 63) >> 3) ^ (rt & 7)) << 4) + (d & 7) * 2;
          if constexpr (E == 4) *reinterpret_cast<uint2*>(at) = make_uint2(h[0], h[1]);
          else *reinterpret_cast<uint32_t*>(at) = h[0];
        }
        if (ct < 8) sNan[ct] = 0u;
        fence_proxy_async_smem();
      }
      __syncthreads();  // the unit's rows are in
#pragma unroll 1
      for (int i = 0; i < u.blocks; ++i) {
        const int x = t + i, st = x & 1;
        const int valid = u.valid(i);
        uint4 codes[kParts];
        float rv = 0.f;
        if (w == 0) {
          // The unit's largest V scale so far, and the block's relative to it (the
          // ratio first: of zeros' 2^-126 the reciprocal times kWScale is no fp32
          // number), worked out while the codes are on their way.
          top = fmaxf(top, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(sv))));  // (scales are >= 0)
          const float even = top > 1.f ? 0x1p-64f : 0x1p64f;  // (the division wants an ordinary divisor)
          rv = top > 0.f ? __fdividef(sv * even, top * even) : 0.f;
        }
        TSV_PWAIT(&kc_full[st], x >> 1);
        take(sK + st * C::kTileBytes, valid, codes);
        dead = named_bar_or(kBarWConv, 256, dead);  // everyone has read, or gives up
        if (dead) break;
        if (w == 0) {
          if (lane < 8) {
            sScale[(x & 3) * 28 + lane] = sk;
            sScale[(x & 3) * 28 + 8 + lane] = rv * kWScale;
            sScale[(x & 3) * 28 + 20 + lane] = fmaxf(__log2f(rv), -(float)kWApart);
          }
          if (lane == 0) sScale[(x & 3) * 28 + 16] = top;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[x & 3]);
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) put(sK + st * C::kTileBytes, first_row + q * kStep, codes[q]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[st]);
        if (i + 1 < u.blocks) scales();
        if (i + 2 < u.blocks) look(i + 2);
        TSV_PWAIT(&vc_full[st], x >> 1);
        take(sV + st * C::kTileBytes, valid, codes);
        dead = named_bar_or(kBarWConv, 256, dead);
        if (dead) break;
        if (u.j + i >= u.nmain) {
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            uint32_t* v = reinterpret_cast<uint32_t*>(&codes[q]);
            uint32_t any = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t bad = nan_codes(v[e]);
              any |= bad;
              v[e] &= ~((bad >> 7) * 0xFFu);
            }
            const int key = u.base(i) + first_row + q * kStep;
            if (any) atomicOr(&sNan[key >> 5], 1u << (key & 31));
          }
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) put(sV + st * C::kTileBytes, first_row + q * kStep, codes[q]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[st]);
      }
      if (!sUnit->whole()) {
        named_bar_sync(kBarWJoin, 512);
        if (*sJoin) join(tid);
        fence_proxy_async_smem();
      }
      end(u);
    }
  } else if (warp >= kWMmaWarp) {
    // ---------------------------------------------------------- issuer
    setmaxnreg_dec<kWRestRegs>();
    int asked = 0;  // blocks that the producer has asked for
    while (begin(u)) {
      __syncthreads();  // the unit's rows are in
      const int q = warp - kWMmaWarp;  // the issuer's tile
      if (q < u.ntiles) {
        constexpr uint32_t idS = idesc_f16_f32(kWTile, kHalf, 0), idPV = idesc_f16_f32(kWTile, D, 1);
        const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk = sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dv = sdesc_sw128(smem_u32(sV), kPBlock * 128, 1024);
        // S of tile and half block: 64 keys, so that a tile has two buffers and
        // the next half's scores are there when its softmax gets to them.
        auto issue_s = [&](int tile, int x, int half) {
          const uint32_t da = (uint32_t)dq + (uint32_t)((tile * C::kTileBytes) >> 4);
          const uint32_t db = (uint32_t)dk + (uint32_t)(((x & 1) * C::kTileBytes + half * (kHalf * 128)) >> 4);
          const uint32_t dst = tmem + (uint32_t)(tile * kPBlock + half * kHalf);
          const bool lead = elect_one();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * (kPBlock * 128) + (kk & 3) * 32) >> 4;
            umma_f16(dst, desc_at(dq, da + o), desc_at(dk, db + o), idS, kk > 0 ? 1u : 0u, lead);
          }
          if (lead) umma_commit(&s_full[2 * tile + half]);
          __syncwarp();
        };
        // O += P V over those keys; P, two keys a column, lies over its S.
        auto issue_pv = [&](int tile, int x, int half, bool more) {
          const uint32_t db = (uint32_t)dv + (uint32_t)(((x & 1) * C::kTileBytes + half * (kHalf * 128)) >> 4);
          const uint32_t pa = tmem + (uint32_t)(tile * kPBlock + half * kHalf), dst = tmem + C::kColO + (uint32_t)(tile * D);
          const bool lead = elect_one();
#pragma unroll
          for (int kk = 0; kk < kHalf / 16; ++kk)
            umma_f16_ts(dst, pa + kk * 8, desc_at(dv, db + ((kk * 16 * 128) >> 4)), idPV, more || kk > 0 ? 1u : 0u, lead);
          if (lead) umma_commit(&pv_done[2 * tile + half]);
          __syncwarp();
        };
        const int both = u.ntiles == 1 ? 2 : 1;  // arrivals at the rings' barriers
        TSV_PWAIT(&k_full[t & 1], t >> 1);
        if (!__any_sync(0xffffffffu, dead)) {
          tc_fence_after();
          issue_s(q, t, 0);
          issue_s(q, t, 1);
          if (elect_one())
            for (int n = 0; n < both; ++n) umma_commit(&k_empty[t & 1]);
          __syncwarp();
        }
#pragma unroll 1
        for (int h = 0; h < 2 * u.blocks; ++h) {
          const int i = h >> 1, half = h & 1, x = t + i;
          const bool more = i + 1 < u.blocks;
          if (half == 0) TSV_PWAIT(&v_full[x & 1], x >> 1);
          TSV_PWAIT(&p_full[2 * q + half], cnt[q] + i);
          if (__any_sync(0xffffffffu, dead)) break;
          tc_fence_after();
          issue_pv(q, x, half, h > 0);
          if (half == 1 && elect_one())
            for (int n = 0; n < both; ++n) umma_commit(&v_empty[x & 1]);
          if (more) {
            if (half == 0) TSV_PWAIT(&k_full[(x + 1) & 1], (x + 1) >> 1);
            if (__any_sync(0xffffffffu, dead)) break;
            tc_fence_after();
            issue_s(q, x + 1, half);
            if (half == 1 && elect_one())
              for (int n = 0; n < both; ++n) umma_commit(&k_empty[(x + 1) & 1]);
          }
          __syncwarp();
        }
      } else if (q >= 2) {
        // ------------------------------------------------------ producers of K and of V
        const bool is_v = q == 3;
        const CUtensorMap* tmap = is_v ? &tmap_v : &tmap_k;
        uint64_t* full = is_v ? vc_full : kc_full;
        uint64_t* empty = is_v ? v_empty : k_empty;
        const uint64_t pol = sUnit->tiles > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
        // Lane p holds page p of the next block.
        auto page_of = [&](int i) {
          if (i >= u.blocks || (lane << lps) >= u.valid(i)) return -1;
          const tsv_page_table& pt = u.j + i < u.nmain ? a.table : a.tree_table;
          return __ldg(pt.ids_d + (int64_t)sUnit->b * pt.stride + (u.base(i) >> lps) + lane);
        };
        int next = page_of(0);
#pragma unroll 1
        for (int i = 0; i < u.blocks; ++i) {
          const int x = t + i, st = x & 1, ids = next;
          next = page_of(i + 1);
          const uint32_t pages = (uint32_t)(u.valid(i) + (1 << lps) - 1) >> lps;
          if (x >= 2) TSV_PWAIT(&empty[st], (x >> 1) - 1);
          if (__any_sync(0xffffffffu, dead)) break;
          const uint32_t at = smem_u32(is_v ? sV : sK) + (uint32_t)(st * C::kTileBytes + C::kTileBytes / 2);
          const bool lead = elect_one();
          if (pages > 0 && lead) mbar_expect_tx(&full[st], (pages << lps) * D);
#pragma unroll 1
          for (uint32_t p = 0; p < pages; ++p)
            tma_load_page(at + (p << lps) * D, tmap, smem_u32(&full[st]), (uint32_t)u.g,
                          (uint32_t)__shfl_sync(0xffffffffu, ids, (int)p), pol, lead);
          __syncwarp();
          if (lead) mbar_arrive(&full[st]);
          if ((uint32_t)next < (uint32_t)a.cache.num_pages) tma_prefetch_4d(tmap, 0, u.g, 0, next);
          asked = x + 1;
        }
      }
      end(u);
    }
    // Every copy has landed before the CTA leaves (whatever the other roles did).
    if (warp >= kWMmaWarp + 2)
      for (int x = max(0, asked - 2); x < asked; ++x)
        mbar_wait(warp == kWMmaWarp + 3 ? &vc_full[x & 1] : &kc_full[x & 1], (x >> 1) & 1, nullptr);
  } else {
    // ---------------------------------------------------------- softmax: a thread owns a row
    setmaxnreg_inc<kWSoftRegs>();
    for (int k = 0; begin(u); ++k) {
      const int tile = warp >> 2, r = tid & (kWTile - 1), row = tile * kWTile + r;
      const bool active = tile < u.ntiles;
      uint32_t* anc = sAnc + row * 9;
      if (tree) {  // the row's ancestors
        const int node = (u.row0 + row) / a.G;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t bits = 0u;
          if (row < u.rows) {
            const int left = node + 1 - 32 * q;
            bits = a.anc ? __ldg(a.anc + (int64_t)(u.off + node) * TSV_ANC_WORDS + q)
                         : left >= 32 ? 0xFFFFFFFFu : left > 0 ? (1u << left) - 1u : 0u;
          }
          anc[q] = bits;
        }
      }
      __syncthreads();  // the unit's rows are in
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t o_col = tmem + lane_base + C::kColO + (uint32_t)(tile * D);
      const float fr = sFr[row];
      float m_ref = -INFINITY, l = 0.f, v_ref = 0.f;
      int room = kWApart;  // how far the reference may still be lowered
      auto half_step = [&](int h, auto masked_c) {
        constexpr bool MASKED = decltype(masked_c)::value;
        const int i = h >> 1, half = h & 1, x = t + i;
        TSV_PWAIT(&s_full[2 * tile + half], cnt[tile] + i);
        if (half == 0) TSV_PWAIT(&sc_full[x & 3], x >> 2);
        if (__any_sync(0xffffffffu, dead)) return;
        tc_fence_after();
        const uint32_t s_col = tmem + lane_base + (uint32_t)(tile * kPBlock + half * kHalf);
        uint32_t s[2][32];
        tmem_ld32_nowait(s_col, s[0]);
        tmem_ld32_nowait(s_col + 32, s[1]);
        const float* sc = sScale + (x & 3) * 28;
        const float4 k4 = *reinterpret_cast<const float4*>(sc + 4 * half);
        const float4 v4 = *reinterpret_cast<const float4*>(sc + 8 + 4 * half);  // times kWScale, relative to v_top
        const float4 g4 = *reinterpret_cast<const float4*>(sc + 20 + 4 * half);  // log2 of that
        const float v_top = sc[16];  // V's largest scale so far
        const float f[4] = {k4.x * fr, k4.y * fr, k4.z * fr, k4.w * fr};  // the row's factor of 16 keys each
        uint32_t see[2] = {~0u, ~0u};
        if (MASKED) {
          const int valid = u.valid(i) - half * kHalf;
          see[0] = valid >= 32 ? ~0u : valid > 0 ? (1u << valid) - 1u : 0u;
          see[1] = valid >= 64 ? ~0u : valid > 32 ? (1u << (valid - 32)) - 1u : 0u;
          if (u.j + i >= u.nmain) {
            const uint32_t* m = anc + 4 * (u.j + i - u.nmain) + 2 * half;
            see[0] &= m[0];
            see[1] &= m[1];
          }
        }
        tmem_wait_ld_tie32(s[0]);
        reg_tie32(s[1]);
        if (MASKED) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (!((see[e >> 5] >> (e & 31)) & 1u)) s[e >> 5][e & 31] = 0xFF800000u;
        }
        float alpha = 1.f;
        if (v_top > v_ref) {  // the same in every thread
          // What was summed up stays, under a reference that is lower by as much as
          // the relative scales of its keys now are (powers of two: l goes with it).
          if (v_ref > 0.f) {
            const float c = v_ref / v_top;
            const int down = min(127 - (int)(__float_as_uint(c) >> 23), room);
            const float up = __uint_as_float((uint32_t)(127 + down) << 23);
            room -= down;
            m_ref -= (float)down;
            l *= up;
            alpha = c * up;  // 1 for scales that are powers of two
          }
          v_ref = v_top;
        }
        const float g[4] = {g4.x, g4.y, g4.z, g4.w};
        float hmax = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t* z = &s[q >> 1][(q & 1) * 16];
          float b0 = fmaxf(__uint_as_float(z[0]), __uint_as_float(z[1]));
          float b1 = fmaxf(__uint_as_float(z[2]), __uint_as_float(z[3]));
#pragma unroll
          for (int e = 4; e < 16; e += 4) {
            b0 = fmax3(b0, __uint_as_float(z[e]), __uint_as_float(z[e + 1]));
            b1 = fmax3(b1, __uint_as_float(z[e + 2]), __uint_as_float(z[e + 3]));
          }
          hmax = fmaxf(hmax, fmaf(fmaxf(b0, b1), f[q], g[q]));
        }
        if (hmax > m_ref + kWThreshold) {
          const float a = fast_exp2(m_ref - hmax);  // 0 when m_ref = -inf
          m_ref = hmax;
          l *= a;
          alpha *= a;
        }
        if (h > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          TSV_PWAIT(&pv_done[2 * tile + (1 - half)], cnt[tile] + ((h - 1) >> 1));
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 16) {
            float o[16];
            tmem_ld16(o_col + cc, o);
            uint32_t z16[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) z16[e] = __float_as_uint(o[e] * alpha);
            tmem_st16u_nowait(o_col + cc, z16);
          }
        }
        const float neg_ref = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t ref2 = f2_pack(neg_ref, neg_ref);
        uint64_t sum[2] = {0ull, 0ull};
        const float fv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int q = 2 * c + (e >> 4);
            const uint64_t x2 = ffma2((uint64_t)s[c][e] | ((uint64_t)s[c][e + 1] << 32), f2_pack(f[q], f[q]), ref2);
            float p0 = fast_exp2(f2_lo(x2)), p1 = fast_exp2(f2_hi(x2));
            if (MASKED) {
              if (!((see[c] >> e) & 1u)) p0 = 0.f;
              if (!((see[c] >> (e + 1)) & 1u)) p1 = 0.f;
            }
            const uint64_t p2 = f2_pack(p0, p1);
            sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], p2);
            const uint64_t y2 = fmul2(p2, f2_pack(fv[q], fv[q]));
            p[e >> 1] = pack_f16x2(f2_lo(y2), f2_hi(y2));
          }
          tmem_st16u_nowait(s_col + 16 * c, p);
        }
        tmem_wait_st();
        const uint64_t both = fadd2(sum[0], sum[1]);
        l += f2_lo(both) + f2_hi(both);
        tc_fence_before();
        parrive(&p_full[2 * tile + half], dead);
      };
      // Blocks of 128 prefix keys need no mask.
      const int whole_main = max(0, min(u.blocks, u.P / kPBlock - u.j));
      if (active) {
#pragma unroll 1
        for (int h = 0; h < 2 * whole_main; ++h) half_step(h, std::false_type{});
#pragma unroll 1
        for (int h = 2 * whole_main; h < 2 * u.blocks; ++h) half_step(h, std::true_type{});
        TSV_PWAIT(&pv_done[2 * tile], cnt[tile] + u.blocks - 1);
        TSV_PWAIT(&pv_done[2 * tile + 1], cnt[tile] + u.blocks - 1);
      }
      const bool stop = named_bar_or(kBarWSoft, 256, dead);  // the same in every softmax thread
      if (!stop) {
        tc_fence_after();
        // Columns of a row whose NaN codes were kept out of the product.
        uint32_t bad[D / 32];
#pragma unroll
        for (int q = 0; q < D / 32; ++q) bad[q] = 0u;
        if (tree && active && row < u.rows) {
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
#pragma unroll 1
            for (uint32_t seen = sNan[q] & anc[q]; seen; seen &= seen - 1) {
              const int key = 32 * q + __ffs(seen) - 1;
              const int id = __ldg(a.tree_table.ids_d + (int64_t)sUnit->b * a.tree_table.stride + (key >> lps));
              if ((uint32_t)id >= (uint32_t)a.cache.num_pages) continue;
              const uint32_t* v = reinterpret_cast<const uint32_t*>(
                  static_cast<const uint8_t*>(a.cache.v_d) + (int64_t)id * a.cache.stride_page +
                  (int64_t)(key & ((1 << lps) - 1)) * a.cache.stride_row + (int64_t)u.g * a.cache.stride_head);
#pragma unroll
              for (int e = 0; e < D / 4; ++e) {
                const uint32_t m = nan_codes(__ldg(v + e)) >> 7;  // bits 0, 8, 16, 24
                bad[e >> 3] |= ((m | (m >> 7) | (m >> 14) | (m >> 21)) & 15u) << (4 * (e & 7));
              }
            }
          }
        }
        // (0 for a row that sees nothing.  v_ref may be 2^-126, a page of zeros', or
        // little more: then it is a factor of its own.)
        const bool tiny = v_ref < 0x1p-60f;
        const float inv = l == 0.f ? 0.f : (1.f / kWScale) / l * (tiny ? 1.f : v_ref);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
        const bool whole = sUnit->whole();
        const int slot = 2 * (int)blockIdx.x + (k == 0 ? 0 : 1);
        if (active) {
          __nv_bfloat16* to = out + (int64_t)(row < u.rows ? sRow[row] : 0) * D;
          // A partial's rows go through shared memory (the tiles are idle), a
          // warp its own 32, so that a store covers a whole row.
          float* po = part_o + ((int64_t)slot * kWRows + (row & ~31)) * D;
          float* mine = reinterpret_cast<float*>(smem) + row * (D + 4);
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) {
            float o[32];
            tmem_ld32(o_col + cc, o);
            if (row < u.rows) {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : (bad[cc / 32] >> e) & 1u ? NAN : o[e] * inv;
              if (tiny) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= v_ref;
              }
              if (whole) {
#pragma unroll
                for (int e = 0; e < 32; e += 8)
                  *reinterpret_cast<uint4*>(to + cc + e) = make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                                                                      pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(mine + cc + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
              }
            }
          }
          if (!whole) {
            __syncwarp();
            constexpr int kOnce = 128 / D;  // rows of a store
            const int rl = lane / (D / 4), d4 = (lane % (D / 4)) * 4;
#pragma unroll 4
            for (int q = rl; q < 32; q += kOnce)
              if ((row & ~31) + q < u.rows)
                *reinterpret_cast<float4*>(po + q * D + d4) =
                    *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + ((row & ~31) + q) * (D + 4) + d4);
          }
          if (!whole && row < u.rows) {  // normalised: its sum is 1
            float* pm = part_ml + (int64_t)slot * 2 * kWRows;
            const bool sees = l != 0.f;
            pm[row] = l > 0.f ? m_ref + log2f(l) : sees ? m_ref : -INFINITY;
            pm[kWRows + row] = l > 0.f ? 1.f : l;
          }
        }
        if (!whole) {
          // The last CTA of the group to arrive joins.
          const Group z = group();
          named_bar_sync(kBarWSoft, 256);
          if (tid == 0) {
            const int before = atom_add_acq_rel_gpu(counters + z.cf, 1);
            const bool last = before == z.parts - 1;
            if (last) counters[z.cf] = 0;
            *sJoin = last ? 1 : 0;
          }
          named_bar_sync(kBarWSoft, 256);
          if (*sJoin) {
            // Weights of the parts of every row (a thread each); the rows follow.
            if (tid < u.rows) {
              float top = -INFINITY, all = 0.f;
#pragma unroll 4
              for (int c = 0; c < z.parts; ++c) top = fmaxf(top, __ldcg(part_ml + z.slot(c) * 2 * kWRows + tid));
#pragma unroll 4
              for (int c = 0; c < z.parts; ++c) {
                const float* ml = part_ml + z.slot(c) * 2 * kWRows + tid;
                const float m = __ldcg(ml), w = m == -INFINITY ? 0.f : fast_exp2(m - top);
                all += w * __ldcg(ml + kWRows);
                weight[c * kWRows + tid] = w;
              }
              const float scale = all == 0.f ? 0.f : 1.f / all;
              for (int c = 0; c < z.parts; ++c) weight[c * kWRows + tid] *= scale;
            }
          }
        }
      }
      if (!sUnit->whole()) {
        named_bar_sync(kBarWJoin, 512);
        if (*sJoin) join(tid);
        fence_proxy_async_smem();  // the next unit's copies come after these accesses of the tiles
      }
      end(u);
      if (tid == 0) {
        PUnit next = *sUnit;
        list.next(next);
        *sUnit = next;
        *sJoin = 0;
      }
    }
  }
  if (warp == kWMmaWarp || warp == kWMmaWarp + 1) {
    if (elect_one()) umma_commit(mma_done);  // every MMA has finished before TMEM is freed
    __syncwarp();
    mbar_wait(mma_done, 0, nullptr);
  } else if (warp == kWMmaWarp + 2) {
    // Every request's lengths and page ids are checked by one CTA.
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      PagedRequest r;
      bool bad = !paged_request(a, b, &r);
      if (!bad) bad = paged_bad_page(a, b, r, lane, 32);
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) report_check(a, words, b, bad);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_v)
    for (PUnit u = *sFirst; u.valid; list.next(u)) report_timeout(a, words, u.b);
  if (warp == kWMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_typed(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int num_sms, void* ws, cudaStream_t st) {
  const int grid = min(num_sms, kPagedWideCtas);
  char* w = static_cast<char*>(ws);
  const PagedAttnLayout lay = paged_attn_layout(grid, kWRows, D);
  return launch_pdl(paged_attn_wide_kernel<D>, dim3(grid), dim3(kWThreads), (size_t)WCfg<D>::kSmem, st, 0u, tk, tv, a,
                    reinterpret_cast<int32_t*>(w), reinterpret_cast<float*>(w + lay.part_o), reinterpret_cast<float*>(w + lay.part_ml));
}

template <int D>
cudaError_t set_typed() {
  // The register split draws on what the block is launched with.
  cudaFuncAttributes attr;
  const cudaError_t e = cudaFuncGetAttributes(&attr, paged_attn_wide_kernel<D>);
  if (e != cudaSuccess) return e;
  if (attr.numRegs < kWRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(paged_attn_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, WCfg<D>::kSmem);
}

}  // namespace

cudaError_t paged_attention_wide_set_attributes(int32_t D) { return D == 64 ? set_typed<64>() : set_typed<128>(); }

cudaError_t launch_paged_attention_wide(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int num_sms, void* ws,
                                        cudaStream_t st) {
  return a.cache.D == 64 ? launch_typed<64>(tk, tv, a, num_sms, ws, st) : launch_typed<128>(tk, tv, a, num_sms, ws, st);
}

}  // namespace tsv
