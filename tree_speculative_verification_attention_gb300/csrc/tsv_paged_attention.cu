// tsv_paged_attention.cu — tree attention over a paged 8-bit cache on the
// tensor cores, keys on the TMEM lanes.
//
//   S^T = K Q^T       M = 128 keys, N = rows, K = D      (A = K tile, B = Q tile)
//   O^T = V^T P^T     M = 128 (d), N = 2 x rows, K = 128 keys (A = V tile, M-major)
//
// Both products run on the e4m3 codes themselves, straight from the bytes that
// TMA brings in: nothing is widened on the way, so a 128-key block of one head
// costs 32 KB of shared memory and of HBM traffic, which is the bound while a
// KV head has few query rows.  The operands that are not e4m3 are split:
//   q = (hi + lo) 2^-k   two e4m3 terms under a power of two per row (the
//                        row's largest value lands in [128, 256)): a bf16's 8
//                        bits exactly down to 2^-17 of the row's largest.
//   p = (hi + lo) / 256  relative to the step's own largest score of the row:
//                        off by 2^-8 of itself or 2^-18 of that largest (256
//                        keys: 2^-10 of the step; of weights times V's scale
//                        2^-14 where scales lie up to 2^4 apart, see below).
// The terms of q accumulate into the same S; those of p lie side by side on the
// N axis of one MMA (an MMA of this shape takes its issue time, not its N) and
// are added in fp32.
// That the reference maximum is the step's own (not a running one) keeps those
// bounds whatever the earlier steps held; O of a step is brought to the running
// maximum in fp32 registers, which also keeps long sums out of the tensor core's
// accumulator.  The scale of a key's page multiplies S, and the scale of its V
// page, relative to the step's largest, multiplies P.  Where V's scales in a step
// lie more than 2^4 apart (a page of zeros has 2^-126), the reference is instead
// the row's largest score plus the logarithm of that ratio, so that a row whose
// weight lies on pages of small values keeps its bits: a second look at S, taken
// by such steps alone.
//
// Work.  The 128-key blocks of all (request, KV head, row tile) groups form one
// list, cut into equal ranges, one per CTA (one CTA per SM): every SM gets the
// same number of blocks whatever the lengths, which the kernel reads from the
// device.  A group that a cut goes through leaves fp32 partials in the
// workspace, and the last of its CTAs to arrive joins them in a fixed order.
// Inside a CTA two blocks make a step: one exchange of maxima, one O and one
// round of barriers for 256 keys.  With few rows the bound is not the bytes but
// the instructions around them (a warp's chain of dependent steps runs at 6 to
// 7 cycles an instruction, a third of it waiting for instruction fetches), so
// what a step costs once matters most.  Measured: 32 requests x 2064 keys x 32
// heads, 16 rows each, 122 us (4.5 TB/s; at 144 us it took 104 without P's
// arithmetic, 137 without O's sums, 122 with one MMA of four for O); one token of
// 8 requests, 64 heads on 8 of the cache, 25 us; a 20-node tree over 1024 keys, 32
// heads, 15.9 us.
//
// Roles (20 warps): two softmax warpgroups (warps 0-3 and 4-7; a thread owns a
// key of each block), which take alternate steps, or, with 64 rows, 32 rows of
// every step each; the accumulating warpgroup (8-11; a thread owns a d); the
// producers (12, 13 of K, 14, 15 of V, each pair taking alternate blocks: page
// ids and scales are looked up a warp's worth ahead, a page is one TMA box, and
// a box costs its warp about 100 cycles); the issuers of S and of O (16, 17);
// and two warps that prepare the next unit's Q tiles and tree mask (18, 19).
// What a role needs from the rows (maxima, factors) is worked out by each of its
// warps for itself: a step costs a softmax group one barrier and the
// accumulating group none.  The register file is split by role.
//
// Tail and tree blocks: V rows past the last key are zeroed in shared memory
// and NaN codes of tree rows are taken out of the product and put back only
// into the rows that see them, so that 0 x NaN reaches nobody.
#include <type_traits>

#include "tsv_paged_tc.cuh"

namespace tsv {

namespace {

constexpr int kPThreads = 640;
constexpr int kPProducerWarp = 12, kPSWarp = 16, kPOWarp = 17, kPPrepWarp = 18;
// Registers a thread: 640 x 96 at launch = 256 x 120 + 128 x 112 + 256 x 64.
constexpr int kPRegs = 96, kPSoftRegs = 120, kPAccRegs = 112, kPRestRegs = 64;
static_assert(256 * kPSoftRegs + 128 * kPAccRegs + 256 * kPRestRegs <= kPThreads * kPRegs, "register split");
// What a unit costs beside its blocks, in blocks (us at 0, 2, 4, 6: a 20-node
// tree x 32 heads over 1024 keys 20.1, 16.1, 16.1, 16.9; 64 requests of one
// token, 64 heads on 8, up to 3000 keys 81.7, 80.5, 78.6, 76.8; 32 requests x 16
// nodes x 32 heads over 2048 keys 141, 144, 143, 142).
// Groups of two or three blocks cost more cut than whole: 13 requests of up to 45
// nodes over up to 144 keys 22 us without, 26 with.
constexpr PPad kPPad{4, 4};
constexpr float kPEven = 16.f, kPApart = 40.f;  // of V's scales: see the softmax
constexpr int kBarSoft = 1;       // and 2: one per softmax warpgroup
constexpr int kBarAcc = 3, kBarFirst = 4;

template <int D, int R>
struct PCfg {
  static constexpr int kTile = kPBlock * D;                 // K tile
  static constexpr int kVTile = kPBlock * 128;              // 128 d; the upper half stays zero when D = 64
  // K tiles go as soon as S is there; V tiles wait for their step's P, so more
  // of them are needed for the same bytes in flight.
  static constexpr int kKStages = D == 64 ? 6 : R == 64 ? 3 : 4;
  static constexpr int kVStages = R == 16 ? 6 : 5;
  static constexpr int kPB = R == 64 ? 1 : 2;               // P buffers (of two blocks)
  static constexpr int kNS = R == 64 ? 2 : 4;               // S buffers (of two blocks)
  static constexpr int kQ = R * D;                          // one term of a Q tile
  static constexpr int kOffK = 0;                                  // K ring
  static constexpr int kOffV = kOffK + kKStages * kTile;           // V ring
  static constexpr int kPRow = R == 64 ? 128 : 64;                 // bytes of a key's P: hi of every row, lo of every row
  static constexpr int kPTile = kPBlock * kPRow;
  static constexpr int kOffP = kOffV + kVStages * kVTile;          // [kPB][2 blocks]
  static constexpr int kOffQ = kOffP + 2 * kPB * kPTile;                 // [2][hi, lo]
  static constexpr int kOffDesc = kOffQ + 4 * kQ;                  // u32 [2][256 keys][2]: rows that see the tree key
  static constexpr int kOffPoison = kOffDesc + 2 * 256 * 8;        // u64 [2][128 d]: rows that see a NaN there
  static constexpr int kOffCum = kOffPoison + 2 * 128 * 8;         // i64 [TSV_MAX_BATCH + 1]
  static constexpr int kOffReq = kOffCum + 8 * (TSV_MAX_BATCH + 2);  // int4 [TSV_MAX_BATCH]: off, n, P, blocks
  static constexpr int kOffFr = kOffReq + 16 * TSV_MAX_BATCH;      // f32 [2][R]: score factor of a row
  static constexpr int kOffRow = kOffFr + 8 * R;                   // i32 [2][R]: output row
  static constexpr int RW = R < 32 ? R : 32;                       // rows of one softmax group
  static constexpr bool kCols = R == 64;                           // the groups split the rows, not the blocks
  static constexpr int kOffWmax = kOffRow + 8 * R;                 // f32 [2 groups][2][4 warps][RW]
  static constexpr int kOffPw = kOffWmax + 64 * RW;                // f32 [8 warps][3][RW]: -maxima, sum factors, rescale
  static constexpr int kOffM = kOffPw + 96 * RW;                   // f32 [4][R]: a block's largest scores
  static constexpr int kOffAB = kOffM + 16 * R;                     // f32 [4 warps][2][R]: accumulation factors
  static constexpr int kOffL = kOffAB + 32 * R;                    // f32 [2][8 warps][RW]
  static constexpr int kOffMw = kOffL + 64 * RW;                   // f32 [2][2 groups][RW]
  static constexpr int kOffFin = kOffMw + 16 * RW;                 // f32 [2][R]: sums of a unit
  static constexpr int kOffUnit = kOffFin + 8 * R;                 // PUnit [2]
  static constexpr int kOffFirst = kOffUnit + 128;                 // PUnit, then i64 [4]: x0, x1, blocks, CTAs
  static constexpr int kOffScale = kOffFirst + 96;                 // f32 [V stages][20]: (K, V) of 8 pages, V's largest and smallest
  static constexpr int kOffSv = kOffScale + kVStages * 80;         // f32 [4]
  static constexpr int kOffBar = kOffSv + 16;
  // k_full, k_empty, v_full, v_empty, sc_full (per stage), s_full[4], p_full[4], o_full[2], o_free[2], q_full[2], unit_free[2],
  // l_full[2], d_full[2], mma_done[2]
  static constexpr int kBars = 2 * kKStages + 3 * kVStages + 22;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kSmem = kOffMisc + 64 + 1024;
  static constexpr int kO = kNS * 2 * R;                           // first column of O: S is [kNS][2 blocks][R], O [2][2 R]
  static constexpr uint32_t kTmem = R == 16 ? 256 : 512;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kTile % 1024 == 0 && kQ % 512 == 0 && kOffQ % 1024 == 0, "swizzle atoms");
};

// Swizzled position of 16-byte chunk c of row r in a tile of ROW-byte rows.
template <int ROW>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return ROW == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Issued by the whole warp: the one lane with `lead` set issues the MMA.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// The bits that any lane has set, in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }
// Instruction descriptor of kind::f8f6f4: e4m3 A and B (format 0), fp32 D.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Descriptor of a tile with 128- or 64-byte rows, swizzled over its rows' width.
template <int ROW>
__device__ __forceinline__ uint64_t sdesc_row(uint32_t saddr, uint32_t lbo) {
  uint64_t d = sdesc_sw128(saddr, lbo, 8 * ROW);
  if (ROW == 64) d = (d & ~(7ull << 61)) | (4ull << 61);
  return d;
}

// 16 lanes x 256 bits, repeated over R columns: thread t holds, of lanes t / 4
// and t / 4 + 8, columns 8 i + 2 (t % 4) and the next, in v[4 i ..] (two of the
// first lane, two of the second).  Does not wait.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// Waits for this thread's TMEM loads and ties registers to the wait.
template <int N>
__device__ __forceinline__ void tmem_wait_tie(uint32_t (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i])::"memory");
}
template <int N>
__device__ __forceinline__ void tmem_tie(uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i])::"memory");
}

// 32 lanes x 32 bits, 16 consecutive columns per thread; does not wait.
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The same with 8 columns.
__device__ __forceinline__ void tmem_ld8_nowait(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

template <int D, int R>
__global__ void __launch_bounds__(kPThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                      const __grid_constant__ PagedAttnArgs a, int32_t* words,
                      float* __restrict__ part_o, float* __restrict__ part_ml) {
  using C = PCfg<D, R>;
  constexpr int SK = C::kKStages, SV = C::kVStages, NS = C::kNS;
  int32_t* counters = words + TSV_MAX_BATCH;  // (the first words: requests that a wait was given up for)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  uint8_t* sP = smem + C::kOffP;
  uint8_t* sQ = smem + C::kOffQ;
  uint32_t* sDesc = reinterpret_cast<uint32_t*>(smem + C::kOffDesc);
  unsigned long long* sPoison = reinterpret_cast<unsigned long long*>(smem + C::kOffPoison);
  int64_t* sCum = reinterpret_cast<int64_t*>(smem + C::kOffCum);
  int4* sReq = reinterpret_cast<int4*>(smem + C::kOffReq);
  float* sFr = reinterpret_cast<float*>(smem + C::kOffFr);
  int32_t* sRow = reinterpret_cast<int32_t*>(smem + C::kOffRow);
  float* sWmax = reinterpret_cast<float*>(smem + C::kOffWmax);
  float* sPw = reinterpret_cast<float*>(smem + C::kOffPw);
  float* sM = reinterpret_cast<float*>(smem + C::kOffM);
  float* sAB = reinterpret_cast<float*>(smem + C::kOffAB);
  float* sL = reinterpret_cast<float*>(smem + C::kOffL);
  float* sMw = reinterpret_cast<float*>(smem + C::kOffMw);
  float* sFin = reinterpret_cast<float*>(smem + C::kOffFin);
  PUnit* sUnit = reinterpret_cast<PUnit*>(smem + C::kOffUnit);
  PUnit* sFirst = reinterpret_cast<PUnit*>(smem + C::kOffFirst);
  int64_t* sRange = reinterpret_cast<int64_t*>(smem + C::kOffFirst + 64);
  float* sScale = reinterpret_cast<float*>(smem + C::kOffScale);
  float* sSv = reinterpret_cast<float*>(smem + C::kOffSv);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_empty = k_full + SK;
  uint64_t* v_full = k_empty + SK;
  uint64_t* v_empty = v_full + SV;
  uint64_t* sc_full = v_empty + SV;  // a block's scales are in
  uint64_t* s_full = sc_full + SV;
  uint64_t* p_full = s_full + 4;
  uint64_t* o_full = p_full + 4;
  uint64_t* o_free = o_full + 2;
  uint64_t* q_full = o_free + 2;
  uint64_t* unit_free = q_full + 2;
  uint64_t* l_full = unit_free + 2;
  uint64_t* d_full = l_full + 2;  // a unit's tree mask is in
  uint64_t* mma_done = d_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  int* abort_flag = reinterpret_cast<int*>(smem + C::kOffMisc + 4);
  int* sPoisoned = reinterpret_cast<int*>(smem + C::kOffMisc + 8);   // [2]
  int* sJoin = reinterpret_cast<int*>(smem + C::kOffMisc + 16);
  volatile int* abort_v = abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lps = __ffs(a.cache.page_size) - 1;  // pages are powers of two
  const bool tree = a.tree_table.ids_d != nullptr;
  bool dead = false;

  if (tid == 0) {
    for (int s = 0; s < SK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
      mbar_init(&sc_full[s], 1);
    }
    for (int x = 0; x < 4; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], C::kCols ? 256 : 128);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&o_full[x], 1);
      mbar_init(&o_free[x], 128);
      mbar_init(&q_full[x], 64);
      mbar_init(&d_full[x], 64);
      mbar_init(&unit_free[x], 128);
      mbar_init(&l_full[x], 256);
    }
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    *abort_flag = 0;
    sPoisoned[0] = sPoisoned[1] = 0;
    mbar_fence_init();
  }
  if (warp == kPSWarp) {
    tmem_alloc(tmem_slot, C::kTmem);
    tmem_relinquish();
  }
  if (warp == kPProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  if (D == 64) {  // the upper half of every V stage stays zero
    for (int i = tid; i < SV * (C::kVTile / 2 / 16); i += kPThreads) {
      const int st = i / (C::kVTile / 2 / 16), o = i % (C::kVTile / 2 / 16);
      reinterpret_cast<uint4*>(sV + st * C::kVTile + C::kVTile / 2)[o] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  if (tid < 256) sPoison[tid] = 0ull;
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();

  if (warp == 0) plist_setup(a, R, kPPad, sCum, sReq, sFirst, sRange);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const PList list{sCum, sReq, a.B, a.G, a.cache.Hkv, R, kPPad, tree, sRange[1]};

  // Rows r_lo .. r_lo + count - 1 of a unit's tile (one warp): their output
  // rows, score factors and two e4m3 terms.
  auto prep_rows = [&](const PUnit& u, int buf, int r_lo, int count) {
    constexpr int E = D / 32;  // elements of a row per lane
    constexpr int kBatch = 8;  // rows loaded together
    const int row0 = u.tile * R;
    const int rows = min(R, u.n * a.G - row0);
    // Row r of the tile: node (row0 + r) / G, query head g G + (row0 + r) % G.
    // Lane i knows row r_lo + i.
    int64_t at_q = 0;
    if (lane < count) {
      const int r = r_lo + lane;
      const int gr = row0 + r;
      const int node = gr / a.G;
      const int head = u.g * a.G + (gr - node * a.G);
      sRow[buf * R + r] = r < rows ? (u.off + node) * a.Hq + head : -1;
      if (r < rows) at_q = (int64_t)(u.off + node) * a.qs_n + (int64_t)head * a.qs_h;
    }
    uint8_t* hi = sQ + buf * 2 * C::kQ;
    uint8_t* lo = hi + C::kQ;
#pragma unroll 1
    for (int r0 = 0; r0 < count; r0 += kBatch) {
      uint32_t raw[kBatch][E / 2];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (r0 + i >= count) break;
        const int64_t at = __shfl_sync(0xffffffffu, at_q, r0 + i);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) raw[i][e] = 0u;
        if (r_lo + r0 + i < rows) {
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + at + lane * E;
          if constexpr (E == 4) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(src));
            raw[i][0] = w.x;
            raw[i][1] = w.y;
          } else {
            raw[i][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (r0 + i >= count) break;
        const int r = r_lo + r0 + i;
        uint32_t top = 0u;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) top = max(top, max((raw[i][e] << 16) & 0x7FFF0000u, raw[i][e] & 0x7FFF0000u));
        top = __reduce_max_sync(0xffffffffu, top);
        const bool fine = top < 0x7F800000u;  // no infinity, no NaN in the row
        // The largest value moves to [128, 256): exponent 134 as biased.
        const int up = top == 0u ? 0 : max(-120, min(120, 134 - (int)(top >> 23)));
        const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
        if (lane == 0) sFr[buf * R + r] = __uint_as_float((uint32_t)(127 - up) << 23) * (a.scale * 1.4426950408889634f);
        uint32_t wh = 0u, wl = 0u;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          // A row with an infinity or a NaN is NaN throughout (its scores are).
          const float y0 = fine ? __uint_as_float(raw[i][e] << 16) * mul : NAN;
          const float y1 = fine ? __uint_as_float(raw[i][e] & 0xFFFF0000u) * mul : NAN;
          const uint32_t h2 = e4m3x2(y0, y1), f2 = f16x2_of_e4m3x2(h2);
          wh |= h2 << (16 * e);
          wl |= e4m3x2(y0 - f16_lo(f2), y1 - f16_hi(f2)) << (16 * e);
        }
        const uint32_t at = swz<D>(r, lane * E / 16) + (lane * E) % 16;
        if constexpr (E == 4) {
          *reinterpret_cast<uint32_t*>(hi + at) = wh;
          *reinterpret_cast<uint32_t*>(lo + at) = wl;
        } else {
          *reinterpret_cast<uint16_t*>(hi + at) = (uint16_t)wh;
          *reinterpret_cast<uint16_t*>(lo + at) = (uint16_t)wl;
        }
      }
    }
    fence_proxy_async_smem();
  };
  // The first unit's rows: every warp but the producers, which start the
  // copies meanwhile.
  if (sFirst->valid && (warp < kPProducerWarp || warp >= kPSWarp)) {
    const int w = warp < kPProducerWarp ? warp : warp - 4;
    prep_rows(*sFirst, 0, w * (R / 16), R / 16);
    named_bar_sync(kBarFirst, 512);
  }

  if (warp >= kPProducerWarp && warp < kPSWarp) {
    // ------------------------------------------------------------ producers of K and of V
    setmaxnreg_dec<kPRestRegs>();
    const bool is_v = warp >= kPProducerWarp + 2;
    const int odd = warp & 1;  // this warp's blocks
    const CUtensorMap* tmap = is_v ? &tmap_v : &tmap_k;
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    uint8_t* ring = is_v ? sV : sK;
    const int tile = is_v ? C::kVTile : C::kTile, stages = is_v ? SV : SK;
    // The lanes stand for the pages of the next 32 / per blocks, per pages to
    // a block: lane i holds page i % per of block i / per of its chunk.  Page ids
    // of the next chunk are loaded as a chunk begins, their scales after its
    // first block.
    const int per = kPBlock >> lps, chunk = 32 >> (7 - lps);  // pages of a block, blocks of a chunk
    const int mine = lane >> (7 - lps), pg = lane & (per - 1);
    struct Look {
      int id, pages, g, tiles;  // id -1: no keys in this lane's page
    };
    PUnit u = *sFirst;  // the unit and block of this lane's page
    auto advance = [&](int n) {
      while (u.valid && n > 0) {
        const int left = u.j1 - u.j;
        if (n < left) {
          u.j += n;
          return;
        }
        n -= left;
        list.next(u);
      }
    };
    auto look_id = [&](Look& k) {
      k.id = -1;
      k.pages = 0;
      k.g = u.g;
      k.tiles = u.tiles;
      if (!u.valid) return;
      const bool main = u.j < u.nmain;
      const int block = main ? u.j : u.j - u.nmain;
      const int keys = (main ? u.P : tree ? u.n : 0) - block * kPBlock;
      k.pages = (max(0, min(keys, kPBlock)) + (1 << lps) - 1) >> lps;
      const tsv_page_table& pt = main ? a.table : a.tree_table;
      if (pg < k.pages) k.id = __ldg(pt.ids_d + (int64_t)u.b * pt.stride + block * per + pg);
    };
    // V's producer brings both scales: V's stage is held until the block is done,
    // so whoever waits for them sees this phase of their barrier (K's goes on).
    auto look_scale = [&](const Look& k) {
      float2 s = make_float2(0.f, 0.f);
      if (is_v && (uint32_t)k.id < (uint32_t)a.cache.num_pages) {
        const int64_t at = (int64_t)k.id * a.cache.Hkv + k.g;
        s = make_float2(__ldg(a.cache.k_scale_d + at), __ldg(a.cache.v_scale_d + at));
      }
      return s;
    };
    Look c0{-1, 0, 0, 0}, c1;
    float2 sc0 = make_float2(0.f, 0.f), sc1 = sc0;
    float top = 0.f, low = 0.f;  // of the lane's block: V's largest scale, and the smallest
    const int blocks = __shfl_sync(0xffffffffu, (int)sRange[0], 0);
    int st = odd, ph = 0;  // of this warp's next block: ring stage and phase
    // Chunk t is issued (c0) while the ids of the next one (c1) are looked up,
    // at its first block, and its scales, at its second.
#pragma unroll 1
    for (int t = -chunk;; t += chunk) {
      advance(t < 0 ? mine : chunk);
      look_id(c1);
#pragma unroll 1
      for (int i = odd; t >= 0 && i < chunk && t + i < blocks; i += 2) {  // this warp's blocks of the chunk
        if (t + i >= stages) TSV_PWAIT(&empty[st], ph ^ 1);
        if (__any_sync(0xffffffffu, dead)) break;
        const int src = i << (7 - lps);
        const bool mine_now = mine == i;
        // Pages, whether several row tiles read them (then they stay in L2), head.
        const uint32_t what = uniform(mine_now ? (uint32_t)c0.pages | (c0.tiles > 1 ? 0x100u : 0u) | ((uint32_t)c0.g << 16) : 0u);
        const uint32_t pages = what & 0xFFu, g = what >> 16;
        const uint64_t pol = (what & 0x100u) ? l2_policy_evict_last() : l2_policy_evict_first();
        const uint32_t at = smem_u32(ring) + (uint32_t)(st * tile), bar = smem_u32(&full[st]);
        const bool lead = elect_one();
        if (pages > 0 && lead) mbar_expect_tx(&full[st], (uint32_t)((pages << lps) * D));
#pragma unroll 1
        for (uint32_t p = 0; p < pages; ++p) {
          const uint32_t id = __shfl_sync(0xffffffffu, (uint32_t)c0.id, src + (int)p);
          tma_load_page(at + (p << lps) * D, tmap, bar, g, id, pol, lead);
        }
        if (is_v && i == odd) {  // (the copies of the first block go before the wait for its scales)
          top = sc0.y;
          low = c0.id >= 0 ? sc0.y : INFINITY;
          for (int o = per >> 1; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
          }
        }
        if (is_v && mine_now) {
          float* sc = sScale + st * 20;
          *reinterpret_cast<float2*>(sc + 2 * pg) = sc0;
          if (pg == 0) *reinterpret_cast<float2*>(sc + 16) = make_float2(top, low);
        }
        __syncwarp();
        if (lead) {
          mbar_arrive(&full[st]);
          if (is_v) mbar_arrive(&sc_full[st]);
        }
        st += 2;
        if (st >= stages) {
          st -= stages;
          ph ^= 1;
        }
        if (i == odd + 2) sc1 = look_scale(c1);
      }
      if (__any_sync(0xffffffffu, dead) || t + chunk >= blocks) break;
      if (t < 0) sc1 = look_scale(c1);
      c0 = c1;
      sc0 = sc1;
    }
    // Every copy has landed before the CTA leaves (whatever the other roles did).
    for (int x = max(0, blocks - stages); x < blocks; ++x)
      if ((x & 1) == odd) mbar_wait(&full[x % stages], (x / stages) & 1, nullptr);
  } else if (warp == kPSWarp) {
    // ------------------------------------------------------------ issuer of S
    setmaxnreg_dec<kPRestRegs>();
    // S of step t needs its unit's Q, the blocks' K, and its buffer: the softmax
    // of step t - NS has read it.
    const uint64_t dK0 = sdesc_row<D>(smem_u32(sK), 16);
    const uint64_t dQ0 = sdesc_row<D>(smem_u32(sQ), 16);
    const uint32_t idS = idesc_e4m3(kPBlock, R, 0, 0);
    int t = 0, st = 0, ph = 0;
    for (int k = 0; !dead; ++k) {
      TSV_PWAIT(&q_full[k & 1], k >> 1);
      const PUnit& u = sUnit[k & 1];
      const int blocks = __shfl_sync(0xffffffffu, u.valid ? u.j1 - u.j : 0, 0);
      if (blocks == 0) break;
      const uint32_t dq = (uint32_t)dQ0 + (uint32_t)((k & 1) * (2 * C::kQ >> 4));
      for (int i = 0; i < blocks; ++i) {
        if ((i & 1) == 0 && t >= NS) TSV_PWAIT(&p_full[(t - NS) & 3], (t - NS) >> 2);
        TSV_PWAIT(&k_full[st], ph);
        if (__any_sync(0xffffffffu, dead)) break;
        tc_fence_after();
        const bool last = (i & 1) || i + 1 == blocks;
        const bool lead = elect_one();
        const uint32_t dk = (uint32_t)dK0 + (uint32_t)(st * (C::kTile >> 4));
        const uint32_t dst = tmem + (uint32_t)((t % NS) * 2 * R + (i & 1) * R);
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            umma_e4m3(dst, desc_at(dK0, dk + kk * 2), desc_at(dQ0, dq + term * (C::kQ >> 4) + kk * 2), idS, term + kk > 0 ? 1u : 0u, lead);
        if (lead) {
          umma_commit(&k_empty[st]);
          if (last) umma_commit(&s_full[t & 3]);
        }
        __syncwarp();
        if (last) ++t;
        if (++st == SK) {
          st = 0;
          ph ^= 1;
        }
      }
      dead = __any_sync(0xffffffffu, dead);
    }
    if (elect_one()) umma_commit(&mma_done[0]);
    __syncwarp();
    mbar_wait(&mma_done[0], 0, nullptr);
  } else if (warp == kPOWarp) {
    // ------------------------------------------------------------ issuer of O
    setmaxnreg_dec<kPRestRegs>();
    // O of step t needs P, the blocks' V and its own buffer: the accumulating
    // group has read step t - 2.
    const uint64_t dV0 = sdesc_row<D>(smem_u32(sV), kPBlock * 64);
    const uint64_t dP0 = sdesc_row<C::kPRow>(smem_u32(sP), kPBlock * 128);
    const uint32_t idO = idesc_e4m3(128, 2 * R, 1, 1);
    int t = 0, st = 0, ph = 0;
    for (int k = 0; !dead; ++k) {
      TSV_PWAIT(&q_full[k & 1], k >> 1);
      const PUnit& u = sUnit[k & 1];
      const int blocks = __shfl_sync(0xffffffffu, u.valid ? u.j1 - u.j : 0, 0);
      if (blocks == 0) break;
      const int u_j = u.j, u_P = u.P, u_n = u.n, nmain = u.nmain;
      for (int i = 0; i < blocks; ++i) {
        if ((i & 1) == 0) {
          if (t >= 2) TSV_PWAIT(&o_free[t & 1], (t >> 1) - 1);
          TSV_PWAIT(&p_full[t & 3], t >> 2);
        }
        TSV_PWAIT(&v_full[st], ph);
        if (__any_sync(0xffffffffu, dead)) break;
        tc_fence_after();
        const bool last = (i & 1) || i + 1 == blocks;
        const bool lead = elect_one();
        const uint32_t dv = (uint32_t)dV0 + (uint32_t)(st * (C::kVTile >> 4));
        const uint32_t dp = (uint32_t)dP0 + (uint32_t)(((t % C::kPB) * 2 + (i & 1)) * (C::kPTile >> 4));
        const uint32_t dst = tmem + (uint32_t)(C::kO + (t & 1) * 2 * R);
        const uint32_t more = (uint32_t)(i & 1);
        // The last blocks of the prefix and of the tree: only the 32-key slices
        // that hold keys (one at least, so that O is written).
        const int block = u_j + i;
        const int keys = (block < nmain ? u_P - block * kPBlock : tree ? u_n - (block - nmain) * kPBlock : 0);
#pragma unroll
        for (int kk = 0; kk < kPBlock / 32; ++kk) if (kk == 0 || 32 * kk < keys)
          umma_e4m3(dst, desc_at(dV0, dv + kk * (32 * D >> 4)), desc_at(dP0, dp + kk * (32 * C::kPRow >> 4)), idO, kk > 0 ? 1u : more, lead);
        if (lead) {
          umma_commit(&v_empty[st]);
          if (last) umma_commit(&o_full[t & 1]);
        }
        __syncwarp();
        if (last) ++t;
        if (++st == SV) {
          st = 0;
          ph ^= 1;
        }
      }
      dead = __any_sync(0xffffffffu, dead);
    }
    if (elect_one()) umma_commit(&mma_done[1]);
    __syncwarp();
    mbar_wait(&mma_done[1], 0, nullptr);
  } else if (warp >= kPPrepWarp) {
    // ------------------------------------------------------------ Q tiles and tree masks
    setmaxnreg_dec<kPRestRegs>();
    const int q = warp - kPPrepWarp;
    PUnit u = *sFirst;
    for (int k = 0;; ++k) {
      const int buf = k & 1;
      if (k >= 2) TSV_PWAIT(&unit_free[buf], (k >> 1) - 1);
      if (__any_sync(0xffffffffu, dead)) break;
      if (q == 0 && lane == 0) sUnit[buf] = u;  // what the other roles walk by
      if (!u.valid) {
        parrive(&q_full[buf], dead);
        break;
      }
      if (k > 0) prep_rows(u, buf, q * (R / 2), R / 2);
      parrive(&q_full[buf], dead);
      // Rows that see tree key j: word q of sDesc[buf][j] holds rows 32 q .. (two warps).
      if (tree && u.j1 > u.nmain) {
        const int r = q * 32 + lane;
        const bool has = r < min(R, u.n * a.G - u.tile * R);
        const int i0 = has ? (u.tile * R + r) / a.G : 0;  // the row's node
        for (int w = 0; w < (u.n + 31) / 32; ++w) {
          uint32_t bits = 0u;
          if (has) {
            const int left = i0 + 1 - 32 * w;
            bits = a.anc ? __ldg(a.anc + (int64_t)(u.off + i0) * TSV_ANC_WORDS + w)
                         : (left >= 32 ? 0xFFFFFFFFu : left > 0 ? (1u << left) - 1u : 0u);
          }
          uint32_t see = 0u;
#pragma unroll 1
          for (int i = 0; i < 32; ++i) {
            const uint32_t m = __ballot_sync(0xffffffffu, (bits >> i) & 1u);
            if (lane == i) see = m;
          }
          sDesc[(buf * 256 + w * 32 + lane) * 2 + q] = see;
        }
      }
      parrive(&d_full[buf], dead);
      list.next(u);
    }
    // Every request's lengths and page ids are checked by one CTA.
    for (int b = blockIdx.x; q == 0 && b < a.B; b += gridDim.x) {
      PagedRequest r;
      bool bad = !paged_request(a, b, &r);
      if (!bad) bad = paged_bad_page(a, b, r, lane, 32);
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) report_check(a, words, b, bad);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax: a thread owns a key
    setmaxnreg_inc<kPSoftRegs>();
    constexpr int RW = C::RW;
    constexpr bool kCols = C::kCols;
    const int wg = warp >> 2, lg = warp & 3;
    const int col0 = kCols ? wg * 32 : 0;      // this group's rows of the tile
    const int kt = tid & 127;                  // thread of the group = key lane
    const uint32_t lane_base = (uint32_t)(lg * 32) << 16;
    float* pw = sPw + warp * 3 * RW;
    int t = 0, st = 0, ph = 0, nth = 0;
    for (int k = 0;; ++k) {
      const int buf = k & 1;
      TSV_PWAIT(&q_full[buf], k >> 1);
      if (named_bar_or(kBarSoft + wg, 128, dead)) break;  // the same in every thread of the group
      const int u_j = sUnit[buf].j, u_j1 = sUnit[buf].j1, u_P = sUnit[buf].P, u_n = sUnit[buf].n, nmain = sUnit[buf].nmain;
      if (!sUnit[buf].valid) break;
      float lsum[RW];
#pragma unroll
      for (int i = 0; i < RW; ++i) lsum[i] = 0.f;
      float mw = -INFINITY;  // lane r < RW: largest score of row r over this group's blocks of the unit
      const float fr = lane < RW ? sFr[buf * R + col0 + lane] : 0.f;
      for (int j = u_j; j < u_j1; j += 2, ++t) {
        const int halves = min(2, u_j1 - j);
        const int st0 = st, ph0 = ph;
        for (int h = 0; h < halves; ++h)
          if (++st == SV) {
            st = 0;
            ph ^= 1;
          }
        if (!kCols && (t & 1) != wg) continue;
        const int st1 = st0 + 1 == SV ? 0 : st0 + 1, ph1 = st0 + 1 == SV ? ph0 ^ 1 : ph0;
        const uint32_t s_col = tmem + lane_base + (uint32_t)((t % NS) * 2 * R + col0);
        // Keys of block j + h: its first row, how many are valid, tree or prefix.
        auto block_base = [&](int h) { return (j + h < nmain ? j + h : j + h - nmain) * kPBlock; };
        auto block_valid = [&](int h) {
          return h >= halves ? 0 : max(0, min(kPBlock, (j + h < nmain ? u_P : tree ? u_n : 0) - block_base(h)));
        };
        const bool all = j + 2 <= u_j1 && (j + 2) * kPBlock <= u_P;  // two blocks that every row sees throughout
        ++nth;
        TSV_PWAIT(&s_full[t & 3], t >> 2);
        tc_fence_after();

        auto step = [&](auto all_c) {
          constexpr bool ALL = decltype(all_c)::value;  // no masks, and V's scales near each other (else: false)
          if (!ALL && j + halves > nmain) TSV_PWAIT(&d_full[buf], k >> 1);
          const int nh = ALL ? 2 : halves;
          // Rows (of this group) that see a key, one bit each.
          auto sees = [&](int h, int key) -> uint32_t {
            if (key >= block_valid(h)) return 0u;
            if (j + h < nmain) return 0xFFFFFFFFu;
            return sDesc[(buf * 256 + block_base(h) + key) * 2 + (kCols ? wg : 0)];
          };
          // Largest score of every row over the warp's 64 keys: of 16 keys a
          // thread holds 2 in 2 columns of 8; then three halving exchanges over
          // the 8 thread rows.  best[2 i + c] is column 8 i + 2 (lane % 4) + c.
          constexpr int N0 = RW / 4;
          float* wmax = sWmax + ((wg * 2 + (nth & 1)) * 4) * RW;
          auto maxima = [&](auto apart_c, float inv_top) {
            constexpr bool APART = decltype(apart_c)::value;
            float best[N0];
#pragma unroll
            for (int i = 0; i < N0; ++i) best[i] = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < nh; ++h) {
              uint32_t sa[RW / 2], sb[RW / 2];  // the warp's keys 0-15 and 16-31
              tmem_ld_16x256(s_col + h * R, sa);
              tmem_ld_16x256(s_col + h * R + (16u << 16), sb);
              TSV_PWAIT(&sc_full[h ? st1 : st0], h ? ph1 : ph0);
              const float2* sc = reinterpret_cast<const float2*>(sScale + (h ? st1 : st0) * 20);
              const float fa = sc[(lg * 32) >> lps].x, fb = sc[(lg * 32 + 16) >> lps].x;
              tmem_wait_tie(sa);
              tmem_tie(sb);
              if (!ALL) {
                const int key = lg * 32 + (lane >> 2);
                const int sh = 2 * (lane & 3);
                const uint32_t v0 = sees(h, key) >> sh, v1 = sees(h, key + 8) >> sh;
                const uint32_t v2 = sees(h, key + 16) >> sh, v3 = sees(h, key + 24) >> sh;
#pragma unroll
                for (int i = 0; i < RW / 8; ++i)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    if (!((v0 >> (8 * i + c)) & 1u)) sa[4 * i + c] = 0xFF800000u;
                    if (!((v1 >> (8 * i + c)) & 1u)) sa[4 * i + 2 + c] = 0xFF800000u;
                    if (!((v2 >> (8 * i + c)) & 1u)) sb[4 * i + c] = 0xFF800000u;
                    if (!((v3 >> (8 * i + c)) & 1u)) sb[4 * i + 2 + c] = 0xFF800000u;
                  }
              }
              if constexpr (APART) {
                const float la = fmaxf(__log2f(sc[(lg * 32) >> lps].y * inv_top), -kPApart);
                const float lb = fmaxf(__log2f(sc[(lg * 32 + 16) >> lps].y * inv_top), -kPApart);
#pragma unroll
                for (int i = 0; i < RW / 8; ++i) {
                  const float2 f2 = *reinterpret_cast<const float2*>(sFr + buf * R + col0 + 8 * i + 2 * (lane & 3));
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const float xa = fmaxf(__uint_as_float(sa[4 * i + c]), __uint_as_float(sa[4 * i + 2 + c])) * fa;
                    const float xb = fmaxf(__uint_as_float(sb[4 * i + c]), __uint_as_float(sb[4 * i + 2 + c])) * fb;
                    const float f = c ? f2.y : f2.x;
                    best[2 * i + c] = fmaxf(best[2 * i + c], fmaxf(fmaf(xa, f, la), fmaf(xb, f, lb)));
                  }
                }
              } else {
#pragma unroll
                for (int i = 0; i < RW / 8; ++i)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const float x = fmaxf(fmaxf(__uint_as_float(sa[4 * i + c]), __uint_as_float(sa[4 * i + 2 + c])) * fa,
                                          fmaxf(__uint_as_float(sb[4 * i + c]), __uint_as_float(sb[4 * i + 2 + c])) * fb);
                    best[2 * i + c] = fmaxf(best[2 * i + c], x);
                  }
              }
            }
            {
              int at = 0;  // first index that this thread is left with: the halvings pick its bits from the top
#pragma unroll
              for (int s = 0; s < 3; ++s) {
                const int half = (N0 >> s) / 2;  // values kept
                const int bit = 16 >> s;
                const bool up = lane & bit;
                if (half >= 1) {
#pragma unroll
                  for (int i = 0; i < (half > 0 ? half : 1); ++i) {
                    const float send = up ? best[i] : best[i + half];
                    const float keep = up ? best[i + half] : best[i];
                    best[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, bit));
                  }
                  at += up ? half : 0;
                } else {
                  best[0] = fmaxf(best[0], __shfl_xor_sync(0xffffffffu, best[0], bit));
                }
              }
              wmax[lg * RW + (at >> 1) * 8 + 2 * (lane & 3) + (at & 1)] = best[0];
            }
          };
          maxima(std::false_type{}, 0.f);
          // V's scales go to P relative to the step's largest (2^-126 at least: there
          // is none above 0 that the library writes below it).  Scales further apart
          // than kPEven: the rows' references are those of p times the scale (as far
          // as 2^-kPApart), so that a row which attends to a page of small values has
          // its bits there.
          const float2 v0 = *reinterpret_cast<const float2*>(sScale + st0 * 20 + 16);
          const float2 v1 = nh == 2 ? *reinterpret_cast<const float2*>(sScale + st1 * 20 + 16) : v0;
          const float top = fmaxf(fmaxf(v0.x, v1.x), 0x1p-126f);
          float inv_top;
          asm("rcp.approx.f32 %0, %1;" : "=f"(inv_top) : "f"(top));  // (of 2^127 too, unlike __fdividef)
          const bool apart = fminf(v0.y, v1.y) * kPEven < top;
          if (apart) {
            if (ALL) return false;
            maxima(std::true_type{}, inv_top);
          }
          named_bar_sync(kBarSoft + wg, 128);
          // Every warp works out the rows' maxima and factors for itself.
          float m = 0.f;
          bool moved = false;
          if (lane < RW) {
            m = fmaxf(fmaxf(wmax[lane], wmax[RW + lane]), fmaxf(wmax[2 * RW + lane], wmax[3 * RW + lane])) * (!ALL && apart ? 1.f : fr);
            if (!(m > -INFINITY)) m = -INFINITY;  // nothing seen, or NaN scores only: P is 0 or NaN
            const float mn = fmaxf(mw, m);
            // P takes 2^8 p (256 over the scale of a page of zeros, 2^-126, would be no
            // fp32 number), the sums p.
            pw[lane] = m == -INFINITY ? 0.f : 8.f - m;
            pw[RW + lane] = m == -INFINITY ? 1.f : fast_exp2(m - mn) * (1.f / 256.f);
            pw[2 * RW + lane] = mn == -INFINITY ? 1.f : mw == -INFINITY ? 0.f : fast_exp2(mw - mn);
            moved = mn != mw;
            mw = mn;
          }
          __syncwarp();
          // P's buffer is free once O of the step kPB before is there.  That
          // waited for the accumulating group to be through with a step at least
          // 3 back, so the group's copies of the maxima (4 deep) are free too.
          if (t >= C::kPB) TSV_PWAIT(&o_full[(t - C::kPB) & 1], (t - C::kPB) >> 1);
          if (lg == 0 && lane < RW) {
            sM[(t & 3) * R + col0 + lane] = m;
            if (lane == 0 && col0 == 0) sSv[t & 3] = top * (1.f / 256.f);
          }
          if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int i = 0; i < RW; i += 4) {
              const float4 al = *reinterpret_cast<const float4*>(pw + 2 * RW + i);
              lsum[i] *= al.x;
              lsum[i + 1] *= al.y;
              lsum[i + 2] *= al.z;
              lsum[i + 3] *= al.w;
            }
          }
#pragma unroll 1
          for (int h = 0; h < nh; ++h) {  // rolled, here and above: the loop's code is fetched once for both blocks
            // O reads the 32-key slices that hold keys (and the first): the
            // other warps have no P to write.
            if (!ALL && lg > 0 && lg * 32 >= block_valid(h)) continue;
            uint32_t sv2[2][16];  // this chunk of 16 rows and the next
            tmem_ld16_nowait(s_col + h * R, sv2[0]);
            const float2 mine = reinterpret_cast<const float2*>(sScale + (h ? st1 : st0) * 20)[kt >> lps];
            const uint32_t vis = ALL ? 0u : sees(h, kt);
            uint8_t* ptile = sP + ((t % C::kPB) * 2 + h) * C::kPTile;
            const uint64_t fk2 = f2_pack(mine.x, mine.x), fv2 = f2_pack(mine.y * inv_top, mine.y * inv_top);
#pragma unroll
            for (int c0 = 0; c0 < RW; c0 += 16) {
              uint32_t(&sv)[16] = sv2[(c0 >> 4) & 1];
              tmem_wait_tie(sv);
              if (c0 + 16 < RW) tmem_ld16_nowait(s_col + h * R + c0 + 16, sv2[((c0 >> 4) + 1) & 1]);
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                const ulonglong2 m4 = *reinterpret_cast<const ulonglong2*>(pw + c0 + 4 * q4);
                const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(pw + RW + c0 + 4 * q4);
                const ulonglong2 f4 = *reinterpret_cast<const ulonglong2*>(sFr + buf * R + col0 + c0 + 4 * q4);
                uint32_t hw = 0u, lw = 0u;
#pragma unroll
                for (int pr = 0; pr < 2; ++pr) {
                  const int r = c0 + 4 * q4 + 2 * pr;
                  const uint64_t s2 = (uint64_t)sv[4 * q4 + 2 * pr] | ((uint64_t)sv[4 * q4 + 2 * pr + 1] << 32);
                  // The same products as in the maximum: x <= 0 up to m's own rounding.
                  const uint64_t x2 = ffma2(fmul2(s2, fk2), pr ? f4.y : f4.x, pr ? m4.y : m4.x);
                  float p0 = fast_exp2(f2_lo(x2)), p1 = fast_exp2(f2_hi(x2));
                  if (!ALL) {
                    if (!((vis >> r) & 1u)) p0 = 0.f;
                    if (!((vis >> (r + 1)) & 1u)) p1 = 0.f;
                  }
                  uint64_t p2 = f2_pack(p0, p1);
                  const uint64_t l2 = ffma2(p2, pr ? b4.y : b4.x, f2_pack(lsum[r], lsum[r + 1]));
                  lsum[r] = f2_lo(l2);
                  lsum[r + 1] = f2_hi(l2);
                  p2 = fmul2(p2, fv2);
                  p0 = f2_lo(p2);
                  p1 = f2_hi(p2);
                  const uint32_t h2 = e4m3x2(p0, p1), g2 = f16x2_of_e4m3x2(h2);
                  hw |= h2 << (16 * pr);
                  lw |= e4m3x2(p0 - f16_lo(g2), p1 - f16_hi(g2)) << (16 * pr);
                }
                hi[q4] = hw;
                lo[q4] = lw;
              }
              *reinterpret_cast<uint4*>(ptile + swz<C::kPRow>(kt, (col0 + c0) / 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(ptile + swz<C::kPRow>(kt, (R + col0 + c0) / 16)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            if (!ALL && (!kCols || wg == 0)) {
              uint8_t* vrow = sV + (h ? st1 : st0) * C::kVTile + kt * D;
              TSV_PWAIT(&v_full[h ? st1 : st0], h ? ph1 : ph0);
              if (kt >= block_valid(h)) {  // whatever the row holds
#pragma unroll
                for (int c = 0; c < D / 16; ++c)  // (a lane starts at its own chunk: no bank conflicts)
                  reinterpret_cast<uint4*>(vrow)[(c + kt) % (D / 16)] = make_uint4(0u, 0u, 0u, 0u);
              } else if (j + h >= nmain) {
                uint32_t any = 0u;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  const uint4 w = reinterpret_cast<const uint4*>(vrow)[(c + kt) % (D / 16)];
                  any |= ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
                         ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
                }
                any &= 0x80808080u;
                const uint32_t* see = sDesc + (buf * 256 + block_base(h) + kt) * 2;
                const unsigned long long rows = (unsigned long long)see[0] | (R > 32 ? (unsigned long long)see[1] << 32 : 0ull);
#pragma unroll 1
                for (int c = 0; any && c < D / 4; ++c) {
                  const uint32_t w = reinterpret_cast<const uint32_t*>(vrow)[c];
                  uint32_t nan = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                  if (nan == 0u) continue;
                  reinterpret_cast<uint32_t*>(vrow)[c] = w & ~((nan >> 7) * 0xFFu);
                  const int chunk = D == 128 ? (c >> 2) ^ (kt & 7) : (c >> 2) ^ ((kt >> 1) & 3);
                  for (; nan; nan &= nan - 1)
                    atomicOr(sPoison + buf * 128 + chunk * 16 + (c & 3) * 4 + ((__ffs(nan) - 1) >> 3), rows);
                  sPoisoned[buf] = 1;
                }
              }
            }
          }
          return true;
        };
        if (!all || !step(std::true_type{})) step(std::false_type{});
        fence_proxy_async_smem();
        tc_fence_before();
        parrive(&p_full[t & 3], dead);
      }
      // Sums of P over the warp's keys (transposed reduction), and their reference.
      if (k >= 2) TSV_PWAIT(&unit_free[buf], (k >> 1) - 1);
      {
        int first = 0;  // row that this thread is left with
#pragma unroll
        for (int s = 0; s < 5; ++s) {
          const int half = (RW >> s) / 2;
          const int bit = 16 >> s;
          const bool up = lane & bit;
          if (half >= 1) {
#pragma unroll
            for (int i = 0; i < (half > 0 ? half : 1); ++i) {
              const float send = up ? lsum[i] : lsum[i + half];
              const float keep = up ? lsum[i + half] : lsum[i];
              lsum[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
            }
            first += up ? half : 0;
          } else {
            lsum[0] += __shfl_xor_sync(0xffffffffu, lsum[0], bit);
          }
        }
        sL[(buf * 8 + warp) * RW + first] = lsum[0];
        if (lg == 0 && lane < RW) sMw[(buf * 2 + wg) * RW + lane] = mw;
      }
      parrive(&l_full[buf], dead);
    }
  } else {
    // ------------------------------------------------------------ accumulation: a thread owns a d
    setmaxnreg_inc<kPAccRegs>();
    const int d = tid & 127, lg = warp & 3;
    const uint32_t lane_base = (uint32_t)(lg * 32) << 16;
    const bool live = d < D;
    int t = 0;
    for (int k = 0;; ++k) {
      const int buf = k & 1;
      TSV_PWAIT(&q_full[buf], k >> 1);
      if (named_bar_or(kBarAcc, 128, dead)) break;  // the same in every thread of the group
      const PUnit& u = sUnit[buf];
      if (!u.valid) break;
      const int u_j = u.j, u_j1 = u.j1;
      uint64_t acc[R / 2];  // rows 2 i and 2 i + 1
#pragma unroll
      for (int i = 0; i < R / 2; ++i) acc[i] = 0ull;
      constexpr int kPer = (R + 31) / 32;  // rows of a lane: lane, lane + 32
      float mt[kPer];                      // their running maxima (each warp keeps its own copy)
#pragma unroll
      for (int i = 0; i < kPer; ++i) mt[i] = -INFINITY;
      float* ab = sAB + lg * 2 * R;        // this warp's factors: rescale, weight of the block
      for (int j = u_j; j < u_j1; j += 2, ++t) {
        const int x = t & 1, x4 = t & 3;
        TSV_PWAIT(&p_full[x4], t >> 2);
        const float sv = sSv[x4];
        bool moved = false;
        __syncwarp();  // the last block's factors have been read
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = lane + 32 * i;
          if (r < R) {
            const float m = sM[x4 * R + r];
            const float mn = fmaxf(mt[i], m);
            ab[r] = mn == -INFINITY ? 1.f : mt[i] == -INFINITY ? 0.f : fast_exp2(mt[i] - mn);
            ab[R + r] = sv * (m == -INFINITY ? 1.f : fast_exp2(m - mn));  // no maximum: P is 0 or NaN
            moved = moved || mn != mt[i];
            mt[i] = mn;
          }
        }
        __syncwarp();
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < R / 2; i += 2) {
            const ulonglong2 al = *reinterpret_cast<const ulonglong2*>(ab + 2 * i);
            acc[i] = fmul2(acc[i], al.x);
            acc[i + 1] = fmul2(acc[i + 1], al.y);
          }
        }
        TSV_PWAIT(&o_full[x], t >> 1);
        tc_fence_after();
        const uint32_t o_col = tmem + lane_base + (uint32_t)(C::kO + x * 2 * R);
        uint32_t h2[2][8], l2[2][8];  // hi and lo of this chunk of 8 rows and the next
        tmem_ld8_nowait(o_col, h2[0]);
        tmem_ld8_nowait(o_col + R, l2[0]);
#pragma unroll
        for (int c0 = 0; c0 < R; c0 += 8) {
          uint32_t(&h)[8] = h2[(c0 >> 3) & 1];
          uint32_t(&l)[8] = l2[(c0 >> 3) & 1];
          tmem_wait_tie(h);
          tmem_tie(l);
          if (c0 + 8 < R) {
            tmem_ld8_nowait(o_col + c0 + 8, h2[((c0 >> 3) + 1) & 1]);
            tmem_ld8_nowait(o_col + R + c0 + 8, l2[((c0 >> 3) + 1) & 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const ulonglong2 be = *reinterpret_cast<const ulonglong2*>(ab + R + c0 + 2 * i);
            const int q = c0 / 2 + i;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint64_t sum = fadd2((uint64_t)h[2 * (i + y)] | ((uint64_t)h[2 * (i + y) + 1] << 32),
                                         (uint64_t)l[2 * (i + y)] | ((uint64_t)l[2 * (i + y) + 1] << 32));
              acc[q + y] = ffma2(sum, y ? be.y : be.x, acc[q + y]);
            }
          }
        }
        tc_fence_before();
        parrive(&o_free[x], dead);
      }
      // The unit is done: denominators, then its rows or its partials.
      TSV_PWAIT(&l_full[buf], k >> 1);
      float* fin = sFin + buf * R;
      if (lg == 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = lane + 32 * i;
          if (r >= R) continue;
          float l = 0.f;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (C::kCols && w != i) continue;  // the group that had the row
            const int rr = C::kCols ? lane : r;
            const float mw = sMw[(buf * 2 + w) * C::RW + rr];
            const float* lw = sL + (buf * 8 + 4 * w) * C::RW + rr;
            const float sum = (lw[0] + lw[C::RW]) + (lw[2 * C::RW] + lw[3 * C::RW]);
            l += mw == -INFINITY ? sum : sum * fast_exp2(mw - mt[i]);
          }
          // A whole group needs the reciprocal (0 for a row that sees nothing).
          fin[r] = !u.whole() ? l : l == 0.f ? 0.f : 1.f / l;
        }
      }
      float* of = reinterpret_cast<float*>(acc);
      if (sPoisoned[buf]) {
        const unsigned long long rows = sPoison[buf * 128 + d];
#pragma unroll
        for (int r = 0; r < R; ++r)
          if ((rows >> r) & 1ull) of[r] = NAN;
        sPoison[buf * 128 + d] = 0ull;
      }
      const bool stop = named_bar_or(kBarAcc, 128, dead);  // the same in every thread
      if (d == 0) sPoisoned[buf] = 0;
      const int rows = min(R, u.n * a.G - u.tile * R);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
      if (u.whole()) {
        __nv_bfloat16* od = out + d;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < rows && live) od[(int64_t)sRow[buf * R + r] * D] = __float2bfloat16_rn(of[r] * fin[r]);
      } else if (!stop) {
        const int slot = 2 * (int)blockIdx.x + (k == 0 ? 0 : 1);
        float* po = part_o + (int64_t)slot * R * D;
        float* pm = part_ml + (int64_t)slot * 2 * R;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < rows && live) po[r * D + d] = of[r];
        if (lg == 0) {
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < R) pm[lane + 32 * i] = mt[i];
        }
        if (d < R) pm[R + d] = fin[d];
        // CTAs cf .. cl share the group; the last to arrive joins.
        const int64_t W = sRange[2], ctas = sRange[3];
        const int64_t g0 = u.gx + list.pad.of(u.T);  // the place of its first block
        const int cf = (int)(((g0 + 1) * ctas - 1) / W), cl = (int)(((g0 + u.T) * ctas - 1) / W);
        named_bar_sync(kBarAcc, 128);
        if (d == 0) {
          const int n = atom_add_acq_rel_gpu(counters + cf, 1);
          const bool last = n == cl - cf;
          if (last) counters[cf] = 0;
          *sJoin = last ? 1 : 0;
        }
        named_bar_sync(kBarAcc, 128);
        if (*sJoin) {
          const int first_slot = (int64_t)cf * W / ctas >= u.gx ? 0 : 1;  // the group is its first unit, or its last
          join_partials<D, R>(part_o, part_ml, cf, cl, first_slot, rows, sRow + buf * R, out, lg, 4, lane);
        }
      }
      parrive(&unit_free[buf], dead);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_v)
    for (PUnit u = *sFirst; u.valid; list.next(u)) report_timeout(a, words, u.b);
  if (warp == kPSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

template <int D, int R>
cudaError_t launch_typed(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int grid, void* ws,
                         cudaStream_t st) {
  char* w = static_cast<char*>(ws);
  const PagedAttnLayout lay = paged_attn_layout(grid, R, D);
  return launch_pdl(paged_attn_kernel<D, R>, dim3(grid), dim3(kPThreads), (size_t)PCfg<D, R>::kSmem, st, 0u, tk, tv, a,
                    reinterpret_cast<int32_t*>(w), reinterpret_cast<float*>(w + lay.part_o),
                    reinterpret_cast<float*>(w + lay.part_ml));
}

template <int D, int R>
cudaError_t set_typed() {
  // The register split draws on what the block is launched with.
  cudaFuncAttributes attr;
  const cudaError_t e = cudaFuncGetAttributes(&attr, paged_attn_kernel<D, R>);
  if (e != cudaSuccess) return e;
  if (attr.numRegs < kPRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(paged_attn_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, PCfg<D, R>::kSmem);
}

}  // namespace

cudaError_t paged_attention_set_attributes(int32_t D, int32_t R) {
  if (D == 64) return R == 16 ? set_typed<64, 16>() : R == 32 ? set_typed<64, 32>() : set_typed<64, 64>();
  return R == 16 ? set_typed<128, 16>() : R == 32 ? set_typed<128, 32>() : set_typed<128, 64>();
}

cudaError_t launch_paged_attention(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int32_t R, int grid,
                                   void* ws, cudaStream_t st) {
  if (a.cache.D == 64)
    return R == 16   ? launch_typed<64, 16>(tk, tv, a, grid, ws, st)
           : R == 32 ? launch_typed<64, 32>(tk, tv, a, grid, ws, st)
                     : launch_typed<64, 64>(tk, tv, a, grid, ws, st);
  return R == 16   ? launch_typed<128, 16>(tk, tv, a, grid, ws, st)
         : R == 32 ? launch_typed<128, 32>(tk, tv, a, grid, ws, st)
                   : launch_typed<128, 64>(tk, tv, a, grid, ws, st);
}

}  // namespace tsv
