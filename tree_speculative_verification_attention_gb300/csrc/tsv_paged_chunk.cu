// tsv_paged_chunk.cu — causal attention of chunks of new tokens over a paged
// 8-bit cache, bf16 rows on the tensor cores.
//
//   S = (Qh + Ql) K^T   M = 128 rows, N = 128 keys, K = D   (e4m3; A = Q, B = K, shared memory)
//   O += P V            M = 128 rows, N = D, K = 128 keys   (fp16; A = P, TMEM; B = V, shared memory)
//
// Rows of a tile are (token, query head of the KV head) pairs, token by token, so
// a KV head's codes are read once for all heads that share it.  K's codes are an
// operand as they lie in the cache: TMA brings a page's rows of a head into the
// swizzled tile.  A row of q is two e4m3 terms under a power of two that moves
// its largest value to [128, 256): a bf16's 8 bits exactly down to 2^-17 of it,
// at the price of one fp16 product, since e4m3 products run at twice the rate.
// V is widened to fp16 (exactly) so that P keeps fp16's 11 bits: P is 2^8 p
// times 2^e of the V scale of its page relative to the unit's largest so far,
// m 2^e, where p is relative to a reference maximum that moves only when a score
// passes it by 2^7 (moving costs a wait for the products and a pass over O: with 2^4
// and 2^11 a chunk of 1024 tokens behind 8192 took 1.06 times as long).  2^e is part
// of the exponent of p and goes out of the row's sum again (a factor per 16 keys); m,
// 1 for scales that are powers of two, goes into V as it is widened.
//
// Work.  Units of up to 256 rows (two tiles) of a KV head and the 128-key blocks
// that any of their rows sees form one list, which is cut into equal ranges, one
// per CTA (one CTA per SM); the lengths are read from the device.  A unit that a
// cut goes through leaves fp32 partials, which a second launch joins.
// Roles (16 warps) run on their own through all units of the range, tied by
// barriers on the buffers alone, so that a unit's end overlaps the next one's
// beginning:
//   0-7    softmax, a thread per row (0-3 tile 0, 4-7 tile 1): they bring their
//          tile's next Q in before they wait for the last product
//   8-11   widening of V, and NaN codes of blocks with masked keys taken out
//   12, 13 MMA issuers of the tiles.  A tile's scores are two buffers of 64 keys, and
//          P lies over its scores: S of a half goes out behind PV of the same half of
//          the block before, under the softmax of the other half and the other tile
//   14, 15 producers of K and of V with the pages' scales
//
// What bounds it: the chain softmax - issuer - tensor cores - softmax of a half, whose
// links wait for one another more than any unit is busy.  A block of 256 rows takes
// 3700 cycles; of those the tensor cores have 2048 to do (an e4m3 product of two
// terms and an fp16 one), the softmax warps 2600 (two on a scheduler), and shared
// memory moves 336 KB, 2700 at 128 bytes a cycle, 128 KB of it Q, which every product
// of 64 keys reads again (TMEM is full of S and O).  Measured: 1024 tokens
// behind 8192, 64 query heads on 8, D = 128: 244 us, 183 with the
// arithmetic and most of the products taken out; 4096 behind 28672: 3.0 ms, 1.37
// PFLOP/s, 0.71 of a large bf16 product's rate.  Short chunks are bound by the way to
// the first score (2 us of list, 4 of Q and the first tiles) and back (1.5 of the
// unit's end, 4 of the second launch): 512 tokens from the start, 32 heads on 8: 21 us.
// A softmax that looks at a block's sum and not at its maximum, two halves in
// registers at once, and two warps on the halves of one tile were no faster.
#include <type_traits>

#include "tsv_paged_tc.cuh"

namespace tsv {

namespace {

constexpr int kCThreads = 512;
constexpr int kCConvWarp = 8, kCMmaWarp = 12, kCKWarp = 14, kCVWarp = 15;
// Registers a thread: 512 x 128 at launch = 256 x 144 + 256 x 112.  (Nothing may
// spill: beside so much shared memory the L1 holds next to nothing.)
constexpr int kCSoftRegs = 144, kCRestRegs = 112;
static_assert(256 * kCSoftRegs + 256 * kCRestRegs <= kCThreads * 128, "register split");
constexpr int kTileRows = 128;
constexpr int kKStages = 3;
constexpr float kRise = 7.f;    // log2: how far a score may pass the reference maximum
constexpr float kUp = 8.f;      // log2 of P's factor: 2^7 x 2^8 is within fp16
constexpr int kFarApart = 40;   // log2: V scales that far apart leave a row's weights their bits
// What a unit costs beside its blocks, in blocks; and how near to a unit's end a cut may come.
constexpr int kUnitCost = 5, kLeastCut = 6, kNearEnd = 2;
constexpr uint32_t kCWaitTries = 1024;  // of a wait before it looks at the clock, too (0.3 to 1.4 us each)
constexpr int kBarConv = 1;
constexpr int kScaleRow = 36;   // of a block, per 16 keys: K's scale, e and 2^-e and m of V's relative scale m 2^e; V's largest scale, whether every m is 1
constexpr int kNanSlots = 6;    // blocks of a unit with masked keys: 3 at each end

// A unit, and the part of it in the CTA's range.
struct CUnit {
  int b, tile, g;
  int off, n, start, tiles;  // of the request
  int row0, rows;
  int first, end;            // blocks of the unit
  int j, j1;                 // and those of this part
  __device__ __forceinline__ bool whole() const { return j == first && j1 == end; }
};

// n / d of 0 <= n < 2^31 by a product: with 2^l >= d, m = 2^(31 + l) / d rounded up is
// too large by less than d / d <= 2^l / d, which n x does not carry to the next quotient.
struct Divisor {
  uint32_t m;
  int shift;
  explicit Divisor(int d) {
    int l = 0;
    while (((int64_t)1 << l) < d) ++l;
    shift = 31 + l;
    m = (uint32_t)((((uint64_t)1 << shift) + d - 1) / d);
  }
  __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> shift); }
};

struct ChunkGeometry {
  Divisor by_heads;  // query heads of a KV head
  int R, window;
  // Blocks that rows r0 .. r1 of request (start) see: first, end.
  __device__ __forceinline__ int2 blocks(int start, int r0, int r1) const {
    const int p0 = start + by_heads.of(r0), p1 = start + by_heads.of(r1);
    const int lo = window > 0 ? max(0, p0 - window + 1) : 0;
    return make_int2(lo / kPBlock, p1 / kPBlock + 1);
  }
};

template <int D>
struct CCfg {
  static constexpr int kQTile = kTileRows * D;       // one term of a Q tile
  static constexpr int kKTile = kPBlock * D;         // codes of a block
  static constexpr int kVTile = kPBlock * D * 2;
  static constexpr int kOffQ = 0;                                   // [tile][hi, lo]
  static constexpr int kOffK = kOffQ + 4 * kQTile;                  // ring of codes
  static constexpr int kOffRaw = kOffK + kKStages * kKTile;         // V's codes
  static constexpr int kOffV = kOffRaw + 2 * kKTile;                // V in fp16
  static constexpr int kOffReq = kOffV + 2 * kVTile;                // int4 [TSV_MAX_BATCH]: off, n, start, tiles
  static constexpr int kOffTiles = kOffReq + 16 * TSV_MAX_BATCH;    // i32 [TSV_MAX_BATCH + 4]: tiles of the requests before
  static constexpr int kOffPre = kOffTiles + 4 * (TSV_MAX_BATCH + 4);  // i64 [17 + 3]
  static constexpr int kOffFr = kOffPre + 8 * 20;                   // f32 [256]: score factor of a row
  static constexpr int kOffScale = kOffFr + 4 * 256;                // f32 [4][kScaleRow]
  static constexpr int kOffNan = kOffScale + 16 * kScaleRow;               // u32 [2][kNanSlots][4]
  static constexpr int kOffCut = kOffNan + 2 * kNanSlots * 16;      // i32 [2][4]: f, g, j of the range's ends
  // k_full[3], k_empty[3], raw_full[2], raw_empty[2], v_full[2], v_empty[2], sc_full[4], s_full[4], p_full[4], pv_done[4],
  // q_full[2], mma_done
  static constexpr int kOffBar = kOffCut + 32;
  static constexpr int kBars = 2 * kKStages + 27;
  static constexpr int kOffMisc = kOffBar + 8 * kBars + 8;
  static constexpr int kSmem = kOffMisc + 64 + 1024;
  static constexpr uint32_t kColO = 2 * kPBlock;  // S0 | S1 | O0 | O1
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kOffPre % 16 == 0 && kOffScale % 16 == 0 && kOffBar % 8 == 0, "alignment");
};

// What a CTA did of groups that others share, for the launch that joins them.
struct alignas(16) ChunkPart {
  int empty, cont, through, lead;  // first unit continues a group (and goes on in the next CTA); the last one begins a cut group
  int off, row0, rows, g;          // of the group that is begun
};

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// e4m3 (kind::f8f6f4) or fp16 (kind::f16) A and B, fp32 D; A K-major, B K-major (0) or N-major (1).
__host__ __device__ constexpr uint32_t idesc_mn(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
template <int ROW>
__device__ __forceinline__ uint64_t sdesc_row(uint32_t saddr, uint32_t lbo) {
  uint64_t d = sdesc_sw128(saddr, lbo, 8 * ROW);
  if (ROW == 64) d = (d & ~(7ull << 61)) | (4ull << 61);
  return d;
}
// Position of 16-byte chunk c of row r in a swizzled tile of ROW-byte rows.
template <int ROW>
__device__ __forceinline__ int swizzled(int r, int c) {
  return ROW == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two fp16 values -> two e4m3 codes, nearest even; the difference of fp16 pairs.
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_minus(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Bytes that are NaN codes, as their top bits.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// As pwait, without a time that the hardware holds the thread for: warps that
// wait here wait shortly (2 % of a long chunk).  But for the softmax warps of a tile that
// sits units out, which wait for as long as those take: a wait is given up when for
// kWaitLimitNs K's producer has asked for no block (abort[1]: the time when it last did,
// the lower 32 bits of ns; it may be later than the clock that was read here).
__device__ __forceinline__ void cwait(uint64_t* bar, uint32_t parity, volatile int* abort, bool& dead) {
#pragma unroll 1
  for (uint32_t n = 0; !mbar_try_wait(bar, parity & 1u); ++n)
    if (dead || *abort || (n >= kCWaitTries && (int)((uint32_t)global_timer_ns() - (uint32_t)abort[1]) > (int)kWaitLimitNs)) {
      *abort = 1;
      dead = true;
      break;
    }
  __syncwarp();
}
// A wait after which the whole warp knows whether it is dead.
#define TSV_CWAIT(bar, parity)                                    \
  do {                                                            \
    cwait((bar), (uint32_t)(parity), abort_v, dead);              \
    dead = __any_sync(0xffffffffu, dead);                         \
  } while (0)

template <int D>
__global__ void __launch_bounds__(kCThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const __grid_constant__ PagedAttnArgs a, const ChunkGeometry geo, int32_t* timeouts, ChunkPart* __restrict__ parts,
                       float* __restrict__ part_o, float* __restrict__ part_ml) {
  using C = CCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sRaw = smem + C::kOffRaw;
  uint8_t* sV = smem + C::kOffV;
  int4* sReq = reinterpret_cast<int4*>(smem + C::kOffReq);
  int32_t* sTiles = reinterpret_cast<int32_t*>(smem + C::kOffTiles);
  int64_t* sPre = reinterpret_cast<int64_t*>(smem + C::kOffPre);
  float* sFr = reinterpret_cast<float*>(smem + C::kOffFr);
  float* sScale = reinterpret_cast<float*>(smem + C::kOffScale);
  uint32_t* sNan = reinterpret_cast<uint32_t*>(smem + C::kOffNan);
  int32_t* sCut = reinterpret_cast<int32_t*>(smem + C::kOffCut);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_empty = k_full + kKStages;
  uint64_t* raw_full = k_empty + kKStages;
  uint64_t* raw_empty = raw_full + 2;
  uint64_t* v_full = raw_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* sc_full = v_empty + 2;   // scales of a block
  uint64_t* s_full = sc_full + 4;    // [tile][half]
  uint64_t* p_full = s_full + 4;     // [tile][half]
  uint64_t* pv_done = p_full + 4;   // [tile][half]
  uint64_t* q_full = pv_done + 4;    // [tile]
  uint64_t* mma_done = q_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  int* abort_flag = reinterpret_cast<int*>(smem + C::kOffMisc + 4);
  volatile int* abort_v = abort_flag;
  volatile int* units_done = reinterpret_cast<int*>(smem + C::kOffMisc + 16);  // [8]: of the softmax warps

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lps = __ffs(a.cache.page_size) - 1;  // pages are powers of two
  const int R = geo.R;
  const int Hkv = a.cache.Hkv;
  bool dead = false;

  if (tid == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);  // both tiles' issuers
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);  // the widening warps
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 2);
      mbar_init(&q_full[s], 4);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sc_full[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    for (int w = 0; w < 8; ++w) units_done[w] = 0;
    mbar_fence_init();
  }
  if (warp == kCMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();

  // ------------------------------------------------------------ the list and this CTA's range
  if (warp == 0) {
    int before = 0;
    if (lane == 0) sTiles[0] = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      int tiles = 0;
      PagedRequest r;
      if (b < a.B && paged_request(a, b, &r) && r.n >= a.least) {
        tiles = (int)(((int64_t)r.n * a.G + R - 1) / R);
        sReq[b] = make_int4(r.off, r.n, r.P - r.n, tiles);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, tiles, o);
        if (lane >= o) tiles += y;
      }
      sTiles[b + 1] = before + tiles;
      before += __shfl_sync(0xffffffffu, tiles, 31);
    }
  }
  if (tid < 8) sCut[tid] = tid & 3 ? 0 : INT32_MAX;  // behind all tiles
  __syncthreads();
  auto request_of = [&](int f) {  // the request that owns tile f of all
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sTiles[mid + 1] > f) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  };
  auto tile_blocks = [&](int b, int tile) {
    const int4 q = sReq[b];
    const int r0 = tile * R, r1 = (int)(min((int64_t)r0 + R, (int64_t)q.y * a.G) - 1);
    return geo.blocks(q.z, r0, r1);
  };
  const int all_tiles = sTiles[(a.B + 31) & ~31];
  const int share = (all_tiles + kCThreads - 1) / kCThreads, f_lo = min(all_tiles, tid * share), f_hi = min(all_tiles, f_lo + share);
  int64_t mine = 0;
  for (int f = f_lo, b = f < f_hi ? request_of(f) : 0; f < f_hi; ++f) {
    while (sTiles[b + 1] <= f) ++b;
    const int2 t = tile_blocks(b, f - sTiles[b]);
    mine += t.y - t.x + kUnitCost;
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sPre[warp + 1] = upto;
  __syncthreads();
  int64_t begin = upto - mine, total = lane < kCThreads / 32 ? sPre[lane + 1] : 0;
#pragma unroll
  for (int o = 1; o < kCThreads / 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, total, o);
    if (lane >= o) total += y;
  }
  if (warp > 0) begin += __shfl_sync(0xffffffffu, total, warp - 1);
  total = __shfl_sync(0xffffffffu, total, kCThreads / 32 - 1);
  begin *= Hkv;
  total *= Hkv;
  {
    const int64_t ctas = gridDim.x;
    const bool small = total < (1 << 21);  // 32-bit products and quotients (at most 1024 CTAs)
    const int64_t x[2] = {small ? (uint32_t)total * blockIdx.x / gridDim.x : total * blockIdx.x / ctas,
                          small ? (uint32_t)total * (blockIdx.x + 1) / gridDim.x : total * (blockIdx.x + 1) / ctas};
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      if (mine == 0 || x[e] < begin || x[e] >= begin + mine * Hkv) continue;
      int64_t at = begin;
      int f = f_lo, b = request_of(f);
      int2 t = tile_blocks(b, f - sTiles[b]);
      while (x[e] >= at + (int64_t)(t.y - t.x + kUnitCost) * Hkv) {
        at += (int64_t)(t.y - t.x + kUnitCost) * Hkv;
        ++f;
        while (sTiles[b + 1] <= f) ++b;
        t = tile_blocks(b, f - sTiles[b]);
      }
      const int T = t.y - t.x;
      int g = small ? (int)((uint32_t)(x[e] - at) / (uint32_t)(T + kUnitCost)) : (int)((x[e] - at) / (T + kUnitCost));
      int j = max(0, (int)(x[e] - at - (int64_t)g * (T + kUnitCost)) - kUnitCost);
      // Short units stay whole, and no part is short.
      if (T < kLeastCut) j = 2 * j < T ? 0 : T;
      else if (j < kNearEnd) j = 0;
      else if (T - j < kNearEnd) j = T;
      if (j == T) {
        j = 0;
        if (++g == Hkv) {
          g = 0;
          ++f;
        }
      }
      sCut[4 * e] = f;
      sCut[4 * e + 1] = g;
      sCut[4 * e + 2] = j;
    }
  }
  if (tid == 0) abort_v[1] = (int)(uint32_t)global_timer_ns();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The units of the range, for every role by itself.
  struct Cut {
    int f, g, j;
  };
  // (Read where they are wanted: registers that lie idle through the blocks are better used.)
  auto cut = [&](int e) {
    const volatile int32_t* c = sCut + 4 * e;
    return Cut{c[0], c[1], c[2]};
  };
  auto tiles_of_all = [&] { return *static_cast<const volatile int32_t*>(sTiles + ((a.B + 31) & ~31)); };
  auto fill_unit = [&](CUnit& u) {  // g, tile and b are set
    const int4 q = sReq[u.b];
    u.off = q.x;
    u.n = q.y;
    u.start = q.z;
    u.tiles = q.w;
    u.row0 = u.tile * R;
    u.rows = (int)min((int64_t)R, (int64_t)u.n * a.G - u.row0);
    const int2 t = geo.blocks(u.start, u.row0, u.row0 + u.rows - 1);
    u.first = t.x;
    u.end = t.y;
  };
  auto load_unit = [&](CUnit& u, int f) {
    const Cut to = cut(1);
    fill_unit(u);
    u.j = u.first;
    u.j1 = f == to.f && u.g == to.g ? u.first + to.j : u.end;
  };
  auto first_unit = [&](CUnit& u) {
    const Cut from = cut(0), to = cut(1);
    if (from.f >= tiles_of_all() || (from.f == to.f && from.g == to.g && from.j == to.j)) return false;
    u.b = request_of(from.f);
    u.tile = from.f - sTiles[u.b];
    u.g = from.g;
    load_unit(u, from.f);
    u.j = u.first + from.j;
    return true;
  };
  auto next_unit = [&](CUnit& u) {
    const Cut to = cut(1);
    if (++u.g == Hkv) {
      u.g = 0;
      if (++u.tile == u.tiles) {
        u.tile = 0;
        do ++u.b;
        while (u.b < a.B && sTiles[u.b + 1] == sTiles[u.b]);
      }
    }
    const int all = tiles_of_all(), f = u.b < a.B ? sTiles[u.b] + u.tile : all;
    if (f > to.f || (f == to.f && (u.g > to.g || (u.g == to.g && to.j == 0))) || f >= all) return false;
    load_unit(u, f);
    return true;
  };
  // Blocks of a tile among those of the part (none: both at its end).
  auto tile_range = [&](const CUnit& u, int q) {
    const int r0 = q * kTileRows, r1 = min(u.rows, r0 + kTileRows) - 1;
    int2 t = make_int2(u.j1, u.j1);
    if (r0 < u.rows) {
      const int2 x = geo.blocks(u.start, u.row0 + r0, u.row0 + r1);
      const int lo = max(u.j, x.x), hi = min(u.j1, x.y);
      if (lo < hi) t = make_int2(lo, hi);
    }
    return t;
  };
  // The blocks whose keys rows r0 .. r1 of the unit see all: from .x up to .y.
  auto full_range = [&](const CUnit& u, int r0, int r1) {
    const int p0 = u.start + geo.by_heads.of(u.row0 + r0), p1 = u.start + geo.by_heads.of(u.row0 + r1);
    return make_int2(a.window > 0 ? (max(p1 - a.window, -1) + kPBlock) / kPBlock : 0, (p0 + 1) / kPBlock);
  };
  CUnit u{};

  if (warp < kCConvWarp) {
    // ---------------------------------------------------------- softmax: a thread owns a row
    setmaxnreg_inc<kCSoftRegs>();
    const int tile = warp >> 2, r = tid & (kTileRows - 1), row = tile * kTileRows + r;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + (uint32_t)(tile * kPBlock);
    const uint32_t o_col = tmem + lane_base + C::kColO + (uint32_t)(tile * D);
    // The warp's rows of q, as two e4m3 terms each.
    auto bring_q = [&](const CUnit& v) {
      constexpr int kLanes = D / 8, kRows = 32 / kLanes, kPasses = 32 / kRows, kBatch = 8;
      int64_t at = -1;
      if (row < v.rows) {
        const int gr = v.row0 + row, token = geo.by_heads.of(gr);
        at = (int64_t)(v.off + token) * a.qs_n + (int64_t)(v.g * a.G + (gr - token * a.G)) * a.qs_h;
      }
      const int part = lane % kLanes, sub = lane / kLanes;
#pragma unroll 1
      for (int p0 = 0; p0 < kPasses; p0 += kBatch) {
        uint4 raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int64_t x = __shfl_sync(0xffffffffu, at, (p0 + i) * kRows + sub);
          raw[i] = make_uint4(0u, 0u, 0u, 0u);
          if (x >= 0) raw[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + x + part * 8));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int rr = (p0 + i) * kRows + sub;  // of the warp
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          // The row's largest value, two at a time: bf16 without sign as whole numbers.
          uint32_t two = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, o));
          const uint32_t top = max(two & 0xFFFFu, two >> 16) << 16;
          const bool fine = top < 0x7F800000u;  // a row with an infinity or a NaN is NaN throughout (its scores are)
          const int up = top == 0u ? 0 : max(-120, min(120, 134 - (int)(top >> 23)));
          const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // fp16 holds a bf16 under 2^8 down to 2^-17 of the row's largest, and what
            // e4m3 leaves of it.
            const uint32_t x2 = pack_f16(__uint_as_float(w[e] << 16) * mul, __uint_as_float(w[e] & 0xFFFF0000u) * mul);
            const uint32_t h = e4m3x2_of_f16x2(x2), l = e4m3x2_of_f16x2(f16x2_minus(x2, f16x2_of_e4m3x2(h)));
            if (e & 1) {
              hi[e >> 1] |= h << 16;
              lo[e >> 1] |= l << 16;
            } else {
              hi[e >> 1] = h;
              lo[e >> 1] = l;
            }
          }
          if (!fine) hi[0] = hi[1] = lo[0] = lo[1] = 0x7F7F7F7Fu;
          const int tr = (warp & 3) * 32 + rr;
          uint8_t* to_hi = sQ + tile * 2 * C::kQTile + swizzled<D>(tr, part >> 1) + 8 * (part & 1);
          *reinterpret_cast<uint2*>(to_hi) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to_hi + C::kQTile) = make_uint2(lo[0], lo[1]);
          if (part == 0) sFr[tile * kTileRows + tr] = __uint_as_float((uint32_t)(127 - up) << 23) * (a.scale * 1.4426950408889634f);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[tile]);
    };
    int t = 0, cnt = 0, units = 0;  // blocks and units of all roles, blocks of the tile
    auto takes_part = [&](const CUnit& v) {
      const int2 x = tile_range(v, tile);
      return x.x < x.y;
    };
    bool going = first_unit(u);
    if (going && takes_part(u)) bring_q(u);
    while (going) {
      const int2 range = tile_range(u, tile);
      const bool active = tile * kTileRows < u.rows;
      const float fr = sFr[row];
      const int pos = u.start + geo.by_heads.of(u.row0 + min(row, u.rows - 1));
      float m_ref = -INFINITY, l = 0.f, v_ref = 0.f;
      int room = kFarApart;  // how far the reference may still be lowered
      // P of 64 keys out of their scores.
      auto half_step = [&](int j, int h, bool masked, float alpha, const float* sc) {
        uint32_t s[2][32];
        tc_fence_after();
        tmem_ld32_nowait(s_col + 64 * h, s[0]);
        tmem_ld32_nowait(s_col + 64 * h + 32, s[1]);
        // Per 16 keys: the factor of the scores, V's exponent.
        float f[4], ex[4];
        *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(sc + 4 * h);
        *reinterpret_cast<float4*>(ex) = *reinterpret_cast<const float4*>(sc + 8 + 4 * h);
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = fmaxf(f[q] * fr, 0x1p-126f);  // (above 0: a masked key's -inf stays one)
        tmem_wait_ld_tie32(s[0]);
        reg_tie32(s[1]);
        if (__builtin_expect(masked, 0)) {
          const int hi = pos - j * kPBlock + 1 - 64 * h, lo = a.window > 0 ? hi - a.window : 0;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t see = bits_below(hi - 32 * c) & ~bits_below(lo - 32 * c);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) s[c][e] = 0xFF800000u;
          }
        }
        float top = -INFINITY;
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
          top = fmaxf(top, fmaf(fmaxf(b0, b1), f[q], ex[q]));
        }
        if (top > m_ref + kRise) {
          const float c = fast_exp2(m_ref - top);  // 0 when m_ref = -inf
          m_ref = top;
          l *= c;
          alpha *= c;
        }
        const float base = m_ref == -INFINITY ? kUp : kUp - m_ref;
        const float4 back = *reinterpret_cast<const float4*>(sc + 16 + 4 * h);  // 2^-exponent
        const float un[4] = {back.x, back.y, back.z, back.w};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int q = 2 * c; q < 2 * c + 2; ++q) {
            const uint64_t ref2 = f2_pack(base + ex[q], base + ex[q]), f2 = f2_pack(f[q], f[q]);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const int k = (q & 1) * 16 + e;
              const uint64_t x2 = ffma2((uint64_t)s[c][k] | ((uint64_t)s[c][k + 1] << 32), f2, ref2);
              const uint64_t w2 = f2_pack(fast_exp2(f2_lo(x2)), fast_exp2(f2_hi(x2)));
              if (e < 4) sum[e >> 1] = w2;
              else sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], w2);
              p[(q & 1) * 8 + (e >> 1)] = pack_f16(f2_lo(w2), f2_hi(w2));
            }
            const uint64_t both = fadd2(sum[0], sum[1]);
            l = fmaf(f2_lo(both) + f2_hi(both), un[q], l);
          }
          tmem_st16u_nowait(s_col + 64 * h + 16 * c, p);
        }
        // O moves only now, with the scores gone from registers: in front of P the copies
        // that this block forced, run or not, cost a long chunk 12 %.
        if (__builtin_expect(j + h > range.x && __any_sync(0xffffffffu, alpha != 1.f), 0)) {
          if (h == 0) TSV_CWAIT(&pv_done[2 * tile + 1], cnt - 1);
          else TSV_CWAIT(&pv_done[2 * tile], cnt);
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            float o[32];
            tmem_ld32(o_col + cc, o);
            uint32_t z16[2][16];
#pragma unroll
            for (int e = 0; e < 32; ++e) z16[e >> 4][e & 15] = __float_as_uint(o[e] * alpha);
            tmem_st16u_nowait(o_col + cc, z16[0]);
            tmem_st16u_nowait(o_col + cc + 16, z16[1]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        dead = __any_sync(0xffffffffu, dead);
        if (lane == 0 && !dead) mbar_arrive(&p_full[2 * tile + h]);
      };
      // Across the blocks the unit is four registers; what follows from them comes again.
      uint32_t who = (uint32_t)u.b | ((uint32_t)u.tile << 8);  // (fewer than 2^24 tiles: 128 rows of 2^31)
      int who_g = u.g;
      const int from_j = u.j, to_j = u.j1, x0 = t - from_j;
      if (range.x < range.y) {
        const int r0 = tile * kTileRows, r1 = min(u.rows, r0 + kTileRows) - 1;
        const int2 full = full_range(u, r0, r1);
#pragma unroll 1
        for (int j = range.x; j < range.y && !dead; ++j) {
          const int x = x0 + j;
          const bool masked = j < full.x || j >= full.y;
          cwait(&s_full[2 * tile], (uint32_t)cnt, abort_v, dead);
          // (Behind s_full: a tile that sits units out is far ahead of the scales' phases.)
          cwait(&sc_full[x & 3], (uint32_t)(x >> 2), abort_v, dead);
          const float* sc = sScale + (x & 3) * kScaleRow;
          const float v_top = sc[32];
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
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (h == 1) cwait(&s_full[2 * tile + 1], (uint32_t)cnt, abort_v, dead);
            half_step(j, h, masked, h == 0 ? alpha : 1.f, sc);
          }
          ++cnt;
        }
      }
      asm volatile("" : "+r"(who), "+r"(who_g));
      u.b = (int)(who & 255u);
      u.tile = (int)(who >> 8);
      u.g = who_g;
      fill_unit(u);
      u.j = from_j;
      u.j1 = to_j;
      const CUnit now = u;
      going = next_unit(u);
      if (dead) break;
      if (going && takes_part(u)) bring_q(u);  // (the tile's last S is there: Q is free)
      if (active) {
        if (range.x < range.y) TSV_CWAIT(&pv_done[2 * tile + 1], cnt - 1);
        if (dead) break;
        tc_fence_after();
        const int gr = now.row0 + row, token = geo.by_heads.of(gr);
        // Columns of a row whose NaN codes were kept out of the product.
        uint32_t bad[D / 32];
#pragma unroll
        for (int q = 0; q < D / 32; ++q) bad[q] = 0u;
        const uint32_t* nan = sNan + (units & 1) * (kNanSlots * 4);
        if (__any_sync(0xffffffffu, lane < kNanSlots * 4 && nan[lane] != 0u) && row < now.rows) {
#pragma unroll 1
          for (int w = 0; w < kNanSlots * 4; ++w) {
            const int slot = w >> 2, jb = slot < 3 ? now.first + slot : now.end - 1 - (slot - 3);
            uint32_t seen = nan[w];
            if (seen == 0u) continue;
            const int base = jb * kPBlock + 32 * (w & 3);
            seen &= bits_below(pos - base + 1) & (a.window > 0 ? ~bits_below(pos - base + 1 - a.window) : ~0u);
#pragma unroll 1
            for (; seen; seen &= seen - 1) {
              const int key = base + __ffs(seen) - 1;
              const int id = __ldg(a.table.ids_d + (int64_t)now.b * a.table.stride + (key >> lps));
              if ((uint32_t)id >= (uint32_t)a.cache.num_pages) continue;
              const uint32_t* v = reinterpret_cast<const uint32_t*>(
                  static_cast<const uint8_t*>(a.cache.v_d) + (int64_t)id * a.cache.stride_page +
                  (int64_t)(key & ((1 << lps) - 1)) * a.cache.stride_row + (int64_t)now.g * a.cache.stride_head);
#pragma unroll
              for (int e = 0; e < D / 4; ++e) {
                const uint32_t m = nan_bytes(__ldg(v + e)) >> 7;  // bits 0, 8, 16, 24
                bad[e >> 3] |= ((m | (m >> 7) | (m >> 14) | (m >> 21)) & 15u) << (4 * (e & 7));
              }
            }
          }
        }
        // (v_ref may be 2^-126, a page of zeros', or little more: then it is a factor of its own.)
        const bool none = range.x >= range.y || l == 0.f, tiny = v_ref < 0x1p-60f;
        const float inv = none ? 0.f : 1.f / l * (tiny ? 1.f : v_ref);
        const bool whole = now.whole();
        const int slot = 2 * (int)blockIdx.x + (now.j > now.first ? 0 : 1);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                             ((int64_t)(now.off + token) * a.Hq + now.g * a.G + (gr - token * a.G)) * D;
        float* po = part_o + ((int64_t)slot * kPagedWideRows + row) * D;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          float o[32];
          tmem_ld32(o_col + cc, o);
          if (row >= now.rows) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * inv;
          if (tiny) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= v_ref;
          }
          uint32_t nans = bad[0];
#pragma unroll
          for (int q = 1; q < D / 32; ++q)
            if (cc == 32 * q) nans = bad[q];
          if (nans) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((nans >> e) & 1u) o[e] = NAN;
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(out + cc + e) = make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                                                                   pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(po + cc + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (!whole && row < now.rows) {  // normalised: its sum is 1
          float* pm = part_ml + (int64_t)slot * 2 * kPagedWideRows;
          pm[row] = none ? -INFINITY : l > 0.f ? m_ref + log2f(l) : m_ref;
          pm[kPagedWideRows + row] = none ? 0.f : l > 0.f ? 1.f : l;
        }
        tc_fence_before();
      }
      t += now.j1 - now.j;
      ++units;
      __syncwarp();
      if (lane == 0) units_done[warp] = units;  // (a warp whose tile sits units out may be far ahead)
    }
  } else {
    setmaxnreg_dec<kCRestRegs>();
    if (warp < kCMmaWarp) {
      // -------------------------------------------------------- V, widened
      const int ct = tid - kCConvWarp * 32;
      constexpr int kLanes = D / 16, kStep = 128 / kLanes, kParts = kPBlock / kStep;  // lanes of a row; rows of a thread
      // Eight lanes take four 16-code chunks of two rows: their stores meet 32 banks.
      const int chunk = D == 128 ? (ct & 3) | ((ct >> 1) & 4) : ct & 3;
      const int first_row = D == 128 ? ((ct >> 2) & 1) | ((ct >> 4) << 1) : ct >> 2;
      int t = 0, units = 0;
      for (bool going = first_unit(u); going; going = next_unit(u)) {
        const int par = units & 1;
        // The rows of the unit before last, which had these words, are done with them.
        for (uint64_t t0 = 0; !__all_sync(0xffffffffu, lane >= 8 || units_done[lane & 7] >= units - 1);) {
          const uint64_t now = global_timer_ns();
          if (t0 == 0) t0 = now;
          if (__any_sync(0xffffffffu, *abort_v != 0 || now - t0 > kWaitLimitNs)) {
            *abort_v = 1;
            dead = true;
            break;
          }
        }
        if (ct < kNanSlots * 4) sNan[par * (kNanSlots * 4) + ct] = 0u;
        dead = named_bar_or(kBarConv, 128, dead);
        if (dead) break;
        const int2 full = full_range(u, 0, u.rows - 1);
        const int keys = u.start + min(u.n, geo.by_heads.of(u.row0 + u.rows - 1) + 1);  // behind the last one that a row sees
#pragma unroll 1
        for (int j = u.j; j < u.j1; ++j) {
          const int x = t + j - u.j, st = x & 1, valid = keys - j * kPBlock;
          TSV_CWAIT(&raw_full[st], x >> 1);
          TSV_CWAIT(&sc_full[x & 3], x >> 2);
          if (x >= 2) TSV_CWAIT(&v_empty[st], (x >> 1) - 1);
          if (dead) break;
          const float* sc = sScale + (x & 3) * kScaleRow;
          const bool plain = sc[33] != 0.f;
          const bool masked = j < full.x || j >= full.y;
          const int slot = j - u.first < 3 ? j - u.first : u.end - 1 - j < 3 ? 3 + u.end - 1 - j : 0;
#pragma unroll 1
          for (int h = 0; h < kParts; h += 2) {
            uint4 codes[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int key = first_row + (h + q) * kStep;
              codes[q] = make_uint4(0u, 0u, 0u, 0u);
              if (key < valid) codes[q] = *reinterpret_cast<const uint4*>(sRaw + st * C::kKTile + swizzled<D>(key, chunk));
            }
            if (masked) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t* v = reinterpret_cast<uint32_t*>(&codes[q]);
                uint32_t any = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t bad = nan_bytes(v[e]);
                  any |= bad;
                  v[e] &= ~((bad >> 7) * 0xFFu);
                }
                const int key = first_row + (h + q) * kStep;
                if (any) atomicOr(&sNan[par * (kNanSlots * 4) + slot * 4 + (key >> 5)], 1u << (key & 31));
              }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int key = first_row + (h + q) * kStep;
              const uint4 c = codes[q];
              uint8_t* to_row = sV + st * C::kVTile + (chunk >> 2) * (kPBlock * 128) + key * 128;
              const int at = (((2 * chunk) & 7) ^ (key & 7)) << 4;  // chunk 2 c of 8 values, and its neighbour
              uint32_t v[8] = {f16x2_of_e4m3x2(c.x & 0xFFFFu), f16x2_of_e4m3x2(c.x >> 16), f16x2_of_e4m3x2(c.y & 0xFFFFu),
                               f16x2_of_e4m3x2(c.y >> 16),     f16x2_of_e4m3x2(c.z & 0xFFFFu), f16x2_of_e4m3x2(c.z >> 16),
                               f16x2_of_e4m3x2(c.w & 0xFFFFu), f16x2_of_e4m3x2(c.w >> 16)};
              if (!plain) {  // rounded to fp16's 11 bits, as P is
                const float m = sc[24 + (key >> 4)];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = pack_f16(f16_lo(v[e]) * m, f16_hi(v[e]) * m);
              }
              *reinterpret_cast<uint4*>(to_row + at) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(to_row + (at ^ 16)) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v_full[st]);
            mbar_arrive(&raw_empty[st]);
          }
        }
        t += u.j1 - u.j;
        ++units;
      }
    } else if (warp < kCKWarp) {
      // -------------------------------------------------------- issuer of a tile
      const int q = warp - kCMmaWarp;
      constexpr uint32_t idS = idesc_mn(kTileRows, 64, 0), idPV = idesc_mn(kTileRows, D, 1);
      const uint64_t dq = sdesc_row<D>(smem_u32(sQ + q * 2 * C::kQTile), 16);
      const uint64_t dk = sdesc_row<D>(smem_u32(sK), 16);
      const uint64_t dv = sdesc_sw128(smem_u32(sV), kPBlock * 128, 1024);
      const uint32_t s_at = tmem + (uint32_t)(q * kPBlock), o_at = tmem + C::kColO + (uint32_t)(q * D);
      // The whole warp waits, one thread issues: behind elect.sync the compiler knows
      // that it is one, and the operands stay in uniform registers (behind a test of
      // the lane a long chunk took 1.13 times as long).
      int t = 0, cnt = 0, mine_units = 0;
      for (bool going = first_unit(u); going && !dead; going = next_unit(u)) {
        const int2 range = tile_range(u, q);
        // A block that no row of the tile sees (or a unit without the tile): the issuer
        // keeps step with the rings, so that no wait is for a phase further on.
        auto skip = [&](int j) {
          const int x = t + j - u.j;
          TSV_CWAIT(&k_full[x % kKStages], x / kKStages);
          TSV_CWAIT(&v_full[x & 1], x >> 1);
          if (!dead && elect_one()) {
            mbar_arrive(&k_empty[x % kKStages]);
            mbar_arrive(&v_empty[x & 1]);
          }
          __syncwarp();
        };
        // S of half a block.
        auto issue_s = [&](int j, int half) {
          const int x = t + j - u.j, st = x % kKStages;
          if (half == 0) TSV_CWAIT(&k_full[st], x / kKStages);
          if (dead) return;
          tc_fence_after();
          const uint32_t db = (uint32_t)dk + (uint32_t)((st * C::kKTile + half * 64 * D) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                umma_e4m3(s_at + half * 64, desc_at(dq, (uint32_t)dq + (uint32_t)((term * C::kQTile) >> 4) + kk * 2),
                          desc_at(dk, db + kk * 2), idS, term + kk > 0 ? 1u : 0u);
            umma_commit(&s_full[2 * q + half]);
            if (half == 1) umma_commit(&k_empty[st]);
          }
          __syncwarp();
        };
        if (range.x < range.y) {
          TSV_CWAIT(&q_full[q], mine_units);
          ++mine_units;
        }
#pragma unroll 1
        for (int j = u.j; j < range.x && !dead; ++j) skip(j);
        if (range.x < range.y && !dead) {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) issue_s(range.x, half);
        }
#pragma unroll 1
        for (int j = range.x; j < range.y && !dead; ++j) {
          const int x = t + j - u.j;
          TSV_CWAIT(&v_full[x & 1], x >> 1);
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            TSV_CWAIT(&p_full[2 * q + half], cnt);
            if (dead) break;
            tc_fence_after();
            const uint32_t db = (uint32_t)dv + (uint32_t)(((x & 1) * C::kVTile + half * 64 * 128) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // 16 keys each; P, two keys a column, lies over its S
                umma_f16_ts(o_at, s_at + half * 64 + kk * 8, desc_at(dv, db + (uint32_t)((kk * 16 * 128) >> 4)), idPV,
                            half + kk > 0 || j > range.x ? 1u : 0u);
              umma_commit(&pv_done[2 * q + half]);
              if (half == 1) umma_commit(&v_empty[x & 1]);
            }
            __syncwarp();
            if (j + 1 < range.y) issue_s(j + 1, half);
          }
          ++cnt;
        }
        if (range.x < range.y) {
#pragma unroll 1
          for (int j = range.y; j < u.j1 && !dead; ++j) skip(j);
        }
        t += u.j1 - u.j;
      }
      if (elect_one()) umma_commit(mma_done);  // every MMA has finished before TMEM is freed
      __syncwarp();
      mbar_wait(mma_done, 0, nullptr);
    } else {
      // -------------------------------------------------------- producers
      const bool is_v = warp == kCVWarp;
      const CUtensorMap* tmap = is_v ? &tmap_v : &tmap_k;
      const tsv_paged_cache& c = a.cache;
      const uint64_t pol = l2_policy_evict_last();
      int t = 0, asked = 0;
      for (bool going = first_unit(u); going && !dead; going = next_unit(u)) {
        const int32_t* ids = a.table.ids_d + (int64_t)u.b * a.table.stride;
        const int keys = u.start + min(u.n, geo.by_heads.of(u.row0 + u.rows - 1) + 1);
        const int page_end = (keys + (1 << lps) - 1) >> lps;
        // Keys in front of the unit's first window, as far as they fill 16: their pages may
        // hold anything, and have no say in V's largest scale.
        const int front = a.window > 0 ? max(0, u.start + geo.by_heads.of(u.row0) - a.window + 1) & ~15 : 0;
        // Lane p holds page p of the next block (of V's producer: of the next two), lanes
        // 0 .. 7 the next block's scales of 16 keys each: asked for a block ahead.
        auto page_of = [&](int j) {
          const int p = ((j * kPBlock) >> lps) + lane;
          return j < u.j1 && (lane << lps) < kPBlock && p < page_end ? __ldg(ids + p) : -1;
        };
        float top = 0.f, sk = 0.f, sv = 0.f;
        auto scales_of = [&](int pages, int j) {
          const int sid = __shfl_sync(0xffffffffu, pages, ((lane * 16) >> lps) & 31);
          const bool on = j < u.j1 && lane < 8 && lane * 16 < keys - j * kPBlock && lane * 16 >= front - j * kPBlock &&
                          (uint32_t)sid < (uint32_t)c.num_pages;
          sk = on ? __ldg(c.k_scale_d + (int64_t)sid * c.Hkv + u.g) : 0.f;
          sv = on ? __ldg(c.v_scale_d + (int64_t)sid * c.Hkv + u.g) : 0.f;
        };
        int now = page_of(u.j), next = page_of(u.j + 1);
        if (is_v) scales_of(now, u.j);
#pragma unroll 1
        for (int j = u.j; j < u.j1; ++j) {
          const int x = t + j - u.j;
          const int valid = min(kPBlock, keys - j * kPBlock);
          const uint32_t pages = (uint32_t)(valid + (1 << lps) - 1) >> lps;
          const float sk_now = sk, sv_now = sv;
          const int pages_now = now;
          now = next;
          next = page_of(j + 2);
          if (is_v) scales_of(now, j + 1);
          const int st = is_v ? x & 1 : x % kKStages;
          uint64_t* full = is_v ? &raw_full[st] : &k_full[st];
          if (is_v && x >= 2) TSV_CWAIT(&raw_empty[st], (x >> 1) - 1);
          if (!is_v && x >= kKStages) TSV_CWAIT(&k_empty[st], x / kKStages - 1);
          if (dead) break;
          const uint32_t at = smem_u32(is_v ? sRaw : sK) + (uint32_t)(st * C::kKTile);
          const bool lead = elect_one();
          if (lead) mbar_expect_tx(full, (pages << lps) * D);
          __syncwarp();
#pragma unroll 1
          for (uint32_t p = 0; p < pages; ++p)
            tma_load_page(at + (p << lps) * D, tmap, smem_u32(full), (uint32_t)u.g, (uint32_t)__shfl_sync(0xffffffffu, pages_now, (int)p), pol,
                          lead);
          __syncwarp();
          if (lead) mbar_arrive(full);
          asked = x + 1;
          if (!is_v && lead) abort_v[1] = (int)(uint32_t)global_timer_ns();
          if (is_v) {
            // The unit's largest V scale so far, and the block's relative to it as m 2^e:
            // 2^e goes into the exponent of P and m, 1 as a rule, into V as it is widened.
            top = fmaxf(top, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(sv_now))));  // (scales are >= 0)
            const float turn = top > 1.f ? 0x1p-64f : 0x1p64f;  // (the division wants an ordinary divisor)
            const bool past = lane * 16 >= valid || lane * 16 < front - j * kPBlock;  // (such keys take part in nothing)
            // (While every scale so far is 0, values are 0 whatever their codes: m is 0 as for a
            // scale of 0 beside others.)
            const float rel = past ? 1.f : top > 0.f ? __fdiv_rn(sv_now * turn, top * turn) : 0.f;
            const int e = max((int)(__float_as_uint(rel) >> 23) - 127, -kFarApart);
            const float m = rel * __uint_as_float((uint32_t)(127 - e) << 23);
            const bool all = __all_sync(0xffffffffu, lane >= 8 || m == 1.f);
            float* sc = sScale + (x & 3) * kScaleRow;
            if (lane < 8) {
              sc[lane] = sk_now;
              sc[8 + lane] = (float)e;
              sc[16 + lane] = __uint_as_float((uint32_t)(127 - e) << 23);
              sc[24 + lane] = m;
            }
            if (lane == 0) {
              sc[32] = top;
              sc[33] = all ? 1.f : 0.f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sc_full[x & 3]);
          }
        }
        t += u.j1 - u.j;
      }
      // Every copy has landed before the CTA leaves (whatever the other roles did).
      const int stages = is_v ? 2 : kKStages;
      for (int x = max(0, asked - stages); x < asked; ++x)
        mbar_wait(is_v ? &raw_full[x & 1] : &k_full[x % kKStages], (x / stages) & 1, nullptr);
    }
  }
  if (warp == kCMmaWarp + 1) {  // what the joining launch has to know
    CUnit v{};
    const bool any = first_unit(v);
    const Cut from = cut(0), to = cut(1);
    ChunkPart p{};
    p.empty = any ? 0 : 1;
    if (any) {
      p.cont = v.j > v.first;
      p.through = p.cont && v.j1 < v.end;
      if (to.j > 0 && !(from.f == to.f && from.g == to.g && from.j > 0)) {  // the last unit begins a group
        p.lead = 1;
        v.b = request_of(to.f);
        v.tile = to.f - sTiles[v.b];
        v.g = to.g;
        load_unit(v, to.f);
        p.off = v.off;
        p.row0 = v.row0;
        p.rows = v.rows;
        p.g = v.g;
      }
    }
    if (lane == 0) parts[blockIdx.x] = p;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_v) {
    CUnit v{};
    for (bool on = first_unit(v); on; on = next_unit(v)) *static_cast<volatile int32_t*>(timeouts + v.b) = 1;
  }
  if (warp == kCMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of a group (in the order of the CTAs) and checks the
// requests: CTA c x kJoinParts + k takes rows k x 256 / kJoinParts .. of the group
// that CTA c of the other launch began.
constexpr int kJoinParts = 16, kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_chunk_join_kernel(const __grid_constant__ PagedAttnArgs a, int ctas,
                                                                        const int32_t* timeouts, const ChunkPart* __restrict__ parts,
                                                                        const float* __restrict__ part_o,
                                                                        const float* __restrict__ part_ml) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < a.B) {
    const int b = blockIdx.x;
    PagedRequest r;
    bool bad = !paged_request(a, b, &r);
    if (!bad) bad = paged_bad_page(a, b, r, tid, kJoinThreads);
    bad = __syncthreads_or(bad);
    if (tid == 0) a.status[b] = timeouts[b] ? TSV_ERR_TIMEOUT : bad ? TSV_ERR_INVALID_ARG : TSV_OK;
  }
  const int c0 = blockIdx.x / kJoinParts, k = blockIdx.x % kJoinParts;
  if (c0 >= ctas) return;
  const ChunkPart p = parts[c0];
  if (!p.lead) return;
  constexpr int kRows = kPagedWideRows / kJoinParts, L4 = D / 4;  // 16 bytes a thread
  for (int i = tid; i < kRows * L4; i += kJoinThreads) {
    const int row = k * kRows + i / L4, d4 = (i % L4) * 4;
    if (row >= p.rows) return;
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int64_t slot) {
      const float m = part_ml[slot * 2 * kPagedWideRows + row], l = part_ml[(slot * 2 + 1) * kPagedWideRows + row];
      const float4 v = *reinterpret_cast<const float4*>(part_o + (slot * kPagedWideRows + row) * D + d4);
      const float t2 = fmaxf(top, m);
      const float f = top == -INFINITY ? 1.f : fast_exp2(top - t2);  // nothing yet: all zero (or NaN)
      const float w = m == -INFINITY ? 1.f : fast_exp2(m - t2);
      top = t2;
      sum = sum * f + l * w;
      o.x = o.x * f + v.x * w;
      o.y = o.y * f + v.y * w;
      o.z = o.z * f + v.z * w;
      o.w = o.w * f + v.w * w;
    };
    add(2 * c0 + 1);
    for (int c = c0 + 1; c < ctas; ++c) {
      if (parts[c].empty) continue;
      add(2 * c);
      if (!parts[c].through) break;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int gr = p.row0 + row, token = gr / a.G;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                              ((int64_t)(p.off + token) * a.Hq + p.g * a.G + (gr - token * a.G)) * D + d4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

template <int D>
cudaError_t launch_typed(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int num_sms, void* ws, cudaStream_t st) {
  char* w = static_cast<char*>(ws);
  const PagedChunkLayout lay = paged_chunk_layout(num_sms, D);
  int32_t* timeouts = reinterpret_cast<int32_t*>(w);
  ChunkPart* parts = reinterpret_cast<ChunkPart*>(w + lay.parts);
  float* po = reinterpret_cast<float*>(w + lay.part_o);
  float* pm = reinterpret_cast<float*>(w + lay.part_ml);
  // Rows of a unit.  The second tile of 256 rows costs a block hardly more, but few
  // units leave SMs idle, unless they are long enough to be cut.  Measured (us; 32
  // query heads on 8, D = 128), 128 / 256 rows: 512 tokens from the start (64 units of
  // 256) 23.6 / 26.5, 1024 (128 units) 51 / 38; behind 8000 tokens 64 tokens (8 units)
  // 44 / 51, 128 54 / 51, 256 78 / 63.
  const int64_t rows = (int64_t)a.max_nodes * a.G, tiles = ((int64_t)a.N * a.G + 255) / 256 * a.cache.Hkv;
  const int64_t keys = (int64_t)a.table.pages * a.cache.page_size;
  const int R = 2 * tiles >= num_sms || (rows > 512 && keys >= 4096) ? 256 : 128;
  const cudaError_t e =
      launch_pdl(paged_chunk_kernel<D>, dim3(num_sms), dim3(kCThreads), (size_t)CCfg<D>::kSmem, st, 0u, tk, tv, a,
                 ChunkGeometry{Divisor(a.G), R, a.window}, timeouts, parts, po, pm);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_chunk_join_kernel<D>, dim3(num_sms * kJoinParts > a.B ? num_sms * kJoinParts : a.B), dim3(kJoinThreads), 0, st, 0u,
                    a, num_sms, timeouts, parts, po, pm);
}

template <int D>
cudaError_t set_typed() {
  // The register split draws on what the block is launched with.
  cudaFuncAttributes attr;
  const cudaError_t e = cudaFuncGetAttributes(&attr, paged_chunk_kernel<D>);
  if (e != cudaSuccess) return e;
  if (attr.numRegs < 128) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(paged_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, CCfg<D>::kSmem);
}

}  // namespace

static_assert(sizeof(ChunkPart) == kPagedChunkPartBytes, "workspace layout");

cudaError_t paged_chunk_set_attributes(int32_t D) { return D == 64 ? set_typed<64>() : set_typed<128>(); }

cudaError_t launch_paged_chunk(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, int num_sms, void* ws,
                               cudaStream_t st) {
  return a.cache.D == 64 ? launch_typed<64>(tk, tv, a, num_sms, ws, st) : launch_typed<128>(tk, tv, a, num_sms, ws, st);
}

}  // namespace tsv
