// Attention over a paged cache for chunks of new tokens (sm_103a): more than
// 16 packed rows a sequence and key head, on tcgen05 tensor cores.
//
//   o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),   x_j = scale log2(e) (q . k_j)
//
// A unit is 256 packed rows (new token, query head of the key head's group):
// two tiles of 128, the M of one tcgen05.mma, that walk the same keys 80 at a
// time.  Two tiles halve the shared-memory fills that a product needs, and the
// tensor pipe has one tile's products while the other's softmax runs.  The
// line of all key tiles of all units is cut into equal parts, one a CTA
// (paged.cuh), so a chunk whose units are few, or uneven, or behind a mask's
// diagonal, still fills every SM.
//
// Why 80 keys: tensor memory has 512 columns, of which the two outputs take
// 256; a tile has 128 left, and 80 FP32 scores with 40 columns of BF16
// probabilities beside them are the most (in steps of 16) that fit without
// overlap.  With P over S, as 128 keys need, S_(j+1) has to wait until PV_j
// has completed: the pipe drains and refills twice a step, and the first form
// of this kernel came to 1171 TFLOP/s where this one has 1447.  Without
// overlap S_(j+1) is issued as soon as the softmax has S_j in registers.
//
// What bounds it is shared memory.  Of a step's (two tiles, 80 keys) products
// S reads Q and K there, 2 x 52 KB, PV reads V, 2 x 20 KB, and the loads write
// 40 KB: 1470 cycles at 128 bytes a cycle, against 1280 of the tensor pipe;
// it runs at about 1500.  In the E4M3 kind the widening moves 60 KB more (and
// the loads 20 KB less), about 1800 cycles; it runs at about 2000.  Q cannot
// come from tensor memory, which is full.
//
// Warps: 0 walks the line and issues the loads; 1 and 2 gather the Q rows of
// tile 0 and 1 (a group of any size, any strides) and issue S; 3 issues PV of
// both; 4-7 and 8-11 are the softmax of tile 0 and 1, one row a thread; E4M3
// pages have four more, 12-15, that widen codes to BF16: a staged tile of
// codes becomes the K or V tile that the BF16 kind loads, scale applied (the
// scales are powers of two: what results is exactly the BF16 value that
// cache_read gives).  A word's codes c0..c3 are taken as the pairs (c0, c2),
// (c1, c3), which need no byte permutation; Q's dimensions are brought into
// that order too, and the output's back.
//
// The loads are one warp's, and one instruction takes it 60 to 150 cycles, so
// their number counts: pages of 64 and 128 tokens come as the one or two runs
// of whole keys that a tile has in them (boxes of 16 to 80 keys, or untiled
// copies for codes), smaller ones as boxes of 16 keys.  2048 tokens over 17000
// keys, 40 query and 8 key heads, BF16: 449 us with boxes of 16 for all, 435
// with runs.
//
// Code that is seldom run is short here (the mask, the output): the softmax
// fills the instruction cache, and what is not in it costs about 100 cycles
// for every eight instructions.
//
// Measured (graphs of four calls, with the joining kernel; tensor rate of the
// visible pairs; the first by the chip's power, 936 to 974 us from run to run):
//   2048 new of 33792, 40 / 8 heads, causal, BF16    960 us  1431 TFLOP/s
//   8704 of 8704, 24 / 24 heads, causal, BF16        344 us  1353
//   1320 new of 9505, 56 / 56 heads, all keys, E4M3  322 us  1117
// (a cuBLAS product of 8192^3 reaches 1949 alone and 1723 for seconds).
//
// Tensor memory: O of tile 0 and 1 in columns [0, 128), [128, 256); S of
// tile t in [256 + 128 t, + 80), P in the 40 columns behind it.
#include <atomic>
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kTileKeys = kPagedChunkKeys;
constexpr int kBoxKeys = 16;             // divides pages and tiles
constexpr int kBoxes = kTileKeys / kBoxKeys;  // pages that a tile touches, at most
constexpr int kUnitRows = kPagedChunkRows;
// A K or V tile: for each 8 keys two blocks of 1 KB, [8 keys x 64 dimensions]
// with 128-byte swizzle, one for each half of the dimensions.
constexpr uint32_t kSlotBytes = kTileKeys * 256;
constexpr uint32_t kGroupBytes = 2048, kHalfBytes = 1024;
constexpr uint32_t kQBytes = 32768;      // of a tile: 2 column halves x [128 rows x 128 B]
constexpr int kSegs = 2;
constexpr int kStageSlots = 4;           // staged code tiles (E4M3): [80 keys x 128 B]
constexpr uint32_t kStageBytes = kTileKeys * 128;
// The reference follows a row's maximum only when that passes it, and then by
// this much more (log2), so that O is seldom rescaled.  Probabilities relative
// to it are at most 1: a sum of them times values overflows only where the one
// relative to the maximum itself would.
constexpr float kLead = 8.0f;
// The line's places of a CTA are those of this many key tiles at least, while
// there are any.  (A unit's beginning has places too, so the first CTAs of a
// unit may have fewer tiles, or none.)  300 tokens over 600 keys,
// 8 / 4 heads, E4M3: 22.6 us with 2 or 3, 24.6 with 4, 26.5 with 6; 20 over
// 8000, 8 / 1 heads, where the parts are to be joined: 46 with 1, 31 with 2.
constexpr int kMinTiles = 3;

template <int kKind>
struct Cfg {
  static constexpr int kThreads = kKind == 0 ? 384 : 512;
  // Registers after the split: the sum over warpgroups stays within the
  // launch allocation (384 x 168 or 512 x 128).
  static constexpr uint32_t kRegsLaunch = kKind == 0 ? 168 : 128;
  static constexpr uint32_t kRegsControl = kKind == 0 ? 88 : 72;
  static constexpr uint32_t kRegsSoftmax = kKind == 0 ? 208 : 176;
  static constexpr uint32_t kRegsConvert = 88;
  static_assert(kRegsControl + 2 * kRegsSoftmax + (kKind ? kRegsConvert : 0) <= (kThreads / 128) * kRegsLaunch, "");
  static constexpr int kSlots = kKind == 0 ? 8 : 6;  // K, V, K, V, ...
  // The line's places (paged.cuh): what a key tile costs under one row tile
  // and under two, and a unit's beginning, edges and end.  A short prompt's
  // units are unequal, so the last counts: 8704 of 8704 tokens, 24 heads, takes
  // 387 us with 2 key tiles for it, 363 with 4, 354 with 6 and 356 with 8; a
  // batch of seven sequences, up to 777 new each, 98, 87, 89 and 90.  Under one
  // row tile a BF16 key tile costs less (no second tile's products): 12
  // sequences of up to 100 new tokens, 63 us with 4 of 4 places, 56 with 3 (a
  // unit's ends at 4); an E4M3 one does not (its widening is the same): 1320
  // of 9505, 56 heads, 339 us with 4 of 4, 346 with 3.
  static constexpr int kHalfPlaces = kKind == 0 ? 3 : 4, kFullPlaces = 4;
  static constexpr int kOver = 6 * kFullPlaces;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffRing = 2 * kQBytes;
  static constexpr uint32_t kOffStage = kOffRing + kSlots * kSlotBytes;
  static constexpr uint32_t kOffExp = kOffStage + (kKind ? kStageSlots * kStageBytes : 0);
  static constexpr uint32_t kOffSeg = kOffExp + (kKind ? kStageSlots * kTileKeys : 0);
  static constexpr uint32_t kOffBar = kOffSeg + kSegs * 64;
  static constexpr uint32_t kOffMisc = kOffBar + 512;
  static constexpr uint32_t kOffOdd = kOffMisc + 64;  // [slots][2][3]: bits of keys with odd values
  static constexpr uint32_t kSmem = kOffOdd + 256 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};
static_assert(sizeof(Segment) <= 64, "");

enum {
  BAR_FULL = 0,     // +slot (8)
  BAR_EMPTY = 8,    // +slot: both tiles' products are done with it (even slots K, odd V)
  BAR_SGFULL = 16,  // +staged tile (4)
  BAR_SGEMPTY = 20,
  BAR_SEGFULL = 24, // +step (2)
  BAR_SEGEMPTY = 26,
  BAR_SFULL = 32,   // +tile
  BAR_SREAD = 34,   // the softmax has S in registers
  BAR_PFULL = 36,
  BAR_PVDONE = 38,
  BAR_VREADY = 42,  // +2 tile, + every other one: V of a tile at the mask's edge is ready
  BAR_DRAIN = 46,   // +issuer (3): products in flight have completed (abort)
  NUM_BARS = 49
};

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Largest of 80 values: three-input maxima.
__device__ __forceinline__ float max80(const uint32_t (&s)[kTileKeys]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 4]));
#pragma unroll
  for (int k = 8; k < kTileKeys; k += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = fmax3(m[i], __uint_as_float(s[k + i]), __uint_as_float(s[k + 4 + i]));
  return fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
}

__device__ __forceinline__ void lds128(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// V of a tile at the mask's edge (by a warp): rows outside [first, end), which
// no row of Q sees, become zeros, and so do rows that hold a NaN or an
// infinity, which set their bit.
__device__ __forceinline__ void edge_values(uint32_t v, int first, int end, uint32_t* bits, int lane) {
  // 16 lanes a row, 16 bytes each; two rows at a time
  auto at = [&](int row) {
    return v + (row / 8) * kGroupBytes + (lane / 8 % 2) * kHalfBytes + (row % 8) * 128 + (lane % 8) * 16;
  };
  const uint32_t zero[4] = {0, 0, 0, 0};
  const int row0 = lane / 16;
  if (lane < 3) bits[lane] = 0;
  if (first > 0 || end < kTileKeys) {
    for (int row = row0; row < kTileKeys; row += 2)
      if (row < first || row >= end) sts128(at(row), zero);
  }
  __syncwarp();
  auto largest = [&](int row) {  // magnitudes as integers, two to a word
    uint32_t z[4];
    lds128(z, at(row));
    return __vmaxu2(__vmaxu2(z[0] & 0x7FFF7FFFu, z[1] & 0x7FFF7FFFu), __vmaxu2(z[2] & 0x7FFF7FFFu, z[3] & 0x7FFF7FFFu));
  };
  auto not_finite = [](uint32_t m) { return (m >> 16) >= 0x7F80u || (m & 0xFFFFu) >= 0x7F80u; };
  uint32_t m = 0;
#pragma unroll 8
  for (int row = row0; row < kTileKeys; row += 2) m = __vmaxu2(m, largest(row));
  if (__any_sync(0xFFFFFFFFu, not_finite(m))) {
#pragma unroll 1
    for (int row = row0; row < kTileKeys; row += 2) {
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, not_finite(largest(row)));
      if ((who >> (16 * row0)) & 0xFFFFu) {
        sts128(at(row), zero);
        if (lane % 16 == 0) atomicOr(&bits[row / 32], 1u << (row % 32));
      }
    }
  }
  fence_proxy_async_smem();  // read by the products
  __syncwarp();
}

// O of this thread's row (tensor memory, the whole warp) += p V of the cached
// row `at`, for the threads that see it: p from Q and K themselves.
__device__ __noinline__ void odd_add(uint32_t o_col, const uint16_t* q, const uint8_t* k_pages, const uint8_t* v_pages,
                                     int64_t at, bool see, float c2, float neg) {
  const uint16_t* k = reinterpret_cast<const uint16_t*>(k_pages) + at * kHeadDim;
  const uint16_t* v = reinterpret_cast<const uint16_t*>(v_pages) + at * kHeadDim;
  float dot = 0.f;
  if (see) {
#pragma unroll 1
    for (int d = 0; d < kHeadDim; d += 2) {
      const uint32_t qv = *reinterpret_cast<const uint32_t*>(q + d), kv = *reinterpret_cast<const uint32_t*>(k + d);
      dot = fmaf(__uint_as_float(qv << 16), __uint_as_float(kv << 16), dot);
      dot = fmaf(__uint_as_float(qv & 0xFFFF0000u), __uint_as_float(kv & 0xFFFF0000u), dot);
    }
  }
  __syncwarp();
  const float p = ex2_approx(fmaf(dot, c2, neg));
#pragma unroll 1
  for (int d = 0; d < kHeadDim; d += 32) {
    uint32_t o[32];
    tmem_ld32(o_col + d, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (see)
        o[e] = __float_as_uint(fmaf(p, __uint_as_float(static_cast<uint32_t>(v[d + e]) << 16), __uint_as_float(o[e])));
    __syncwarp();
    tmem_st32(o_col + d, o);
    tmem_wait_st();
  }
}

template <int kKind>
__global__ void __launch_bounds__(Cfg<kKind>::kThreads, 1)
paged_chunk_kernel(const __grid_constant__ ChunkMaps maps, const PagedAttnArgs a, const PagedScratch ws) {
  using C = Cfg<kKind>;
  const PagedArgs& c = a.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(base);
  auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * i; };
  Segment* segs = reinterpret_cast<Segment*>(base + C::kOffSeg);
  volatile int32_t* s_abort = reinterpret_cast<volatile int32_t*>(base + C::kOffMisc);
  int32_t* s_bad = reinterpret_cast<int32_t*>(base + C::kOffMisc + 4);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(base + C::kOffMisc + 8);
  int32_t* s_loads = reinterpret_cast<int32_t*>(base + C::kOffMisc + 12);  // tiles that the producer has loaded
  uint32_t* s_odd = reinterpret_cast<uint32_t*>(base + C::kOffOdd);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  if (threadIdx.x < 64) s_odd[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    *s_abort = 0;
    *s_bad = 0;
    for (int i = 0; i < NUM_BARS; ++i) mbar_init(bar(i), 1);
    for (int i = 0; i < C::kSlots; ++i) {
      if (kKind) mbar_init(bar(BAR_FULL + i), 2);  // the widening warps
      mbar_init(bar(BAR_EMPTY + i), i % 2 ? 1 : 2);  // K: both tiles' issuers; V: one issuer
    }
    for (int i = 0; i < kStageSlots; ++i) mbar_init(bar(BAR_SGEMPTY + i), 2);
    for (int i = 0; i < kSegs; ++i) mbar_init(bar(BAR_SEGEMPTY + i), kKind ? 15 : 11);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(BAR_SREAD + t), 4);
      mbar_init(bar(BAR_PFULL + t), 4);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tslot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tslot, 0);

  auto wait = [&](int b, int parity) -> bool { return mbar_wait(bar(b), parity & 1, a.wait_limit); };
  // What is in flight completes before the CTA ends, whatever the limit.
  auto drain = [&](int b, int parity) { mbar_wait(bar(b), parity & 1, kWaitLimitNs); };
  // By a whole warp: one wait; two at once (parity < 0: only the first).  They
  // also fail once another warp has given up, which is looked at only by those
  // that have to wait (whoever goes on without a wait soon needs one).
  auto all_wait = [&](int b, int parity) {
    if (__all_sync(0xFFFFFFFFu, mbar_test_wait(bar(b), parity & 1))) return true;
    return __all_sync(0xFFFFFFFFu, wait(b, parity) && *s_abort == 0) != 0;
  };
  auto all_wait2 = [&](int b, int parity, int b2, int parity2) {
    const bool one = mbar_test_wait(bar(b), parity & 1), two = parity2 < 0 || mbar_test_wait(bar(b2), parity2 & 1);
    if (__all_sync(0xFFFFFFFFu, one && two)) return true;
    return __all_sync(0xFFFFFFFFu, wait(b, parity) && (parity2 < 0 || wait(b2, parity2)) && *s_abort == 0) != 0;
  };
  // The next step's description; false when waiting failed.
  auto next_seg = [&](int k, Segment& g) -> bool {
    if (!all_wait(BAR_SEGFULL + k % kSegs, k / kSegs)) return false;
    g = segs[k % kSegs];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(BAR_SEGEMPTY + k % kSegs));
    return true;
  };
  // K's slot of the CTA's x-th key tile is 2x, V's 2x + 1 of one sequence.
  constexpr int kSlots = C::kSlots;
  // What the producer loads into: the ring, or the staged codes.
  constexpr int kBufs = kKind ? kStageSlots : kSlots;
  constexpr int kFull = kKind ? BAR_SGFULL : BAR_FULL, kEmpty = kKind ? BAR_SGEMPTY : BAR_EMPTY;
  bool ok = true;

  if (warp < 4) setmaxnreg_dec<C::kRegsControl>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (kKind == 0 && lane < 2 * min(kBoxes, c.page_size / kBoxKeys)) tma_prefetch_desc(&maps.m[lane % 2][lane / 2]);
    LineWalk w;
    bool bad = false;
    using Line = LineShape<kUnitRows, kTileKeys, C::kHalfPlaces, C::kFullPlaces, C::kOver, kMinTiles * C::kFullPlaces, false>;
    walk_begin<Line>(a, w, blockIdx.x, gridDim.x, bad);
    JoinDesc join;
    join.pieces = 0;
    int q = 0, buf = 0, round = 0;  // tiles of K or V so far, the next one's slot and use of it
    const uint32_t elect = elect_one();
    auto next_buf = [&] {
      ++q;
      if (++buf == kBufs) {
        buf = 0;
        ++round;
      }
    };
    for (int k = 0; ok; ++k) {
      const Segment g = walk_next<Line>(a, w, blockIdx.x, join);
      ok = k < kSegs || all_wait(BAR_SEGEMPTY + k % kSegs, k / kSegs - 1);
      if (!ok) break;
      if (lane == 0) {
        segs[k % kSegs] = g;
        mbar_arrive(bar(BAR_SEGFULL + k % kSegs));
      }
      if (!g.valid) break;
      const int32_t* table = c.table + g.s * c.table_stride;
      const int p_lo = g.lo >> c.page_shift, p_hi = (g.hi + c.page_size - 1) >> c.page_shift;
      int have = -64, entry = 0;  // entry: page index have + lane
      for (int t = g.t0; t < g.t0 + g.nt && ok; ++t) {
        const int page0 = t * kTileKeys >> c.page_shift, page1 = (t * kTileKeys + kTileKeys - 1) >> c.page_shift;
        if (page1 >= have + 32) {
          have = page0;
          const int at = have + lane;
          entry = at >= p_lo && at < p_hi ? __ldg(table + at) : 0;
          const bool wrong = entry < 0 || entry >= c.pages;
          bad |= wrong;
          if (wrong) entry = -1;
        }
        // Keys n of the cache from row r on, to the tile's place `first`.
        auto load = [&](int kv, int b, uint32_t r, int first, int n) {
          if constexpr (kKind == 0) {
            tma_load_4d(sbase + C::kOffRing + b * kSlotBytes + first * 256, &maps.m[kv][n / kBoxKeys - 1],
                        bar(kFull + b), 0, 0, 0, r / 8);
          } else {
            bulk_load(sbase + C::kOffStage + b * kStageBytes + first * 128,
                      (kv ? c.v_pages : c.k_pages) + static_cast<uint64_t>(r) * 128, n * 128, bar(kFull + b));
            bulk_load(sbase + C::kOffExp + b * kTileKeys + first, (kv ? c.v_exp : c.k_exp) + r, n, bar(kFull + b));
          }
        };
        const int key0 = t * kTileKeys;
        if (c.page_shift >= 6) {
          // at most two pages
          const int key1 = page1 << c.page_shift, n0 = page0 == page1 ? kTileKeys : key1 - key0;
          const int e0 = __shfl_sync(0xFFFFFFFFu, entry, (page0 - have) & 31);
          const int e1 = __shfl_sync(0xFFFFFFFFu, entry, (page1 - have) & 31);
          const bool on0 = page0 >= p_lo && page0 < p_hi && e0 >= 0, on1 = n0 < kTileKeys && page1 < p_hi && e1 >= 0;
          const uint32_t r0 = ((static_cast<uint32_t>(e0) * c.H + g.h) << c.page_shift) + (key0 & (c.page_size - 1));
          const uint32_t r1 = (static_cast<uint32_t>(e1) * c.H + g.h) << c.page_shift;
          const int all = (on0 ? n0 : 0) + (on1 ? kTileKeys - n0 : 0);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            ok = q < kBufs || all_wait(kEmpty + buf, round - 1);
            if (!ok) break;
            if (elect) {
              mbar_arrive_expect_tx(bar(kFull + buf), all * (kKind ? 128 + 1 : 256));
              if (on0) load(kv, buf, r0, 0, n0);
              if (on1) load(kv, buf, r1, n0, kTileKeys - n0);
            }
            __syncwarp();
            next_buf();
          }
        } else {
          // lane i < 5: row of the cache where the i-th 16 keys begin (-1: not to be loaded)
          const int key = key0 + lane * kBoxKeys, at = key >> c.page_shift;
          const int page = __shfl_sync(0xFFFFFFFFu, entry, (at - have) & 31);
          const bool mine = lane < kBoxes && at >= p_lo && at < p_hi && page >= 0;
          const int row = mine ? static_cast<int>(((static_cast<uint32_t>(page) * c.H + g.h) << c.page_shift) +
                                                  (key & (c.page_size - 1)))
                               : -1;
          const int loads = __popc(__ballot_sync(0xFFFFFFFFu, mine));
          int rows[kBoxes];
#pragma unroll
          for (int i = 0; i < kBoxes; ++i) rows[i] = __shfl_sync(0xFFFFFFFFu, row, i);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            ok = q < kBufs || all_wait(kEmpty + buf, round - 1);
            if (!ok) break;
            if (elect) {
              mbar_arrive_expect_tx(bar(kFull + buf), loads * kBoxKeys * (kKind ? 128 + 1 : 256));
#pragma unroll
              for (int i = 0; i < kBoxes; ++i)
                if (rows[i] >= 0) load(kv, buf, rows[i], i * kBoxKeys, kBoxKeys);
            }
            __syncwarp();
            next_buf();
          }
        }
      }
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (!ok) {
      *s_abort = 1;
      // (the block's end waits for them as well; without these lines the
      // compiler's loop above is slower: a batch of seven sequences, up to 777
      // new each, 85.6 us against 82.8)
      for (int x = max(0, q - kBufs); x < q; ++x) drain(kFull + x % kBufs, x / kBufs);
    }
    if (lane == 0) {
      ws.join[blockIdx.x] = join;
      if (bad) *s_bad = 1;
      *s_loads = q;
    }
  } else if (warp < 3) {
    // ------------------------------------------------------------ Q and S of tile t
    const int t = warp - 1;
    const uint32_t id_s = idesc_bf16(128, kTileKeys, false, false);
    const uint32_t s_col = tmem + 256 + 128 * t;
    auto qmaj_off = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4); };
    auto kmaj_off = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4); };
    const uint64_t q_base = sdesc_sw128(sbase + C::kOffQ + t * kQBytes, 16, 1024);
    const uint32_t elect = elect_one();
    const int q_row = lane / 16, q_chunk = lane % 16;  // 16 bytes of Q's rows q_row, q_row + 2, ..
    const uint32_t q_to = sbase + C::kOffQ + t * kQBytes + (q_chunk / 8) * 16384;
    int slot = 0, phase = 0;  // K's slot of the next key tile, and its phase
    int y = 0;                // key tiles of this row tile so far
    bool issued = false;
    for (int k = 0; ok; ++k) {
      Segment g;
      ok = next_seg(k, g);
      if (!ok || !g.valid) break;
      const bool rows = g.rows > 128 * t;
      if (rows) {
        // Q: rows past the last are zeros.  The last unit's last S, the last
        // reader of the tile's Q, has completed when its barrier says so.
        // (What follows takes as long as the last unit's softmax and output.)
        ok = y == 0 || all_wait(BAR_SFULL + t, y - 1);
        if (!ok) break;
        const int rho = g.rho0 + 128 * t + q_row, left = g.rows - 128 * t;
        int i = div_group(a, rho), e = rho - i * a.group;
        const uint16_t* src = a.q + static_cast<int64_t>(g.row0 + i) * a.q_token +
                              static_cast<int64_t>(g.h * a.group + e) * a.q_head + q_chunk * 8;
        const int i2 = a.group == 1 ? 2 : a.group == 2 ? 1 : 0, e2 = 2 - i2 * a.group;  // two rows on: tokens and heads
        const int64_t step = i2 * a.q_token + e2 * a.q_head, wrap = a.q_token - a.group * a.q_head;
        auto at = [&](int r) { return q_to + r * 128 + ((q_chunk ^ r) & 7) * 16; };
#pragma unroll 4
        for (int r = q_row; r < 128; r += 2) {
          const bool is = r < left;
          cp_async16(at(r), is ? src : a.q, is);
          src += step;
          e += e2;
          if (e >= a.group) {
            e -= a.group;
            src += wrap;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (kKind != 0) {  // the order of dimensions that K gets (each lane its own 16 bytes)
#pragma unroll 8
          for (int r = q_row; r < 128; r += 2) {
            uint32_t v[4], z[4];
            lds128(v, at(r));
#pragma unroll
            for (int w = 0; w < 4; w += 2) {
              z[w] = __byte_perm(v[w], v[w + 1], 0x5410);
              z[w + 1] = __byte_perm(v[w], v[w + 1], 0x7632);
            }
            sts128(at(r), z);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
#pragma unroll 1
      for (int j = 0; j < g.nt; ++j) {
        // S_j goes over S_(j-1), which the softmax has in registers.  (Without
        // rows the slots are released as they come.)
        ok = all_wait2(BAR_FULL + slot, phase, BAR_SREAD + t, rows && y + j > 0 ? y + j - 1 : -1);
        if (!ok) break;
        if (rows) {
          tc_fence_after();
          const uint64_t ks = sdesc_sw128(sbase + C::kOffRing + slot * kSlotBytes, 16, kGroupBytes);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ss_elect(s_col, q_base + qmaj_off(kk), ks + kmaj_off(kk), id_s, kk > 0 ? 1u : 0u, elect);
          if (elect) {
            umma_commit(bar(BAR_EMPTY + slot));
            umma_commit(bar(BAR_SFULL + t));
          }
          issued = true;
        } else if (elect) {
          mbar_arrive(bar(BAR_EMPTY + slot));
        }
        __syncwarp();
        slot += 2;
        if (slot == kSlots) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (rows) y += g.nt;
    }
    if (!ok) *s_abort = 1;
    if (elect && issued) {  // products in flight complete before the CTA ends
      umma_commit(bar(BAR_DRAIN + t));
      drain(BAR_DRAIN + t, 0);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ O += P V of both tiles
    // (the softmax makes O zeros before a unit's first P)
    const uint32_t id_o = idesc_bf16(128, 128, false, true);
    auto vmaj_off = [](int kk) { return static_cast<uint64_t>((kk * 2 * kGroupBytes) >> 4); };
    const uint32_t elect = elect_one();
    int slot = 1, phase = 0;
    int y0 = 0, y1 = 0;          // key tiles of row tile 0 and 1
    int edges0 = 0, edges1 = 0;  // those of them at the mask's edge
    bool issued = false;
    for (int k = 0; ok; ++k) {
      Segment g;
      ok = next_seg(k, g);
      if (!ok || !g.valid) break;
      const int tiles = g.rows > 128 ? 2 : 1;
      // V at the mask's edge (see the softmax), a tile ahead of its product
      auto prepare = [&](int j, int at, int parity) -> bool {
        const int key0 = (g.t0 + j) * kTileKeys;
        if (key0 >= g.all_lo && key0 + kTileKeys <= g.all_hi) return true;
        if (!all_wait(BAR_FULL + at, parity)) return false;
        if constexpr (kKind == 0)
          edge_values(sbase + C::kOffRing + at * kSlotBytes, g.lo - key0, g.hi - key0, &s_odd[6 * at], lane);
        if (lane < tiles) mbar_arrive(bar(BAR_VREADY + 2 * lane + ((lane ? edges1 : edges0) & 1)));
        ++edges0;
        if (tiles == 2) ++edges1;
        return true;
      };
      ok = prepare(0, slot, phase);
#pragma unroll 1
      for (int j = 0; j < g.nt && ok; ++j) {
        const int slot2 = slot + 2 > kSlots ? 1 : slot + 2, phase2 = slot + 2 > kSlots ? phase ^ 1 : phase;
        ok = j + 1 == g.nt || prepare(j + 1, slot2, phase2);
        if (!ok) break;
        const uint64_t vs = sdesc_sw128(sbase + C::kOffRing + slot * kSlotBytes, kHalfBytes, kGroupBytes);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= tiles) break;
          ok = all_wait2(BAR_FULL + slot, phase, BAR_PFULL + t, (t ? y1 : y0) + j);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kTileKeys / 16; ++kk)
            umma_ts_elect(tmem + 128 * t, tmem + 256 + 128 * t + kTileKeys + kk * 8, vs + vmaj_off(kk), id_o,
                          1u, elect);
          if (elect) {
            if (t + 1 == tiles) umma_commit(bar(BAR_EMPTY + slot));
            umma_commit(bar(BAR_PVDONE + t));
          }
          __syncwarp();
          issued = true;
        }
        slot = slot2;
        phase = phase2;
      }
      y0 += g.nt;
      if (tiles == 2) y1 += g.nt;
    }
    if (!ok) *s_abort = 1;
    if (elect && issued) {
      umma_commit(bar(BAR_DRAIN + 2));
      drain(BAR_DRAIN + 2, 0);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax of tile t
    setmaxnreg_inc<C::kRegsSoftmax>();
    const int t = (warp - 4) / 4;
    const int row = (warp & 3) * 32 + lane;  // of the tile: a lane of tensor memory
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_addr + 256 + 128 * t, p_col = s_col + kTileKeys, o_col = tmem + lane_addr + 128 * t;
    const float c2 = a.scale * 1.4426950408889634f;
    int x = 0, y = 0, edges = 0;
    for (int k = 0; ok; ++k) {
      Segment g;
      ok = next_seg(k, g);
      if (!ok || !g.valid) break;
      if (g.rows <= 128 * t) {
        x += g.nt;
        continue;
      }
      const int rho = g.rho0 + 128 * t + row;
      const bool real = 128 * t + row < g.rows;
      const int i = div_group(a, rho);
      const int pos = g.len - g.n + i;
      // a row that does not exist has Q = 0: no mask, and no output
      const int lo = real ? row_lo(a, pos) : 0;
      const int hi = real ? (a.causal ? min(g.len, pos + 1) : g.len) : 0x7FFFFFFF;
      float ref = -INFINITY, l = 0.f;
      float whole = 1.f;  // NaN once the row has seen a value that is NaN as a whole
      // O starts as zeros (PV accumulates; the last unit's O has been read)
      {
        uint32_t zero[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) zero[e] = 0;
#pragma unroll
        for (int b = 0; b < 128; b += 32) tmem_st32(o_col + b, zero);
      }
      // One key tile; false when a wait gave up.  edge: some row of the unit
      // does not see some key of it.
      auto tile = [&](bool edge, int j) -> bool {
        if (!all_wait(BAR_SFULL + t, y + j)) return false;
        tc_fence_after();
        const int key0 = (g.t0 + j) * kTileKeys;
        if (edge) {
          // masked in place: what most tiles skip stays small and takes no
          // registers from the rest (a second copy of the code, with the mask
          // in it, cost more than it saved: it was never in the instruction cache)
#pragma unroll 1
          for (int b = 0; b < kTileKeys; b += 16) {
            const int from = lo - key0 - b, to = hi - key0 - b;
            if (__all_sync(0xFFFFFFFFu, !real || (from <= 0 && to >= 16))) continue;
            uint32_t z[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(-INFINITY);
            // (a load's way there and back is most of the 400 cycles of a block)
            if (!__all_sync(0xFFFFFFFFu, !real || to <= 0 || from >= 16)) {
              tmem_ld16(s_col + b, z);
              tmem_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < from || e >= to) z[e] = __float_as_uint(-INFINITY);
            tmem_st8(s_col + b, *reinterpret_cast<uint32_t(*)[8]>(&z[0]));
            tmem_st8(s_col + b + 8, *reinterpret_cast<uint32_t(*)[8]>(&z[8]));
          }
          tmem_wait_st();
        }
        uint32_t s[kTileKeys];
        tmem_ld32(s_col, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
        tmem_ld32(s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
        tmem_ld16(s_col + 64, *reinterpret_cast<uint32_t(*)[16]>(&s[64]));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_SREAD + t));
        const float mx = max80(s) * c2;  // (scale > 0)
        const float prev = ref;
        if (mx > prev) ref = mx + kLead;
        const bool moved = prev != -INFINITY && ref != prev;
        const float neg = ref == -INFINITY ? 0.f : -ref;
        const uint64_t c2x = f2(c2, c2), negx = f2(neg, neg);
        uint64_t sum[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) sum[b] = f2(0.f, 0.f);
        uint32_t p[kTileKeys / 2];
#pragma unroll
        for (int b = 0; b < kTileKeys / 2; ++b) {
          float x0, x1;
          unf2(ffma2(f2(__uint_as_float(s[2 * b]), __uint_as_float(s[2 * b + 1])), c2x, negx), x0, x1);
          const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
          sum[b & 3] = fadd2(sum[b & 3], f2(e0, e1));
          p[b] = pack_bf16x2(e0, e1);
        }
        // O holds the tiles before j, and P_(j-1)'s place is free, when PV_(j-1) has completed
        if (j > 0) {
          if (!all_wait(BAR_PVDONE + t, y + j - 1)) return false;
          tc_fence_after();
        }
        if (__any_sync(0xFFFFFFFFu, moved)) {
          const float f = moved ? ex2_approx(prev - ref) : 1.0f;
          l *= f;
#pragma unroll 1
          for (int b = 0; b < 128; b += 32) {
            uint32_t o[32];
            tmem_ld32(o_col + b, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(o_col + b, o);
          }
        }
        {
          float z0, z1;
          unf2(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])), z0, z1);
          l += z0 + z1;
        }
        tmem_st32(p_col, *reinterpret_cast<uint32_t(*)[32]>(&p[0]));
        tmem_st8(p_col + 32, *reinterpret_cast<uint32_t(*)[8]>(&p[32]));
        if (edge) {
          // At the mask's edge a key of the tile may be hidden from a row that
          // its probability 0 would still multiply with what V holds, and
          // 0 * NaN is not 0.  Slots that no row sees may hold anything; keys
          // that only some rows see hold tokens, but these may have a NaN or
          // an infinity.  The PV warp (in the E4M3 kind the widening warps)
          // has made zeros of both; the tokens among them, a bit each in
          // s_odd, are added here one by one.
          if (!all_wait(BAR_VREADY + 2 * t + (edges & 1), edges / 2)) return false;
          ++edges;
          const int slot = (2 * (x + j) + 1) % kSlots;
          uint32_t odd[3];
#pragma unroll
          for (int w = 0; w < 3; ++w) {
            odd[w] = *reinterpret_cast<volatile uint32_t*>(&s_odd[6 * slot + w]);
            if (kKind != 0) odd[w] |= *reinterpret_cast<volatile uint32_t*>(&s_odd[6 * slot + 3 + w]);
          }
          if (odd[0] | odd[1] | odd[2]) {
            tmem_wait_st();
#pragma unroll 1
            for (int b = 0; b < kTileKeys; ++b) {
              if (!((b < 32 ? odd[0] : b < 64 ? odd[1] : odd[2]) >> (b % 32) & 1)) continue;
              const int key = key0 + b;
              const bool see = real && key >= lo && key < hi;
              if constexpr (kKind != 0) {
                if (see) whole = __uint_as_float(0x7FFFFFFFu);  // all of the value is NaN
              } else {
                const int page = c.table[g.s * c.table_stride + (key >> c.page_shift)];
                if (page < 0 || page >= c.pages) continue;  // (reported by the producer)
                odd_add(o_col,
                        a.q + static_cast<int64_t>(g.row0 + i) * a.q_token +
                            static_cast<int64_t>(g.h * a.group + rho - i * a.group) * a.q_head,
                        c.k_pages, c.v_pages,
                        ((static_cast<int64_t>(page) * c.H + g.h) << c.page_shift) + (key & (c.page_size - 1)), see, c2,
                        neg);
              }
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_PFULL + t));
        return true;
      };
#pragma unroll 1
      for (int j = 0; j < g.nt && ok; ++j) {
        const int key0 = (g.t0 + j) * kTileKeys;
        ok = tile(key0 < g.all_lo || key0 + kTileKeys > g.all_hi, j);
      }
      // ---- the unit's output, or this step's part of it (the widened codes of
      // four dimensions lie in the order 0, 2, 1, 3)
      auto dim = [](int d) constexpr { return kKind == 0 || d % 4 == 0 || d % 4 == 3 ? d : d % 4 == 1 ? d + 1 : d - 1; };
      ok = ok && all_wait(BAR_PVDONE + t, y + g.nt - 1);
      if (!ok) break;
      tc_fence_after();
      const int64_t at = g.part < 0 ? static_cast<int64_t>(g.row0 + i) * a.Hq + g.h * a.group + (rho - i * a.group)
                                    : (static_cast<int64_t>(blockIdx.x) * 2 + g.part) * kUnitRows + 128 * t + row;
      float* part = ws.part + (static_cast<int64_t>(blockIdx.x) * 2 + g.part) * kUnitRows * kHeadDim;  // (g.part >= 0)
      const float inv = (g.part >= 0 ? 1.f : l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) * whole;  // (NaN stays)
      // Output rows are Hq rows apart, and a store of one row a lane touches 32
      // lines: lanes 4 x .. 4 x + 3 exchange their rows' quarters of 64 bytes
      // first, so that each store has 8 rows of them.
      int64_t to[4];
      const uint32_t reals = __ballot_sync(0xFFFFFFFFu, real);
#pragma unroll
      for (int f = 0; f < 4; ++f) to[f] = __shfl_sync(0xFFFFFFFFu, at, (lane & ~3) + f) * kHeadDim + lane % 4 * 8;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t o[32];
        tmem_ld32(o_col + 32 * b, o);
        tmem_wait_ld();
        if (g.part < 0) {
          uint32_t z[4][4];  // [quarter][word], then [row][word]
#pragma unroll
          for (int f = 0; f < 16; ++f)
            z[f / 4][f % 4] = pack_bf16x2(__uint_as_float(o[dim(2 * f)]) * inv, __uint_as_float(o[dim(2 * f + 1)]) * inv);
#pragma unroll
          for (int d = 1; d < 4; d *= 2) {
            const bool upper = lane & d;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              if (f & d) continue;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, upper ? z[f][w] : z[f + d][w], d);
                if (upper)
                  z[f][w] = got;
                else
                  z[f + d][w] = got;
              }
            }
          }
#pragma unroll
          for (int f = 0; f < 4; ++f)
            if (reals >> ((lane & ~3) + f) & 1)
              *reinterpret_cast<uint4*>(a.o + to[f] + 32 * b) = make_uint4(z[f][0], z[f][1], z[f][2], z[f][3]);
        } else if (real) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t z[8];
#pragma unroll
            for (int f = 0; f < 8; ++f) z[f] = __float_as_uint(__uint_as_float(o[dim(8 * e + f)]) * inv);
            // [8 columns][row]: a warp's stores lie side by side
            st_global_v8(part + ((4 * b + e) * kUnitRows + 128 * t + row) * 8, z);
          }
        }
      }
      if (real) {
        if (g.part >= 0)
          ws.ml[at] = make_float2(ref, l);
        else if (a.lse)
          a.lse[at] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
      }
      x += g.nt;
      y += g.nt;
    }
    if (!ok) {
      tmem_wait_st();  // stores in flight complete before tensor memory is freed
      *s_abort = 1;
    }
  } else if constexpr (kKind != 0) {
    // ------------------------------------------------------------ widening
    setmaxnreg_dec<C::kRegsConvert>();
    // Two warps take the K tiles, two the V tiles (and so, with even numbers
    // of slots, the same slots always: they see every phase of their barriers).
    static_assert(kSlots % 2 == 0 && kStageSlots % 2 == 0, "slots of the widening warps");
    const int kv = (warp - 12) / 2;
    int x = kv;
    for (int k = 0; ok; ++k) {
      Segment g;
      ok = next_seg(k, g);
      if (!ok || !g.valid) break;
      for (int j = 0; j < g.nt; ++j, x += 2) {
        const int b = x % kStageSlots, slot = x % kSlots;
        ok = all_wait2(BAR_SGFULL + b, x / kStageSlots, BAR_EMPTY + slot, x >= kSlots ? x / kSlots - 1 : -1);
        if (!ok) break;
        const int key0 = (g.t0 + j) * kTileKeys;
        const uint32_t src = sbase + C::kOffStage + b * kStageBytes, dst = sbase + C::kOffRing + slot * kSlotBytes;
        // A warp takes 16 codes of 4 rows x 8 chunks at a time.  Eight lanes
        // are two rows, half of the chunks of one and the other half of the
        // other, so that neither their loads nor their stores (every other
        // chunk of a half of the dimensions) meet in a bank.
        const int ch = lane % 4 + 4 * ((lane / 4 ^ lane / 8) % 2), row0 = (warp % 2) * 4 + lane / 4 % 2 + 2 * (lane / 16);
        const bool inside = key0 >= g.lo && key0 + kTileKeys <= g.hi;
        const bool edge = key0 < g.all_lo || key0 + kTileKeys > g.all_hi;
        if (kv == 1 && edge) {
          // (see the softmax) values that are NaN: a bit, and exponent 0 for zeros
          uint32_t* bits = &s_odd[6 * slot + 3 * (warp % 2)];
          if (lane < 3) bits[lane] = 0;
          __syncwarp();
          for (int row = lane; row < kTileKeys; row += 32) {
            uint8_t* e = base + C::kOffExp + b * kTileKeys + row;
            if (*e == 255 && key0 + row >= g.lo && key0 + row < g.hi) {
              atomicOr(&bits[row / 32], 1u << (row % 32));
              *e = 0;
            }
          }
          __syncwarp();
        }
        const uint32_t from = src + row0 * 128 + ch * 16, exps = sbase + C::kOffExp + b * kTileKeys + row0;
        const uint32_t to0 = dst + (ch / 4) * kHalfBytes + row0 * 128 + ((2 * ch % 8) ^ row0) * 16;
        const uint32_t to1 = dst + (ch / 4) * kHalfBytes + row0 * 128 + (((2 * ch + 1) % 8) ^ row0) * 16;
        // Codes land as the value times 2^-120; one factor then, of 2^120 and
        // the row's scale.
        auto widen = [&](const uint32_t(&in)[4], uint32_t two, uint32_t(&out)[8]) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {  // (c0, c2) and (c1, c3) of a word
            const uint32_t v = in[w];
            out[2 * w] = bf16x2_mul(((v * 16) & 0x07F007F0u) | ((v * 256) & 0x80008000u), two);
            out[2 * w + 1] = bf16x2_mul(((v >> 4) & 0x07F007F0u) | (v & 0x80008000u), two);
          }
        };
        bool plain = inside;  // every row seen, and every factor at most 2^127
        for (int row = lane; row < kTileKeys; row += 32)
          plain = plain && lds8(sbase + C::kOffExp + b * kTileKeys + row) - 1u < 134u;
        if (__all_sync(0xFFFFFFFFu, plain)) {
#pragma unroll 1
          for (int i0 = 0; i0 < kTileKeys / 8; i0 += 5) {
            uint32_t in[5][4], e[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) {  // all loads first
              lds128(in[i], from + (i0 + i) * 1024);
              e[i] = lds8(exps + (i0 + i) * 8);
            }
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              uint32_t out[8];
              widen(in[i], (e[i] + 120) * 0x00800080u, out);
              sts128(to0 + (i0 + i) * kGroupBytes, *reinterpret_cast<uint32_t(*)[4]>(&out[0]));
              sts128(to1 + (i0 + i) * kGroupBytes, *reinterpret_cast<uint32_t(*)[4]>(&out[4]));
            }
          }
        } else {
          // 0 where no row sees the key, whatever was there; NaN for the
          // exponent byte 255 (a byte of 0 is no exponent of cache_write); a
          // second factor for large scales
#pragma unroll 1
          for (int i = 0; i < kTileKeys / 8; ++i) {
            uint32_t in[4], out[8], e = lds8(exps + i * 8);
            lds128(in, from + i * 1024);
            if (key0 + row0 + 8 * i < g.lo || key0 + row0 + 8 * i >= g.hi) e = 0;
            const uint32_t e1 = min(e, 134u), more = (e - e1 + 127) * 0x00800080u;
            widen(in, e == 0 ? 0u : e == 255 ? 0x7FFF7FFFu : (e1 + 120) * 0x00800080u, out);
#pragma unroll
            for (int w = 0; w < 8; ++w) out[w] = bf16x2_mul(out[w], more);
            sts128(to0 + i * kGroupBytes, *reinterpret_cast<uint32_t(*)[4]>(&out[0]));
            sts128(to1 + i * kGroupBytes, *reinterpret_cast<uint32_t(*)[4]>(&out[4]));
          }
        }
        fence_proxy_async_smem();  // read by the products
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(BAR_FULL + slot));
          mbar_arrive(bar(BAR_SGEMPTY + b));
        }
      }
    }
    if (!ok) *s_abort = 1;
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Where a warp has given up, nobody may have waited for the last loads: they
  // land before the CTA ends (bounded).  Only here is it known: the producer
  // may have issued all its loads before another warp's wait fails.
  if (warp == 0 && *s_abort) {
    const int n = *s_loads;
    for (int x = max(0, n - kBufs); x < n; ++x) drain(kFull + x % kBufs, x / kBufs);
  }
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) ws.cta_status[blockIdx.x] = *s_abort ? 5 /* SA_ETIMEOUT */ : (*s_bad ? kPagedInvalid : 0);
  griddep_launch_dependents();
}

template <int kKind>
cudaError_t launch(const ChunkMaps& maps, const PagedAttnArgs& a, const PagedScratch& ws, int ctas, cudaStream_t s) {
  using C = Cfg<kKind>;
  auto* kern = paged_chunk_kernel<kKind>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(kern), C::kSmem);
  if (e != cudaSuccess) return e;
  // The register split redistributes the launch allocation; a build with
  // fewer registers a thread would make setmaxnreg.inc wait forever.
  static std::atomic<int> known{0};
  int regs = known.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
    known.store(regs, std::memory_order_relaxed);
  }
  const int split = C::kRegsControl + 2 * C::kRegsSoftmax + (kKind ? C::kRegsConvert : 0);
  if (regs * (C::kThreads / 128) < split) return cudaErrorInvalidConfiguration;
  kern<<<ctas, C::kThreads, C::kSmem, s>>>(maps, a, ws);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_chunk(const ChunkMaps& maps, const PagedAttnArgs& a, const PagedScratch& ws, int ctas,
                               cudaStream_t s) {
  return a.c.kind == 0 ? launch<0>(maps, a, ws, ctas, s) : launch<1>(maps, a, ws, ctas, s);
}

}  // namespace sa
