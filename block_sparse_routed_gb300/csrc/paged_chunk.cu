// Attention over a paged cache for chunks of new tokens (sm_103a): more than
// 16 packed rows a sequence and key head, on tcgen05 tensor cores.
//
//   o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),   x_j = scale log2(e) (q . k_j)
//
// A unit is 256 packed rows (new token, query head of the key head's group):
// two tiles of 128, the M of one tcgen05.mma, that walk the same keys 128 at a
// time.  Two tiles halve the shared-memory fills a product needs (64 KB of K
// and V for 256 x 128 x 128 x 4 flops), and while one tile's softmax runs the
// tensor pipe has the other's products.  The line of all key tiles of all
// units is cut into equal parts, one a CTA (paged.cuh), so a chunk whose units
// are few, or uneven, or behind a mask's diagonal, still fills every SM.
//
// Warps: 0 walks the line and issues the TMA loads (one box a page); 1 and 2
// issue the products of tile 0 and 1; 3 brings Q into shared memory (rows are
// gathered: a group of any size, any strides); 4-7 and 8-11 are the softmax of
// tile 0 and 1, one row a thread; E4M3 pages have four more, 12-15, that widen
// codes to BF16: a staged tile of codes becomes the K or V tile that the BF16
// kind loads, scale applied (the scales are powers of two: what results is
// exactly the BF16 value that cache_read gives).
//
// A tile's chain is S_j = Q K_j^T, softmax, O += P_j V_j; P (BF16) goes over
// S's first half in tensor memory.  S_(j+1) is issued when PV_j has completed,
// so a softmax that sees S_j may rescale O at once; it does so only when a
// row's maximum has passed its reference by 2^32.
//
// Tensor memory: S of tile 0 and 1 in columns [0, 128), [128, 256), O in
// [256, 384), [384, 512).
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kKeyShift = 7;  // 128 keys a tile
constexpr int kTileKeys = 1 << kKeyShift;
constexpr int kUnitRows = 256;
constexpr int kSlots = 4;                // K, V, K, V, ...
constexpr uint32_t kSlotBytes = 32768;   // 2 column halves x [128 keys x 128 B]
constexpr uint32_t kQBytes = 32768;      // of a tile: 2 column halves x [128 rows x 128 B]
constexpr int kSegs = 2;
constexpr int kStageSlots = 2;           // staged code tiles (E4M3): [128 keys x 128 B]
constexpr uint32_t kStageBytes = 16384;
constexpr float kRescaleLog2 = 32.0f;
constexpr int kMinTiles = 4;             // key tiles of a CTA at least, while there are any

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
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffRing = 2 * kQBytes;
  static constexpr uint32_t kOffStage = kOffRing + kSlots * kSlotBytes;
  static constexpr uint32_t kOffExp = kOffStage + (kKind ? kStageSlots * kStageBytes : 0);
  static constexpr uint32_t kOffSeg = kOffExp + (kKind ? kStageSlots * kTileKeys : 0);
  static constexpr uint32_t kOffBar = kOffSeg + kSegs * 64;
  static constexpr uint32_t kOffMisc = kOffBar + 256;
  static constexpr uint32_t kSmem = kOffMisc + 64 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};
static_assert(sizeof(Segment) <= 64, "");

enum {
  BAR_FULL = 0,     // +slot (4)
  BAR_EMPTY = 4,    // +slot: both tiles' products are done with it
  BAR_SGFULL = 8,   // +staged tile (2)
  BAR_SGEMPTY = 10,
  BAR_SEGFULL = 12, // +step (2)
  BAR_SEGEMPTY = 14,
  BAR_QFULL = 16,   // +tile (2)
  BAR_QEMPTY = 18,  // +tile: the unit's last S has completed
  BAR_SFULL = 20,   // +tile
  BAR_PFULL = 22,
  BAR_PVDONE = 24,
  BAR_OEMPTY = 26,  // the output has been read
  BAR_DRAIN = 28,   // +tile: products in flight have completed (abort)
  NUM_BARS = 30
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

// Largest of 128 values: three-input maxima.
__device__ __forceinline__ float max128(const uint32_t (&s)[128]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 4]));
#pragma unroll
  for (int k = 8; k < 128; k += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = fmax3(m[i], __uint_as_float(s[k + i]), __uint_as_float(s[k + 4 + i]));
  return fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 16 bytes, or zeros when !real.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

template <int kKind>
__global__ void __launch_bounds__(Cfg<kKind>::kThreads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const PagedAttnArgs a, const PagedScratch ws) {
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
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    *s_abort = 0;
    *s_bad = 0;
    for (int i = 0; i < NUM_BARS; ++i) mbar_init(bar(i), 1);
    for (int i = 0; i < kSlots; ++i) {
      if (kKind) mbar_init(bar(BAR_FULL + i), 4);  // the widening warps
      mbar_init(bar(BAR_EMPTY + i), 2);
    }
    for (int i = 0; i < kStageSlots; ++i) mbar_init(bar(BAR_SGEMPTY + i), 4);
    for (int i = 0; i < kSegs; ++i) mbar_init(bar(BAR_SEGEMPTY + i), kKind ? 15 : 11);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(BAR_PFULL + t), 4);
      mbar_init(bar(BAR_OEMPTY + t), 4);
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
  const uint32_t tmem = *tslot;

  auto wait = [&](int b, int parity) -> bool { return mbar_wait(bar(b), parity & 1, kWaitLimitNs); };
  // The next step's description; false when waiting failed.
  auto next_seg = [&](int k, Segment& g) -> bool {
    if (!__all_sync(0xFFFFFFFFu, wait(BAR_SEGFULL + k % kSegs, k / kSegs))) return false;
    g = segs[k % kSegs];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(BAR_SEGEMPTY + k % kSegs));
    return true;
  };
  // K's slot of the CTA's x-th key tile is 2x, V's 2x + 1 of one sequence.
  auto slot_addr = [&](int q) { return sbase + C::kOffRing + (q % kSlots) * kSlotBytes; };
  bool ok = true;

  if (warp < 4) setmaxnreg_dec<C::kRegsControl>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    LineWalk w;
    bool bad = false;
    walk_begin(a, w, kUnitRows, kKeyShift, blockIdx.x, gridDim.x, kMinTiles, bad);
    JoinDesc join;
    join.pieces = 0;
    int q = 0;  // tiles of K or V so far
    const int tile_pages = kTileKeys >> c.page_shift;  // (pages of 16 to 128 keys)
    const int sub = lane % 2, pg = lane / 2;
    constexpr int kBufs = kKind ? kStageSlots : kSlots;
    constexpr int kFull = kKind ? BAR_SGFULL : BAR_FULL, kEmpty = kKind ? BAR_SGEMPTY : BAR_EMPTY;
    for (int k = 0; ok; ++k) {
      const Segment g = walk_next(a, w, kUnitRows, kKeyShift, blockIdx.x, join);
      ok = k < kSegs || __all_sync(0xFFFFFFFFu, wait(BAR_SEGEMPTY + k % kSegs, k / kSegs - 1));
      if (!ok) break;
      if (lane == 0) {
        segs[k % kSegs] = g;
        mbar_arrive(bar(BAR_SEGFULL + k % kSegs));
      }
      if (!g.valid) break;
      const int32_t* table = c.table + g.s * c.table_stride;
      const int p_lo = g.lo >> c.page_shift, p_hi = (g.hi + c.page_size - 1) >> c.page_shift;
      int have = -1, entry = 0;  // entry: page index 32 * have + lane
      for (int t = g.t0; t < g.t0 + g.nt && ok; ++t) {
        const int page0 = t * tile_pages;
        if (page0 / 32 != have) {
          have = page0 / 32;
          const int at = have * 32 + lane;
          entry = at >= p_lo && at < p_hi ? __ldg(table + at) : 0;
          const bool wrong = entry < 0 || entry >= c.pages;
          bad |= wrong;
          if (wrong) entry = -1;
        }
        const int at = page0 + pg;
        const int page = __shfl_sync(0xFFFFFFFFu, entry, at % 32);
        const bool mine = pg < tile_pages && at >= p_lo && at < p_hi && page >= 0;
        const int loads = __popc(__ballot_sync(0xFFFFFFFFu, mine && sub == 0));
        const int row = static_cast<int>((static_cast<int64_t>(page) * c.H + g.h) << c.page_shift);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++q) {
          const int b = q % kBufs;
          ok = q < kBufs || __all_sync(0xFFFFFFFFu, wait(kEmpty + b, q / kBufs - 1));
          if (!ok) break;
          if (lane == 0)
            mbar_arrive_expect_tx(bar(kFull + b), (loads << c.page_shift) * (kKind ? 128 + 1 : 256));
          __syncwarp();
          if (mine) {
            const CUtensorMap* map = kv ? &tm_v : &tm_k;
            if constexpr (kKind == 0) {
              tma_load_2d(slot_addr(q) + sub * (kTileKeys * 128) + (pg << c.page_shift) * 128, map, bar(kFull + b),
                          sub * 64, row);
            } else if (sub == 0) {
              tma_load_2d(sbase + C::kOffStage + b * kStageBytes + (pg << c.page_shift) * 128, map, bar(kFull + b), 0,
                          row);
            } else {
              bulk_load(sbase + C::kOffExp + b * kTileKeys + (pg << c.page_shift), (kv ? c.v_exp : c.k_exp) + row,
                        c.page_size, bar(kFull + b));
            }
          }
        }
        if (__any_sync(0xFFFFFFFFu, *s_abort != 0)) ok = false;
      }
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (!ok) {
      *s_abort = 1;
      // copies in flight land before the CTA ends (bounded)
      for (int x = max(0, q - kBufs); x < q; ++x) wait(kFull + x % kBufs, x / kBufs);
    }
    if (lane == 0) {
      ws.join[blockIdx.x] = join;
      if (bad) *s_bad = 1;
    }
  } else if (warp < 3) {
    // ------------------------------------------------------------ products of tile t
    const int t = warp - 1;
    const uint32_t id_s = idesc_bf16(128, 128, false, false), id_o = idesc_bf16(128, 128, false, true);
    const uint32_t s_col = tmem + 128 * t, o_col = tmem + 256 + 128 * t;
    auto kmaj_off = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4); };
    auto vmaj_off = [](int kk) { return static_cast<uint64_t>((kk * 2048) >> 4); };
    const uint64_t q_base = sdesc_sw128(sbase + C::kOffQ + t * kQBytes, 16, 1024);
    int x = 0;     // key tiles of the CTA so far
    int y = 0;     // key tiles of this row tile so far
    int units = 0; // units in which the row tile has rows
    bool issued = false;
    for (int k = 0; ok; ++k) {
      Segment g;
      ok = next_seg(k, g);
      if (!ok || !g.valid) break;
      if (g.rows <= 128 * t) {
        // no rows: the slots are released as they come
        if (lane == 0)
          for (int j = 0; j < 2 * g.nt && ok; ++j) {
            const int q = 2 * x + j;
            ok = wait(BAR_FULL + q % kSlots, q / kSlots) && *s_abort == 0;
            if (ok) mbar_arrive(bar(BAR_EMPTY + q % kSlots));
          }
        x += g.nt;
        ok = __all_sync(0xFFFFFFFFu, ok);
        continue;
      }
      if (lane == 0) {
        auto issue_s = [&](int j) {
          const int q = 2 * (x + j);
          if (!wait(BAR_FULL + q % kSlots, q / kSlots)) return false;
          tc_fence_after();
          const uint64_t ks = sdesc_sw128(slot_addr(q), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) umma_ss(s_col, q_base + kmaj_off(kk), ks + kmaj_off(kk), id_s, kk > 0 ? 1u : 0u);
          umma_commit(bar(BAR_EMPTY + q % kSlots));
          umma_commit(bar(BAR_SFULL + t));
          if (j == g.nt - 1) umma_commit(bar(BAR_QEMPTY + t));
          issued = true;
          return true;
        };
        ok = wait(BAR_QFULL + t, units) && issue_s(0);
        for (int j = 0; j < g.nt && ok; ++j) {
          const int q = 2 * (x + j) + 1;
          ok = wait(BAR_FULL + q % kSlots, q / kSlots) && wait(BAR_PFULL + t, y + j);
          // the unit's first PV overwrites O: the last unit's must have been read
          if (ok && j == 0 && units > 0) ok = wait(BAR_OEMPTY + t, units - 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vs = sdesc_sw128(slot_addr(q), 16384, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(o_col, s_col + kk * 8, vs + vmaj_off(kk), id_o, (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(bar(BAR_EMPTY + q % kSlots));
          umma_commit(bar(BAR_PVDONE + t));
          // S_(j+1) overwrites P_j
          ok = wait(BAR_PVDONE + t, y + j);
          if (ok && j + 1 < g.nt) ok = issue_s(j + 1);
          if (*s_abort) ok = false;
        }
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      x += g.nt;
      y += g.nt;
      ++units;
    }
    if (!ok) {
      *s_abort = 1;
      if (lane == 0 && issued) {  // products in flight complete before the CTA ends (bounded)
        umma_commit(bar(BAR_DRAIN + t));
        wait(BAR_DRAIN + t, 0);
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ Q
    int units[2] = {0, 0};
    const int chunk = lane % 16;  // 16 bytes of a row
    for (int k = 0; ok; ++k) {
      Segment g;
      ok = next_seg(k, g);
      if (!ok || !g.valid) break;
      for (int t = 0; t < 2 && ok; ++t) {
        if (g.rows <= 128 * t) continue;
        ok = units[t] == 0 || __all_sync(0xFFFFFFFFu, wait(BAR_QEMPTY + t, units[t] - 1));
        if (!ok) break;
        ++units[t];
        const uint32_t to = sbase + C::kOffQ + t * kQBytes + (chunk / 8) * 16384;
        int rho = g.rho0 + 128 * t + lane / 16;
        int i = rho / a.group, e = rho - i * a.group;
        const int real = g.rho0 + g.rows - rho;  // rows 0, 2, .. below this are
#pragma unroll 4
        for (int r = 0; r < 128; r += 2) {
          const bool is = r < real;
          const uint16_t* src = a.q;
          if (is)
            src += static_cast<int64_t>(g.row0 + i) * a.q_token + static_cast<int64_t>(g.h * a.group + e) * a.q_head +
                   chunk * 8;
          const int row = r + lane / 16;
          cp_async16(to + row * 128 + ((chunk % 8) ^ (row & 7)) * 16, src, is);
          e += 2;
          while (e >= a.group) {
            e -= a.group;
            ++i;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_QFULL + t));
      }
    }
    if (!ok) *s_abort = 1;
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax of tile t
    setmaxnreg_inc<C::kRegsSoftmax>();
    const int t = (warp - 4) / 4;
    const int row = (warp & 3) * 32 + lane;  // of the tile: a lane of tensor memory
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_addr + 128 * t, o_col = tmem + lane_addr + 256 + 128 * t;
    const float c2 = a.scale * 1.4426950408889634f;
    int x = 0, y = 0;
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
      const int i = rho / a.group;
      const int pos = g.len - g.n + i;
      // a row that does not exist has Q = 0: no mask, and no output
      const int lo = real ? row_lo(a, pos) : 0;
      const int hi = real ? (a.causal ? min(g.len, pos + 1) : g.len) : 0x7FFFFFFF;
      float ref = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < g.nt; ++j) {
        ok = __all_sync(0xFFFFFFFFu, wait(BAR_SFULL + t, y + j));
        if (!ok) break;
        tc_fence_after();
        const int key0 = (g.t0 + j) << kKeyShift;
        // BF16 pages: slots that no row sees may hold anything, and their V
        // must become zeros (their probabilities are 0, and 0 * NaN is not).
        // Both tiles' warps write them, each before its own products.
        if (kKind == 0 && (key0 < g.lo || key0 + kTileKeys > g.hi)) {
          const int q = 2 * (x + j) + 1;
          ok = __all_sync(0xFFFFFFFFu, wait(BAR_FULL + q % kSlots, q / kSlots));
          if (!ok) break;
          if (key0 + row < g.lo || key0 + row >= g.hi) {
            uint8_t* v = base + C::kOffRing + (q % kSlots) * kSlotBytes + row * 128;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              *reinterpret_cast<uint4*>(v + 16 * b) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(v + 16384 + 16 * b) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
        }
        // Pass 1 takes the maximum of the row's 128 scores, pass 2 reads them
        // again, 64 at a time, and turns them into P (fewer registers live).
        // Where the mask cuts the tile, pass 1 writes -inf back.
        float mx;
        {
          uint32_t s[128];
#pragma unroll
          for (int b = 0; b < 4; ++b) tmem_ld32(s_col + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * b]));
          tmem_wait_ld();
          if (!__all_sync(0xFFFFFFFFu, key0 >= lo && key0 + kTileKeys <= hi)) {
            const int a0 = lo - key0, a1 = hi - key0;
#pragma unroll
            for (int b = 0; b < 128; ++b)
              if (b < a0 || b >= a1) s[b] = __float_as_uint(-INFINITY);
#pragma unroll
            for (int b = 0; b < 4; ++b) tmem_st32(s_col + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * b]));
            tmem_wait_st();
          }
          mx = max128(s) * c2;  // (scale > 0)
        }
        const float prev = ref;
        if (prev == -INFINITY || mx > prev + kRescaleLog2) ref = fmaxf(prev, mx);
        const bool moved = prev != -INFINITY && ref != prev;
        if (__any_sync(0xFFFFFFFFu, moved)) {
          // O holds the tiles before j, all completed: S_j was issued after PV_(j-1)
          const float f = moved ? ex2_approx(prev - ref) : 1.0f;
          l *= f;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t o[32];
            tmem_ld32(o_col + 32 * b, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(o_col + 32 * b, o);
          }
        }
        const float neg = ref == -INFINITY ? 0.f : -ref;
        const uint64_t c2x = f2(c2, c2), negx = f2(neg, neg);
        uint64_t sum[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) sum[b] = f2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32], s[64];
          tmem_ld32(s_col + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
          tmem_ld32(s_col + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
          tmem_wait_ld();
#pragma unroll
          for (int b = 0; b < 32; ++b) {
            float x0, x1;
            unf2(ffma2(f2(__uint_as_float(s[2 * b]), __uint_as_float(s[2 * b + 1])), c2x, negx), x0, x1);
            const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
            sum[b & 3] = fadd2(sum[b & 3], f2(e0, e1));
            p[b] = pack_bf16x2(e0, e1);
          }
          tmem_st32(s_col + 32 * h, p);
        }
        {
          float z0, z1;
          unf2(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])), z0, z1);
          l += z0 + z1;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_PFULL + t));
        if (__any_sync(0xFFFFFFFFu, *s_abort != 0)) {
          ok = false;
          break;
        }
      }
      // ---- the unit's output, or this step's part of it
      ok = ok && __all_sync(0xFFFFFFFFu, wait(BAR_PVDONE + t, y + g.nt - 1));
      if (!ok) break;
      tc_fence_after();
      const int64_t at = g.part < 0 ? static_cast<int64_t>(g.row0 + i) * a.Hq + g.h * a.group + (rho - i * a.group)
                                    : (static_cast<int64_t>(blockIdx.x) * 2 + g.part) * kUnitRows + 128 * t + row;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (NaN stays)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t o[32];
        tmem_ld32(o_col + 32 * b, o);
        tmem_wait_ld();
        if (real) {
          if (g.part < 0) {
            uint4* dst = reinterpret_cast<uint4*>(a.o + at * kHeadDim + 32 * b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t z[4];
#pragma unroll
              for (int f = 0; f < 4; ++f)
                z[f] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * f]) * inv, __uint_as_float(o[8 * e + 2 * f + 1]) * inv);
              dst[e] = make_uint4(z[0], z[1], z[2], z[3]);
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(ws.part + at * kHeadDim + 32 * b);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
      if (real) {
        if (g.part >= 0)
          ws.ml[at] = make_float2(ref, l);
        else if (a.lse)
          a.lse[at] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_OEMPTY + t));
      x += g.nt;
      y += g.nt;
    }
    if (!ok) *s_abort = 1;
  } else if constexpr (kKind != 0) {
    // ------------------------------------------------------------ widening
    setmaxnreg_dec<C::kRegsConvert>();
    const int row = threadIdx.x - 384;  // a key of the tile
    int q = 0;
    for (int k = 0; ok; ++k) {
      Segment g;
      ok = next_seg(k, g);
      if (!ok || !g.valid) break;
      for (int j = 0; j < 2 * g.nt; ++j, ++q) {
        const int b = q % kStageSlots, slot = q % kSlots;
        ok = __all_sync(0xFFFFFFFFu, wait(BAR_SGFULL + b, q / kStageSlots));
        if (ok && q >= kSlots) ok = __all_sync(0xFFFFFFFFu, wait(BAR_EMPTY + slot, q / kSlots - 1));
        if (ok) ok = !__any_sync(0xFFFFFFFFu, *s_abort != 0);
        if (!ok) break;
        const int key = ((g.t0 + j / 2) << kKeyShift) + row;
        const bool seen = key >= g.lo && key < g.hi;  // else zeros, whatever was there
        const uint32_t e = base[C::kOffExp + b * kTileKeys + row];
        // codes land as the value times 2^-120; then the row's scale, a
        // power of two (NaN for 255; a byte of 0 is no exponent of cache_write)
        const uint32_t two = e == 255 ? 0x7FFF7FFFu : e * 0x00800080u;
        const uint8_t* src = base + C::kOffStage + b * kStageBytes + row * 128;
        uint8_t* dst = base + C::kOffRing + slot * kSlotBytes + row * 128;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + (ch ^ (row & 7)) * 16);
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t out[8];
#pragma unroll
          for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t p = __byte_perm(in[w], 0, h ? 0x3424 : 0x1404);  // a code in each upper byte
              const uint32_t z = ((p >> 4) & 0x07F007F0u) | (p & 0x80008000u);
              out[2 * w + h] = seen ? bf16x2_mul(bf16x2_mul(z, 0x7B807B80u), two) : 0u;
            }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int cc = 2 * ch + h;
            *reinterpret_cast<uint4*>(dst + (cc / 8) * 16384 + ((cc % 8) ^ (row & 7)) * 16) =
                make_uint4(out[4 * h], out[4 * h + 1], out[4 * h + 2], out[4 * h + 3]);
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
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) ws.cta_status[blockIdx.x] = *s_abort ? 5 /* SA_ETIMEOUT */ : (*s_bad ? kPagedInvalid : 0);
  griddep_launch_dependents();
}

template <int kKind>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, const PagedScratch& ws,
                   int ctas, cudaStream_t s) {
  using C = Cfg<kKind>;
  auto* kern = paged_chunk_kernel<kKind>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
  if (e != cudaSuccess) return e;
  // The register split redistributes the launch allocation; a build with
  // fewer registers a thread would make setmaxnreg.inc wait forever.
  static int regs = -1;
  if (regs < 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  const int split = C::kRegsControl + 2 * C::kRegsSoftmax + (kKind ? C::kRegsConvert : 0);
  if (regs * (C::kThreads / 128) < split) return cudaErrorInvalidConfiguration;
  kern<<<ctas, C::kThreads, C::kSmem, s>>>(tk, tv, a, ws);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_chunk(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a,
                               const PagedScratch& ws, int ctas, cudaStream_t s) {
  return a.c.kind == 0 ? launch<0>(tk, tv, a, ws, ctas, s) : launch<1>(tk, tv, a, ws, ctas, s);
}

}  // namespace sa
