// Attention over a paged cache for few rows a sequence and key head: single
// tokens and short drafts (at most 16 packed rows), sm_103a.
//
//   o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),   x_j = scale log2(e) (q . k_j)
//
// Every cached row is used once for all rows of the unit, so the kernel is
// bound by memory: 512 bytes a token and key head (258 in the E4M3 kind)
// against 8 or 16 rows' worth of products.  What it needs is many bytes in
// flight and an even share for every SM however ragged the batch is: the line
// of all key tiles is cut into equal parts, one a CTA (paged.cuh), and each
// CTA streams its part through a ring of 64-key stages of K and V.  A
// producer warp fills the ring with TMA boxes, one a page (the keys of one
// page and head are contiguous), and each consumer warp takes 16 keys of a
// stage, with a softmax reference, sum and output of its own until the unit's
// keys end: nothing passes between warps inside the loop.
//
// Products are mma.sync m16n8k16 with the keys (then the dimensions) as M and
// eight rows as N:  S^T = K Q^T,  O^T = V^T P^T.  A tcgen05 instruction takes
// 128 rows, of which seven eighths or more would be padding, and here the
// tensor pipe is not what bounds; with the rows as M, eight of sixteen would
// still be.  P^T leaves the first product's accumulators as pairs of rows and
// enters the second as pairs of keys: one movmatrix for eight keys.
//
// E4M3 (exact in both products).  K: two cvt make four FP16 values of a word;
// Q is held in FP16 too, each row scaled by a power of two that brings its
// largest magnitude to 2^13 or 2^14: exact down to 2^-30 of that (FP16's
// subnormals hold BF16's 8 bits from 2^-17 on); smaller ones lose bits and
// vanish below 2^-38 of it, which shows only where a key is 0 in every
// dimension that is larger.  V: BF16, since a probability times its key's
// scale can leave FP16's range; a word's codes c0..c3 are two dimensions of two keys,
// and exponent and fraction shifted into place, times a power of two, give the pairs
// (c0, c2) and (c1, c3) without a byte permutation.  A key's scale is a power
// of two: K's multiplies the logit, V's the probability.  So that the latter
// stays in BF16's normal range as far down as can be, probabilities are 2^7
// times what they are in the BF16 kind, and V's codes 2^-7 times: a key of
// probability p keeps all 8 bits of it for scales down to 2^-126 / p.
//
// Two CTAs an SM: four consumer warps and three stages of 32 KB, or, for up
// to eight rows over E4M3 pages, where the widening takes more instructions
// than the products, eight warps (four on every other stage) and six of 16 KB.
// (For sixteen rows eight warps leave 96 registers, 64 of them accumulators:
// 366 us against 229 for 64 sequences of 8704 keys.)
//
// Measured (bytes of the cached keys a second; a copy reaches 6.78 TB/s):
//   64 sequences of 512 to 33792 keys, 40 / 8 heads, BF16, one new   238 us  6.79 TB/s
//   96 of them, 56 / 8 heads, E4M3, one new                          268 us  6.25
//   64 of 8704, 24 / 8 heads, four new (12 rows): BF16               348 us  6.56
//                                                 E4M3               229 us  5.02
// The last is bound by the instructions of the widening and of two products.
// Small calls are bound by what comes once: about 2 us until the line is
// walked, 1.5 us for joining the warps, and the
// joining kernel (16 sequences of 300 to 8704 keys, window 4096, 24 / 8 heads,
// E4M3, four new: 25.4 us in a graph of such calls, of which the keys' bytes
// are 10).  Code that runs
// once is fetched as it runs, about 100 cycles for every eight instructions,
// so a unit's beginning and end are kept short.
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kKeyShift = 6;  // 64 keys a stage
constexpr int kTileKeys = kPagedFewKeys;
static_assert(kTileKeys == 1 << kKeyShift, "");
constexpr uint32_t kQRow = 272;  // bytes of a row of Q in shared memory (256 and padding: other banks for each row)
// The reference follows a row's maximum only when that passes it, and then by
// this much more (log2), so that O is seldom rescaled.  Probabilities relative
// to it are at most 1: a sum of them times values overflows only where the one
// relative to the maximum itself would.
constexpr float kLead = 7.0f;
// A unit's beginning (its Q) and end (joining the warps), in stages.
constexpr int kOverBf16 = 2, kOverE4m3 = 3;
constexpr uint32_t kRegionBytes = 4096;  // of the merge area: 8 rows x 128 floats

template <int kKind, int kN>
struct Cfg {
  // Probabilities reach 2^kTop: what V's codes are short of (E4M3).
  static constexpr float kTop = kKind == 0 ? 0.0f : 7.0f;
  static constexpr int kGroups = kKind == 1 && kN == 1 ? 2 : 1;  // of four consumer warps, on stages in turn
  static constexpr int kConsumers = 4 * kGroups;
  static constexpr int kThreads = 32 * (kConsumers + 1);
  // Every stage belongs to one group: a group that skipped phases of a stage
  // could take the phase before the awaited one for it.
  static constexpr int kStages = kKind == 0 ? 3 : 6;
  static_assert(kStages % kGroups == 0, "stages of a group");
  static constexpr uint32_t kRow = kKind == 0 ? 256 : 128;            // bytes of a cached row
  static constexpr uint32_t kHalf = kTileKeys * kRow;                 // K or V of a stage
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kExp = kKind == 0 ? 0 : 2 * kTileKeys;    // exponent bytes of a stage
  // Shared memory, from a 1024-byte boundary.
  static constexpr uint32_t kOffExp = kStages * kStage;
  static constexpr uint32_t kOffMerge = kOffExp + kStages * kExp;     // kRegions x 8 rows
  static constexpr int kRegions = 2;
  static constexpr int kSegs = kN == 1 ? 2 : 1;                       // steps described ahead, with their Q
  static constexpr uint32_t kQBytes = 8 * kN * kQRow;
  static constexpr uint32_t kOffQ = kOffMerge + kRegions * kRegionBytes;
  static constexpr uint32_t kOffMl = kOffQ + kSegs * kQBytes;  // [8 warps][16 rows] float2, then by row
  static constexpr uint32_t kOffSeg = kOffMl + 1024 + 16 * 24 + 64;       // kSegs x Segment
  static constexpr uint32_t kOffBar = kOffSeg + kSegs * 64;
  static constexpr uint32_t kOffMisc = kOffBar + 256;
  static constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
};
static_assert(sizeof(Segment) <= 64, "");

enum { BAR_FULL = 0, BAR_EMPTY = 8, BAR_SFULL = 16, BAR_SEMPTY = 20, NUM_BARS = 24 };

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_b32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_f4(uint32_t addr, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
template <bool kHalfs>  // FP16 operands, else BF16
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (kHalfs)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes (c0, c2) and (c1, c3) of a word as BF16 pairs: the seven magnitude
// bits land on BF16's exponent and upper fraction as the value times 2^-120
// (subnormal codes as subnormals); what is returned is the value times 2^-7.
__device__ __forceinline__ uint32_t times_2_113(uint32_t v) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x78007800u));
  return d;
}
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
  return times_2_113(((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u));
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
  return times_2_113(((w >> 4) & 0x07F007F0u) | (w & 0x80008000u));
}
// Codes (c0, c1) and (c2, c3) as FP16 pairs.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// The consumers meet (barrier 1) and agree: true for all when it is for one
// (a wait that gave up in one warp must not leave the others at a barrier).
template <int kThreads>
__device__ __forceinline__ bool bar_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "n"(kThreads)
      : "memory");
  return r != 0;
}
template <int kThreads>
__device__ __forceinline__ void bar_all() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

template <int kKind, int kN>  // kN: tiles of eight rows
__global__ void __launch_bounds__(Cfg<kKind, kN>::kThreads, 2)
paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const PagedAttnArgs a, const PagedScratch ws) {
  using C = Cfg<kKind, kN>;
  constexpr int kRows = 8 * kN, kSegs = C::kSegs;
  constexpr int kWorkers = 32 * C::kConsumers;
  const PagedArgs& c = a.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(base);
  auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * i; };
  Segment* segs = reinterpret_cast<Segment*>(base + C::kOffSeg);
  volatile int32_t* s_abort = reinterpret_cast<volatile int32_t*>(base + C::kOffMisc);
  int32_t* s_bad = reinterpret_cast<int32_t*>(base + C::kOffMisc + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    *s_abort = 0;
    *s_bad = 0;
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(bar(BAR_FULL + i), 1);
      mbar_init(bar(BAR_EMPTY + i), 4);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(bar(BAR_SFULL + i), 33);  // the description; 32 lanes' copies of Q
      mbar_init(bar(BAR_SEMPTY + i), C::kConsumers);
    }
    fence_barrier_init();
  }
  __syncthreads();
  // Token of a packed row: there are at most 16, so FP32 divides exactly (and
  // takes the fewest registers).
  const float inv_group = 1.0f / static_cast<float>(a.group);
  auto token_of = [&](int row) { return static_cast<int>((static_cast<float>(row) + 0.5f) * inv_group); };
  int seq = 0, steps = 0;  // producer: stages and descriptions so far

  if (warp == C::kConsumers) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    LineWalk w;
    bool bad = false;
    using Line = LineShape<kRows, kTileKeys, 1, 1, kKind == 0 ? kOverBf16 : kOverE4m3, 1, true>;
    walk_begin<Line>(a, w, blockIdx.x, gridDim.x, bad);
    JoinDesc join;
    join.pieces = 0;
    bool ok = true;
    int stage = 0;
    const int per_page = min(c.page_size, kTileKeys);        // keys of a tile in one page
    const int tile_pages = kTileKeys / per_page;
    const uint32_t elect = elect_one();
    for (int k = 0; ok; ++k) {
      const Segment g = walk_next<Line>(a, w, blockIdx.x, join);
      ok = k < kSegs ||
           __all_sync(0xFFFFFFFFu, mbar_wait(bar(BAR_SEMPTY + k % kSegs), ((k / kSegs) & 1) ^ 1, a.wait_limit));
      if (!ok) break;
      // pages of this step's tiles, 32 table entries at a time (the first load
      // is under way while Q's are issued)
      const int p_lo = g.lo >> c.page_shift, p_hi = (g.hi + c.page_size - 1) >> c.page_shift;
      int have = g.valid ? (g.t0 << kKeyShift >> c.page_shift) / 32 : 0;  // entry: page index 32 * have + lane
      const int32_t* table = c.table + (g.valid ? g.s * c.table_stride : 0);
      auto fetch = [&] {
        const int at = have * 32 + lane;
        return at >= p_lo && at < p_hi ? __ldg(table + at) : 0;
      };
      auto checked = [&](int e) {
        const bool wrong = e < 0 || e >= c.pages;
        bad |= wrong;
        return wrong ? -1 : e;
      };
      int entry = 0;
      if (g.valid) {  // (a unit is one row tile here: rho0 is 0)
        entry = fetch();
#pragma unroll
        for (int x = 0; x < kRows / 2; ++x) {
          const int row = 2 * x + lane / 16, i = token_of(row);
          const uint16_t* src = a.q;
          if (row < g.rows)
            src += static_cast<int64_t>(g.row0 + i) * a.q_token +
                   static_cast<int64_t>(g.h * a.group + row - i * a.group) * a.q_head + lane % 16 * 8;
          cp_async16(sbase + C::kOffQ + k % kSegs * C::kQBytes + row * kQRow + lane % 16 * 16, src, row < g.rows);
        }
      }
      cp_async_arrive(bar(BAR_SFULL + k % kSegs));
      if (lane == 0) {
        segs[k % kSegs] = g;
        mbar_arrive(bar(BAR_SFULL + k % kSegs));
      }
      ++steps;
      if (!g.valid) break;
      entry = checked(entry);
      for (int t = g.t0; t < g.t0 + g.nt; ++t) {
        const int key0 = t << kKeyShift;
        const int page0 = key0 >> c.page_shift;
        if (page0 / 32 != have) {
          have = page0 / 32;
          entry = checked(fetch());
        }
        // lane i: row of the cache where the tile's i-th page begins (-1: not to be loaded)
        const int at = page0 + lane;
        const int page = __shfl_sync(0xFFFFFFFFu, entry, at % 32);
        const bool mine = lane < tile_pages && at >= p_lo && at < p_hi && page >= 0;
        const int row = mine ? static_cast<int>(((static_cast<int64_t>(page) * c.H + g.h) << c.page_shift) +
                                                (key0 & (c.page_size - 1)))
                             : -1;
        const int loads = __popc(__ballot_sync(0xFFFFFFFFu, mine));
        int rows[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = __shfl_sync(0xFFFFFFFFu, row, i);
        ok = seq < C::kStages || __all_sync(0xFFFFFFFFu, mbar_wait(bar(BAR_EMPTY + stage),
                                                                  ((seq / C::kStages) & 1) ^ 1, a.wait_limit));
        if (!ok) break;
        if (elect) {
          mbar_arrive_expect_tx(bar(BAR_FULL + stage), loads * per_page * (2 * C::kRow + (kKind ? 2 : 0)));
          const uint32_t to = sbase + stage * C::kStage;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (rows[i] < 0) continue;
            if constexpr (kKind == 0) {
              tma_load_4d(to + i * per_page * C::kRow, &tm_k, bar(BAR_FULL + stage), 0, 0, 0, rows[i] / 8);
              tma_load_4d(to + C::kHalf + i * per_page * C::kRow, &tm_v, bar(BAR_FULL + stage), 0, 0, 0, rows[i] / 8);
            } else {
              tma_load_2d(to + i * per_page * C::kRow, &tm_k, bar(BAR_FULL + stage), 0, rows[i]);
              tma_load_2d(to + C::kHalf + i * per_page * C::kRow, &tm_v, bar(BAR_FULL + stage), 0, rows[i]);
              // (by the same lane: copies of eight lanes through their registers' path cost 8% of the call)
              const uint32_t ex = sbase + C::kOffExp + stage * C::kExp + i * per_page;
              bulk_load(ex, c.k_exp + rows[i], per_page, bar(BAR_FULL + stage));
              bulk_load(ex + kTileKeys, c.v_exp + rows[i], per_page, bar(BAR_FULL + stage));
            }
          }
        }
        __syncwarp();
        ++seq;
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
        ok = !__any_sync(0xFFFFFFFFu, *s_abort != 0);
        if (!ok) break;
      }
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (!ok) *s_abort = 1;
    if (lane == 0) {
      ws.join[blockIdx.x] = join;
      if (bad) *s_bad = 1;
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int u = lane / 4, t4 = lane % 4;
    const int quarter = warp % 4, grp = warp / 4;  // 16 keys of the stages that are the group's
    float2* s_ml = reinterpret_cast<float2*>(base + C::kOffMl);  // [warp][row]: reference, sum
    float2* s_row = s_ml + 8 * 16;                                  // [row]: of all warps
    int64_t* s_at = reinterpret_cast<int64_t*>(s_row + 16);         // [row]: where its output goes
    float* s_inv = reinterpret_cast<float*>(s_at + 16);             // [row]: its factor
    float* s_qinv = s_inv + 16;                                     // [row]: 2^(-e / 2) of its Q
    const float c2 = a.scale * 1.4426950408889634f;
    // ldmatrix rows: lane l gives row l % 8 of matrix l / 8.  K: (keys 0-7,
    // chunk i), (8-15, i), (0-7, i + 1), (8-15, i + 1); V the same in the
    // E4M3 kind, else (0-7, i), (0-7, i + 1), (8-15, i), (8-15, i + 1).
    const int mrow = lane % 8, mat = lane / 8;
    const int krow = 16 * quarter + (mat & 1) * 8 + mrow, kchunk = mat / 2;
    const int vrow = kKind == 0 ? 16 * quarter + (mat / 2) * 8 + mrow : krow;
    const int vchunk = kKind == 0 ? (mat & 1) : kchunk;
    auto chunk_at = [](int row, int chunk) -> uint32_t {
      if (kKind == 0) return (row / 8) * 2048 + (chunk / 8) * 1024 + (row % 8) * 128 + ((chunk % 8) ^ (row & 7)) * 16;
      return row * 128 + (chunk ^ (row & 7)) * 16;
    };
    // 128 bytes of a V row in a stage: of the second half of the dimensions if `half`
    auto half_row = [](int row, int half) -> uint32_t {
      return kKind == 0 ? (row / 8) * 2048 + half * 1024 + (row % 8) * 128 : row * 128;
    };
    bool ok = true;
    int tile = 0;  // tiles of the CTA so far
    for (int k = 0; ok; ++k) {
      ok = !bar_any<kWorkers>(!mbar_wait(bar(BAR_SFULL + k % kSegs), (k / kSegs) & 1, a.wait_limit));
      if (!ok) break;
      const Segment g = segs[k % kSegs];
      if (!g.valid) break;
      const uint32_t q_rows = sbase + C::kOffQ + k % kSegs * C::kQBytes;
      if constexpr (kKind != 0) {
        // Q in FP16, in place, a warp a row: a lane has dimensions 4 lane ..
        // of it, and within 16 the pairs get K's order (first the first two
        // codes of each word).
#pragma unroll 1
        for (int row = warp; row < kRows; row += C::kConsumers) {
          const uint32_t at = q_rows + row * kQRow;
          const uint32_t q0 = lds_b32(at + 8 * lane), q1 = lds_b32(at + 8 * lane + 4);
          const uint32_t m2 = __vmaxu2(q0 & 0x7FFF7FFFu, q1 & 0x7FFF7FFFu);
          const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(m2 >> 16, m2 & 0xFFFFu));
          // largest magnitude 2^(E - 127): times 2^(141 - E) or half of it (e is even), at most 2^126
          const int e = min(126, (141 - static_cast<int>(m >> 7)) & ~1);
          const float f = pow2(e);
          const uint32_t to = at + lane / 4 * 32 + lane % 4 * 4;
          sts_b32(to, pack_f16x2(bf_lo(q0) * f, bf_hi(q0) * f));
          sts_b32(to + 16, pack_f16x2(bf_lo(q1) * f, bf_hi(q1) * f));
          if (lane == 0) s_qinv[row] = pow2(-e / 2);
        }
        bar_all<kWorkers>();
      }
      // Q as the second operand: row u of each tile, dimensions 2t, 2t + 1
      // and 2t + 8, 2t + 9 of 16
      uint32_t qf[kN][8][2];
      float qinv[kN][2];  // E4M3: its square undoes the scaling of rows 2t, 2t + 1
#pragma unroll
      for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int kk = 0; kk < 8; kk += 2) {
          uint32_t b[4];
          ldsm4(b, q_rows + (8 * n + lane % 8) * kQRow + kk * 32 + lane / 8 * 16);
          qf[n][kk][0] = b[0];
          qf[n][kk][1] = b[1];
          qf[n][kk + 1][0] = b[2];
          qf[n][kk + 1][1] = b[3];
        }
        if constexpr (kKind != 0) {
          qinv[n][0] = s_qinv[8 * n + 2 * t4];
          qinv[n][1] = s_qinv[8 * n + 2 * t4 + 1];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_SEMPTY + k % kSegs));
      // keys that this thread's rows 2t, 2t + 1 of each tile see
      int lo[kN][2], hi[kN][2];
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * n + 2 * t4 + e;
          const int pos = g.len - g.n + token_of(row);
          lo[n][e] = row < g.rows ? row_lo(a, pos) : 0;
          hi[n][e] = row < g.rows ? (a.causal ? min(g.len, pos + 1) : g.len) : 0;
        }
      float acc[kN][8][4], ref[kN][2], sum[kN][2];
#pragma unroll
      for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ref[n][e] = -INFINITY;
          sum[n][e] = 0.f;
        }
      }
      const int step = C::kGroups;
      const int skip = (grp - tile % C::kGroups + C::kGroups) % C::kGroups;  // the group's first tile of this unit
#pragma unroll 1
      for (int t = skip; t < g.nt; t += step) {
        const int use = tile + t, stage = use % C::kStages;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(BAR_FULL + stage), (use / C::kStages) & 1, a.wait_limit));
        if (!ok) break;
        const uint32_t sk = sbase + stage * C::kStage, sv = sk + C::kHalf;
        const int key0 = ((g.t0 + t) << kKeyShift) + 16 * quarter;
        // Slots that no row sees may hold anything: this warp's V rows there
        // become zeros (their probabilities are 0, and 0 * NaN is not).
        const bool ragged = key0 < g.lo || key0 + 16 > g.hi;
        if (ragged) {
          const int x = lane / 2;
          if (key0 + x < g.lo || key0 + x >= g.hi) {
            const uint32_t v = sv + half_row(16 * quarter + x, lane % 2) + (kKind == 0 ? 0 : (lane % 2) * 64);
#pragma unroll
            for (int i = 0; i < (kKind == 0 ? 8 : 4); ++i) sts_f4(v + 16 * i, make_float4(0.f, 0.f, 0.f, 0.f));
          }
          __syncwarp();
        }
        // ---- S^T = K Q^T: keys u and u + 8, rows 2t and 2t + 1
        float s[kN][4];
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < (kKind == 0 ? 8 : 4); ++kk) {
          uint32_t b[4];
          ldsm4(b, sk + chunk_at(krow, 2 * kk + kchunk));
          if constexpr (kKind == 0) {
#pragma unroll
            for (int n = 0; n < kN; ++n) mma<false>(s[n], b[0], b[1], b[2], b[3], qf[n][kk][0], qf[n][kk][1]);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // 16 dimensions of chunk 2 kk + i
              uint32_t l0, h0, l1, h1;
              codes_f16(b[2 * i], l0, h0);
              codes_f16(b[2 * i + 1], l1, h1);
#pragma unroll
              for (int n = 0; n < kN; ++n)
                mma<true>(s[n], l0, l1, h0, h1, qf[n][2 * kk + i][0], qf[n][2 * kk + i][1]);
            }
          }
        }
        // A key's scale as two factors of half its exponent, as Q's: the
        // product of one of each is a number, whatever the two scales are, and
        // a logit leaves FP32's range on the way only if it does in the end.
        float ks[2][2];
        float vs[2];
        if constexpr (kKind != 0) {
          const uint8_t* ex = base + C::kOffExp + stage * C::kExp + 16 * quarter + u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = ex[8 * e], half = k >> 1;
            ks[e][0] = pow2(half - 64);
            ks[e][1] = (k - 1u < 254u ? pow2(k - half - 63) : exp_scale(k)) * c2;
            vs[e] = exp_scale(ex[kTileKeys + 8 * e]);
          }
        }
        const bool cut = ragged || key0 < g.all_lo || key0 + 16 > g.all_hi;  // some row misses some key
        // BF16, rows of several tokens: a value of a key that one row sees and
        // another does not must not reach that other one as 0 * NaN or
        // 0 * infinity.  Keys with such values (a bit each) are left out of
        // the product and added one by one.
        uint32_t odd_keys = 0;
        if (kKind == 0 && cut && g.n > 1) {
          const uint32_t v = sv + half_row(16 * quarter + lane / 2, lane % 2);
          uint32_t m2 = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 f = lds_f4(v + 16 * i);
            m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(__float_as_uint(f.x) & 0x7FFF7FFFu, __float_as_uint(f.y) & 0x7FFF7FFFu),
                                       __vmaxu2(__float_as_uint(f.z) & 0x7FFF7FFFu, __float_as_uint(f.w) & 0x7FFF7FFFu)));
          }
          const uint32_t by_lane = __ballot_sync(0xFFFFFFFFu, (m2 >> 16) >= 0x7F80u || (m2 & 0xFFFFu) >= 0x7F80u);
          odd_keys = (by_lane | by_lane >> 1) & 0x55555555u;  // key x at bit 2x
        }
        uint32_t p[kN][2];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (kKind == 0)
              s[n][e] *= c2;
            else
              s[n][e] = s[n][e] * (qinv[n][e & 1] * ks[e / 2][0]) * (qinv[n][e & 1] * ks[e / 2][1]);
          }
          if (cut) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + u + 8 * (e / 2);
              if (key < lo[n][e & 1] || key >= hi[n][e & 1]) s[n][e] = -INFINITY;
            }
          }
          // The lanes need not agree on a maximum before some key passes the
          // reference (by 2^kTop).
          float mx[2] = {fmaxf(s[n][0], s[n][2]), fmaxf(s[n][1], s[n][3])};
          if (__any_sync(0xFFFFFFFFu, mx[0] > ref[n][0] + C::kTop || mx[1] > ref[n][1] + C::kTop)) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int d = 4; d < 32; d *= 2) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], d));
              const float to = mx[e] > ref[n][e] + C::kTop ? mx[e] + (kLead - C::kTop) : ref[n][e];
              f[e] = to == ref[n][e] ? 1.f : ex2_approx(ref[n][e] - to);  // the first keys: 2^-inf = 0
              ref[n][e] = to;
              sum[n][e] *= f[e];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[n][i][e] *= f[e & 1];
          }
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = ex2_approx(s[n][e] - (ref[n][e & 1] == -INFINITY ? 0.f : ref[n][e & 1]));
            sum[n][e & 1] += x;
            // (a hidden key's scale may be NaN; that of a key which is seen counts whatever its probability)
            y[e] = kKind == 0 ? x : (s[n][e] == -INFINITY ? 0.f : x * vs[e / 2]);
          }
          p[n][0] = transpose8(pack_bf16x2(y[0], y[1]));
          p[n][1] = transpose8(pack_bf16x2(y[2], y[3]));
          for (uint32_t left = odd_keys; left; left &= left - 1) {
            const int x = (__ffs(left) - 1) / 2;  // key of the sixteen
            const int from = (x % 8) * 4 + t4;    // the lane that has its probabilities of this thread's rows
            const float p0 = __shfl_sync(0xFFFFFFFFu, x < 8 ? y[0] : y[2], from);
            const float p1 = __shfl_sync(0xFFFFFFFFu, x < 8 ? y[1] : y[3], from);
            const bool see0 = key0 + x >= lo[n][0] && key0 + x < hi[n][0];
            const bool see1 = key0 + x >= lo[n][1] && key0 + x < hi[n][1];
            const int row = 16 * quarter + x;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // dimension 16 j + 8 e + u
                uint16_t b;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(sv + chunk_at(row, 2 * j + e) + 2 * u));
                const float v = __uint_as_float(static_cast<uint32_t>(b) << 16);
                if (see0) acc[n][j][2 * e] = fmaf(p0, v, acc[n][j][2 * e]);
                if (see1) acc[n][j][2 * e + 1] = fmaf(p1, v, acc[n][j][2 * e + 1]);
              }
          }
        }
        if (odd_keys) {
          __syncwarp();
          if ((odd_keys >> (lane & ~1)) & 1) {
            const uint32_t v = sv + half_row(16 * quarter + lane / 2, lane % 2);
#pragma unroll
            for (int i = 0; i < 8; ++i) sts_f4(v + 16 * i, make_float4(0.f, 0.f, 0.f, 0.f));
          }
          __syncwarp();
        }
        // ---- O^T += V^T P^T: dimensions u, u + 8 of 16 (2u, 2u + 1 in the E4M3 kind)
#pragma unroll
        for (int j = 0; j < (kKind == 0 ? 8 : 4); ++j) {
          uint32_t b[4];
          ldsm4_t(b, sv + chunk_at(vrow, 2 * j + vchunk));
          if constexpr (kKind == 0) {
#pragma unroll
            for (int n = 0; n < kN; ++n) mma<false>(acc[n][j], b[0], b[1], b[2], b[3], p[n][0], p[n][1]);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t e0 = codes_even(b[2 * i]), o0 = codes_odd(b[2 * i]);
              const uint32_t e1 = codes_even(b[2 * i + 1]), o1 = codes_odd(b[2 * i + 1]);
#pragma unroll
              for (int n = 0; n < kN; ++n) mma<false>(acc[n][2 * j + i], e0, o0, e1, o1, p[n][0], p[n][1]);
            }
          }
        }
        if (ragged || odd_keys) fence_proxy_async_smem();  // zeros written here, TMA writes next
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_EMPTY + stage));
      }
      tile += g.nt;
      // ---- the warps' results into one: references and sums first
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) sum[n][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][e], d);
          if constexpr (kKind != 0) {  // relative to the reference that the outputs have
            ref[n][e] += C::kTop;
            sum[n][e] *= 1.0f / 128;
          }
          if (u == 0) s_ml[warp * kRows + 8 * n + 2 * t4 + e] = make_float2(ref[n][e], sum[n][e]);
        }
      ok = !bar_any<kWorkers>(!ok || *s_abort != 0);
      if (!ok) break;
      if (warp == 0) {  // a row over all warps: 32 / kRows lanes share them
        constexpr int kSteps = C::kConsumers * kRows / 32;
        float2 ml[kSteps];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          ml[i] = s_ml[i * 32 + lane];  // [warp][row]
          m = fmaxf(m, ml[i].x);
        }
#pragma unroll
        for (int d = kRows; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
#pragma unroll
        for (int i = 0; i < kSteps; ++i)  // (a warp without a reference has the sum 0, or NaN if its logits are)
          l += ml[i].x == -INFINITY ? ml[i].y : ml[i].y * ex2_approx(ml[i].x - m);
#pragma unroll
        for (int d = kRows; d < 32; d *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        if (lane < kRows) s_row[lane] = make_float2(m, l);
      }
      bar_all<kWorkers>();
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        float f[2];  // rows 8n + 2t, 2t + 1
#pragma unroll
        for (int e = 0; e < 2; ++e)
          f[e] = ref[n][e] == -INFINITY ? 0.f : ex2_approx(ref[n][e] - s_row[8 * n + 2 * t4 + e].x);
        // (the last warp's turn comes last: meanwhile, what concerns whole rows)
        if (n == 0 && warp == C::kConsumers - 1 && lane < kRows) {
          const float2 ml = s_row[lane];
          const int i = token_of(lane);
          const bool real = lane < g.rows;
          const int64_t at = g.part < 0 ? static_cast<int64_t>(g.row0 + i) * a.Hq + g.h * a.group + lane - i * a.group
                                        : (static_cast<int64_t>(blockIdx.x) * 2 + g.part) * kRows + lane;
          s_at[lane] = real ? at * kHeadDim : -1;
          s_inv[lane] = g.part >= 0 ? 1.f : ml.y > 0.f ? 1.f / ml.y : (ml.y == 0.f ? 0.f : ml.y);  // (NaN stays)
          if (real && g.part >= 0) ws.ml[at] = ml;
          if (real && g.part < 0 && a.lse)
            a.lse[at] = ml.y == 0.f ? -INFINITY : (ml.x + log2f(ml.y)) * 0.6931471805599453f;
        }
        // The outputs, in the accumulators' own order (a float4 of 16
        // dimensions j for each lane): warp after warp adds to its region.
        const uint32_t mine = sbase + C::kOffMerge + (warp % C::kRegions) * kRegionBytes + lane * 16;
#pragma unroll 1
        for (int gr = 0; gr < C::kConsumers / C::kRegions; ++gr) {
          if (warp / C::kRegions == gr) {
#pragma unroll
            for (int j0 = 0; j0 < 8; j0 += 4) {
              float4 y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (gr > 0) y[j] = lds_f4(mine + (j0 + j) * 512);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float(&c4)[4] = acc[n][j0 + j];
                sts_f4(mine + (j0 + j) * 512, make_float4(fmaf(c4[0], f[0], y[j].x), fmaf(c4[1], f[1], y[j].y),
                                                          fmaf(c4[2], f[0], y[j].z), fmaf(c4[3], f[1], y[j].w)));
              }
            }
          }
          bar_all<kWorkers>();
        }
        // Each warp writes 8 / kConsumers of the 8 times 16 dimensions.
        int64_t at[2];
        float inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          at[e] = s_at[8 * n + 2 * t4 + e];
          inv[e] = s_inv[8 * n + 2 * t4 + e];
        }
#pragma unroll
        for (int x = 0; x < 8 / C::kConsumers; ++x) {
          const int j = warp * (8 / C::kConsumers) + x;
          float4 y = lds_f4(sbase + C::kOffMerge + lane * 16 + j * 512);
#pragma unroll
          for (int w = 1; w < C::kRegions; ++w) {
            const float4 z = lds_f4(sbase + C::kOffMerge + w * kRegionBytes + lane * 16 + j * 512);
            y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
          }
          y.x *= inv[0];
          y.y *= inv[1];
          y.z *= inv[0];
          y.w *= inv[1];
          // two neighbouring dimensions of a row: d and d + 1
          auto put = [&](int e, int d, float lo, float hi) {
            const int64_t to = (e ? at[1] : at[0]) + d;
            if ((e ? at[1] : at[0]) < 0) return;  // no such row
            if (g.part < 0)
              *reinterpret_cast<uint32_t*>(a.o + to) = pack_bf16x2(lo, hi);
            else
              *reinterpret_cast<float2*>(ws.part + to) = make_float2(lo, hi);
          };
          if constexpr (kKind != 0) {  // the lane has dimensions 2u, 2u + 1 of both rows
            put(0, 16 * j + 2 * u, y.x, y.z);
            put(1, 16 * j + 2 * u, y.y, y.w);
          } else {  // dimensions u and u + 8: lanes u and u ^ 1 exchange rows
            const bool odd = u & 1;
            const float a0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? y.x : y.y, 4);
            const float a1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? y.z : y.w, 4);
            put(odd, 16 * j + (u & ~1), odd ? a0 : y.x, odd ? y.y : a0);
            put(odd, 16 * j + 8 + (u & ~1), odd ? a1 : y.z, odd ? y.w : a1);
          }
        }
        if (n + 1 < kN) bar_all<kWorkers>();  // (the next unit's first barrier otherwise)
      }
    }
    if (!ok) *s_abort = 1;
  }
  __syncthreads();
  // Where a warp has given up, nobody may have waited for the last loads: they
  // land before the CTA ends (bounded).  Only here is it known: the producer
  // may have issued all its loads before another warp's wait fails.
  if (warp == C::kConsumers && *s_abort) {
    for (int k = max(0, steps - kSegs); k < steps; ++k)
      mbar_wait(bar(BAR_SFULL + k % kSegs), (k / kSegs) & 1, kWaitLimitNs);
    for (int q = max(0, seq - C::kStages); q < seq; ++q)
      mbar_wait(bar(BAR_FULL + q % C::kStages), (q / C::kStages) & 1, kWaitLimitNs);
  }
  if (threadIdx.x == 0) ws.cta_status[blockIdx.x] = *s_abort ? 5 /* SA_ETIMEOUT */ : (*s_bad ? kPagedInvalid : 0);
  griddep_launch_dependents();
}

template <int kKind, int kN>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, const PagedScratch& ws,
                   int ctas, cudaStream_t s) {
  using C = Cfg<kKind, kN>;
  static SmemOnce once;
  const cudaError_t e = once.set(reinterpret_cast<const void*>(paged_few_kernel<kKind, kN>), C::kSmem);
  if (e != cudaSuccess) return e;
  paged_few_kernel<kKind, kN><<<ctas, C::kThreads, C::kSmem, s>>>(tk, tv, a, ws);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_few(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a,
                             const PagedScratch& ws, int row_tile, int ctas, cudaStream_t s) {
  if (a.c.kind == 0)
    return row_tile == 8 ? launch<0, 1>(tk, tv, a, ws, ctas, s) : launch<0, 2>(tk, tv, a, ws, ctas, s);
  return row_tile == 8 ? launch<1, 1>(tk, tv, a, ws, ctas, s) : launch<1, 2>(tk, tv, a, ws, ctas, s);
}

}  // namespace sa
