// Attention over a paged cache for few rows a sequence and key head: single
// tokens and short drafts (at most 32 packed rows), sm_103a.
//
//   o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),   x_j = scale log2(e) (q . k_j)
//
// Every cached row is used once for all rows of the unit, so the kernel is
// bound by memory: 512 bytes a token and key head (258 in the E4M3 kind)
// against 16 to 32 rows' worth of products.  What it needs is many bytes in
// flight and an even share for every SM however ragged the batch is: the line
// of all key tiles is cut into equal parts, one a CTA (paged.cuh), and each
// CTA streams its part through a ring of 64-key stages of K and V.  A
// producer warp fills the ring with TMA boxes, one a page (64 keys of one
// page and head are contiguous), and four warps take 16 keys of a stage each,
// with a softmax reference, sum and output of their own until the unit's keys
// end: nothing passes between warps inside the loop.
//
// Products are mma.sync m16n8k16: with 16 rows a tcgen05 instruction (128
// rows) would be seven eighths padding, and the tensor pipe is not what
// bounds the kernel.  A warp's keys are the N of Q K^T and the K of P V, so
// the probabilities go from one accumulator layout to the other operand's
// without leaving the registers.
//
// E4M3 codes are widened to BF16 in registers (exact): exponent and fraction
// moved into place, then one packed multiplication by 2^120.  A 32-bit word of
// four codes c0..c3 gives the pairs (c0, c2) and (c1, c3) without a byte
// permutation; for K the dimensions' order within 16 is free (Q's fragment
// takes the same one), for V, read transposed, the pairs are two keys of one
// dimension.  A key's scale is a power of two: K's multiplies the logit, V's
// the probability.
//
// Two CTAs of 160 threads an SM; three 32 KB stages each (six in the E4M3
// kind).
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kKeyShift = 6;  // 64 keys a stage
constexpr int kTileKeys = 1 << kKeyShift;
constexpr int kConsumers = 4;  // warps
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kSegs = 4;       // steps described ahead
constexpr float kRescaleLog2 = 8.0f;

template <int kKind>
struct Ring {
  static constexpr int kStages = kKind == 0 ? 3 : 6;
  static constexpr uint32_t kRow = kKind == 0 ? 256 : 128;              // bytes of a cached row
  static constexpr uint32_t kHalf = kTileKeys * kRow;                   // K or V of a stage
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kExp = kKind == 0 ? 0 : 2 * kTileKeys;      // exponent bytes of a stage
};
constexpr uint32_t kRingBytes = 3 * 32768;
static_assert(Ring<0>::kStages * Ring<0>::kStage == kRingBytes && Ring<1>::kStages * Ring<1>::kStage == kRingBytes, "");

// Shared memory, from a 1024-byte boundary.
constexpr uint32_t kOffExp = kRingBytes;                 // 6 x 128 exponent bytes
constexpr uint32_t kOffMerge = kOffExp + 768;            // 8 KB: merging the warps' outputs
constexpr uint32_t kOffMl = kOffMerge + 8192;            // [2][4][32] floats
constexpr uint32_t kOffSeg = kOffMl + 1024;              // kSegs x Segment
constexpr uint32_t kOffBar = kOffSeg + kSegs * 64;
constexpr uint32_t kOffMisc = kOffBar + 256;
constexpr uint32_t kSmemBytes = kOffMisc + 128 + 1024;
static_assert(sizeof(Segment) <= 64 && sizeof(LineStart) <= 64, "");
static_assert(kLineSeqs * 8 <= kRingBytes, "the scan's scratch lies over the ring");
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs an SM");

enum { BAR_FULL = 0, BAR_EMPTY = 6, BAR_SFULL = 12, BAR_SEMPTY = 16, NUM_BARS = 20 };

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
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Codes (c0, c2) and (c1, c3) of a word as BF16 pairs.  The seven magnitude
// bits land on BF16's exponent and upper fraction, as x 2^-120 (subnormal
// codes as subnormals).
__device__ __forceinline__ uint32_t times_2_120(uint32_t v) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x7B807B80u));
  return d;
}
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
  return times_2_120(((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u));
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
  return times_2_120(((w >> 4) & 0x07F007F0u) | (w & 0x80008000u));
}
// The consumers agree: true for all when it is for one (a wait that gave up in
// one warp must not leave the others at a barrier).
__device__ __forceinline__ bool bar_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

template <int kKind, int kM>  // kM: m-tiles of 16 rows
__global__ void __launch_bounds__(kThreads, 2)
paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const PagedAttnArgs a, const PagedScratch ws) {
  using R = Ring<kKind>;
  constexpr int kRows = 16 * kM;
  const PagedArgs& c = a.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(base);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * i; };
  Segment* segs = reinterpret_cast<Segment*>(base + kOffSeg);
  volatile int32_t* s_abort = reinterpret_cast<volatile int32_t*>(base + kOffMisc);
  int32_t* s_bad = reinterpret_cast<int32_t*>(base + kOffMisc + 4);
  LineStart* line = reinterpret_cast<LineStart*>(base + kOffMisc + 16);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    *s_abort = 0;
    *s_bad = 0;
    for (int i = 0; i < R::kStages; ++i) {
      mbar_init(bar(BAR_FULL + i), 1);
      mbar_init(bar(BAR_EMPTY + i), kConsumers);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(bar(BAR_SFULL + i), 1);
      mbar_init(bar(BAR_SEMPTY + i), kConsumers);
    }
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  // (a unit is one row tile here: the host chose the form by max_new)
  line_start<false>(a, kRows, kKeyShift, blockIdx.x, gridDim.x, reinterpret_cast<int64_t*>(base), line, s_bad);
  fence_proxy_async_smem();  // the scan's scratch is written by TMA next
  __syncthreads();

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    LineWalk w;
    walk_begin(a, *line, w, kRows, kKeyShift);
    JoinDesc join;
    join.pieces = 0;
    bool ok = true, bad_page = false;
    int stage = 0, seq = 0;
    const int per_page = min(c.page_size, kTileKeys);        // keys of a tile in one page
    const int tile_pages = kTileKeys / per_page;
    const int sub = lane % 4, pg = lane / 4;                  // lane: page pg of the tile, box sub
    for (int k = 0; ok; ++k) {
      const Segment g = walk_next(a, w, kRows, kKeyShift, blockIdx.x, join);
      ok = k < kSegs ||
           __all_sync(0xFFFFFFFFu, mbar_wait(bar(BAR_SEMPTY + k % kSegs), ((k / kSegs) & 1) ^ 1, kWaitLimitNs));
      if (!ok) break;
      if (lane == 0) {
        segs[k % kSegs] = g;
        mbar_arrive(bar(BAR_SFULL + k % kSegs));
      }
      if (!g.valid) break;
      const int32_t* table = c.table + g.s * c.table_stride;
      // pages of this step's tiles, 32 table entries at a time
      const int p_lo = g.lo >> c.page_shift, p_hi = (g.hi + c.page_size - 1) >> c.page_shift;
      int have = -1, entry = 0;  // entry: page index 32 * have + lane
      for (int t = g.t0; t < g.t0 + g.nt; ++t) {
        const int key0 = t << kKeyShift;
        const int page0 = key0 >> c.page_shift;
        if (page0 / 32 != have) {
          have = page0 / 32;
          const int at = have * 32 + lane;
          entry = at >= p_lo && at < p_hi ? __ldg(table + at) : 0;
          const bool wrong = entry < 0 || entry >= c.pages;
          bad_page |= wrong;
          if (wrong) entry = -1;
        }
        const int first = max(page0, p_lo), last = min(page0 + tile_pages, p_hi);  // [first, last)
        ok = seq < R::kStages || __all_sync(0xFFFFFFFFu, mbar_wait(bar(BAR_EMPTY + stage),
                                                                  ((seq / R::kStages) & 1) ^ 1, kWaitLimitNs));
        if (!ok) break;
        const int at = page0 + pg;
        const int page = __shfl_sync(0xFFFFFFFFu, entry, at % 32);
        const bool mine = pg < tile_pages && at >= first && at < last && page >= 0;
        const int loads = __popc(__ballot_sync(0xFFFFFFFFu, mine && sub == 0));
        if (lane == 0)
          mbar_arrive_expect_tx(bar(BAR_FULL + stage),
                                loads * per_page * (2 * R::kRow + (kKind ? 2 : 0)));
        __syncwarp();
        if (mine) {
          const int64_t row = ((static_cast<int64_t>(page) * c.H + g.h) << c.page_shift) + (key0 & (c.page_size - 1));
          const uint32_t to = sbase + stage * R::kStage + (sub / 2) * R::kHalf + pg * per_page * 128;
          const CUtensorMap* map = sub / 2 ? &tm_v : &tm_k;
          if constexpr (kKind == 0) {
            tma_load_2d(to + (sub % 2) * (kTileKeys * 128), map, bar(BAR_FULL + stage), (sub % 2) * 64,
                        static_cast<int>(row));
          } else if (sub % 2 == 0) {
            tma_load_2d(to, map, bar(BAR_FULL + stage), 0, static_cast<int>(row));
          } else {
            bulk_load(sbase + kOffExp + stage * R::kExp + (sub / 2) * kTileKeys + pg * per_page,
                      (sub / 2 ? c.v_exp : c.k_exp) + row, per_page, bar(BAR_FULL + stage));
          }
        }
        ++seq;
        stage = stage + 1 == R::kStages ? 0 : stage + 1;
        ok = !__any_sync(0xFFFFFFFFu, *s_abort != 0);
        if (!ok) break;
      }
    }
    bad_page = __any_sync(0xFFFFFFFFu, bad_page);
    if (!ok) {
      *s_abort = 1;
      // copies in flight land before the CTA ends (bounded)
      for (int q = max(0, seq - R::kStages); q < seq; ++q)
        mbar_wait(bar(BAR_FULL + q % R::kStages), (q / R::kStages) & 1, kWaitLimitNs);
    }
    if (lane == 0) {
      ws.join[blockIdx.x] = join;
      if (bad_page) *s_bad = 1;
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int r = lane / 4, t4 = lane % 4;
    float* merge = reinterpret_cast<float*>(base + kOffMerge);
    float* s_m = reinterpret_cast<float*>(base + kOffMl);
    float* s_l = s_m + 4 * 32;
    const float c2 = a.scale * 1.4426950408889634f;
    // ldmatrix rows: lane l gives row l % 8 of matrix l / 8
    const int mrow = lane % 8, mat = lane / 8;
    bool ok = true;
    int stage = 0, seq = 0;
    for (int k = 0; ok; ++k) {
      ok = !bar_any(!mbar_wait(bar(BAR_SFULL + k % kSegs), (k / kSegs) & 1, kWaitLimitNs));
      if (!ok) break;
      const Segment g = segs[k % kSegs];
      if (!g.valid) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_SEMPTY + k % kSegs));
      // Q fragments and the keys that this thread's rows see
      uint32_t qf[kM][8][4];
      int lo[kM][2], hi[kM][2];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rho = g.rho0 + 16 * m + r + 8 * e;
          const bool real = 16 * m + r + 8 * e < g.rows;
          const int i = rho / a.group;
          const int pos = g.len - g.n + i;
          lo[m][e] = real ? row_lo(a, pos) : 0;
          hi[m][e] = real ? (a.causal ? min(g.len, pos + 1) : g.len) : 0;
          const uint16_t* src = a.q + static_cast<int64_t>(g.row0 + i) * a.q_token +
                                static_cast<int64_t>(g.h * a.group + rho % a.group) * a.q_head;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t x = 0, y = 0;
            if (real) {
              if constexpr (kKind == 0) {
                x = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 2 * t4));
                y = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 8 + 2 * t4));
              } else {  // dimensions 4t, 4t + 2 and 4t + 1, 4t + 3, as the codes come
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + 16 * kk + 4 * t4));
                x = __byte_perm(v.x, v.y, 0x5410);
                y = __byte_perm(v.x, v.y, 0x7632);
              }
            }
            qf[m][kk][e] = x;
            qf[m][kk][2 + e] = y;
          }
        }
      }
      const int all_lo = row_lo(a, g.len - g.n + (g.rho0 + g.rows - 1) / a.group);
      const int all_hi = a.causal ? min(g.len, g.len - g.n + g.rho0 / a.group + 1) : g.len;
      float acc[kM][16][4], ref[kM][2], sum[kM][2];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ref[m][e] = -INFINITY;
          sum[m][e] = 0.f;
        }
      }
#pragma unroll 1
      for (int t = g.t0; t < g.t0 + g.nt; ++t) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(BAR_FULL + stage), (seq / R::kStages) & 1, kWaitLimitNs));
        if (!ok) break;
        const uint32_t sk = sbase + stage * R::kStage, sv = sk + R::kHalf;
        uint8_t* ex = base + kOffExp + stage * R::kExp;
        const int key0 = (t << kKeyShift) + 16 * warp;
        // Slots that no row sees may hold anything: this warp's V rows there
        // become zeros (their probabilities are 0, and 0 * NaN is not).
        const bool ragged = key0 < g.lo || key0 + 16 > g.hi;
        if (ragged) {
          const int u = lane / 2;
          if (key0 + u < g.lo || key0 + u >= g.hi) {
            uint8_t* v = base + stage * R::kStage + R::kHalf + (16 * warp + u) * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              *reinterpret_cast<uint4*>(v + (lane % 2) * 64 + 16 * i) = make_uint4(0, 0, 0, 0);
              if (kKind == 0)
                *reinterpret_cast<uint4*>(v + kTileKeys * 128 + (lane % 2) * 64 + 16 * i) = make_uint4(0, 0, 0, 0);
            }
          }
          __syncwarp();
        }
        // ---- S = Q K^T of 16 keys: two n-tiles
        float s[kM][2][4];
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[m][0][e] = s[m][1][e] = 0.f;
        {
          // matrices: keys 0-7 chunk c, c + 1, keys 8-15 chunk c, c + 1
          const int row = 16 * warp + (mat / 2) * 8 + mrow;
          const uint32_t rb = sk + row * 128;
#pragma unroll
          for (int kk = 0; kk < (kKind == 0 ? 8 : 4); ++kk) {
            const int chunk = 2 * kk + (mat & 1);
            uint32_t b[4];
            ldsm4(b, rb + (kKind == 0 ? (chunk / 8) * (kTileKeys * 128) : 0) + ((chunk % 8) ^ (row & 7)) * 16);
            if constexpr (kKind == 0) {
#pragma unroll
              for (int m = 0; m < kM; ++m) {
                mma(s[m][0], qf[m][kk], b[0], b[1]);
                mma(s[m][1], qf[m][kk], b[2], b[3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // keys 8 (i / 2).., dimensions 16 (2 kk + i % 2)..
                const uint32_t b0 = codes_even(b[i]), b1 = codes_odd(b[i]);
#pragma unroll
                for (int m = 0; m < kM; ++m) mma(s[m][i / 2], qf[m][2 * kk + i % 2], b0, b1);
              }
            }
          }
        }
        float ks[2][2], vs[2][2];
        if constexpr (kKind != 0) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int u = 16 * warp + 8 * nt + 2 * t4;
            const uint32_t ke = *reinterpret_cast<const uint16_t*>(ex + u);
            const uint32_t ve = *reinterpret_cast<const uint16_t*>(ex + kTileKeys + u);
            ks[nt][0] = exp_scale(ke & 255u) * c2;
            ks[nt][1] = exp_scale(ke >> 8) * c2;
            vs[nt][0] = exp_scale(ve & 255u);
            vs[nt][1] = exp_scale(ve >> 8);
          }
        }
        const bool cut = ragged || key0 < all_lo || key0 + 16 > all_hi;  // some row misses some key
        uint32_t p[kM][4];
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          bool moves = false;
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x = s[m][nt][e] * (kKind == 0 ? c2 : ks[nt][e & 1]);
              if (cut) {
                const int key = key0 + 8 * nt + 2 * t4 + (e & 1);
                if (key < lo[m][e / 2] || key >= hi[m][e / 2]) x = -INFINITY;
              }
              s[m][nt][e] = x;
              mx[e / 2] = fmaxf(mx[e / 2], x);
            }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 2));
            moves |= mx[e] > ref[m][e] + kRescaleLog2;
          }
          // The reference follows the maximum only when it is passed by 2^8:
          // p <= 256 keeps the sums far inside FP32.
          if (__any_sync(0xFFFFFFFFu, moves)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float to = mx[e] > ref[m][e] + kRescaleLog2 ? mx[e] : ref[m][e];
              const float f = to == ref[m][e] ? 1.f : ex2_approx(ref[m][e] - to);  // first keys: 2^-inf = 0
              ref[m][e] = to;
              sum[m][e] *= f;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                acc[m][i][2 * e] *= f;
                acc[m][i][2 * e + 1] *= f;
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float rf = ref[m][e / 2] == -INFINITY ? 0.f : ref[m][e / 2];
              const float x = ex2_approx(s[m][nt][e] - rf);
              sum[m][e / 2] += x;
              // a hidden key's scale may be NaN
              y[e] = kKind == 0 ? x : (x == 0.f ? 0.f : x * vs[nt][e & 1]);
            }
            p[m][2 * nt] = pack_bf16x2(y[0], y[1]);
            p[m][2 * nt + 1] = pack_bf16x2(y[2], y[3]);
          }
        }
        // ---- O += P V: matrices keys 0-7, 8-15 of chunk c, then of chunk c + 1
        {
          const int row = 16 * warp + (mat & 1) * 8 + mrow;
          const uint32_t rb = sv + row * 128;
#pragma unroll
          for (int j = 0; j < (kKind == 0 ? 8 : 4); ++j) {
            const int chunk = 2 * j + mat / 2;
            uint32_t b[4];
            ldsm4_t(b, rb + (kKind == 0 ? (chunk / 8) * (kTileKeys * 128) : 0) + ((chunk % 8) ^ (row & 7)) * 16);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if constexpr (kKind == 0) {
#pragma unroll
                for (int m = 0; m < kM; ++m) mma(acc[m][2 * j + i], p[m], b[2 * i], b[2 * i + 1]);
              } else {  // even and odd dimensions of 16
                const uint32_t e0 = codes_even(b[2 * i]), e1 = codes_even(b[2 * i + 1]);
                const uint32_t o0 = codes_odd(b[2 * i]), o1 = codes_odd(b[2 * i + 1]);
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                  mma(acc[m][4 * j + 2 * i], p[m], e0, e1);
                  mma(acc[m][4 * j + 2 * i + 1], p[m], o0, o1);
                }
              }
            }
          }
        }
        if (ragged) fence_proxy_async_smem();  // zeros written here, TMA writes next
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_EMPTY + stage));
        ++seq;
        stage = stage + 1 == R::kStages ? 0 : stage + 1;
      }
      ok = !bar_any(!ok || *s_abort != 0);
      if (!ok) break;
      // ---- the four warps' results into one
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[m][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[m][e], 1);
          sum[m][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[m][e], 2);
          if (t4 == 0) {
            s_m[warp * 32 + 16 * m + r + 8 * e] = ref[m][e];
            s_l[warp * 32 + 16 * m + r + 8 * e] = sum[m][e];
          }
        }
      bar_consumers();
      float f[kM][2];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 16 * m + r + 8 * e;
          const float mt = fmaxf(fmaxf(s_m[row], s_m[32 + row]), fmaxf(s_m[64 + row], s_m[96 + row]));
          f[m][e] = ref[m][e] == -INFINITY ? 0.f : ex2_approx(ref[m][e] - mt);
        }
      constexpr int kCols = 128 / kM;  // columns a pass: 8 KB of FP32
#pragma unroll
      for (int pass = 0; pass < kM; ++pass) {
        for (int w = 0; w < kConsumers; ++w) {
          if (warp == w) {
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
              for (int i = 0; i < 16 / kM; ++i) {
                const int n = pass * (16 / kM) + i;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int col = kKind == 0 ? 8 * i + 2 * t4 + (e & 1)
                                             : 16 * (i / 2) + 4 * t4 + 2 * (e & 1) + (i & 1);
                  float* d = merge + (16 * m + r + 8 * (e / 2)) * kCols + col;
                  const float y = acc[m][n][e] * f[m][e / 2];
                  *d = w == 0 ? y : *d + y;
                }
              }
          }
          bar_consumers();
        }
        // 16 kM rows x kCols columns: 16 values a thread, in one row
        const int row = threadIdx.x * 16 / kCols, col = threadIdx.x * 16 % kCols;
        const float mt = fmaxf(fmaxf(s_m[row], s_m[32 + row]), fmaxf(s_m[64 + row], s_m[96 + row]));
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w)
          l += s_m[32 * w + row] == -INFINITY ? 0.f : s_l[32 * w + row] * ex2_approx(s_m[32 * w + row] - mt);
        const float* src = merge + row * kCols + col;
        if (row < g.rows) {
          if (g.part < 0) {
            const int rho = g.rho0 + row;
            const int64_t at = static_cast<int64_t>(g.row0 + rho / a.group) * a.Hq + g.h * a.group + rho % a.group;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (NaN stays)
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = pack_bf16x2(src[2 * i] * inv, src[2 * i + 1] * inv);
            uint4* dst = reinterpret_cast<uint4*>(a.o + at * kHeadDim + pass * kCols + col);
            dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
            dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
            if (a.lse && pass == 0 && col == 0)
              a.lse[at] = l == 0.f ? -INFINITY : (mt + log2f(l)) * 0.6931471805599453f;
          } else {
            const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + g.part) * kRows + row;
            float4* dst = reinterpret_cast<float4*>(ws.part + at * kHeadDim + pass * kCols + col);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = reinterpret_cast<const float4*>(src)[i];
            if (pass == 0 && col == 0) ws.ml[at] = make_float2(mt, l);
          }
        }
        bar_consumers();
      }
    }
    if (!ok) *s_abort = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) ws.cta_status[blockIdx.x] = *s_abort ? 5 /* SA_ETIMEOUT */ : (*s_bad ? kPagedInvalid : 0);
  griddep_launch_dependents();
}

}  // namespace

size_t paged_few_smem() { return kSmemBytes; }

cudaError_t launch_paged_few(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a,
                             const PagedScratch& ws, int row_tile, int ctas, cudaStream_t s) {
  auto* kern = a.c.kind == 0 ? (row_tile == 16 ? paged_few_kernel<0, 1> : paged_few_kernel<0, 2>)
                             : (row_tile == 16 ? paged_few_kernel<1, 1> : paged_few_kernel<1, 2>);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kThreads, kSmemBytes, s>>>(tk, tv, a, ws);
  return cudaGetLastError();
}

}  // namespace sa
