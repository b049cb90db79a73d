// The attention weight that cached keys receive (sm_103a):
//
//   w_j (+)= sum over rows r that see key j, and query heads of its group, of
//            2^(x_rj - L_r),   x_rj = scale log2(e) (q_r . k_j),  L_r = log2(e) lse_r
//
// A key's weight depends on its own K alone, so whoever has a key adds up all
// rows for it: nothing is joined, and no atomics change an order.  This is the
// form for few rows (at most 128 packed rows a sequence and key head), in two
// kernels: rows in registers up to 16, in shared memory above.
//
// Bound by memory: K once (256 bytes a key and head, 129 in the E4M3 kind), the
// weight read and written.  The line of all tiles of 16 keys is cut into equal
// parts, one a warp, however ragged the batch is; warps share nothing, so a call
// is a launch, a walk of the line and as many tiles as a warp has.  K goes from
// memory into the registers of mma.sync m16n8k16 as its first operand (the
// order of dimensions inside a product is free), a tile while the last one is
// multiplied.
//
// Measured:
//   64 sequences of 512 to 33792 keys, 40 / 8 heads, BF16, one new   127 us  6.58 TB/s
//                                                    E4M3             79 us  5.48
//   64 of 8704, 24 / 8 heads, four new (12 rows): BF16               186 us  6.32
//                                                 E4M3               129 us  4.76
//   one of 1152, 8 / 2 heads, BF16                                   4.2 us  (latency; 6.4 with a status to clear)
// Without the loads ahead the first takes 153 us; in E4M3 what a tile costs
// besides its bytes counts: finding the next one from the last (113 -> 89 us)
// and codes as FP16 instead of BF16.  Two tiles ahead: no better (registers).
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4;
// Blocks an SM: what the registers of so many rows allow (BF16, up to eight rows:
// with 86 bytes spilled).
template <int kN>
constexpr int kBlocks = kN == 1 ? 4 : 3;
constexpr int kTileKeys = 16;  // keys of a warp's tile: inside one page

// Keys of sequence q whose weight the call writes.
struct KeySpan {
  int lo, hi;  // [lo, hi), empty for hi <= lo
  int t0, nt;  // tiles of 16 keys
};
__device__ __forceinline__ KeySpan key_span(const WeighArgs& w, const PagedSeq& q) {
  KeySpan k;
  k.lo = w.accumulate ? max(w.first, row_lo(w.a, q.len - q.n)) : w.first;
  k.hi = q.n > 0 ? q.len : 0;
  k.t0 = k.lo / kTileKeys;
  k.nt = k.hi > k.lo ? (k.hi + kTileKeys - 1) / kTileKeys - k.t0 : 0;
  return k;
}

__device__ __forceinline__ int lane_tiles16(const WeighArgs& w, int s, PagedSeq& q) {
  q.n = q.len = q.row0 = 0;
  if (s >= w.a.c.seqs) return 0;
  bool bad;
  q = paged_seq(w.a.c, s, bad);
  return key_span(w, q).nt;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes (c0, c1) and (c2, c3) as FP16 pairs.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t v;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  return v;
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Rows of Q: as the second operand of K Q^T, 8 kN of them.  A lane has row
// lane / 4 of each eight, and 16-byte chunks lane % 4 + 4 i of it, as of K's
// rows: the order of dimensions inside a product is free as long as both have
// the same.
// E4M3: K's codes become FP16 (two instructions for four), and so does Q, each row
// scaled by the even power of two that brings its largest magnitude to 2^13 or
// 2^14 or just below: exact down to 2^-30 of that.
template <int kKind, int kN>
struct Rows {
  uint32_t q[kN][8][2];
  float neg[kN][2];        // -L of rows 2 t, 2 t + 1 of each eight (-inf: counts nothing)
  float undo[kN][2];       // E4M3: their squares undo the rows' scaling
  int lo[kN][2], hi[kN][2];  // keys that they see

  __device__ __forceinline__ void load(const WeighArgs& w, const PagedSeq& s, int h, int rho0, int lane) {
    const PagedAttnArgs& a = w.a;
    const int rows = s.n * a.group, u = lane / 4, t4 = lane % 4;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int rho = rho0 + 8 * n + u;
      const int i = div_group(a, rho);
      const uint16_t* src = a.q + static_cast<int64_t>(s.row0 + i) * a.q_token +
                            static_cast<int64_t>(h * a.group + rho - i * a.group) * a.q_head;
      uint4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = make_uint4(0, 0, 0, 0);
        // (16 codes of K are 32 bytes here)
        const int at = kKind == 0 ? 8 * (t4 + 4 * e) : 16 * (t4 + 4 * (e / 2)) + 8 * (e % 2);
        if (rho < rows) x[e] = __ldg(reinterpret_cast<const uint4*>(src + at));
      }
      if constexpr (kKind != 0) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[e].x & 0x7FFF7FFFu, x[e].y & 0x7FFF7FFFu),
                                   __vmaxu2(x[e].z & 0x7FFF7FFFu, x[e].w & 0x7FFF7FFFu)));
        m = max(m >> 16, m & 0xFFFFu);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        // largest magnitude 2^(E - 127): times 2^(141 - E) or half of it, at most 2^126
        const int e2 = min(126, (141 - static_cast<int>(m >> 7)) & ~1);
        const float f = pow2(e2), back = pow2(-e2 / 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t* v = reinterpret_cast<uint32_t*>(&x[e]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = pack_f16x2(__uint_as_float(v[k] << 16) * f, __uint_as_float(v[k] & 0xFFFF0000u) * f);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) undo[n][e] = __shfl_sync(0xFFFFFFFFu, back, 4 * (2 * t4 + e));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[n][2 * e][0] = x[e].x;
        q[n][2 * e][1] = x[e].y;
        q[n][2 * e + 1][0] = x[e].z;
        q[n][2 * e + 1][1] = x[e].w;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rho0 + 8 * n + 2 * t4 + e;
        const int j = div_group(a, r), pos = s.len - s.n + j;
        const bool real = r < rows;
        float l = INFINITY;
        if (real) l = __ldg(w.lse + static_cast<int64_t>(s.row0 + j) * a.Hq + h * a.group + r - j * a.group);
        // (a row that counts nothing sees nothing here: its products may be NaN)
        const bool counts = l != -INFINITY && real;
        neg[n][e] = counts ? -l * 1.4426950408889634f : -INFINITY;
        lo[n][e] = counts ? row_lo(a, pos) : 0;
        hi[n][e] = counts ? (a.causal ? min(s.len, pos + 1) : s.len) : 0;
      }
    }
  }
};

// A tile of 16 keys: keys u and u + 8 of the lanes of a row.
template <int kKind>
struct Tile {
  uint4 x[2][kKind == 0 ? 4 : 2];
  uint32_t exp[2];  // E4M3: their exponents
  float old;       // the weight that this lane writes
  int64_t row0;    // first row of the cache; -1: not to be looked at
  int key0, lo, hi;  // of the tile, and keys of its unit whose weight is written
  bool fresh;      // the first of its unit
  PagedSeq q;
  int h;
};

template <int kKind, int kN>  // kN: tiles of eight rows
__global__ void __launch_bounds__(32 * kWarps, kBlocks<kN>) weigh_kernel(const WeighArgs w) {
  const PagedAttnArgs& a = w.a;
  const PagedArgs& c = a.c;
  const int lane = threadIdx.x % 32, u = lane / 4, t4 = lane % 4;
  if (blockIdx.x == 0) paged_check_all(c);
  const int worker = blockIdx.x * kWarps + threadIdx.x / 32, workers = gridDim.x * kWarps;
  // The line of all tiles, in the order (sequence, head, tile), in equal parts.
  PagedSeq q;
  const int first_tiles = lane_tiles16(w, lane, q);  // of the first 32 sequences
  int64_t total = first_tiles;
#pragma unroll 1
  for (int base = 32; base < c.seqs; base += 32) total += lane_tiles16(w, base + lane, q);
  total = warp_sum(total) * c.H;
  int64_t at = muldiv(worker, total, workers);
  const int64_t end = muldiv(worker + 1, total, workers);
  if (at >= end) return;
  int s = 0, h = 0, t = 0;
  {
    int64_t left = at;
#pragma unroll 1
    for (int base = 0;; base += 32) {
      const int64_t mine = static_cast<int64_t>(base ? lane_tiles16(w, base + lane, q) : first_tiles) * c.H;
      const int64_t upto = warp_scan(mine, lane);
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, upto > left);
      if (hit) {
        const int src = __ffs(hit) - 1;
        s = base + src;
        left = __shfl_sync(0xFFFFFFFFu, left - (upto - mine), src);
        break;
      }
      left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    bool bad;
    q = paged_seq(c, s, bad);
    const int nt = key_span(w, q).nt;
    h = static_cast<int>(muldiv(left, 1, nt));
    t = static_cast<int>(left - static_cast<int64_t>(h) * nt);
  }
  KeySpan k = key_span(w, q);
  bool fresh = true;
  int have = -1, entry = 0;  // table entries 32 have + lane
  const float c2 = a.scale * 1.4426950408889634f;
  constexpr int kRow = kKind == 0 ? 256 : 128, kLoads = kKind == 0 ? 4 : 2;
  auto load = [&](Tile<kKind>& n, int64_t from) {
    n.row0 = from;
    n.lo = k.lo;
    n.hi = k.hi;
    n.q = q;
    n.h = h;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) n.x[e][i] = ld_stream(c.k_pages + (from + u + 8 * e) * kRow + 16 * (t4 + 4 * i));
#pragma unroll
    for (int e = 0; e < 2; ++e) n.exp[e] = kKind == 0 ? 0u : __ldg(c.k_exp + from + u + 8 * e);
    // lanes t = 0 and 1 of each four write keys u and u + 8
    const int key = n.key0 + u + 8 * t4;
    n.old = 0.f;
    if (t4 < 2 && key >= k.lo && key < q.len - q.n && w.accumulate) n.old = w.weights[from + u + 8 * t4];
  };
  // The next tile of the part, its loads under way.
  int64_t row0 = -1;
  int more = 0;  // tiles of the same page and unit that follow
  auto fetch = [&](Tile<kKind>& n) {
    if (more > 0 && row0 >= 0) {
      --more;
      ++t;
      row0 += kTileKeys;
      n.key0 = (k.t0 + t - 1) * kTileKeys;
      n.fresh = false;
      load(n, row0);
      return;
    }
    if (t == k.nt) {
      t = 0;
      fresh = true;
      if (++h == c.H) {
        h = 0;
        have = -1;
        do {
          bool bad;
          if (++s >= c.seqs) {
            n.row0 = -1;
            return;
          }
          q = paged_seq(c, s, bad);
          k = key_span(w, q);
        } while (k.nt == 0);
      }
    }
    n.key0 = (k.t0 + t) * kTileKeys;
    more = min(k.nt - t, (c.page_size - (n.key0 & (c.page_size - 1))) / kTileKeys) - 1;
    n.fresh = fresh;
    fresh = false;
    ++t;
    const int pi = n.key0 >> c.page_shift;
    if (pi / 32 != have) {
      have = pi / 32;
      const int e = have * 32 + lane;
      entry = (static_cast<int64_t>(e) << c.page_shift) < k.hi && (static_cast<int64_t>(e + 1) << c.page_shift) > k.lo
                  ? __ldg(c.table + s * c.table_stride + e) : 0;
    }
    const int page = __shfl_sync(0xFFFFFFFFu, entry, pi % 32);
    row0 = n.row0 = -1;
    if (page < 0 || page >= c.pages) {
      if (lane == 0) paged_fail(c);
      return;
    }
    row0 = ((static_cast<int64_t>(page) * c.H + h) << c.page_shift) + (n.key0 & (c.page_size - 1));
    load(n, row0);
  };
  Rows<kKind, kN> rows;
  bool need = false;  // the unit's rows are to be loaded
  Tile<kKind> tiles[2];
  fetch(tiles[0]);
  Tile<kKind>& now = tiles[0];
#pragma unroll 1
  for (; at < end; ++at) {
    if (at + 1 < end) fetch(tiles[1]);
    need |= now.fresh;
    if (now.row0 >= 0) {
      if (need) rows.load(w, now.q, now.h, 0, lane);
      need = false;
      float d[kN][4];
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[n][e] = 0.f;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t k0[4] = {now.x[0][i].x, now.x[0][i].y, now.x[0][i].z, now.x[0][i].w};
        const uint32_t k1[4] = {now.x[1][i].x, now.x[1][i].y, now.x[1][i].z, now.x[1][i].w};
        if constexpr (kKind == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < kN; ++n)
              mma_bf16(d[n], k0[2 * e], k1[2 * e], k0[2 * e + 1], k1[2 * e + 1], rows.q[n][2 * i + e][0], rows.q[n][2 * i + e][1]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t l0, h0, l1, h1;
            codes_f16(k0[e], l0, h0);
            codes_f16(k1[e], l1, h1);
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_f16(d[n], l0, l1, h0, h1, rows.q[n][4 * i + e][0], rows.q[n][4 * i + e][1]);
          }
        }
      }
      // A key's scale as two factors of half its exponent, as Q's: the product
      // of one of each is a number, whatever the two scales are.
      float ks[2][2] = {};
      if constexpr (kKind != 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int x = now.exp[e], half = x >> 1;
          ks[e][0] = pow2(half - 64);
          ks[e][1] = (x - 1u < 254u ? pow2(x - half - 63) : exp_scale(x)) * c2;
        }
      }
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // key u + 8 (e / 2), row 2 t + e % 2
          const int j = now.key0 + u + 8 * (e / 2);
          float x = d[n][e], f = c2;
          if constexpr (kKind != 0) {
            x *= rows.undo[n][e & 1] * ks[e / 2][0];
            f = rows.undo[n][e & 1] * ks[e / 2][1];
          }
          const float p = ex2_approx(fmaf(x, f, rows.neg[n][e & 1]));
          if (j >= rows.lo[n][e & 1] && j < rows.hi[n][e & 1]) sum[e / 2] += p;
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 2);
      }
      const int key = now.key0 + u + 8 * t4;
      if (t4 < 2 && key >= now.lo && key < now.hi) w.weights[now.row0 + u + 8 * t4] = now.old + (t4 ? sum[1] : sum[0]);
    }
    tiles[0] = tiles[1];
  }
}

// ---- 17 to 128 packed rows a sequence and key head
//
// The same products, with more rows than a warp's registers hold: a block takes a
// part of the line, the rows of its unit lie in shared memory (in the order of a
// lane's reads), and each warp multiplies every fourth tile with all of them.  A tile
// costs what its rows cost, and rows differ from sequence to sequence, so the line
// is measured in that.
// Bound by mma.sync where there are 64 rows (about three quarters of its rate), by
// memory where there are few.  Eight sequences, 24 heads, up to so many rows each,
// here and by the form of paged_weigh_chunk.cu, which multiplies six times as fast
// but has to fill and drain 256 keys for however many rows come:
//   rows   keys            E4M3            BF16
//     17   1152          16 /  30 us     18 /  34 us
//     17   17408         98 / 269       143 / 338
//     64   1152          25 /  30        25 /  35
//     64   17408        135 / 278       162 / 345
//    128   17408        173 / 282       181 / 361
// and as many rows each, over 17408 keys: 64 rows 208 / 282 and 209 / 364, 96 rows
// 283 / 238 and 285 / 282, 128 rows 356 / 301 and 352 / 323 (so above 64 rows the
// mean decides).  Two tiles a warp (54 against 46 us for eight sequences of 1152
// to 8704 keys, up to 64 rows) and two accumulators a product (no change) did not
// help: loads of rows did, all under way at once and behind the first keys' (46 ->
// 43 us).
constexpr int kMidRow = 320;   // bytes of a row: other banks for the next one
constexpr int kMidBlocks = 4;  // blocks an SM

template <int kRows>  // at most so many rows
struct MidRows {
  alignas(16) uint8_t q[kRows * kMidRow];
  float4 use[kRows / 2];  // of a pair of rows: -L (-inf: counts nothing); E4M3: the roots of what undoes their scaling
  int pos[kRows];         // the last key that the row sees (-1: its lse is -infinity, it counts nothing)
};

// The rows of unit (q, h), by the whole block: half a warp has a row at a time, and
// eight of them are on their way before the first is looked at.  True where this
// thread's rows have one that counts nothing: its products may be NaN and are to
// be left out.
template <int kKind, int kRows>
__device__ __forceinline__ bool mid_rows(const WeighArgs& w, const PagedSeq& q, int h, MidRows<kRows>& m) {
  const PagedAttnArgs& a = w.a;
  constexpr int kTurns = 8;
  static_assert(kRows % (kTurns * 8) == 0 && 2 * kWarps == 8, "a turn is eight rows");
  const int rows = q.n * a.group, lane = threadIdx.x % 32, sub = lane % 16;
  bool nothing = false;
#pragma unroll 1
  for (int r0 = 0; r0 < kRows; r0 += kTurns * 8) {
    if (r0 >= rows) break;
    uint4 x[kTurns];
    float l[kTurns];
#pragma unroll
    for (int n = 0; n < kTurns; ++n) {
      // (past the last: the last again, counting nothing)
      const int rho = r0 + 8 * n + threadIdx.x / 16, real = min(rho, rows - 1), i = div_group(a, real), e = real - i * a.group;
      x[n] = make_uint4(0, 0, 0, 0);
      l[n] = INFINITY;
      if (r0 + 8 * n < rows)
        x[n] = __ldg(reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(q.row0 + i) * a.q_token +
                                                    static_cast<int64_t>(h * a.group + e) * a.q_head + sub * 8));
      if (rho < rows) l[n] = __ldg(w.lse + static_cast<int64_t>(q.row0 + i) * a.Hq + h * a.group + e);
    }
#pragma unroll
    for (int n = 0; n < kTurns; ++n) {
      const int rho = r0 + 8 * n + threadIdx.x / 16;
      if (r0 + 8 * n >= rows) break;
      nothing |= l[n] == -INFINITY;
      int at = sub;
      float* use = reinterpret_cast<float*>(m.use + rho / 2) + rho % 2;
      if constexpr (kKind != 0) {  // (see Rows)
        uint32_t z = __vmaxu2(__vmaxu2(x[n].x & 0x7FFF7FFFu, x[n].y & 0x7FFF7FFFu),
                              __vmaxu2(x[n].z & 0x7FFF7FFFu, x[n].w & 0x7FFF7FFFu));
        z = max(z >> 16, z & 0xFFFFu);
#pragma unroll
        for (int d = 1; d < 16; d *= 2) z = max(z, __shfl_xor_sync(0xFFFFFFFFu, z, d));
        const int e2 = min(126, (141 - static_cast<int>(z >> 7)) & ~1);
        const float f = pow2(e2);
        uint32_t* v = reinterpret_cast<uint32_t*>(&x[n]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = pack_f16x2(__uint_as_float(v[k] << 16) * f, __uint_as_float(v[k] & 0xFFFF0000u) * f);
        if (sub == 0) use[2] = pow2(-e2 / 2);
        // 16 codes of K are two of these: the first ones of the lanes t = 0 .. 3, then the second
        at = (sub >> 3) * 8 + (sub & 1) * 4 + (sub >> 1 & 3);
      }
      *reinterpret_cast<uint4*>(m.q + rho * kMidRow + at * 16) = x[n];
      if (sub == 0) {
        use[0] = l[n] == -INFINITY ? -INFINITY : -l[n] * 1.4426950408889634f;
        m.pos[rho] = rho >= rows || l[n] == -INFINITY ? -1 : a.causal ? q.len - q.n + div_group(a, rho) : 0x7FFFFFFF;
      }
    }
  }
  return nothing;
}

using f2 = unsigned long long;  // two floats in a register pair
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(f2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// What a tile of a sequence costs, in units of eight rows' products (kTileCost: what
// it costs beside them); the line is measured in it.
constexpr int kTileCost = 4;
__device__ __forceinline__ int tile_cost(const WeighArgs& w, const PagedSeq& q) { return kTileCost + (q.n * w.a.group + 7) / 8; }
__device__ __forceinline__ int64_t lane_cost(const WeighArgs& w, int s, PagedSeq& q) {
  const int nt = lane_tiles16(w, s, q);
  return static_cast<int64_t>(nt) * tile_cost(w, q) * w.a.c.H;
}

template <int kKind, int kRows>
__global__ void __launch_bounds__(32 * kWarps, kMidBlocks) weigh_mid_kernel(const WeighArgs w) {
  const PagedAttnArgs& a = w.a;
  const PagedArgs& c = a.c;
  __shared__ MidRows<kRows> m;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, u = lane / 4, t4 = lane % 4;
  if (blockIdx.x == 0) paged_check_all(c);
  // The block's part of the line (every warp finds it for itself): the tiles that
  // begin in it.
  PagedSeq q;
  const int64_t first = lane_cost(w, lane, q);  // of the first 32 sequences
  int64_t total = first;
#pragma unroll 1
  for (int base = 32; base < c.seqs; base += 32) total += lane_cost(w, base + lane, q);
  total = warp_sum(total);
  int64_t left = muldiv(blockIdx.x, total, gridDim.x);
  int64_t more = muldiv(static_cast<int64_t>(blockIdx.x) + 1, total, gridDim.x) - left;
  if (more <= 0) return;
  int s = 0;
#pragma unroll 1
  for (int base = 0;; base += 32) {
    const int64_t mine = base ? lane_cost(w, base + lane, q) : first;
    const int64_t upto = warp_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, upto > left);
    if (hit) {
      const int src = __ffs(hit) - 1;
      s = base + src;
      left = __shfl_sync(0xFFFFFFFFu, left - (upto - mine), src);
      break;
    }
    left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  bool bad;
  q = paged_seq(c, s, bad);
  KeySpan k = key_span(w, q);
  int cost = tile_cost(w, q);
  int64_t unit = static_cast<int64_t>(k.nt) * cost;
  int h = static_cast<int>(muldiv(left, 1, unit));
  left -= h * unit;
  const float c2 = a.scale * 1.4426950408889634f;
  constexpr int kRow = kKind == 0 ? 256 : 128, kLoads = kKind == 0 ? 4 : 2;
  for (;;) {
    const int t0 = static_cast<int>(muldiv(left + cost - 1, 1, cost));
    const int t1 = left + more >= unit ? k.nt : static_cast<int>(muldiv(left + more + cost - 1, 1, cost));
    if (t0 < t1) {
      const int tiles = (q.n * a.group + 7) / 8;
      // keys that all rows see
      const int all_lo = row_lo(a, q.len - 1), all_hi = a.causal ? q.len - q.n + 1 : q.len;
      const int32_t* table = c.table + s * c.table_stride;
      int have = -1, entry = 0;  // table entries 32 have + lane
      struct Keys {
        uint4 x[2][kLoads];
        uint32_t exp[2];
        float old;
        int64_t row0;  // -1: not to be looked at
      } now, next;
      auto fetch = [&](int t) {
        const int key0 = (k.t0 + t) * kTileKeys, pi = key0 >> c.page_shift;
        if (pi / 32 != have) {
          have = pi / 32;
          const int e = have * 32 + lane;
          entry = (static_cast<int64_t>(e) << c.page_shift) < k.hi && (static_cast<int64_t>(e + 1) << c.page_shift) > k.lo ? __ldg(table + e) : 0;
        }
        const int page = __shfl_sync(0xFFFFFFFFu, entry, pi % 32);
        next.row0 = -1;
        if (page < 0 || page >= c.pages) {
          if (lane == 0) paged_fail(c);
          return;
        }
        next.row0 = ((static_cast<int64_t>(page) * c.H + h) << c.page_shift) + (key0 & (c.page_size - 1));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) next.x[e][i] = ld_stream(c.k_pages + (next.row0 + u + 8 * e) * kRow + 16 * (t4 + 4 * i));
          next.exp[e] = kKind == 0 ? 0u : __ldg(c.k_exp + next.row0 + u + 8 * e);
        }
        const int key = key0 + u + 8 * t4;
        next.old = 0.f;
        if (t4 < 2 && key >= k.lo && key < q.len - q.n && w.accumulate) next.old = w.weights[next.row0 + u + 8 * t4];
      };
      if (t0 + warp < t1) fetch(t0 + warp);
      __syncthreads();
      const bool nothing = __syncthreads_or(mid_rows<kKind, kRows>(w, q, h, m));
#pragma unroll 1
      for (int t = t0 + warp; t < t1; t += kWarps) {
        now = next;
        if (t + kWarps < t1) fetch(t + kWarps);
        if (now.row0 < 0) continue;
        const int key0 = (k.t0 + t) * kTileKeys;
        const bool edge = key0 < all_lo || key0 + kTileKeys > all_hi || nothing;
        uint32_t f[2][16];  // E4M3: keys u and u + 8 in FP16
        f2 ks[2][2];
        if constexpr (kKind != 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
              const uint32_t v[4] = {now.x[e][i].x, now.x[e][i].y, now.x[e][i].z, now.x[e][i].w};
#pragma unroll
              for (int g = 0; g < 4; ++g) codes_f16(v[g], f[e][8 * i + 2 * g], f[e][8 * i + 2 * g + 1]);
            }
            const int x = now.exp[e], half = x >> 1;
            const float near = pow2(half - 64), far = (x - 1u < 254u ? pow2(x - half - 63) : exp_scale(x)) * c2;
            ks[e][0] = pair(near, near);
            ks[e][1] = pair(far, far);
          }
        }
        f2 sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll 2
        for (int n = 0; n < tiles; ++n) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          const uint4* rq = reinterpret_cast<const uint4*>(m.q + (8 * n + u) * kMidRow) + t4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 b = rq[4 * i];
            if constexpr (kKind == 0) {
              mma_bf16(d, now.x[0][i].x, now.x[1][i].x, now.x[0][i].y, now.x[1][i].y, b.x, b.y);
              mma_bf16(d, now.x[0][i].z, now.x[1][i].z, now.x[0][i].w, now.x[1][i].w, b.z, b.w);
            } else {
              mma_f16(d, f[0][4 * i], f[1][4 * i], f[0][4 * i + 1], f[1][4 * i + 1], b.x, b.y);
              mma_f16(d, f[0][4 * i + 2], f[1][4 * i + 2], f[0][4 * i + 3], f[1][4 * i + 3], b.z, b.w);
            }
          }
          const float4 use = m.use[4 * n + t4];
          const f2 neg = pair(use.x, use.y), undo = pair(use.z, use.w);
          float p[2][2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // key u + 8 e, rows 2 t and 2 t + 1
            f2 x = pair(d[2 * e], d[2 * e + 1]), g = pair(c2, c2);
            if constexpr (kKind != 0) {
              x = mul2(x, mul2(undo, ks[e][0]));
              g = mul2(undo, ks[e][1]);
            }
            unpair(fma2(x, g, neg), p[e][0], p[e][1]);
            p[e][0] = ex2_approx(p[e][0]);
            p[e][1] = ex2_approx(p[e][1]);
          }
          if (edge) {
            const int2 pos = *reinterpret_cast<const int2*>(&m.pos[8 * n + 2 * t4]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + u + 8 * (e / 2), at = e & 1 ? pos.y : pos.x;
              if (key < row_lo(a, at) || key > at) p[e / 2][e % 2] = 0.f;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) sum[e] = add2(sum[e], pair(p[e][0], p[e][1]));
        }
        float all[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float lo, hi;
          unpair(sum[e], lo, hi);
          all[e] = lo + hi;
          all[e] += __shfl_xor_sync(0xFFFFFFFFu, all[e], 1);
          all[e] += __shfl_xor_sync(0xFFFFFFFFu, all[e], 2);
        }
        const int key = key0 + u + 8 * t4;
        if (t4 < 2 && key >= k.lo && key < k.hi) w.weights[now.row0 + u + 8 * t4] = now.old + (t4 ? all[1] : all[0]);
      }
    }
    more -= unit - left;  // on to the next unit
    left = 0;
    if (more <= 0) return;
    if (++h == c.H) {
      h = 0;
      do {
        if (++s >= c.seqs) return;
        q = paged_seq(c, s, bad);
        k = key_span(w, q);
      } while (k.nt == 0);
      cost = tile_cost(w, q);
      unit = static_cast<int64_t>(k.nt) * cost;
    }
  }
}

template <int kKind, int kN>
cudaError_t launch(const WeighArgs& w, int sms, int64_t ctas, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(kBlocks<kN>) * sms;
  weigh_kernel<kKind, kN><<<static_cast<unsigned>(ctas < most ? ctas : most), 32 * kWarps, 0, s>>>(w);
  return cudaGetLastError();
}

template <int kKind, int kRows>
cudaError_t launch_mid(const WeighArgs& w, int sms, int64_t ctas, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(kMidBlocks) * sms;
  weigh_mid_kernel<kKind, kRows><<<static_cast<unsigned>(ctas < most ? ctas : most), 32 * kWarps, 0, s>>>(w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs& w, int64_t rows, int sms, int64_t key_tiles, cudaStream_t s) {
  const int64_t ctas = (key_tiles + kWarps - 1) / kWarps;
  static_assert(kWeighFewRows == 128, "the most rows of a kernel here");
  if (rows > 64) return w.a.c.kind == 0 ? launch_mid<0, 128>(w, sms, ctas, s) : launch_mid<1, 128>(w, sms, ctas, s);
  if (rows > 16) return w.a.c.kind == 0 ? launch_mid<0, 64>(w, sms, ctas, s) : launch_mid<1, 64>(w, sms, ctas, s);
  if (w.a.c.kind == 0) return rows <= 8 ? launch<0, 1>(w, sms, ctas, s) : launch<0, 2>(w, sms, ctas, s);
  return rows <= 8 ? launch<1, 1>(w, sms, ctas, s) : launch<1, 2>(w, sms, ctas, s);
}

}  // namespace sa
