// The attention weight that cached keys receive (sm_103a):
//
//   w_j (+)= sum over rows r that see key j, and query heads of its group, of
//            2^(x_rj - L_r),   x_rj = scale log2(e) (q_r . k_j),  L_r = log2(e) lse_r
//
// A key's weight depends on its own K alone, so whoever has a key adds up all
// rows for it: nothing is joined, and no atomics change an order.
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4, kBlocks = 4;  // blocks an SM
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
// Codes (c0, c2) and (c1, c3) of a word as BF16 pairs, times 2^-7.
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

// Rows of Q: as the second operand of K Q^T, 8 kN of them.  A lane has row
// lane / 4 of each eight, and 16-byte chunks lane % 4 + 4 i of it, as of K's
// rows: the order of dimensions inside a product is free as long as both have
// the same.
template <int kKind, int kN>
struct Rows {
  uint32_t q[kN][8][2];
  float neg[kN][2];        // -L of rows 2 t, 2 t + 1 of each eight (-inf: counts nothing)
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
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (kKind == 0) {
          if (rho < rows) x = __ldg(reinterpret_cast<const uint4*>(src + 8 * (t4 + 4 * e)));
          q[n][2 * e][0] = x.x;
          q[n][2 * e][1] = x.y;
          q[n][2 * e + 1][0] = x.z;
          q[n][2 * e + 1][1] = x.w;
        } else {
          // 16 codes of K are 32 bytes here; a word's codes are taken as (c0, c2), (c1, c3)
          if (rho < rows) x = __ldg(reinterpret_cast<const uint4*>(src + 16 * (t4 + 4 * (e / 2)) + 8 * (e % 2)));
          q[n][2 * e][0] = __byte_perm(x.x, x.y, 0x5410);
          q[n][2 * e][1] = __byte_perm(x.x, x.y, 0x7632);
          q[n][2 * e + 1][0] = __byte_perm(x.z, x.w, 0x5410);
          q[n][2 * e + 1][1] = __byte_perm(x.z, x.w, 0x7632);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rho0 + 8 * n + 2 * t4 + e;
        const int j = div_group(a, r), pos = s.len - s.n + j;
        const bool real = r < rows;
        float l = INFINITY;
        if (real) l = __ldg(w.lse + static_cast<int64_t>(s.row0 + j) * a.Hq + h * a.group + r - j * a.group);
        neg[n][e] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
        lo[n][e] = real ? row_lo(a, pos) : 0;
        hi[n][e] = real ? (a.causal ? min(s.len, pos + 1) : s.len) : 0;
      }
    }
  }
};

// A tile of 16 keys: keys u and u + 8 of the lanes of a row.
template <int kKind>
struct Tile {
  uint4 x[2][kKind == 0 ? 4 : 2];
  float scale[2];  // of their logits
  float old;       // the weight that this lane writes
  int64_t row0;    // first row of the cache; -1: not to be looked at
  int key0, lo, hi;
  bool fresh;      // the first of its unit
  PagedSeq q;
  int h;
};

template <int kKind, int kN>  // kN: tiles of eight rows
__global__ void __launch_bounds__(32 * kWarps, kBlocks) weigh_kernel(const WeighArgs w) {
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
  // The next tile of the part, its loads under way.
  auto fetch = [&](Tile<kKind>& n) {
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
    n.lo = k.lo;
    n.hi = k.hi;
    n.fresh = fresh;
    n.q = q;
    n.h = h;
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
    n.row0 = -1;
    if (page < 0 || page >= c.pages) {
      if (lane == 0) paged_fail(c);
      return;
    }
    n.row0 = ((static_cast<int64_t>(page) * c.H + h) << c.page_shift) + (n.key0 & (c.page_size - 1));
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) n.x[e][i] = ld_stream(c.k_pages + (n.row0 + u + 8 * e) * kRow + 16 * (t4 + 4 * i));
#pragma unroll
    for (int e = 0; e < 2; ++e) n.scale[e] = kKind == 0 ? c2 : exp_scale(__ldg(c.k_exp + n.row0 + u + 8 * e)) * (128.0f * c2);
    // lanes t = 0 and 1 of each four write keys u and u + 8
    const int key = n.key0 + u + 8 * t4;
    n.old = 0.f;
    if (t4 < 2 && key >= k.lo && key < q.len - q.n && w.accumulate) n.old = w.weights[n.row0 + u + 8 * t4];
  };
  Rows<kKind, kN> rows;
  bool need = false;  // the unit's rows are to be loaded
  Tile<kKind> now, next;
  fetch(now);
#pragma unroll 1
  for (; at < end; ++at) {
    if (at + 1 < end) fetch(next);
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
            const uint32_t e0 = codes_even(k0[e]), o0 = codes_odd(k0[e]), e1 = codes_even(k1[e]), o1 = codes_odd(k1[e]);
#pragma unroll
            for (int n = 0; n < kN; ++n) mma_bf16(d[n], e0, e1, o0, o1, rows.q[n][4 * i + e][0], rows.q[n][4 * i + e][1]);
          }
        }
      }
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // key u + 8 (e / 2), row 2 t + e % 2
          const int j = now.key0 + u + 8 * (e / 2);
          const float p = ex2_approx(fmaf(d[n][e], now.scale[e / 2], rows.neg[n][e & 1]));
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
    now = next;
  }
}

template <int kKind, int kN>
cudaError_t launch(const WeighArgs& w, int ctas, cudaStream_t s) {
  weigh_kernel<kKind, kN><<<ctas, 32 * kWarps, 0, s>>>(w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs& w, int64_t rows, int sms, int64_t key_tiles, cudaStream_t s) {
  int64_t ctas = (key_tiles + kWarps - 1) / kWarps;
  if (ctas > kBlocks * sms) ctas = kBlocks * sms;
  const int n = static_cast<int>(ctas);
  if (w.a.c.kind == 0) return rows <= 8 ? launch<0, 1>(w, n, s) : launch<0, 2>(w, n, s);
  return rows <= 8 ? launch<1, 1>(w, n, s) : launch<1, 2>(w, n, s);
}

}  // namespace sa
