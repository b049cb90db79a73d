// Writing rows of K and V into a paged cache and reading them back, for
// sm_103a: BF16 rows are moved as they are; E4M3 rows are quantised with one
// power-of-two scale a row (see include/sparse_attn.h for the format).
//
// Both are bound by memory: a row of one head is 256 bytes of BF16 against
// 256, or 128 + 1, in the cache.  A warp takes one token and kHeads heads of
// it; its halves take K and V, 16 lanes a row, 8 elements a lane, so a row's
// largest magnitude is a 16-bit integer maximum over 8 values and four
// shuffles.  The rows' loads do not wait for the look-up of the sequence and
// its page; in cache_read they have to.
//
// Measured (a copy reaches 6.78 TB/s): writing 9505 tokens of 56 heads as E4M3
// 68 us, 6.0 TB/s (four tokens a warp instead of one: slower); reading
// 67608 tokens of 24 heads back 186 us, 6.72 TB/s; one token of 32 sequences
// and 8 heads 5.3 us alone and 3.2 among others, a launch and two dependent
// look-ups.
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;
// Heads a warp moves at once, 16 bytes a lane of each in flight.  Eight take as
// long for 56 heads (70 us) and longer for one token of 8 heads (6.2 against
// 5.3 us); fourteen 75 us.
constexpr int kHeads = 4;

// 16 bytes that this kernel reads once.
__device__ __forceinline__ uint4 ld_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The row of page table that holds the token of packed row r, as the index
// page * page_size * H + slot of head 0 (heads are page_size rows apart); -1
// when there is none.  `pos` is the token's position (below 0: no token).
__device__ __forceinline__ int64_t slot_of(const PagedArgs& c, int r, int lane, bool& member, int& pos) {
  member = false;
  pos = -1;
  const int s = paged_find(c, r, lane);
  if (s < 0) return -1;
  bool bad;
  const PagedSeq q = paged_seq(c, s, bad);
  if (bad) {
    if (lane == 0) paged_fail(c);
    return -1;
  }
  if (r < q.row0 || r >= q.row0 + q.n) return -1;
  member = true;
  pos = q.len - q.n + (r - q.row0);
  if (pos < 0) return -1;
  const int page = c.table[s * c.table_stride + (pos >> c.page_shift)];
  if (page < 0 || page >= c.pages) {
    if (lane == 0) paged_fail(c);
    return -1;
  }
  return (static_cast<int64_t>(page) * c.H << c.page_shift) + (pos & (c.page_size - 1));
}

// Eight codes (BF16 pairs scaled by 2^-e already).
__device__ __forceinline__ uint2 to_codes(const uint32_t (&v)[4]) {
  uint16_t half[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(half[k])
        : "f"(__uint_as_float(v[k] & 0xFFFF0000u)), "f"(__uint_as_float(v[k] << 16)));
  return make_uint2(half[0] | (static_cast<uint32_t>(half[1]) << 16), half[2] | (static_cast<uint32_t>(half[3]) << 16));
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t v;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(a), "r"(b));
  return v;
}

// From 248 * 2^120 on, the nearest code would stand for 256 * 2^120, which is
// no BF16 number: such elements take 240's, like the largest that round to it.
// Only rows of the exponent 120 have them.  One thread writes such a row once
// more, after the barrier behind its first writing: in the kernel's main path
// a test for it took 2 to 4 us of 67 (9505 tokens of 56 heads).
constexpr int kLargestExp = 247;
__device__ __noinline__ void rewrite_largest(const uint16_t* src, uint8_t* dst) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    const uint4 x = ld_once(src + 8 * i);
    uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = bf16x2_mul(__vminu2(v[k] & 0x7FFF7FFFu, 0x7F777F77u) | (v[k] & 0x80008000u), (254 - kLargestExp) * 0x00800080u);
    *reinterpret_cast<uint2*>(dst + 8 * i) = to_codes(v);
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const PagedArgs c, const CacheRows rows, int blocks_h) {
  if (blockIdx.x == 0) paged_check_all(c);
  constexpr int kTile = kThreads / 32;  // rows of the CTA, one a warp
  __shared__ int64_t s_slot[kTile];
  __shared__ uint8_t s_exp[2][kHeads][kTile];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int r = static_cast<int>(blockIdx.x / blocks_h) * kTile + warp, h0 = static_cast<int>(blockIdx.x % blocks_h) * kHeads;
  const bool is_v = lane >= 16;
  const int sub = lane % 16;
  const int64_t head = is_v ? rows.v_head : rows.k_head, token = is_v ? rows.v_token : rows.k_token;
  const uint16_t* src = (is_v ? rows.v : rows.k) + r * token + h0 * head + sub * 8;
  uint4 x[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    if (r < c.rows && h0 + i < c.H) x[i] = ld_once(src + i * head);
  }
  uint8_t* pages = is_v ? c.v_pages : c.k_pages;
  bool member;
  int pos;
  const int64_t slot = r < c.rows ? slot_of(c, r, lane, member, pos) : -1;
  if (kE4m3 && lane == 0) s_slot[warp] = slot;
  // E4M3: the largest magnitude of a row over its 16 lanes.  BF16 bits without
  // the sign order as integers; two heads' maxima share a word.
  uint32_t top[kHeads / 2];
  if constexpr (kE4m3) {
#pragma unroll
    for (int i = 0; i < kHeads; i += 2) {
      uint32_t m[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 v = x[i + k];
        m[k] = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
      }
      uint32_t y = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
#pragma unroll
      for (int d = 1; d < 16; d *= 2) y = __vmaxu2(y, __shfl_xor_sync(0xFFFFFFFFu, y, d));
      top[i / 2] = y;
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int64_t row = slot + (static_cast<int64_t>(h0 + i) << c.page_shift);
    const bool real = slot >= 0 && h0 + i < c.H;
    if constexpr (!kE4m3) {
      if (real) *reinterpret_cast<uint4*>(pages + row * 256 + sub * 16) = x[i];
    } else {
      const uint32_t m = i % 2 ? top[i / 2] >> 16 : top[i / 2] & 0xFFFFu;
      // amax = (1 + M / 128) 2^(E - 127) <= 1.75 * 2^8 * 2^e with M <= 96 for e = E - 135
      const bool finite = m < 0x7F80u;
      const int e = finite ? max(1, static_cast<int>((m + 31) >> 7) - 8) : 255;
      // times 2^(127 - e), exact in BF16; NaN makes every code of the row one
      const uint32_t inv = finite ? (254 - e) * 0x00800080u : 0x7FFF7FFFu;
      const uint32_t v[4] = {bf16x2_mul(x[i].x, inv), bf16x2_mul(x[i].y, inv), bf16x2_mul(x[i].z, inv),
                             bf16x2_mul(x[i].w, inv)};
      if (real) *reinterpret_cast<uint2*>(pages + row * 128 + sub * 8) = to_codes(v);
      if (sub == 0) s_exp[is_v][i][warp] = static_cast<uint8_t>(e);
    }
  }
  if constexpr (kE4m3) {
    // the exponents of consecutive tokens of one head lie side by side
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kHeads * kTile; i += kThreads) {
      const int t = i % kTile, h = i / kTile % kHeads, v = i / (kTile * kHeads);
      if (s_slot[t] >= 0 && h0 + h < c.H) {
        const int64_t row = s_slot[t] + (static_cast<int64_t>(h0 + h) << c.page_shift);
        const uint8_t e = s_exp[v][h][t];
        (v ? c.v_exp : c.k_exp)[row] = e;
        if (e == kLargestExp) {
          const int r1 = r - warp + t;
          rewrite_largest(v ? rows.v + r1 * rows.v_token + (h0 + h) * rows.v_head
                            : rows.k + r1 * rows.k_token + (h0 + h) * rows.k_head,
                          (v ? c.v_pages : c.k_pages) + row * 128);
        }
      }
    }
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const PagedArgs c, const CacheRows rows, int blocks_h) {
  if (blockIdx.x == 0) paged_check_all(c);
  const int lane = threadIdx.x % 32;
  const int r = static_cast<int>(blockIdx.x / blocks_h) * (kThreads / 32) + threadIdx.x / 32;
  const int h0 = static_cast<int>(blockIdx.x % blocks_h) * kHeads;
  if (r >= c.rows) return;
  const bool is_v = lane >= 16;
  const int sub = lane % 16;
  uint16_t* dst = (is_v ? rows.v + r * rows.v_token : rows.k + r * rows.k_token) + sub * 8;
  const int64_t head = is_v ? rows.v_head : rows.k_head;
  bool member;
  int pos;
  const int64_t slot = slot_of(c, r, lane, member, pos);
  if (!member) return;
  const uint8_t* pages = is_v ? c.v_pages : c.k_pages;
  const uint8_t* exps = is_v ? c.v_exp : c.k_exp;
  uint4 x[kHeads];
  uint32_t e[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    e[i] = 0;
    if (h0 + i >= c.H || slot < 0) continue;
    const int64_t row = slot + (static_cast<int64_t>(h0 + i) << c.page_shift);
    if constexpr (!kE4m3) {
      x[i] = __ldg(reinterpret_cast<const uint4*>(pages + row * 256 + sub * 16));
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(pages + row * 128 + sub * 8));
      x[i].x = v.x;
      x[i].y = v.y;
      e[i] = __ldg(exps + row);
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (h0 + i >= c.H) break;
    if constexpr (kE4m3) {
      const float two = exp_scale(e[i]);
      const uint32_t v[2] = {x[i].x, x[i].y};
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float lo, hi;
        e4m3x2_f32(static_cast<uint16_t>(v[k / 2] >> (16 * (k % 2))), lo, hi);
        w[k] = pack_bf16x2(lo * two, hi * two);  // exact: 4 significant bits
      }
      x[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(dst + (h0 + i) * head) = x[i];
  }
}

template <typename K>
cudaError_t launch_rows(K kern, const PagedArgs& c, const CacheRows& r, cudaStream_t s) {
  const int blocks_h = (c.H + kHeads - 1) / kHeads;
  const int64_t grid = (static_cast<int64_t>(c.rows) + kThreads / 32 - 1) / (kThreads / 32) * blocks_h;
  kern<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(c, r, blocks_h);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const PagedArgs& c, const CacheRows& r, cudaStream_t s) {
  return c.kind ? launch_rows(cache_write_kernel<true>, c, r, s) : launch_rows(cache_write_kernel<false>, c, r, s);
}

cudaError_t launch_cache_read(const PagedArgs& c, const CacheRows& r, cudaStream_t s) {
  return c.kind ? launch_rows(cache_read_kernel<true>, c, r, s) : launch_rows(cache_read_kernel<false>, c, r, s);
}

}  // namespace sa
