// The attention weight that cached keys receive from chunks of rows (sm_103a):
// more than 128 packed rows (64, if most have many) a sequence and key head, on tcgen05 tensor cores.
//
//   w_j (+)= sum_r 2^(x_rj - L_r),   x_rj = scale log2(e) (q_r . k_j),  L_r = log2(e) lse_r
//
// The sum runs over rows, so keys are the products' M: a unit is 256 keys of
// one sequence and key head, two tiles of 128 that stay in tensor memory as
// the products' first operand while the rows that see some of them come by 96
// at a time.  A thread has a key: it reads the key's scores of 96 rows, and
// adds up their exponentials in registers.  Nothing passes between threads.
//
// A row's lse belongs to a column, which all threads read: from shared memory
// that is 768 cycles a step.  So the products subtract it, in a ninth block of
// 16 dimensions: 1 in the keys, and in the rows -lse / scale as three BF16
// parts, which hold all of its 24 bits (604 -> 580 us for 2048 rows that see all
// of 33792 keys).  A kernel in front makes the rows' blocks (made by the warps
// that bring the rows, these were what the rest waited for: 580 -> 555).  It marks
// rows whose lse is -infinity, and who issues products writes zeros over them
// first: such a row counts nothing, whatever it holds.
//
// Keys are in tensor memory because shared memory would not feed both operands:
// of a step (two tiles, 96 rows) products read Q there twice, 2 x 24 KB, and the
// copies write 24 KB, 560 cycles at 128 bytes a cycle, against 864 of the tensor
// pipe; with the keys in shared memory it would be 1060.
//
// What bounds it is the warps of keys: a step takes them 1400 cycles.  The
// exponentials are 768 of a scheduler's two warps, but a warp alone takes 650 for
// its own (their latency), reading 96 columns of tensor memory 240, and waiting
// for them and releasing them 200.  Three tiles with one place for their scores
// take 2115 cycles a step, 16 warps of 48 columns each 1650 for two tiles, a
// loop that reads ahead in thirds 1440, one of 32 columns 1640: tried, not kept.
//
// The line of all steps of all units is cut into equal parts, one a CTA; a
// unit that a cut divides is joined from its parts in order by another kernel.
//
// Warps: 0 and 1 bring the rows of Q, a box of whole tokens a step (and gather,
// 48 rows each, what is no whole box: a sequence's last rows, strides that no
// box has); 2 and 3 issue the products of tile 1 and 0 (one warp for both: 556
// against 538 us), and 3 walks the line; 4-7 and 8-11 are the keys of tile 0
// and 1.  They bring the next unit's keys into shared memory while the present
// one's rows pass, widen codes, and write them to tensor memory.
//
// Measured (graphs of four calls; tensor rate of the visible pairs):
//   2048 new of 33792, 40 / 8 heads, causal, BF16      573 us  1199 TFLOP/s
//                                            E4M3      569 us  1208
//   8704 of 8704, 24 / 24 heads, causal, BF16          212 us  1096
//
// Tensor memory: K of tile t in columns [64 t, + 64); scores of tile t, every
// other step, in [128 + 96 (2 t + b), + 96).
#include <atomic>
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kKeys = kWeighKeys;  // of a unit
constexpr int kRows = 96;          // packed rows of a step
constexpr int kStages = 5, kAhead = 2;
constexpr int kSegs = 3;
constexpr uint32_t kHalfBytes = kRows * 128;  // of a stage: 64 dimensions of its rows
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
// A unit's beginning and end, in steps.
constexpr int kOver = 3;
constexpr int kMinPlaces = 4;

constexpr int kKeyWarps = 8;
constexpr int kThreads = 32 * (4 + kKeyWarps);
// Registers after the split: their sum over warpgroups stays within the
// launch allocation (384 x 168).
constexpr uint32_t kRegsLaunch = 168, kRegsControl = 88, kRegsKeys = 208;
static_assert(kRegsControl + 2 * kRegsKeys <= 3 * kRegsLaunch, "");

// Shared memory, from a 1024-byte boundary.  The ninth blocks are laid out
// without a swizzle: 8 rows x 16 bytes together, eight rows after eight, and
// the second 16 bytes of all rows behind the first.
constexpr uint32_t kOnesBytes = 128 * 32, kShiftBytes = kRows * 32;
constexpr uint32_t kOffKeys = kStages * kStageBytes;            // the next unit's keys, as they lie in the cache
constexpr uint32_t kOffOnes = kOffKeys + kKeys * 256;           // the ninth block of the keys
constexpr uint32_t kOffShift = kOffOnes + kOnesBytes;           // [stages]: of the rows
constexpr uint32_t kOffTok = kOffShift + kStages * kShiftBytes; // [rows]: token of a step's row
constexpr uint32_t kOffSeg = kOffTok + kRows * 4;
constexpr uint32_t kOffBar = kOffSeg + kSegs * 64;
constexpr uint32_t kOffMisc = kOffBar + 512;
constexpr uint32_t kSmem = kOffMisc + 64 + 1024;
static_assert(kSmem <= 232448, "shared memory");

enum {
  BAR_QFULL = 0,     // +stage (5): warps 0 and 1, and the box
  BAR_QEMPTY = 8,    // +stage: both tiles' products
  BAR_SFULL = 16,    // +2 tile, + every other step
  BAR_SEMPTY = 20,
  BAR_KREADY = 24,   // +tile
  BAR_SEGFULL = 26,  // +segment (3)
  BAR_SEGEMPTY = 29,
  BAR_DRAIN = 32,    // +tile
  NUM_BARS = 34
};

// A matrix descriptor of a ninth block: no swizzle; 16 bytes on, and 8 rows on.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t next16, uint32_t next8) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(next16 >> 4) << 16 |
         static_cast<uint64_t>(next8 >> 4) << 32 | 1ull << 46;
}

// One step of the walk: some steps of a unit.
struct Work {
  int valid;
  int row0, n, len, h, s;
  int key0;    // first key of the unit
  int lo, hi;  // its keys whose weight is written
  int i0, i1;  // tokens of the unit's rows
  int j0;      // first of its steps
  int steps;
  int part;    // -1: the unit's weights; else the partial sums' slot (0 or 1)
};
static_assert(sizeof(Work) <= 64, "");

struct Unit {
  int lo, hi;      // keys whose weight is written
  int i0, i1;      // tokens whose rows see some of them
  int steps, places;
};

// Keys of a sequence whose weights are written: [lo, hi).
__device__ __forceinline__ void seq_span(const WeighArgs& w, const PagedSeq& q, int& lo, int& hi) {
  lo = w.accumulate ? max(w.first, row_lo(w.a, q.len - q.n)) : w.first;
  hi = q.n > 0 ? q.len : 0;
}
__device__ __forceinline__ int blocks_of(int lo, int hi) {
  return hi > lo ? (hi + kKeys - 1) / kKeys - lo / kKeys : 0;
}

// Unit b of a sequence with the span [lo, hi).
__device__ __forceinline__ Unit unit_of(const WeighArgs& w, const PagedSeq& q, int lo, int hi, int b) {
  Unit u;
  const int key0 = (lo / kKeys + b) * kKeys;
  u.lo = max(lo, key0);
  u.hi = min(hi, key0 + kKeys);
  int i0 = 0, i1 = q.n;
  const int base = q.len - q.n;  // position of the first row
  if (w.a.causal) {
    i0 = min(max(u.lo - base, 0), q.n);
    if (w.a.window) i1 = static_cast<int>(min(int64_t(q.n), max(int64_t(i0), int64_t(u.hi) - 1 + w.a.window - base)));
  }
  u.i0 = i0;
  u.i1 = i1;
  u.steps = max(1, (i1 - i0 + w.tokens - 1) / w.tokens) * w.slices;
  u.places = u.steps + kOver;
  return u;
}

// Places of one head of the sequences base + lane, one a lane.  All keys that
// lie before the first row and inside the last row's window have all rows:
// only the units beside them are looked at one by one, many of them by the
// whole warp.
__device__ __forceinline__ int64_t lane_places(const WeighArgs& w, int base, int lane, bool& bad) {
  const int s = base + lane;
  PagedSeq q;
  q.n = q.len = q.row0 = 0;
  if (s < w.a.c.seqs) {
    bool b;
    q = paged_seq(w.a.c, s, b);
    bad |= b;
  }
  int lo, hi;
  seq_span(w, q, lo, hi);
  const int n = blocks_of(lo, hi);
  int from = 0, to = n;  // units with all rows: [from, to)
  if (w.a.causal) {
    const int first = lo / kKeys;
    to = min(n, max(0, (q.len - q.n) / kKeys + 1 - first));  // those that begin at or before the first row
    if (w.a.window) {  // those that end behind what the last row sees last
      const int64_t cut = int64_t(q.len) - w.a.window;
      while (from < to && int64_t(first + from + 1) * kKeys <= cut) ++from;
    }
    if (to > 0 && max(lo, (first + to - 1) * kKeys) > q.len - q.n) --to;
    to = max(to, from);
  }
  int64_t t = 0;
  if (to > from) t = static_cast<int64_t>(to - from) * unit_of(w, q, lo, hi, from).places;
  const int others = n - (to - from);
  if (others <= 4)
#pragma unroll 1
    for (int i = 0; i < others; ++i) t += unit_of(w, q, lo, hi, i < from ? i : i + to - from).places;
  unsigned many = __ballot_sync(0xFFFFFFFFu, others > 4);
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    PagedSeq r;
    r.row0 = 0;
    r.n = __shfl_sync(0xFFFFFFFFu, q.n, src);
    r.len = __shfl_sync(0xFFFFFFFFu, q.len, src);
    const int rlo = __shfl_sync(0xFFFFFFFFu, lo, src), rhi = __shfl_sync(0xFFFFFFFFu, hi, src);
    const int rfrom = __shfl_sync(0xFFFFFFFFu, from, src), rto = __shfl_sync(0xFFFFFFFFu, to, src);
    const int rothers = __shfl_sync(0xFFFFFFFFu, others, src);
    int64_t y = 0;
#pragma unroll 1
    for (int i = lane; i < rothers; i += 32) y += unit_of(w, r, rlo, rhi, i < rfrom ? i : i + rto - rfrom).places;
    y = warp_sum(y);
    if (lane == src) t += y;
  }
  return t;
}

struct Walk {
  int64_t at, end, total;
  int ctas;
  int s, h, b;
  int skip;  // places of the unit that earlier CTAs have
  PagedSeq q;
  int lo, hi, blocks;
};

__device__ __forceinline__ void walk_to(const WeighArgs& w, Walk& k) {
  bool bad;
  k.q = paged_seq(w.a.c, k.s, bad);
  seq_span(w, k.q, k.lo, k.hi);
  k.blocks = blocks_of(k.lo, k.hi);
}

__device__ __forceinline__ void walk_start(const WeighArgs& w, Walk& k, bool& bad) {
  const int lane = threadIdx.x % 32, cta = blockIdx.x;
  const PagedArgs& c = w.a.c;
  int64_t t = 0;
#pragma unroll 1
  for (int base = 0; base < c.seqs; base += 32) t += lane_places(w, base, lane, bad);
  k.total = warp_sum(t) * c.H;
  k.ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (k.total + kMinPlaces - 1) / kMinPlaces));
  k.at = k.end = 0;
  k.s = k.h = k.b = k.skip = 0;
  if (cta >= k.ctas) return;
  k.at = muldiv(cta, k.total, k.ctas);
  k.end = muldiv(cta + 1, k.total, k.ctas);
  int64_t left = k.at;
#pragma unroll 1
  for (int base = 0;; base += 32) {
    bool b;
    const int64_t mine = lane_places(w, base, lane, b) * c.H;
    const int64_t upto = warp_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, upto > left);
    if (hit) {
      const int src = __ffs(hit) - 1;
      k.s = base + src;
      left = __shfl_sync(0xFFFFFFFFu, left - (upto - mine), src);
      t = __shfl_sync(0xFFFFFFFFu, mine, src);
      break;
    }
    left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  walk_to(w, k);
  t = muldiv(t, 1, c.H);
  k.h = static_cast<int>(muldiv(left, 1, t));
  left -= k.h * t;
  for (int b0 = 0;; b0 += 32) {
    const int64_t mine = b0 + lane < k.blocks ? unit_of(w, k.q, k.lo, k.hi, b0 + lane).places : 0;
    const int64_t upto = warp_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, upto > left);
    if (hit) {
      const int src = __ffs(hit) - 1;
      k.b = b0 + src;
      k.skip = static_cast<int>(__shfl_sync(0xFFFFFFFFu, left - (upto - mine), src));
      return;
    }
    left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
}

__device__ __forceinline__ Work walk_step(const WeighArgs& w, Walk& k, WeighJoin& join) {
  Work g;
  g.valid = 0;
  while (k.at < k.end) {
    while (k.b >= k.blocks) {  // next head, next sequence with keys
      k.b = 0;
      if (k.blocks == 0 || ++k.h >= w.a.c.H) {
        k.h = 0;
        ++k.s;
        walk_to(w, k);
      }
    }
    const Unit u = unit_of(w, k.q, k.lo, k.hi, k.b);
    const int take = static_cast<int>(min(static_cast<int64_t>(u.places - k.skip), k.end - k.at));
    const int from = max(0, k.skip - kOver), to = max(0, k.skip + take - kOver);
    if (to > from) {
      g.valid = 1;
      g.row0 = k.q.row0;
      g.n = k.q.n;
      g.len = k.q.len;
      g.h = k.h;
      g.s = k.s;
      g.key0 = (k.lo / kKeys + k.b) * kKeys;
      g.lo = u.lo;
      g.hi = u.hi;
      g.i0 = u.i0;
      g.i1 = u.i1;
      g.j0 = from;
      g.steps = to - from;
      g.part = from == 0 ? (to == u.steps ? -1 : 1) : 0;
      if (g.part == 1) {  // the CTA that holds the unit's last place
        join.pieces = static_cast<int>(muldiv((k.at - k.skip + u.places) * k.ctas - 1, 1, k.total)) - static_cast<int>(blockIdx.x) + 1;
        join.s = g.s;
        join.h = g.h;
        join.key0 = g.key0;
        join.lo = g.lo;
        join.hi = g.hi;
        join.fresh = w.accumulate ? g.len - g.n : 0;
      }
    }
    k.at += take;
    k.skip = 0;
    ++k.b;
    if (g.valid) break;
  }
  return g;
}

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
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
__device__ __forceinline__ float bf16_of(float x) {  // rounded to BF16
  return __uint_as_float(pack_bf16x2(0.f, x) & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void lds_i4(int (&v)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}

// Sums of a warp's keys over the rows of a unit's steps, once more where they are
// not numbers and the key holds an infinity or NaN: that times the zeros of rows
// that count nothing is none, though each row's own product may be.  (Other sums
// are not numbers because of a row that counts, and stay so.)  A lane has a key,
// its row of the cache (-1: none) and its sum; the lanes share the key's rows, and
// the first that is not a number ends it.  With NaN in a row or a key the long
// chunk takes 585 to 605 us as a call, 590 without; an infinite key that all of its
// 10240 rows reject adds 620.
template <int kKind>
__device__ __noinline__ float weigh_again(const WeighArgs& w, const Work& g, int key, int64_t at, float sum) {
  const PagedAttnArgs& a = w.a;
  const int lane = threadIdx.x % 32;
  bool odd = false;
  if (at >= 0 && sum != sum) {
    if constexpr (kKind != 0) {
      odd = __ldg(a.c.k_exp + at) == 255;
    } else {
      const uint4* k = reinterpret_cast<const uint4*>(a.c.k_pages + at * 256);
#pragma unroll 4
      for (int f = 0; f < 16; ++f) {
        const uint4 v = __ldg(k + f);
        for (uint32_t x : {v.x, v.y, v.z, v.w}) odd |= (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
      }
    }
  }
#pragma unroll 1
  for (unsigned left = __ballot_sync(0xFFFFFFFFu, odd); left; left &= left - 1) {
    const int src = __ffs(left) - 1, of = __shfl_sync(0xFFFFFFFFu, key, src);
    const uint4* k = reinterpret_cast<const uint4*>(a.c.k_pages + __shfl_sync(0xFFFFFFFFu, at, src) * 256);
    float part = 0.f;
    bool end = false;
#pragma unroll 1
    for (int j = g.j0; j < g.j0 + g.steps && !end; ++j) {
      const int tile = j / w.slices, e0 = (j - tile * w.slices) * w.heads, heads = min(w.heads, a.group - e0);
      const int i0 = g.i0 + tile * w.tokens, rows = (min(i0 + w.tokens, g.i1) - i0) * heads;
#pragma unroll 1
      for (int r = lane; r < rows; r += 32) {
        const int i = i0 + r / heads, pos = g.len - g.n + i;
        if ((a.causal && of > pos) || of < row_lo(a, pos)) continue;
        const int64_t row = g.row0 + i, head = static_cast<int64_t>(g.h) * a.group + e0 + r % heads;
        const float l = w.lse[row * a.Hq + head];
        if (l == -INFINITY) continue;
        if constexpr (kKind != 0) {
          part = NAN;
        } else {
          const uint4* q = reinterpret_cast<const uint4*>(a.q + row * a.q_token + head * a.q_head);
          float x = 0.f;
#pragma unroll 4
          for (int f = 0; f < 16; ++f) {
            const uint4 u = __ldg(q + f), v = __ldg(k + f);
            const uint32_t m[4] = {u.x, u.y, u.z, u.w}, n[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              x = fmaf(__uint_as_float(m[z] << 16), __uint_as_float(n[z] << 16), x);
              x = fmaf(__uint_as_float(m[z] & 0xFFFF0000u), __uint_as_float(n[z] & 0xFFFF0000u), x);
            }
          }
          part += ex2_approx((x * a.scale - l) * 1.4426950408889634f);
        }
      }
      end = __any_sync(0xFFFFFFFFu, part != part);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) part += __shfl_xor_sync(0xFFFFFFFFu, part, d);
    if (lane == src) sum = part;
  }
  return sum;
}

template <int kKind>
__global__ void __launch_bounds__(kThreads, 1)
weigh_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_shift,
                   const WeighArgs w, const WeighScratch ws) {
  const PagedAttnArgs& a = w.a;
  const PagedArgs& c = a.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(base);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * i; };
  Work* segs = reinterpret_cast<Work*>(base + kOffSeg);
  volatile int32_t* s_abort = reinterpret_cast<volatile int32_t*>(base + kOffMisc);
  int32_t* s_bad = reinterpret_cast<int32_t*>(base + kOffMisc + 4);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(base + kOffMisc + 8);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  // A step's rows: `tokens` tokens of `heads` heads (a slice of the group).
  const int step_rows = w.tokens * w.heads;

  auto shift_at = [&](int st, int row) { return reinterpret_cast<uint4*>(base + kOffShift + st * kShiftBytes + row * 16); };
  const uint4 kNothing = make_uint4(0x0000FF80u, 0, 0, 0);  // -infinity: a row that counts nothing

  // Rows of a stage that no step has are zeros throughout.
  for (int i = step_rows * 8 + threadIdx.x; i < kRows * 8; i += kThreads)
    for (int st = 0; st < 2 * kStages; ++st)
      *reinterpret_cast<uint4*>(base + st * kHalfBytes + i * 16) = make_uint4(0, 0, 0, 0);
  // The ninth blocks: three ones in each key; nothing yet in the rows.
  for (int i = threadIdx.x; i < static_cast<int>((kOnesBytes + kStages * kShiftBytes) / 16); i += kThreads) {
    const bool ones = i < 128, row = i >= 256 && (i - 256) % (2 * kRows) < kRows;
    *reinterpret_cast<uint4*>(base + kOffOnes + i * 16) =
        ones ? make_uint4(0x3F803F80u, 0x3F80u, 0, 0) : row ? kNothing : make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x < kRows) *reinterpret_cast<int*>(base + kOffTok + threadIdx.x * 4) = threadIdx.x / w.heads;
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    *s_abort = 0;
    *s_bad = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(BAR_QFULL + i), 2);
      mbar_init(bar(BAR_QEMPTY + i), 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(BAR_SFULL + i), 1);
      mbar_init(bar(BAR_SEMPTY + i), 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(BAR_KREADY + t), 4);
      mbar_init(bar(BAR_DRAIN + t), 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(bar(BAR_SEGFULL + i), 1);
      mbar_init(bar(BAR_SEGEMPTY + i), 3 + kKeyWarps);
    }
    fence_barrier_init();
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(tslot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tslot, 0);

  // By a whole warp; fails once another warp has given up, too.
  auto all_wait = [&](int b, int parity) {
    if (__all_sync(0xFFFFFFFFu, mbar_test_wait(bar(b), parity & 1))) return true;
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar(b), parity & 1, a.wait_limit) && *s_abort == 0) != 0;
  };
  auto next_seg = [&](int k, Work& g) -> bool {
    if (!all_wait(BAR_SEGFULL + k % kSegs, k / kSegs)) return false;
    g = segs[k % kSegs];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(BAR_SEGEMPTY + k % kSegs));
    return true;
  };
  bool ok = true;

  if (warp < 4) setmaxnreg_dec<kRegsControl>();
  if (warp < 2) {
    // ------------------------------------------------------------ rows
    if (warp == 0 && lane == 0 && w.boxes) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_shift);
    }
    griddep_wait();  // the rows' ninth blocks
    const uint32_t elect = elect_one();
    int x = 0, done = 0;  // steps so far; those whose copies have landed, or are boxes
    auto publish = [&](int to) {
      if (done >= to) return;
      fence_proxy_async_smem();
      __syncwarp();
      for (; done < to; ++done)
        if (lane == 0) mbar_arrive(bar(BAR_QFULL + done % kStages));
    };
    auto flush = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      publish(x);
    };
    Work g;
    int k = 0, j = 0;
    ok = next_seg(0, g);
    while (ok && g.valid) {
      const int st = x % kStages;
      ok = x < kStages || all_wait(BAR_QEMPTY + st, x / kStages - 1);
      if (!ok) break;
      const int tile = w.slices == 1 ? g.j0 + j : (g.j0 + j) / w.slices, slice = g.j0 + j - tile * w.slices;
      const int first = g.i0 + tile * w.tokens;  // token of the step's first row
      if (w.boxes && first + w.tokens <= g.i1 && (slice + 1) * w.heads <= a.group) {
        if (warp == 0 && elect) {
          mbar_arrive_expect_tx(bar(BAR_QFULL + st), step_rows * (2 * 128 + 16));
#pragma unroll
          for (int half = 0; half < 2; ++half)
            tma_load_4d(sbase + st * kStageBytes + half * kHalfBytes, &tm_q, bar(BAR_QFULL + st), half * 64,
                        slice * w.heads, g.h, g.row0 + first);
          tma_load_4d(sbase + kOffShift + st * kShiftBytes, &tm_shift, bar(BAR_QFULL + st), 0, slice * w.heads, g.h,
                      g.row0 + first);
        } else if (warp != 0 && lane == 0) {
          mbar_arrive(bar(BAR_QFULL + st));
        }
        __syncwarp();
        if (done < x) flush();
        done = ++x;
      } else {
        // a lane has row lane of the warp's 48, and half of the lanes a second one, 32 behind it
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          const int at = 48 * warp + 32 * e + lane, tok = at / w.heads, i = first + tok, sub = slice * w.heads + at - tok * w.heads;
          const bool real = (e == 0 || lane < 16) && at < step_rows && i < g.i1 && sub < a.group;
          const uint16_t* src0 = a.q;
          if (real) {
            src0 += static_cast<int64_t>(g.row0 + i) * a.q_token + static_cast<int64_t>(g.h * a.group + sub) * a.q_head;
            cp_async16(smem_u32(shift_at(st, at)), ws.shift + static_cast<int64_t>(g.row0 + i) * a.Hq + g.h * a.group + sub, true);
          } else if (e == 0 || lane < 16) {
            *shift_at(st, at) = kNothing;
          }
          const uint32_t to = sbase + st * kStageBytes + (lane % 16 / 8) * kHalfBytes + (48 * warp + 32 * e) * 128;
          const unsigned reals = __ballot_sync(0xFFFFFFFFu, real);
#pragma unroll 4
          for (int y = 0; y < (e ? 16 : 32); y += 2) {
            const int z = y + lane / 16;
            const uint16_t* src = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(src0), z));
            const bool is = reals >> z & 1;
            cp_async16(to + z * 128 + ((lane ^ z) & 7) * 16, src + (is ? lane % 16 * 8 : 0), is);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++x;
        if (x - done > kAhead) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
          publish(x - kAhead);
        }
      }
      if (++j == g.steps) {
        j = 0;
        ++k;
        // The next description may come only once the products of these steps are under way.
        if (done < x && !__all_sync(0xFFFFFFFFu, mbar_test_wait(bar(BAR_SEGFULL + k % kSegs), (k / kSegs) & 1))) flush();
        ok = next_seg(k, g);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok) publish(x);
    if (!ok) *s_abort = 1;
    if (lane == 0 && warp == 0) *reinterpret_cast<int32_t*>(base + kOffMisc + 12) = x;
  } else if (warp < 4) {
    // ------------------------------------------------------------ products of tile t; warp 3 walks the line
    const int t = 3 - warp;
    Walk walk;
    WeighJoin join;
    Work g;
    bool bad = false;
    int k = 0;  // descriptions so far
    auto give = [&]() -> bool {  // the next one, to the others
      g = walk_step(w, walk, join);
      if (k >= kSegs && !all_wait(BAR_SEGEMPTY + k % kSegs, k / kSegs - 1)) return false;
      if (lane == 0) {
        segs[k % kSegs] = g;
        mbar_arrive(bar(BAR_SEGFULL + k % kSegs));
      }
      __syncwarp();
      ++k;
      return true;
    };
    if (t == 0) {
      walk_start(w, walk, bad);
      join.pieces = 0;
      ok = give();
    } else {
      ok = next_seg(k++, g);
    }
    // (whole thirds: what is no row counts nothing)
    const uint32_t id = idesc_bf16(128, kRows, false, false);
    auto off = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4); };
    const uint64_t ones = sdesc_plain(sbase + kOffOnes, 128 * 16, 128);
    const uint32_t elect = elect_one();
    // Zeros over a stage's marked rows (both warps that read it write the same).
    auto blank_rows = [&](int st) {
      uint32_t mark[kRows / 32], any = 0;
#pragma unroll
      for (int e = 0; e < kRows / 32; ++e) any |= mark[e] = lds_u32(smem_u32(shift_at(st, 32 * e + lane)) + 12);
      if (!__any_sync(0xFFFFFFFFu, any)) return;
#pragma unroll 1
      for (int e = 0; e < kRows / 32; ++e)
        for (unsigned m = __ballot_sync(0xFFFFFFFFu, e == 0 ? mark[0] : e == 1 ? mark[1] : mark[2]); m; m &= m - 1)
          if (lane < 16)
            *reinterpret_cast<uint4*>(base + st * kStageBytes + lane / 8 * kHalfBytes + (32 * e + __ffs(m) - 1) * 128 + lane % 8 * 16) =
                make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
    };
    int st = 0, phase = 0;  // the next step's stage
    int y = 0, u = 0;       // steps and units of the tile
    bool issued = false;
    while (ok && g.valid) {
      const int steps = g.steps;
      const bool mine = g.hi > g.key0 + 128 * t;
      ok = t == 0 ? give() : next_seg(k++, g);  // (g is the next unit's from here on)
      if (!ok) break;
      if (mine) ok = all_wait(BAR_KREADY + t, u++);
#pragma unroll 1
      for (int j = 0; j < steps && ok; ++j) {
        ok = all_wait(BAR_QFULL + st, phase);
        if (!ok) break;
        if (mine) {
          blank_rows(st);
          const int s = 2 * t + (y & 1);
          ok = y < 2 || all_wait(BAR_SEMPTY + s, y / 2 - 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + 128 + kRows * s;
          const uint64_t qs = sdesc_sw128(sbase + st * kStageBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) umma_ts_elect(d, tmem + 64 * t + 8 * kk, qs + off(kk), id, kk > 0 ? 1u : 0u, elect);
          umma_ss_elect(d, ones, sdesc_plain(sbase + kOffShift + st * kShiftBytes, kRows * 16, 128), id, 1u, elect);
          if (elect) {
            umma_commit(bar(BAR_SFULL + s));
            umma_commit(bar(BAR_QEMPTY + st));
          }
          issued = true;
          ++y;
        } else if (elect) {
          mbar_arrive(bar(BAR_QEMPTY + st));
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) *s_abort = 1;
    if (elect && issued) {  // products in flight complete before the CTA ends
      umma_commit(bar(BAR_DRAIN + t));
      mbar_wait(bar(BAR_DRAIN + t), 0, kWaitLimitNs);
    }
    if (t == 0) {
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (lane == 0) {
        ws.join[blockIdx.x] = join;
        if (bad) *s_bad = 1;
      }
    }
  } else {
    // ------------------------------------------------------------ keys of tile t
    setmaxnreg_inc<kRegsKeys>();
    const int t = (warp - 4) / 4;
    const int row = (warp & 3) * 32 + lane;  // of the tile: a lane of tensor memory
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t k_col = tmem + lane_addr + 64 * t;
    const float c2 = a.scale * 1.4426950408889634f;
    const uint64_t c2x = f2(c2, c2);
    auto has = [&](const Work& g) { return g.valid && g.hi > g.key0 + 128 * t; };
    // The next unit's key comes into shared memory (a thread's own row, its 16-byte
    // chunks in another order in every row for the banks' sake).
    constexpr int kRow = kKind == 0 ? 256 : 128, kChunks = kRow / 16;
    uint32_t exp = 0;
    float next_old = 0.f;
    int64_t next_at = -1;  // of its weight; -1: none is written
    const uint32_t mine = sbase + kOffKeys + (t * 128 + row) * kRow;
    auto load = [&](const Work& g) {
      next_at = -1;
      next_old = 0.f;
      exp = 0;
      const int j = g.key0 + 128 * t + row;
      if (has(g) && j >= g.lo && j < g.hi) {
        const int page = __ldg(c.table + g.s * c.table_stride + (j >> c.page_shift));
        if (page < 0 || page >= c.pages)
          *s_bad = 1;
        else
          next_at = ((static_cast<int64_t>(page) * c.H + g.h) << c.page_shift) + (j & (c.page_size - 1));
      }
      const bool is = next_at >= 0;
      const uint8_t* src = c.k_pages + (is ? next_at * kRow : 0);
#pragma unroll
      for (int e = 0; e < kChunks; ++e) cp_async16(mine + (e ^ (row % 8)) * 16, src + (is ? 16 * e : 0), is);
      if (is) {
        if constexpr (kKind != 0) exp = __ldg(c.k_exp + next_at);
        if (w.accumulate && j < g.len - g.n) next_old = w.weights[next_at];
      }
    };
    // The key in BF16 into tensor memory, 32 columns at a time.
    auto store = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      // codes land as the value times 2^-120; two factors, of 2^120 and the row's scale
      const uint32_t e1 = min(exp, 134u), two = exp == 255 ? 0x7FFF7FFFu : (e1 + 120) * 0x00800080u;
      const uint32_t more = (exp == 255 ? 127u : exp - e1 + 127) * 0x00800080u;
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        uint32_t z[32];
#pragma unroll
        for (int e = 0; e < kChunks / 2; ++e) {
          uint32_t in[4];
          lds_i4(reinterpret_cast<int(&)[4]>(in), mine + ((b * (kChunks / 2) + e) ^ (row % 8)) * 16);
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const uint32_t v = in[f];
            if constexpr (kKind == 0) {
              z[4 * e + f] = v;
            } else {
              const uint32_t even = bf16x2_mul(bf16x2_mul(((v * 16) & 0x07F007F0u) | ((v * 256) & 0x80008000u), two), more);
              const uint32_t odd = bf16x2_mul(bf16x2_mul(((v >> 4) & 0x07F007F0u) | (v & 0x80008000u), two), more);
              z[8 * e + 2 * f] = __byte_perm(even, odd, 0x5410);
              z[8 * e + 2 * f + 1] = __byte_perm(even, odd, 0x7632);
            }
          }
        }
        tmem_st32(k_col + 32 * b, z);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_KREADY + t));
    };
    int y = 0;  // steps of the tile
    Work g, next;
    int64_t at = -1;
    float old = 0.f;
    ok = next_seg(0, g);
    if (ok) {
      load(g);
      if (has(g)) store();
      at = next_at;
      old = next_old;
    }
    for (int k = 0; ok && g.valid; ++k) {
      ok = next_seg(k + 1, next);
      if (!ok) break;
      load(next);
      if (!has(g)) {
        if (has(next)) store();
      } else {
        const int j0 = g.key0 + 128 * t + row;
        // Steps [0, e0) and [e1, ..) have rows that miss some key of the unit.
        int e0 = 0, e1 = g.j0 + g.steps;
        if (a.causal) {
          const int64_t p0 = g.len - g.n + g.i0;  // position of the unit's first row
          e0 = static_cast<int>((max(int64_t(0), g.hi - 1 - p0) + w.tokens - 1) / w.tokens) * w.slices;
          if (a.window) {
            const int64_t far = g.lo + int64_t(a.window) + 1 - p0;  // tokens until one misses the unit's first key
            e1 = static_cast<int>(min(int64_t(e1), far <= w.tokens ? 0 : (far - 1) / w.tokens * w.slices));
          }
        }
        uint64_t acc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[b] = f2(0.f, 0.f);
        uint32_t z[kRows / 32][32];
        // The scores of the unit's step j are there, and on their way.
        auto arrived = [&](int j) -> bool {
          const int s = 2 * t + (y & 1);
          if (!all_wait(BAR_SFULL + s, y / 2)) return false;
          tc_fence_after();
          const uint32_t col = tmem + lane_addr + 128 + kRows * s;
          if (g.j0 + j < e0 || g.j0 + j >= e1) {
            // masked in place: a second copy of the sums, with the mask in it,
            // is not in the instruction cache (1002 us against 846 for the long chunk)
            const int tile = w.slices == 1 ? g.j0 + j : (g.j0 + j) / w.slices;
            const int p0 = g.len - g.n + g.i0 + tile * w.tokens, k0 = j0 - lane;  // the step's first row, the warp's first key
#pragma unroll 1
            for (int b = 0; b < kRows; b += 16) {
              int tok[16];
#pragma unroll
              for (int e = 0; e < 16; e += 4) lds_i4(*reinterpret_cast<int(*)[4]>(&tok[e]), sbase + kOffTok + 4 * (b + e));
              const int pa = p0 + tok[0], pz = p0 + tok[15];
              if (k0 + 31 <= pa && (!a.window || k0 > pz - a.window)) continue;  // all are seen
              uint32_t v[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(-INFINITY);
              if (k0 <= pz && (!a.window || k0 + 31 > pa - a.window)) {  // some are
                tmem_ld16(col + b, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (j0 > p0 + tok[e] || (a.window && j0 <= p0 + tok[e] - a.window)) v[e] = __float_as_uint(-INFINITY);
              }
              tmem_st16(col + b, v);
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int b = 0; b < kRows / 32; ++b) tmem_ld32(col + 32 * b, z[b]);
          // no product reads the unit's keys any more
          if (j + 1 == g.steps && has(next)) store();
          return true;
        };
#pragma unroll 1
        for (int j = 0; j < g.steps; ++j) {
          ok = arrived(j);
          if (!ok) break;
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_SEMPTY + 2 * t + (y & 1)));
          ++y;
#pragma unroll
          for (int b = 0; b < kRows / 32; ++b) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float p0, p1;
              unf2(fmul2(f2(__uint_as_float(z[b][e]), __uint_as_float(z[b][e + 1])), c2x), p0, p1);
              acc[e / 2 % 4] = fadd2(acc[e / 2 % 4], f2(ex2_approx(p0), ex2_approx(p1)));
            }
          }
        }
        if (!ok) break;
        float p, q;
        unf2(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), p, q);
        float sum = p + q;
        if (__any_sync(0xFFFFFFFFu, sum != sum && at >= 0)) sum = weigh_again<kKind>(w, g, j0, at, sum);
        if (g.part >= 0)
          ws.part[(static_cast<int64_t>(blockIdx.x) * 2 + g.part) * kKeys + 128 * t + row] = sum;
        else if (at >= 0)
          w.weights[at] = old + sum;
      }
      at = next_at;
      old = next_old;
      g = next;
    }
    if (!ok) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      tmem_wait_st();
      *s_abort = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Where a warp has given up, nobody may have waited for the last boxes: they
  // land before the CTA ends (bounded; a stage without a box may not fill).
  if (warp == 0 && *s_abort) {
    const int n = *reinterpret_cast<volatile int32_t*>(base + kOffMisc + 12);
    for (int x = max(0, n - kStages); x < n; ++x) mbar_wait(bar(BAR_QFULL + x % kStages), (x / kStages) & 1, kWaitLimitNs / 100);
  }
  if (warp == 3) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) ws.cta_status[blockIdx.x] = *s_abort ? 5 /* SA_ETIMEOUT */ : (*s_bad ? kPagedInvalid : 0);
  griddep_launch_dependents();
}

// The rows' ninth blocks: -lse / scale = hi + mid + lo in BF16; and ones, which the
// keys multiply by 0, as the mark of a row that counts nothing.
__global__ void __launch_bounds__(256) weigh_shift_kernel(const WeighArgs w, const WeighScratch ws) {
  griddep_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= static_cast<int64_t>(w.a.c.rows) * w.a.Hq) return;
  const float l = w.lse[at];
  const float v = l == -INFINITY ? -INFINITY : -l / w.a.scale;
  const float hi = bf16_of(v);
  const float mid = isfinite(hi) ? bf16_of(v - hi) : 0.f, lo = isfinite(hi) ? v - hi - mid : 0.f;
  ws.shift[at] = make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(lo, 0.f), 0, l == -INFINITY ? 0x3F803F80u : 0u);
}

// The units that a cut divided, their parts in order; and the call's status.
__global__ void __launch_bounds__(kKeys) weigh_join_kernel(const WeighArgs w, const WeighScratch ws) {
  griddep_wait();
  const PagedArgs& c = w.a.c;
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    int st = 0;
    for (int i = threadIdx.x; i < gridDim.x; i += 32) st = max(st, ws.cta_status[i]);
    st = __reduce_max_sync(0xFFFFFFFFu, st);
    if (threadIdx.x == 0) *c.status = st;
  }
  const WeighJoin d = ws.join[blockIdx.x];
  const int j = d.key0 + threadIdx.x;
  if (d.pieces == 0 || j < d.lo || j >= d.hi) return;
  const int page = c.table[d.s * c.table_stride + (j >> c.page_shift)];
  if (page < 0 || page >= c.pages) return;  // (reported)
  float sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < d.pieces; ++i)
    sum += ws.part[(static_cast<int64_t>(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * kKeys + threadIdx.x];
  float* to = w.weights + ((static_cast<int64_t>(page) * c.H + d.h) << c.page_shift) + (j & (c.page_size - 1));
  *to = (j < d.fresh ? *to : 0.f) + sum;
}

template <int kKind>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_shift, const WeighArgs& w, const WeighScratch& ws, int ctas, cudaStream_t s) {
  auto* kern = weigh_chunk_kernel<kKind>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(kern), kSmem);
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
  if (regs * 3 < static_cast<int>(kRegsControl + 2 * kRegsKeys)) return cudaErrorInvalidConfiguration;
  const int64_t all = static_cast<int64_t>(w.a.c.rows) * w.a.Hq;
  weigh_shift_kernel<<<static_cast<unsigned>((all + 255) / 256), 256, 0, s>>>(w, ws);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_dependent(kern, dim3(ctas), dim3(kThreads), kSmem, s, tm_q, tm_shift, w, ws);
  if (e != cudaSuccess) return e;
  return launch_dependent(weigh_join_kernel, dim3(ctas), dim3(kKeys), 0, s, w, ws);
}

}  // namespace

cudaError_t launch_weigh_chunk(WeighArgs w, const WeighScratch& ws, int ctas, cudaStream_t s) {
  const PagedAttnArgs& a = w.a;
  w.heads = a.group < kRows ? a.group : kRows;
  w.tokens = kRows / w.heads;
  w.slices = (a.group + w.heads - 1) / w.heads;
  CUtensorMap tm_q{}, tm_shift{};
  w.boxes = make_map_heads(&tm_q, a.q, a.c.rows, a.c.H, a.group, a.q_token, a.q_head, w.tokens, w.heads) &&
            make_map_heads16(&tm_shift, ws.shift, a.c.rows, a.c.H, a.group, w.tokens, w.heads);
  return a.c.kind == 0 ? launch<0>(tm_q, tm_shift, w, ws, ctas, s) : launch<1>(tm_q, tm_shift, w, ws, ctas, s);
}

}  // namespace sa
