// The batch description of the paged-cache calls, read and checked on the
// device (see include/sparse_attn.h): a sequence that fails a check has no
// rows, a page out of range is skipped, and both set the status word.
#pragma once

#include <cstdint>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace sa {

constexpr int kPagedInvalid = 1;  // SA_EINVAL

__device__ __forceinline__ void paged_fail(const PagedArgs& c) {
  if (c.status) atomicCAS(c.status, 0, kPagedInvalid);
}

struct PagedSeq {
  int row0;  // first row
  int n;     // rows (new tokens)
  int len;   // cached tokens, the new ones among them
};

// One of the line's sequences where some share a prefix (SharedAttnArgs).
struct SharedSeq : PagedSeq {
  int row;    // of the table
  int page0;  // first page (0: all keys are its own); -1: the keys are a prefix, and all rows of its group see all of them
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& c, int s, bool& bad) {
  PagedSeq q;
  const int r0 = c.row_start[s], r1 = c.row_start[s + 1];
  q.len = c.kv_len[s];
  bad = r0 < 0 || r1 < r0 || r1 > c.rows || r1 - r0 > c.max_new || q.len < 0 ||
        q.len > (static_cast<int64_t>(c.table_width) << c.page_shift);
  q.row0 = r0;
  q.n = bad ? 0 : r1 - r0;
  return q;
}

// Reports a bad sequence that no row may lead to (one CTA of a grid does it).
__device__ __forceinline__ void paged_check_all(const PagedArgs& c) {
  if (!c.status) return;
  for (int s = threadIdx.x; s < c.seqs; s += blockDim.x) {
    bool bad;
    paged_seq(c, s, bad);
    if (bad) paged_fail(c);
  }
}

// The last sequence that starts at or before row r (-1 if none), by the whole
// warp: 32 starts are compared at a time.
__device__ __forceinline__ int paged_find(const PagedArgs& c, int r, int lane) {
  int lo = 0, n = c.seqs;
  while (true) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool below = at < n && c.row_start[lo + at] <= r;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, below));
    if (k == 0) return lo == 0 ? -1 : lo - 1;  // (only an unsorted array gets here with lo > 0)
    lo += (k - 1) * step;
    if (step == 1) return lo;
    n = min(step, n - (k - 1) * step);
  }
}

// 2^(e - 127) of an exponent byte; 255 is a row that is not a number.
__device__ __forceinline__ float exp_scale(uint32_t e) {
  return __uint_as_float(e == 255 ? 0x7FFFFFFFu : e << 23);
}

// Arrives on `bar` when this thread's cp.async so far have completed (counted
// among the barrier's arrivals).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

// An untiled copy into shared memory, counted on `bar` (both ends 16-byte
// aligned, bytes a multiple of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 16 bytes, or zeros when !real.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// Two E4M3 codes (the low 16 bits) as FP32 values.
__device__ __forceinline__ void e4m3x2_f32(uint16_t v, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

// ---- work of paged_fwd
//
// The rows of a sequence under one key head are packed as rho = i * group + g
// (new token i, query head g of the group), so that a tile of them reads the
// same keys.  A unit is a tile of `row_tile` packed rows of one sequence and
// key head; its work is the tiles of key_tile keys between the first
// key of its first row and the last key of its last one (one empty tile when
// there is none, so that every unit writes its rows).  All key tiles of all
// units, in the order (sequence, head, row tile, key tile), are one line that
// is cut into equal parts, one a CTA: every CTA streams the same number of
// however ragged the batch is.  A unit's beginning and end cost time too:
// in front of its key tiles the line has `over` places without one.  Nor does
// a key tile cost the same under few rows as under many: it has `half` places
// in units that fill at most half of the row tile, else `full`, and belongs to
// the CTA that has the first of them.  A unit that a cut divides is joined
// from its parts by the joining kernel.

template <int kRowTile, int kKeyTile, int kHalf, int kFull, int kOver, int kMinPlaces, bool kSingle>
struct LineShape {
  static constexpr int row_tile = kRowTile;           // packed rows of a unit
  static constexpr int key_tile = kKeyTile;           // keys of a tile
  static constexpr int half = kHalf, full = kFull;    // places of a key tile
  static constexpr int over = kOver;                  // places of a unit without a key tile
  static constexpr int min_places = kMinPlaces;       // of a CTA at least (>= full), while there are any
  static constexpr bool single = kSingle;             // a sequence and key head are one unit at most
};

// x / group (x >= 0).
__device__ __forceinline__ int div_group(const PagedAttnArgs& a, int x) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(x)) * a.group_mul) >> a.group_shift);
}

struct UnitKeys {
  int lo, hi;  // keys that some row of the unit sees: [lo, hi)
  int t0, nt;  // key tiles
  int each;    // places of one
  int places;  // of the unit
};

// First key that the row at position pos sees.
__device__ __forceinline__ int row_lo(const PagedAttnArgs& a, int pos) {
  return a.window ? static_cast<int>(max(int64_t(0), int64_t(pos) + 1 - a.window)) : 0;
}

__device__ __forceinline__ int row_tiles(const PagedAttnArgs& a, const PagedSeq& q, int row_tile) {
  return static_cast<int>((static_cast<uint32_t>(q.n) * static_cast<uint32_t>(a.group) + row_tile - 1) /
                          static_cast<uint32_t>(row_tile));
}

// The sequences of a line: those of the batch, or, where some share a prefix,
// the prefixes of the groups (the rows of all of a group's sequences over the
// whole pages of its prefix) and then the sequences with their own keys.
__device__ __forceinline__ int line_seqs(const PagedAttnArgs& a) { return a.c.seqs; }
__device__ __forceinline__ PagedSeq line_seq(const PagedAttnArgs& a, int s, bool& bad) { return paged_seq(a.c, s, bad); }
__device__ __forceinline__ bool line_causal(const PagedAttnArgs& a, const PagedSeq&) { return a.causal; }

__device__ __forceinline__ int line_seqs(const SharedAttnArgs& a) {
  return (a.parts & 1 ? a.groups : 0) + (a.parts & 2 ? a.c.seqs : 0);
}
__device__ __forceinline__ bool line_causal(const SharedAttnArgs& a, const SharedSeq& q) { return a.causal && q.page0 >= 0; }

// Shared pages of group g (0 where it has less than two sequences), and its
// sequences [s0, s1).
__device__ __forceinline__ int shared_pages(const SharedAttnArgs& a, int g, int& s0, int& s1, bool& bad) {
  s0 = a.group_start[g];
  s1 = a.group_start[g + 1];
  const int len = a.prefix_len[g];
  bad = s0 < 0 || s1 < s0 || s1 > a.c.seqs || len < 0 || len > (static_cast<int64_t>(a.c.table_width) << a.c.page_shift);
  return bad || s1 - s0 < 2 ? 0 : len >> a.c.page_shift;
}

// Shared pages of sequence s.
__device__ __forceinline__ int shared_before(const SharedAttnArgs& a, int s, bool& bad) {
  int lo = 0, hi = a.groups;  // groups that start at or before s: [0, lo), behind it: [hi, ..)
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.group_start[mid] <= s) lo = mid + 1;
    else hi = mid;
  }
  bad = false;
  if (lo == 0) return 0;
  int s0, s1;
  const int pages = shared_pages(a, lo - 1, s0, s1, bad);
  return s < s1 ? pages : 0;
}

// The first sequence of [s0, s1) that has rows, where s0 has none: the last one
// that starts at row r0, as s0 does.  (Empty slots' table rows may name any page.)
__device__ __forceinline__ int first_with_rows(const SharedAttnArgs& a, int s0, int s1, int r0) {
  int lo = s0, hi = s1 - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.c.row_start[mid] <= r0) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ SharedSeq line_seq(const SharedAttnArgs& a, int v, bool& bad) {
  SharedSeq q;
  q.row0 = q.n = q.len = q.row = 0;
  q.page0 = -1;
  if (!(a.parts & 1)) v += a.groups;
  if (v < a.groups) {
    int s1;
    const int pages = shared_pages(a, v, q.row, s1, bad);
    if (pages > 0) {
      const int s0 = q.row, r0 = a.c.row_start[s0], r1 = a.c.row_start[s1], next = a.c.row_start[s0 + 1];
      bad = r0 < 0 || r1 < r0 || r1 > a.c.rows;
      if (!bad) {
        if (next <= r0) q.row = first_with_rows(a, s0, s1, r0);
        q.row0 = r0;
        q.n = r1 - r0;
        q.len = pages << a.c.page_shift;
      }
    }
    return q;
  }
  bool wrong;
  static_cast<PagedSeq&>(q) = paged_seq(a.c, v - a.groups, bad);
  q.row = v - a.groups;
  q.page0 = shared_before(a, q.row, wrong);
  const int before = q.page0 << a.c.page_shift;
  bad |= wrong || (before > 0 && q.n > 0 && q.len - q.n < before);
  if (bad) q.n = 0;
  q.len -= before;
  return q;
}

// Where a row's result lies: `at` = row * Hq + head.
__device__ __forceinline__ int64_t shared_ref(const SharedAttnArgs& a, int own, int64_t at) {
  return own * (static_cast<int64_t>(a.c.rows) * a.Hq) + at;
}
__device__ __forceinline__ int64_t shared_sums(const SharedAttnArgs& a, int own, int chunk, int64_t at) {
  return ((own * 16 + chunk) * (static_cast<int64_t>(a.c.rows) * a.Hq) + at) * 8;
}

// What a step's description says of its sequence besides: 1, or for a
// SharedSeq 1 for a prefix, else 2 + its first page.
__device__ __forceinline__ int line_kind(const PagedSeq&) { return 1; }
__device__ __forceinline__ int line_kind(const SharedSeq& q) { return 2 + q.page0; }
__device__ __forceinline__ int line_row(const PagedSeq&, int s) { return s; }
__device__ __forceinline__ int line_row(const SharedSeq& q, int) { return q.row; }
template <class Line, class Args, class Seq>
__device__ __forceinline__ UnitKeys unit_keys(const Args& a, const Seq& q, int p) {
  constexpr int row_tile = Line::row_tile, key_tile = Line::key_tile;
  const int rows = q.n * a.group;
  int i0 = 0, i1 = q.n - 1;  // first and last new token of the tile
  if (!Line::single && rows > row_tile) {
    i0 = div_group(a, p * row_tile);
    i1 = div_group(a, min((p + 1) * row_tile, rows) - 1);
  }
  UnitKeys u;
  u.hi = line_causal(a, q) ? min(q.len, q.len - q.n + i1 + 1) : q.len;
  u.lo = row_lo(a, q.len - q.n + i0);
  if (u.hi <= u.lo) u.lo = u.hi = 0;
  u.t0 = u.lo / static_cast<uint32_t>(key_tile);
  u.nt = max(1, static_cast<int>((u.hi + static_cast<uint32_t>(key_tile) - 1) / static_cast<uint32_t>(key_tile)) - u.t0);
  u.each = Line::half == Line::full || rows - p * row_tile > row_tile / 2 ? Line::full : Line::half;
  u.places = u.nt * u.each + Line::over;
  return u;
}

__device__ __forceinline__ int64_t warp_sum(int64_t t) {
#pragma unroll
  for (int d = 16; d; d /= 2) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
  return t;
}
__device__ __forceinline__ int64_t warp_scan(int64_t t, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, t, d);
    if (lane >= d) t += y;
  }
  return t;
}

// x * y / z, in 32 bits where they hold it (a 64-bit division is long).
__device__ __forceinline__ int64_t muldiv(int64_t x, int64_t y, int64_t z) {
  const uint64_t v = static_cast<uint64_t>(x) * static_cast<uint64_t>(y);
  if ((v | static_cast<uint64_t>(z)) >> 32 == 0) return static_cast<uint32_t>(v) / static_cast<uint32_t>(z);
  return static_cast<int64_t>(v / static_cast<uint64_t>(z));
}

// Places of one head of the sequences base + lane, one a lane (0 past the
// last).  Sequences of many row tiles are summed by the whole warp.
template <class Line, class Args>
__device__ __forceinline__ int64_t lane_tiles(const Args& a, int base, int lane, bool& bad) {
  using Seq = decltype(line_seq(a, 0, bad));
  const int s = base + lane;
  Seq q;
  q.n = q.len = 0;
  if (s < line_seqs(a)) {
    bool b;
    q = line_seq(a, s, b);
    bad |= b;
  }
  if constexpr (Line::single) {
    return q.n > 0 ? unit_keys<Line>(a, q, 0).places : 0;
  } else {
    const int tiles = row_tiles(a, q, Line::row_tile);
    int64_t t = 0;
    if (tiles <= 4)
#pragma unroll 1
      for (int p = 0; p < tiles; ++p) t += unit_keys<Line>(a, q, p).places;
    unsigned many = __ballot_sync(0xFFFFFFFFu, tiles > 4);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      Seq r;
      r.row0 = 0;
      if constexpr (Args::shared) r.page0 = __shfl_sync(0xFFFFFFFFu, q.page0, src);
      r.n = __shfl_sync(0xFFFFFFFFu, q.n, src);
      r.len = __shfl_sync(0xFFFFFFFFu, q.len, src);
      const int n = __shfl_sync(0xFFFFFFFFu, tiles, src);
      int64_t y = 0;
#pragma unroll 1
      for (int p = lane; p < n; p += 32) y += unit_keys<Line>(a, r, p).places;
      y = warp_sum(y);
      if (lane == src) t = y;
    }
    return t;
  }
}
// The same for sequences behind the first 32, out of the way where it is long:
// a small batch's time is that of fetching the code that it runs.
template <class Line, class Args>
__device__ __noinline__ int64_t far_call(const Args& a, int base, bool& bad) {
  return lane_tiles<Line>(a, base, threadIdx.x % 32, bad);
}
template <class Line, class Args>
__device__ __forceinline__ int64_t far_tiles(const Args& a, int base, bool& bad) {
  if constexpr (Line::single) return lane_tiles<Line>(a, base, threadIdx.x % 32, bad);
  else return far_call<Line>(a, base, bad);
}

// One step of a CTA: some key tiles of a unit.
struct Segment {
  int valid;       // 0: no more; else line_kind of the sequence
  int row0, n, len, h, rho0, rows;
  int lo, hi;      // keys that some row sees
  int all_lo, all_hi;  // keys that every row sees
  int t0, nt;      // key tiles of this step
  int part;        // -1: the unit's output; else the partial result's slot (0 or 1)
  int s;           // row of the table
};

// Walks the steps of a CTA's part of the line (by a whole warp, all lanes
// alike).
template <class Seq>
struct LineWalkOf {
  int64_t at, end, total;
  int ctas;     // CTAs with work: all, or fewer when tiles are few
  int s, h, p;
  int skip;     // places of the unit that earlier CTAs have
  Seq q;
  int tiles;    // row tiles of the sequence
};
using LineWalk = LineWalkOf<PagedSeq>;

template <class Line, class Args, class Seq>
__device__ __forceinline__ void walk_seq(const Args& a, LineWalkOf<Seq>& w) {
  bool bad;
  w.q = line_seq(a, w.s, bad);
  w.tiles = row_tiles(a, w.q, Line::row_tile);
}

// Finds the part of CTA `cta` of `ctas`.  Sets `bad` when a sequence fails its
// checks.
template <class Line, class Args, class Seq>
__device__ __forceinline__ void walk_begin(const Args& a, LineWalkOf<Seq>& w, int cta, int ctas, bool& bad) {
  const int lane = threadIdx.x % 32;
  const int64_t first = lane_tiles<Line>(a, 0, lane, bad);
  int64_t t = first;
#pragma unroll 1
  for (int base = 32; base < line_seqs(a); base += 32) t += far_tiles<Line>(a, base, bad);
  w.total = warp_sum(t) * a.c.H;
  const int64_t most = (w.total + Line::min_places - 1) / Line::min_places;
  w.ctas = static_cast<int>(min(static_cast<int64_t>(ctas), most));
  // (a part without tiles must not lie between two of one unit)
  w.at = w.end = 0;
  w.s = w.h = w.p = w.skip = 0;
  if (cta >= w.ctas) return;
  w.at = muldiv(cta, w.total, w.ctas);
  w.end = muldiv(cta + 1, w.total, w.ctas);
  int64_t left = w.at;
#pragma unroll 1
  for (int base = 0;; base += 32) {
    bool b;
    const int64_t mine = (base == 0 ? first : far_tiles<Line>(a, base, b)) * a.c.H;
    const int64_t upto = warp_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, upto > left);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w.s = base + src;
      left = __shfl_sync(0xFFFFFFFFu, left - (upto - mine), src);
      t = __shfl_sync(0xFFFFFFFFu, mine, src);  // of all heads
      break;
    }
    left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  walk_seq<Line>(a, w);
  t = muldiv(t, 1, a.c.H);
  w.h = static_cast<int>(muldiv(left, 1, t));
  left -= w.h * t;
  w.skip = static_cast<int>(left);
  if constexpr (!Line::single) {
    for (int p0 = 0; w.tiles > 1; p0 += 32) {
      const int64_t mine = p0 + lane < w.tiles ? unit_keys<Line>(a, w.q, p0 + lane).places : 0;
      const int64_t upto = warp_scan(mine, lane);
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, upto > left);
      if (hit) {
        const int src = __ffs(hit) - 1;
        w.p = p0 + src;
        w.skip = static_cast<int>(__shfl_sync(0xFFFFFFFFu, left - (upto - mine), src));
        return;
      }
      left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
  }
}

// The next step (valid = 0 at the end); `join` is filled when it leaves a
// unit unfinished that it began.
template <class Line, class Args, class Seq>
__device__ __forceinline__ Segment walk_next(const Args& a, LineWalkOf<Seq>& w, int cta, JoinDesc& join) {
  Segment g;
  g.valid = 0;
  while (w.at < w.end) {
    while (w.p >= w.tiles) {  // next head, next sequence with rows
      w.p = 0;
      if (w.tiles == 0 || ++w.h >= a.c.H) {
        w.h = 0;
        ++w.s;
        walk_seq<Line>(a, w);
      }
    }
    const UnitKeys u = unit_keys<Line>(a, w.q, w.p);
    const int take = static_cast<int>(min(static_cast<int64_t>(u.places - w.skip), w.end - w.at));
    // key tiles whose first place is among [skip, skip + take)
    const auto tiles_before = [&](int place) { return (max(0, place - Line::over) + u.each - 1) / u.each; };
    const int from = tiles_before(w.skip), to = tiles_before(w.skip + take);
    if (to > from) {
      g.valid = line_kind(w.q);
      g.row0 = w.q.row0;
      g.n = w.q.n;
      g.len = w.q.len;
      g.h = w.h;
      g.s = line_row(w.q, w.s);
      g.rho0 = w.p * Line::row_tile;
      g.rows = min(Line::row_tile, w.q.n * a.group - g.rho0);
      g.lo = u.lo;
      g.hi = u.hi;
      const int base = w.q.len - w.q.n;
      g.all_lo = row_lo(a, base + div_group(a, g.rho0 + g.rows - 1));
      g.all_hi = line_causal(a, w.q) ? min(w.q.len, base + div_group(a, g.rho0) + 1) : w.q.len;
      g.t0 = u.t0 + from;
      g.nt = to - from;
      g.part = from == 0 ? (to == u.nt ? -1 : 1) : 0;
      if (g.part == 1) {
        // the CTA that holds the first place of the unit's last tile
        const int owner = static_cast<int>(muldiv((w.at - w.skip + u.places - u.each + 1) * w.ctas - 1, 1, w.total));
        join.pieces = owner - cta + 1;
        join.row0 = g.row0;
        join.rho0 = g.rho0;
        join.rows = g.rows;
        join.h = g.h;
        if constexpr (Args::shared) join.own = g.valid > 1;
      }
    }
    w.at += take;
    w.skip = 0;
    ++w.p;
    if (g.valid) break;
  }
  return g;
}

}  // namespace sa
