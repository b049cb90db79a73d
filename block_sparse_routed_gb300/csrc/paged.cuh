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

// 2^(e - 127) of an exponent byte.
__device__ __forceinline__ float exp_scale(uint32_t e) { return __uint_as_float(e << 23); }

// Two E4M3 codes (the low 16 bits) as FP32 values.
__device__ __forceinline__ void e4m3x2_f32(uint16_t v, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

}  // namespace sa
