// Joining the partial results of attention over a paged cache (sm_103a): for
// each row of a unit that a cut of the work divided, over its parts in the
// order of their keys,
//   o = sum_i 2^(m_i - m) a_i / sum_i 2^(m_i - m) l_i,  m = max m_i.
// Bound by latency and by what the parts weigh (512 bytes a row and part).
// A warp takes a row, four columns a lane; where a unit of the form for few
// rows has been cut into many parts (one long context alone on the GPU), four
// warps share a row's parts.
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4;

// kShare: the block's warps share one row's parts, else each takes a row.
template <bool kShare>
__global__ void __launch_bounds__(32 * kWarps) paged_join_kernel(const PagedAttnArgs a, const PagedScratch ws,
                                                                 int row_tile) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  griddep_wait();
  const JoinDesc d = ws.join[blockIdx.x];
  // One status word of the CTAs' words.
  if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
    int st = 0;
    for (int i = lane; i < gridDim.x; i += 32) st = max(st, ws.cta_status[i]);
    st = __reduce_max_sync(0xFFFFFFFFu, st);
    if (lane == 0) *a.c.status = st;
  }
  const int rows_here = kShare ? 1 : kWarps;
  for (int row = blockIdx.y * rows_here + (kShare ? 0 : warp); row < d.rows && d.pieces > 0;
       row += gridDim.y * rows_here) {
    auto slot = [&](int i) -> int64_t {
      return (static_cast<int64_t>(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * row_tile + row;
    };
    const int first = kShare ? warp : 0, step = kShare ? kWarps : 1;
    // The references of 32 parts, one a lane, give the maximum so far; then
    // the parts themselves, relative to it.
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = first; i0 < d.pieces; i0 += 32 * step) {
      const int mine = i0 + lane * step;
      const float2 ml = mine < d.pieces ? ws.ml[slot(mine)] : make_float2(-INFINITY, 0.f);
      float top = ml.x;
#pragma unroll
      for (int k = 16; k; k /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
      const float to = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.f : ex2_approx(m - to);
      m = to;
      l *= f;
      o.x *= f;
      o.y *= f;
      o.z *= f;
      o.w *= f;
      const float w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
      const int n = min(32, (d.pieces - i0 + step - 1) / step);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float4 x = reinterpret_cast<const float4*>(ws.part + slot(i0 + i * step) * kHeadDim)[lane];
        const float wi = __shfl_sync(0xFFFFFFFFu, w, i), li = __shfl_sync(0xFFFFFFFFu, ml.y, i);
        l += wi * li;
        o.x += wi * x.x;
        o.y += wi * x.y;
        o.z += wi * x.z;
        o.w += wi * x.w;
      }
    }
    if constexpr (kShare) {
      __shared__ float s_m[kWarps], s_l[kWarps];
      __shared__ float4 s_o[kWarps][32];
      __syncthreads();  // (the last row's have been read)
      s_o[warp][lane] = o;
      if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
      }
      __syncthreads();
      if (warp != 0) continue;
      m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
      l = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w] == -INFINITY ? 0.f : ex2_approx(s_m[w] - m);
        const float4 x = s_o[w][lane];
        l += f * s_l[w];
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
    }
    const int rho = d.rho0 + row, i = rho / a.group;
    const int64_t at = static_cast<int64_t>(d.row0 + i) * a.Hq + d.h * a.group + rho - i * a.group;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (NaN stays)
    reinterpret_cast<uint2*>(a.o + at * kHeadDim)[lane] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttnArgs& a, const PagedScratch& ws, int row_tile, int ctas, cudaStream_t s) {
  if (row_tile <= kPagedFewRows)
    return launch_dependent(paged_join_kernel<true>, dim3(ctas, row_tile), dim3(32 * kWarps), 0, s, a, ws, row_tile);
  return launch_dependent(paged_join_kernel<false>, dim3(ctas, 16), dim3(32 * kWarps), 0, s, a, ws, row_tile);
}

}  // namespace sa
