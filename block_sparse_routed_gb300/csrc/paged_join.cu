// Joining the partial results of attention over a paged cache (sm_103a).
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

// Joins the parts of the units that a cut divided: a warp takes a row, four
// columns a lane, and adds the parts in the order of their keys,
//   o = sum_i 2^(m_i - m) a_i / sum_i 2^(m_i - m) l_i,  m = max m_i.
// The first CTA also makes one status word of the CTAs' words.
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedAttnArgs a, const PagedScratch ws, int row_tile) {
  griddep_wait();
  const int lane = threadIdx.x % 32, row = blockIdx.y * 4 + threadIdx.x / 32;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) {
    int st = 0;
    for (int i = lane; i < gridDim.x; i += 32) st = max(st, ws.cta_status[i]);
    st = __reduce_max_sync(0xFFFFFFFFu, st);
    if (lane == 0) *a.c.status = st;
  }
  const JoinDesc d = ws.join[blockIdx.x];
  if (d.pieces == 0 || row >= d.rows) return;
  auto slot = [&](int i) -> int64_t {
    return (static_cast<int64_t>(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * row_tile + row;
  };
  float m = -INFINITY;
  for (int i = lane; i < d.pieces; i += 32) m = fmaxf(m, ws.ml[slot(i)].x);
#pragma unroll
  for (int k = 16; k; k /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < d.pieces; ++i) {
    const int64_t at = slot(i);
    const float2 ml = ws.ml[at];
    const float4 x = reinterpret_cast<const float4*>(ws.part + at * kHeadDim)[lane];
    const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
    l += f * ml.y;
    o.x += f * x.x;
    o.y += f * x.y;
    o.z += f * x.z;
    o.w += f * x.w;
  }
  const int rho = d.rho0 + row;
  const int64_t at = static_cast<int64_t>(d.row0 + rho / a.group) * a.Hq + d.h * a.group + rho % a.group;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (NaN stays)
  reinterpret_cast<uint2*>(a.o + at * kHeadDim)[lane] =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttnArgs& a, const PagedScratch& ws, int row_tile, int ctas, cudaStream_t s) {
  return launch_dependent(paged_join_kernel, dim3(ctas, row_tile / 4), dim3(128), 0, s, a, ws, row_tile);
}

}  // namespace sa
