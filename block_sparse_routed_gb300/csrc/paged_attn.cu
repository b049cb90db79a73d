// Attention of new tokens over a paged cache (sm_103a): the plainest form.
// One CTA takes one row and one query head; each of its four warps walks
// every fourth visible key with an online softmax
//   m' = max(m, x),  l' = l 2^(m - m') + 2^(x - m'),  a' = a 2^(m - m') + 2^(x - m') v
// (x the logit in log2 units, four dimensions a lane) and the four partial
// results are merged the same way.
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

__device__ __forceinline__ float4 row4(const uint8_t* pages, const uint8_t* exps, int kind, int64_t row, int lane) {
  float4 f;
  if (kind == 0) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(pages + row * 256 + lane * 8));
    f = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                    __uint_as_float(v.y & 0xFFFF0000u));
  } else {
    const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(pages + row * 128 + lane * 4));
    const float two = exp_scale(__ldg(exps + row));
    e4m3x2_f32(static_cast<uint16_t>(v), f.x, f.y);
    e4m3x2_f32(static_cast<uint16_t>(v >> 16), f.z, f.w);
    f.x *= two;
    f.y *= two;
    f.z *= two;
    f.w *= two;
  }
  return f;
}

__global__ void __launch_bounds__(128) paged_simple_kernel(const PagedAttnArgs a) {
  const PagedArgs& c = a.c;
  __shared__ float sm[4], sl[4], sacc[4][kHeadDim];
  const int r = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int h = hq / a.group;
  if (r == 0 && hq == 0) paged_check_all(c);
  const int s = paged_find(c, r, lane);
  if (s < 0) return;
  bool bad;
  const PagedSeq q = paged_seq(c, s, bad);
  if (bad) {
    if (threadIdx.x == 0) paged_fail(c);
    return;
  }
  if (r < q.row0 || r >= q.row0 + q.n) return;
  const int pos = q.len - q.n + (r - q.row0);
  const int hi = a.causal ? min(q.len, pos + 1) : q.len;
  const int lo = a.window ? max(0, pos + 1 - a.window) : 0;
  const uint2 qv = __ldg(reinterpret_cast<const uint2*>(a.q + r * a.q_token + hq * a.q_head + lane * 4));
  const float c2 = a.scale * 1.4426950408889634f;
  const float4 qf = make_float4(__uint_as_float(qv.x << 16), __uint_as_float(qv.x & 0xFFFF0000u),
                                __uint_as_float(qv.y << 16), __uint_as_float(qv.y & 0xFFFF0000u));
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = lo + warp; j < hi; j += 4) {
    const int page = c.table[s * c.table_stride + (j >> c.page_shift)];
    if (page < 0 || page >= c.pages) {
      if (lane == 0) paged_fail(c);
      continue;
    }
    const int64_t row = ((static_cast<int64_t>(page) * c.H + h) << c.page_shift) + (j & (c.page_size - 1));
    const float4 k = row4(c.k_pages, c.k_exp, c.kind, row, lane);
    const float4 v = row4(c.v_pages, c.v_exp, c.kind, row, lane);
    float x = qf.x * k.x + qf.y * k.y + qf.z * k.z + qf.w * k.w;
#pragma unroll
    for (int d = 16; d; d /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    x *= c2;
    const float mn = fmaxf(m, x);
    const float f = (m == -INFINITY) ? 0.f : exp2f(m - mn), p = (mn == -INFINITY) ? 0.f : exp2f(x - mn);
    l = l * f + p;
    acc.x = acc.x * f + p * v.x;
    acc.y = acc.y * f + p * v.y;
    acc.z = acc.z * f + p * v.z;
    acc.w = acc.w * f + p * v.w;
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  *reinterpret_cast<float4*>(&sacc[warp][lane * 4]) = acc;
  __syncthreads();
  if (threadIdx.x >= kHeadDim) return;
  const float mt = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float lt = 0.f, o = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float f = (sm[w] == -INFINITY) ? 0.f : exp2f(sm[w] - mt);
    lt += f * sl[w];
    o += f * sacc[w][threadIdx.x];
  }
  const int64_t at = static_cast<int64_t>(r) * a.Hq + hq;
  const float y = lt > 0.f ? o / lt : 0.f;
  a.o[at * kHeadDim + threadIdx.x] = static_cast<uint16_t>(pack_bf16x2(y, 0.f));
  if (a.lse && threadIdx.x == 0) a.lse[at] = lt > 0.f ? (mt + log2f(lt)) * 0.6931471805599453f : -INFINITY;
}

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

cudaError_t launch_paged_simple(const PagedAttnArgs& a, cudaStream_t s) {
  paged_simple_kernel<<<dim3(a.c.rows, a.Hq), 128, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_paged_join(const PagedAttnArgs& a, const PagedScratch& ws, int row_tile, int ctas, cudaStream_t s) {
  return launch_dependent(paged_join_kernel, dim3(ctas, row_tile / 4), dim3(128), 0, s, a, ws, row_tile);
}

}  // namespace sa
