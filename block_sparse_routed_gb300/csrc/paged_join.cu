// Joining the partial results of attention over a paged cache (sm_103a): for
// each row of a unit that a cut of the work divided, over its parts in the
// order of their keys,
//   o = sum_i 2^(m_i - m) a_i / sum_i 2^(m_i - m) l_i,  m = max m_i.
// Bound by latency (with its launch and the attention kernel's last stores 3
// to 4 us after it in the form for few rows) and in the form for chunks by what
// the parts weigh too: 512 bytes a row and part, two parts a CTA, 6 to 9 us.
// The first CTA also makes one status word of the CTAs' words.
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4;

// (of a call's second join: with what the first one found)
template <class Args>
__device__ __forceinline__ void join_status(const Args& a, const PagedScratch& ws, bool first = true) {
  if (blockIdx.x != 0 || blockIdx.y != 0 || threadIdx.x >= 32) return;
  int st = 0;
  for (int i = threadIdx.x; i < gridDim.x; i += 32) st = max(st, ws.cta_status[i]);
  st = __reduce_max_sync(0xFFFFFFFFu, st);
  if (threadIdx.x == 0) *a.c.status = first ? st : max(st, *a.c.status);
}

// Row of the i-th part of the unit that begins in CTA blockIdx.x.
__device__ __forceinline__ int64_t part_row(int i, int row_tile, int row) {
  return (static_cast<int64_t>(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * row_tile + row;
}

__device__ __forceinline__ float join_inverse(float l) {
  return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (NaN stays)
}

__device__ __forceinline__ float join_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// The form for few rows.  A block takes a row; its warps share the parts (one
// long context alone on the GPU has 150 of them), four columns a lane.
template <class Args>
__global__ void __launch_bounds__(32 * kWarps) join_few_kernel(const Args a, const PagedScratch ws, int row_tile, bool first) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, row = blockIdx.y;
  if constexpr (Args::shared) griddep_launch_dependents();
  griddep_wait();
  const JoinDesc d = ws.join[blockIdx.x];
  join_status(a, ws, first);
  if (d.pieces == 0 || row >= d.rows) return;
  // The references of 32 parts, one a lane, give the maximum so far; then the
  // parts themselves, relative to it.
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < d.pieces; i0 += 32 * kWarps) {
    const int mine = i0 + lane * kWarps;
    const float2 ml = mine < d.pieces ? ws.ml[part_row(mine, row_tile, row)] : make_float2(-INFINITY, 0.f);
    float top = ml.x;
#pragma unroll
    for (int k = 16; k; k /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
    const float to = fmaxf(m, top);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - to);
    m = to;
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    const float w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
    const int n = min(32, (d.pieces - i0 + kWarps - 1) / kWarps);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float4 x = reinterpret_cast<const float4*>(ws.part + part_row(i0 + i * kWarps, row_tile, row) * kHeadDim)[lane];
      const float wi = __shfl_sync(0xFFFFFFFFu, w, i), li = __shfl_sync(0xFFFFFFFFu, ml.y, i);
      l += wi * li;
      o.x += wi * x.x;
      o.y += wi * x.y;
      o.z += wi * x.z;
      o.w += wi * x.w;
    }
  }
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ float4 s_o[kWarps][32];
  s_o[warp][lane] = o;
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  if (warp != 0) return;
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
  const int rho = d.rho0 + row, i = div_group(a, rho);
  const int64_t at = static_cast<int64_t>(d.row0 + i) * a.Hq + d.h * a.group + rho - i * a.group;
  if constexpr (Args::shared) {
    *reinterpret_cast<float4*>(a.sums + shared_sums(a, d.own, lane / 2, at) + lane % 2 * 4) = o;
    if (lane == 0) a.refs[shared_ref(a, d.own, at)] = make_float2(m, l);
    return;
  }
  const float inv = join_inverse(l);
  reinterpret_cast<uint2*>(a.o + at * kHeadDim)[lane] =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (a.lse && lane == 0) a.lse[at] = join_lse(m, l);
}

// The form for chunks.  A warp takes 8 rows x 32 columns: the parts are read
// 256 bytes, the output written 64 bytes at a time.  kGroups sets of warps
// share the parts of a unit: where few units are cut into many parts they are
// what keeps enough loads in flight (60 tokens over 30000 keys, 16 / 2 heads,
// 38 parts a unit: 41 us with one set, 37 with four); with two or three parts
// a unit they only wait (128 over 1000, 8 / 4 heads: 20.5 us with one, 24 with
// four).
template <int kGroups, class Args>
__global__ void __launch_bounds__(32 * kWarps * kGroups)
join_chunk_kernel(const Args a, const PagedScratch ws) {
  constexpr int kRows = kPagedChunkRows;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 % kWarps, group = threadIdx.x / (32 * kWarps);
  if constexpr (Args::shared) griddep_launch_dependents();
  griddep_wait();
  const JoinDesc d = ws.join[blockIdx.x];
  join_status(a, ws);
  if (d.pieces == 0 || blockIdx.y * 8 >= d.rows) return;
  // warp: columns 32 w ..; lane: row, 8 columns
  const int row = blockIdx.y * 8 + lane % 8, chunk = warp * 4 + lane / 8;
  if (kGroups == 1 && row >= d.rows) return;  // (else they load what nobody wrote, and write nothing)
  // Four parts at a time, references, sums and values by one round of loads.
  float m = -INFINITY, l = 0.f;
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int i0 = 4 * group; i0 < d.pieces; i0 += 4 * kGroups) {
    float2 ml[4];
    float4 x[4], y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = min(i0 + u, d.pieces - 1);
      ml[u] = ws.ml[part_row(i, kRows, row)];
      const float4* src = reinterpret_cast<const float4*>(ws.part + part_row(i, kRows, 0) * kHeadDim + (chunk * kRows + row) * 8);
      x[u] = src[0];
      y[u] = src[1];
    }
    float to = m;
#pragma unroll
    for (int u = 0; u < 4; ++u) to = fmaxf(to, ml[u].x);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - to);
    m = to;
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i0 + u >= d.pieces) break;
      const float w = ml[u].x == -INFINITY ? 0.f : ex2_approx(ml[u].x - m);
      l += w * ml[u].y;
      o[0] += w * x[u].x;
      o[1] += w * x[u].y;
      o[2] += w * x[u].z;
      o[3] += w * x[u].w;
      o[4] += w * y[u].x;
      o[5] += w * y[u].y;
      o[6] += w * y[u].z;
      o[7] += w * y[u].w;
    }
  }
  if constexpr (kGroups > 1) {
    __shared__ float2 s_ml[kGroups - 1][32 * kWarps];
    __shared__ float4 s_o[kGroups - 1][2][32 * kWarps];
    const int at = threadIdx.x % (32 * kWarps);
    if (group > 0) {
      s_ml[group - 1][at] = make_float2(m, l);
      s_o[group - 1][0][at] = make_float4(o[0], o[1], o[2], o[3]);
      s_o[group - 1][1][at] = make_float4(o[4], o[5], o[6], o[7]);
    }
    __syncthreads();
    if (group > 0) return;
    const float own = m;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) m = fmaxf(m, s_ml[k][at].x);
    const float f = own == -INFINITY ? 0.f : ex2_approx(own - m);
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= f;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
      const float2 ml = s_ml[k][at];
      const float w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
      const float4 x = s_o[k][0][at], y = s_o[k][1][at];
      l += w * ml.y;
      o[0] += w * x.x;
      o[1] += w * x.y;
      o[2] += w * x.z;
      o[3] += w * x.w;
      o[4] += w * y.x;
      o[5] += w * y.y;
      o[6] += w * y.z;
      o[7] += w * y.w;
    }
  }
  if (kGroups > 1 && row >= d.rows) return;
  const int rho = d.rho0 + row, i = div_group(a, rho);
  const int64_t at = static_cast<int64_t>(d.row0 + i) * a.Hq + d.h * a.group + rho - i * a.group;
  if constexpr (Args::shared) {
    float4* to = reinterpret_cast<float4*>(a.sums + shared_sums(a, d.own, chunk, at));
    to[0] = make_float4(o[0], o[1], o[2], o[3]);
    to[1] = make_float4(o[4], o[5], o[6], o[7]);
    if (chunk == 0) a.refs[shared_ref(a, d.own, at)] = make_float2(m, l);
    return;
  }
  const float inv = join_inverse(l);
  uint32_t z[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) z[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  reinterpret_cast<uint4*>(a.o + at * kHeadDim)[chunk] = make_uint4(z[0], z[1], z[2], z[3]);
  if (a.lse && chunk == 0) a.lse[at] = join_lse(m, l);
}

// Rows over their group's prefix and over their own keys: one result.  A warp
// takes 8 heads x 4 of the 16 times 8 dimensions of a row.  What it needs comes at
// once: the sequence that a row belongs to while the joins run, and both sums
// before it is known whether the row has a prefix (102 -> 98.5 us for 64 rows of 40
// heads, 138 -> 135 for 464 of 56).
__global__ void __launch_bounds__(32 * kWarps) shared_merge_kernel(const SharedAttnArgs a) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, r = blockIdx.x;
  const int s = paged_find(a.c, r, lane);
  bool bad;
  SharedSeq q = line_seq(a, a.groups + max(s, 0), bad);
  bad |= s < 0 || r < q.row0 || r >= q.row0 + q.n;  // (a sequence that is refused, or none)
  griddep_wait();
  if (bad) return;
  for (int x = blockIdx.y * kWarps + warp; x < (a.Hq + 7) / 8 * 4; x += gridDim.y * kWarps) {
    const int head = x / 4 * 8 + lane % 8, chunk = x % 4 * 4 + lane / 8;
    if (head >= a.Hq) continue;
    const int64_t at = static_cast<int64_t>(r) * a.Hq + head;
    const float2 own = a.refs[shared_ref(a, 1, at)];
    const float4* from = reinterpret_cast<const float4*>(a.sums + shared_sums(a, 1, chunk, at));
    float4 u = from[0], v = from[1];
    float m = own.x, l = own.y;
    if (q.page0 > 0) {
      const float2 pre = a.refs[shared_ref(a, 0, at)];
      const float4* other = reinterpret_cast<const float4*>(a.sums + shared_sums(a, 0, chunk, at));
      const float4 y = other[0], z = other[1];
      m = fmaxf(own.x, pre.x);
      const float f = own.x == -INFINITY ? 0.f : ex2_approx(own.x - m);
      const float g = pre.x == -INFINITY ? 0.f : ex2_approx(pre.x - m);
      // (a part without a reference has the sum 0, or NaN if its logits are)
      l = (own.x == -INFINITY ? own.y : f * own.y) + (pre.x == -INFINITY ? pre.y : g * pre.y);
      u = make_float4(f * u.x + g * y.x, f * u.y + g * y.y, f * u.z + g * y.z, f * u.w + g * y.w);
      v = make_float4(f * v.x + g * z.x, f * v.y + g * z.y, f * v.z + g * z.z, f * v.w + g * z.w);
    }
    const float inv = join_inverse(l);
    reinterpret_cast<uint4*>(a.o + at * kHeadDim)[chunk] =
        make_uint4(pack_bf16x2(u.x * inv, u.y * inv), pack_bf16x2(u.z * inv, u.w * inv),
                   pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    if (a.lse && chunk == 0) a.lse[at] = join_lse(m, l);
  }
}

}  // namespace

cudaError_t launch_shared_join(const SharedAttnArgs& a, const PagedScratch& ws, int row_tile, int ctas, bool many_parts,
                               bool first, cudaStream_t s) {
  if (row_tile <= kPagedFewRows)
    return launch_dependent(join_few_kernel<SharedAttnArgs>, dim3(ctas, row_tile), dim3(32 * kWarps), 0, s, a, ws, row_tile,
                            first);
  const dim3 grid(ctas, kPagedChunkRows / 8);
  if (many_parts)
    return launch_dependent(join_chunk_kernel<4, SharedAttnArgs>, grid, dim3(32 * kWarps * 4), 0, s, a, ws);
  return launch_dependent(join_chunk_kernel<1, SharedAttnArgs>, grid, dim3(32 * kWarps), 0, s, a, ws);
}

cudaError_t launch_shared_merge(const SharedAttnArgs& a, cudaStream_t s) {
  const int pieces = min(((a.Hq + 7) / 8 * 4 + kWarps - 1) / kWarps, 65535);
  return launch_dependent(shared_merge_kernel, dim3(a.c.rows, pieces), dim3(32 * kWarps), 0, s, a);
}

cudaError_t launch_paged_join(const PagedAttnArgs& a, const PagedScratch& ws, int row_tile, int ctas, bool many_parts,
                              cudaStream_t s) {
  if (row_tile <= kPagedFewRows)
    return launch_dependent(join_few_kernel<PagedAttnArgs>, dim3(ctas, row_tile), dim3(32 * kWarps), 0, s, a, ws, row_tile, true);
  const dim3 grid(ctas, kPagedChunkRows / 8);
  if (many_parts) return launch_dependent(join_chunk_kernel<4, PagedAttnArgs>, grid, dim3(32 * kWarps * 4), 0, s, a, ws);
  return launch_dependent(join_chunk_kernel<1, PagedAttnArgs>, grid, dim3(32 * kWarps), 0, s, a, ws);
}

}  // namespace sa
