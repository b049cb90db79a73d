// Host side of the paged-cache entry points declared in include/sparse_attn.h:
// argument checks, workspace layout and launches.  Every check happens before
// anything is enqueued.
#include <atomic>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "sparse_attn.h"

#define SA_API extern "C" __attribute__((visibility("default")))

namespace {
using namespace sa;

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

bool bad_stride(int64_t s) { return s < 0 || s % 8 != 0; }

// The fields that every call reads.
sa_status check_paged(const sa_paged_params* p) {
  if (p == nullptr) return SA_EINVAL;
  if (p->abi_version != SA_ABI_VERSION) return SA_EINVAL;
  if (p->D != kHeadDim) return SA_EUNSUPPORTED;
  if (p->kind != SA_CACHE_BF16 && p->kind != SA_CACHE_E4M3) return SA_EINVAL;
  if (p->pages < 1 || p->H < 1) return SA_EINVAL;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) return SA_EINVAL;
  if (p->seqs < 0 || p->rows < 0 || p->max_new < 0 || p->table_width < 0 || p->table_stride < 0) return SA_EINVAL;
  const int64_t lim = int64_t(1) << 31;
  if (int64_t(p->pages) * p->H >= lim || int64_t(p->pages) * p->H * p->page_size >= lim) return SA_EUNSUPPORTED;
  if (int64_t(p->table_width) * p->page_size >= lim - 256) return SA_EUNSUPPORTED;
  if (int64_t(p->rows) * p->H >= lim) return SA_EUNSUPPORTED;
  return SA_OK;
}

sa_status check_attn(const sa_paged_params* p) {
  const sa_status st = check_paged(p);
  if (st != SA_OK) return st;
  if (p->Hq < 1 || p->Hq % p->H != 0) return SA_EINVAL;
  if (int64_t(p->rows) * p->Hq >= (int64_t(1) << 31) - 4096) return SA_EUNSUPPORTED;  // (whole tiles of rows)
  if (p->causal != 0 && p->causal != 1) return SA_EINVAL;
  if (p->window < 0 || (p->window > 0 && !p->causal)) return SA_EINVAL;
  if (!std::isfinite(p->scale) || !(p->scale > 0.0f)) return SA_EINVAL;
  return SA_OK;
}

// The pointers of the cache and the batch.
sa_status check_pointers(const sa_paged_params* p, const void* kp, const void* vp, const void* ke,
                         const void* ve, const void* table, const void* row_start, const void* kv_len,
                         const void* ws) {
  if (!kp || !vp || !row_start) return SA_EINVAL;
  if (p->seqs > 0 && (!kv_len || (!table && p->table_width > 0))) return SA_EINVAL;
  if (p->kind == SA_CACHE_E4M3 && (!ke || !ve)) return SA_EINVAL;
  if (!aligned(kp, 16) || !aligned(vp, 16) || !aligned(table, 4) || !aligned(row_start, 4) ||
      !aligned(kv_len, 4) || !aligned(ws, 256))
    return SA_EINVAL;
  if (p->kind == SA_CACHE_E4M3 && (!aligned(ke, 16) || !aligned(ve, 16))) return SA_EINVAL;
  return SA_OK;
}

PagedArgs paged_args(const sa_paged_params* p, const void* kp, const void* vp, const uint8_t* ke,
                     const uint8_t* ve, const int32_t* table, const int32_t* row_start,
                     const int32_t* kv_len, void* ws) {
  PagedArgs c;
  c.kind = p->kind;
  c.pages = p->pages;
  c.H = p->H;
  c.page_size = p->page_size;
  c.page_shift = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  c.seqs = p->seqs;
  c.table_width = p->table_width;
  c.rows = p->rows;
  c.max_new = p->max_new;
  c.table_stride = p->table_stride;
  c.table = table;
  c.row_start = row_start;
  c.kv_len = kv_len;
  c.k_pages = static_cast<uint8_t*>(const_cast<void*>(kp));
  c.v_pages = static_cast<uint8_t*>(const_cast<void*>(vp));
  c.k_exp = const_cast<uint8_t*>(ke);
  c.v_exp = const_cast<uint8_t*>(ve);
  c.status = static_cast<int32_t*>(ws);
  return c;
}

// The form that computes a call: by the most packed rows of one sequence and
// key head, from the host's bound.
PagedForm form_of(const sa_paged_params* p) {
  PagedForm f;
  const int64_t rows = int64_t(p->max_new < p->rows ? p->max_new : p->rows) * (p->Hq / p->H);
  f.few = rows <= kPagedFewRows;
  f.row_tile = rows <= 8 ? 8 : (f.few ? kPagedFewRows : kPagedChunkRows);
  f.max_ctas = f.few ? kPagedFewCtas : kPagedChunkCtas;
  return f;
}

// Of the current device (0: none could be asked).
int multiprocessors() {
  static std::atomic<int> cached[128];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

constexpr uint64_t align256(uint64_t x) { return (x + 255u) & ~uint64_t(255); }

// Workspace layout; returns its bytes.
uint64_t scratch_of(void* ws, const PagedForm& f, PagedScratch* out) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint64_t off = kStatusBytes;
  const uint64_t n = f.max_ctas;
  const uint64_t status = off; off += align256(n * 4);
  const uint64_t join = off;   off += align256(n * sizeof(JoinDesc));
  const uint64_t ml = off;     off += align256(n * 2 * f.row_tile * 8);
  const uint64_t part = off;   off += n * 2 * f.row_tile * kHeadDim * 4;
  if (out) {
    out->cta_status = reinterpret_cast<int32_t*>(w + status);
    out->join = reinterpret_cast<JoinDesc*>(w + join);
    out->ml = reinterpret_cast<float2*>(w + ml);
    out->part = reinterpret_cast<float*>(w + part);
  }
  return off;
}

sa_status clear_status(void* ws, cudaStream_t stream) {
  if (ws && cuda_failed(cudaMemsetAsync(ws, 0, kStatusBytes, stream))) return SA_ECUDA;
  return SA_OK;
}

}  // namespace

SA_API sa_status sparse_attn_cache_write(const sa_paged_params* p, const void* k, const void* v, void* k_pages,
                                         void* v_pages, uint8_t* k_exp, uint8_t* v_exp, const int32_t* table,
                                         const int32_t* row_start, const int32_t* kv_len, void* ws,
                                         cudaStream_t stream) {
  sa_status st = check_paged(p);
  if (st != SA_OK) return st;
  if (bad_stride(p->a_token_stride) || bad_stride(p->a_head_stride) || bad_stride(p->b_token_stride) ||
      bad_stride(p->b_head_stride))
    return SA_EINVAL;
  if (p->rows > 0 && (!k || !v)) return SA_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16)) return SA_EINVAL;
  st = check_pointers(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws);
  if (st != SA_OK) return st;
  st = static_cast<sa_status>(device_status());
  if (st != SA_OK) return st;
  st = clear_status(ws, stream);
  if (st != SA_OK || p->rows == 0 || p->seqs == 0) return st;
  const PagedArgs c = paged_args(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws);
  CacheRows r;
  r.k = static_cast<uint16_t*>(const_cast<void*>(k));
  r.v = static_cast<uint16_t*>(const_cast<void*>(v));
  r.k_token = p->a_token_stride;
  r.k_head = p->a_head_stride;
  r.v_token = p->b_token_stride;
  r.v_head = p->b_head_stride;
  return cuda_failed(launch_cache_write(c, r, stream)) ? SA_ECUDA : SA_OK;
}

SA_API sa_status sparse_attn_cache_read(const sa_paged_params* p, const void* k_pages, const void* v_pages,
                                        const uint8_t* k_exp, const uint8_t* v_exp, const int32_t* table,
                                        const int32_t* row_start, const int32_t* kv_len, void* k, void* v,
                                        void* ws, cudaStream_t stream) {
  sa_status st = check_paged(p);
  if (st != SA_OK) return st;
  if (p->rows > 0 && (!k || !v)) return SA_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16)) return SA_EINVAL;
  st = check_pointers(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws);
  if (st != SA_OK) return st;
  st = static_cast<sa_status>(device_status());
  if (st != SA_OK) return st;
  st = clear_status(ws, stream);
  if (st != SA_OK || p->rows == 0 || p->seqs == 0) return st;
  const PagedArgs c = paged_args(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws);
  CacheRows r;
  r.k = static_cast<uint16_t*>(k);
  r.v = static_cast<uint16_t*>(v);
  r.k_token = r.v_token = int64_t(p->H) * kHeadDim;
  r.k_head = r.v_head = kHeadDim;
  return cuda_failed(launch_cache_read(c, r, stream)) ? SA_ECUDA : SA_OK;
}

SA_API sa_status sparse_attn_paged_ws_bytes(const sa_paged_params* p, uint64_t* out) {
  if (out == nullptr) return SA_EINVAL;
  const sa_status st = check_attn(p);
  if (st != SA_OK) return st;
  const PagedForm f = form_of(p);
  *out = scratch_of(nullptr, f, nullptr);
  return SA_OK;
}

SA_API sa_status sparse_attn_paged_fwd(const sa_paged_params* p, const void* q, const void* k_pages,
                                       const void* v_pages, const uint8_t* k_exp, const uint8_t* v_exp,
                                       const int32_t* table, const int32_t* row_start,
                                       const int32_t* kv_len, void* o, float* lse, void* ws,
                                       size_t ws_bytes, cudaStream_t stream) {
  uint64_t need = 0;
  sa_status st = sparse_attn_paged_ws_bytes(p, &need);
  if (st != SA_OK) return st;
  if (bad_stride(p->a_token_stride) || bad_stride(p->a_head_stride)) return SA_EINVAL;
  if (!ws || (p->rows > 0 && (!q || !o))) return SA_EINVAL;
  if (!aligned(q, 16) || !aligned(o, 32) || !aligned(lse, 4)) return SA_EINVAL;
  st = check_pointers(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws);
  if (st != SA_OK) return st;
  if (ws_bytes < need) return SA_EINVAL;
  st = static_cast<sa_status>(device_status());
  if (st != SA_OK) return st;
  if (p->rows == 0 || p->seqs == 0) return clear_status(ws, stream);
  PagedAttnArgs a;
  a.c = paged_args(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws);
  a.q = static_cast<const uint16_t*>(q);
  a.q_token = p->a_token_stride;
  a.q_head = p->a_head_stride;
  a.Hq = p->Hq;
  a.group = p->Hq / p->H;
  // with 2^l >= group: m = ceil(2^(31 + l) / group) is off by less than 2^l / group, and x < 2^31
  int l = 0;
  while ((int64_t(1) << l) < a.group) ++l;
  a.group_shift = 31 + l;
  a.group_mul = static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + a.group - 1) / a.group);
  a.causal = p->causal;
  a.window = p->window;
  a.scale = p->scale;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.wait_limit = wait_limit_ns();
  const PagedForm f = form_of(p);
  PagedScratch scratch;
  scratch_of(ws, f, &scratch);
  const uint64_t cached = uint64_t(p->pages) * p->H * p->page_size;
  const int tile = f.few ? kPagedFewKeys : kPagedChunkKeys;
  CUtensorMap tk, tv;
  ChunkMaps boxes{};
  bool maps = true;
  if (f.few) {  // a box holds the keys of a page that fall into a tile
    const uint32_t box = p->page_size < tile ? p->page_size : tile;
    if (p->kind == SA_CACHE_E4M3)
      maps = make_map_rows(&tk, k_pages, cached, kHeadDim, 1, box) &&
             make_map_rows(&tv, v_pages, cached, kHeadDim, 1, box);
    else
      maps = make_map_groups(&tk, k_pages, cached, box) && make_map_groups(&tv, v_pages, cached, box);
  } else if (p->kind == SA_CACHE_BF16) {
    for (int i = 0; 16 * i < tile && 16 * i < p->page_size; ++i)
      maps = maps && make_map_groups(&boxes.m[0][i], k_pages, cached, 16 * (i + 1)) &&
             make_map_groups(&boxes.m[1][i], v_pages, cached, 16 * (i + 1));
  }
  if (!maps) return SA_ECUDA;
  // no more CTAs than units times the key tiles of the longest context that the table can hold
  const int64_t units = p->seqs + (int64_t(p->rows) * a.group + f.row_tile - 1) / f.row_tile;
  const int64_t tiles = (int64_t(p->table_width) * p->page_size + tile - 1) / tile;
  const int64_t most = units * p->H * (tiles + 1);
  int ctas = (f.few ? 2 : 1) * multiprocessors();
  if (ctas <= 0) return SA_ECUDA;
  if (ctas > f.max_ctas) ctas = f.max_ctas;
  if (most < ctas) ctas = static_cast<int>(most);
  const cudaError_t e = f.few ? launch_paged_few(tk, tv, a, scratch, f.row_tile, ctas, stream)
                              : launch_paged_chunk(boxes, a, scratch, ctas, stream);
  if (cuda_failed(e)) return SA_ECUDA;
  // a dozen parts a unit and more (an estimate: the chunks' parts have the places of three key tiles at least)
  const bool many_parts = units * p->H * 12 < ctas && tiles >= 48;
  return cuda_failed(launch_paged_join(a, scratch, f.row_tile, ctas, many_parts, stream)) ? SA_ECUDA : SA_OK;
}
