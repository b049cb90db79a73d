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

PagedAttnArgs attn_args(const sa_paged_params* p, const void* q, const PagedArgs& c, void* o, float* lse) {
  PagedAttnArgs a;
  a.c = c;
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
  return a;
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

// K's and V's boxes of the form for chunks (BF16 pages).
bool chunk_maps(const sa_paged_params* p, const void* k_pages, const void* v_pages, ChunkMaps* boxes) {
  const uint64_t cached = uint64_t(p->pages) * p->H * p->page_size;
  bool ok = true;
  if (p->kind == SA_CACHE_BF16)
    for (int i = 0; 16 * i < kPagedChunkKeys && 16 * i < p->page_size; ++i)
      ok = ok && make_map_groups(&boxes->m[0][i], k_pages, cached, 16 * (i + 1)) &&
           make_map_groups(&boxes->m[1][i], v_pages, cached, 16 * (i + 1));
  return ok;
}

// Whether a call with groups of sequences goes by them: its workspace, too.
bool shares(const sa_paged_params* p, int32_t groups) { return groups > 0 && p->seqs > 1 && p->rows > 0; }

PagedForm chunk_form() { return {kPagedChunkRows, kPagedChunkCtas, false}; }

// How a call with groups is computed: all of it by the form for few rows where
// all rows of a key head fit into its tile; else by the form for chunks, in one
// launch, but for own keys of few rows in E4M3, which that form widens for 256
// rows: two tiles of the form for few rows are faster there.  64 sequences
// behind 4096 tokens, with 1000 to 1500 own ones, 40 / 8 heads, own keys by
// chunks and by few rows: BF16, 5 rows 86 and 99 us, 20 rows 92 and 122; E4M3, 20
// rows 121 and 104; 32 sequences of 4096 to 8704, E4M3, 5 rows 180 and 114.
struct SharedForms {
  bool few_prefix, few_own;
  int row_tile;  // of the form for few rows
};
SharedForms shared_forms(const sa_paged_params* p) {
  const int64_t group = p->Hq / p->H, all = p->rows * group, own = int64_t(p->max_new < p->rows ? p->max_new : p->rows) * group;
  SharedForms f;
  f.few_prefix = all <= kPagedFewRows;
  f.few_own = f.few_prefix || (p->kind == SA_CACHE_E4M3 && own <= 2 * kPagedFewRows);
  f.row_tile = (f.few_prefix ? all : own) <= 8 ? 8 : kPagedFewRows;
  return f;
}

uint64_t shared_scratch_of(const sa_paged_params* p, void* ws, PagedScratch* chunk, PagedScratch* few, SharedAttnArgs* a) {
  const SharedForms f = shared_forms(p);
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint64_t off = kStatusBytes;  // (of which each part below has its own, not used)
  if (!f.few_prefix) off += align256(scratch_of(w + off, chunk_form(), chunk));
  if (f.few_own) off += align256(scratch_of(w + off, {f.row_tile, kPagedFewCtas, true}, few));
  const uint64_t rows = uint64_t(p->rows) * p->Hq;
  const uint64_t sums = off; off += align256(2 * rows * kHeadDim * 4);
  const uint64_t refs = off; off += align256(2 * rows * 8);
  if (a) {
    a->sums = reinterpret_cast<float*>(w + sums);
    a->refs = reinterpret_cast<float2*>(w + refs);
  }
  return off;
}

// Maps of the form for few rows: a box holds the keys of a page that fall into a tile.
bool few_maps(const sa_paged_params* p, const void* k_pages, const void* v_pages, CUtensorMap* tk, CUtensorMap* tv) {
  const uint64_t cached = uint64_t(p->pages) * p->H * p->page_size;
  const uint32_t box = p->page_size < kPagedFewKeys ? p->page_size : kPagedFewKeys;
  if (p->kind == SA_CACHE_E4M3)
    return make_map_rows(tk, k_pages, cached, kHeadDim, 1, box) && make_map_rows(tv, v_pages, cached, kHeadDim, 1, box);
  return make_map_groups(tk, k_pages, cached, box) && make_map_groups(tv, v_pages, cached, box);
}

// CTAs of a form for `seqs` sequences whose packed rows fill `full` tiles: no
// more than units times the key tiles of the longest context that the table can
// hold (0: the device could not be asked).  many_parts: a dozen parts a unit and
// more (an estimate: the chunks' parts have the places of three key tiles at least).
int form_ctas(const sa_paged_params* p, const PagedForm& f, int64_t seqs, int64_t full, bool* many_parts) {
  const int tile = f.few ? kPagedFewKeys : kPagedChunkKeys;
  const int64_t units = seqs + full;
  const int64_t tiles = (int64_t(p->table_width) * p->page_size + tile - 1) / tile;
  const int64_t most = units * p->H * (tiles + 1);
  int ctas = (f.few ? 2 : 1) * multiprocessors();
  if (ctas > f.max_ctas) ctas = f.max_ctas;
  if (most < ctas) ctas = static_cast<int>(most);
  *many_parts = units * p->H * 12 < ctas && tiles >= 48;
  return ctas;
}

// Whether weights are taken by the form for few rows (both measured in
// paged_weigh.cu): what it costs goes with the rows that there are, what the form
// for chunks costs with whole steps of 96.
bool weighs_few(const sa_paged_params* p) {
  const int64_t group = p->Hq / p->H, most = int64_t(p->max_new < p->rows ? p->max_new : p->rows) * group;
  return most <= 64 || (most <= kWeighFewRows && p->rows * group <= int64_t(80) * p->seqs);
}

uint64_t weigh_scratch_of(const sa_paged_params* p, void* ws, WeighScratch* out) {
  if (weighs_few(p)) return kStatusBytes;
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint64_t off = kStatusBytes;
  const uint64_t status = off; off += align256(kWeighCtas * 4);
  const uint64_t join = off;   off += align256(kWeighCtas * sizeof(WeighJoin));
  const uint64_t part = off;   off += kWeighCtas * 2 * kWeighKeys * 4;
  const uint64_t shift = off;  off += uint64_t(p->rows) * p->Hq * 16;
  if (out) {
    out->shift = reinterpret_cast<uint4*>(w + shift);
    out->cta_status = reinterpret_cast<int32_t*>(w + status);
    out->join = reinterpret_cast<WeighJoin*>(w + join);
    out->part = reinterpret_cast<float*>(w + part);
  }
  return off;
}

// Whether the n numbers from `out` on share one with `rows` rows of `width` numbers, `stride` apart.
bool overlaps(const int32_t* out, int64_t n, const int32_t* in, int64_t rows, int64_t width, int64_t stride) {
  if (!out || !in || n <= 0 || rows <= 0 || width <= 0) return false;
  const int64_t at = (reinterpret_cast<intptr_t>(out) - reinterpret_cast<intptr_t>(in)) / 4;  // (both aligned)
  if (at + n <= 0) return false;
  // the last row that begins at or before `out` (none: -1), and the next one
  const int64_t row = at < 0 ? -1 : stride == 0 || at / stride >= rows ? rows - 1 : at / stride;
  return (row >= 0 && at < row * stride + width) || (row + 1 < rows && (row + 1) * stride < at + n);
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
  const PagedAttnArgs a =
      attn_args(p, q, paged_args(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws), o, lse);
  const PagedForm f = form_of(p);
  PagedScratch scratch;
  scratch_of(ws, f, &scratch);
  CUtensorMap tk, tv;
  ChunkMaps boxes{};
  if (!(f.few ? few_maps(p, k_pages, v_pages, &tk, &tv) : chunk_maps(p, k_pages, v_pages, &boxes))) return SA_ECUDA;
  bool many_parts;
  const int ctas = form_ctas(p, f, p->seqs, (int64_t(p->rows) * a.group + f.row_tile - 1) / f.row_tile, &many_parts);
  if (ctas <= 0) return SA_ECUDA;
  const cudaError_t e = f.few ? launch_paged_few(tk, tv, a, scratch, f.row_tile, ctas, stream)
                              : launch_paged_chunk(boxes, a, scratch, ctas, stream);
  if (cuda_failed(e)) return SA_ECUDA;
  return cuda_failed(launch_paged_join(a, scratch, f.row_tile, ctas, many_parts, stream)) ? SA_ECUDA : SA_OK;
}

SA_API sa_status sparse_attn_prefix_ws_bytes(const sa_paged_params* p, int32_t groups, uint64_t* out) {
  if (out == nullptr) return SA_EINVAL;
  const sa_status st = check_attn(p);
  if (st != SA_OK) return st;
  if (groups < 0 || p->window != 0) return SA_EINVAL;
  *out = shares(p, groups) ? shared_scratch_of(p, nullptr, nullptr, nullptr, nullptr) : scratch_of(nullptr, form_of(p), nullptr);
  return SA_OK;
}

SA_API sa_status sparse_attn_prefix_fwd(const sa_paged_params* p, int32_t groups, const void* q, const void* k_pages,
                                        const void* v_pages, const uint8_t* k_exp, const uint8_t* v_exp,
                                        const int32_t* table, const int32_t* row_start, const int32_t* kv_len,
                                        const int32_t* group_start, const int32_t* prefix_len, void* o, float* lse,
                                        void* ws, size_t ws_bytes, cudaStream_t stream) {
  uint64_t need = 0;
  sa_status st = sparse_attn_prefix_ws_bytes(p, groups, &need);
  if (st != SA_OK) return st;
  if (!group_start || (groups > 0 && !prefix_len)) return SA_EINVAL;
  if (!aligned(group_start, 4) || !aligned(prefix_len, 4)) return SA_EINVAL;
  if (!shares(p, groups))
    return sparse_attn_paged_fwd(p, q, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, o, lse, ws, ws_bytes,
                                 stream);
  if (bad_stride(p->a_token_stride) || bad_stride(p->a_head_stride)) return SA_EINVAL;
  if (!ws || !q || !o) return SA_EINVAL;
  if (!aligned(q, 16) || !aligned(o, 32) || !aligned(lse, 4)) return SA_EINVAL;
  st = check_pointers(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws);
  if (st != SA_OK) return st;
  if (ws_bytes < need) return SA_EINVAL;
  st = static_cast<sa_status>(device_status());
  if (st != SA_OK) return st;
  SharedAttnArgs a;
  static_cast<PagedAttnArgs&>(a) =
      attn_args(p, q, paged_args(p, k_pages, v_pages, k_exp, v_exp, table, row_start, kv_len, ws), o, lse);
  a.groups = groups;
  a.group_start = group_start;
  a.prefix_len = prefix_len;
  PagedScratch chunk, few;
  shared_scratch_of(p, ws, &chunk, &few, &a);
  const SharedForms f = shared_forms(p);
  const int64_t rows = int64_t(p->rows) * a.group;
  const PagedForm few_form = {f.row_tile, kPagedFewCtas, true};
  CUtensorMap tk, tv;
  ChunkMaps boxes{};
  if (f.few_own && !few_maps(p, k_pages, v_pages, &tk, &tv)) return SA_ECUDA;
  if (!f.few_prefix && !chunk_maps(p, k_pages, v_pages, &boxes)) return SA_ECUDA;
  // (every row is in a unit over its prefix, and in one over its own keys)
  bool many = false, many_few = false;
  int ctas = 0, few_ctas = 0;
  a.parts = f.few_own ? 1 : 3;
  if (!f.few_prefix) {
    const int64_t full = (rows + kPagedChunkRows - 1) / kPagedChunkRows;
    ctas = form_ctas(p, chunk_form(), groups + (f.few_own ? 0 : p->seqs), (f.few_own ? 1 : 2) * full, &many);
    if (ctas <= 0 || cuda_failed(launch_shared_chunk(boxes, a, chunk, ctas, stream))) return SA_ECUDA;
  }
  SharedAttnArgs own = a;
  own.parts = f.few_prefix ? 3 : 2;
  if (f.few_own) {
    const int64_t full = (rows + f.row_tile - 1) / f.row_tile;
    few_ctas = form_ctas(p, few_form, p->seqs + (f.few_prefix ? groups : 0), 2 * full, &many_few);
    if (few_ctas <= 0 || cuda_failed(launch_shared_few(tk, tv, own, few, f.row_tile, few_ctas, !f.few_prefix, stream)))
      return SA_ECUDA;
  }
  if (!f.few_prefix && cuda_failed(launch_shared_join(a, chunk, kPagedChunkRows, ctas, many, true, stream))) return SA_ECUDA;
  if (f.few_own && cuda_failed(launch_shared_join(own, few, f.row_tile, few_ctas, many_few, f.few_prefix, stream)))
    return SA_ECUDA;
  a.parts = 3;
  return cuda_failed(launch_shared_merge(a, stream)) ? SA_ECUDA : SA_OK;
}

SA_API sa_status sparse_attn_weigh_ws_bytes(const sa_paged_params* p, uint64_t* out) {
  if (out == nullptr) return SA_EINVAL;
  const sa_status st = check_attn(p);
  if (st != SA_OK) return st;
  // (lse / scale, which the form for chunks subtracts, and its parts are numbers then; so is
  // the half of a key's exponent that has scale in it in the forms for few rows, 2^64 at most
  // without, and an E4M3 key of the largest values gives a row of zeros the logit 0)
  if (p->scale < 0x1p-100f || p->scale > 0x1p60f) return SA_EUNSUPPORTED;
  *out = weigh_scratch_of(p, nullptr, nullptr);
  return SA_OK;
}

SA_API sa_status sparse_attn_cache_weigh(const sa_paged_params* p, int32_t first, int32_t accumulate, const void* q,
                                         const float* lse, const void* k_pages, const uint8_t* k_exp,
                                         const int32_t* table, const int32_t* row_start, const int32_t* kv_len,
                                         float* weights, void* ws, size_t ws_bytes, cudaStream_t stream) {
  uint64_t need = 0;
  sa_status st = sparse_attn_weigh_ws_bytes(p, &need);
  if (st != SA_OK) return st;
  if (bad_stride(p->a_token_stride) || bad_stride(p->a_head_stride)) return SA_EINVAL;
  if (first < 0 || (accumulate != 0 && accumulate != 1)) return SA_EINVAL;
  const bool unreported = !ws && ws_bytes == 0 && need == kStatusBytes;
  if ((!ws && !unreported) || !weights || (p->rows > 0 && (!q || !lse))) return SA_EINVAL;
  if (!aligned(q, 16) || !aligned(lse, 4) || !aligned(weights, 16)) return SA_EINVAL;
  // (V is not read: K stands in for it)
  st = check_pointers(p, k_pages, k_pages, k_exp, k_exp, table, row_start, kv_len, ws);
  if (st != SA_OK) return st;
  if (ws_bytes < need && !unreported) return SA_EINVAL;
  st = static_cast<sa_status>(device_status());
  if (st != SA_OK) return st;
  const int64_t longest = int64_t(p->table_width) * p->page_size;
  const bool few = weighs_few(p);
  if (few || p->rows == 0 || p->seqs == 0) {
    st = clear_status(ws, stream);
    if (st != SA_OK || p->rows == 0 || p->seqs == 0) return st;
  }
  WeighArgs w;
  w.a = attn_args(p, q, paged_args(p, k_pages, nullptr, k_exp, nullptr, table, row_start, kv_len, ws), nullptr, nullptr);
  w.lse = lse;
  w.weights = weights;
  w.first = first;
  w.accumulate = accumulate;
  const int sms = multiprocessors();
  if (sms <= 0) return SA_ECUDA;
  if (few) {
    const int64_t rows = int64_t(p->max_new < p->rows ? p->max_new : p->rows) * w.a.group;
    const int64_t tiles = (longest + 15) / 16 * p->seqs * p->H;
    // (at least one block: it reports what is wrong with the batch)
    return cuda_failed(launch_weigh(w, rows, sms, tiles > 0 ? tiles : 1, stream)) ? SA_ECUDA : SA_OK;
  }
  WeighScratch scratch;
  weigh_scratch_of(p, ws, &scratch);
  // no more CTAs than key blocks times steps that the call can have
  const int64_t blocks = (longest / kWeighKeys + 2) * p->seqs * p->H;
  const int64_t most = blocks * (int64_t(p->rows) * w.a.group / 96 + 2);
  int ctas = sms > kWeighCtas ? kWeighCtas : sms;
  if (most < ctas) ctas = static_cast<int>(most);
  return cuda_failed(launch_weigh_chunk(w, scratch, ctas, stream)) ? SA_ECUDA : SA_OK;
}

SA_API sa_status sparse_attn_cache_evict(const sa_paged_params* p, const sa_evict_params* e, void* k_pages,
                                         void* v_pages, uint8_t* k_exp, uint8_t* v_exp, float* weights,
                                         const int32_t* table, const int32_t* kv_len, const int32_t* to_table,
                                         int32_t* kept, int32_t* new_len, void* ws, cudaStream_t stream) {
  sa_status st = check_paged(p);
  if (st != SA_OK) return st;
  if (e == nullptr) return SA_EINVAL;
  if (e->keep < 1 || e->first < 0 || e->last < 0 || int64_t(e->first) + e->last > e->keep) return SA_EINVAL;
  if (to_table && (e->to_width < 0 || e->to_stride < 0)) return SA_EINVAL;
  // (the blocks of a launch, and positions that a block's step passes)
  if (e->keep > 1 << 30 || int64_t(p->seqs) * p->H >= int64_t(1) << 27 || int64_t(p->table_width) * p->page_size > int64_t(1) << 30)
    return SA_EUNSUPPORTED;
  if (!weights || (p->seqs > 0 && (!kept || !new_len))) return SA_EINVAL;
  if (!aligned(weights, 16) || !aligned(to_table, 4) || !aligned(kept, 4) || !aligned(new_len, 4)) return SA_EINVAL;
  // Lengths and tables are read by all blocks while others write what was kept.
  const int64_t all = int64_t(p->seqs) * p->H * e->keep;
  if (overlaps(new_len, p->seqs, kv_len, 1, p->seqs, 0) || overlaps(kept, all, kv_len, 1, p->seqs, 0) ||
      overlaps(kept, all, new_len, 1, p->seqs, 0) || overlaps(kept, all, table, p->seqs, p->table_width, p->table_stride) ||
      overlaps(new_len, p->seqs, table, p->seqs, p->table_width, p->table_stride) ||
      overlaps(kept, all, to_table, p->seqs, e->to_width, e->to_stride) ||
      overlaps(new_len, p->seqs, to_table, p->seqs, e->to_width, e->to_stride))
    return SA_EINVAL;
  st = check_pointers(p, k_pages, v_pages, k_exp, v_exp, table, k_pages /* no row_start */, kv_len, ws);
  if (st != SA_OK) return st;
  st = static_cast<sa_status>(device_status());
  if (st != SA_OK) return st;
  st = clear_status(ws, stream);
  if (st != SA_OK || p->seqs == 0) return st;
  const PagedArgs c = paged_args(p, k_pages, v_pages, k_exp, v_exp, table, nullptr, kv_len, ws);
  EvictArgs a;
  a.weights = weights;
  a.to_table = to_table;
  a.to_stride = e->to_stride;
  a.to_width = e->to_width;
  a.keep = e->keep;
  a.first = e->first;
  a.last = e->last;
  a.kept = kept;
  a.new_len = new_len;
  const int sms = multiprocessors();
  if (sms <= 0) return SA_ECUDA;
  return cuda_failed(launch_evict(c, a, sms, stream)) ? SA_ECUDA : SA_OK;
}
