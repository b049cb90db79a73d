// Definitions shared by the host side of the C ABI and the kernels.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sa {

constexpr int kBlock = 64;         // tokens per physical block
constexpr int kHeadDim = 128;      // head dimension
constexpr int kStatusBytes = 256;  // device status area at the start of a workspace
constexpr int kMaxList = 1024;     // largest supported block-list width (maxl)
constexpr int kMaxVideoBlocks = 8192;
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // bounded on-device waits: 1 s

// Block bookkeeping derived from sa_params (see sparse_attn.h).
struct Geometry {
  int T, H, Nv;
  int nvk;    // full video blocks
  int tail;   // Nv - 64 nvk
  int nblk;   // ceil(T / 64)
  int nq;     // sparse query blocks
  int K;      // Top-K budget
  int R;      // forced local radius
  int pad;    // 1 when the video tail block is routed (pad mode with tail > 0)
  int nsink;  // nblk - nvk
  int maxl;   // block-list width
  int r0;     // first dense query row
};

struct PlanArgs {
  const uint16_t* q;  // BF16 bits [T, H, 128]
  const uint16_t* k;
  float* qc;          // [H, nq, 128]
  float* kc;          // [H, nvk, 128]
  int32_t* idx;       // [H, nq, maxl]
  int32_t* cnt;       // [H, nq]
  float* scores;      // [H, nq, nvk] or null
  int32_t* status;    // the call's status words, zeroed by the pool kernel (or null)
  Geometry g;
};

struct AttnArgs {
  const int32_t* idx;
  const int32_t* cnt;
  const float* b2;     // key bias in log2 units [T], or null
  uint16_t* o;         // BF16 bits [T, H, 128]
  int32_t* status;     // device status word
  int32_t* unit_counter;  // next work unit (zeroed before the launch)
  const int32_t* bias_nz; // 1 when some key bias is nonzero (set by the bias prep)
  Geometry g;
  int n_dense;         // dense 128-row tiles per head
  int n_pairs;         // sparse query-block pairs per head
  float scale_log2;    // log2(e) / sqrt(128)
  // merged (Spark) mode: skipped video blocks enter as summary keys
  int merged;
  const float* lm2;    // log-mass in log2 units [H, nblkp]
  int nblkp;           // row stride of lm2 (a multiple of 64)
  float* vbias;        // per CTA and descriptor slot: summary-key logits [nvc][2][64]
  int vstride;         // floats per (CTA, slot): nvc * 2 * 64
  // fused mode: the kernel routes each unit from the block means and
  // exports the lists to idx_w / cnt_w (then read back as idx / cnt)
  int fused;
  const float* qc;     // [H, nq, 128]
  const float* kc;     // [H, nvk, 128]
  int32_t* idx_w;
  int32_t* cnt_w;
  int probe_once;      // testing build: every pipeline wait is a single probe
};

constexpr int kMaxFusedVideoBlocks = 256;  // video key blocks a fused route supports

constexpr int kMaxMergedCtas = 256;  // CTAs a merged launch may use (summary-key logit rows)

struct ReweightArgs {
  const uint16_t* a;   // BF16 anchors [P, H, 128]
  const uint16_t* k;   // BF16 [T, H, 128]
  const uint16_t* v;
  uint16_t* ak;        // BF16 [P, H, nblk, 128]
  uint16_t* av;
  float* lm;           // [P, H, nblk]
  int T, H, P, nblk;
  // Optional (merged forward, P = 1): lm in log2 units for the attention
  // kernel, [H, nblkp], 0 for blocks >= nvk and the padding.
  float* lm2;
  int nvk, nblkp;
};

// Launches `kern` with programmatic stream serialization: it may start while
// the stream's previous kernel finishes, and waits for that kernel on the
// device (griddep_wait) before touching what it wrote.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                             Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

// Raises a kernel's shared-memory limit once on each device (a static member
// of each launcher; setting it again is harmless).
struct SmemOnce {
  std::atomic<uint8_t> done[128] = {};
  cudaError_t set(const void* kern, uint32_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess && dev >= 0 && dev < 128) done[dev].store(1, std::memory_order_release);
    return e;
  }
};

// Records a failed CUDA call for sparse_attn_last_cuda_error (thread-local,
// defined in api.cu); returns true when `e` is an error.
bool cuda_failed(cudaError_t e);

// SA_OK when the current device is an sm_103 part (cached per device), else
// SA_EUNSUPPORTED or SA_ECUDA; an int of enum sa_status.
int device_status();

// Limit of a pipeline wait: kWaitLimitNs, or 0 while the testing hook is on.
uint64_t wait_limit_ns();

// Launchers (defined in the kernel translation units).
cudaError_t launch_pool(const PlanArgs& a, cudaStream_t s);
cudaError_t launch_route_topk(const PlanArgs& a, cudaStream_t s);
cudaError_t launch_bias_prep(const float* bias, float* b2, int32_t* status, const Geometry& g,
                             cudaStream_t s);
cudaError_t launch_attention(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const CUtensorMap& tak, const CUtensorMap& tav, const AttnArgs& a,
                             cudaStream_t s);
cudaError_t launch_spark_reweight(const ReweightArgs& r, cudaStream_t s);

// Spark token reblocking (landmark tree).
constexpr int kReblockMaxLandmarks = 64;
constexpr int kReblockMaxFanout = 16;
constexpr int kReblockMaxLevelNodes = 2000;  // split nodes per launch (the list is a kernel parameter)

struct ReblockArgs {
  const uint16_t* x;     // BF16 samples: row (t, h) at x + t * token_stride + h * head_stride
  int64_t token_stride;  // elements
  int64_t head_stride;   // elements
  int T, H, fanout, landmarks;
  int32_t* perm;         // [H, T]
  int32_t* inv;          // [H, T]
  void* ws;              // reblock_layout(T, H).total bytes, 256-byte aligned
};

struct ReblockLayout {
  size_t xh, keys, ord0, ord1, pairs, total;  // byte offsets: FP16 unit rows [H, N, 128], keys [H, N],
                                              // orders [H, N], landmark pairs int2 [H, N / 64]
};

ReblockLayout reblock_layout(int T, int H);
int reblock_depth(int m, int fanout);
cudaError_t launch_reblock(const ReblockArgs& r, cudaStream_t s);
int anchor_chunks(int Nv);
cudaError_t launch_video_query_mean(const uint16_t* q, float* partial, uint16_t* anchor, int H, int Nv,
                                    cudaStream_t s);

// Paged key/value cache (see sparse_attn.h for the batch and its checks).
struct PagedArgs {
  int kind;                  // sa_cache_kind
  int pages, H, page_size, page_shift;
  int seqs, table_width, rows, max_new;
  int64_t table_stride;
  const int32_t* table;
  const int32_t* row_start;  // [seqs + 1]
  const int32_t* kv_len;     // [seqs]
  uint8_t* k_pages;          // BF16 or E4M3 [pages, H, page_size, 128]
  uint8_t* v_pages;
  uint8_t* k_exp;            // [pages, H, page_size] (E4M3)
  uint8_t* v_exp;
  int32_t* status;           // device status word, or null
};

// Rows in (cache_write) or out (cache_read: contiguous).
struct CacheRows {
  uint16_t* k;
  uint16_t* v;
  int64_t k_token, k_head, v_token, v_head;  // strides, elements
};

struct PagedAttnArgs {
  static constexpr bool shared = false;
  PagedArgs c;
  const uint16_t* q;
  int64_t q_token, q_head;
  int Hq, group;             // group = Hq / H query heads a key head
  uint32_t group_mul;        // x / group = x group_mul >> group_shift for x < 2^31
  int group_shift;
  int causal, window;
  float scale;
  uint16_t* o;               // BF16 [rows, Hq, 128]
  float* lse;                // [rows, Hq] or null
  uint64_t wait_limit;       // of a pipeline wait, ns (0, the testing hook: a single probe)
};

// Attention where groups of sequences share the whole pages of a prefix: each
// row's result over the prefix and over its sequence's own keys, which
// launch_shared_merge joins.
struct SharedAttnArgs : PagedAttnArgs {
  static constexpr bool shared = true;
  int parts;      // of the line: 1 the prefixes, 2 the sequences with their own keys, 3 both
  int groups;
  const int32_t* group_start;  // [groups + 1]
  const int32_t* prefix_len;   // [groups]
  float* sums;    // [2: prefix, own][16][rows * Hq][8]: FP32 sums relative to the reference, eight dimensions together
  float2* refs;   // [2][rows * Hq]: reference in log2 units, sum
};

// Weights of cached keys [pages, H, page_size].
struct WeighArgs {
  PagedAttnArgs a;    // (its outputs and V are not used)
  const float* lse;   // [rows, Hq]
  float* weights;
  int first;          // keys below are left as they are
  int accumulate;     // 0: weights are set; 1: added to those of the tokens before the call's own
  // the form for chunks: a step's rows are `tokens` tokens of `heads` heads, of
  // which a group has `slices`; boxes: the tensor map of Q can be used
  int tokens, heads, slices, boxes;
};

// What the join needs of the unit (keys of one sequence and head) that begins
// in a CTA's part of the work and does not end there.
struct WeighJoin {
  int pieces;  // 0: none
  int s, h, key0;
  int lo, hi;  // keys whose weight is written
  int fresh;   // weights of keys below are added to
  int pad;
};
constexpr int kWeighKeys = 256;  // keys of a unit of the form for chunks
constexpr int kWeighCtas = 160;  // most CTAs of it
constexpr int kWeighFewRows = 128;  // most packed rows that paged_weigh.cu takes
struct WeighScratch {
  int32_t* cta_status;  // [ctas]
  WeighJoin* join;      // [ctas]
  float* part;          // [ctas][2][keys]
  uint4* shift;         // [rows, Hq]: -lse / scale as three BF16 parts, and zeros
};

struct EvictArgs {
  float* weights;
  const int32_t* to_table;  // pages of the tokens that stay, or null: the sequence's first ones
  int64_t to_stride;
  int to_width;
  int keep, first, last;
  int32_t* kept;            // [seqs, H, keep]
  int32_t* new_len;         // [seqs]
};

// What the joining kernel needs of the unit (a tile of packed rows of one
// sequence and key head) that begins in a CTA's part of the work and does not
// end there.
struct JoinDesc {
  int pieces;  // 0: none
  int row0;    // first row of the sequence
  int rho0;    // first packed row of the tile
  int rows;    // packed rows of the tile
  int h;
  int own;     // SharedAttnArgs: 0 over a prefix, 1 over own keys
  int pad[2];
};

// Workspace of paged_fwd: the status words, then a word and a JoinDesc of each
// CTA, then two partial results of each: FP32 sums relative to the row's
// reference, [row_tile][128] in the form for few rows and [16][row_tile][8] in
// the form for chunks, and [row_tile] (reference in log2 units, sum).
struct PagedScratch {
  int32_t* cta_status;  // [ctas]
  JoinDesc* join;       // [ctas]
  float* part;          // [ctas][2][row_tile * 128]
  float2* ml;           // [ctas][2][row_tile]
};

constexpr int kPagedFewRows = 16;   // most packed rows of the form for few rows
constexpr int kPagedFewKeys = 64;   // keys of its tiles
constexpr int kPagedFewCtas = 320;  // most CTAs of it (two an SM)
constexpr int kPagedChunkRows = 256;  // packed rows of a unit of the form for chunks
constexpr int kPagedChunkKeys = 80;   // keys of its tiles
constexpr int kPagedChunkCtas = 160;

struct PagedForm {
  int row_tile;  // packed rows of a unit
  int max_ctas;
  bool few;
};

cudaError_t launch_cache_write(const PagedArgs& c, const CacheRows& r, cudaStream_t s);
cudaError_t launch_cache_read(const PagedArgs& c, const CacheRows& r, cudaStream_t s);
cudaError_t launch_weigh(const WeighArgs& w, int64_t rows, int sms, int64_t key_tiles, cudaStream_t s);
cudaError_t launch_weigh_chunk(WeighArgs w, const WeighScratch& ws, int ctas, cudaStream_t s);
cudaError_t launch_evict(const PagedArgs& c, const EvictArgs& e, int sms, cudaStream_t s);
cudaError_t launch_paged_few(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a,
                             const PagedScratch& ws, int row_tile, int ctas, cudaStream_t s);
// K's and V's maps of the form for chunks, of BF16 pages: boxes of 16 (i + 1)
// keys, as many as a page and a key tile can have in common.
struct ChunkMaps {
  CUtensorMap m[2][kPagedChunkKeys / 16];
};
cudaError_t launch_paged_chunk(const ChunkMaps& maps, const PagedAttnArgs& a, const PagedScratch& ws, int ctas,
                               cudaStream_t s);
cudaError_t launch_paged_join(const PagedAttnArgs& a, const PagedScratch& ws, int row_tile, int ctas, bool many_parts,
                              cudaStream_t s);
// The same for rows that share prefixes (a.parts), and the join of a row's two
// results.  behind: the stream's previous kernel may still run (the other part).
cudaError_t launch_shared_chunk(const ChunkMaps& maps, const SharedAttnArgs& a, const PagedScratch& ws, int ctas,
                                cudaStream_t s);
cudaError_t launch_shared_few(const CUtensorMap& tk, const CUtensorMap& tv, const SharedAttnArgs& a, const PagedScratch& ws,
                              int row_tile, int ctas, bool behind, cudaStream_t s);
cudaError_t launch_shared_join(const SharedAttnArgs& a, const PagedScratch& ws, int row_tile, int ctas, bool many_parts,
                               bool first, cudaStream_t s);
cudaError_t launch_shared_merge(const SharedAttnArgs& a, cudaStream_t s);

// Tensor map of a row-major 2-D array of `elem`-byte elements, box
// [box_rows, 128 bytes], 128-byte swizzle, zeros past the last row.
bool make_map_rows(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, int elem, uint32_t box_rows);

// Tensor map of BF16 rows [rows, 128] (rows a multiple of 8) as [rows / 8][2
// halves][8 rows][64 columns]: a box is box_rows rows, written as one 1 KB
// block (8 rows x 128 bytes, 128-byte swizzle) for each half of each 8 rows.
bool make_map_groups(CUtensorMap* m, const void* ptr, uint64_t rows, uint32_t box_rows);

// Tensor map of BF16 rows of 128 at token * token_stride + head * head_stride
// (elements), heads in groups: [tokens][H][group][128]; a box is 64 columns of
// `box_heads` heads of one group and `box_tokens` tokens, 128-byte swizzle,
// zeros past a group's last head.  False where strides allow no map.
bool make_map_heads(CUtensorMap* m, const void* ptr, int tokens, int H, int group, int64_t token_stride,
                    int64_t head_stride, int box_tokens, int box_heads);

// The same of 16 bytes a head, contiguous [tokens, H * group], no swizzle.
bool make_map_heads16(CUtensorMap* m, const void* ptr, int tokens, int H, int group, int box_tokens, int box_heads);

size_t route_topk_smem_bytes(const Geometry& g);
size_t attention_smem_bytes();

}  // namespace sa
