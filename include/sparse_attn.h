/*
 * sparse_attn.h -- C ABI of the GB300 (sm_103a) Top-K block-sparse routed
 * attention library (forward pass, one GPU, one process).
 *
 * The method (sources are web pages, cited by title and section):
 *
 *   Q, K, V are contiguous BF16 [B=1, T, H, 128] ("Sol-Attn and Spark for
 *   MiniMax-H3", section "Install").  T is a target-video prefix of
 *   `video_tokens` tokens followed by a context suffix (same page, "H3
 *   pipeline integration").  Blocks are 64 tokens.  Let
 *     nvk  = floor(video_tokens / 64)      full video blocks (routed keys)
 *     nblk = ceil(T / 64)                  physical key blocks
 *     sinks = blocks nvk .. nblk-1         context sink blocks (always exact)
 *     K    = min(nvk, ceil(topk_ratio * nvk))
 *   sparse_attn_plan mean-pools Q and K per block, scores every video query
 *   block against every video key block, s = Qmean . Kmean / sqrt(128)
 *   ("Spark inference integration": native mean Top-K routing, packed route
 *   exported once), keeps the K best blocks by FP32 score (ties to the lower
 *   index) among the non-local video blocks, and adds the self block, its
 *   +-radius neighbours and every sink block outside the budget ("H3
 *   pipeline integration", sol_exact_block_radius; "Add key bias to chunked
 *   Sol-Attn producers", "Tests and source audit": sinks go straight into the
 *   exact list).
 *   sparse_attn_fwd runs exact softmax attention of each video query block
 *   over the union of its list, and dense attention over every key for the
 *   context rows and, with tail_mode = SA_TAIL_DENSE, for the rows of a video
 *   block cut by the boundary ("H3 pipeline integration").  With
 *   SA_TAIL_PAD that block is routed and attends sparsely; its centroid is
 *   the mean of its real video rows.  An optional key bias in natural-log
 *   units is added to the logits of sink keys only ("Add key bias to chunked
 *   Sol-Attn producers", "Summary" and "Contract").
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers on the current CUDA device,
 *     owned by the caller, 16-byte aligned and contiguous; the output `o` of
 *     the attention calls is 32-byte aligned (its rows are written by
 *     32-byte stores).  No entry point
 *     allocates device memory (the one fixed scratch array of
 *     sparse_attn_plan_static is part of the loaded library).
 *   - All GPU work is enqueued on `stream`; plan and fwd never synchronise
 *     the host.  Argument errors are returned before anything is enqueued.
 *   - A workspace `ws` of the size reported by sparse_attn_query belongs to
 *     one stream at a time; its first 256 bytes hold a device status word.
 *   - No fallback: when the GPU path cannot run, the call fails.
 */
#ifndef SPARSE_ATTN_H_
#define SPARSE_ATTN_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SA_ABI_VERSION 1u

typedef enum sa_status {
  SA_OK = 0,
  SA_EINVAL = 1,        /* bad argument, shape, pointer, size or key-bias value  */
  SA_EUNSUPPORTED = 2,  /* outside what this build supports (B != 1, D != 128,
                           a device that is not sm_103, sizes past the limits) */
  SA_ENOSINKBIAS = 3,   /* nonzero key bias on a routed video key (u < 64 nvk)  */
  SA_ECUDA = 4,         /* a CUDA runtime call or a kernel launch failed        */
  SA_ETIMEOUT = 5       /* a bounded on-device wait gave up; outputs invalid    */
} sa_status;

typedef enum sa_tail_mode { SA_TAIL_DENSE = 0, SA_TAIL_PAD = 1 } sa_tail_mode;

/* Problem description, passed by pointer to every call. */
typedef struct sa_params {
  uint32_t abi_version; /* must be SA_ABI_VERSION                               */
  int32_t B;            /* batch, must be 1 (packed batch size one)             */
  int32_t T;            /* packed tokens, >= 1                                  */
  int32_t H;            /* heads, >= 1                                          */
  int32_t D;            /* head dimension, must be 128                          */
  int32_t video_tokens; /* target-video prefix length Nv, 64 <= Nv <= T         */
  int32_t radius;       /* forced local radius R >= 0                           */
  int32_t tail_mode;    /* sa_tail_mode                                         */
  double topk_ratio;    /* Top-K ratio in (0, 1]; K = min(nvk, ceil(r * nvk)),
                           the product rounded as a decimal: a relative slack
                           of 1e-9 absorbs the binary representation of r     */
} sa_params;

/* Derived sizes and workspace requirements. */
typedef struct sa_sizes {
  int32_t nvk;             /* full video blocks                               */
  int32_t tail;            /* video_tokens - 64 nvk                           */
  int32_t nblk;            /* ceil(T / 64)                                    */
  int32_t nq;              /* sparse query blocks: nvk, +1 for a pad tail     */
  int32_t topk;            /* K                                               */
  int32_t nsink;           /* nblk - nvk                                      */
  int32_t maxl;            /* list width: min(nvk, 2R + 1 + K) + nsink        */
  int32_t dense_row_start; /* first densely evaluated query row               */
  uint64_t plan_ws_bytes;  /* workspace bytes for sparse_attn_plan            */
  uint64_t fwd_ws_bytes;   /* workspace bytes for sparse_attn_fwd             */
} sa_sizes;

/*
 * Validates `p` and fills `out`.  Host only: touches no device.
 * Errors: SA_EINVAL (null pointer, abi_version mismatch, T < 1, H < 1,
 * video_tokens outside [64, T], topk_ratio outside (0, 1], radius < 0,
 * unknown tail_mode, pad mode with T < 64 (nvk + 1) when the video tail is
 * nonempty); SA_EUNSUPPORTED (B != 1, D != 128, nvk > 8192, maxl > 1024,
 * T * H * 128 beyond 2^31 elements).
 */
sa_status sparse_attn_query(const sa_params* p, sa_sizes* out);

/*
 * Routing: pool + route scores + Top-K + block lists.
 *   q, k          BF16 [1, T, H, 128]
 *   idx           int32 [1, H, nq, maxl]: row (h, i) holds the sorted block
 *                 list of query block i in head h, padded with -1
 *   cnt           int32 [1, H, nq]: list lengths
 *   route_scores  optional (may be NULL) float32 [H, nq, nvk]: the scores
 *                 the selection compared (Qmean . Kmean / sqrt(128))
 *   ws, ws_bytes  workspace of at least plan_ws_bytes.  Layout after the
 *                 256-byte status area: Qmean float32 [H, nq, 128], then
 *                 Kmean float32 [H, nvk, 128], each 256-byte aligned.
 * Errors before launch: as sparse_attn_query, plus SA_EINVAL for a null or
 * misaligned required pointer or a short workspace.  SA_ECUDA if a launch
 * fails.
 */
sa_status sparse_attn_plan(const sa_params* p, const void* q, const void* k, int32_t* idx,
                           int32_t* cnt, float* route_scores, void* ws, size_t ws_bytes,
                           cudaStream_t stream);

/*
 * Attention: sparse video blocks over their lists, dense rows over all keys.
 *   q, k, v   BF16 [1, T, H, 128]
 *   key_bias  optional (may be NULL) float32 [B * T] in natural-log units.
 *             Converted once to log2 units.  Must be 0 on every key
 *             u < 64 nvk (else SA_ENOSINKBIAS); NaN or +inf anywhere gives
 *             SA_EINVAL; -inf removes the key.  Both are device-detected:
 *             read them with sparse_attn_last_device_status.
 *   idx, cnt  block lists from sparse_attn_plan (same params).  Lists are
 *             checked on the device before any of their blocks is loaded:
 *             1 <= cnt <= maxl, entries in [0, nblk) and strictly increasing,
 *             else SA_EINVAL (device-detected)
 *   o         BF16 [1, T, H, 128], 32-byte aligned; every row is written
 *             when the device status is SA_OK
 *   ws        workspace of at least fwd_ws_bytes (may alias none of the
 *             tensors above)
 * Errors before launch: as sparse_attn_plan.  Device-detected conditions
 * leave `o` unspecified and are reported by sparse_attn_last_device_status.
 */
sa_status sparse_attn_fwd(const sa_params* p, const void* q, const void* k, const void* v,
                          const float* key_bias, const int32_t* idx, const int32_t* cnt, void* o,
                          void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Routing without a caller workspace: the same computation and outputs as
 * sparse_attn_plan, with its scratch (status word and block means) kept in a
 * file-scope device array of SA_PLAN_STATIC_SCRATCH_BYTES instead of `ws`.
 * The source pages have no counterpart to this entry point.  It is for
 * callers that cannot give the library device scratch memory: plugins in a
 * host application whose device memory belongs to the host's own pool
 * allocator with no allocation hook for plugins, and code that must not call
 * cudaMalloc because it synchronises the device.  It allocates nothing.
 *   - Every GPU that loads the library holds the array until process exit.
 *   - Problems whose plan workspace (sparse_attn_query's plan_ws_bytes)
 *     exceeds SA_PLAN_STATIC_SCRATCH_BYTES return SA_EUNSUPPORTED before any
 *     launch.  The five reference workloads need at most 25.2 MiB.
 *   - The first call on a device looks up the array's device address with
 *     that device current (cudaGetSymbolAddress) and caches it; make that
 *     first call before any stream capture.
 *   - All calls share the array and it keeps the last call's contents: calls
 *     that overlap on the GPU (several streams or host threads) race, and the
 *     caller must serialise them.  The status area is cleared on each call.
 * Errors: as sparse_attn_plan (no workspace arguments).
 */
#define SA_PLAN_STATIC_SCRATCH_BYTES (32u * 1024u * 1024u)
sa_status sparse_attn_plan_static(const sa_params* p, const void* q, const void* k, int32_t* idx,
                                  int32_t* cnt, float* route_scores, cudaStream_t stream);

/*
 * Spark virtual summaries ("Sol-Attn and Spark for MiniMax-H3", section
 * "Spark primitives", spark_reweight; default numerics from section "Spark
 * inference integration").  For every anchor p, head h and physical 64-token
 * block b of K/V (a partial last block uses only its T - 64 b real keys):
 *     s_u = a[p, h] . k[u, h] / sqrt(128),   w = softmax over the block's u
 *     ak[p, h, b] = sum_u w_u k[u, h]        BF16 (round to nearest even)
 *     av[p, h, b] = sum_u w_u v[u, h]        BF16
 *     lm[p, h, b] = logsumexp_u(s_u) - a[p, h] . ak[p, h, b] / sqrt(128)
 * where the ak in lm is the stored BF16 value.  Scores, weights and sums are
 * FP32.  It does not choose anchors, routes or merge outputs.
 *   a        BF16 [1, P, H, 128] anchors (query representatives)
 *   k, v     BF16 [1, T, H, 128]
 *   ak, av   BF16 [1, P, H, nblk, 128], nblk = ceil(T / 64)
 *   lm       float32 [1, P, H, nblk]
 * Errors before launch: SA_EINVAL (null params or tensor pointer,
 * abi_version mismatch, T < 1, H < 1, P < 1, a tensor pointer not 16-byte
 * aligned, lm not 4-byte aligned); SA_EUNSUPPORTED (B != 1, D != 128,
 * T * H * 128 or P * H * nblk * 128 beyond 2^31 elements, a device that is
 * not sm_103).  SA_ECUDA if the launch fails.  Nothing is device-detected.
 */
typedef struct sa_reweight_params {
  uint32_t abi_version; /* must be SA_ABI_VERSION                               */
  int32_t B;            /* batch, must be 1                                     */
  int32_t T;            /* tokens of K and V, >= 1                              */
  int32_t H;            /* heads, >= 1                                          */
  int32_t D;            /* head dimension, must be 128                          */
  int32_t P;            /* anchors per head, >= 1                               */
} sa_reweight_params;

sa_status sparse_attn_spark_reweight(const sa_reweight_params* p, const void* a, const void* k,
                                     const void* v, void* ak, void* av, float* lm,
                                     cudaStream_t stream);

/*
 * Spark's merged attention ("Sol-Attn and Spark for MiniMax-H3", section
 * "Spark inference integration": one global representative per head formed
 * by averaging all target-video queries, stored as BF16; global-anchor K/V
 * and log-mass summaries merged with exact attention).  Same arguments,
 * lists and exact part as sparse_attn_fwd; in addition, per head, the
 * anchor a = BF16(mean of q rows t < video_tokens) is formed, its summaries
 * of every key block are computed as by sparse_attn_spark_reweight (P = 1),
 * and every video key block j < nvk that a sparse query block's list skips
 * enters that block's softmax as one extra key: ak[h, j] with logit
 * q . ak[h, j] / sqrt(128) + lm[h, j] and value av[h, j].  Dense rows are
 * exact over all keys as in sparse_attn_fwd.  The source pages have no
 * separate name for this call.
 *   ws  workspace of at least sparse_attn_spark_ws_bytes(p) bytes, 256-byte
 *       aligned.  Layout after the 256-byte status area (each part 256-byte
 *       aligned): key bias in log2 units float32 [T]; anchors BF16 [H, 128];
 *       anchor partial sums float32 [H, ceil(video_tokens / 1024), 128];
 *       ak, av BF16 [H, nblk, 128]; lm float32 [H, nblk]; lm in log2 units
 *       float32 [H, 64 ceil(nvk / 64)]; summary-key logits of each
 *       attention CTA float32 [256][2][ceil(nvk / 64)][2][64].
 * Errors: as sparse_attn_fwd (with this workspace size); SA_EUNSUPPORTED
 * also when H * nblk * 128 reaches 2^31.
 */
sa_status sparse_attn_spark_ws_bytes(const sa_params* p, uint64_t* out);
sa_status sparse_attn_spark_fwd(const sa_params* p, const void* q, const void* k, const void* v,
                                const float* key_bias, const int32_t* idx, const int32_t* cnt,
                                void* o, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Routing and attention in one call, with the Top-K taken inside the
 * attention kernel ("Sol-Attn and Spark for MiniMax-H3", section "Spark
 * inference integration": CTA-local fused Top-K routing, which removes the
 * external route pass).  Computes exactly what sparse_attn_plan followed by
 * sparse_attn_fwd computes, with the same FP32 scores and selection rule:
 * block means first, then each attention work unit scores its query blocks
 * against every video key block's mean, selects, and walks the lists it
 * made.  The lists are exported to idx / cnt (the layout of
 * sparse_attn_plan's outputs; here outputs of this call).
 *   ws  workspace of at least sparse_attn_fused_ws_bytes(p) bytes, 256-byte
 *       aligned: 256-byte status area, key bias in log2 units float32 [T],
 *       Qmean float32 [H, nq, 128], Kmean float32 [H, nvk, 128] (each part
 *       256-byte aligned).
 * Errors: as sparse_attn_fwd (with this workspace size); SA_EUNSUPPORTED
 * also when nvk > 256 (rows of at most 256 video blocks are routed in one
 * warp's registers).
 */
sa_status sparse_attn_fused_ws_bytes(const sa_params* p, uint64_t* out);
sa_status sparse_attn_fused(const sa_params* p, const void* q, const void* k, const void* v,
                            const float* key_bias, int32_t* idx, int32_t* cnt, void* o, void* ws,
                            size_t ws_bytes, cudaStream_t stream);

/*
 * Spark token reblocking ("Sol-Attn and Spark for MiniMax-H3", section
 * "Spark primitives", spark_reblock: a permutation of each head's tokens
 * into 64-token blocks by a landmark tree, with its inverse; fanout with
 * power-of-two scheduling and cosine scoring on normalized FP16 vectors from
 * section "Spark inference integration").  The pages name the ingredients,
 * not the steps; this call computes, per head h independently:
 *   N = 64 floor(T / 64); tokens t >= N (the flat order's remainder) keep
 *   their place at the end.  Each token is scored as its FP16 unit vector
 *   (FP32 norm, zero rows stay zero).  The root node is [0, N) in flat
 *   order; a node of m > 1 blocks splits into c children, c the largest
 *   power of two <= min(fanout, m), child i taking floor(m / c) + [i < m % c]
 *   blocks.  Its landmarks are the tokens at positions floor(j n / L),
 *   j < L = min(landmarks, n), of its current order (n tokens); the pair
 *   with the smallest cosine (ties to the lower (j, j')) gives a and b;
 *   tokens ranked by (cos(t, a) - cos(t, b), position) fill child 0, 1, ...
 *   in turn, and each child keeps the node's order.  Leaves are the blocks.
 *   Cosines are FP32 sums of exact FP16 products in a fixed order (per
 *   lane four consecutive terms left to right, then a butterfly over 32
 *   lanes), so the integer result is reproducible bit for bit.
 *   x      BF16 samples, row (t, h) at x + t * token_stride + h * head_stride
 *          (elements; [1, T, H, 128] has token_stride = 128 H, head_stride =
 *          128); 16-byte aligned, strides multiples of 8.  Read only.
 *   perm   int32 [H, T]: perm[h, i] = original token at new position i;
 *          the blocks are perm[h, 64 b : 64 b + 64], the excluded remainder
 *          perm[h, N:].
 *   inv    int32 [H, T]: inv[h, perm[h, i]] = i.
 *   ws     workspace of sparse_attn_reblock_ws_bytes(p) bytes, 256-byte
 *          aligned: FP16 unit rows [H, N, 128], keys uint64 [H, N], two
 *          orders int32 [H, N], landmark pairs int32 [H, N / 64, 2] (each
 *          256-byte aligned).  Owned by the caller.
 * Errors before launch: SA_EINVAL (null params or pointer, abi_version
 * mismatch, T < 1, H < 1, fanout not a power of two in [2, 16], landmarks
 * outside [2, 64], a negative stride or one not a multiple of 8, x not
 * 16-byte aligned, perm or inv not 4-byte aligned, ws not 256-byte aligned or
 * short); SA_EUNSUPPORTED (D != 128, H > 65535, T * H >= 2^31, a device that
 * is not sm_103).  SA_ECUDA if a launch fails.  Nothing is device-detected.
 */
typedef struct sa_reblock_params {
  uint32_t abi_version; /* must be SA_ABI_VERSION                               */
  int32_t T;            /* tokens, >= 1                                         */
  int32_t H;            /* heads (independent sample matrices), >= 1            */
  int32_t D;            /* feature dimension, must be 128                       */
  int32_t fanout;       /* children per split at most: 2, 4, 8 or 16            */
  int32_t landmarks;    /* landmarks per split, [2, 64] (32 by default)         */
  int64_t token_stride; /* elements between tokens t and t + 1 of one head      */
  int64_t head_stride;  /* elements between heads h and h + 1 of one token      */
} sa_reblock_params;

sa_status sparse_attn_reblock_ws_bytes(const sa_reblock_params* p, uint64_t* out);
sa_status sparse_attn_spark_reblock(const sa_reblock_params* p, const void* x, int32_t* perm,
                                    int32_t* inv, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Paged key/value cache, and attention of new tokens over it.  Whoever
 * generates chunk by chunk (a video continued from a cached clip, a language
 * model that serves many users) keeps K and V between calls, for many
 * sequences of uneven length, and attends from the new tokens only.
 *
 * Cache.  k_pages, v_pages [pages, H, page_size, 128], contiguous, in one of
 *   two kinds:
 *   SA_CACHE_BF16  BF16 rows as they came.
 *   SA_CACHE_E4M3  8-bit E4M3 codes, each row (one token of one head) with
 *                  a power-of-two scale: with amax the row's largest
 *                  magnitude, e is the smallest integer >= -126 such that
 *                  amax <= 448 * 2^e, a code is x * 2^-e rounded to nearest
 *                  even, and k_exp, v_exp uint8 [pages, H, page_size] hold
 *                  e + 127.  Scaling by 2^e is exact both ways, so the
 *                  code's own rounding is the only one, and what a code
 *                  stands for is a BF16 value, a finite one (for e = 120 the
 *                  largest code used is 240's: 256 * 2^120 would not be).  A
 *                  row that holds a NaN or an infinity has the exponent byte
 *                  255 and NaN codes: all of it stands for NaN.  Two things
 *                  that cache_write never makes stand for nothing certain: a
 *                  NaN code under another exponent byte (to paged_fwd it is a
 *                  NaN or 480, by the form that a call takes) and a code that
 *                  with its exponent byte is past the largest BF16 value
 *                  (outputs of that sequence are unspecified).
 * Batch (device memory, int32, read by every call).  Sequence s < seqs has
 *   kv_len[s] tokens; token j is in slot j % page_size of page
 *   table[s * table_stride + j / page_size].  The rows row_start[s] ..
 *   row_start[s + 1] - 1 of a packed tensor are its last tokens: with n of
 *   them, row i is the token at position kv_len[s] - n + i.  A position below
 *   0 is no token: it is not written, reads as zeros and attends to nothing
 *   (with causal = 0, to every token, like the others).  Rows before
 *   row_start[0] or from row_start[seqs] on belong to no sequence and are
 *   left as they were.
 *   Table entries of pages that no token of the call needs are not read.  A
 *   page may stand in several rows of the table (a shared prefix); a slot
 *   that two rows of one write call reach holds either row's values after it,
 *   in the E4M3 kind possibly one's codes and the other's exponent.
 * Checked on the device, before any access that depends on it: 0 <=
 *   row_start[s] <= row_start[s + 1] <= rows, at most max_new rows a sequence,
 *   0 <= kv_len[s] <= table_width * page_size, and every page used in
 *   [0, pages).  What fails is SA_EINVAL in the status word of `ws`
 *   (sparse_attn_last_device_status): the sequence, or the tokens of the
 *   page, are left out, and the outputs of that sequence are unspecified.
 */
typedef enum sa_cache_kind { SA_CACHE_BF16 = 0, SA_CACHE_E4M3 = 1 } sa_cache_kind;

typedef struct sa_paged_params {
  uint32_t abi_version;  /* must be SA_ABI_VERSION                              */
  int32_t kind;          /* sa_cache_kind                                       */
  int32_t pages;         /* pages of the pool, >= 1                             */
  int32_t H;             /* key heads, >= 1                                     */
  int32_t page_size;     /* tokens a page: 16, 32, 64 or 128                    */
  int32_t D;             /* head dimension, must be 128                         */
  int32_t seqs;          /* sequences, >= 0                                     */
  int32_t table_width;   /* page-table entries a sequence, >= 0                 */
  int64_t table_stride;  /* elements between the table rows, >= 0               */
  int32_t rows;          /* rows of the packed tensors, >= 0                    */
  int32_t max_new;       /* most rows of one sequence, >= 0 (rows is always
                            right; a tight bound lets paged_fwd pick the form
                            for few tokens)                                     */
  int32_t Hq;            /* query heads, a multiple of H: query head i reads
                            key head i / (Hq / H) (paged_fwd only)              */
  int32_t causal;        /* 1: a row sees keys up to its own position; 0: all
                            kv_len keys of its sequence (paged_fwd only)        */
  int32_t window;        /* w > 0: only the last w of the keys a causal row
                            sees, its own among them; 0: all (paged_fwd only)   */
  float scale;           /* logit of a key: scale * (q . k); > 0, finite (paged_fwd) */
  int64_t a_token_stride, a_head_stride; /* elements, of k (cache_write) or q
                            (paged_fwd): multiples of 8                         */
  int64_t b_token_stride, b_head_stride; /* of v (cache_write)                  */
} sa_paged_params;

/*
 * Writes rows of K and V into the cache.
 *   k, v   BF16 rows (r, h) at k + r * a_token_stride + h * a_head_stride and
 *          v + r * b_token_stride + h * b_head_stride, 128 contiguous elements
 *   ws     optional (may be NULL): 256 bytes whose first word takes the
 *          status; without it what is left out is not reported
 * Errors before launch: SA_EINVAL (null or misaligned pointer: 16 bytes for
 * k, v and the pages, 4 for the batch, 256 for ws; k_exp, v_exp null with
 * SA_CACHE_E4M3; a field outside its range; a stride that is negative or no
 * multiple of 8; kind or page_size unknown); SA_EUNSUPPORTED (D != 128,
 * pages * H * page_size >= 2^31, table_width * page_size >= 2^31 - 256,
 * rows * H >= 2^31 or rows * Hq >= 2^31 - 4096, a device that is not sm_103).  SA_ECUDA if a launch fails.
 */
sa_status sparse_attn_cache_write(const sa_paged_params* p, const void* k, const void* v, void* k_pages,
                                  void* v_pages, uint8_t* k_exp, uint8_t* v_exp, const int32_t* table,
                                  const int32_t* row_start, const int32_t* kv_len, void* ws,
                                  cudaStream_t stream);

/*
 * Reads cached rows back as BF16: the inverse of sparse_attn_cache_write, and
 * with row_start spanning whole contexts the packed [T, H, 128] tensors that
 * sparse_attn_plan and sparse_attn_fwd take.
 *   k, v   BF16 [rows, H, 128], contiguous
 * Errors: as sparse_attn_cache_write.
 */
sa_status sparse_attn_cache_read(const sa_paged_params* p, const void* k_pages, const void* v_pages,
                                 const uint8_t* k_exp, const uint8_t* v_exp, const int32_t* table,
                                 const int32_t* row_start, const int32_t* kv_len, void* k, void* v, void* ws,
                                 cudaStream_t stream);

/*
 * Attention of rows of Q over the cached keys of their sequence (their own
 * tokens' K and V are in the cache already).  One softmax a row, in FP32;
 * logits scale * (q . k).
 *   q     BF16 rows (r, h) at q + r * a_token_stride + h * a_head_stride
 *   o     BF16 [rows, Hq, 128], contiguous, 32-byte aligned; zeros for a row
 *         that sees no key
 *   lse   optional (may be NULL) float32 [rows, Hq]: natural logarithm of the
 *         sum of exp(logit), -inf for a row that sees no key, NaN for one
 *         that sees a logit which is NaN
 *   ws    workspace of sparse_attn_paged_ws_bytes(p) bytes: the status word
 *         in the first 256, then scratch of this call
 * Cached values behind kv_len, or below the window of every row, are never
 * used, whatever they are.
 * Logits and sums are FP32.  A row's probabilities are taken relative to a
 * reference that is never below its largest logit so far: o is finite where
 * sum exp(logit - largest) |v| stays under 2^128, and a key 2^118 times less
 * probable than the most probable one may count as 0.
 * For few rows over E4M3 pages, elements of a query head's row below 2^-30 of
 * its largest one lose bits.
 * Errors: as sparse_attn_cache_write, and SA_EINVAL for Hq not a multiple of
 * H, causal not 0 or 1, window < 0 or with causal = 0, scale not positive and finite, o
 * not 32-byte or lse not 4-byte aligned, a short workspace.
 */
sa_status sparse_attn_paged_ws_bytes(const sa_paged_params* p, uint64_t* out);
sa_status sparse_attn_paged_fwd(const sa_paged_params* p, const void* q, const void* k_pages,
                                const void* v_pages, const uint8_t* k_exp, const uint8_t* v_exp,
                                const int32_t* table, const int32_t* row_start, const int32_t* kv_len,
                                void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * The same attention for a batch in which groups of sequences begin with the
 * same tokens (one instruction before many questions, several continuations of
 * one clip): the keys of a prefix are read and multiplied once for all rows of
 * its group, and joined with each row's own keys in one softmax.
 *   groups       groups, >= 0
 *   group_start  int32 [groups + 1], device memory, ascending: group g is the
 *                sequences group_start[g] .. group_start[g + 1] - 1 (others
 *                share nothing)
 *   prefix_len   int32 [groups], device memory: the first prefix_len[g] tokens
 *                of all sequences of group g are the same.  Those in whole
 *                pages are read once, from the pages of the group's first
 *                sequence that has rows, which the others' table rows name
 *                too (or pages that hold the same); the rest of them, as all
 *                other tokens, by each sequence's own row.  A group of one
 *                sequence shares nothing; of one without rows, neither kv_len
 *                nor the table's row has to agree with its group
 * Everything else is as in sparse_attn_paged_fwd, and so is the result, up to
 * the order of sums.  window must be 0.  It is the faster one where the shared
 * keys, counted once for each sequence, are about 130000 or more (64 sequences
 * of one token behind 4096 keys: 56 us and 72; behind 1024: 48 and 32).
 *   ws  workspace of sparse_attn_prefix_ws_bytes(p, groups) bytes (1040 for
 *       each row and query head, besides those of sparse_attn_paged_fwd)
 * Checked on the device besides: 0 <= group_start[g] <= group_start[g + 1] <=
 * seqs, 0 <= prefix_len[g] <= table_width * page_size, and that a sequence's
 * own rows lie behind its group's whole shared pages; else SA_EINVAL in the
 * status word, and the outputs of the group, or of the sequence, are
 * unspecified.  Where seqs < 2 or rows is 0 nothing can be shared: the call is
 * sparse_attn_paged_fwd's, and the groups are not looked at.
 * Errors: as sparse_attn_paged_fwd; SA_EINVAL also for groups < 0, window not
 * 0, a null or misaligned group_start, or prefix_len with groups > 0.
 */
sa_status sparse_attn_prefix_ws_bytes(const sa_paged_params* p, int32_t groups, uint64_t* out);
sa_status sparse_attn_prefix_fwd(const sa_paged_params* p, int32_t groups, const void* q, const void* k_pages,
                                 const void* v_pages, const uint8_t* k_exp, const uint8_t* v_exp,
                                 const int32_t* table, const int32_t* row_start, const int32_t* kv_len,
                                 const int32_t* group_start, const int32_t* prefix_len, void* o, float* lse,
                                 void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * The attention weight that cached keys receive, by which
 * sparse_attn_cache_evict chooses: for each key head h and key j >= first of a
 * sequence with rows in the call,
 *     w[j] = (what w[j] was, or 0) + sum exp(scale * (q . k_j) - lse)
 * over the rows that see key j and the query heads that read key head h, in
 * FP32.  What w[j] was counts with accumulate = 1 and only for tokens before
 * the call's own rows; a token's own call, and every call with accumulate = 0,
 * sets it.  Fields of `p`, batch, q and checks as in sparse_attn_paged_fwd
 * (causal, window, scale as in the call that gave lse); V is not read.
 *   lse      float32 [rows, Hq], contiguous: sparse_attn_paged_fwd's or
 *            sparse_attn_prefix_fwd's of the same rows.  A row whose lse is
 *            -inf counts nothing
 *   weights  float32 [pages, H, page_size], contiguous, 16-byte aligned: the
 *            weight of the token in a page's slot
 *   first    keys at positions below it keep their weights (those that an
 *            eviction keeps anyway, or a prefix that several sequences share)
 *   accumulate  0 or 1
 *   ws       workspace of sparse_attn_weigh_ws_bytes(p) bytes, the status word first.
 *            Where that is 256 (the status alone) it may be NULL with ws_bytes
 *            0, as in sparse_attn_cache_write
 * With accumulate = 1 a key that no row sees is left as it was, with 0 it gets
 * 0.  Sequences without rows are left as they were.  A page that stands in
 * several rows of the table must lie below `first` in all of them but one;
 * else its weights are unspecified.  Results do not depend on the order in
 * which the device works.
 * For few rows over E4M3 pages, elements of a query head's row below 2^-30 of
 * its largest one lose bits.
 * Errors: as sparse_attn_paged_fwd; SA_EINVAL also for first < 0, accumulate
 * not 0 or 1, a null or misaligned lse or weights; SA_EUNSUPPORTED also for a
 * scale outside [2^-100, 2^60].
 */
sa_status sparse_attn_weigh_ws_bytes(const sa_paged_params* p, uint64_t* out);
sa_status sparse_attn_cache_weigh(const sa_paged_params* p, int32_t first, int32_t accumulate, const void* q,
                                  const float* lse, const void* k_pages, const uint8_t* k_exp,
                                  const int32_t* table, const int32_t* row_start, const int32_t* kv_len,
                                  float* weights, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Eviction: of every sequence with more than `keep` tokens each key head keeps
 * `keep` of them: the first `first` and the last `last`, and of those between
 * the ones with the largest weights (of equal ones the earlier; +0 and -0 are
 * equal, NaN is above all).  The tokens that a head keeps move, in their
 * order, to the positions 0 .. of the sequence: rows of K and V as they are,
 * exponents, and weights.  Heads keep different tokens; what a position was is
 * told by `kept`.  A sequence of at most `keep` tokens keeps all.
 *   to_table  NULL: in place, the sequence's first pages.  Then no page that
 *             holds a token at position `first` or later may stand in another
 *             row of the table.  Else int32 table [seqs] rows of to_width
 *             entries, to_stride apart: the pages that the tokens go to, none
 *             of which holds a token of the call.  The old pages stay as they
 *             were, and sequences that keep all are copied.
 *   weights   float32 [pages, H, page_size], 16-byte aligned
 *   kept      int32 [seqs, H, keep]: the former position of the token at
 *             position i, -1 from the new length on
 *   new_len   int32 [seqs]: min(kv_len, keep)
 * kept and new_len must not overlap each other, kv_len or a table.
 *   ws        optional (may be NULL): 256 bytes whose first word takes the status
 * Slots from the new length on are left as they were.  Later rows see kept
 * tokens by their new positions (a window counts kept tokens).
 * Of `p`, rows, max_new, Hq, causal, window, scale and the strides are not
 * used.  Checked on the device: 0 <= kv_len[s] <= table_width * page_size, all
 * pages of its tokens and of their destinations in [0, pages), room for them
 * in to_width pages; else SA_EINVAL in the status word: nothing of that
 * sequence moves, kept is -1 throughout and new_len is kv_len.
 * Errors before launch: as sparse_attn_cache_write; SA_EINVAL also for keep <
 * 1, first or last < 0, first + last > keep, a null or misaligned weights,
 * kept or new_len, outputs that overlap as above; SA_EUNSUPPORTED also for keep > 2^30,
 * seqs * H >= 2^27, table_width * page_size > 2^30.
 */
typedef struct sa_evict_params {
  int32_t keep;       /* tokens that a sequence may have after the call, >= 1   */
  int32_t first;      /* tokens at its start that stay, >= 0                    */
  int32_t last;       /* tokens at its end that stay, >= 0                      */
  int32_t to_width;   /* entries of a row of to_table, >= 0                     */
  int64_t to_stride;  /* elements between the rows of to_table, >= 0            */
} sa_evict_params;

sa_status sparse_attn_cache_evict(const sa_paged_params* p, const sa_evict_params* e, void* k_pages, void* v_pages,
                                  uint8_t* k_exp, uint8_t* v_exp, float* weights, const int32_t* table,
                                  const int32_t* kv_len, const int32_t* to_table, int32_t* kept, int32_t* new_len,
                                  void* ws, cudaStream_t stream);

/*
 * Reads the device status word of `ws` (written by the last plan or fwd
 * enqueued with it).  Synchronises `stream`.  SA_ECUDA if the copy fails.
 */
sa_status sparse_attn_last_device_status(const void* ws, cudaStream_t stream, sa_status* out);

/*
 * Testing hook (the source pages have no counterpart).  Every on-device
 * pipeline wait of the attention kernels gives up after 1 s: the kernel then
 * records SA_ETIMEOUT in the workspace status word, lets its own copies and
 * MMAs in flight finish (those waits keep the 1 s limit), frees its tensor
 * memory and returns; the outputs of that call are invalid.  With `on`
 * nonzero, later launches by sparse_attn_fwd, sparse_attn_spark_fwd,
 * sparse_attn_fused, sparse_attn_paged_fwd, sparse_attn_prefix_fwd and (its form
 * for chunks) sparse_attn_cache_weigh are ones in which every pipeline
 * wait is a single probe, so that a call almost surely times out: it exists to
 * test that path.  Process-wide; returns the previous setting (0 or 1).
 * Host only: touches no device.
 */
int sparse_attn_set_single_probe_waits(int on);

/*
 * The last CUDA runtime error that made an entry point return SA_ECUDA on
 * the calling host thread (0 = none since the thread started), and its
 * message when `message` is not NULL.  Host only.
 */
int sparse_attn_last_cuda_error(const char** message);

/* Static, human-readable name of a status code. */
const char* sparse_attn_status_string(sa_status s);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_ATTN_H_ */
