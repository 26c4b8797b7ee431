/*
 * infllmv2.h -- C ABI of the InfLLM v2 block-sparse attention library (sm_103a).
 *
 * The method is the trainable sparse attention of the MiniCPM4 technical
 * report ("MiniCPM4: Ultra-Efficient LLMs on End Devices", section "InfLLM v2:
 * Trainable Sparse Attention for Both Prefilling and Decoding"; cited below as
 * [InfLLM v2 > paragraph, equation]).  Three stages:
 *
 *   1. infllmv2_compress_keys       semantic-kernel key means
 *                                   [InfLLM v2 > Semantic kernels, eq. S_j]
 *   2. infllmv2_select_blocks       per-head kernel softmax, GQA group mean,
 *                                   block max, forced blocks, top-k
 *                                   [InfLLM v2 > Semantic kernels, eqs. r_kernel,
 *                                   r_block; > Query group sharing, eq. r_group;
 *                                   > Top-K implementation and the LSE bottleneck;
 *                                   > Initial and local tokens always selected]
 *   3. infllmv2_sparse_attn_decode  exact softmax attention over the selected
 *      infllmv2_sparse_attn_prefill KV blocks [InfLLM v2 > Block-level key-value
 *                                   partitioning, eq. B_j; > Complexity analysis]
 *
 * Around them: infllmv2_append_kv and infllmv2_decode_step (a whole decode
 * step, one launch for n_q = 1), infllmv2_append_decode_step (both as one
 * launch), infllmv2_coarse_means and
 * infllmv2_select_blocks_coarse_lse (the coarse-kernel LSE approximation),
 * and infllmv2_sparse_attn_backward (gradients of stage 3 with the selection
 * fixed [InfLLM v2 > Training-time considerations]).
 *
 * Beside the contiguous caches above, a cache of pages for serving many
 * sequences from one pool, attended densely: infllmv2_paged_append_kv,
 * infllmv2_paged_attn_decode and infllmv2_paged_evict (see there; they have
 * shapes and types of their own).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every tensor argument is a DEVICE pointer owned by the caller (the few
 *   arguments documented as possibly host memory excepted).  The
 *   library never allocates, frees or synchronises in these calls; all work
 *   is enqueued on `stream` (a cudaStream_t passed as void*, NULL = legacy
 *   default stream) and the calls return before it runs.  (One exception:
 *   the prefill selection past 327360 tokens of capacity reads the device's
 *   SM-identifier bound once per device with a small synchronous query on a
 *   private stream; see infllmv2_select_blocks.)
 * - Shapes (row-major, innermost last; d = head_dim, G = group_size,
 *   Hq = n_kv_heads * G, n_c(L) = floor((L - p)/s) + 1 complete kernels,
 *   n_b(L) = ceil(L / m) blocks):
 *       q          bf16  [batch, n_q, Hq, d]        (heads h*G .. h*G+G-1 share KV head h)
 *       k_cache    bf16  [batch, n_kv_heads, max_kv_len, d]
 *       v_cache    bf16  [batch, n_kv_heads, max_kv_len, d]
 *       kv_lens    int32 [batch]                    (L_b, including the n_q query tokens)
 *       kc         bf16  [batch, n_kv_heads, 2, n_c(max_kv_len), d]
 *                  plane 0 holds hi = bf16(mean), plane 1 lo = bf16(mean - hi):
 *                  hi + lo is the fp32 kernel mean to 16 significant bits.
 *       block_idx  int32 [batch, n_kv_heads, n_q, k_max]   ascending, padded with -1
 *       n_selected int32 [batch, n_kv_heads, n_q]
 *       out        bf16  [batch, n_q, Hq, d]
 *       lse        fp32  [batch, n_q, Hq]           natural-log sum of exp of the
 *                                                   scaled scores of the attended keys
 * - Query t (0 <= t < n_q) of sequence b sits at position i = L_b - n_q + t; it
 *   attends keys 0..i of its selected blocks (inclusive causal mask).  The
 *   same rule serves decode (n_q = 1), speculative verification (small n_q)
 *   and causal prefill (n_q = L_b).
 * - Pointers must be 16-byte aligned.  Supported shape: head_dim 128,
 *   group_size 16, block_size 64, kernel_size 32, kernel_stride 16;
 *   anything else returns INFLLMV2_UNSUPPORTED.
 * - Return codes are INFLLMV2_* below; on failure nothing was launched and
 *   infllmv2_last_error() describes why (thread-local string).  Problems only
 *   the device can see (a kv_len outside [n_q, max_kv_len], a bounded wait
 *   that gave up) are recorded in a device status word read by
 *   infllmv2_get_device_status(); the affected unit writes zeros / an empty
 *   selection instead of reading out of bounds.
 * - No C++ exception crosses this boundary.
 */
#ifndef INFLLMV2_H
#define INFLLMV2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define INFLLMV2_OK                  0
#define INFLLMV2_INVALID_ARGUMENT    1  /* null pointer, bad size, topk < forced count, ... */
#define INFLLMV2_UNSUPPORTED         2  /* shape outside the supported set, misaligned pointer */
#define INFLLMV2_WORKSPACE_TOO_SMALL 3
#define INFLLMV2_CUDA_ERROR          4  /* launch failed; message from the CUDA runtime */

/* Device status bits (infllmv2_get_device_status). */
#define INFLLMV2_DEVICE_BAD_KV_LEN   0x1u  /* kv_lens[b] < n_q or > max_kv_len */
#define INFLLMV2_DEVICE_TIMEOUT      0x2u  /* a bounded mbarrier wait expired */
#define INFLLMV2_DEVICE_BOUNDS       0x4u  /* checked build only: a caller-given index out of range */
#define INFLLMV2_DEVICE_BAD_PAGE     0x8u  /* a page-table entry in use is outside [0, num_pages) */

/* Workspace kinds for infllmv2_workspace_size. */
#define INFLLMV2_OP_SELECT  1
#define INFLLMV2_OP_DECODE  2
#define INFLLMV2_OP_PREFILL 3
#define INFLLMV2_OP_DECODE_STEP 4
#define INFLLMV2_OP_BACKWARD 5
/* For infllmv2_paged_workspace_size. */
#define INFLLMV2_OP_PAGED_DECODE 6
#define INFLLMV2_OP_PAGED_EVICT  7

typedef struct infllmv2_params {
  int32_t batch;                 /* B */
  int32_t n_kv_heads;            /* Hkv */
  int32_t group_size;            /* G, query heads per KV head (16) */
  int32_t head_dim;              /* d (128) */
  int32_t block_size;            /* m (64)  [InfLLM v2 > Block-level key-value partitioning] */
  int32_t kernel_size;           /* p (32)  [InfLLM v2 > Semantic kernels] */
  int32_t kernel_stride;         /* s (16)  [InfLLM v2 > Semantic kernels] */
  int32_t topk;                  /* k, blocks per query group */
  int32_t n_init_blocks;         /* forced initial blocks (1) [InfLLM v2 > Initial and local tokens] */
  int32_t n_local_blocks;        /* forced local blocks ending at the query's block (2) */
  int32_t topk_includes_forced;  /* 1: forced blocks count toward k; 0: k scored blocks on top */
  int32_t max_kv_len;            /* cache capacity per (b, h) in tokens */
  float score_scale;             /* scale inside the kernel softmax (default 1/sqrt(d)) */
  float attn_scale;              /* attention softmax scale (default 1/sqrt(d)) */
} infllmv2_params;

/* Fill `p` with the recommended shape (d 128, G 16, m 64, p 32, s 16, one
 * initial and two local blocks, both scales 1/sqrt(128)). */
void infllmv2_default_params(infllmv2_params* p, int32_t batch, int32_t n_kv_heads,
                             int32_t max_kv_len, int32_t topk, int32_t topk_includes_forced);

/* Width of a block_idx row: topk if forced blocks are included, else
 * topk + n_init_blocks + n_local_blocks.  Negative on invalid params. */
int32_t infllmv2_max_selected(const infllmv2_params* p);

/* n_c(max_kv_len): rows of each kc plane. */
int32_t infllmv2_num_kernels(const infllmv2_params* p);

/* Bytes of scratch that `op` (INFLLMV2_OP_*) needs for n_q query tokens per
 * sequence.  0 on invalid arguments. */
size_t infllmv2_workspace_size(const infllmv2_params* p, int32_t n_q, int32_t op);

/*
 * Stage 1: kc[b, h, :, j, :] = split(Mean(k_cache[b, h, j s : j s + p, :])) for
 * complete kernels j in [kernel_begin, kernel_end) of each sequence.
 * [InfLLM v2 > Semantic kernels for block relevance scoring, eqs. S_j, r_kernel]
 *   kernel_begin >= 0 : absolute first kernel;  < 0 : n_c(L_b) + kernel_begin
 *                       (so -1 recomputes only the newest complete kernel).
 *   kernel_end   >= 0 : absolute end (clipped to n_c(L_b));  < 0 : n_c(L_b).
 * Kernels outside the range are left untouched.  The mean is an fp32 sum of
 * the 32 bf16 keys times 1/32.
 */
int infllmv2_compress_keys(const infllmv2_params* p, const void* k_cache, const int32_t* kv_lens,
                           int32_t kernel_begin, int32_t kernel_end, void* kc, void* stream);

/*
 * Stage 2: choose the KV blocks of every (b, h_kv, t).
 *   z[h, j]  = score_scale * q_h . Mean_j            for kernels j visible to i
 *   g[j]     = (1/G) sum_h softmax_j(z[h, :])         (exact two-pass LSE)
 *   r[blk]   = max of g over visible kernels meeting the block, -inf if none
 *   selected = forced blocks (first n_init, the n_local ending at floor(i/m))
 *              + the best other finite-score blocks ordered by (r desc, index asc):
 *              topk - |forced| of them if topk_includes_forced, else topk.
 * block_scores (nullable) receives r as fp32 [B, Hkv, n_q, n_b(max_kv_len)]
 * (-inf past floor(i/m)).  n_q >= 1; workspace from
 * infllmv2_workspace_size(p, n_q, INFLLMV2_OP_SELECT).  For n_q > 16 the
 * selection keeps 8 tokens' block scores on chip up to max_kv_len 327360
 * (no workspace); above that they take one slot per SM of the workspace
 * (SM identifiers x 8 x n_b(max_kv_len) x 4 bytes), up to about 680K tokens
 * (INFLLMV2_UNSUPPORTED above).  The number of SM identifiers is read from
 * the device once, by a small synchronous query the first time it is
 * needed: make that first call (or the workspace-size query) outside
 * stream capture.
 */
int infllmv2_select_blocks(const infllmv2_params* p, const void* q, int32_t n_q, const void* kc,
                           const int32_t* kv_lens, int32_t* block_idx, int32_t* n_selected,
                           float* block_scores, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * infllmv2_select_blocks without a caller workspace.  The MiniCPM4 pages have
 * no counterpart of this entry point; it exists for embedders that cannot
 * hand the library device scratch at the call site: inference engines whose
 * device memory is laid out once at start-up, and plain C hosts that have no
 * device allocator of their own.
 *   Same arguments and result as infllmv2_select_blocks, minus the
 *   workspace.  Scratch comes from a fixed 8 MiB array inside the library
 *   (held by every device that loads it until the process exits); a
 *   selection whose scratch (infllmv2_workspace_size(p, n_q,
 *   INFLLMV2_OP_SELECT)) exceeds 8 MiB returns INFLLMV2_WORKSPACE_TOO_SMALL
 *   and launches nothing.  It allocates and frees nothing.
 *   The first call on a device looks up that device's address of the array
 *   (once); make that first call before any stream capture.  Every call
 *   shares the one array: calls whose work overlaps on the GPU (different
 *   streams, no ordering) race.  Nothing in the array has to start at zero;
 *   each call writes what it reads first.
 */
int infllmv2_select_blocks_static(const infllmv2_params* p, const void* q, int32_t n_q, const void* kc,
                                  const int32_t* kv_lens, int32_t* block_idx, int32_t* n_selected,
                                  float* block_scores, void* stream);

/*
 * Coarse-grained LSE approximation [InfLLM v2 > Efficient LSE approximation]
 * (off the default path; the exact LSE is the reference selection).
 *
 * infllmv2_coarse_means: kcc[b, h, 0 / 1, j, :] = hi / lo bf16 planes of the
 * mean of keys [j coarse, (j + 1) coarse) for every complete window of
 * sequence b (j < kv_lens[b] / coarse); kcc is bf16
 * [batch, n_kv_heads, 2, max_kv_len / coarse, d].  `coarse` is a multiple of
 * 16 in [32, 4096].
 *
 * infllmv2_select_blocks_coarse_lse: infllmv2_select_blocks for the prefill
 * path (n_q > 16) with each head's kernel-softmax normaliser taken over the
 * visible coarse windows (all keys <= i) instead of the fine kernels; a query
 * with no complete window keeps the exact LSE.  This cuts the first pass over
 * the kernel means by coarse / kernel_stride.  The decode path (n_q <= 16)
 * already computes the exact LSE without a second pass over memory, so it
 * has no coarse form (n_q <= 16 returns INFLLMV2_UNSUPPORTED).  Needs no
 * workspace; max_kv_len up to 327360 (the block scores stay on chip).
 */
int infllmv2_coarse_means(const infllmv2_params* p, const void* k_cache, const int32_t* kv_lens, int32_t coarse,
                          void* kcc, void* stream);
int infllmv2_select_blocks_coarse_lse(const infllmv2_params* p, const void* q, int32_t n_q, const void* kc,
                                      int32_t coarse, const void* kcc, const int32_t* kv_lens,
                                      int32_t* block_idx, int32_t* n_selected, float* block_scores,
                                      void* stream);

/*
 * Stage 3, few queries per sequence (decode n_q = 1, speculative verification
 * n_q <= 16): the selected blocks of each (b, h_kv, t) are dealt to the CTAs
 * of a thread-block cluster; each CTA computes an online-softmax partial and
 * the partials are merged through distributed shared memory.  out/lse as
 * documented above (lse nullable).  Only the first n_selected[b, h, t]
 * entries of block_idx are read; each must lie in [0, floor(i/m)] (entries
 * outside are skipped).  Needs no workspace (infllmv2_workspace_size
 * returns 0; workspace may be NULL).
 */
int infllmv2_sparse_attn_decode(const infllmv2_params* p, const void* q, int32_t n_q,
                                const void* k_cache, const void* v_cache, const int32_t* kv_lens,
                                const int32_t* block_idx, const int32_t* n_selected, void* out,
                                float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Stage 3, many queries per sequence (chunked or full causal prefill): same
 * arguments and result as the decode entry point, any n_q up to max_kv_len.
 */
int infllmv2_sparse_attn_prefill(const infllmv2_params* p, const void* q, int32_t n_q,
                                 const void* k_cache, const void* v_cache, const int32_t* kv_lens,
                                 const int32_t* block_idx, const int32_t* n_selected, void* out,
                                 float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Cache append of a decode step: k_new / v_new (bf16 [batch, n_kv_heads, n_q,
 * d], the keys and values of each sequence's n_q newest tokens) are written
 * to cache rows kv_lens[b] - n_q .. kv_lens[b] - 1 of (b, h), so that kv_lens
 * already counts them [InfLLM v2 > Block-level key-value partitioning: the
 * cache grows by the decoded tokens].  A sequence whose kv_lens[b] lies
 * outside [n_q, max_kv_len] is left untouched and sets
 * INFLLMV2_DEVICE_BAD_KV_LEN.  q_src / q_dst (both NULL, or both given):
 * also copy the step's queries, bf16 [batch, n_q, Hq, d], from q_src to q_dst.
 * k_new, v_new and q_src are read with ordinary loads, so they may be
 * page-locked host memory mapped for the device: a decode step whose inputs
 * sit in host memory then needs no separate copy.  The launch may start
 * while the previous kernel of the stream drains; it writes only after that
 * kernel has finished, and infllmv2_decode_step on the same stream reads
 * what it wrote.
 */
int infllmv2_append_kv(const infllmv2_params* p, int32_t n_q, const void* k_new, const void* v_new,
                       const int32_t* kv_lens, void* k_cache, void* v_cache, const void* q_src, void* q_dst,
                       void* stream);

/*
 * One whole decode step: stages 1-3 for the newest n_q tokens of each
 * sequence, whose keys and values the caller has already written to the
 * caches (kv_lens counts them) [InfLLM v2 > Semantic kernels, eq. S_j;
 * > Top-K implementation and the LSE bottleneck; > Block-level key-value
 * partitioning; > Complexity analysis, stage 2].
 *   kc      in/out: every kernel mean that ends before the step's tokens must
 *           be present; the kernels that end inside them (for n_q = 1: the
 *           newest complete kernel n_c(L) - 1) are recomputed from k_cache
 *           and written back.
 *   block_idx, n_selected, out, lse: as from infllmv2_select_blocks followed
 *           by infllmv2_sparse_attn_decode (lse nullable).  out and lse are
 *           written with ordinary stores, so they may also be page-locked host
 *           memory mapped for the device (e.g. from cudaHostAlloc on a system
 *           with unified addressing): the result then reaches the host without
 *           a separate copy.
 *   n_q in [1, 16].  With n_q = 1 the step is one launch of a thread-block
 *   cluster of C CTAs per (b, h_kv), one CTA per SM, that keeps every
 *   intermediate on chip and needs no workspace.  C (at most 16) is chosen
 *   for the device and batch so that all batch * n_kv_heads clusters are
 *   resident at once; the form applies while the cache holds at most
 *   256 C blocks of 64 tokens and at most 4096 blocks (262144 tokens).
 *   Otherwise the step enqueues the three stages in order.  Workspace:
 *   infllmv2_workspace_size(p, n_q, INFLLMV2_OP_DECODE_STEP) bytes (0 for
 *   the single-launch form; workspace may then be NULL).
 */
int infllmv2_decode_step(const infllmv2_params* p, const void* q, int32_t n_q, const void* k_cache,
                         const void* v_cache, const int32_t* kv_lens, void* kc, int32_t* block_idx,
                         int32_t* n_selected, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * infllmv2_append_kv followed by infllmv2_decode_step for one new token per
 * sequence (n_q = 1), as a single launch of the decode step's cluster form
 * [InfLLM v2 > Block-level key-value partitioning: the cache grows by the
 * decoded token; the step's stages as for infllmv2_decode_step].
 *   q       bf16 [batch, 1, Hq, d]: the token's queries.
 *   k_new, v_new  bf16 [batch, n_kv_heads, 1, d]: its key and value, written
 *           to cache row kv_lens[b] - 1 of k_cache / v_cache (kv_lens
 *           already counts the token); the step reads the key from k_new
 *           where it needs it before the store is visible.
 *   q, k_new and v_new are read with ordinary loads and out / lse written
 *   with ordinary stores, so any of them may be page-locked host memory mapped
 *   for the device: a step whose inputs and result live in host memory is one
 *   launch and no copy.  kc, block_idx, n_selected, out, lse: as for
 *   infllmv2_decode_step.  No workspace.
 * INFLLMV2_UNSUPPORTED for n_q != 1 or a shape outside the single-launch
 * form (see infllmv2_decode_step): call infllmv2_append_kv and
 * infllmv2_decode_step there.  A sequence whose kv_lens[b] lies outside
 * [1, max_kv_len] is left untouched (no row written, out zero, block_idx
 * -1) and sets INFLLMV2_DEVICE_BAD_KV_LEN.
 */
int infllmv2_append_decode_step(const infllmv2_params* p, const void* q, int32_t n_q, const void* k_new,
                                const void* v_new, void* k_cache, void* v_cache, const int32_t* kv_lens, void* kc,
                                int32_t* block_idx, int32_t* n_selected, void* out, float* lse, void* stream);

/*
 * Backward of stage 3 with the selection held fixed [InfLLM v2 >
 * Training-time considerations: top-k passes no gradient, the keys learn
 * through the gradient of the sparse attention]: for an upstream gradient
 * dout of `out`,
 *     P = exp(attn_scale q.k - lse) over each query's attended keys,
 *     D = rowsum(dout * out),  dS = P * (dout . v - D),
 *     dq = attn_scale sum_k dS k,  dk = attn_scale sum_q dS q,  dv = sum_q P dout.
 *   q, k_cache, v_cache, kv_lens, block_idx, n_selected: as given to the
 *           forward call; out (bf16) and lse (fp32, required) are its results.
 *   dout    bf16 [batch, n_q, Hq, d].
 *   dq      fp32 [batch, n_q, Hq, d], every row written.
 *   dk, dv  fp32 [batch, n_kv_heads, max_kv_len, d], every row written: keys
 *           no query attends get 0 (the call zeroes both, then adds the
 *           contributions of all queries of all heads of the group).
 * The contributions to one key row are added in an order that depends on
 * scheduling, so dk and dv may differ in the last bits from run to run.
 * Workspace: infllmv2_workspace_size(p, n_q, INFLLMV2_OP_BACKWARD) bytes
 * (an inverse block -> query index, D, work lists).
 */
int infllmv2_sparse_attn_backward(const infllmv2_params* p, const void* q, int32_t n_q, const void* k_cache,
                                  const void* v_cache, const int32_t* kv_lens, const int32_t* block_idx,
                                  const int32_t* n_selected, const void* out, const float* lse, const void* dout,
                                  float* dq, float* dk, float* dv, void* workspace, size_t workspace_bytes,
                                  void* stream);

/*
 * ---------------------------------------------------------------- pages ----
 *
 * A paged cache: one pool of pages of `page_size` token slots, shared by all
 * sequences.  Slot s of sequence b is row s % page_size of page
 * page_table[b][s / page_size]; page_table is int32 [batch, max_pages], and
 * only the entries that cover slots [0, kv_lens[b]) are read.  kv_lens is
 * int32 [batch], each in [0, max_pages * page_size]; a length outside sets
 * INFLLMV2_DEVICE_BAD_KV_LEN and counts as 0.  An entry in use outside
 * [0, num_pages) sets INFLLMV2_DEVICE_BAD_PAGE, and its page is not touched.
 *
 * k_pages and v_pages hold the row of (page, kv head, slot) at
 * page * strides[0] + head * strides[1] + slot * strides[2], in elements, the
 * head_dim values of a row consecutive: head-major and token-major storage
 * and a buffer that holds keys and values side by side are all described so.
 * weights and positions (both may be NULL) are contiguous [num_pages,
 * n_kv_heads, page_size]: per slot the attention weight it has received so
 * far, and the token's position in its sequence.  Eviction makes them
 * differ: a sequence that has seen seq_lens[b] tokens may hold kv_lens[b] of
 * them.  seq_lens (int32 [batch]) may be NULL: nothing was ever evicted.
 *
 * Supported: bf16 and fp16, head_dim 64 and 128, page_size a multiple of 16,
 * up to 4096 sequences and 2^30 slots each, fewer than 2^31 slots in the pool,
 * strides that are multiples of 8 elements, pointers 16-byte aligned.
 *
 * The conventions above hold: device pointers, work enqueued on `stream`,
 * no allocation, no synchronisation, bounded waits.  A workspace is written
 * before it is read in every call: calls that may overlap on the GPU, graphs
 * captured with it among them, need workspaces of their own; one stream's
 * calls can share one.
 */
#define INFLLMV2_BF16 0
#define INFLLMV2_FP16 1

typedef struct infllmv2_paged_cache {
  int32_t dtype;         /* INFLLMV2_BF16 or INFLLMV2_FP16: the pages, q, out and new rows */
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t page_size;     /* token slots of a page */
  int32_t num_pages;     /* pages of the pool */
  int32_t reserved;      /* 0 */
  int64_t k_strides[3];  /* elements between pages, KV heads and slots of k_pages */
  int64_t v_strides[3];
  void* k_pages;
  void* v_pages;
  float* weights;
  int32_t* positions;
} infllmv2_paged_cache;

/* Bytes of workspace of `op` (INFLLMV2_OP_PAGED_DECODE, with group_size query
 * heads per KV head; INFLLMV2_OP_PAGED_EVICT, which ignores group_size).  A
 * cache with weights needs room for every score of a decode: batch *
 * n_kv_heads * group_size * max_pages * page_size floats.  0 on invalid
 * arguments. */
size_t infllmv2_paged_workspace_size(const infllmv2_paged_cache* cache, int32_t batch, int32_t max_pages,
                                     int32_t group_size, int32_t op);

/*
 * Write new tokens into the pages: token t < n_new[b] of sequence b goes to
 * slot kv_lens[b] - n_new[b] + t (kv_lens already counts the new tokens); its
 * weight becomes 0 and its position seq_lens[b] - n_new[b] + t (seq_lens
 * counts them too; NULL: kv_lens).
 *   k_new, v_new  [batch, n_kv_heads, n_q, head_dim]; new_strides (host
 *           memory, NULL for contiguous): the elements between sequences,
 *           heads and tokens of k_new, then of v_new.  Read with ordinary
 *           loads: they may be page-locked host memory mapped for the device.
 *   n_new   int32 [batch], each in [0, n_q], or NULL: n_q for all.
 * A sequence with n_new[b] outside [0, n_q] or kv_lens[b] outside
 * [n_new[b], max_pages * page_size] is left untouched and sets
 * INFLLMV2_DEVICE_BAD_KV_LEN; a token whose page is bad is not written.  The
 * slots written must be pairwise different, and k_new and v_new apart from them.
 */
int infllmv2_paged_append_kv(const infllmv2_paged_cache* cache, int32_t batch, int32_t max_pages, int32_t n_q,
                             const void* k_new, const void* v_new, const int64_t* new_strides,
                             const int32_t* page_table, const int32_t* kv_lens, const int32_t* n_new,
                             const int32_t* seq_lens, void* stream);

/*
 * Attention of one new token per sequence over all its slots:
 *     z[h, s] = attn_scale q_h . k_s,  P = softmax_s(z),  out_h = sum_s P v_s,
 *     lse_h = ln sum_s exp(z[h, s]).
 *   q, out  [batch, 1, n_kv_heads * group_size, head_dim] in the cache's type
 *           (heads h*G .. h*G+G-1 share KV head h); group_size in [1, 32].
 *   lse     fp32 [batch, 1, n_kv_heads * group_size], may be NULL.
 *   accumulate = 1: weights[slot] += sum of P over the group's heads, for
 *           every slot attended (needs the cache's weights).  Sequences may
 *           share pages (a common prefix); the weights of a shared slot are
 *           then summed in an order that depends on scheduling.
 * A sequence with kv_lens[b] = 0 gets out = 0 and lse = -inf.  Slots of bad
 * pages, and whatever rows past kv_lens[b] hold, take no part.  Infinities and
 * NaN in attended rows act as in the formula, in their own sequence and KV head
 * only, but for an infinity in a value row whose probability is below 2^-28
 * (fp16; bf16: 2^-110) of the largest: it may give NaN instead.
 *   attn_scale  > 0, and finite in fp32 also times log2(e).
 * Workspace: infllmv2_paged_workspace_size(.., INFLLMV2_OP_PAGED_DECODE).
 */
int infllmv2_paged_attn_decode(const infllmv2_paged_cache* cache, int32_t batch, int32_t max_pages,
                               int32_t group_size, const void* q, const int32_t* page_table, const int32_t* kv_lens,
                               float attn_scale, int32_t accumulate, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Evict from every (sequence, KV head) that holds more than `budget` slots
 * all but `budget`: kept are first the slots whose position is < n_init or
 * >= seq_lens[b] - n_local, then those with the largest weights (equal
 * weights: the lowest slots; a NaN weight counts as less than any number).
 * n_init + n_local <= budget.  In place: kept slots at or past `budget` move,
 * in ascending order, into the evicted slots below it, with their weights and
 * positions, so a cache's slots are no longer in order of position; slots at
 * or past `budget` are left as they were, and the pages past
 * ceil(budget / page_size) are free.  Each KV head keeps slots of its own.
 *   new_lens  int32 [batch]: min(kv_lens[b], budget); kv_lens itself, or an
 *           array apart from kv_lens and seq_lens (with which a page table of at
 *           most 128 slots past the budget takes one launch instead of two).
 * A sequence with a bad page among its slots is left as it is (new_lens =
 * kv_lens[b]).  The pages in use must be pairwise different: a page that
 * sequences share must not be evicted from.  max_pages * page_size <= 524288.
 * Workspace: infllmv2_paged_workspace_size(.., INFLLMV2_OP_PAGED_EVICT).
 */
int infllmv2_paged_evict(const infllmv2_paged_cache* cache, int32_t batch, int32_t max_pages,
                         const int32_t* page_table, const int32_t* kv_lens, int32_t budget, int32_t n_init,
                         int32_t n_local, const int32_t* seq_lens, int32_t* new_lens, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * The page tables and the token maps of one step, from its requests' lengths.
 * Sequence b holds kv_lens[b] tokens and gets n_new[b] more (0: none).  It owns
 * the first held[b] entries of its row of page_table, and needs
 * ceil((kv_lens[b] + n_new[b]) / page_size); the call takes the pages it lacks
 * from the free pages and gives back those it no longer needs: all of them for
 * kv_lens[b] = n_new[b] = 0 (a finished sequence), the ones past the budget after
 * an eviction.  No page may be owned twice.
 *   page_table  int32 [batch, max_pages], in/out; entries past held[b] are left
 *           as they were.
 *   held    int32 [batch], in/out.
 *   free_pages, n_free  int32 [num_pages] and [1], in/out: a stack of
 *           n_free[0] free pages.  Pages are taken from its top, sequence by
 *           sequence; once it is empty, of those given back, in order; the rest
 *           of those go onto it.  Entries from n_free[0] on are left as they were.
 *   seq_lens  int32 [batch], the tokens each sequence has seen, without the new
 *           ones, or NULL: kv_lens.
 *   new_lens  int32 [batch]: kv_lens + n_new; may be kv_lens or n_new.
 *   starts  int32 [batch + 1]: sequence b's new tokens are tokens starts[b] ..
 *           starts[b + 1] - 1 of the step.
 *   slots, positions  int32 [max_tokens], each may be NULL: of every token of the
 *           step its slot in the pool, page * page_size + row, and its position,
 *           seq_lens[b] + t; past the last token -1 and 0.  max_tokens counts where one of
 *           the two is there.
 *   missing int32 [1]: 0, or the number of free pages that lack, or -1: a length,
 *           held[b] or n_free is out of range (a row has max_pages entries; the
 *           pages given back and the free ones are at most num_pages), or
 *           the step has more than max_tokens tokens; then also
 *           INFLLMV2_DEVICE_BAD_KV_LEN.  Where it is not 0 nothing is taken or
 *           given back, new_lens is kv_lens, every start 0 and every slot -1: the
 *           step is empty.
 * Page sizes, batch and pool as for the paged cache (any page size from 1 on).
 */
typedef struct infllmv2_reserve_args {
  int32_t page_size, num_pages, batch, max_pages, max_tokens;
  int32_t reserved;        /* 0 */
  int32_t* page_table;
  int32_t* held;
  int32_t* free_pages;
  int32_t* n_free;
  int32_t* missing;
  const int32_t* kv_lens;
  const int32_t* n_new;
  const int32_t* seq_lens;
  int32_t* new_lens;
  int32_t* starts;
  int32_t* slots;
  int32_t* positions;
} infllmv2_reserve_args;

int infllmv2_paged_reserve(const infllmv2_reserve_args* args, void* stream);

/*
 * Write the tokens of a packed step into the pages: row t of k_new and v_new
 * [tokens, n_kv_heads, head_dim] goes to slot slots[t] (page * page_size + row;
 * below 0: nowhere); the slot's weight becomes 0 and its position positions[t].
 *   strides (host memory, NULL for contiguous): the elements between tokens and
 *           heads of k_new, then of v_new.  Read with ordinary loads: they may be
 *           page-locked host memory mapped for the device.
 *   positions  int32 [tokens]; NULL only where the cache has none.
 *   tokens  1 .. 2^30.
 * A slot past the pool is not written and sets INFLLMV2_DEVICE_BAD_PAGE.  The
 * slots written must be pairwise different, and k_new and v_new apart from them.
 */
int infllmv2_paged_append_packed(const infllmv2_paged_cache* cache, int32_t tokens, const void* k_new,
                                 const void* v_new, const int64_t* strides, const int32_t* slots,
                                 const int32_t* positions, void* stream);

/*
 * --------------------------------------------------------- packed steps ----
 *
 * The tokens of several sequences one after the other: starts int32 [batch + 1],
 * sequence b's are rows starts[b] .. starts[b + 1] - 1 of tensors [tokens, heads,
 * head_dim] with any strides between tokens and heads (multiples of 16 bytes; the
 * values of a head are consecutive), as views of one projection's output have.
 * Rows of no sequence are neither read into a result nor written.
 */

/*
 * The frequencies of rotary positions: pair i of rotary_dim / 2 turns by
 * base^(-2 i / rotary_dim) radians per position, scaled for contexts longer than
 * the trained original_len by
 *   INFLLMV2_ROTARY_PLAIN    nothing;
 *   INFLLMV2_ROTARY_LINEAR   all divided by factor;
 *   INFLLMV2_ROTARY_BASE     base times factor^(d / (d - 2)), so that the slowest
 *           pair is divided by factor and the fastest stays (d = rotary_dim > 2);
 *   INFLLMV2_ROTARY_PARTS    pairs that turn more than fast_turns times in
 *           original_len positions stay, those that turn less than slow_turns times
 *           are divided by factor, a linear ramp over the pairs' index between
 *           (its ends rounded outwards); values times 0.1 ln(factor) + 1
 *           (Peng et al. 2023, "YaRN");
 *   INFLLMV2_ROTARY_FACTORS  pair i divided by factors[i]; values times
 *           sqrt(1 + ln(factor) / ln(original_len)) (Ding et al. 2024, "LongRoPE").
 * Host code: turns and scale are host memory.  turns[i] is 2^64 times the turns
 * per position, scale what infllmv2_rotary multiplies the values by.
 */
#define INFLLMV2_ROTARY_PLAIN 0
#define INFLLMV2_ROTARY_LINEAR 1
#define INFLLMV2_ROTARY_BASE 2
#define INFLLMV2_ROTARY_PARTS 3
#define INFLLMV2_ROTARY_FACTORS 4

typedef struct infllmv2_rotary_config {
  int32_t rotary_dim;    /* even, 2 .. 512 */
  int32_t scaling;       /* INFLLMV2_ROTARY_* */
  double base;           /* > 1 */
  double factor;         /* >= 1 */
  int32_t original_len;  /* > 1; read by PARTS and FACTORS */
  int32_t reserved;      /* 0 */
  double fast_turns, slow_turns;   /* PARTS: fast > slow > 0 (32 and 1) */
  const double* factors; /* FACTORS: rotary_dim / 2 divisors, >= 1 */
} infllmv2_rotary_config;

int infllmv2_rotary_frequencies(const infllmv2_rotary_config* config, uint64_t* turns, float* scale);

/*
 * Rotary positions of a packed step's queries and keys: of every head the first
 * rotary_dim values are pairs (x, y), value i with i + rotary_dim / 2, or
 * (interleaved) 2 i with 2 i + 1.  Pair i of token t becomes
 *     scale (x cos a - y sin a, x sin a + y cos a),  a = 2 pi positions[t] turns[i] / 2^64,
 * with transpose = 1 the same with -a: the gradient of the inputs from that of
 * the outputs.  The other head_dim - rotary_dim values are copied.
 *   q, k    INFLLMV2_BF16, INFLLMV2_FP16 or INFLLMV2_FP32 (dtype); no k where
 *           k_heads is 0.  Strides in elements between tokens and heads.  q_out may be
 *           q, with the same strides; otherwise the two must not overlap; k likewise.
 *           q_out must be apart from k and k_out, and k_out from q.
 *   tokens  1 .. 2^30.
 *   positions  int32 [tokens], any value.
 *   turns   device memory, [rotary_dim / 2], from infllmv2_rotary_frequencies.
 * head_dim and rotary_dim: multiples of 16, rotary_dim <= head_dim <= 512.
 * Angles are exact to 2^-27 turn whatever the position.
 */
#define INFLLMV2_FP32 2

typedef struct infllmv2_rotary_args {
  int32_t dtype, tokens, head_dim, rotary_dim, q_heads, k_heads, interleaved, transpose;
  float scale;
  int32_t reserved;        /* 0 */
  const int32_t* positions;
  const uint64_t* turns;
  const void* q;           /* [tokens, q_heads, head_dim] */
  void* q_out;
  const void* k;           /* [tokens, k_heads, head_dim] */
  void* k_out;
  int64_t q_strides[2], q_out_strides[2], k_strides[2], k_out_strides[2];
} infllmv2_rotary_args;

int infllmv2_rotary(const infllmv2_rotary_args* args, void* stream);

/*
 * Causal attention over packed sequences with grouped heads.  Sequence b has the
 * query rows q_starts[b] .. q_starts[b + 1] - 1 and the key rows k_starts[b] ..
 * k_starts[b + 1] - 1; the last of each are the same token, so query i of n_q
 * attends the keys j <= n_k - n_q + i of n_k (more keys than queries: tokens
 * of earlier steps come first).  Of its n_kv_heads * group_size heads the ones
 * h * group_size .. (h + 1) * group_size - 1 share KV head h:
 *     z_j = scale q . k_j,  P = softmax_j(z),  out = sum_j P_j v_j,
 *     lse = ln sum_j exp(z_j).
 * A row that attends no key (n_k < n_q) gets out = 0 and lse = -inf.  Rows of other
 * sequences and of none take no part, whatever they hold.  Within a sequence,
 * infinities and NaN act as in the formula, and what a query does not attend
 * does not reach it.
 *   dtype   INFLLMV2_BF16 or INFLLMV2_FP16: q, k, v, out and the gradients.
 *   head_dim 64 or 128; group_size 1 .. 32; up to 4096 sequences; fewer than
 *           2^31 / (n_kv_heads * group_size) tokens, at least one of each.
 *   strides elements between tokens and heads, multiples of 8; rows of one tensor
 *           must not overlap.  Pointers 16-byte aligned.
 *   q_starts, k_starts  int32 [batch + 1], not descending, within [0, q_tokens] and
 *           [0, k_tokens]; k_starts NULL: q_starts.  A sequence whose starts are out of
 *           range or descend sets INFLLMV2_DEVICE_BAD_KV_LEN and counts as empty.
 *   scale   > 0, and finite in fp32 also times log2(e).
 * lse is contiguous fp32 [q_tokens, heads] and may be NULL in the forward call.
 * Outputs must not overlap inputs or each other.
 */
typedef struct infllmv2_packed_attn_args {
  int32_t dtype, batch, n_kv_heads, group_size, head_dim, q_tokens, k_tokens;
  float scale;
  const void* q;   /* [q_tokens, n_kv_heads * group_size, head_dim] */
  const void* k;   /* [k_tokens, n_kv_heads, head_dim] */
  const void* v;
  int64_t q_strides[2], k_strides[2], v_strides[2];
  const int32_t* q_starts;
  const int32_t* k_starts;
} infllmv2_packed_attn_args;

int infllmv2_packed_attn(const infllmv2_packed_attn_args* args, void* out, const int64_t* out_strides, float* lse,
                         void* stream);

/*
 * Its gradient: for the upstream gradient dout of out,
 *     P = exp(z - lse),  D = rowsum(dout * out),  dS = P * (dout . v - D),
 *     dq = scale sum_j dS k_j,  dk_j = scale sum dS q,  dv_j = sum P dout,
 * the sums for a key over all queries of all heads of its group that attend it.
 * Every row of a sequence is written, in an order of sums that does not change from
 * run to run; keys that no query attends get 0.
 *   out, lse  as the forward call on the same arguments wrote them.
 *   D is summed from the scores where a row attends up to 1024 keys.  Longer rows take it
 *           from out and correct it by the scores; a tile of rows whose dq the rounding of out has moved more than
 *           the 16-bit rounding of dS may is done once more, which takes its time once more.
 *   grad_strides (host memory): between tokens and heads of out, dout, dq, dk, dv.
 *   P and dS enter the sums in the type of q, in fp16 times powers of two (of a row, and of the
 *           rows that share keys), so that neither small nor large upstream gradients leave
 *           its range.  A non-finite dout or q row reaches every
 *           key row of its own sequence and KV head, a non-finite key every query row.
 * Workspace: infllmv2_packed_workspace_size(args) bytes (D and lse of each row).  Written before
 * it is read in every call: calls that may overlap on the GPU need their own.
 */
size_t infllmv2_packed_workspace_size(const infllmv2_packed_attn_args* args);
int infllmv2_packed_attn_backward(const infllmv2_packed_attn_args* args, const void* out, const float* lse,
                                  const void* dout, void* dq, void* dk, void* dv, const int64_t* grad_strides,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * The checked build.  The library can also be built with INFLLMV2_CHECKED
 * (libinfllmv2_checked.so), in place of a memory checker.  It verifies
 * every index that comes from the caller before use (each counted
 * block_idx entry within [0, floor(i/m)], each n_selected within
 * [0, k_max]) and the start of every K/V tile formed from one; a violation
 * sets INFLLMV2_DEVICE_BOUNDS and the access is skipped (the product build
 * skips the same accesses without reporting them).  Its bounded waits give
 * up after 2^16 polls instead of 2^22.
 *
 * infllmv2_is_checked_build: 1 in the checked build, 0 otherwise.
 *
 * infllmv2_test_hooks: fault injection for the library's own tests, checked
 * build only (the product build returns INFLLMV2_UNSUPPORTED and changes
 * nothing).  flags = 1: in every later infllmv2_decode_step of the
 * single-launch form, one warp per CTA withholds the release of its first
 * ring stage, so a bounded wait expires: the call still returns, sets
 * INFLLMV2_DEVICE_TIMEOUT and leaves no copy in flight.  flags = 0 turns it
 * off.  Process-wide; not for concurrent use with other calls.
 */
int infllmv2_is_checked_build(void);
int infllmv2_test_hooks(uint32_t flags);

/* Human-readable name of an INFLLMV2_* return code. */
const char* infllmv2_status_string(int status);

/* Message of the last failed call on this thread ("" if none). */
const char* infllmv2_last_error(void);

/* Read (and if `clear` is nonzero, reset) the device status word of the
 * current device.  Synchronises the device; not for the hot path.
 * The library looks up the device addresses of its status word and of the
 * built-in selection scratch once per device and keeps them: it assumes the
 * device's primary context (the one the CUDA runtime uses) for the life of
 * the process, and does not support a cudaDeviceReset or a separately
 * created driver context on that device after its first call there. */
int infllmv2_get_device_status(uint32_t* status_out, int clear);

#ifdef __cplusplus
}
#endif

#endif /* INFLLMV2_H */
