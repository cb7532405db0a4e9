/*
 * bsa.h -- C ABI of libbsa.so: content-dependent block-sparse attention on
 * one NVIDIA GB300 (sm_103a): the forward, its backward, rotary positions,
 * a paged cache in 16 or 8 bits, decoding of single tokens over it, and
 * attention of new tokens to all of it, a window, or a tree.
 *
 * The method (page "sparse-attention-triton-bench", section "Two-stage
 * block indexer"):
 *   Stage 1  mean-pool every B-token key block into a representative Kbar_b,
 *            score every query against every block (q . Kbar_b) and keep the
 *            k best blocks per query, ties to the lower block index;
 *   Stage 2  softmax attention, scale 1/sqrt(d) by default, over only the
 *            k*B tokens of the selected blocks, accumulated with an online
 *            softmax state (running max m, running sum l, accumulator acc;
 *            same page, section "The Triton kernel").
 * The fine stage also runs over static block lists (page "yayme/CUDA-kernel"
 * README: local window |i-j| <= w plus global stride j % s == 0, walked as a
 * precomputed active-tile list; page "Block-Sparse & Linear Attention
 * Kernels", section 2: block-sparse loop and the causal sliding window).
 *
 * Conventions shared by every entry point
 *   - Tensors Q, K, V, O are [bh][n][d] row-major (d fastest), contiguous,
 *     element type given by bsa_shape.dtype.  bh = batch * heads.
 *   - Every tensor pointer is a DEVICE pointer unless the parameter says
 *     host.  Device pointers must be 16-byte aligned (int32 arrays 4-byte);
 *     workspaces 256-byte.
 *   - The caller owns every buffer.  The library never allocates device
 *     memory and keeps no per-call state (handles -- graphs, page managers --
 *     hold host memory until destroyed); calls only enqueue work on `stream` (a
 *     cudaStream_t passed as void*, NULL = legacy default stream) and return
 *     at once.  Results are ready when the stream reaches that point.
 *   - Argument errors are detected on the host and returned synchronously;
 *     nothing is enqueued then.  bsa_last_error() gives a one-line reason.
 *   - Errors found by a kernel (a listed block index outside [0, nb), a
 *     bounded wait that ran out) never trap: the kernel skips the offending
 *     work, records the first such code in a device status word and
 *     returns.  bsa_get_device_status() reads and clears that word.
 *   - Supported: d in {64, 128}; key_block B in {16, 32, 64, 128};
 *     dtype bf16 everywhere, fp32 for the fine stage and the rotary
 *     positions.
 */
#ifndef BSA_H_
#define BSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BSA_OK = 0,
    BSA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, bad enum value      */
    BSA_ERR_UNSUPPORTED = 2,   /* valid request outside the supported set     */
    BSA_ERR_BAD_INDEX = 3,     /* (device) a listed block id outside [0, nb)  */
    BSA_ERR_WORKSPACE = 4,     /* workspace null or smaller than required;
                                  page pool, table or pair array too small    */
    BSA_ERR_CUDA = 5,          /* a CUDA runtime call failed                  */
    BSA_ERR_TIMEOUT = 6,       /* (device) a bounded barrier wait ran out     */
    BSA_ERR_ALIGNMENT = 7      /* pointer not 16-byte (workspace: 256) aligned */
} bsa_status;

typedef enum { BSA_BF16 = 0, BSA_FP32 = 1 } bsa_dtype;

/* Shape of Q, K, V and O: [bh][n][d], element type `dtype` (bsa_dtype). */
typedef struct {
    int64_t bh;
    int64_t n;
    int32_t d;
    int32_t dtype;
} bsa_shape;

typedef enum {
    BSA_MASK_NONE = 0,          /* every token of a listed block is attended   */
    BSA_MASK_LOCAL_GLOBAL = 1,  /* |i-j| <= window  or  j % stride == 0        */
    BSA_MASK_SLIDING = 2,       /* causal window: i - sliding < j <= i         */
    BSA_MASK_CAUSAL = 3         /* causal: j <= i                              */
} bsa_mask_kind;

/*
 * Token-level predicate applied inside the listed blocks (page
 * "yayme/CUDA-kernel" README, sparsity pattern; page "Block-Sparse & Linear
 * Attention Kernels", section 2, sliding window, and section 1, the causal
 * lower triangle).  LOCAL_GLOBAL: window < 0 disables the band, stride <= 0
 * disables the global columns.  SLIDING: sliding >= 1 is W, the number of
 * keys up to and including the query.  CAUSAL takes no parameter; with
 * per-query lists (q_group = 1) it is what a causal selection needs inside
 * the query's own block.
 */
typedef struct {
    int32_t kind;
    int32_t window;
    int32_t stride;
    int32_t sliding;
} bsa_mask;

/*
 * Layout of a block-index list.  The list is int32
 *   [per_head ? bh : 1][ceil(n / q_group)][max_blocks]:
 * row r serves queries [r*q_group, (r+1)*q_group); each row holds key-block
 * ids (block b = tokens [b*key_block, min(n, (b+1)*key_block))) in strictly
 * ascending order, padded with -1 at the tail only.
 *   dynamic lists (stage 2):  q_group = 1, max_blocks = k, per_head = 1;
 *   static lists:             q_group = the query-tile height, per_head = 0.
 */
typedef struct {
    int32_t q_group;
    int32_t key_block;
    int32_t max_blocks;
    int32_t per_head;
} bsa_list_desc;

/*
 * Stage 1, pooling (page "sparse-attention-triton-bench", Two-stage block
 * indexer, Stage 1: "mean-pooling the keys within" each block).
 *   k     [bh][n][d] bf16 keys (device).
 *   kbar  [bh][nb][d] fp32 output, nb = ceil(n / key_block) (device);
 *         kbar[h][b] = mean of the valid keys of block b (a ragged last
 *         block averages its n - b*key_block tokens).
 */
bsa_status bsa_pool_blocks(bsa_shape shape, const void *k, int32_t key_block,
                           float *kbar, void *stream);

/*
 * Stage 1 scoring + Stage 2 selection (same page and section: score every
 * query against every block representative, "take the top-k
 * highest-scoring blocks").  Scores are q . Kbar_b (unscaled: a positive
 * scale cannot change the ranking) and are never written to memory.
 *   q     [bh][n][d] bf16 queries (device).
 *   kbar  [bh][nb][d] fp32 block means, as written by bsa_pool_blocks.
 *   idx   [bh][n][topk] int32 output (device): the min(topk, nb) selected
 *         block ids of each query in ascending order, ties in score going to
 *         the lower block id; entries past nb are -1.
 *   ws    device workspace of bsa_coarse_topk_workspace_size() bytes.
 * topk in [1, 32].
 */
size_t bsa_coarse_topk_workspace_size(bsa_shape shape, int32_t key_block,
                                      int32_t topk);
bsa_status bsa_coarse_topk(bsa_shape shape, const void *q, const float *kbar,
                           int32_t key_block, int32_t topk, int32_t *idx,
                           void *ws, size_t ws_bytes, void *stream);

/*
 * Options of the selection (NULL = none, which is bsa_coarse_topk).
 *   head_topk    optional DEVICE int32 [bh]: the budget k_h of each
 *                (batch * head) row, in [0, topk] (page
 *                "sparse-attention-triton-bench", What's next: per-head
 *                sparsity budgets chosen at run time on the per-head stage-1
 *                scores).  Row h of idx then holds min(k_h, eligible) ids and
 *                -1 after them.  A value outside [0, topk] is clamped into it
 *                and reported as BSA_ERR_INVALID_ARG through
 *                bsa_get_device_status().  NULL: topk for every row.
 *   causal       nonzero: query i may select only blocks b <= i / key_block
 *                (blocks holding some key j <= i; page "Block-Sparse &
 *                Linear Attention Kernels", section 1, the causal pattern),
 *                and the fine stage of bsa_forward_ex attends only keys
 *                j <= i.
 *   local_block  nonzero: the query's own block i / key_block is always
 *                selected (when its budget is >= 1); the other k_h - 1 are
 *                the best-scoring eligible blocks except it.
 * Ties and output order as bsa_coarse_topk.
 */
typedef struct {
    const int32_t *head_topk;
    int32_t causal;
    int32_t local_block;
} bsa_select;

bsa_status bsa_coarse_topk_ex(bsa_shape shape, const void *q, const float *kbar,
                              int32_t key_block, int32_t topk,
                              const bsa_select *sel, int32_t *idx, void *ws,
                              size_t ws_bytes, void *stream);

/*
 * Stage 2, fine attention over a block list (page
 * "sparse-attention-triton-bench", Stage 2 and "The Triton kernel": dense
 * softmax attention over the listed blocks' tokens with an online-softmax
 * state; page "Block-Sparse & Linear Attention Kernels", section 2: skip
 * every unlisted block).
 *   q, k, v  [bh][n][d] of shape.dtype (bf16 or fp32), device.
 *   list     int32 block list laid out as `ld` says (device), or NULL for
 *            every block of the sequence.
 *   mask     token-level predicate inside listed blocks.
 *   scale    softmax scale; <= 0 selects 1/sqrt(d).
 *   out      [bh][n][d] of shape.dtype (device); a query whose list admits
 *            no key gets zeros.
 *   ws       device workspace of bsa_fine_attention_workspace_size() bytes.
 *            Per-query lists need it.  For static tile lists (and no list)
 *            of bf16 inputs on the tensor-core path it is optional: with it
 *            the kernel first takes each block's largest key norm and runs
 *            one pass with a per-row bound on the scores (the exact two-pass
 *            kernel redoes only the tiles the bound does not serve); without
 *            it (NULL) every tile runs two passes.  The results agree to
 *            rounding.
 * A listed id outside [0, nb) is skipped and reported as BSA_ERR_BAD_INDEX
 * through bsa_get_device_status().
 */
size_t bsa_fine_attention_workspace_size(bsa_shape shape, bsa_list_desc ld,
                                         bsa_mask mask);
bsa_status bsa_fine_attention(bsa_shape shape, const void *q, const void *k,
                              const void *v, const int32_t *list,
                              bsa_list_desc ld, bsa_mask mask, float scale,
                              void *out, void *ws, size_t ws_bytes,
                              void *stream);

/*
 * bsa_fine_attention that also returns each query's log2-sum-exp
 * lse_i = log2 sum_{j in T_i} 2^(s_ij * scale * log2 e), the softmax's
 * normaliser in base 2 ("The Triton kernel": the row statistics m and l of
 * the online softmax, lse = m + log2 l), for a backward pass to reuse
 * (bsa_fine_backward_lse).  A query whose list admits no key gets -inf.
 *   lse_out  [bh][n] fp32 (device), 4-byte aligned.
 * Only where bsa_fine_attention takes its block-major path: per-query lists
 * (q_group 1, per_head 1, max_blocks <= 32), bf16, d in {64, 128},
 * key_block 64, at most 16384 blocks, no mask or the causal one; other calls
 * return BSA_ERR_UNSUPPORTED.  Workspace and everything else as
 * bsa_fine_attention.
 */
bsa_status bsa_fine_attention_lse(bsa_shape shape, const void *q, const void *k,
                                  const void *v, const int32_t *list,
                                  bsa_list_desc ld, bsa_mask mask, float scale,
                                  void *out, float *lse_out, void *ws,
                                  size_t ws_bytes, void *stream);

/*
 * Backward pass of the fine stage (page "sparse-attention-triton-bench",
 * What's next: a backward pass through the sparse softmax-weighted sum over
 * the selected blocks).  The selection is a discrete choice and is held
 * fixed: the gradients flow through the fine stage only.  For query i with
 * token set T_i (its listed blocks' keys; only j <= i under
 * BSA_MASK_CAUSAL) and the output gradient dO:
 *   D_i = dO_i . O_i,  dS_ij = p_ij (dO_i . v_j - D_i),
 *   dQ_i = scale sum_j dS_ij k_j,  dK_j = scale sum_i dS_ij q_i,
 *   dV_j = sum_i p_ij dO_i.
 * The row statistics of the softmax are recomputed from q, k and the list.
 *   q, k, v   [bh][n][d] bf16 (device), as given to the forward.
 *   out       [bh][n][d] bf16: the forward's output O for this list.
 *   dout      [bh][n][d] bf16: dO.
 *   list, ld  per-query lists as the forward took them (q_group 1,
 *             per_head 1, max_blocks <= 64; ascending ids, -1 padding).
 *   mask      BSA_MASK_NONE or BSA_MASK_CAUSAL.
 *   scale     softmax scale; <= 0 selects 1/sqrt(d).
 *   dq, dk, dv  [bh][n][d] fp32 outputs (device); every element is written
 *             (keys no query listed get zeros).
 *   ws        device workspace of bsa_fine_backward_workspace_size() bytes.
 * d in {64, 128}, key_block * d <= 8192; bf16 only.  Listed ids outside
 * [0, nb) are skipped and
 * reported as BSA_ERR_BAD_INDEX through bsa_get_device_status().
 */
size_t bsa_fine_backward_workspace_size(bsa_shape shape, bsa_list_desc ld);
bsa_status bsa_fine_backward(bsa_shape shape, const void *q, const void *k,
                             const void *v, const void *out, const void *dout,
                             const int32_t *list, bsa_list_desc ld,
                             bsa_mask mask, float scale, float *dq, float *dk,
                             float *dv, void *ws, size_t ws_bytes,
                             void *stream);

/*
 * bsa_fine_backward given the forward's log2-sum-exp per query (as
 * bsa_fine_attention_lse writes it, for the same inputs, lists, mask and
 * scale), so that the softmax statistics are not recomputed: on the
 * tensor-core path (key_block 64, max_blocks <= 32) the call inverts the
 * lists and runs the gradient kernels only.  Other shapes recompute the
 * statistics as bsa_fine_backward does and ignore lse.
 *   lse  [bh][n] fp32 (device), 4-byte aligned; not modified.
 * Same workspace (bsa_fine_backward_workspace_size) and outputs as
 * bsa_fine_backward.
 */
bsa_status bsa_fine_backward_lse(bsa_shape shape, const void *q, const void *k,
                                 const void *v, const void *out, const void *dout,
                                 const int32_t *list, bsa_list_desc ld,
                                 bsa_mask mask, float scale, const float *lse,
                                 float *dq, float *dk, float *dv, void *ws,
                                 size_t ws_bytes, void *stream);

/*
 * The whole dynamic forward: pool -> score + top-k -> fine attention, all
 * enqueued on `stream` (page "sparse-attention-triton-bench", Two-stage
 * block indexer).  bf16 only, non-causal (bsa_forward_ex below takes the causal and
 * per-head options).
 *   idx_out  optional [bh][n][topk] int32 (device) receiving the selection;
 *            NULL keeps it in the workspace.
 *   ws       device workspace of bsa_forward_workspace_size() bytes.
 */
size_t bsa_forward_workspace_size(bsa_shape shape, int32_t key_block,
                                  int32_t topk);
bsa_status bsa_forward(bsa_shape shape, const void *q, const void *k,
                       const void *v, int32_t key_block, int32_t topk,
                       float scale, void *out, int32_t *idx_out, void *ws,
                       size_t ws_bytes, void *stream);

/*
 * bsa_forward with selection options (bsa_select above; NULL = none).  With
 * `causal` the fine stage attends, for query i, only the keys j <= i of its
 * selected blocks.  Same workspace as bsa_forward (its size does not depend
 * on the options); same errors.
 */
bsa_status bsa_forward_ex(bsa_shape shape, const void *q, const void *k,
                          const void *v, int32_t key_block, int32_t topk,
                          const bsa_select *sel, float scale, void *out,
                          int32_t *idx_out, void *ws, size_t ws_bytes,
                          void *stream);

/*
 * bsa_forward_ex that also writes each query's log2-sum-exp (as
 * bsa_fine_attention_lse defines it) for a backward pass over the same
 * selection (bsa_fine_backward_lse with idx_out as the list), so that a
 * training step computes the softmax statistics once.  The forward then
 * always runs as separate launches (the one-launch form for small problems
 * keeps no statistics).
 *   lse_out  [bh][n] fp32 (device), 4-byte aligned.
 * Only where the fine stage takes its block-major path (key_block 64, at most
 * 16384 blocks); other shapes return BSA_ERR_UNSUPPORTED.  Workspace and
 * everything else as bsa_forward_ex.
 */
bsa_status bsa_forward_lse(bsa_shape shape, const void *q, const void *k,
                           const void *v, int32_t key_block, int32_t topk,
                           const bsa_select *sel, float scale, void *out,
                           int32_t *idx_out, float *lse_out, void *ws,
                           size_t ws_bytes, void *stream);

/*
 * The whole forward as one CUDA graph (page "sparse-attention-triton-bench",
 * The Triton kernel: the forward as a few fused launches instead of the
 * hundreds of a Python loop; here every launch of bsa_forward_ex is captured
 * once and the caller replays them with one host call).
 *   bsa_forward_graph_create  captures bsa_forward_ex for these exact
 *       pointers and arguments (same validation and errors) on a private
 *       stream and instantiates it; *graph receives the handle (NULL on
 *       error).  Nothing runs at creation.
 *   bsa_graph_launch  enqueues one replay on `stream`: it reads whatever the
 *       captured q, k, v (and head_topk) buffers hold at that time and writes
 *       out (and idx_out); the workspace must stay allocated and unshared
 *       while replays can run.
 *   bsa_graph_destroy  releases the handle (NULL is a no-op); replays already
 *       enqueued complete.
 */
typedef struct bsa_graph_s *bsa_graph;
bsa_status bsa_forward_graph_create(bsa_shape shape, const void *q,
                                    const void *k, const void *v,
                                    int32_t key_block, int32_t topk,
                                    const bsa_select *sel, float scale,
                                    void *out, int32_t *idx_out, void *ws,
                                    size_t ws_bytes, bsa_graph *graph);
bsa_status bsa_graph_launch(bsa_graph graph, void *stream);
bsa_status bsa_graph_destroy(bsa_graph graph);

/*
 * bsa_forward without a workspace argument, for callers that must not
 * allocate device memory at call time (e.g. a plugin inside an application
 * whose memory manager owns the device, or a latency-bound loop that cannot
 * afford cudaMalloc).  The pages have no counterpart: this is a packaging
 * variant of bsa_forward, same kernels, same results.
 *   - Scratch is a static device array of 32 MiB inside the library; every
 *     device that loads the library holds it until the process exits.  A
 *     problem whose bsa_forward_workspace_size() exceeds 32 MiB is rejected
 *     with BSA_ERR_WORKSPACE (2 heads x 1024 tokens, top-4 needs about
 *     2.1 MiB and fits; 8 heads x 8192 tokens, top-16 needs about 25 MiB
 *     and fits; 8 heads x 32768 tokens, top-16 needs about 100 MiB and is
 *     rejected; the workspace grows with heads * n * k).
 *   - Allocates nothing: no cudaMalloc/cudaFree and no allocating library
 *     call.  The first call on each device looks up the array's device
 *     address (cudaGetSymbolAddress) with that device current; make that
 *     first call before any stream capture.  The address is kept for the
 *     life of the process (like the status word's, see
 *     bsa_get_device_status): calls after a cudaDeviceReset of that device
 *     are not supported.
 *   - Every call on a device shares the one array: calls whose work can
 *     overlap on the GPU (different streams, or different host threads)
 *     race on it and must be serialised by the caller.
 * Other arguments and errors as bsa_forward.
 */
bsa_status bsa_forward_noalloc(bsa_shape shape, const void *q, const void *k,
                               const void *v, int32_t key_block, int32_t topk,
                               float scale, void *out, int32_t *idx_out,
                               void *stream);

/*
 * Rotary positions, on q and k before bsa_forward, bsa_cache_append or
 * bsa_paged_decode, and their gradient.  (The pages do not rotate; a model
 * around the method does.)  Pair i of a token at position p turns by
 * t = p * f_i:
 *   x_a' = m (x_a cos t - x_b sin t),  x_b' = m (x_b cos t + x_a sin t),
 * with (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved; channels
 * from rot on are copied.  Products of a position and the table (below) are
 * exact modulo one turn, so an angle is off by fp32 rounding and by 2^-52 of
 * p f, the fp64 frequency's; the rotation is computed in fp32 and rounded once.
 *
 * The frequencies f_i are made on the host, in two steps so that a caller
 * can put its own in between:
 *   bsa_rope_frequencies  inv_freq[i] = theta^(-2i/rot), i < rot/2, scaled
 *       for longer contexts (s = factor):
 *         LINEAR  f / s;
 *         BASE    theta * s^(rot/(rot-2)) in place of theta (rot >= 4);
 *         PARTS   by the turns r = original * f / 2 pi a frequency makes
 *                 over the original context: f where r >= high, f / s where
 *                 r <= low, in between g f + (1 - g) f / s with
 *                 g = (r - low) / (high - low).
 *   bsa_rope_table        f as turns per position modulo one turn, in units
 *       of 2^-64.  Products with a position wrap modulo one turn exactly.
 * Both write HOST arrays; the caller copies the table to the device once.
 */
typedef enum {
    BSA_ROPE_NONE = 0,
    BSA_ROPE_LINEAR = 1,
    BSA_ROPE_BASE = 2,
    BSA_ROPE_PARTS = 3
} bsa_rope_scaling;

typedef struct {
    int32_t rot;            /* rotated channels, even                       */
    int32_t scaling;        /* bsa_rope_scaling                             */
    double theta;           /* base of the frequencies                      */
    double factor;          /* s (ignored by NONE)                          */
    double original;        /* PARTS: tokens of the original context        */
    double low, high;       /* PARTS: bounds on the turns, low < high       */
} bsa_rope_params;

bsa_status bsa_rope_frequencies(bsa_rope_params params, double *inv_freq);
bsa_status bsa_rope_table(const double *inv_freq, int32_t count, uint64_t *table);

/*
 * x and out are [batch][heads][n][d] in any order of strides (in elements;
 * the d channels of a row contiguous), so that q and k can be rotated where a
 * projection left them and come out in the layout bsa_forward takes.
 *   positions  int32 [batch][n] (device), or NULL: token i is at first + i.
 *              Any int32 value, negative ones too.  (first may lie beyond, at
 *              2^-52 of p f an angle means nothing from about 2^50 on.)
 *   rotation   table (DEVICE uint64 [rot/2], from bsa_rope_table), rot even
 *              and in [2, d], layout, and the factor m on cos and sin.
 *   out        may be x itself, with x's strides; otherwise the two must not
 *              overlap.  Rows of out must not overlap (no stride 0); x may be
 *              broadcast.
 * bf16 or fp32; d in {64, 128}; strides multiples of 16 bytes, not negative;
 * the table 16-byte aligned; n = 0 does nothing.
 * bsa_rope_backward: dx = the gradient with respect to x given dout (the
 * same map with -t; m applies again, the map being linear).
 */
typedef struct {
    int64_t batch, n;
    int32_t heads, d, dtype;
} bsa_heads;

typedef struct {
    int64_t batch, head, token;
} bsa_strides;

typedef struct {
    const uint64_t *table;
    int32_t rot;
    int32_t interleaved;
    float factor;
} bsa_rotation;

bsa_status bsa_rope(bsa_heads shape, const void *x, bsa_strides x_strides,
                    const int32_t *positions, int64_t first, bsa_rotation rotation,
                    void *out, bsa_strides out_strides, void *stream);
bsa_status bsa_rope_backward(bsa_heads shape, const void *dout, bsa_strides dout_strides,
                             const int32_t *positions, int64_t first, bsa_rotation rotation,
                             void *dx, bsa_strides dx_strides, void *stream);

/*
 * A paged key/value cache.  A page is one key block of the selection: it
 * holds `page` tokens' K and V of every head, and the mean of its keys, so
 * that decoding scores pages without reading their keys.  Sequence s's block
 * b (tokens [b * page, (b + 1) * page)) is in page table[s][b].
 *   k, v   [num_pages][heads][page][d] bf16 (device)
 *   kbar   [num_pages][heads][d] fp32 (device): the mean of the rows the last
 *          append left filled
 * page in {16, 32, 64, 128}, d in {64, 128}, heads <= 65535.
 */
typedef struct {
    void *k;
    void *v;
    float *kbar;
    int64_t num_pages;
    int32_t heads, page, d;
} bsa_cache;

/*
 * Appends new tokens' K and V to their sequences' pages and writes the means
 * of the pages they fall in (over all of a page's filled rows, so a call may
 * be repeated, and a sequence that was cut short may be appended to).
 *   k, v        [tokens][heads][d] bf16 (device), the tokens of sequence 0
 *               first; k_stride, v_stride: elements from a token to the next
 *               (multiples of 8, >= heads * d).  They must not overlap the
 *               cache.
 *   cu_tokens   int32 [seqs + 1] (device): sequence s has the tokens
 *               [cu[s], cu[s + 1]), possibly none; tokens before cu[0] and
 *               from cu[seqs] on are ignored.  NULL: tokens / seqs each (it must divide).
 *   start       int32 [seqs] (device): tokens each sequence holds already.
 *   table       int32 [seqs][table_width] (device).  A page may be listed by
 *               several sequences, but a page that is written to by one only.
 * A sequence whose new tokens do not fit its table (or whose cu_tokens or
 * start make no sense) is skipped and reported as BSA_ERR_INVALID_ARG
 * through bsa_get_device_status(), a page outside [0, num_pages) is skipped
 * and reported as BSA_ERR_BAD_INDEX.  Where cu_tokens fall or leave [0,
 * tokens], which is always reported, the other sequences may get only some of
 * their pages' tokens.
 */
bsa_status bsa_cache_append(bsa_cache cache, const void *k, int64_t k_stride, const void *v,
                            int64_t v_stride, int64_t tokens, int64_t seqs,
                            const int32_t *cu_tokens, const int32_t *start,
                            const int32_t *table, int32_t table_width, void *stream);

/*
 * Copies whole pages (K, V and means): pairs int32 [count][2] (device) of
 * (from, to).  No page may be the target of two pairs, nor the target of one
 * and the source of another (bsa_pages_take_copies and bsa_pages_compact
 * give such lists).  A pair with a page outside [0, num_pages) is skipped and
 * reported as BSA_ERR_BAD_INDEX.
 */
bsa_status bsa_cache_copy_pages(bsa_cache cache, const int32_t *pairs, int64_t count,
                                void *stream);

/*
 * Decoding: the two stages of the method for single tokens over the paged
 * cache, in one launch.  Token t of sequence token_seq[t] sees its first
 * lens[t] keys.  Every query head h scores the ceil(lens[t] / page) blocks of
 * cache head h / (q_heads / heads) (score = q . kbar, unscaled), keeps its
 * topk best, and attends to their keys j < lens[t].  The selection is that of
 * the scores' exact values for the given kbar (close calls are settled in
 * fp64, one block after another: means that differ by rounding only, or one
 * that is not finite, in thousands of blocks, cost milliseconds), ties to the
 * lower block id; a NaN score ranks as -inf.  A kbar is that of the rows its
 * page held at the last append: without local_block, a token with rows behind
 * it in its own block (drafts; a sequence that was cut short) scores that
 * block by a mean they are part of, although it does not attend to them.
 *   q          [tokens][q_heads][d] bf16 (device); q_stride: elements from a
 *              token to the next (multiple of 8, >= q_heads * d).
 *   table      int32 [seqs][table_width] (device), table_width <= 16384.
 *   token_seq  int32 [tokens] (device) in [0, seqs), or NULL: token t is
 *              sequence t's (seqs >= tokens then).
 *   lens       int32 [tokens] (device), the token itself included.  0: the
 *              output row is zero.
 *   options    NULL = none;
 *              local_block  the last block (the token's own) is always
 *                           selected; topk - 1 others compete.
 *              share_group  the query heads of a cache head share one
 *                           selection, made on the sum of their scores.
 *   scale      softmax scale; <= 0 selects 1/sqrt(d).
 *   out        [tokens][q_heads][d] bf16 (device); not q, nor in the cache.
 *   idx_out    optional int32 (device) [tokens][q_heads][topk], or
 *              [tokens][heads][topk] with share_group: the selected blocks,
 *              ascending, -1 after the last.
 * topk in [1, 32]; q_heads a multiple of heads, at most 128 per cache head.
 * Only pages that hold one of the first lens[t] keys are looked up.  One
 * outside [0, num_pages) is reported as BSA_ERR_BAD_INDEX; its block scores
 * -inf, and its keys are skipped if it is selected all the same.  lens
 * outside [0, table_width * page] is clamped and reported as
 * BSA_ERR_INVALID_ARG; a token_seq outside [0, seqs) is reported as
 * BSA_ERR_BAD_INDEX and the token's row is zero.
 */
typedef struct {
    int32_t local_block;
    int32_t share_group;
} bsa_decode_options;

bsa_status bsa_paged_decode(bsa_cache cache, const void *q, int64_t q_stride, int64_t tokens,
                            int32_t q_heads, const int32_t *table, int32_t table_width,
                            int64_t seqs, const int32_t *token_seq, const int32_t *lens,
                            int32_t topk, const bsa_decode_options *options, float scale,
                            void *out, int32_t *idx_out, void *stream);

/*
 * The paged cache in 8 bits.  A row (one token's d channels of one head) is
 * held as codes c_i = 127 x_i / a, rounded to the nearest whole number (ties
 * to the even one), a = max |x_i|, and the scale a / 127: it stands for
 * c_i * scale, off by a / 254 at most.  Codes are those of the exact quotients;
 * a row of zeros has scale 0; a row with a value that is not finite has scale
 * NaN (and codes 0), so all of it reads as NaN.
 *   k, v              [num_pages][heads][page][d] int8 (device)
 *   k_scale, v_scale  [num_pages][heads][page] fp32 (device)
 *   kbar              [num_pages][heads][d] fp32 (device): the mean of what
 *                     the page's filled rows stand for
 * Sizes as bsa_cache.
 */
typedef struct {
    int8_t *k;
    int8_t *v;
    float *k_scale;
    float *v_scale;
    float *kbar;
    int64_t num_pages;
    int32_t heads, page, d;
} bsa_cache8;

/*
 * bsa_cache_append, bsa_cache_copy_pages and bsa_paged_decode over the 8-bit
 * cache: arguments, results and errors are theirs.  Appending quantises the
 * bf16 rows; copies take the codes, the scales and the means; decoding attends
 * to what the rows stand for (no second rounding of K and V).  A key's weight
 * is off by 2^-11 of itself at most, or, where that is more, its part of an
 * output by 2^-31 of the largest 127 * v_scale among the keys that the same
 * query row attends to.  Keys that a row does not attend to do not count.
 */
bsa_status bsa_cache8_append(bsa_cache8 cache, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, int64_t tokens, int64_t seqs,
                             const int32_t *cu_tokens, const int32_t *start,
                             const int32_t *table, int32_t table_width, void *stream);
bsa_status bsa_cache8_copy_pages(bsa_cache8 cache, const int32_t *pairs, int64_t count,
                                 void *stream);
bsa_status bsa_paged_decode8(bsa_cache8 cache, const void *q, int64_t q_stride, int64_t tokens,
                             int32_t q_heads, const int32_t *table, int32_t table_width,
                             int64_t seqs, const int32_t *token_seq, const int32_t *lens,
                             int32_t topk, const bsa_decode_options *options, float scale,
                             void *out, int32_t *idx_out, void *stream);

/*
 * Reads cached tokens back: positions [start[s], start[s] + n_s) of every
 * sequence s, as bf16 rows (of an 8-bit cache code * scale in fp32, rounded
 * once), for instance a prefix for bsa_forward.
 *   tokens, cu_tokens, seqs, start, table, table_width  as bsa_cache_append;
 *              token cu[s] + i of the output is position start[s] + i.
 *   k, v       outputs (device) with the strides `out` in elements (batch is
 *              ignored): [tokens][heads][d] has token = heads * d, head = d;
 *              [heads][tokens][d] has token = d, head = tokens * d.  Strides
 *              are multiples of 8, rows must not overlap, nor k, v and the
 *              cache.
 * A sequence whose tokens lie beyond its table is skipped and reported as
 * BSA_ERR_INVALID_ARG, a page outside [0, num_pages) is skipped and reported
 * as BSA_ERR_BAD_INDEX; rows that are skipped and tokens that no sequence has
 * are left as they were.
 */
bsa_status bsa_cache_read(bsa_cache cache, int64_t tokens, int64_t seqs, const int32_t *cu_tokens,
                          const int32_t *start, const int32_t *table, int32_t table_width,
                          void *k, void *v, bsa_strides out, void *stream);
bsa_status bsa_cache8_read(bsa_cache8 cache, int64_t tokens, int64_t seqs,
                           const int32_t *cu_tokens, const int32_t *start, const int32_t *table,
                           int32_t table_width, void *k, void *v, bsa_strides out, void *stream);

/*
 * Attention of new tokens to the cache that holds them (append first, with
 * the same cu_tokens, start and table): the last token of each sequence, a
 * prompt's chunk, or a tree of drafted tokens.  Nothing is selected; with a
 * window it is what a sliding-window model does around the block selection
 * (page "Block-Sparse & Linear Attention Kernels", section 2, sliding window).
 * New token i of sequence s has its K and V at slot start[s] + i.
 *   Without tree   its position is its slot, and it sees the keys of the
 *                  slots up to its own.
 *   tree           uint64 [tokens] (device), 8-byte aligned: bit j of token
 *                  i's word says that it sees new token j of its sequence (its
 *                  ancestors, and itself); it sees all keys of slots before
 *                  start[s].  At most 64 new tokens each.  Its position is
 *                  start[s] + the number of other new tokens it sees.
 *   window         NULL: all of these.  Otherwise only those at positions
 *                  above its own less `window`, and those below `sinks`
 *                  (window >= 1, sinks >= 0).
 *   q              [tokens][q_heads][d] bf16 (device); q_stride: elements from
 *                  a token to the next (multiple of 8, >= q_heads * d).
 *   scale          softmax scale; <= 0 selects 1/sqrt(d).
 *   out            [tokens][q_heads][d] bf16 (device); not q, nor in the
 *                  cache.  A token that sees no key gets zeros (as does one
 *                  whose scores are all -inf).
 * Softmax statistics and sums are fp32; the weighted values are divided by the
 * weights' sum at the end, so |v| times the number of keys has to stay below
 * 2^119.  A weight enters the product with V
 * off by at most 2^-17 of itself where a sequence has few query rows per cache
 * head on average (8, or 16 with at most 1024 keys), by at most 2^-8 (half a
 * bf16 step) where it has more; over 8-bit pages as bsa_paged_decode8 says.
 * q_heads a multiple of heads, at most 128 per cache head.  A masked key does
 * not count whatever its K and V hold; a key of the cache that is not finite
 * costs time where it is masked (its rows are computed again, one by one).
 * A sequence with start below 0, more keys than its table has room for or
 * than 2^31 - 256, or more than 64 new tokens and a tree, is skipped and
 * reported as BSA_ERR_INVALID_ARG, like one whose cu_tokens make no sense; its
 * rows, and those of tokens that no sequence has, are left as they were.
 * The keys of a page outside [0, num_pages) are skipped and reported as
 * BSA_ERR_BAD_INDEX; only pages that hold a key some row sees are looked up
 * for certain.
 */
typedef struct {
    int32_t window;
    int32_t sinks;
} bsa_window;

bsa_status bsa_paged_attention(bsa_cache cache, const void *q, int64_t q_stride, int64_t tokens,
                               int32_t q_heads, const int32_t *table, int32_t table_width,
                               int64_t seqs, const int32_t *cu_tokens, const int32_t *start,
                               const uint64_t *tree, const bsa_window *window, float scale,
                               void *out, void *stream);
bsa_status bsa_paged_attention8(bsa_cache8 cache, const void *q, int64_t q_stride, int64_t tokens,
                                int32_t q_heads, const int32_t *table, int32_t table_width,
                                int64_t seqs, const int32_t *cu_tokens, const int32_t *start,
                                const uint64_t *tree, const bsa_window *window, float scale,
                                void *out, void *stream);

/*
 * Which sequence owns which page, on the host: page counts of references,
 * copy on write, and the copies that bsa_cache_copy_pages has to make.  It
 * touches no device memory; a handle is used by one thread at a time.
 *   create      a pool of num_pages pages of `page` tokens, max_seqs empty
 *               sequences with at most table_width pages each.
 *   reserve     makes room for `tokens` more tokens of a sequence and counts
 *               them as there.  If its partly filled last page is shared, the
 *               sequence gets a page of its own and a copy is queued.
 *               All or nothing: BSA_ERR_WORKSPACE when the pool or the table
 *               is too small.
 *   fork        the empty sequence `to` gets all of `from`'s tokens, sharing
 *               the pages.  Tokens that are reserved but not appended yet come
 *               with the shared pages once they are appended to `from`; if
 *               one of the two grows before that, see take_copies.
 *   truncate    keeps the first `length` tokens; pages nobody holds any more
 *               become free (length 0: all of them).
 *   take_copies hands out the queued copies, pairs HOST int32 [capacity][2],
 *               and empties the queue.  Run them (in stream order) before
 *               anything is appended to the cache.  pairs NULL: only
 *               *count is written.  A page that a queued copy reads is not
 *               given away until then.  BSA_ERR_WORKSPACE when capacity is
 *               too small (nothing is taken).
 *               A copy brings the tokens that are in the page when it runs.
 *               BSA_ERR_INVALID_ARG, and nothing is taken, when a sequence
 *               was forked and grew after tokens were reserved that no
 *               take_copies or tables has followed: its copy would miss them.
 *               Free the fork, and make it again after the append.  A call of
 *               tables says that they are appended by now, or will be to
 *               every sequence that has them, and lifts the refusal.
 *   compact     moves the pages in use to the lowest ids; pairs as above, at
 *               most num_pages / 2 of them.  Not while copies are queued
 *               (BSA_ERR_INVALID_ARG).
 *   tables      HOST int32 [max_seqs][table_width] (-1 after a sequence's
 *               pages) and int32 [max_seqs] lengths; either may be NULL.
 *   free_pages  pages nobody holds; -BSA_ERR_INVALID_ARG without a handle.
 * A sequence's length is at most 2^31 - 1.
 */
typedef struct bsa_pages_s *bsa_pages;
bsa_status bsa_pages_create(int64_t num_pages, int32_t page, int32_t max_seqs,
                            int32_t table_width, bsa_pages *pages);
bsa_status bsa_pages_destroy(bsa_pages pages);
bsa_status bsa_pages_reserve(bsa_pages pages, int32_t seq, int64_t tokens);
bsa_status bsa_pages_fork(bsa_pages pages, int32_t from, int32_t to);
bsa_status bsa_pages_truncate(bsa_pages pages, int32_t seq, int64_t length);
bsa_status bsa_pages_take_copies(bsa_pages pages, int32_t *pairs, int64_t capacity,
                                 int64_t *count);
bsa_status bsa_pages_compact(bsa_pages pages, int32_t *pairs, int64_t capacity, int64_t *count);
bsa_status bsa_pages_tables(bsa_pages pages, int32_t *table, int32_t *lengths);
int64_t bsa_pages_free_pages(bsa_pages pages);

/* Number of kernel launches one bsa_forward call enqueues for this problem
 * (for launch accounting by callers); negative bsa_status on bad arguments. */
int32_t bsa_forward_launches(bsa_shape shape, int32_t key_block, int32_t topk);

/*
 * Static block lists, built on the host, synchronously (page
 * "yayme/CUDA-kernel" README: "precompute the list of active (row_tile,
 * col_tile) pairs on the CPU and pass it in").  A key block is listed for a
 * query tile iff at least one (query, key) pair inside it satisfies `mask`
 * (BSA_MASK_NONE lists every block).
 *   list          HOST int32 [ceil(n/q_group)][max_blocks], -1 padded.
 *   counts        optional HOST int32 [ceil(n/q_group)]: blocks per row.
 *   active_pairs  optional HOST int64: number of (i, j) pairs the mask
 *                 admits over the whole sequence (one head).
 * bsa_static_max_blocks() returns the smallest max_blocks that fits, or a
 * negative bsa_status on invalid arguments.
 */
int32_t bsa_static_max_blocks(int64_t n, int32_t q_group, int32_t key_block,
                              bsa_mask mask);
bsa_status bsa_static_blocks(int64_t n, int32_t q_group, int32_t key_block,
                             bsa_mask mask, int32_t *list, int32_t max_blocks,
                             int32_t *counts, int64_t *active_pairs);

/*
 * Reads the device status word into *status (a bsa_status value), then
 * clears it.  Synchronises `stream` first.  The word is a static device
 * variable of the library, one per device; its address is looked up on the
 * first call that needs it on a device and kept for the life of the process
 * (a cudaDeviceReset of that device is not supported afterwards).
 */
bsa_status bsa_get_device_status(int32_t *status, void *stream);

/*
 * Failure-path self-test (the pages have no counterpart; it tests this
 * library's own error handling).  Enqueues one small kernel that runs the
 * library's bounded wait on something nothing will ever complete -- kind 0:
 * an mbarrier no thread arrives on (the wait every TMA / MMA hand-off of the
 * tensor-core kernels uses); kind 1: a counter in global memory no thread
 * raises (the wait the block-major fine stage uses between its query ranges
 * and merges).  After about limit_ns (1e3 .. 2e9 ns; the kernels use 2e9)
 * the wait gives up, records BSA_ERR_TIMEOUT in the device status word and
 * the kernel returns; the CUDA context stays usable.  If the status word
 * already holds BSA_ERR_TIMEOUT the wait gives up at once.  Read (and clear)
 * the result with bsa_get_device_status().  BSA_ERR_INVALID_ARG for another
 * kind or a limit outside the range.
 */
bsa_status bsa_selftest_wait_timeout(int32_t kind, uint64_t limit_ns, void *stream);

/* Static description of a status code. */
const char *bsa_status_string(int32_t status);

/* One-line reason for the last error returned on the calling thread. */
const char *bsa_last_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t bsa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BSA_H_ */
