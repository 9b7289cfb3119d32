/*
 * dfl.h -- C ABI of one DFlash speculative-decode step over Q4_1 weights on one GB300 (sm_103a).
 *
 * The step (pages, by title and section):
 *   1. Draft: an 8-row block [last token, mask x 7] conditioned on the target's tapped layer outputs
 *      through the draft's fc projection proposes up to 7 tokens in one pass (model card
 *      "Nemotron-3.5-Bolt-E4B-DFlash-NPU2", spec table and "How it is used"; 1bit engine PR "a Gemma4
 *      pack stops re-reading its weights every token; tools/dflash_acceptance", item 2).
 *   2. Verify: one batched pass of the target over the k drafted rows, every projection one M-row
 *      product, attention over per-layer-width KV planes: sliding and full layers, and KV-shared
 *      layers that read their owner's plane and append nothing (1bit engine PR "npu forward: Gemma4
 *      verifies a draft in one batched pass; KV row width per layer", "What changes").
 *   3. Accept the longest agreeing prefix plus one target token (greedy, first maximum; or sampled
 *      per position), then commit_verify_rows: keep that many rows, pure index arithmetic.
 *
 * Conventions
 *  - Every call returns DFL_OK (0) or a negative DFL_E_* code; dfl_last_error() gives the message.
 *    On any error the state (positions held, planes, draft context) is unchanged.
 *  - Memory: the library never allocates device memory. The caller allocates the three device buffers
 *    sized by dfl_required_bytes() and keeps them alive until dfl_destroy(). Device pointers below
 *    are marked "device"; everything else is host memory.
 *  - Calls enqueue work on the stream given to dfl_init(). Calls with host outputs (tokens, counts,
 *    logits) synchronise that stream before returning, so the outputs are valid on return. Calls
 *    without host outputs return without synchronising.
 *  - Numbers: activations, KV planes and taps are fp32 (the pages' "floats"); weights are Q4_1 or bf16.
 *  - Formats: bf16 = upper half of IEEE binary32. Q4_1 matrix ("container" layout): uint8
 *    [N][K/32][20]; block = fp16 scale d, fp16 minimum m, 16 bytes of 4-bit codes, element i of the
 *    block in byte 4 + i/2 (low nibble for even i); weight w = d*q + m ("Q4_1: 5 bits per weight with
 *    scales and minimums", model card spec table). N = output columns, K = inputs (reduction).
 *  - Not thread-safe: one host thread per context.
 */
#ifndef DFL_H
#define DFL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DFL_MAX_LAYERS 64
#define DFL_MAX_TAPS 8
#define DFL_MAX_ROWS 16          /* rows of one verify or prefill chunk (R_max) */

enum {
    DFL_OK = 0,
    DFL_E_INVALID_ARG = -1,      /* bad pointer, size, token id or configuration */
    DFL_E_STATE = -2,            /* call not legal in the current state (e.g. verify while pending) */
    DFL_E_CAPACITY = -3,         /* positions would exceed max_ctx */
    DFL_E_UNSUPPORTED = -4,      /* e.g. k > DFL_MAX_ROWS, a shape the kernels do not take */
    DFL_E_CUDA = -5,             /* a CUDA call failed; the message names it */
    DFL_E_TIMEOUT = -6           /* a bounded device wait gave up (about 1 s); reported by the next call
                                    that reads the device state, with the state of the last good call */
};

enum { DFL_SLIDING = 0, DFL_FULL = 1 };

/* Model and capacity. Layer l is KV-shared when kv_owner[l] != l: it reads the plane of layer
 * kv_owner[l] (the last non-shared layer of the same attention type) and appends nothing. */
typedef struct dfl_config {
    /* target */
    int32_t n_layers, hidden, vocab, n_heads, head_dim;
    int32_t window;                        /* sliding window: keys p-window+1..p visible to position p */
    int32_t ple_dim;                       /* per-layer-embedding width; 0 = none (and no layer scalar) */
    int32_t layer_type[DFL_MAX_LAYERS];    /* DFL_SLIDING / DFL_FULL */
    int32_t kv_heads[DFL_MAX_LAYERS];
    int32_t kv_owner[DFL_MAX_LAYERS];
    int32_t ffn[DFL_MAX_LAYERS];
    float rope_base_sliding, rope_base_full, eps, emb_scale;
    /* draft (hidden width = target hidden) */
    int32_t d_layers, d_ffn, d_heads, d_kv_heads, d_head_dim;
    int32_t d_window;                      /* context keys visible to a block; 0 = all */
    int32_t block;                         /* rows of a draft block (proposals = block - 1) */
    int32_t n_taps, mask_token;
    int32_t taps[DFL_MAX_TAPS];            /* target layers whose outputs feed fc, ascending */
    float d_rope_base, d_eps, d_emb_scale;
    /* capacity */
    int32_t max_ctx;                       /* positions the KV arena holds */
    int32_t prefill_rows;                  /* 0, or 128..8192 (a multiple of 16): dfl_prefill takes up to
                                              this many prompt rows in one pass whose products run on the
                                              tcgen05 tensor cores (the buffers of such a pass, and sliding
                                              rings of window + prefill_rows - 1 slots, are sized in) */
    int32_t kv8;                           /* 0, or 1: the planes of full layers, which grow with the context,
                                              are held in 8 bits (the dfl_kv8 cache below: blocks of 32 committed
                                              positions as codes, newer positions fp32), a quarter of the
                                              memory and of the bytes that attention reads. A row sees the blocks
                                              committed before its pass as their codes' values, so results differ
                                              from those of fp32 planes by the codes' rounding, and a
                                              position's by how its passes were cut. Needs prefill_rows = 0 and
                                              at most 16 query heads a key/value head */
} dfl_config;

typedef struct dfl_sizes {
    uint64_t weights_bytes;                /* packed weight image, tables */
    uint64_t state_bytes;                  /* KV planes, draft context, taps, device counters */
    uint64_t workspace_bytes;              /* activations and reduction scratch of one pass */
} dfl_sizes;

typedef struct dfl_buffers {
    void *weights;                         /* device, >= weights_bytes, 256-byte aligned */
    void *state;                           /* device, >= state_bytes, 256-byte aligned */
    void *workspace;                       /* device, >= workspace_bytes, 256-byte aligned */
} dfl_buffers;

/* Sampling: temperature > 0 samples every verified position with the uniform
 * U(seed, position) = top 53 bits of SplitMix64(seed XOR position * 0x9E3779B97F4A7C15) * 2^-53,
 * and picks the smallest token whose running sum of exp((l - max)/T) exceeds U * sum.
 * A NULL dfl_sampling, or temperature <= 0, means greedy (first maximum). */
typedef struct dfl_sampling {
    float temperature;
    uint64_t seed;
} dfl_sampling;

typedef struct dfl_ctx dfl_ctx;

/* sizeof(dfl_config) of the library. Headers of later builds may add fields at the end of dfl_config, and the
 * library reads all that its own has: a client that loads a library it was not built beside first compares
 * this with its own sizeof(dfl_config), and passes no dfl_config where they differ. */
int64_t dfl_config_bytes(void);

/* Sizes of the three device buffers for a configuration. Fails with DFL_E_INVALID_ARG or
 * DFL_E_UNSUPPORTED on a configuration the library does not take (it states which field). */
int dfl_required_bytes(const dfl_config *cfg, dfl_sizes *out);

/* Create a context over caller-owned device buffers (sizes from dfl_required_bytes) and a CUDA
 * stream (cudaStream_t, may be NULL for the legacy stream). Positions held start at 0. Every tensor
 * must then be given once with dfl_load_tensor before the first pass. The context does not own the
 * buffers or the stream. */
int dfl_init(const dfl_config *cfg, const dfl_buffers *buf, void *cuda_stream, dfl_ctx **out);

/* Load one tensor from DEVICE memory in its container format; the library packs it into its own
 * layout in the weights buffer (Q4_1 matrices into a tile-major image of the same bytes per weight).
 * Names: "emb" bf16 [vocab][hidden]; "head" bf16 [vocab][hidden]; "final_norm" bf16 [hidden];
 * "ple_table" bf16 [vocab][n_layers*ple_dim]; per target layer l, "t<l>.": attn_norm, q_norm,
 * k_norm (owners), post_attn_norm, pre_ffn_norm, post_ffn_norm, ple_norm (bf16), lambda (bf16 [1]),
 * wqkv (owners: q|k|v) or wq (shared), wo, wgu (gate|up), wd, wple_g, wple_p (Q4_1);
 * draft: "d.fc" bf16 [hidden][n_taps*hidden], "d.hidden_norm", "d.final_norm", and per draft
 * layer "d<l>.": attn_norm, q_norm, k_norm, ffn_norm, wqkv, wo, wgu, wd.
 * `bytes` must equal the tensor's container size. The source may be freed once the stream has
 * passed this call (it is read by kernels enqueued here). */
int dfl_load_tensor(dfl_ctx *ctx, const char *name, const void *dev_src, size_t bytes);

/* Prefill (extend the context; 1bit engine PR "npu forward: Gemma4 verifies a draft in one batched
 * pass; KV row width per layer", "What changes" item 1, extend_context): run the n tokens at positions
 * held..held+n-1 in passes, commit them, bring the draft context up to date,
 * and write the target's token for the next position to *next_tok (greedy or sampled). The output
 * head runs on the last prompt row only: only that row's token is needed. Passes: with prefill_rows > 0,
 * min(prefill_rows, remaining) rows while 128 or more remain (products on tcgen05), then passes of at
 * most DFL_MAX_ROWS rows; with prefill_rows = 0, passes of at most DFL_MAX_ROWS rows. Fails with
 * DFL_E_CAPACITY if held + n exceeds max_ctx; on any error positions held stay as they were. An error
 * after the first pass was enqueued (DFL_E_TIMEOUT, DFL_E_CUDA) on a context that held positions
 * leaves it refusing passes and snapshots with DFL_E_STATE until dfl_restore succeeds: the passes that
 * ran may have overwritten sliding-ring and draft-context slots those positions still need. */
int dfl_prefill(dfl_ctx *ctx, const int32_t *tokens, int n, const dfl_sampling *s, int32_t *next_tok);

/* Draft block (model card "Nemotron-3.5-Bolt-E4B-DFlash-NPU2", "How it is used"; 1bit engine PR "a
 * Gemma4 pack stops re-reading its weights every token; tools/dflash_acceptance", item 2) at positions
 * held..held+block-1 for rows [last_tok, mask x (block-1)]: first makes the committed rows not yet in
 * the draft context into context (fc of their taps, then each draft layer's key and value), then runs
 * the block. Proposals (block-1 tokens for positions held+1..) are kept on the device for
 * dfl_verify_block(rows = NULL) and copied to `proposals` when it is not NULL (which synchronises; with
 * NULL the call does not synchronise, and a device error surfaces at the next synchronising call). */
int dfl_draft_block(dfl_ctx *ctx, int32_t last_tok, int32_t *proposals);

/* Batched verify (1bit engine PR "npu forward: Gemma4 verifies a draft in one batched pass; KV row
 * width per layer", "What changes": every projection one M-row product, a KV-shared layer reads its
 * owner's plane and appends nothing; acceptance: model card "How it is used") of k rows at positions
 * held..held+k-1. rows = [last token, proposal 1, .., proposal k-1]; rows == NULL takes last_tok of the
 * last draft block and its k-1 first proposals. Writes the target's token for positions
 * held+1..held+k to target_tok[0..k-1] (if not NULL) and the accepted length a (longest prefix with
 * proposal i == target token i-1) to *accepted (if not NULL). The tokens the pass emits are
 * target_tok[0..a] (the accepted proposals equal the target's tokens before them, plus the target's
 * token after the last one). The rows stay pending until dfl_commit_verify_rows / dfl_commit_accepted.
 * k in 1..DFL_MAX_ROWS. */
int dfl_verify_block(dfl_ctx *ctx, const int32_t *rows, int k, const dfl_sampling *s,
                     int32_t *target_tok, int32_t *accepted);

/* commit_verify_rows (1bit engine PR "npu forward: Gemma4 verifies a draft in one batched pass",
 * "What changes" item 1 and "Proof": 3 held, commit_verify_rows(2), 5 held): keep the first `keep` rows
 * of the pending verify (0 <= keep <= k); positions held become held + keep. Pure index arithmetic: no
 * data moves; later rows are overwritten by the next pass. keep = DFL_KEEP_ACCEPTED keeps accepted + 1
 * rows (the accepted proposals and the row of the last token) as counted by the last verify. */
#define DFL_KEEP_ACCEPTED (-1)
int dfl_commit_verify_rows(dfl_ctx *ctx, int keep);
/* The acceptance step's commit (model card "How it is used": the longest agreeing prefix plus one
 * target token are kept): keep min(accepted + 1, max_keep) rows of the pending verify, where max_keep
 * caps the tokens a caller still wants (a token budget), and write that count to *kept (if not NULL).
 * The tokens the kept rows emit are target_tok[0..*kept-1] of the verify. With stop_token >= 0, a kept
 * row whose token is the stop token ends the count there: that token is emitted, but no row for it is
 * ever committed (single-turn serving, FastFlowLM PR #899 "gemma4e-dflash-flash", "Changes": no KV row
 * for the stop token); *stopped (if not NULL) is then 1, else 0. */
int dfl_commit_accepted(dfl_ctx *ctx, int max_keep, int32_t stop_token, int32_t *kept, int32_t *stopped);

/* Snapshot (1bit engine PR "npu forward: Gemma4 verifies a draft in one batched pass", "What changes"
 * item 1: snapshot and restore cut each plane at its own layer's width; a KV-shared layer's plane stays
 * empty) of the committed state (positions held, every owner plane, the draft context, the taps of
 * committed rows not yet in the draft context) into a DEVICE buffer of at least dfl_snapshot_bytes()
 * bytes; restore replaces the state with a snapshot taken from a context with the same configuration.
 * Both need the committed state (no pending verify). KV-shared layers have no plane and contribute
 * nothing. A snapshot taken once after a pinned prefix may be restored any number of times (FastFlowLM
 * PR #899 "gemma4e-dflash-flash", "Changes": the pinned prefix must not be overwritten by a request).
 * Planes in 8 bits hold counts of their own. Where a snapshot's are out of order, the next prefill or verify
 * meets it on the device: it fails with DFL_E_STATE, and so do passes and snapshots until a sound one is restored. */
int64_t dfl_snapshot_bytes(const dfl_ctx *ctx);
int dfl_snapshot(dfl_ctx *ctx, void *dev_dst, size_t bytes);
int dfl_restore(dfl_ctx *ctx, const void *dev_src, size_t bytes);

/* Per-layer KV row width in floats per position (1bit engine PR "npu forward: Gemma4 verifies a draft
 * in one batched pass", "What changes" item 1, kv_widths(): 2 x 256 on E4B's sliding layers, 2 x 512 on
 * its full layers): 2 * kv_heads * head_dim for a layer with its own plane, 0 for a KV-shared layer.
 * out: n_layers entries. */
int dfl_kv_widths(const dfl_ctx *ctx, int32_t *out);

/* Positions held (committed), counted over owner planes only (same PR, "What changes" item 1: the
 * positions-held count ignores shared layers). -1 on a NULL context. */
int64_t dfl_positions_held(const dfl_ctx *ctx);

/* Options. DFL_OPT_KEEP_LOGITS = 1 makes verify and draft passes also store their fp32 logits
 * (otherwise only the fused argmax runs); DFL_OPT_GRAPHS = 0 launches kernels one by one instead of
 * replaying captured CUDA graphs; DFL_OPT_STOP_LAYER = l >= 0 (inspection only) makes target passes
 * stop after layer l, without the head, so dfl_debug_read shows that layer's intermediates; -1 = off;
 * DFL_OPT_PROFILE = 1 times the kernel launches of every pass on the device (read with
 * dfl_profile_read; setting the option clears the totals; each profiled pass synchronises once, to read
 * its time stamps); DFL_OPT_ATTN_CLUSTER = 16 (default), 8 or 4
 * caps the number of CTAs over which attention spreads one pair of query heads (the largest size up to
 * the cap whose clusters all fit on the device at once is taken; sizes differ in the order in which
 * the partial softmax states are added, so logits may differ in the last bits); other values are
 * DFL_E_INVALID_ARG. Changing it drops the captured graphs. */
enum { DFL_OPT_KEEP_LOGITS = 1, DFL_OPT_GRAPHS = 2, DFL_OPT_STOP_LAYER = 3, DFL_OPT_PROFILE = 4,
       DFL_OPT_ATTN_CLUSTER = 5, DFL_OPT_TEST_STALL = 6, DFL_OPT_FUSE_STEPS = 7, DFL_OPT_PLE_SPLIT = 8 };
/* DFL_OPT_PLE_SPLIT = 1 runs the per-layer-embedding tail's gate and projection (PR-batched "What
 * changes": gate = silu(x Wg) times the layer's per-layer input, then its projection) as two products
 * (0, the default, runs them as one launch on a cluster of ple_dim / 16 CTAs when the pass has at most
 * 16 rows and ple_dim is a multiple of 16 up to 256). Both give results within the parity tolerance of
 * each other. Changing it drops the captured graphs. */
/* DFL_OPT_FUSE_STEPS = 1 runs the row steps (residual, norms, layer scalar, taps) and the q/k steps
 * (norm, rotation, KV store) on the last CTAs of the product that feeds them instead of as separate
 * kernels (0, the default). Both give results within the parity tolerance of each other (the sums are
 * taken in different orders); on the E4B-shaped pair the separate kernels are faster. Changing it drops
 * the captured graphs. */
/* DFL_OPT_TEST_STALL = 1 (tests of the error path only): the Q4_1 products of the following passes
 * issue no copies, so the first one's bounded waits give up after about a second and the call that reads
 * the device state returns DFL_E_TIMEOUT with the state unchanged; set it back to 0 and the context
 * works as before. */
int dfl_set_option(dfl_ctx *ctx, int option, int value);

/* Copy the fp32 logits of the last pass (rows x vocab, row-major) to host memory. which = 0: the
 * last verify block (rows <= its k) or, after dfl_prefill, the last prompt row (rows = 1); which = 1:
 * the last draft block (rows 1..block-1, rows <= block-1). Needs DFL_OPT_KEEP_LOGITS. */
int dfl_read_logits(dfl_ctx *ctx, int which, float *host_dst, int rows);

/* Copy the fp32 taps of positions pos0..pos0+rows-1 (n_taps*hidden each) to host memory. */
int dfl_read_taps(dfl_ctx *ctx, int pos0, int rows, float *host_dst);

/* Draft-only context: make `rows` rows of given taps (DEVICE fp32 [rows][n_taps*hidden]) context at
 * positions held..held+rows-1 and advance positions held, without running the target. A context used
 * this way refuses dfl_verify_block and dfl_prefill (DFL_E_STATE). */
int dfl_draft_append_taps(dfl_ctx *ctx, const void *dev_taps, int rows);

/* Inspection: copy the first `bytes` of an internal buffer of the last pass to host memory. Names:
 * "x" [16][hidden] residual rows, "y" [16][hidden] last projection output, "qkv" [16][width],
 * "q" [16][heads*head_dim] (normed, rotated), "x_d" [16][hidden] draft residual rows; "k<l>" and "v<l>"
 * the key and value plane of target layer l, [slots][kv_heads][head_dim] with position p in slot p
 * (full layers) or p mod (window + 15) (sliding layers); all fp32. A KV-shared layer has no plane
 * (DFL_E_INVALID_ARG). */
int dfl_debug_read(dfl_ctx *ctx, const char *name, void *host_dst, size_t bytes);

/* Planted drafts (measurement workloads that control acceptance): after dfl_draft_block, replace its
 * proposals on the device with dev_table[held+1 .. held+block-1], a DEVICE int32 table indexed by
 * absolute position with at least held+block entries. The draft block itself has run. */
int dfl_plant_proposals(dfl_ctx *ctx, const int32_t *dev_table, int table_len);

/* Kernels this context has launched so far (every launch counted once). */
int64_t dfl_launch_count(const dfl_ctx *ctx);

/* Totals of the launches profiled while DFL_OPT_PROFILE was on, per class: 0 = Q4_1 products,
 * 1 = bf16 products (fc), 2 = the bf16 head with its fused argmax, 3 = attention, 4 = q/k norm,
 * rotation and KV store, 5 = the row kernels (residual and norms, taps), embedding and sampling (the
 * small state and copy kernels are not timed). A launch's time is its in-pass duration on the device
 * clock: from the earliest of its CTAs past its dependency wait to the latest of its CTAs done, so the
 * overlap of consecutive launches (programmatic dependent launch) is kept and the durations of a
 * pass's launches add up to at most the pass. *ms = their sum; *bytes = the launches' algorithmic
 * bytes for classes 0-2 (weights at 0.625 B (Q4_1) or 2 B (bf16) per weight, fp32 activations in and
 * products out), 0 for the others. Error DFL_E_INVALID_ARG for a class outside 0..5. Synchronises the
 * stream. */
int dfl_profile_read(dfl_ctx *ctx, int cls, int64_t *launches, double *ms, double *bytes);

const char *dfl_last_error(const dfl_ctx *ctx);
void dfl_destroy(dfl_ctx *ctx);

/* ---- the Q4_1 product on its own (used for the isolated GEMM measurements) ----------------------- */

/* Bytes of the packed tile image of a K x N Q4_1 matrix (K padded up to a multiple of 64). */
int64_t dfl_q41_image_bytes(int K, int N);
/* Pack a container-layout Q4_1 matrix (DEVICE) into the tile image (DEVICE). */
int dfl_q41_pack(const void *dev_src, int K, int N, void *dev_image, void *cuda_stream);
/* Bytes of an activation operand buffer for up to 16 rows of K inputs (K % 16 == 0). */
int64_t dfl_act_bytes(int M, int K);
/* Pack fp32 rows x (DEVICE [M][K]) into an activation operand buffer (DEVICE, dfl_act_bytes): bf16
 * hi + lo fragments in the order the tensor cores consume them, and per-16-input sums. */
int dfl_act_pack(const float *dev_x, int M, int K, void *dev_act, void *cuda_stream);
/* Scratch bytes dfl_q41_gemm needs for K, N, M. */
int64_t dfl_q41_gemm_scratch_bytes(int K, int N, int M);
/* y[m][n] = sum_k x[m][k] * w[k][n] (fp32), x given as an activation operand buffer (DEVICE, from
 * dfl_act_pack), y fp32 DEVICE [M][N], from the tile image; M in 1..16; N a multiple of 32. The
 * scratch (DEVICE, 256-byte aligned, >= dfl_q41_gemm_scratch_bytes) holds an error word (its first 4
 * bytes), arrival counters and partial sums; it must be zeroed once before the first call (each call
 * leaves the counters zero). Calls on one scratch must not overlap on the GPU. A row's result does not
 * depend on M. The call only enqueues; a bounded wait that gave up sets the error word (read it with
 * dfl_q41_gemm_status) and leaves y undefined. */
int dfl_q41_gemm(const void *dev_image, int K, int N, const void *act, int M, float *dev_y,
                 void *dev_scratch, size_t scratch_bytes, void *cuda_stream);
/* Status of the products enqueued on a scratch so far: synchronises the stream, returns DFL_OK, or
 * DFL_E_TIMEOUT (and clears the error word) when a bounded wait of one of them gave up. */
int dfl_q41_gemm_status(const void *dev_scratch, void *cuda_stream);

/* ---- the Q4_1 product at many rows (prompt ingest) on the tcgen05 tensor cores -------------------- */

/* Scratch bytes dfl_q41_gemm_tc needs for K, N, M (the weights expanded to bf16 hi + lo, N x Kp x 4
 * bytes, and the rows split the same way, M x Kp x 4 bytes, Kp = K rounded up to 64, plus a 1 KiB
 * header), or -1 for a shape it does not take (K and N multiples of 32 as for the tile image, M >= 1). */
int64_t dfl_q41_gemm_tc_scratch_bytes(int K, int N, int M);
/* y[m][n] = sum_k x[m][k] * w[k][n] for a Q4_1 tile image (DEVICE, dfl_q41_pack), fp32 rows x (DEVICE
 * [M][K], row-major) and fp32 y (DEVICE [M][N], row-major). 1bit engine PR "npu forward: Gemma4
 * verifies a draft in one batched pass", "What changes" item 1: a prompt goes through the layer
 * products in chunks of rows; this is that product for chunks of hundreds of rows, where it is a
 * dense contraction. w = d q + m is formed in fp32 and split into bf16 hi + lo, x likewise; the
 * tensor cores add hi*hi + hi*lo + lo*hi in fp32, so y carries about the error of an fp32 dot
 * product (it is not bit-identical to dfl_q41_gemm's). The scratch (DEVICE, 1024-byte aligned, >=
 * dfl_q41_gemm_tc_scratch_bytes) starts with the error word of dfl_q41_gemm_status, which must be
 * zero before the first call and reports (DFL_E_TIMEOUT) a bounded device wait that gave up, leaving
 * y undefined. Calls on one scratch must not overlap on the GPU. The call only enqueues three kernels
 * on the stream (weight expansion, row split, product). DFL_E_INVALID_ARG for a shape, pointer, size
 * or alignment it rejects; DFL_E_CUDA when the tensor-map encoder is unavailable or a launch fails. */
int dfl_q41_gemm_tc(const void *dev_image, int K, int N, const float *dev_x, int M, float *dev_y,
                    void *dev_scratch, size_t scratch_bytes, void *cuda_stream);

/* ---- the bf16 head on its own (the isolated sweep's bf16 2560 x 262144 comparison shape) ---------- */

/* Bytes of the packed tile image of a bf16 K x N matrix (K a multiple of 64, N of 16). */
int64_t dfl_bf16_image_bytes(int K, int N);
/* Pack a bf16 matrix [N][K] (DEVICE, row n = output n) into the tile image (DEVICE). */
int dfl_bf16_pack(const void *dev_src, int K, int N, void *dev_image, void *cuda_stream);
/* Scratch bytes dfl_bf16_head_argmax needs. */
int64_t dfl_bf16_head_scratch_bytes(int K, int N, int M);
/* The head product of the step with its fused argmax (model card "Nemotron-3.5-Bolt-E4B-DFlash-NPU2",
 * "How it is used": greedy proposals and target tokens are the first maximum of the logits):
 * argmax[m] = the first n maximising sum_k x[m][k] * w[k][n] (DEVICE int32 [M]); logits (DEVICE fp32
 * [M][N], nullable) receives the products themselves. Activations as for dfl_q41_gemm; the scratch
 * (DEVICE, 256-byte aligned, zeroed once before the first call; each call leaves it reusable) must not
 * be shared by calls that overlap on the GPU. */
int dfl_bf16_head_argmax(const void *dev_image, int K, int N, const void *dev_act, int M, int32_t *dev_argmax,
                         float *dev_logits, void *dev_scratch, size_t scratch_bytes, void *cuda_stream);

/* The same product for callers that cannot allocate device memory per call and have no scratch
 * buffer of their own to pass: code that must keep every device allocation out of its call path (a
 * fixed device-memory budget reserved up front), or hosts whose plug-in interface hands over only the
 * input and output pointers. Nothing in the DFlash method corresponds to this entry point; it is a
 * packaging of dfl_q41_gemm.
 * Scratch: one array of dfl_q41_gemm_noalloc_max_scratch() bytes (4 MiB) in the library's static device
 * memory. The first call on a device looks up that device's copy of the array (cudaGetSymbolAddress,
 * with the device current) and caches its address; make that first call outside any stream capture.
 * The cached address belongs to the device's context of that moment: after cudaDeviceReset (or any
 * other teardown of the primary context) call dfl_q41_gemm_noalloc_reset before the next product.
 * No call allocates or frees memory. Every call on a device uses the same array and leaves the last
 * call's contents in it: the arrival counters at its start must be zero, which the zero-initialised
 * array gives and every completed call restores; calls that overlap on the GPU race on it.
 * Errors: DFL_E_INVALID_ARG for the shapes or pointers dfl_q41_gemm rejects; DFL_E_CAPACITY when
 * dfl_q41_gemm_scratch_bytes(K, N, M) exceeds the array; DFL_E_CUDA when the address lookup or the
 * launch fails. Arguments as for dfl_q41_gemm. */
int dfl_q41_gemm_noalloc(const void *dev_image, int K, int N, const void *dev_act, int M, float *dev_y,
                         void *cuda_stream);
/* Bytes of the static scratch array behind dfl_q41_gemm_noalloc. */
int64_t dfl_q41_gemm_noalloc_max_scratch(void);
/* dfl_q41_gemm_status for the static array of the current device. */
int dfl_q41_gemm_noalloc_status(void *cuda_stream);
/* Look the current device's array up again and zero all of it (cudaMemsetAsync on the given stream):
 * after a context teardown, or to start from a known state. Must not overlap a product on the GPU. */
int dfl_q41_gemm_noalloc_reset(void *cuda_stream);

/* ---- a key/value cache in 8 bits: rows in, attention over it, eviction, rows out ------------------- */

/* The fp32 planes of the step take 4 bytes a value. This cache takes one: it holds blocks of
 * DFL_KV8_BLOCK tokens per key/value head as unsigned codes with one fp32 scale for the block's keys and
 * one for its values:  value = (code - 128) * scale,  scale = amax / 127 rounded to fp32 (amax = the
 * largest magnitude of the block's tokens x head_dim values),  code = 128 + the integer nearest to
 * value / scale (ties to even, limited to -127..127; 128 where the scale is 0). A block that holds an
 * infinity or a NaN gets the scale NaN and codes 128. Attention rows that see one of its tokens (or, in the
 * tail, a token that holds an infinity or a NaN) get NaN; the others are not touched by it.
 * The newest tokens, which are not a complete block yet or may still be rolled back, stay fp32 in a tail
 * of DFL_KV8_TAIL rows, so a verify's rows are never quantised before they are committed and a block is
 * quantised once, from its original rows.
 *
 * Everything is DEVICE memory of the caller's, in these layouts (all 16-byte aligned); the calls below
 * read the struct on the host and enqueue on the stream given. Lengths are device arrays, int32 [n_seq],
 * so that a captured graph replays at any position; `len` counts a sequence's committed tokens and is
 * never written here (layers of one model share it): the caller adds the rows that it commits. `cnt`
 * (nullable: `rows` for every sequence) holds each sequence's rows of this call; values outside 0..rows
 * are limited to it, and rows behind it are neither read nor written. */
#define DFL_KV8_BLOCK 32
#define DFL_KV8_TAIL 48
typedef struct dfl_kv8 {
    int32_t n_seq, n_kv, head_dim, n_blocks;  /* head_dim 64, 128 or 256; capacity 32 * n_blocks tokens
                                                 a sequence; n_seq <= 65535, n_kv <= 1024,
                                                 n_blocks <= 2^20 */
    uint8_t *k;         /* [n_seq][n_kv][n_blocks][head_dim/64][32 tokens][64] */
    uint8_t *v;         /* [n_seq][n_kv][n_blocks][head_dim][32 tokens] */
    float *k_scale;     /* [n_seq][n_kv][n_blocks], of the block stored there */
    float *v_scale;
    float *k_tail;      /* [n_seq][n_kv][48 tokens][head_dim]: the tokens from 32 * sealed on */
    float *v_tail;      /* [n_seq][n_kv][head_dim][48 tokens] */
    int32_t *table;     /* [n_seq][n_kv][n_blocks]: where logical block b is stored; a permutation of
                           0..n_blocks-1 */
    int32_t *sealed;    /* [n_seq][n_kv]: logical blocks held as codes */
    float *score;       /* [n_seq][n_kv][n_blocks]: attention weight that logical block b has received
                           (nullable: a cache without scores) */
    int32_t *err;       /* [1] sticky error bits, read and cleared by dfl_kv8_status */
} dfl_kv8;

/* An empty cache: table = identity, sealed, score and err = 0. Codes, scales and tails need no values. */
int dfl_kv8_init(const dfl_kv8 *c, void *cuda_stream);
/* Status of the calls enqueued on a cache so far: synchronises the stream, then DFL_OK, or (clearing the
 * word) one of these. DFL_E_CAPACITY: a sequence's len + rows passed the capacity or was negative.
 * DFL_E_STATE: a len lay further behind the sealed blocks than the tail reaches (tokens that no call has
 * written), or does not hold what is sealed where a call does not cut back (attn, evict), or the sealed counts
 * of a sequence's heads differ where a call needs them equal (evict; attn leaves the heads that differ from the
 * first). DFL_E_INVALID_ARG: a table entry or a sealed count outside 0..n_blocks. A sequence (or head) with
 * such a fault was left as it was by the call that met it, its output rows among them; a read leaves out only
 * the blocks whose entries are bad. Calls leave the heads of a sequence with equal counts, except where a bad
 * entry kept one head from going on with the others. */
int dfl_kv8_status(const dfl_kv8 *c, void *cuda_stream);
/* Append committed rows (a prompt's, or a draft's context): rows k, v (DEVICE fp32, row m of sequence s
 * at k + (s * rows + m) * ld, [n_kv][head_dim] each; ld in floats, a multiple of 4, >= n_kv * head_dim)
 * become tokens len..len+cnt-1. Blocks that are complete are sealed, the rest stays in the tail. Where
 * more is sealed than len holds, the cache is first cut back to len (the tokens of the block that the
 * cut goes through return to the tail as the values of their codes). Scores of blocks that begin among
 * the new rows start at 0. The caller then adds cnt to len. */
int dfl_kv8_append(const dfl_kv8 *c, const int32_t *len, const int32_t *cnt, int rows, const float *k,
                   const float *v, int64_t ld, void *cuda_stream);
/* Stage at most DFL_MAX_ROWS rows that may still be rolled back (a verify's, or a draft block's): first
 * seals the block that the commits since the last call completed, then writes the rows into the tail as
 * tokens len..len+cnt-1. To commit the first r of them the caller adds r to len; to roll the others back
 * it does nothing. Cuts back like dfl_kv8_append. */
int dfl_kv8_stage(const dfl_kv8 *c, const int32_t *len, const int32_t *cnt, int rows, const float *k,
                  const float *v, int64_t ld, void *cuda_stream);
/* Scratch bytes that dfl_kv8_attn needs for n_q query heads, rows, window and score, or -1 for a shape it does
 * not take. */
int64_t dfl_kv8_attn_scratch_bytes(const dfl_kv8 *c, int n_q, int rows, int window, int score);
/* Grouped-query attention of the staged rows (1..DFL_MAX_ROWS) over the cache:
 *   out[s][m][h] = sum_j softmax_j(scale * q[s][m][h] . k_j) v_j,  key/value head h / (n_q / n_kv).
 * Row m of sequence s sits at position p = len + m. causal != 0: it sees the tokens j <= p, with
 * window > 0 only j > p - window. causal == 0 (a draft's block): every row sees the tokens len - window
 * <= j < len (all of them with window = 0) and all cnt staged ones. n_q / n_kv is at most 16. q and out
 * are DEVICE fp32, row m of sequence s at (s * rows + m) * ld, [n_q][head_dim] each. score != 0 adds each
 * logical block's share of row 0's weights, summed over the head's group of query heads in a fixed order,
 * to c->score (row 0 is the one row of a verify that is always committed; weights come from queries and
 * keys, so values that are not finite make outputs NaN but no score). Sums and softmax statistics
 * are fp32; queries and weights enter the tensor cores as two fp16 halves each, which hold 22 bits.
 * What a token adds is held to about 2^-32 of the row's largest weight times its own value, whatever the
 * values of other tokens, seen or not; the sums stay finite for values up to 2^87. One call gives the same
 * bits each time.
 * Where heads, rows and sequences are so many that a call shares its work out evenly (n_seq * n_kv * groups
 * of 8 or 16 rows above 152, above 76 for 9 rows and more of 256 channels, and less where the capacity is
 * long), the last bits of a sequence may depend on the other sequences' lengths, as they decide where its
 * sums are cut; below that they depend on nothing else in the batch. len must not lie below what is sealed
 * (dfl_kv8_stage cuts back). out overlaps none of the inputs. Calls on one scratch (DEVICE, 256-byte
 * aligned) must not overlap on the GPU; nothing is kept in it from one call to the next. */
int dfl_kv8_attn(const dfl_kv8 *c, const float *q, int64_t ldq, int n_q, int rows, const int32_t *len,
                 const int32_t *cnt, int window, int causal, float scale, int score, float *out, int64_t ldo,
                 void *scratch, size_t scratch_bytes, void *cuda_stream);
/* Evict whole blocks (the unit that shares a scale, so no code changes and none moves): of each head's
 * sealed blocks keep at most `keep`: the first `sink`, the last `recent`, and of the others those with the
 * largest scores (equal scores: the lower index; a NaN counts as the smallest), in their order. Needs
 * sink + recent <= keep. Writes, for every head, the table (kept blocks, then those evicted, which are
 * free again, then the rest as it was), the scores (kept ones, the two blocks that the tail holds, zeros)
 * and the sealed count to table_out, score_out and sealed_out, and len - 32 * (blocks evicted) to len_out
 * (all DEVICE, shaped like c's and len; they overlap neither each other nor an input). The caller goes on
 * with these. A sequence whose len lies below what is sealed, or more than the tail behind it, keeps all
 * it has (the outputs are its inputs; DFL_E_STATE). Tokens then have new positions in the cache, which len, windows and causality count by; a
 * model's rotary positions are the caller's own. */
int dfl_kv8_evict(const dfl_kv8 *c, const int32_t *len, int keep, int sink, int recent, int32_t *table_out,
                  float *score_out, int32_t *sealed_out, int32_t *len_out, void *cuda_stream);
/* Read rows out in fp32: tokens first..first+rows-1 of each sequence (first: int32 [n_seq], nullable: 0),
 * as far as they lie below len, to k_out and v_out (DEVICE fp32 [n_seq][rows][n_kv][head_dim]); entries of
 * other tokens are left as they were. A len that counts staged rows reads these too. */
int dfl_kv8_read(const dfl_kv8 *c, const int32_t *len, const int32_t *first, int rows, float *k_out,
                 float *v_out, void *cuda_stream);

/* ---- a paged key/value cache in 16 bits: pages planned from lengths, rows in, attention ------------ */

/* dfl_kv8 gives every sequence its whole capacity. This cache is one pool of pages that sequences of any
 * lengths share, in bf16 or fp16. A page holds `page` tokens of every key/value head; a sequence's tokens lie
 * in the pages that its row of the table names, in order. A step over it:
 *   dfl_paged_plan(len, cnt)       which pages each sequence needs for its len tokens and cnt new rows
 *   dfl_paged_append(slots)        a layer's new keys and values into their pages
 *   dfl_paged_prompt               attention of whole prompts among their own rows, or
 *   dfl_paged_attn                 attention of a token, or of a verify's rows, over the pages
 * The caller then adds the rows that it keeps to len; the others' places are written again by the next step
 * (a rollback is index arithmetic). A sequence that has ended gets len = cnt = 0, and its pages go back.
 * The layers of a model that share lengths share the plan: one table, held, ring and queue, a k and v each.
 *
 * Rows of a call (at most 2^30) are packed: sequence s has rows cu[s] .. cu[s+1]-1 (cu: DEVICE int32 [n_seq+1])
 * of buffers [rows][heads][head_dim], row r at r * ld elements (at most 2^22), heads and channels contiguous. Rows from cu[n_seq] on
 * are neither read for anything that shows nor written.
 *
 * Everything is DEVICE memory of the caller's; the calls read the struct on the host and enqueue on the
 * stream given. k and v are 16-byte aligned, the int32 arrays 4-byte aligned. */
#define DFL_PAGED_MAX_SEQ 4096
enum { DFL_BF16 = 0, DFL_F16 = 1 };
typedef struct dfl_paged {
    int32_t n_seq, n_kv, head_dim;   /* n_seq <= DFL_PAGED_MAX_SEQ, n_kv <= 1024, head_dim 64, 128 or 256 */
    int32_t page;                    /* tokens of a page: 16, 32, 64 or 128 */
    int32_t n_pages, max_pages;      /* of the pool, and of one sequence; both times page at most 2^30 */
    int32_t type;                    /* DFL_BF16 or DFL_F16: of k, v and the rows of all calls */
    void *k, *v;                     /* [n_pages][n_kv][page][head_dim] */
    int32_t *table;                  /* [n_seq][max_pages]: the page of each `page` tokens; entries from held on
                                        mean nothing */
    int32_t *held;                   /* [n_seq]: pages that a sequence has */
    int32_t *ring;                   /* [n_pages]: the pages that no sequence has, a ring: queue[1] of them
                                        from place queue[0] on */
    int32_t *queue;                  /* [4]: where the ring begins, the pages in it, and two words of the
                                        library's, which are 0 between calls */
    int32_t *err;                    /* [1] sticky error bits, read and cleared by dfl_paged_status */
} dfl_paged;

/* An empty cache: no sequence holds a page, the ring has all of them in order, err = 0. */
int dfl_paged_init(const dfl_paged *c, void *cuda_stream);
/* Status of the calls enqueued on a cache so far: synchronises the stream, then DFL_OK, or (clearing the word)
 * the first of these that a call met. DFL_E_TIMEOUT: a bounded device wait of dfl_paged_prompt gave up, and its
 * output is undefined. DFL_E_INVALID_ARG: a row count out of order (cu descending or past the buffers, a negative
 * len or cnt, more rows of a sequence than the call's `rows`), a slot past the pool, or a table or ring entry
 * outside 0..n_pages-1. DFL_E_STATE: held or the queue out of order, or attention over tokens that the sequence has
 * no pages for, or over 2^36 tokens and more in one call. DFL_E_CAPACITY: a sequence longer than max_pages, more rows than slots, or no pages left. */
int dfl_paged_status(const dfl_paged *c, void *cuda_stream);
/* Plan a step: sequence s is to hold ceil((len + cnt) / page) pages. What it has beyond them goes to the ring's
 * end, then what it lacks comes from the ring's front, both in the order of the sequences and of their pages, so
 * that a plan is the same each time. Writes
 *   cu     [n_seq+1]  sums of cnt: where each sequence's rows begin (limited to `rows`)
 *   slots  [rows]     each row's place, page * (tokens of a page) + the token's place in it, and -1 for rows
 *                     behind the last sequence's (a captured graph's spare ones)
 * A sequence that a plan cannot serve keeps the pages that it has, and its rows have slots -1: with DFL_E_CAPACITY one
 * longer than max_pages, one whose rows reach past `rows` and all behind it (those without rows too: what has ended gives
 * its pages back in the next plan whose rows fit), and one whose pages are not there (after it no sequence of the call
 * gets new pages); a negative len or cnt (DFL_E_INVALID_ARG) counts as no rows.
 * A plan takes steps of any kind, but each attention below one kind: rows of whole prompts, or at most DFL_MAX_ROWS rows
 * a sequence behind the tokens that it has. Where requests of both kinds are there, they are two steps: the prompts with
 * cnt = 0 for the others, whose len keeps their pages, then the others with the prompts' rows in len.
 * len and cnt: int32 [n_seq]; cu and slots share no memory with anything else. Calls of a cache must not overlap on
 * the GPU. */
int dfl_paged_plan(const dfl_paged *c, const int32_t *len, const int32_t *cnt, int32_t *cu, int32_t *slots, int rows,
                   void *cuda_stream);
/* Rows k, v (row r at r * ldk, r * ldv elements, [n_kv][head_dim] each; 16-byte aligned, ld a multiple of 8) into
 * the places of slots[0..rows-1]; a negative slot's row is left out. Two rows of one call must not have one slot
 * (a plan's have not).
 * k and v lie outside the pages. */
int dfl_paged_append(const dfl_paged *c, const int32_t *slots, int rows, const void *k, int64_t ldk, const void *v,
                     int64_t ldv, void *cuda_stream);
/* Causal grouped-query attention of packed prompts among their own rows (of a sequence's first tokens; the cache's
 * pages are not read):  out[i][h] = sum_j softmax_j(scale * q[i][h] . k[j][h / g]) v[j][h / g],  g = n_q / n_kv at
 * most 16, over the rows j <= i of the same sequence, with window > 0 only j > i - window. scale > 0. The buffers
 * have `rows` rows, 16-byte aligned, ld multiples of 8. Scores (of any size that fp32 holds), softmax
 * statistics and sums are fp32; a row's weights are rounded once to the cache's type, as what the tensor cores take,
 * and the output once. A value that is not finite leaves nothing finite of its channel in the rows that see it, and
 * touches no other output. A key or query that is not finite counts by the scores that it makes: one of minus infinity
 * takes no weight, and a row that meets one of plus infinity or NaN, or nothing but minus infinity, is NaN. The sums
 * stay finite for values up to 2^90. out shares no memory with an input (rows may lie in the gaps of others that are as
 * far apart). Each row's bits depend on its own sequence alone. */
int dfl_paged_prompt(const dfl_paged *c, const void *q, int64_t ldq, int n_q, const void *k, int64_t ldk, const void *v,
                     int64_t ldv, const int32_t *cu, int rows, int window, float scale, void *out, int64_t ldo,
                     void *cuda_stream);
/* Tests of the error path only, for the whole process: the items of the following dfl_paged_prompt calls issue no more
 * than `copies` > 0 of their copies (of keys and values in turn), or with copies < 0 no more than -copies in the pass
 * over values that are not finite, so that their bounded waits give up after about a second. 0: as always. */
int dfl_paged_test_stall(int copies);
/* Scratch bytes that dfl_paged_attn needs for n_q query heads and at most `rows` rows a sequence, or -1 for a shape
 * it does not take. */
int64_t dfl_paged_attn_scratch_bytes(const dfl_paged *c, int n_q, int rows);
/* Grouped-query attention over the pages, of at most `rows` (1..DFL_MAX_ROWS) rows a sequence: row m of sequence s
 * (row cu[s] + m of q and out, which have `total` rows) sits at position p = len[s] + m. causal != 0: it sees the
 * tokens j <= p, with window > 0 only j > p - window. causal == 0 (a draft's block): every row sees the tokens
 * len - window <= j < len (all of them with window = 0) and all the sequence's new ones. The new rows' keys and
 * values are in the pages (dfl_paged_append). Numbers, groups and scale as for dfl_paged_prompt (up to
 * 16 rows x heads of a group, weights as two numbers of the type each). A sequence with
 * more rows than `rows`, or without the pages that it needs, is left as it is and reported; rows that see a page
 * whose table entry is bad get NaN (reported). out shares no memory with q or the pages. Calls on one scratch
 * (DEVICE, 256-byte aligned) must not overlap on the GPU; nothing is kept in it from one call to the next. One call
 * gives the same bits each time; the last bits of a sequence may depend on the other sequences' lengths, which
 * decide where its sums are cut. */
int dfl_paged_attn(const dfl_paged *c, const void *q, int64_t ldq, int n_q, int total, const int32_t *cu,
                   const int32_t *len, int rows, int window, int causal, float scale, void *out, int64_t ldo,
                   void *scratch, size_t scratch_bytes, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* DFL_H */
