/*
 * moe_mi355x.h — C interface of the sparse top-K routed MoE FFN forward
 * (renormalised gates, optional always-on shared experts) for MI355X (gfx950).
 *
 * Sources, cited by page title and section:
 *   [TopK]  "Sparse MoE Top-Kルーティング" glossary page (jisaku.com):
 *           section ルーティングの仕組み (router scores for every expert, keep
 *           the K best, masked re-softmax gives the gates, gate-weighted sum);
 *           section 解決策2: エキスパートキャパシティファクター (per-expert token
 *           limit, overflow tokens dropped / left to the residual).
 *   [DSMoE] "論文解説: DeepSeekMoE — 細粒度エキスパート分割と共有エキスパートによる
 *           MoE効率化" (0h-n0.github.io): section 共有エキスパート機構 (output
 *           equation: sum of shared experts plus gate-weighted routed experts);
 *           section ルーティングとバランス損失 (gate equation
 *           g_j = s_j / sum_{k in TopK} s_k, s = softmax(W_r x)); section
 *           アルゴリズム (layer arguments d_model, n_routed, n_shared, top_k,
 *           d_ff; router Linear without bias; expert Linear-SiLU-Linear).
 *   [EP]    "エキスパート並列（Expert Parallelism）" glossary page (jisaku.com):
 *           section 推論フロー (gate selects experts, tokens are sent to their
 *           experts, results are sent back); on one GPU that exchange is the
 *           on-device permutation below.
 *
 * Conventions shared by every entry point
 *   - Every pointer argument of type void*, float*, int32_t* that names a
 *     tensor is a DEVICE pointer owned by the caller; the library allocates
 *     nothing and keeps no state between calls.  `cfg` and `w` (the structs)
 *     are HOST pointers read during the call only.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Calls only enqueue work on it; none synchronises with the host and none
 *     copies device data to the host.  Results are ready when the stream is.
 *   - Tensors are dense and row-major in the shapes given; "act" denotes the
 *     activation / expert-weight type chosen by cfg->dtype (MOE_F32: float,
 *     MOE_BF16: bfloat16 bits).  Router weights, router bias, logits and
 *     gates are always float32.  Every device pointer must be 16-byte aligned.
 *   - Return value: MOE_OK, or a negative moe_status.  Argument errors are
 *     detected on the host before anything is enqueued.  Launch failures
 *     return MOE_ERR_HIP.  Device-side contents (for example an expert index
 *     outside [0, N) handed to moe_permute) are not validated; behaviour is
 *     then undefined.  No C++ exception crosses this interface.
 *   - T == 0 is a successful no-op.
 *   - Supported sizes: 1 <= top_k <= n_routed (top_k > n_routed or
 *     top_k < 1 is MOE_ERR_INVALID_ARG); n_routed <= 1024 and top_k <= 64
 *     (the top-K kernel keeps slot k of a token in lane k of one 64-wide
 *     wave, and the combine stages a token's slot rows in 64 entries);
 *     n_shared <= 64; d_model and d_ff multiples of 64 for MOE_BF16 (one
 *     64-element reduction step of the matrix-core kernels, 128 bytes) and of
 *     16 for MOE_F32; T * top_k < 2^31.  Sizes outside these limits return
 *     MOE_ERR_UNSUPPORTED.
 *
 * Numerical contract
 *   - Logits: float32, per (t, e) one fused multiply-add chain over k
 *     ascending starting at +0, then + router_bias[e] with one rounding
 *     (with MOE_BIAS_SELECTION_ONLY the bias is added to the selection key
 *     only).
 *   - Selection: the K largest logits, key (logit desc, expert id asc); slot
 *     k of a token holds its k-th best expert.
 *   - Gates: softmax over the K kept logits (float32), which equals
 *     s_j / sum_{k in TopK} s_k of [DSMoE] gate equation.
 *   - Capacity: C = cfg->capacity when >= 0, else ceil(cf * T * K / N)
 *     evaluated in double as ((cf * T) * K) / N when cf > 0, else no limit.
 *     An expert keeps its first C tokens in token order; a dropped
 *     (token, slot) contributes nothing; gates are not renormalised again.
 *   - Output: y_t = sum_i S_i(x_t) + sum_{k kept} g[t,k] * E_{idx[t,k]}(x_t),
 *     accumulated in float32, shared experts first, then k ascending; no
 *     residual term (that add belongs to the caller).
 *   - Expert E(z) = W2 SiLU(W1 z + b1) + b2; bf16 configurations round the
 *     hidden activations and the expert outputs to bf16, accumulate in fp32.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,   /* NULL where required, negative size, K > N ... */
    MOE_ERR_UNSUPPORTED = -2,   /* sizes outside the supported ranges above      */
    MOE_ERR_WORKSPACE = -3,     /* workspace missing or smaller than required    */
    MOE_ERR_HIP = -4            /* a HIP runtime call or kernel launch failed    */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

/* Layer shape ([DSMoE] アルゴリズム: d_model, n_routed, n_shared, top_k, d_ff). */
typedef struct {
    int64_t T;                /* tokens (batch * seq_len, flattened)              */
    int32_t d_model;          /* d                                                 */
    int32_t n_routed;         /* N routed experts                                  */
    int32_t top_k;            /* K experts kept per token                          */
    int32_t n_shared;         /* K_s always-active shared experts (may be 0)       */
    int32_t d_ff;             /* f, hidden width of every expert                   */
    int32_t dtype;            /* moe_dtype of x, expert weights/biases, hidden, y  */
    float capacity_factor;    /* <= 0: no factor-derived limit                     */
    int32_t capacity;         /* >= 0: explicit per-expert limit; -1: use factor   */
    int32_t bias_mode;        /* MOE_BIAS_IN_LOGIT or MOE_BIAS_SELECTION_ONLY      */
    int32_t dispatch;         /* MOE_DISPATCH_BF16 or MOE_DISPATCH_FP8             */
} moe_config;

/* Precision of the token rows the routed experts receive (the dispatch).
 *   MOE_DISPATCH_BF16: the rows as given (act dtype).
 *   MOE_DISPATCH_FP8: the FP8 dispatch of [DeepEP] ("DeepEP とは？" item 5;
 *     "DeepEP の性能": FP8 dispatch, BF16 combine).  Each token row is sent as
 *     OCP FP8 E4M3 codes (bias 7, 3 mantissa bits, largest value 448) with one
 *     power-of-two scale 2^E per row, E the smallest integer with
 *     max|x[t]| <= 448 * 2^E (0 for an all-zero row); codes are x / 2^E
 *     rounded to nearest, ties to even.  The pass that makes the codes (the
 *     payload an exchange between GPUs would carry) also widens them back,
 *     as the receiving side would, to bf16 rows of exactly 2^E * code value,
 *     and the routed experts' first Linear reads those rows through the
 *     dispatch permutation; the router and the shared experts use x; the
 *     combine is unchanged (bf16).  MOE_BF16 layers only
 *     (MOE_ERR_UNSUPPORTED otherwise); honoured by moe_layer_forward and
 *     moe_layer_forward_noalloc, ignored by the other entry points. */
enum { MOE_DISPATCH_BF16 = 0, MOE_DISPATCH_FP8 = 1 };

/* How router_bias enters the routing.
 *   MOE_BIAS_IN_LOGIT: the bias is part of the logit, for selection and gates.
 *   MOE_BIAS_SELECTION_ONLY: the bias-based balancing of [TopK] section
 *     負荷均衡 (steers the load without changing the loss): selection uses the
 *     key fl32(logit + bias[e]); the gates are the softmax over the K kept
 *     unbiased logits, and the logits written are the unbiased ones. */
enum { MOE_BIAS_IN_LOGIT = 0, MOE_BIAS_SELECTION_ONLY = 1 };

/* Expert and router weights, nn.Linear layout (out_features, in_features). */
typedef struct {
    const float *w_router;    /* [N][d] float32                                   */
    const float *router_bias; /* [N] float32 or NULL                              */
    const void *w1;           /* [N][f][d] act                                    */
    const void *b1;           /* [N][f] act or NULL                               */
    const void *w2;           /* [N][d][f] act                                    */
    const void *b2;           /* [N][d] act or NULL                               */
    const void *ws1;          /* [K_s][f][d] act (NULL when K_s == 0)             */
    const void *bs1;          /* [K_s][f] act or NULL                             */
    const void *ws2;          /* [K_s][d][f] act (NULL when K_s == 0)             */
    const void *bs2;          /* [K_s][d] act or NULL                             */
} moe_weights;

/*
 * moe_route — router scores, top-K selection and renormalised gates
 * ([TopK] ルーティングの仕組み; [DSMoE] gate equation).
 *   x           [T][d] act
 *   w_router    [N][d] float32;  router_bias [N] float32 or NULL (part of the
 *               logit for both selection and gates)
 *   logits      [T][N] float32 output, required: the top-K pass reads the
 *               logits back from here.  The logits of one token are computed
 *               by many workgroups (one logit per lane, each a d-long fixed
 *               order chain), so no single workgroup holds a token's N
 *               logits on chip; a pass that did would serialise N/64 of those
 *               chains per wave, far slower than this T*N*4-byte round trip
 *               (4 MB, under a microsecond of HBM time, at 4096 tokens and
 *               256 experts).
 *   topk_idx    [T][K] int32 output, expert ids in slot order
 *   topk_gate   [T][K] float32 output, sums to 1 per token
 */
int moe_route(const moe_config *cfg, const void *x, const float *w_router,
              const float *router_bias, float *logits, int32_t *topk_idx,
              float *topk_gate, void *stream);

/*
 * moe_permute — dispatch as an on-device permutation: per-expert histogram,
 * capacity clip, exclusive scan, stable scatter ([EP] 推論フロー steps 2-3 on
 * one GPU; [TopK] capacity section).
 *   topk_idx    [T][K] int32 input, values in [0, N)
 *   x           [T][d] act input, read only when x_perm != NULL
 *   counts      [N] int32 output: kept rows per expert
 *   offsets     [N+1] int32 output: exclusive scan of counts
 *   row_token   [T*K] int32 output: rows 0..offsets[N]-1 hold the token of
 *               each row, experts in order, tokens ascending within one
 *   slot_row    [T*K] int32 output: row of (t, k), or -1 when dropped
 *   n_dropped   [1] int32 output
 *   x_perm      [T*K][d] act output (rows 0..offsets[N]-1) or NULL to skip
 *   ws          device workspace of moe_permute_workspace_size(cfg) bytes
 */
int moe_permute(const moe_config *cfg, const int32_t *topk_idx, const void *x,
                int32_t *counts, int32_t *offsets, int32_t *row_token, int32_t *slot_row,
                int32_t *n_dropped, void *x_perm, void *ws, size_t ws_bytes, void *stream);
size_t moe_permute_workspace_size(const moe_config *cfg);

/*
 * moe_grouped_ffn — every group's expert FFN over its contiguous rows:
 * rows offsets[g] .. offsets[g+1]-1 get E_g(x_rows[r]) ([DSMoE] アルゴリズム,
 * expert Linear(d, f) - SiLU - Linear(f, d)).
 *   n_groups    number of experts in w1/w2 (>= 1)
 *   x_rows      [max_rows][d] act input
 *   offsets     [n_groups+1] int32 DEVICE array, non-decreasing, offsets[0]=0
 *   max_rows    host-side upper bound on offsets[n_groups].  The offsets
 *               stay on the device (no call copies them back), so the host
 *               sizes the persistent launch and the split scratch from this
 *               bound; the kernels read the true row counts on the device.
 *               Rows at or beyond offsets[n_groups] are neither read nor
 *               written; offsets[n_groups] > max_rows is undefined.
 *   w1 [G][f][d], b1 [G][f] or NULL, w2 [G][d][f], b2 [G][d] or NULL (act)
 *   h           [max_rows][f] act output (hidden activations)
 *   y_rows      [max_rows][d] act output
 *   ws          optional device scratch of moe_grouped_ffn_workspace_size
 *               bytes (NULL allowed); with it, products with too few row
 *               blocks to fill the GPU are split along their reduction
 *               dimension and the parts summed in a fixed order.  A non-NULL
 *               ws smaller than that size is MOE_ERR_WORKSPACE.
 * Only cfg->d_model, cfg->d_ff and cfg->dtype are read.
 */
int moe_grouped_ffn(const moe_config *cfg, int32_t n_groups, const void *x_rows,
                    const int32_t *offsets, int64_t max_rows, const void *w1, const void *b1,
                    const void *w2, const void *b2, void *h, void *y_rows, void *ws,
                    size_t ws_bytes, void *stream);
size_t moe_grouped_ffn_workspace_size(const moe_config *cfg, int32_t n_groups,
                                      int64_t max_rows);

/*
 * moe_combine — y_t = sum_i S_i[t] + sum_{k: slot_row[t,k] >= 0}
 * g[t,k] * y_rows[slot_row[t,k]] ([DSMoE] 共有エキスパート機構 equation).
 *   y_rows      [*][d] act, indexed by slot_row
 *   slot_row    [T][K] int32, topk_gate [T][K] float32
 *   shared_out  [K_s][T][d] act or NULL (K_s from cfg->n_shared)
 *   y           [T][d] act output
 */
int moe_combine(const moe_config *cfg, const void *y_rows, const int32_t *slot_row,
                const float *topk_gate, const void *shared_out, void *y, void *stream);

/*
 * moe_layer_forward — the whole layer of [DSMoE] 共有エキスパート機構 (output
 * equation: the shared experts' sum plus the gate-weighted routed experts),
 * with the routing of [TopK] ルーティングの仕組み and [DSMoE] gate equation and
 * the capacity limit of [TopK] 解決策2: route, permute (the gather is fused
 * into the first expert GEMM), routed and shared expert FFNs, combine.
 *   x [T][d] act input, y [T][d] act output.
 *   topk_idx, topk_gate ([T][K]) and counts ([N]) are optional outputs of the
 *   routing (NULL to skip).  When one is given, the layer writes that array
 *   there instead of into its workspace region.
 *   ws          device workspace of moe_workspace_size(cfg) bytes.  After the
 *               call has run on the stream, the regions named by
 *               moe_workspace_layout hold the layer's routing: logits,
 *               offsets, n_dropped, row_token and slot_row always, and
 *               topk_idx, topk_gate and counts when their optional output is
 *               NULL.  The rest of ws is scratch.
 */
int moe_layer_forward(const moe_config *cfg, const moe_weights *w, const void *x, void *y,
                      int32_t *topk_idx, float *topk_gate, int32_t *counts,
                      void *ws, size_t ws_bytes, void *stream);

/*
 * moe_layer_forward_noalloc — moe_layer_forward for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc): the same stages and kernels, with the
 * workspace taken from a library-owned device array instead of `ws`.
 *   - The array holds MOE_NOALLOC_SCRATCH_BYTES (64 MiB) per GPU, from the
 *     first use of the library on that GPU until the process ends.  The
 *     call allocates nothing (no hipMalloc, hipFree or allocating library
 *     routine); its first call on a device looks up the array's address there.
 *   - A layer whose workspace, without the expert GEMMs' optional K-split
 *     scratch, exceeds that size returns MOE_ERR_WORKSPACE before anything is
 *     enqueued.  The K-split scratch gets what is left (a DeepSeek-V3-shaped
 *     decode layer of 128 tokens needs about 22 MB plus 32 MB of it); with
 *     less, fewer products are split.  Batches of a few hundred tokens at
 *     DeepSeek-V3 widths fit; 4096-token prefill layers do not.
 *   - Every call on one GPU uses that GPU's one array.  Calls that overlap on
 *     one GPU (on different streams, or from several host threads without
 *     ordering) race and give undefined results; calls on one stream are
 *     ordered and safe.  Each call writes every part of the array it later
 *     reads, so nothing left by an earlier call is used.
 *   Arguments as moe_layer_forward; the routing arrays are not readable
 *   through moe_workspace_layout here (pass topk_idx, topk_gate, counts).
 */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int moe_layer_forward_noalloc(const moe_config *cfg, const moe_weights *w, const void *x,
                              void *y, int32_t *topk_idx, float *topk_gate, int32_t *counts,
                              void *stream);

/* Bytes of device workspace moe_layer_forward needs for cfg (0 when cfg is
 * invalid or unsupported). */
size_t moe_workspace_size(const moe_config *cfg);

/* Byte offsets, from the start of moe_layer_forward's workspace, of the
 * routing arrays the layer leaves there (shapes as in moe_permute; every
 * offset is a multiple of 256). */
typedef struct {
    size_t logits;      /* [T][N] float32                                     */
    size_t topk_idx;    /* [T][K] int32                                       */
    size_t topk_gate;   /* [T][K] float32                                     */
    size_t counts;      /* [N] int32: kept rows per expert                    */
    size_t offsets;     /* [N+1] int32                                        */
    size_t n_dropped;   /* [1] int32                                          */
    size_t row_token;   /* [T*K] int32 (rows 0 .. offsets[N]-1 hold tokens)   */
    size_t slot_row;    /* [T][K] int32 (-1 = dropped)                        */
    size_t x_fp8;       /* MOE_DISPATCH_FP8: [T][d] uint8 E4M3 codes, else 0  */
    size_t x_fp8_exp;   /* MOE_DISPATCH_FP8: [T] int32 scale exponents, else 0 */
    size_t x_fp8_wide;  /* MOE_DISPATCH_FP8: [T][d] bf16, the codes widened back
                           (2^E times each code's value: the rows the first
                           Linear reads), else 0                             */
    size_t total;       /* moe_workspace_size(cfg)                            */
} moe_ws_layout;

/* Fills *out for cfg; MOE_OK, or the status moe_layer_forward would return
 * for cfg's shape. */
int moe_workspace_layout(const moe_config *cfg, moe_ws_layout *out);

/* Stages of moe_layer_forward, in launch order. */
enum {
    MOE_STAGE_ROUTER = 0,   /* router logits                                   */
    MOE_STAGE_TOPK = 1,     /* top-K selection and gates                       */
    MOE_STAGE_DISPATCH = 2, /* histogram, scan, scatter                        */
    MOE_STAGE_UP = 3,       /* first Linear + SiLU, routed and shared experts  */
    MOE_STAGE_DOWN = 4,     /* second Linear, routed and shared experts        */
    MOE_STAGE_COMBINE = 5,  /* gate-weighted sum + shared outputs              */
    MOE_STAGE_COUNT = 6
};

/*
 * moe_layer_forward_events — moe_layer_forward that also records caller-owned
 * HIP events on `stream` at every stage boundary, for timing the stages on the
 * stream they run on.  stage_events points to MOE_STAGE_COUNT + 1 hipEvent_t
 * handles (as void*): event i is recorded just before stage i is launched and
 * event MOE_STAGE_COUNT after the last one.  NULL behaves like
 * moe_layer_forward.  The events are only recorded, never waited on.
 */
int moe_layer_forward_events(const moe_config *cfg, const moe_weights *w, const void *x,
                             void *y, int32_t *topk_idx, float *topk_gate, int32_t *counts,
                             void *ws, size_t ws_bytes, void *const *stage_events,
                             void *stream);

/*
 * moe_balance_stats — load statistics of one routing ([DSMoE] section
 * ルーティングとバランス損失, balance-loss equation):
 *   f[j]  = (number of (t, k) with topk_idx[t][k] == j) / (T * K)
 *   P[j]  = (1/T) * sum_t softmax(logits[t])_j   (softmax over all N)
 *   *loss = alpha * N * sum_j f[j] * P[j]
 *   logits      [T][N] float32 (as written by moe_route)
 *   topk_idx    [T][K] int32, values in [0, N)
 *   f, P        [N] float32 outputs; loss [1] float32 output (device)
 *   ws          device workspace of moe_balance_stats_workspace_size(cfg) bytes
 * Counts are exact; P and the loss are float32 sums in a fixed order, so the
 * results do not depend on timing.  Only T, n_routed and top_k are read.
 */
int moe_balance_stats(const moe_config *cfg, const float *logits, const int32_t *topk_idx,
                      float alpha, float *f, float *P, float *loss, void *ws, size_t ws_bytes,
                      void *stream);
size_t moe_balance_stats_workspace_size(const moe_config *cfg);

/*
 * MXFP4 — rows of 4-bit floating point with a scale for every 32 elements.
 *   codes   [rows][d/2] uint8: E2M1 codes (sign, 2 exponent bits with bias 1,
 *           1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives), element
 *           2i in the low four bits of byte i and element 2i+1 in the high four
 *   scales  [rows][d/32] uint8: byte B stands for 2^(B - 127), 255 for NaN
 * Weights are quantised along their reduction axis (the last one of the
 * nn.Linear layout), so a stack [G][out][in] is G * out rows of d = in.
 */

/*
 * moe_quantize_mxfp4 — rows to MXFP4.  The rule is the FP8 dispatch's: per
 * block of 32 elements the scale is 2^E, E the smallest integer with
 * max|x| <= 6 * 2^E (0 for a block of zeros, at least -127), and a code is
 * x / 2^E rounded to the nearest value, ties to the even code; nothing is
 * clipped.  A block that holds an infinity or a NaN gets scale byte 255 and
 * codes 0.
 *   dtype       moe_dtype of x and widened
 *   x           rows of d elements, x_stride elements apart (x_stride >= d; a
 *               row starts on a 16-byte boundary, so x_stride is a multiple
 *               of 8 for MOE_BF16 and of 4 for MOE_F32; ignored for one row)
 *   widened     [rows][d] dtype output or NULL: the values the codes stand
 *               for, 2^E times each code's value (exact unless the product
 *               leaves the type's range: a block whose largest element is
 *               above 1.75 * 2^127 widens that element to infinity; blocks
 *               marked NaN widen to NaN)
 * d is a multiple of 32 (else MOE_ERR_UNSUPPORTED); rows * d < 2^42.
 */
int moe_quantize_mxfp4(int32_t dtype, int64_t rows, int32_t d, const void *x, int64_t x_stride,
                       uint8_t *codes, uint8_t *scales, void *widened, void *stream);

/*
 * moe_grouped_linear_mxfp4 — one Linear of every group's expert on MXFP4
 * rows and MXFP4 weights, on the scaled matrix instructions:
 *   y_rows[r] = act(X[row_index[r]] W_g^T + bias_g),  offsets[g] <= r < offsets[g+1]
 * with float32 sums, rounded to bf16 once.  A block whose scale byte is 255
 * makes the outputs it enters NaN.  Equal calls give equal bits; the order of a
 * row's sums depends on how many rows all groups have.
 *   x_rows      rows of x_codes and x_scales, the token rows (k elements each)
 *   row_index   [max_rows] int32 or NULL: source row of each row (a dispatch's
 *               row_token, so that a token is quantised once however many
 *               experts it meets), values in [0, x_rows); NULL: row r reads
 *               source row r, and x_rows >= max_rows
 *   offsets     [n_groups+1] int32 DEVICE array, non-decreasing, offsets[0]=0
 *   max_rows    host-side upper bound on offsets[n_groups], as for
 *               moe_grouped_ffn; rows at or beyond offsets[n_groups] are
 *               neither read nor written
 *   w_codes [G][n_out][k/2], w_scales [G][n_out][k/32]
 *   bias        [G][n_out] bf16 or NULL;  silu 1: act = SiLU, 0: none
 *   y_rows      [max_rows][n_out] bf16 output
 *   ws          device scratch of moe_grouped_linear_mxfp4_workspace_size
 *               bytes.  That is 0 in this version: ws may be NULL, and calls may
 *               overlap in time.
 * k is a multiple of 128 (one step of the matrix instruction) and n_out of 8
 * (16-byte output rows), n_groups <= 1088, and the codes of all token rows
 * and those of one group's matrix take less than 4 GiB each (32-bit offsets);
 * else MOE_ERR_UNSUPPORTED.
 */
int moe_grouped_linear_mxfp4(int32_t n_groups, int32_t n_out, int32_t k, int64_t x_rows,
                             const uint8_t *x_codes, const uint8_t *x_scales,
                             const int32_t *row_index,
                             const int32_t *offsets, int64_t max_rows, const uint8_t *w_codes,
                             const uint8_t *w_scales, const void *bias, int32_t silu, void *y_rows,
                             void *ws, size_t ws_bytes, void *stream);
size_t moe_grouped_linear_mxfp4_workspace_size(int32_t n_groups, int32_t n_out, int32_t k,
                                               int64_t max_rows);

/*
 * moe_layer_forward_few — moe_layer_forward for 1 to MOE_FEW_TOKENS tokens (a
 * decode step) in two kernels instead of one per stage.  Arguments, shapes,
 * capacity rule and optional outputs as moe_layer_forward, with these
 * differences:
 *   - T > MOE_FEW_TOKENS, cfg->dispatch == MOE_DISPATCH_FP8, an expert matrix
 *     of 4 GiB or more in cfg->dtype, and T * (top_k + n_shared) + 1 hidden rows
 *     of 2^30 elements or more together (d_ff rounded up to 64 for MOE_F32)
 *     return MOE_ERR_UNSUPPORTED;
 *   - the logits are float32 sums in a fixed tree order, not moe_route's
 *     chain, so two experts whose logits differ by no more than their rounding
 *     may be ordered differently than there; ties still go to the lower id;
 *   - hidden activations keep at least 16 significant bits (float32 layers:
 *     all; one too large for bf16 is not finite in a bf16 layer, as in
 *     moe_layer_forward) and expert outputs are not rounded before the sum over
 *     experts: y is rounded once.  Routed experts are summed in ascending expert
 *     id, the shared experts after them;
 *   - ws holds moe_few_workspace_size(cfg) bytes, all scratch.  Nothing in it
 *     needs to be initialised.  Calls that overlap in time (other streams,
 *     parallel branches of a graph) need a workspace of their own each.
 * Equal calls give equal bits; where a token's sums are cut depends on the experts
 * that all tokens of the call meet, so in another batch its last bits may differ.
 * A weight or token element that is not finite
 * reaches the tokens it enters and no others (their outputs may be NaN where a sum
 * would be infinite).  A call takes no longer for a token or hidden value that is not
 * finite; an infinity or NaN among the weights of a second Linear costs it up to some
 * milliseconds, as the sums it enters are added up again one element after the other.
 */
#define MOE_FEW_TOKENS 16
int moe_layer_forward_few(const moe_config *cfg, const moe_weights *w, const void *x, void *y,
                          int32_t *topk_idx, float *topk_gate, int32_t *counts, void *ws,
                          size_t ws_bytes, void *stream);

/* Device workspace of the two few-token calls (0 when cfg is invalid or
 * unsupported there). */
size_t moe_few_workspace_size(const moe_config *cfg);

/* moe_weights with the expert matrices in MXFP4 (codes and scale bytes);
 * biases are bf16. */
typedef struct {
    const float *w_router;      /* [N][d] float32                               */
    const float *router_bias;   /* [N] float32 or NULL                          */
    const uint8_t *w1;          /* [N][f][d/2] codes                            */
    const uint8_t *w1_scales;   /* [N][f][d/32]                                 */
    const void *b1;             /* [N][f] bf16 or NULL                          */
    const uint8_t *w2;          /* [N][d][f/2] codes                            */
    const uint8_t *w2_scales;   /* [N][d][f/32]                                 */
    const void *b2;             /* [N][d] bf16 or NULL                          */
    const uint8_t *ws1;         /* [K_s][f][d/2] (NULL when K_s == 0)           */
    const uint8_t *ws1_scales;  /* [K_s][f][d/32]                               */
    const void *bs1;            /* [K_s][f] bf16 or NULL                        */
    const uint8_t *ws2;         /* [K_s][d][f/2] (NULL when K_s == 0)           */
    const uint8_t *ws2_scales;  /* [K_s][d][f/32]                               */
    const void *bs2;            /* [K_s][d] bf16 or NULL                        */
} moe_weights_mxfp4;

/* moe_layer_forward_few on MXFP4 expert weights.  The codes go into the scaled
 * matrix instructions as they are, against tokens and hidden rows as sums of
 * E4M3 parts with a power-of-two scale for every 32 elements:
 *   tokens  two parts, exact for a bf16 element down to 2^-13 of the largest of
 *           its 32, and within 2^-21 of that largest below;
 *   hidden  three parts, the rest at most 2^-12 of the element or 2^-25 of the
 *           largest of its 32.
 * That is for a largest of 2^-111 or more; below, tokens are off by at most 2^-133 and
 * hidden values by 2^-137.
 * cfg->dtype is MOE_BF16 and d_model and d_ff are multiples of 128, else
 * MOE_ERR_UNSUPPORTED. */
int moe_layer_forward_few_mxfp4(const moe_config *cfg, const moe_weights_mxfp4 *w, const void *x,
                                void *y, int32_t *topk_idx, float *topk_gate, int32_t *counts,
                                void *ws, size_t ws_bytes, void *stream);

/*
 * Training the layer as a block of a model.  The calls below are the single
 * Linears of the experts with their gradients, the block around the layer
 * (norms, gate, residual) with its gradients, and dropout.  A step goes
 *   moe_block_join (first norm) - moe_route - moe_permute -
 *   moe_grouped_linear (W1, SiLU, pre) - moe_dropout - moe_grouped_linear (W2) -
 *   moe_block_join
 * and back through moe_block_join_grad - weight and input gradient of W2 -
 * moe_dropout - weight and input gradient of W1 - moe_combine with gates of one
 * (the sum of a token's rows over its slots) - moe_block_join_grad.  The router's
 * gradient is not among them: from d_topk_gate through the softmax over the kept
 * logits to w_router and to the token's row is left to the caller, who adds the
 * latter to moe_combine's sum before the last call.
 */

/*
 * moe_grouped_linear — one Linear of every group's expert on its own rows:
 *   y[r] = act(x[row_index[r]] W_g^T + bias_g),   offsets[g] <= r < offsets[g+1]
 * with float32 sums, rounded once.  The SiLU and its derivative, here and in the gradients,
 * are float32's: for MOE_F32 within 12 * 2^-24 of the terms that they are made of, for
 * MOE_BF16 (by the hardware's exp2) within 2^-19 (1 + |z|) of them.
 *   dtype       moe_dtype of x, w, bias, y and pre
 *   x           [x_rows][k], row_index [max_rows] int32 or NULL: source row of
 *               each row (a dispatch's row_token), values in [0, x_rows); NULL:
 *               row r reads row r, and x_rows >= max_rows
 *   offsets     [n_groups+1] int32 DEVICE array, non-decreasing, offsets[0]=0
 *   max_rows    host-side upper bound on offsets[n_groups], as for
 *               moe_grouped_ffn; rows at or beyond offsets[n_groups] are
 *               neither read nor written, here and in the gradients
 *   w [G][n_out][k], bias [G][n_out] or NULL
 *   silu        1: act = SiLU, 0: none
 *   y           [max_rows][n_out] output
 *   pre         [max_rows][n_out] output or NULL, with silu 1 only: the values
 *               before the SiLU, which its gradient reads
 *   ws          device scratch of moe_grouped_linear_workspace_size bytes, which
 *               is one size for the three calls; nothing in it needs to be
 *               initialised, and calls that overlap in time need one each
 * n_out and k are multiples of 64 for MOE_BF16 and of 16 for MOE_F32 (as d_model
 * and d_ff of the layer), n_groups <= 1088, max_rows < 2^30; else
 * MOE_ERR_UNSUPPORTED.  Here and in the gradients, outputs overlap no input.
 */
int moe_grouped_linear(int32_t dtype, int32_t n_groups, int32_t n_out, int32_t k, int64_t x_rows,
                       const void *x, const int32_t *row_index, const int32_t *offsets,
                       int64_t max_rows, const void *w, const void *bias, int32_t silu, void *y,
                       void *pre, void *ws, size_t ws_bytes, void *stream);

/* moe_grouped_linear_input_grad — the gradient of moe_grouped_linear's rows from
 * that of its outputs (before its own SiLU, if it has one):
 *   dx[r] = (dy[r] W_g) silu'(pre[r])
 *   dy [max_rows][n_out], dx [max_rows][k] output
 *   pre         [max_rows][k] or NULL: the values before the SiLU that made the
 *               rows (moe_grouped_linear's pre of the Linear before); NULL: no
 *               such factor
 * Rows are those of the groups: where the forward read them through row_index,
 * the sum over a token's rows is moe_combine with gates of one. */
int moe_grouped_linear_input_grad(int32_t dtype, int32_t n_groups, int32_t n_out, int32_t k,
                                  const void *dy, const int32_t *offsets, int64_t max_rows,
                                  const void *w, const void *pre, void *dx, void *ws,
                                  size_t ws_bytes, void *stream);

/* moe_grouped_linear_weight_grad — the gradients of weights and bias, sums over
 * each group's rows in float32, rounded once:
 *   dw_g (+)= sum_r dy[r]^T x[row_index[r]],   dbias_g (+)= sum_r dy[r]
 *   grad_dtype  moe_dtype of dw and dbias: MOE_F32, or MOE_BF16 for MOE_BF16 rows
 *   dw          [G][n_out][k] output; dbias [G][n_out] output or NULL
 *   accumulate  1: the sums are added to what dw and dbias hold; 0: they replace
 *               it, and groups without rows (all of them, for max_rows 0) get
 *               zeros
 * Equal calls give equal bits. */
int moe_grouped_linear_weight_grad(int32_t dtype, int32_t grad_dtype, int32_t n_groups,
                                   int32_t n_out, int32_t k, const void *dy, int64_t x_rows,
                                   const void *x, const int32_t *row_index,
                                   const int32_t *offsets, int64_t max_rows, void *dw,
                                   void *dbias, int32_t accumulate, void *ws, size_t ws_bytes,
                                   void *stream);

/* Device workspace of the three calls (0 when the sizes are invalid or
 * unsupported, and where none is needed: ws may then be NULL). */
size_t moe_grouped_linear_workspace_size(int32_t dtype, int32_t n_groups, int32_t n_out, int32_t k,
                                         int64_t max_rows);

/* Norm of a row v of d elements, with float32 statistics:
 *   MOE_NORM_NONE   v w + b
 *   MOE_NORM_RMS    v / sqrt(mean(v^2) + eps) w + b
 *   MOE_NORM_LAYER  (v - m) / sqrt(mean((v - m)^2) + eps) w + b,  m = mean(v)
 * Squares are float32's: rows with elements above about 1e18 do not normalise. */
enum { MOE_NORM_NONE = 0, MOE_NORM_RMS = 1, MOE_NORM_LAYER = 2 };

/* Shape and constants of a block around the layer. */
typedef struct {
    int64_t T;                /* tokens                                            */
    double dropout_p;         /* probability of a dropped branch element, see
                                 moe_dropout; 0: none                              */
    int32_t d_model;          /* d, a multiple of 8, at most 16384                 */
    int32_t dtype;            /* moe_dtype of the branch, expert rows and next rows */
    int32_t res_dtype;        /* moe_dtype of the residual stream: dtype or MOE_F32 */
    int32_t norm_out;         /* MOE_NORM_*: norm of the branch                    */
    int32_t norm_in;          /* MOE_NORM_*: norm of the next block's input        */
    int32_t top_k;            /* K, with expert rows (at most 64), else ignored    */
    int32_t n_shared;         /* shared experts' rows beside them (at most 64)     */
    float eps;                /* of both norms, > 0 where there is one             */
    float scale;              /* of the branch                                     */
} moe_block;

/* Tensors that moe_block_join and its gradient read. */
typedef struct {
    const void *residual;       /* [T][d] res_dtype (not read by the gradient)     */
    const void *branch;         /* [T][d] dtype or NULL, see below                 */
    const void *y_rows;         /* expert rows [*][d] dtype, as in moe_combine, or NULL */
    const int32_t *slot_row;    /* [T][K] with y_rows: row of (t, k), or -1        */
    const float *topk_gate;     /* [T][K] with y_rows                              */
    const void *shared_out;     /* [n_shared][T][d] dtype with y_rows and n_shared
                                   > 0 (not read by the gradient)                  */
    const float *gate;          /* [T] or NULL (one)                               */
    const float *w_out, *b_out; /* [d] or NULL (one, zero): norm of the branch     */
    const float *w_in, *b_in;   /* [d] or NULL (one, zero): norm of the next input */
    const uint64_t *rng;        /* {seed, stream} for dropout_p > 0, see moe_dropout */
} moe_block_tensors;

/*
 * moe_block_join — a block's branch into the residual stream, and the next
 * block's input, in one pass over each token's row:
 *   b    = branch[t], or moe_combine of y_rows, slot_row, topk_gate, shared_out
 *   out  = residual[t] + scale gate[t] Drop(Norm_out(b))
 *   next = Norm_in(out)
 * in float32 (next from out before its rounding), each output rounded once.
 * branch and y_rows exclude each other; without both, out is the residual (the
 * norm before a model's first block) and everything of the branch is ignored.
 *   out         [T][d] res_dtype output or NULL; it may be the residual itself
 *   next        [T][d] dtype output or NULL
 *   branch_out  [T][d] dtype output or NULL: b, which the gradient reads (with
 *               y_rows; ignored without)
 * Outputs overlap no input but that one.
 */
int moe_block_join(const moe_block *cfg, const moe_block_tensors *in, void *out, void *next,
                   void *branch_out, void *stream);

/* Gradients that moe_block_join_grad writes; each may be NULL. */
typedef struct {
    void *d_residual;           /* [T][d] res_dtype                                */
    void *d_branch;             /* [T][d] dtype: of b, which is that of each shared
                                   expert's row too                                */
    void *d_y_rows;             /* rows slot_row[t][k] of [*][d] dtype: of the expert
                                   rows; others stay as they are                   */
    float *d_topk_gate;         /* [T][K], 0 where slot_row is -1                  */
    float *d_gate;              /* [T]                                             */
    float *d_w_out, *d_b_out;   /* [d], sums over the tokens                       */
    float *d_w_in, *d_b_in;     /* [d], sums over the tokens                       */
} moe_block_grads;

/*
 * moe_block_join_grad — the gradients of moe_block_join's inputs from those of
 * its outputs.  Statistics, masks and normalised rows are made again from out
 * and the branch as they were stored.
 *   out         [T][d] res_dtype: the forward's out (needed with d_next)
 *   d_out       [T][d] res_dtype or NULL (zero): gradient of out from behind
 *   d_next      [T][d] dtype or NULL (zero): gradient of next
 *   in->branch  the branch, or the forward's branch_out where it had y_rows;
 *               NULL: the block had none, and its gradients must be NULL (sums
 *               over tokens: zeros)
 *   in->y_rows  needed for d_topk_gate; in->slot_row and in->topk_gate for
 *               d_y_rows and d_topk_gate
 *   ws          device scratch of moe_block_join_grad_workspace_size bytes where a
 *               sum over tokens is asked for (else it may be NULL)
 * d_residual may be d_out itself, else outputs overlap no input.  With d_y_rows no
 * row is named twice in slot_row (a dispatch names none twice).  T == 0 writes zeros to the sums over tokens.
 * Equal calls give equal bits.
 */
int moe_block_join_grad(const moe_block *cfg, const moe_block_tensors *in, const void *out,
                        const void *d_out, const void *d_next, const moe_block_grads *grads,
                        void *ws, size_t ws_bytes, void *stream);
size_t moe_block_join_grad_workspace_size(const moe_block *cfg);

/*
 * moe_dropout — rows with elements dropped at random, and its own gradient:
 *   y[i] = x[i] / (1 - q) where element i stays, 0 where it is dropped
 * The probability is q = p rounded to a multiple of 2^-16, and exact: element i
 * of the rows (flat index) is dropped where the 16-bit number i % 8 of block i / 8
 * is below 65536 q.  Block j is Philox4x32-10 (Salmon et al., SC 2011) of the
 * counter (j, stream) under the key seed; its four words are taken in order, low
 * half first.  No mask is stored: the gradient of y, put through the same call,
 * is that of x.
 *   x, y        [rows][d] dtype; y may be x
 *   n_rows      [1] int32 DEVICE value or NULL: rows at or beyond it (a
 *               dispatch's offsets[N], 4-byte aligned) are neither read nor written
 *   p           in [0, 1), at most 1 - 2^-16 after rounding
 *   rng         [2] uint64 DEVICE array {seed, stream}, read when the call runs (a
 *               captured graph draws anew when they change); NULL where q is 0
 * rows * d < 2^42.
 */
int moe_dropout(int32_t dtype, int64_t rows, int64_t d, const void *x, void *y,
                const int32_t *n_rows, double p, const uint64_t *rng, void *stream);

/* Per-expert capacity the library applies for cfg (-1 = unlimited). */
int64_t moe_capacity(const moe_config *cfg);

/* Static text for a moe_status value. */
const char *moe_status_string(int status);

/* Interface version, 0x00MMmmpp: the library returns MOE_VERSION of the
 * header it was built with; a caller built against another version should not
 * use it (struct layouts may differ).  It stays as it is where calls are only
 * added: a library from before them has the same version and lacks their
 * symbols. */
#define MOE_VERSION 0x000200
int moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_H */
