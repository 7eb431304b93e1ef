/*
 * moe.h — C ABI of the sparse Mixture-of-Experts layer forward for AMD
 * Instinct MI355X (gfx950).
 *
 * The layer (page 1, "Mixture of Experts (MoE) 12段階極小ビジュアル解剖シミュレーター",
 * STEP 1-12; nanoMoE slides, "nanoMoEの深層解剖：Mixture of Expertsにおける
 * 条件分岐を排除した並列演算実装", slides 11-40) computes, for every token row x_t:
 *
 *   s      = W_g x_t + noise_t                         (STEP 2-4; slide 11)
 *   I_t    = the k largest scores, in descending order  (STEP 5; slide 12)
 *   g_t,j  = softmax of the k kept scores               (STEP 6; slide 13)
 *   slot   = rank of (j, t) among all assignments to expert I_t[j], counted
 *            over every token's first choice in token order, then every
 *            second choice, ...; ranks >= C are dropped  (slides 14-23)
 *   y_t    = sum over kept j of g_t,j * W_down[e] ReLU(W_up[e] x_t),
 *            e = I_t[j]; 0 when every choice is dropped (STEP 7-12; slides 33-40)
 *
 * with capacity C = ceil(capacity_factor * k * N / E) for a call of N tokens
 * (slide 14's get_capacity(num_tokens); its body is not shown, this is the
 * plain reading).
 *
 * Conventions for every entry point:
 *  - All tensor data pointers are DEVICE pointers owned by the caller; the
 *    library never allocates, frees or retains device memory, and keeps no
 *    global mutable state (every value a call needs, the device's compute
 *    unit count and kernel occupancy included, is queried within the call),
 *    except the per-device address of moe_dispatch_noalloc's static scratch.
 *    Tensors are row-major and contiguous.
 *  - Work is enqueued on the given HIP stream (hipStream_t passed as void*;
 *    NULL = the default stream). Calls return without synchronising; the
 *    results are valid once the stream reaches them.
 *  - Arguments are validated on the host before anything is enqueued. On
 *    error nothing is enqueued and nothing is written; the return value is a
 *    negative MOE_ERR_* code (see moe_error_string). MOE_ERR_HIP reports a
 *    failed launch; earlier launches of the same call may already be queued.
 *  - Work on one stream is ordered; two calls sharing a workspace must not
 *    run concurrently on different streams.
 *  - Results are deterministic: no floating-point atomics, fixed summation
 *    orders; two calls on the same inputs give bitwise-identical outputs.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
enum { MOE_F32 = 0, MOE_BF16 = 1 };

/* return codes */
enum {
    MOE_OK = 0,
    MOE_ERR_NULL = -1,        /* a required pointer is NULL                      */
    MOE_ERR_SHAPE = -2,       /* tensor ranks or extents are inconsistent        */
    MOE_ERR_DTYPE = -3,       /* element type not allowed for this tensor        */
    MOE_ERR_ARG = -4,         /* k < 1, k > E, capacity_factor <= 0 or not finite, negative sizes */
    MOE_ERR_WORKSPACE = -5,   /* workspace smaller than moe_workspace_size()     */
    MOE_ERR_UNSUPPORTED = -6, /* outside the documented limits below             */
    MOE_ERR_ALIGN = -7,       /* pointer not aligned as required                 */
    MOE_ERR_HIP = -8          /* a HIP launch failed                             */
};

/* Limits (MOE_ERR_UNSUPPORTED beyond them): E <= 256 experts, k <= 16,
 * N * k < 2^31 assignments, E * min(C, N) < 2^31 slots. bf16 tensors need
 * d and d_ff to be multiples of 8 and 16-byte aligned data pointers. A launch
 * holds fewer than 2^32 threads: moe_router and the whole layer take up to 64 a
 * token and return MOE_ERR_HIP for the tokens (2^26) that pass it. */
#define MOE_MAX_EXPERTS 256
#define MOE_MAX_TOPK 16
#define MOE_FEW_MAX_TOKENS 64      /* tokens of moe_forward_few */
#define MOE_FEW_MAX_WIDTH (1 << 20)  /* d and d_ff of moe_forward_few */
#define MOE_NORM_MAX_WIDTH 16384   /* row width of moe_layer_norm */
#define MOE_LINEAR_MAX_EXTENT (1 << 28)  /* rows and widths of moe_linear */
#define MOE_ROUTE_MAX_WIDTH (1 << 25)    /* d of moe_router_ex and moe_router_backward */
#define MOE_ROUTE_MAX_GRAD_ROWS (1 << 29)  /* tokens of moe_router_backward */

/* A tensor view: data (device), element type, rank and extents (row-major,
 * contiguous). A 3-D activation [B, T, d] is read as [B*T, d]. */
typedef struct {
    void *data;
    int32_t dtype;     /* MOE_F32 or MOE_BF16 */
    int32_t ndim;      /* 1..4 */
    int64_t shape[4];
} moe_tensor;

/* Launch context and optional exports of moe_forward.
 * Inputs:  stream, workspace (device, 256-byte aligned) and its size.
 * Optional device outputs (NULL = not exported; the library then keeps the
 * values in the workspace):
 *   topk_idx       int32 [N, k]  expert ids, highest score first
 *   topk_gate      fp32  [N, k]  gates of those experts (sum to 1 per token)
 *   slot           int32 [N, k]  capacity slot of each assignment, -1 = dropped
 *   used_capacity  int32 [E]     kept assignments per expert (= min(count, C))
 * Router statistics (optional device outputs, NULL = not computed). The
 * pages name load imbalance and capacity drops as what a router must be
 * watched for ("MoE（Mixture of Experts）とは？", section on MoE's weak
 * points; "게이팅 위기(Gating Crisis)", section on the load-balancing
 * challenge and its capacity-drop panel) and give no loss formula, so these
 * are the counts that define them, with used_capacity (nanoMoE slide 14):
 *   expert_demand    int32 [E]  assignments routed to expert e before the
 *                               capacity clip (count[e] of slide 14)
 *   expert_drops     int32 [E]  of those, the ones past the capacity
 *                               (= expert_demand - used_capacity)
 *   expert_gate_sum  fp32  [E]  sum of the gates of every assignment routed
 *                               to e (kept or dropped), fp32, summed in a
 *                               fixed order (identical on every run)
 * Host output: capacity (C), written before anything is enqueued.
 * aux_stream (input, moe_backward* only; ignored by the forward): a second
 * HIP stream of the same device, owned by the caller, that the backward may
 * run part of its work on (the router-weight and down-projection weight
 * gradients) while the rest runs on `stream`. The call forks it from and
 * joins it back to `stream` with two events it creates and destroys within
 * the call, so the call stays one stream-ordered operation on `stream` and
 * can be captured in a graph. NULL: everything runs on `stream`.
 * Dropped assignments per call = N*k - sum(used_capacity). */
typedef struct {
    void *stream;
    void *workspace;
    size_t workspace_bytes;
    int32_t *topk_idx;
    float *topk_gate;
    int32_t *slot;
    int32_t *used_capacity;
    int64_t capacity;
    int32_t *expert_demand;
    int32_t *expert_drops;
    float *expert_gate_sum;
    void *aux_stream;
} moe_stats;

/* The whole layer forward (page 1 STEP 1-12; nanoMoE slides 11-40).
 *   x      [N, d] (or [B, T, d])   MOE_F32 or MOE_BF16
 *   W_g    [E, d]                  MOE_F32 (the router runs in full precision, slide 11)
 *   noise  [N, E] MOE_F32, or NULL for sigma = 0. The caller draws it: it is
 *          sigma * eps with eps ~ N(0, 1) (STEP 3-4) plus any constant score
 *          offset; the library has no random number generator.
 *   W_up   [E, d_ff, d]            same dtype as x (row f of expert e is the
 *          f-th hidden neuron: z = W_up[e] x, STEP 8)
 *   W_down [E, d, d_ff]            same dtype as x (E_i(x) = W_down[e] h, STEP 10)
 *   k      experts per token, 1 <= k <= min(E, 16)
 *   capacity_factor  > 0, finite
 *   out    [N, d] (same shape as x) same dtype as x; every row is written
 *   stats  launch context and optional exports (required)
 * Numerics: scores, top-k and gates in fp32; expert products accumulate in
 * fp32 (bf16 inputs on matrix cores); the hidden activation is stored in
 * the dtype of x. Each expert's output row is stored in fp32 for an fp32
 * layer; for a bf16 layer it is stored compact in the workspace: every group
 * of 32 columns as fp16 values of y * 2^sh with one power-of-two shift sh
 * per group, chosen from the group's largest finite magnitude (relative
 * error at most 2^-11, no overflow at any magnitude). The combine
 * accumulates in fp32 in choice order and rounds once to the dtype of out
 * (round to nearest even).
 * N = 0 is valid: capacity is 0, used_capacity (if given) is zeroed. */
int moe_forward(const moe_tensor *x, const moe_tensor *W_g, const moe_tensor *noise,
                const moe_tensor *W_up, const moe_tensor *W_down, int k,
                float capacity_factor, moe_tensor *out, moe_stats *stats);

/* The expert variant of the nanoMoE slides (slide 32: a bias after each
 * projection and GELU between them) for moe_forward_ex and moe_experts_ex.
 * activation: MOE_ACT_RELU (page 1 STEP 9) or MOE_ACT_GELU, x * Phi(x) with
 * Phi the standard normal distribution function (erf form), evaluated in
 * fp32 before H is rounded (by a formula within 2.2e-7 of x Phi(x), besides
 * fp32 rounding; an absolute bound: the far negative tail is not as close
 * relative to its size); MOE_ERR_ARG for any other value.
 * b_up:   [E, d_ff] MOE_F32 added to W_up[e] x before the activation, or NULL
 * b_down: [E, d]    MOE_F32 added to W_down[e] h, or NULL
 * Bias data are device pointers, 16-byte aligned (MOE_ERR_ALIGN), checked
 * for dtype and extents like every other tensor.
 * dropout: training-mode dropout on each expert output row (slide 32: the
 *   expert ends in a dropout), after b_down; 0 (the default of a
 *   zero-initialised struct) applies none; MOE_ERR_ARG outside [0, 1).
 *   Element i of the row of assignment a = t k + j is kept when its 32-bit
 *   random word is >= floor(dropout 2^32), and is then scaled by
 *   1 / (1 - dropout); dropped elements are 0. The words of elements
 *   8q .. 8q+7 are the Philox4x64-10 block (Salmon et al., SC 2011) at
 *   counter (q, a, dropout_offset, 0) under key (dropout_seed, 0): element
 *   i takes half i % 2 (low half first) of output word (i % 8) / 2. A call
 *   with the same seed and offset draws the same mask, so moe_backward_ex
 *   differentiates exactly the forward's dropped-out layer.
 * Zero-initialise the struct and set the fields used. */
enum { MOE_ACT_RELU = 0, MOE_ACT_GELU = 1, MOE_ACT_NONE = 2 /* moe_linear only */ };
typedef struct {
    int32_t activation;
    const moe_tensor *b_up;
    const moe_tensor *b_down;
    float dropout;
    uint64_t dropout_seed;
    uint64_t dropout_offset;
} moe_expert_opts;

/* moe_forward with the expert variant above; opts NULL is moe_forward. */
int moe_forward_ex(const moe_tensor *x, const moe_tensor *W_g, const moe_tensor *noise,
                   const moe_tensor *W_up, const moe_tensor *W_down,
                   const moe_expert_opts *opts, int k, float capacity_factor, moe_tensor *out,
                   moe_stats *stats);

/* Bytes of workspace moe_forward needs for these sizes (0 on invalid sizes). */
size_t moe_workspace_size(int64_t N, int64_t d, int64_t E, int64_t d_ff, int k,
                          float capacity_factor, int32_t dtype);

/* Per-expert capacity C = ceil(capacity_factor * k * N / E), in double
 * (nanoMoE slide 14, get_capacity of the call's token count), INT64_MAX
 * where that passes 64 bits. -1 on invalid arguments; 0 when N = 0. */
int64_t moe_capacity(int64_t N, int64_t E, int k, float capacity_factor);

/* Static description of a return code. */
const char *moe_error_string(int code);

/* ---------------------------------------------------------------------------
 * The four stages moe_forward enqueues, exported for callers that run them
 * separately (and for per-stage testing). Same conventions as above.
 * ------------------------------------------------------------------------- */

/* Router (page 1 STEP 2-6; slides 11-13): fp32 scores s = W_g x + noise,
 * top-k in descending order (equal scores: lower expert id first), softmax
 * over the k kept scores. Writes topk_idx [N, k] int32 and topk_gate [N, k]
 * fp32 (device). x, W_g, noise as in moe_forward. workspace: device scratch
 * of moe_router_workspace_size() bytes, 256-byte aligned (may be NULL when
 * that size is 0). */
int moe_router(const moe_tensor *x, const moe_tensor *W_g, const moe_tensor *noise,
               int k, int32_t *topk_idx, float *topk_gate, void *workspace,
               size_t workspace_bytes, void *stream);

/* Bytes of router scratch for N tokens of width d and E experts (0 on invalid
 * sizes or when the dtype needs none). */
size_t moe_router_workspace_size(int64_t N, int64_t d, int64_t E, int32_t dtype);

/* Capacity-limited dispatch plan (slides 14-29). From topk_idx [N, k] and the
 * capacity C (moe_capacity), writes:
 *   slot        int32 [N, k]          rank among the expert's assignments in
 *                                     (choice, token) order, -1 if >= C
 *   used        int32 [E]             kept assignments per expert
 *   slot_token  int32 [E, min(C, N)]  for r < used[e]: the assignment id
 *                                     t*k + j holding slot r of expert e
 *                                     (rows past used[e] are left untouched)
 *   tiles       int32 [2*(E+1)]       prefix sums of ceil(used[e]/128) and
 *                                     ceil(used[e]/256): the expert kernels'
 *                                     tile schedule
 * and, each when not NULL, the router statistics of moe_stats:
 * expert_demand, expert_drops (int32 [E]) and expert_gate_sum (fp32 [E],
 * which reads topk_gate [N, k]; topk_gate may be NULL otherwise).
 * workspace: device scratch of moe_dispatch_workspace_size() bytes (256-byte
 * aligned; may be NULL when that size is 0, i.e. for N*k <= 4096). An id
 * outside [0, E) in topk_idx is not counted and its slot is -1. */
int moe_dispatch(int64_t N, int64_t E, int k, int64_t capacity, const int32_t *topk_idx,
                 const float *topk_gate, int32_t *slot, int32_t *used, int32_t *slot_token,
                 int32_t *tiles, int32_t *expert_demand, int32_t *expert_drops,
                 float *expert_gate_sum, void *workspace, size_t workspace_bytes,
                 void *stream);

/* Name of the kernel instantiation moe_forward launches for one expert
 * product of a layer of these sizes (product 0: the up product, 1: the down
 * product; dropout != 0: the down product's training-dropout variant), as a
 * profiler lists it, e.g. "expert_gemm_kernel<256, 256, 4, 4, 1, 64, 2, 0>".
 * Written to buf, NUL-terminated and truncated to len bytes; returns the
 * length of the full name, or a negative MOE_ERR_* code (N = 0 is
 * MOE_ERR_ARG: nothing is launched). For measurement tools that match
 * profiles to the layer's stages. */
int moe_expert_kernel_name(int64_t N, int64_t d, int64_t E, int64_t d_ff, int k,
                           float capacity_factor, int32_t dtype, int product, int dropout,
                           char *buf, size_t len);

/* moe_dispatch for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same plan, outputs and limits as moe_dispatch, but the per-chunk
 * scratch lives in a static device array of the library (4 MiB, held by
 * each GPU the library runs on until the process ends) instead of a
 * workspace argument, and the call allocates nothing. MOE_ERR_UNSUPPORTED
 * when moe_dispatch_workspace_size(N, E, k) exceeds 4 MiB (about 2 million
 * assignments at E = 256, more with fewer experts). The library keeps the
 * array's device address per device (taken once per device on its first
 * call there). Calls that overlap on one GPU (on different streams, or from
 * several host threads) share that GPU's array and race; calls ordered on
 * one stream do not (the array holds the last call's partials, which the
 * next call overwrites before it reads them). */
int moe_dispatch_noalloc(int64_t N, int64_t E, int k, int64_t capacity,
                         const int32_t *topk_idx, const float *topk_gate, int32_t *slot,
                         int32_t *used, int32_t *slot_token, int32_t *tiles,
                         int32_t *expert_demand, int32_t *expert_drops,
                         float *expert_gate_sum, void *stream);

/* Bytes of dispatch scratch for N tokens, E experts and top-k (0 on invalid
 * sizes or when a call needs none). */
size_t moe_dispatch_workspace_size(int64_t N, int64_t E, int k);

/* Grouped expert FFN (page 1 STEP 7-10; slides 32-37) over the dispatch plan.
 * For each expert e and r < used[e], with a = slot_token[e, r], t = a / k:
 *   H[e, r, :] = ReLU(W_up[e] x_t)      stored in the dtype of x   [E, min(C,N), d_ff]
 *   Y[a, :]    = W_down[e] H[e, r, :]   stored in fp32             [N*k, d]
 * Both products accumulate in fp32; H is rounded once to the dtype of x (the
 * slides' experts run under bf16 autocast), Y is kept in fp32 so that the
 * combine rounds each output once. The gather of token rows is fused into
 * the first product. Rows of Y whose assignment was dropped are not written.
 * H and Y are caller device buffers (16-byte aligned for bf16).
 * workspace: optional device scratch of workspace_bytes (256-byte aligned,
 * MOE_ERR_ALIGN otherwise) in which the bf16 path keeps fp32 partial tiles
 * when it cuts the K loop of a product's last, partly idle round of tiles
 * into ranges; NULL, or too few bytes for one partial tile per workgroup the
 * device runs at once, computes every tile whole (moe_expert_workspace_size()
 * bytes are enough on a device with up to 256 compute units). Either way the
 * result is deterministic; the two differ only in fp32 summation order.
 * Calls that share a workspace must not overlap. */
int moe_experts(const moe_tensor *x, const moe_tensor *W_up, const moe_tensor *W_down,
                int k, int64_t capacity, const int32_t *used, const int32_t *slot_token,
                const int32_t *tiles, void *H, void *Y, void *workspace,
                size_t workspace_bytes, void *stream);

/* moe_experts with the expert variant of moe_expert_opts (NULL: ReLU, no
 * biases). */
int moe_experts_ex(const moe_tensor *x, const moe_tensor *W_up, const moe_tensor *W_down,
                   const moe_expert_opts *opts, int k, int64_t capacity, const int32_t *used,
                   const int32_t *slot_token, const int32_t *tiles, void *H, void *Y,
                   void *workspace, size_t workspace_bytes, void *stream);

/* moe_expert_up and moe_expert_down with the expert variant of
 * moe_expert_opts: the up product adds b_up and applies the activation, the
 * down product adds b_down (b_up and the activation are ignored there). */
int moe_expert_up_ex(const moe_tensor *x, const moe_tensor *W_up, const moe_expert_opts *opts,
                     int k, int64_t capacity, const int32_t *used, const int32_t *slot_token,
                     const int32_t *tiles, void *H, void *workspace, size_t workspace_bytes,
                     void *stream);
int moe_expert_down_ex(int64_t N, const moe_tensor *W_down, const moe_expert_opts *opts, int k,
                       int64_t capacity, const int32_t *used, const int32_t *slot_token,
                       const int32_t *tiles, const void *H, void *Y, void *workspace,
                       size_t workspace_bytes, void *stream);

/* Bytes of expert scratch that enable the K-split on any device with up to
 * 256 compute units (0 for MOE_F32 and for an unknown dtype). */
size_t moe_expert_workspace_size(int32_t dtype);

/* The two halves of moe_experts, one product each (page 1 STEP 8-9 and STEP
 * 10): moe_expert_up writes H from x and W_up; moe_expert_down writes Y from
 * H and W_down ([E, d, d_ff]; H has W_down's dtype and [E, min(C,N), d_ff]
 * rows, Y is [N*k, d] fp32). workspace as for moe_experts. */
int moe_expert_up(const moe_tensor *x, const moe_tensor *W_up, int k, int64_t capacity,
                  const int32_t *used, const int32_t *slot_token, const int32_t *tiles,
                  void *H, void *workspace, size_t workspace_bytes, void *stream);
int moe_expert_down(int64_t N, const moe_tensor *W_down, int k, int64_t capacity,
                    const int32_t *used, const int32_t *slot_token, const int32_t *tiles,
                    const void *H, void *Y, void *workspace, size_t workspace_bytes,
                    void *stream);

/* moe_expert_down_ex writing Y compact, the form in which the fused entry
 * points of a bf16 layer keep it (see moe_forward's numerics): Y16 [N*k, d]
 * fp16 bits and Ysh [N][ceil(d / 32)][k] int8 shifts, assignment a = t*k + j
 * standing for y[a, c] = Y16[a, c] * 2^-Ysh[t][c / 32][j] (a token's k
 * shifts of one group adjacent). Y16 16-byte aligned. bf16 layers
 * only (MOE_ERR_DTYPE otherwise); rows of dropped assignments are not
 * written. Callers that time or check the fused layer's stages use it. */
int moe_expert_down_compact(int64_t N, const moe_tensor *W_down, const moe_expert_opts *opts,
                            int k, int64_t capacity, const int32_t *used,
                            const int32_t *slot_token, const int32_t *tiles, const void *H,
                            void *Y16, int8_t *Ysh, void *workspace, size_t workspace_bytes,
                            void *stream);

/* Combine (page 1 STEP 11-12; slides 38-40): out[t] = sum over j < k with
 * slot[t, j] >= 0 of topk_gate[t, j] * Y[t*k + j], accumulated in fp32 in
 * order j = 0..k-1, rounded once to out's dtype; rows with every choice
 * dropped become 0. Y is [N*k, d] MOE_F32 or MOE_BF16 (read as exact fp32
 * values), out is [N, d] MOE_F32 or MOE_BF16. */
int moe_combine(int64_t N, int64_t d, int k, const moe_tensor *Y, const float *topk_gate,
                const int32_t *slot, moe_tensor *out, void *stream);

/* moe_combine over compact rows (Y16, Ysh as moe_expert_down_compact writes
 * them), each value taken as Y16 * 2^-Ysh exactly; d % 8 == 0
 * (MOE_ERR_UNSUPPORTED otherwise), Y16 and out 16-byte aligned. */
int moe_combine_compact(int64_t N, int64_t d, int k, const void *Y16, const int8_t *Ysh,
                        const float *topk_gate, const int32_t *slot, moe_tensor *out,
                        void *stream);

/* Backward pass of the layer (the row after the forward: gradients through
 * the gates to the router and through the experts), for bf16 layers with
 * ReLU experts and no biases (moe_backward_ex: the GELU / bias / dropout
 * variants). For a loss whose
 * gradient with respect to out is dout, by the chain rule of moe_forward:
 *   combine: dy = g * dout, dg = <dout, y> (kept choices; dropped: 0);
 *   masked softmax over the kept scores: ds_j = g_j (dg_j - sum_l g_l dg_l),
 *   and no gradient through the top-k choice or to experts outside it;
 *   scores: dW_g = ds^T x, dx += ds W_g;
 *   experts: dZ = (dY W_down) where H > 0, dW_down = dY^T H, dW_up = dZ^T X,
 *   dx += the kept choices' dZ W_up rows, summed in choice order.
 * The forward state (routing, dispatch plan, H and the experts' output
 * rows, as the forward combined them) is recomputed from the inputs in
 * the workspace, so the call takes the forward's arguments plus:
 *   dout    [N, d]         same dtype as x (MOE_BF16)
 *   dx      [N, d]         MOE_F32, written
 *   dW_g    [E, d]         MOE_F32, written
 *   dW_up   [E, d_ff, d]   MOE_F32, written
 *   dW_down [E, d, d_ff]   MOE_F32, written
 *   stats   as for moe_forward, with moe_backward_workspace_size() bytes
 * Products run on the matrix cores with bf16 operands (dy and dZ are rounded
 * to bf16; fp32 ds is split exactly into three bf16 terms) and fp32
 * accumulation; every sum has a fixed order. MOE_ERR_UNSUPPORTED for fp32
 * layers. Device pointers 16-byte aligned (MOE_ERR_ALIGN).
 * Streams: with stats->aux_stream set, part of the work (the router-weight
 * gradient and dW_down) runs on that caller-owned stream, forked from and
 * joined to stats->stream inside the call (see moe_stats); with NULL every
 * launch goes to stats->stream. The results are the same bit for bit. */
int moe_backward(const moe_tensor *x, const moe_tensor *W_g, const moe_tensor *noise,
                 const moe_tensor *W_up, const moe_tensor *W_down, int k, float capacity_factor,
                 const moe_tensor *dout, moe_tensor *dx, moe_tensor *dW_g, moe_tensor *dW_up,
                 moe_tensor *dW_down, moe_stats *stats);

/* moe_backward for the expert variants of moe_forward_ex (page 2, slide
 * 32): opts as there (NULL: ReLU, no biases, no dropout). With GELU,
 * dZ = dH gelu'(z), gelu'(z) = Phi(z) + z phi(z), on the bf16
 * pre-activations z the recomputed up product keeps. With dropout, the
 * same mask as the forward's (same seed and offset): dg = <dout, y m> and
 * dY = g dout m, m the dropout factor (1 / (1 - p) or 0) of each element. Bias gradients, fp32, written exactly when the layer has
 * that bias (else they must be NULL: MOE_ERR_ARG; a missing one:
 * MOE_ERR_NULL), each the sum over the expert's kept assignments in a fixed
 * order:
 *   db_up   [E, d_ff]   sum of the dZ rows
 *   db_down [E, d]      sum of the dY rows (g * dout)
 * Same workspace as moe_backward. */
int moe_backward_ex(const moe_tensor *x, const moe_tensor *W_g, const moe_tensor *noise,
                    const moe_tensor *W_up, const moe_tensor *W_down,
                    const moe_expert_opts *opts, int k, float capacity_factor,
                    const moe_tensor *dout, moe_tensor *dx, moe_tensor *dW_g, moe_tensor *dW_up,
                    moe_tensor *dW_down, moe_tensor *db_up, moe_tensor *db_down,
                    moe_stats *stats);

/* Training step without recomputation: moe_forward_train is moe_forward_ex
 * for a bf16 layer (same arguments, same out bit for bit) that also leaves
 * the forward state the backward needs (routing, dispatch plan, H, the
 * experts' output rows and, for GELU, the pre-activations) in
 * stats->workspace, which must hold moe_backward_workspace_size() bytes
 * (and in stats' exported routing arrays when given).
 * moe_backward_after_forward then takes moe_backward_ex's arguments and
 * computes the same gradients from that state instead of recomputing it:
 * pass the same inputs, options and moe_stats (workspace and exported
 * arrays) as to the forward, with no other call on that workspace in
 * between. The state serves one backward call (the GELU pre-activations are
 * overwritten by dZ). For callers that keep activations between the passes
 * of a training step; it saves the two recomputed expert products. */
int moe_forward_train(const moe_tensor *x, const moe_tensor *W_g, const moe_tensor *noise,
                      const moe_tensor *W_up, const moe_tensor *W_down,
                      const moe_expert_opts *opts, int k, float capacity_factor, moe_tensor *out,
                      moe_stats *stats);
int moe_backward_after_forward(const moe_tensor *x, const moe_tensor *W_g,
                               const moe_tensor *noise, const moe_tensor *W_up,
                               const moe_tensor *W_down, const moe_expert_opts *opts, int k,
                               float capacity_factor, const moe_tensor *dout, moe_tensor *dx,
                               moe_tensor *dW_g, moe_tensor *dW_up, moe_tensor *dW_down,
                               moe_tensor *db_up, moe_tensor *db_down, moe_stats *stats);

/* Bytes of workspace moe_backward needs (0 on invalid sizes or a dtype
 * other than MOE_BF16). */
size_t moe_backward_workspace_size(int64_t N, int64_t d, int64_t E, int64_t d_ff, int k,
                                   float capacity_factor, int32_t dtype);

/* ---------------------------------------------------------------------------
 * The rest of a transformer block's feed-forward half: the layer for a few
 * tokens, the linear product of a shared or dense expert, the norm in front.
 * Same conventions as above.
 * ------------------------------------------------------------------------- */

/* moe_forward_ex for at most MOE_FEW_MAX_TOKENS tokens and widths d, d_ff up
 * to MOE_FEW_MAX_WIDTH (MOE_ERR_UNSUPPORTED beyond), the form of a decoding
 * step: the same arguments, routing, capacity drops, options and exports, on
 * kernels that stream each hit expert's weights once instead of computing row
 * tiles. Training-mode dropout is refused (MOE_ERR_UNSUPPORTED). Numerics: as
 * moe_forward's (scores differ from its only in fp32 summation order), except
 * that a bf16 layer keeps the hidden activation to 16 significant bits (two
 * bf16 terms) and the experts' output rows in fp32, so that out carries only
 * its own rounding (an infinite weight in W_down meets both terms: where
 * moe_forward gives an infinity, out may be NaN); GELU of -inf is 0 (there:
 * NaN) and ReLU keeps a NaN (there: 0); each token's choices are added in a
 * fixed order.
 * stats->workspace holds moe_few_workspace_size() bytes (256-byte aligned;
 * a size for more tokens serves fewer). Bias data 16-byte aligned, as there.
 * Neither out, the workspace nor an export may overlap an input or one of each
 * other (MOE_ERR_ARG). */
int moe_forward_few(const moe_tensor *x, const moe_tensor *W_g, const moe_tensor *noise,
                    const moe_tensor *W_up, const moe_tensor *W_down,
                    const moe_expert_opts *opts, int k, float capacity_factor, moe_tensor *out,
                    moe_stats *stats);

/* Bytes of workspace moe_forward_few needs (0 on invalid sizes, or beyond
 * MOE_FEW_MAX_TOKENS). */
size_t moe_few_workspace_size(int64_t N, int64_t d, int64_t E, int64_t d_ff, int k,
                              float capacity_factor, int32_t dtype);

/* Linear product with its epilogue, the dense feed-forward layer or shared
 * expert beside the routed ones:
 *   z = x W^T + bias,  out = act(z) + residual
 *   x        [N, K] (or [B, T, K])  MOE_BF16 (MOE_ERR_UNSUPPORTED for fp32)
 *   W        [M, K]                 MOE_BF16 (row m: output neuron m)
 *   bias     [M] MOE_F32 or NULL
 *   activation  MOE_ACT_NONE, MOE_ACT_RELU or MOE_ACT_GELU (as
 *            moe_expert_opts); MOE_ERR_ARG otherwise
 *   residual [N, M] MOE_BF16 or NULL; may be the buffer of out
 *   out      [N, M] MOE_BF16, every row written
 *   z        [N, M] MOE_BF16 or NULL: the pre-activations, for the backward
 *            (a buffer of its own: MOE_ERR_ARG)
 * fp32 accumulation, bias, activation and residual; out and z are each rounded
 * once. Otherwise out, z and the workspace must not overlap an input or each
 * other (MOE_ERR_ARG). K and M are multiples of 8 and N, K, M at
 * most MOE_LINEAR_MAX_EXTENT (MOE_ERR_UNSUPPORTED); data 16-byte aligned
 * (MOE_ERR_ALIGN). workspace: device scratch of moe_linear_workspace_size()
 * bytes, 256-byte aligned (may be NULL when that is 0): fp32 partial products
 * of a product too small to fill the GPU. N = 0 is valid. */
int moe_linear(const moe_tensor *x, const moe_tensor *W, const moe_tensor *bias,
               int32_t activation, const moe_tensor *residual, moe_tensor *out, moe_tensor *z,
               void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of scratch of moe_linear (0 when it needs none, or for invalid sizes). */
size_t moe_linear_workspace_size(int64_t N, int64_t K, int64_t M);

/* Its backward, for dout [N, M] MOE_BF16 the gradient of out:
 *   dz = dout act'(z),  dx = dz W,  dW = dz^T x,  dbias = sum of the dz rows
 * (the residual's gradient is dout itself; act' of MOE_ACT_RELU is 0 where
 * z <= 0 and 1 elsewhere, a NaN included). z: the forward's, required with an
 * activation, NULL without one (MOE_ERR_ARG). dx [N, K] and dW [M, K] are
 * MOE_BF16 or MOE_F32, dbias [M] MOE_F32; each may be NULL and is then not
 * computed (all three NULL: MOE_ERR_NULL). The products read dz rounded once
 * to bf16 (the dz of MOE_ACT_NONE is dout, exactly), so that with an activation
 * an MOE_F32 dx or dW carries that rounding too; dbias sums the fp32
 * values. No output, nor the workspace, may overlap an input, another output or
 * each other (MOE_ERR_ARG). Each
 * gradient has the same bits whichever others are computed with it. Widths and
 * alignment as moe_linear's. workspace:
 * moe_linear_backward_workspace_size() bytes, 256-byte aligned. N = 0: dW and
 * dbias are zero. */
int moe_linear_backward(const moe_tensor *x, const moe_tensor *W, const moe_tensor *z,
                        int32_t activation, const moe_tensor *dout, moe_tensor *dx,
                        moe_tensor *dW, moe_tensor *dbias, void *workspace,
                        size_t workspace_bytes, void *stream);

/* Bytes of scratch of moe_linear_backward (0 for N = 0 or invalid sizes). */
size_t moe_linear_backward_workspace_size(int64_t N, int64_t K, int64_t M, int32_t activation);

/* Layer norm over the last dimension, the norm in front of the router:
 *   h = x + residual, rounded to the type of x (h = x without a residual)
 *   out = (h - mean) rstd weight + bias,
 *   mean = sum h / d, rstd = 1 / sqrt(sum (h - mean)^2 / d + eps)
 *   x        [N, d] (or [B, T, d])  MOE_F32 or MOE_BF16
 *   residual same shape and dtype as x, or NULL
 *   weight   [d] MOE_F32; bias [d] MOE_F32 or NULL
 *   eps      > 0, finite
 *   h        as x; required with a residual, NULL without one (MOE_ERR_ARG)
 *   out      as x, every row written
 *   mean, rstd  [N] MOE_F32 or NULL: what the backward needs
 * Statistics are fp32, of the values h holds after its rounding. out or h may
 * be the buffer of x or of residual (each element is read before it is
 * written), but must not overlap each other, or one of those any other way;
 * nor may mean or rstd overlap any tensor, or h or out weight or bias
 * (MOE_ERR_ARG). d <= MOE_NORM_MAX_WIDTH;
 * bf16 rows need d % 8 == 0 (MOE_ERR_UNSUPPORTED) and 16-byte aligned x,
 * residual, h, out, weight and bias (MOE_ERR_ALIGN); fp32 rows any d. */
int moe_layer_norm(const moe_tensor *x, const moe_tensor *residual, const moe_tensor *weight,
                   const moe_tensor *bias, float eps, moe_tensor *h, moe_tensor *out,
                   moe_tensor *mean, moe_tensor *rstd, void *stream);

/* Its backward, for dout the gradient of out and dres (or NULL) the gradient
 * that reaches h along the residual path:
 *   g = dout weight, xh = (x - mean) rstd,
 *   dx = rstd (g - sum g / d - xh (sum g xh) / d) + dres
 *   dweight = sum over rows of dout xh, dbias = sum over rows of dout
 * x is the h of the forward (or its x without a residual); with a residual
 * dx is the gradient of both summands. dx, dout and dres have x's shape and
 * dtype. dx may be the buffer of dout or dres; otherwise no output, nor the
 * workspace, may overlap an input, another output or each other (MOE_ERR_ARG).
 * weight, dweight and dbias [d], mean and rstd [N] MOE_F32; dbias may be
 * NULL. Sums are fp32 in a fixed order. workspace: device scratch of
 * moe_layer_norm_backward_workspace_size() bytes, 256-byte aligned. Widths
 * and alignment as moe_layer_norm's. N = 0: the sums are zero. */
int moe_layer_norm_backward(const moe_tensor *x, const moe_tensor *weight, const moe_tensor *mean,
                            const moe_tensor *rstd, const moe_tensor *dout,
                            const moe_tensor *dres, moe_tensor *dx, moe_tensor *dweight,
                            moe_tensor *dbias, void *workspace, size_t workspace_bytes,
                            void *stream);

/* Bytes of scratch of moe_layer_norm_backward (0 for N = 0 or invalid sizes). */
size_t moe_layer_norm_backward_workspace_size(int64_t N, int64_t d);

/* ---------------------------------------------------------------------------
 * Weights of 4 bits with group scales, for decoding: the linear product and
 * the routed experts for up to MOE_FEW_MAX_TOKENS rows. Same conventions as
 * above.
 * ------------------------------------------------------------------------- */

/* A matrix (or E matrices) of 4-bit weights,
 *   w[.., m, k] = (q[.., m, k] - zero[.., m, k / group]) scale[.., m, k / group]
 *   data   [.., M, K / 2] bytes: q of columns 2i and 2i + 1 in the low and the
 *          high half of byte i
 *   scale  [.., M, K / group] bf16
 *   zero   [.., M, K / group] bf16, or NULL: 8 everywhere
 *   group  32, 64 or 128 (MOE_ERR_UNSUPPORTED otherwise); K % group == 0
 *          (MOE_ERR_SHAPE)
 *   ndim   2 ([M, K]) or 3 ([E, M, K]), and shape, the logical extents
 * Device pointers of the caller, 16-byte aligned (MOE_ERR_ALIGN). */
typedef struct {
    void *data;
    void *scale;
    void *zero;
    int32_t group;
    int32_t ndim;      /* 2 or 3 */
    int64_t shape[3];
} moe_q4;

/* Nearest 4-bit weights of W (MOE_F32 or MOE_BF16, finite, the extents of q, fewer
 * than 2^35 of them (MOE_ERR_UNSUPPORTED), 16-byte aligned) into q's buffers, group by
 * group. Without q->zero: scale =
 * max |w| / 7 rounded to bf16, q = 8 + the nearest integer to w / scale in
 * [-8, 7]. With it: the range [min(w, 0), max(w, 0)], scale = its length / 15
 * rounded to bf16, zero = the nearest integer to -min / scale and q = zero +
 * the nearest integer to w / scale, both in [0, 15]. Ties to even; a group
 * whose scale is 0 stands for zeros (past 2^127 a weight's value may round to
 * infinity, as the scale is rounded). q's buffers must not overlap W or each
 * other (MOE_ERR_ARG). */
int moe_quantize(const moe_tensor *W, moe_q4 *q, void *stream);

/* W (MOE_F32 or MOE_BF16, 16-byte aligned) = the values q stands for, each
 * rounded once: the weights of moe_linear, moe_forward and the other entry
 * points for more rows than the calls below take. */
int moe_dequantize(const moe_q4 *q, moe_tensor *W, void *stream);

/* moe_linear for N <= MOE_FEW_MAX_TOKENS rows (MOE_ERR_UNSUPPORTED beyond) and
 * 4-bit weights:  out = act(x W^T + bias) + residual
 *   x [N, K] MOE_BF16 (MOE_ERR_UNSUPPORTED for fp32), W [M, K] as moe_q4,
 *   bias [M] MOE_F32 or NULL, activation as moe_linear's, residual [N, M]
 *   MOE_BF16 or NULL (may be the buffer of out), out [N, M] MOE_BF16
 * The weights enter exactly, sums are fp32, out is rounded once. The kernels add
 * x (128 + q) and x (128 + zero) of a group apart, so sum |x| over each group of
 * columns must stay below 2^119 (zero points in [0, 15]): past it finite values may
 * give infinities or NaN, and an infinite one gives NaN in every output of its row. K and M at most
 * MOE_LINEAR_MAX_EXTENT; x 16-byte, the other data aligned to their types
 * (MOE_ERR_ALIGN). out must not overlap an input otherwise (MOE_ERR_ARG).
 * workspace: moe_linear_quant_workspace_size() bytes, 256-byte aligned (may be
 * NULL when that is 0). N = 0 is valid. */
int moe_linear_quant(const moe_tensor *x, const moe_q4 *W, const moe_tensor *bias,
                  int32_t activation, const moe_tensor *residual, moe_tensor *out,
                  void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of scratch of moe_linear_quant (0 when it needs none, or for invalid sizes). */
size_t moe_linear_quant_workspace_size(int64_t N, int64_t K, int64_t M, int32_t group);

/* The routed experts of N <= MOE_FEW_MAX_TOKENS tokens with 4-bit weights:
 *   out_t = sum over j of topk_gate[t, j] (W_down[e] act(W_up[e] x_t + b_up[e])
 *           + b_down[e]),  e = topk_idx[t, j]
 * for a routing given by the caller (moe_router, moe_router_ex): ids int32 and
 * gates fp32 [N, k], device; an id outside [0, E) contributes nothing, and no
 * capacity applies.
 *   x, out [N, d] MOE_BF16; W_up [E, d_ff, d], W_down [E, d, d_ff] as moe_q4
 *   of one group; opts as moe_forward_few's (activation, biases; no dropout)
 * Numerics: weights as moe_linear_quant's, whose range x and the hidden activations
 * have to keep; the hidden activation keeps 16 significant bits, the experts' rows
 * fp32; a token's choices are added in order and out is rounded once. An infinite
 * value of x gives NaN. E and k
 * within the layer's limits, d and d_ff multiples of group and at most
 * MOE_FEW_MAX_WIDTH; x 16-byte aligned. workspace:
 * moe_experts_quant_workspace_size() bytes, 256-byte aligned; calls that share
 * one must not overlap. Neither out nor the workspace may overlap an input or
 * each other (MOE_ERR_ARG). N = 0 is valid. */
int moe_experts_quant(const moe_tensor *x, const int32_t *topk_idx, const float *topk_gate, int k,
                   const moe_q4 *W_up, const moe_q4 *W_down, const moe_expert_opts *opts,
                   moe_tensor *out, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace of moe_experts_quant (0 for N = 0, invalid sizes, or beyond
 * MOE_FEW_MAX_TOKENS). */
size_t moe_experts_quant_workspace_size(int64_t N, int64_t d, int64_t E, int64_t d_ff, int k,
                                     int32_t group);

/* ---------------------------------------------------------------------------
 * Routing with a balance bias, groups and renormalised gates, and the layer for
 * a routing that the caller has. Same conventions as above.
 * ------------------------------------------------------------------------- */

/* How moe_router_ex chooses and weighs experts. Zero-initialise the struct and
 * set the fields used: all zeros are softmax scores over all experts, the k
 * largest of them as the gates.
 * score        MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID of s = W_g x + noise: p
 * bias         [E] MOE_F32 or NULL, added to p for the choice alone (c = p +
 *              bias), as a balance of the experts' load adjusts it
 * groups       the experts in this many groups of E / groups adjacent ones (0:
 *              1; MOE_ERR_SHAPE unless it divides E, MOE_ERR_UNSUPPORTED past 64)
 * keep_groups  groups whose experts may be chosen (0: all): those with the
 *              largest scores, equal ones by the lower group
 * group_best   1 or 2 (0: 1): a group's score is the sum of its that many
 *              largest c (of one in a group of one)
 * renormalize  nonzero: gates are divided by the sum of the chosen p
 * scale        gates are multiplied by it; finite, >= 0 (0: 1)
 * gates        moe_router_backward with renormalize alone: the topk_gate that the
 *              forward wrote (fp32 [N, k], device, 4-byte aligned), or NULL */
enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
typedef struct {
    int32_t score;
    const moe_tensor *bias;
    int32_t groups;
    int32_t keep_groups;
    int32_t group_best;
    int32_t renormalize;
    float scale;
    const float *gates;
} moe_router_opts;

/* moe_router with these options (NULL: all zeros): topk_idx [N, k] int32, the k
 * largest c in descending order (equal values: lower id first), and their gates
 * topk_gate [N, k] fp32; scores, if not NULL, the p of all experts, [N, E]
 * MOE_F32, for an auxiliary loss or the backward (which takes bf16 x alone). k at most the experts of the
 * kept groups (MOE_ERR_ARG). x, W_g and noise as moe_router's, d at most
 * MOE_ROUTE_MAX_WIDTH (MOE_ERR_UNSUPPORTED), all arithmetic fp32. A NaN score counts as -inf (p = 0); where the chosen p sum to 0,
 * renormalised gates are 0 (those of a softmax are formed from the scores and do
 * not underflow together); softmax scores with infinities share 1 equally. No
 * output, nor the workspace, may overlap an input, another output or each other
 * (MOE_ERR_ARG). workspace: moe_router_ex_workspace_size() bytes, 256-byte
 * aligned (may be NULL when that is 0). N = 0 is valid. */
int moe_router_ex(const moe_tensor *x, const moe_tensor *W_g, const moe_tensor *noise,
                  const moe_router_opts *opts, int k, int32_t *topk_idx, float *topk_gate,
                  moe_tensor *scores, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of scratch of moe_router_ex (0 when it needs none, or on invalid sizes). */
size_t moe_router_ex_workspace_size(int64_t N, int64_t d, int64_t E, int32_t dtype);

/* Its backward, for dgate [N, k] MOE_F32 the gradient of the gates and dscores
 * [N, E] MOE_F32 (or NULL) that of the exported scores, from an auxiliary loss:
 *   ds the gradient of s: through the scaling, the renormalisation and the
 *   softmax or sigmoid (the choice passes none),
 *   dW_g = ds^T x,  dx = ds W_g + dres
 * topk_idx and scores are the forward's; an id outside [0, E) has no gate. The
 * gradient of renormalised gates takes each one's share p / sum of the chosen p from
 * opts->gates; without them from the scores, which for a softmax underflow where the
 * forward's gates do not: chosen p below fp32's normal range (2^-126) then give shares
 * of as few bits as they have, and where all are 0 no gradient.
 * x [N, d] and W_g [E, d] as the forward's, bf16 x (MOE_ERR_UNSUPPORTED for
 * fp32, and past MOE_ROUTE_MAX_GRAD_ROWS tokens). dx [N, d] MOE_F32 or MOE_BF16, dres (or NULL) like it: a gradient that
 * reaches x another way, as the layer's own; dx may be its buffer. dW_g [E, d]
 * MOE_F32. dx or dW_g may be NULL and is then not computed (both:
 * MOE_ERR_NULL; dres without dx: MOE_ERR_ARG). Sums are fp32 in a fixed order,
 * products as accurate as fp32 ones. x, W_g, dres, dx and dW_g 16-byte aligned. No output, nor the workspace, may overlap
 * an input otherwise, another output or each other (MOE_ERR_ARG). workspace:
 * moe_router_backward_workspace_size() bytes, 256-byte aligned. N = 0: dW_g is
 * zero. */
int moe_router_backward(const moe_tensor *x, const moe_tensor *W_g, const moe_router_opts *opts,
                        int k, const int32_t *topk_idx, const moe_tensor *scores,
                        const moe_tensor *dgate, const moe_tensor *dscores,
                        const moe_tensor *dres, moe_tensor *dx, moe_tensor *dW_g, void *workspace,
                        size_t workspace_bytes, void *stream);

/* Bytes of scratch of moe_router_backward (0 for N = 0 or invalid sizes). */
size_t moe_router_backward_workspace_size(int64_t N, int64_t d, int64_t E, int k);

/* moe_forward_ex for a routing that the caller has: stats->topk_idx and
 * stats->topk_gate are inputs (required for N > 0, 4-byte aligned), the rest is as
 * there (an id outside [0, E) takes no slot). The workspace of moe_forward serves it;
 * no written buffer may overlap the routing or another one (MOE_ERR_ARG). */
int moe_forward_routed(const moe_tensor *x, const moe_tensor *W_up, const moe_tensor *W_down,
                       const moe_expert_opts *opts, int k, float capacity_factor, moe_tensor *out,
                       moe_stats *stats);

/* Its backward: moe_backward_ex without the router. dx is the experts' part
 * alone (moe_router_backward's dres), dgate [N, k] MOE_F32 the gradient of each
 * gate, <dout, y> (0 for dropped choices): moe_router_backward's. The workspace
 * of moe_backward serves it; stats as moe_forward_routed's. No written buffer may
 * overlap the routing or another one, nor dgate any input (MOE_ERR_ARG). */
int moe_backward_routed(const moe_tensor *x, const moe_tensor *W_up, const moe_tensor *W_down,
                        const moe_expert_opts *opts, int k, float capacity_factor,
                        const moe_tensor *dout, moe_tensor *dx, moe_tensor *dgate,
                        moe_tensor *dW_up, moe_tensor *dW_down, moe_tensor *db_up,
                        moe_tensor *db_down, moe_stats *stats);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
