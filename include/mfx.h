/*
 * mfx.h -- C ABI of libmfx, fused transformer MLP and residual epilogues for
 * NVIDIA GB300 (sm_103a).
 *
 * Each entry point is one fused, bandwidth-bound pass written as a CUDA
 * kernel.  The operations are those of Megatron-LM's megatron/core/fusions/
 * as the web page "Megatron-LM operator fusion walkthrough"
 * (www.wmrh.cn/news/51426) describes them; each declaration cites the
 * section of that page ("fusions page §N") that defines it.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are dense, contiguous, row-major.  `rows` is the token count
 *    (sequence x batch flattened), `cols` the hidden width.  The GLU ops take
 *    an input of width 2F whose first F columns are the activated ("gate")
 *    half and whose last F columns are the linear ("up") half.
 *  - Every data pointer is a DEVICE pointer owned by the caller.  The library
 *    never allocates, frees or synchronises.  Any alignment is accepted; a
 *    16-byte aligned pointer with a width that is a multiple of 8 takes the
 *    fastest path, other cases take a slower path with the same results.
 *  - dtype codes: MFX_F32 or MFX_BF16.  Outputs take the dtype of the main
 *    input (y or x); the bias has that dtype too; the SwiGLU weight and its
 *    gradient are always fp32.  All arithmetic is fp32 inside the kernels,
 *    with one rounding at each output store.
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream).  Calls are asynchronous: they enqueue one kernel and return.
 *  - An empty tensor (rows == 0 or a zero width) is a no-op returning MFX_OK
 *    without reading any pointer.  Negative sizes, and sizes whose element
 *    count or byte count overflows int64, return MFX_ERR_SHAPE.
 *  - Return value: an mfx_status.  Arguments are validated on the host before
 *    anything is launched, so an error status means nothing was enqueued.
 *    MFX_ERR_CUDA reports a failed launch; mfx_last_cuda_error() then gives
 *    the cudaError_t (thread-local).  Besides that and the device error word
 *    described at mfx_device_error(), the library has no global state.
 *  - Thread safety: calls from several host threads are safe; calls that
 *    overlap on the GPU and write the same buffers race, as with any kernel.
 */
#ifndef MFX_H
#define MFX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The 8-bit codes are for the quantised norm's outputs alone. */
typedef enum { MFX_F32 = 0, MFX_BF16 = 1, MFX_E4M3 = 2, MFX_E5M2 = 3, MFX_E8M0 = 4 } mfx_dtype;

typedef enum {
    MFX_OK = 0,
    MFX_ERR_NULL = 1,  /* a required pointer is NULL                          */
    MFX_ERR_SHAPE = 2, /* negative or overflowing sizes                        */
    MFX_ERR_DTYPE = 3, /* unknown dtype code                                   */
    MFX_ERR_PROB = 4,  /* dropout probability outside [0, 1) or NaN           */
    MFX_ERR_ALIAS = 5, /* buffers overlap in a way the op does not allow       */
    MFX_ERR_CUDA = 6,  /* the kernel launch failed (see mfx_last_cuda_error)   */
    MFX_ERR_DEVICE = 7, /* a kernel gave up a bounded wait (mfx_device_error)  */
    MFX_ERR_WORKSPACE = 8, /* workspace too small or not 16-byte aligned       */
    MFX_ERR_VALUE = 9  /* a scalar argument outside its range                  */
} mfx_status;

/* ------------------------------------------------------------------------ */
/* Bias + GeLU (tanh approximation), fusions page §4.2 bias_gelu(bias, y) and */
/* §4.2 bias_gelu_back(g, bias, y).                                           */
/* ------------------------------------------------------------------------ */

/* out[r,c] = gelu(x), x = y[r,c] + bias[c],
 *   gelu(x) = x * 0.5 * (1 + tanh(0.79788456 * x * (1 + 0.044715 * x * x))).
 * y, out: [rows, cols] of dtype dt.  bias: [cols] of dtype dt, or NULL (no
 * bias).  out may equal y (in place); any other overlap -> MFX_ERR_ALIAS. */
int mfx_bias_gelu_fwd(int dt, int64_t rows, int64_t cols,
                      const void* bias, const void* y, void* out, void* stream);

/* dy[r,c] = g[r,c] * gelu'(x), x = y[r,c] + bias[c], with the page's
 * derivative of the tanh form (its constant 0.1070322243 = 3 * 0.79788456 *
 * 0.044715):  gelu'(x) = 0.5 x (1 - t^2)(0.79788456 + 0.1070322243 x^2)
 *                        + 0.5 (1 + t),  t = tanh(0.79788456 x (1 + 0.044715 x^2)).
 * g, y, dy: [rows, cols] of dtype dt; bias: [cols] or NULL.  The bias
 * gradient is the column sum of dy (the page's backward returns the same
 * tensor for input and bias); this call does not form it.  dy may equal g or
 * y; any other overlap -> MFX_ERR_ALIAS. */
int mfx_bias_gelu_bwd(int dt, int64_t rows, int64_t cols,
                      const void* g, const void* bias, const void* y, void* dy,
                      void* stream);

/* ------------------------------------------------------------------------ */
/* Bias + gated linear units, fusions page §2 (fused_bias_geglu,              */
/* fused_bias_swiglu with its weighted variant) and §9 (the weighted-SwiGLU   */
/* test).  The page names these ops; the split is: z = x + bias over the full */
/* width 2F, a = z[:, :F] is activated, b = z[:, F:] is linear.               */
/* ------------------------------------------------------------------------ */

/* out[r,c] = gelu(a) * b with the §4.2 tanh GeLU.
 * x: [rows, 2F]; bias: [2F] or NULL; out: [rows, F]; all dtype dt.
 * out must not overlap x -> MFX_ERR_ALIAS. */
int mfx_bias_geglu_fwd(int dt, int64_t rows, int64_t F,
                       const void* x, const void* bias, void* out, void* stream);

/* dx[r, c]   = g[r,c] * b * gelu'(a)
 * dx[r, F+c] = g[r,c] * gelu(a)
 * g: [rows, F]; x: [rows, 2F]; bias: [2F] or NULL; dx: [rows, 2F].
 * dx may equal x (in place); other overlaps -> MFX_ERR_ALIAS. */
int mfx_bias_geglu_bwd(int dt, int64_t rows, int64_t F,
                       const void* g, const void* x, const void* bias, void* dx,
                       void* stream);

/* out[r,c] = silu(a) * b * weight[r], silu(a) = a / (1 + exp(-a)).
 * weight: [rows] fp32 per-token weight, or NULL for the plain SwiGLU.
 * x: [rows, 2F]; bias: [2F] or NULL; out: [rows, F]; dtype dt.
 * out must not overlap x or weight -> MFX_ERR_ALIAS. */
int mfx_bias_swiglu_fwd(int dt, int64_t rows, int64_t F,
                        const void* x, const void* bias, const float* weight,
                        void* out, void* stream);

/* With gw = g[r,c] * weight[r] (or g[r,c] without weight), s = sigma(a):
 *   dx[r, c]    = gw * b * s * (1 + a * (1 - s))
 *   dx[r, F+c]  = gw * silu(a)
 *   dweight[r]  = sum_c g[r,c] * silu(a) * b        (fp32)
 * dweight: [rows] fp32, required iff weight != NULL (else MFX_ERR_NULL); the
 * row sum runs in a fixed order inside one thread block, so it is bitwise
 * reproducible run to run and GPU to GPU.  dx may equal x; other overlaps
 * -> MFX_ERR_ALIAS. */
int mfx_bias_swiglu_bwd(int dt, int64_t rows, int64_t F,
                        const void* g, const void* x, const void* bias,
                        const float* weight, void* dx, float* dweight, void* stream);

/* ------------------------------------------------------------------------ */
/* Weighted squared ReLU, fusions page §2 (fused_weighted_squared_relu, the  */
/* per-token weighted MoE activation named beside the weighted SwiGLU).  The */
/* page names the fusion without its formula; the reading here is the        */
/* squared ReLU scaled by the token's fp32 router weight, with no bias.      */
/* ------------------------------------------------------------------------ */

/* out[r,c] = relu(x[r,c])^2 * weight[r], relu(v) = max(v, 0) (NaN -> 0).
 * x, out: [rows, cols] of dtype dt; weight: [rows] fp32 (required).
 * out may equal x (in place); any other overlap of out with x or weight
 * -> MFX_ERR_ALIAS. */
int mfx_weighted_squared_relu_fwd(int dt, int64_t rows, int64_t cols,
                                  const void* x, const float* weight, void* out, void* stream);

/* dx[r,c]    = g[r,c] * weight[r] * 2 relu(x[r,c])           (dtype dt)
 * dweight[r] = sum_c g[r,c] * relu(x[r,c])^2                  (fp32)
 * g, x, dx: [rows, cols] of dtype dt; weight, dweight: [rows] fp32 (both
 * required).  One thread block owns each row's sum and adds it in a fixed
 * order, so dweight is bitwise reproducible.  dx may equal g or x; other
 * overlaps (dweight with anything, dx with weight) -> MFX_ERR_ALIAS. */
int mfx_weighted_squared_relu_bwd(int dt, int64_t rows, int64_t cols,
                                  const void* g, const void* x, const float* weight,
                                  void* dx, float* dweight, void* stream);

/* ------------------------------------------------------------------------ */
/* Scale-mask-softmax, fusions page §6.2-§6.3: ScaledSoftmax,                */
/* ScaledMaskedSoftmax and ScaledUpperTriangMaskedSoftmax, the three         */
/* autograd functions fused_softmax wraps around CUDA kernels, and the one   */
/* backward they share.  Softmax along the last dimension; fp32 arithmetic;  */
/* inputs and outputs in the dtype dt.  Unlike the page's kernels these take */
/* any row length, any sizes and any alignment (the page's kernels require   */
/* 16 < sk <= 4096 and sizes divisible by 4 and fall back to PyTorch         */
/* otherwise, §6.3).                                                         */
/* ------------------------------------------------------------------------ */

/* y = softmax(x * scale + mask) over the last dimension, x and y: [b, np,
 * sq, sk].  mask: NULL (ScaledSoftmax) or an ADDITIVE mask of dtype dt
 * (§6.2 describes it as a broadcastable additive mask) of shape [mask_b,
 * mask_np, mask_sq, sk], where each of mask_b, mask_np, mask_sq is 1
 * (broadcast) or equal to b, np, sq (else MFX_ERR_SHAPE); -inf excludes a
 * position (a boolean padding mask is the additive mask 0 / -inf).  A row
 * whose every score is -inf (nothing left) is all zeros.  Scores whose fp32
 * product x * scale overflows make their row NaN.  y may equal x (in place);
 * any other overlap of y with x or the mask -> MFX_ERR_ALIAS. */
int mfx_scaled_masked_softmax_fwd(int dt, int64_t b, int64_t np, int64_t sq, int64_t sk,
                                  const void* x, const void* mask,
                                  int64_t mask_b, int64_t mask_np, int64_t mask_sq,
                                  float scale, void* y, void* stream);

/* Causal: y = softmax over k of x * scale with k > q excluded, x and y:
 * [attn_batches, sq, sq] (the page's upper-triangle mask for GPT's causal
 * self-attention; sq == sk as §6.4's causal check demands).  Excluded
 * positions are written as exact zeros and are never read.  y may equal x;
 * other overlaps -> MFX_ERR_ALIAS. */
int mfx_scaled_upper_triang_masked_softmax_fwd(int dt, int64_t attn_batches, int64_t sq,
                                               const void* x, float scale, void* y, void* stream);

/* Backward of mfx_scaled_masked_softmax_fwd (with or without a mask): from
 * the forward's output y and the upstream gradient dy, both [rows, sk]
 * (rows = b * np * sq),
 *   dx[r, k] = scale * y[r, k] * (dy[r, k] - sum_j dy[r, j] * y[r, j]).
 * The row sum is accumulated with compensated (error-free) arithmetic.  dx
 * may equal dy or y (in place); other overlaps -> MFX_ERR_ALIAS. */
int mfx_scaled_masked_softmax_bwd(int dt, int64_t rows, int64_t sk,
                                  const void* dy, const void* y, float scale, void* dx, void* stream);

/* Backward of the causal forward, on [attn_batches, sq, sq]: the same
 * formula, with positions k > q written as exact zeros without reading dy
 * or y there. */
int mfx_scaled_upper_triang_masked_softmax_bwd(int dt, int64_t attn_batches, int64_t sq,
                                               const void* dy, const void* y, float scale,
                                               void* dx, void* stream);

/* ------------------------------------------------------------------------ */
/* Scale-mask-softmax with a learned relative position bias by buckets and   */
/* dropout: the attention-score path of encoder-decoder layers in one pass   */
/* each way.  Beside mfx_scaled_masked_softmax_fwd it needs no [np, sq, sk]  */
/* bias tensor, no stored keep mask and no stored probabilities.             */
/* ------------------------------------------------------------------------ */

/* For score row (i, h, q) of x [b, np, sq, sk], with the query at position
 * pos = q_start + (seq_start ? seq_start[i] : 0) + q of the keys 0 .. sk - 1:
 *   s_k = x_k * scale + table[bucket(k - pos), h] + mask_k
 *   P   = softmax of s over the keys that take part
 *   y_k = keep_k ? P_k * (1 / (1 - p)) : 0.
 * table: [num_buckets, np] of dtype table_dt (either code), or NULL (no bias;
 * num_buckets, max_distance and bidirectional are then not looked at).
 * Buckets of a direction, n = |k - pos|: with S of them (num_buckets / 2 per
 * direction when bidirectional, keys after the query in the upper half; else
 * num_buckets, with n = 0 for every key after the query), F = S / 2 rounded
 * down: n itself below F, else
 *   min(S - 1, F + floor((S - F) * log(n / F) / log(max_distance / F))),
 * whose borders are exact (whole-number powers are compared, so a border that
 * is a whole number belongs to the upper bucket).  2 <= S <= 128, num_buckets
 * even when bidirectional, F < max_distance <= 2048, else MFX_ERR_SHAPE.
 * mask: NULL or an ADDITIVE mask of dtype dt, [mask_b, mask_np, mask_sq, sk]
 * with each size 1 or x's; a key whose mask is -inf takes no part whatever x
 * holds there.  Finite masks are added exactly in effect: a row whose every
 * mask is the type's lowest value is the softmax of its scores.  (Scores
 * x_k * scale + table[...] beyond fp32's range over log2 e, 2.36e38, count as
 * infinite; a score of -inf leaves its key out, one of +inf or NaN makes its
 * row NaN.)  causal != 0 leaves out the keys k > pos, whose x is not read (with
 * seq_start: each sequence's unwritten part of a longer key axis).  A row in
 * which no key takes part is zeros.
 * Dropout: element (r, k), r = (i * np + h) * sq + q, has the index e =
 * elem_base + r * sk + k, and keep as in mfx_bias_dropout_add_train (same
 * generator, words and threshold); p = 0 keeps everything.
 * stats: [b, np, sq, 3] fp32, what the backward needs of each row (the shift
 * of its mask, the maximum of its scores in base-2 units and one over the sum
 * of its exponentials), or NULL (inference).
 * y: x's shape and dtype; y may equal x (in place, when no backward follows).
 * b, np, sq, sk and |q_start| at most 2^29, b * sq at most 2^30.  One query
 * per sequence over a long key axis (decoding) splits a row over several
 * thread blocks. */
int mfx_relbias_softmax_dropout_fwd(int dt, int64_t b, int64_t np, int64_t sq, int64_t sk,
                                    const void* x, float scale,
                                    int table_dt, const void* table, int64_t num_buckets, int64_t max_distance,
                                    int bidirectional,
                                    const void* mask, int64_t mask_b, int64_t mask_np, int64_t mask_sq,
                                    int causal, int64_t q_start, const int32_t* seq_start,
                                    float p, uint64_t seed, uint64_t offset, uint64_t elem_base,
                                    void* y, float* stats, void* stream);

/* Backward, from the forward's inputs and stats and the gradient dy of y:
 *   dP_k = keep_k ? dy_k * (1 / (1 - p)) : 0,  D = sum_k dP_k P_k
 *   dS_k = P_k (dP_k - D)
 *   dx_k = scale * dS_k                        (dtype dt; zeros where left out)
 *   dtable[u, h] = sum of dS over the positions of head h in bucket u
 * P and keep are formed again; dy does not count at keys that take no part.  dtable:
 * [num_buckets, np] of dtype table_dt, from fp32 sums rounded once, or NULL
 * (not formed; needs no workspace).  The sums run in a fixed order, so dtable
 * is bitwise reproducible on a given GPU model; with an empty x it is set to
 * zero.  The workspace protocol is that of the fused bias gradients below
 * (workspace == NULL with workspace_bytes given asks for the size).  dx may
 * equal dy or x; other overlaps -> MFX_ERR_ALIAS.  The other arguments are
 * the forward's. */
int mfx_relbias_softmax_dropout_bwd(int dt, int64_t b, int64_t np, int64_t sq, int64_t sk,
                                    const void* dy, const void* x, const float* stats, float scale,
                                    int table_dt, const void* table, int64_t num_buckets, int64_t max_distance,
                                    int bidirectional,
                                    const void* mask, int64_t mask_b, int64_t mask_np, int64_t mask_sq,
                                    int causal, int64_t q_start, const int32_t* seq_start,
                                    float p, uint64_t seed, uint64_t offset, uint64_t elem_base,
                                    void* dx, void* dtable, void* workspace, size_t* workspace_bytes,
                                    void* stream);

/* ------------------------------------------------------------------------ */
/* Tokens sorted by expert and back, with weights applied, and the gradients: */
/* what makes, and takes up again, the rows of expert MLPs (whose activations */
/* are the weighted SwiGLU and the weighted squared ReLU above).             */
/*                                                                           */
/* Slot t * topk + j is choice j of token t.  The sorted layout has the slots */
/* of expert 0, then of expert 1, ..., in slot order within an expert; each   */
/* expert's rows begin at a multiple of `align` (1 = packed; tiles of a       */
/* grouped matrix product otherwise).  Rows without a slot are padding.       */
/* ------------------------------------------------------------------------ */

/* Rows that the layout needs at most: tokens * topk + min(experts, tokens *
 * topk) * (align - 1); -1 for negative or overflowing sizes. */
int64_t mfx_moe_rows(int64_t tokens, int64_t topk, int64_t experts, int64_t align);

/* The maps of the sorted layout, by a stable counting sort.
 * expert_of: [tokens, topk]; a value outside [0, experts) has no row (a
 * choice that the router dropped).  capacity > 0 keeps the first `capacity`
 * slots of each expert and drops the others; 0 keeps all.
 * rows: rows of the sorted buffers, at least mfx_moe_rows() (or, with a
 * capacity, experts * capacity rounded up to align, if that is less), else
 * MFX_ERR_SHAPE.  1 <= experts <= 4096; tokens * topk and rows below 2^31.
 * row_of:  [tokens, topk] row of each slot, -1 for none.
 * slot_of: [rows] slot of each row, -1 for padding.
 * offsets: [experts + 1] first row of each expert, and the end of the last.
 * counts:  [experts] slots of each expert that have a row.
 * All int32.  Workspace protocol as for the fused bias gradients.  The size
 * may be 0 (up to 2048 slots need none, and one kernel does it all); then
 * workspace and workspace_bytes may both be NULL. */
int mfx_moe_sort(int64_t tokens, int64_t topk, int64_t experts, int64_t align, int64_t capacity, int64_t rows,
                 const int32_t* expert_of, int32_t* row_of, int32_t* slot_of, int32_t* offsets, int32_t* counts,
                 void* workspace, size_t* workspace_bytes, void* stream);

/* out[row_of[t, j]] = x[t], padding rows zero; with weight, also
 * out_weight[row_of[t, j]] = weight[t, j] (0 on padding), the per-row weight
 * that the weighted activations take.
 * x: [tokens, cols], out: [rows, cols] of dtype dt; weight: [tokens, topk]
 * fp32 or NULL; out_weight: [rows] fp32, required iff weight.  Outputs must
 * not overlap anything else -> MFX_ERR_ALIAS.  Entries of the maps outside
 * their range count as -1 (here and below).  With cols 0 the outputs of fp32
 * weights are written all the same (here and below; sums over no columns are 0). */
int mfx_moe_permute_fwd(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows,
                        const void* x, const int32_t* row_of, const int32_t* slot_of, const float* weight,
                        void* out, float* out_weight, void* stream);

/* dx[t] = sum_j g[row_of[t, j]] (fp32 sum in choice order, rounded once), and
 * with g_weight (the gradient [rows] of out_weight) dweight[t, j] =
 * g_weight[row_of[t, j]], 0 where the slot has no row. */
int mfx_moe_permute_bwd(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows,
                        const void* g, const int32_t* row_of, const float* g_weight,
                        void* dx, float* dweight, void* stream);

/* out[t] = sum_j weight[t, j] * y[row_of[t, j]] (fp32 sum in choice order,
 * rounded once); weight NULL counts as ones (weights that the activation has
 * applied).  A token without rows is zeros.  y: [rows, cols], out: [tokens,
 * cols]; out must not overlap anything else -> MFX_ERR_ALIAS. */
int mfx_moe_unpermute_fwd(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows,
                          const void* y, const int32_t* row_of, const float* weight,
                          void* out, void* stream);

/* dy[row_of[t, j]] = weight[t, j] * g[t] (dtype dt), padding rows zero;
 * dweight[t, j] = sum_c g[t, c] * y[row_of[t, j], c] (fp32, in a fixed order;
 * 0 where the slot has no row), or NULL (not formed; y is then not read).
 * Outputs must not overlap anything else -> MFX_ERR_ALIAS. */
int mfx_moe_unpermute_bwd(int dt, int64_t tokens, int64_t topk, int64_t cols, int64_t rows,
                          const void* g, const void* y, const int32_t* row_of, const int32_t* slot_of,
                          const float* weight, void* dy, float* dweight, void* stream);

/* ------------------------------------------------------------------------ */
/* Root-mean-square norm with the residual's addition: what stands between    */
/* the residual path (bias-dropout-add) and the next block's first product.   */
/* The fusions page names the fused norm beside these ops without describing  */
/* it; the formulas are those of the literature (Zhang and Sennrich, 2019).   */
/*   h = x + residual,   rstd = 1 / sqrt(mean(h^2) + eps),                    */
/*   y = h * rstd * (weight + weight_offset)                                  */
/* ------------------------------------------------------------------------ */

/* x, y: [rows, cols] dtype x_dt; residual, h: [rows, cols] dtype res_dt;
 * weight: [cols] dtype w_dt, or NULL (a factor of 1); weight_offset is 1 for
 * weights that are kept around zero, else 0.  residual NULL: h = x (and h must
 * be NULL).  h (NULL: not written) is the new residual stream; y is formed
 * from it before it is rounded.  rstd: [rows] fp32, what the backward needs,
 * or NULL.  Norms are fp32: squares of values beyond 1.8e19 overflow, h *
 * (weight + weight_offset) is formed before rstd comes to it and has to be
 * within fp32's range too, and a row of zeros with eps = 0 gives NaN.
 * eps >= 0 and finite, else MFX_ERR_VALUE; cols up to 2^30.  y and h may each
 * be x's or the residual's very buffer; other overlaps -> MFX_ERR_ALIAS. */
int mfx_add_rmsnorm_fwd(int x_dt, int res_dt, int w_dt, int64_t rows, int64_t cols,
                        const void* x, const void* residual, const void* weight,
                        float eps, float weight_offset,
                        void* y, void* h, float* rstd, void* stream);

/* The same with y in 8 bits.  q: [rows, cols] of q_dt (MFX_E4M3 or MFX_E5M2),
 * q = y / s rounded to nearest even and saturated, where s is the scale of the
 * element's group: group = 0 the whole row, 32 or 128 that many columns of it
 * (a row's last group may be shorter), else MFX_ERR_VALUE.
 * s = max |y| / 448 (e4m3) or / 57344 (e5m2), at least 2^-126 and 1 for a
 * group of zeros; scale: [rows, groups of a row], MFX_F32, or MFX_E8M0: s
 * rounded up to a power of two, stored as its exponent + 127 in a byte.
 * Both are products in fp32: beside rstd's own error, an fp32 scale is off by
 * up to 2^-21 of it, and what is rounded to q by up to 2^-21 of y / s (with the
 * stored s), so that a y / s next to the middle of two values may go to either.
 * NaN stays NaN (and counts for nothing in max |y|), infinities saturate.
 * y is not rounded to x_dt on the way.  q and scale overlap nothing else. */
int mfx_add_rmsnorm_quant_fwd(int x_dt, int res_dt, int w_dt, int64_t rows, int64_t cols,
                              const void* x, const void* residual, const void* weight,
                              float eps, float weight_offset,
                              int q_dt, int64_t group, int scale_dt,
                              void* q, void* scale, void* h, float* rstd, void* stream);

/* Gradients from the stored h (x where there was no residual; dtype res_dt)
 * and rstd.  dy: [rows, cols] x_dt; dh: [rows, cols] res_dt, the gradient that
 * reaches h from further on, or NULL.  With n = h * rstd, u = dy * (weight +
 * weight_offset):
 *   d = rstd * (u - n * mean(u * n)) + dh,   dweight[c] = sum_r dy * n.
 * d is the gradient of x and of the residual alike: dx gets it as x_dt,
 * dresidual as res_dt; either may be NULL.  dweight: [cols] w_dt, or NULL.
 * The output in 8 bits is passed straight through (dy is y's gradient).
 * dweight is the same bits from run to run on a given GPU model; the workspace
 * protocol is that of the fused bias gradients below (the size may be 0: then
 * NULL sizes and workspaces run).  dx and dresidual may each be the very
 * buffer of dy, h or dh; other overlaps -> MFX_ERR_ALIAS. */
int mfx_add_rmsnorm_bwd(int x_dt, int res_dt, int w_dt, int64_t rows, int64_t cols,
                        const void* dy, const void* h, const float* rstd,
                        const void* weight, float weight_offset, const void* dh,
                        void* dx, void* dresidual, void* dweight,
                        void* workspace, size_t* workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Operators on logits [rows, vocab] of dtype dt, whose rows begin ld >= vocab */
/* elements apart (a vocabulary padded in memory; what lies between counts for */
/* nothing and is not written).  p = softmax(scale * z) over a row, scale > 0 and finite */
/* (one over the temperature), else MFX_ERR_VALUE.  Columns at -inf have p = 0,*/
/* and so have those whose scale * (z - max) passes fp32's range (log p = -inf);*/
/* powers below 2^-126 add nothing to sums and gradients.                      */
/* A row with a NaN or +inf gives NaN, unless it is left out: nothing comes of */
/* the logits of a row without a token, or without entries, whatever they are. */
/* index_bits: 32 or 64, the width of the integers that name columns, else     */
/* MFX_ERR_DTYPE.  vocab up to 2^30.                                           */
/* ------------------------------------------------------------------------ */

/* Log probabilities of given tokens, the distribution's entropy, and the `top`
 * (0 to 64, else MFX_ERR_VALUE) largest logits' log probabilities and columns.
 * tokens: [rows]; a token outside [0, vocab) leaves its row out: its results
 * are 0, its alternatives (-inf, -1), and nothing comes of its logits.
 * logprob[r] = log p[token], entropy[r] = -sum p log p (fp32).
 * top_logprob, top_index: [rows, top] in falling order, equal logits by the
 * lower column; (-inf, -1) where fewer than `top` are above -inf; columns with
 * NaN are never among them.  stats: [rows, 3] fp32, what the backward needs,
 * or NULL.  A row that is all -inf: logprob -inf, entropy 0.
 * Workspace protocol as for the fused bias gradients; the size may be 0 (no
 * alternatives, or few rows): then NULL sizes and workspaces run, and two
 * kernels otherwise.  Outputs must not overlap anything -> MFX_ERR_ALIAS. */
int mfx_token_logprobs_fwd(int dt, int64_t rows, int64_t vocab, int64_t ld,
                           const void* logits, int index_bits, const void* tokens,
                           float scale, int64_t top,
                           float* logprob, float* entropy,
                           float* top_logprob, int32_t* top_index, float* stats,
                           void* workspace, size_t* workspace_bytes, void* stream);

/* dlogits[r, k] = scale * (g (1[token = k] - p) - ge p (log p + entropy)) in
 * dtype dt, rows ld_out apart, from the gradients g of logprob and ge of
 * entropy ([rows] fp32; either may be NULL) and the forward's inputs and stats.
 * Rows that are left out or all -inf get zeros.  dlogits may be the very
 * buffer of logits (with ld_out == ld); other overlaps -> MFX_ERR_ALIAS. */
int mfx_token_logprobs_bwd(int dt, int64_t rows, int64_t vocab, int64_t ld,
                           const float* g_logprob, const float* g_entropy,
                           const void* logits, int index_bits, const void* tokens,
                           const float* stats, float scale,
                           void* dlogits, int64_t ld_out, void* stream);

/* Distillation from a teacher's top logits.  index, teacher: [rows, k] columns
 * and the teacher's logits t there (dtype t_dt), 0 <= k <= 1024; a column
 * outside [0, vocab) is no entry, and a column may come twice (its entries'
 * q add up).  q = softmax(scale * t) over a row's entries, or, with
 * teacher_lse [rows] fp32, exp(scale * t - teacher_lse): the teacher's own
 * normalisation over its whole vocabulary.
 *   loss[r] = sum_j q_j (log q_j - log p[column j])           (fp32)
 * (+inf where a column with q > 0 has p = 0).  A row whose list names no column,
 * or whose entries are all -inf, has no entries: loss 0, whatever teacher_lse
 * says of it.
 * stats: [rows, 4] fp32, what the backward needs, or NULL. */
int mfx_topk_distill_fwd(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k,
                         const void* logits, int index_bits, const void* index,
                         const void* teacher, const float* teacher_lse, float scale,
                         float* loss, float* stats, void* stream);

/* dlogits = g * scale * (sum(q) p - q at its columns), from the gradient g
 * [rows] (fp32) of the loss; rows without entries, and rows that are all -inf,
 * get zeros.  dlogits as for the log probabilities. */
int mfx_topk_distill_bwd(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k,
                         const float* g, const void* logits, int index_bits, const void* index,
                         const void* teacher, const float* stats, float scale,
                         void* dlogits, int64_t ld_out, void* stream);

/* Both in one call, for a loss whose gradient is known before it (a weight for
 * each row, [rows] fp32, in the place of g): the logits are read from memory
 * once instead of twice. */
int mfx_topk_distill_fwd_bwd(int dt, int t_dt, int64_t rows, int64_t vocab, int64_t ld, int64_t k,
                             const void* logits, int index_bits, const void* index,
                             const void* teacher, const float* teacher_lse,
                             const float* weight, float scale,
                             float* loss, void* dlogits, int64_t ld_out, void* stream);

/* ------------------------------------------------------------------------ */
/* Bias + dropout + residual add, fusions page §3.2-§3.3                     */
/* (_bias_dropout_add_func(x_with_bias, residual, prob, training) and its    */
/* two entry points bias_dropout_add_fused_train / _inference).              */
/* ------------------------------------------------------------------------ */

/* Training:  out = r~ + dropout(x + bias, p), where r~ is the residual cast
 * to x's dtype ("residual.to(x.dtype)", §3.2) and dropout keeps an element
 * with probability 1 - p and scales it by 1 / (1 - p) (computed in fp32).
 * x: [rows, cols] dtype x_dt; bias: [cols] x_dt or NULL; residual: [rows,
 * cols] dtype res_dt (either code); out: [rows, cols] x_dt; keep_mask:
 * [rows, cols] uint8, 1 = kept, 0 = dropped (a dropped element contributes
 * exactly +0, so out == r~ there).
 * Randomness: element (r, c) has global index e = elem_base + r * cols + c;
 * Philox4x32-10 (Salmon et al., SC'11) with key (lo32 seed, hi32 seed) and
 * counter (lo32 e/8, hi32 e/8, lo32 offset, hi32 offset) gives 128 bits, of
 * which 16-bit word e % 8 (little-endian) is the element's uniform u; the
 * element is kept iff u >= min(65535, ceil(p * 65536)).  The mask is thus a
 * pure function of (seed, offset, e): shards of one tensor processed with
 * their own elem_base reproduce the unsharded mask.
 * p must lie in [0, 1) (else MFX_ERR_PROB); p = 0 keeps everything.
 * out may equal x; out must not overlap residual or keep_mask, keep_mask
 * must not overlap any input -> MFX_ERR_ALIAS. */
int mfx_bias_dropout_add_train(int x_dt, int res_dt, int64_t rows, int64_t cols,
                               const void* x, const void* bias, const void* residual,
                               float p, uint64_t seed, uint64_t offset, uint64_t elem_base,
                               void* out, uint8_t* keep_mask, void* stream);

/* mfx_bias_dropout_add_train with the keep mask as bits instead of bytes:
 * bit (i mod 8) of keep_bits[i / 8] (least significant bit first) is the keep
 * flag of element i = r * cols + c of this call, so the mask takes
 * ceil(rows * cols / 8) bytes (the last byte's unused high bits are 0).  The
 * same elements are kept and out is the same bits as with the byte mask;
 * the mask traffic drops from 1 to 1/8 byte per element (bf16 x with an
 * fp32 residual: 8.125 instead of 9 bytes per element).  Fastest when x,
 * out and the residual are 16-byte aligned.  keep_bits must not overlap any
 * other buffer -> MFX_ERR_ALIAS; the other rules are the training call's. */
int mfx_bias_dropout_add_train_packed(int x_dt, int res_dt, int64_t rows, int64_t cols,
                                      const void* x, const void* bias, const void* residual,
                                      float p, uint64_t seed, uint64_t offset, uint64_t elem_base,
                                      void* out, uint8_t* keep_bits, void* stream);

/* mfx_bias_dropout_add_train without a mask: the same elements are kept and
 * out is the same bits, but no keep flags are written.  The backward draws
 * them again: mfx_bias_dropout_add_bwd (or _dbias) with keep_mask NULL and
 * this call's p, seed, offset and elem_base.  8 instead of 9 bytes per
 * element (bf16 x, fp32 residual). */
int mfx_bias_dropout_add_train_nomask(int x_dt, int res_dt, int64_t rows, int64_t cols,
                                      const void* x, const void* bias, const void* residual,
                                      float p, uint64_t seed, uint64_t offset, uint64_t elem_base,
                                      void* out, void* stream);

/* Plain dropout (embeddings, a layer stack's last output) whose mask is never
 * stored: out[i] = keep ? x[i] * (1 / (1 - p)) : 0 for n elements of dtype dt,
 * element i having the index elem_base + i of the generator described at
 * mfx_bias_dropout_add_train.  The backward does the same to the gradient:
 * dx[i] = keep ? g[i] * (1 / (1 - p)) : 0.  out may equal x (dx g); any other
 * overlap -> MFX_ERR_ALIAS.  Bit-exact: fp32 multiply, one rounding. */
int mfx_dropout_fwd(int dt, int64_t n, const void* x, float p, uint64_t seed, uint64_t offset,
                    uint64_t elem_base, void* out, void* stream);
int mfx_dropout_bwd(int dt, int64_t n, const void* g, float p, uint64_t seed, uint64_t offset,
                    uint64_t elem_base, void* dx, void* stream);

/* Inference: x = (x + bias) + r~, IN PLACE in x (§3.2: when not training the
 * bias add, dropout and residual add all run in place).  p, seed and offset
 * are accepted for symmetry with the training call and ignored (p is still
 * validated).  x must not overlap residual or bias -> MFX_ERR_ALIAS. */
int mfx_bias_dropout_add_inference(int x_dt, int res_dt, int64_t rows, int64_t cols,
                                   void* x, const void* bias, const void* residual,
                                   float p, uint64_t seed, uint64_t offset, void* stream);

/* Backward of the training call (the gradients the fusions page's §3.4 unit
 * test compares between fused and unfused versions), given the upstream
 * gradient g = dL/dout [rows, cols] of dtype x_dt:
 *   dx[i]        = keep[i] ? g[i] * (1 / (1 - p)) : 0      (x_dt)
 *                  -- also the bias gradient before its column sum
 *   dresidual[i] = g[i] in the residual's dtype res_dt      (the cast's backward)
 * keep_mask: the forward's mask, or NULL to regenerate it from (seed, offset,
 * elem_base, p), which must then be the forward's values (no mask read: two
 * bytes per element less traffic in bf16).  dresidual may be NULL (not
 * written), or equal g when res_dt == x_dt (nothing to write).  dx may equal
 * g (in place); other overlaps -> MFX_ERR_ALIAS.  Bit-exact: fp32 multiply,
 * one rounding. */
int mfx_bias_dropout_add_bwd(int x_dt, int res_dt, int64_t rows, int64_t cols,
                             const void* g, const uint8_t* keep_mask,
                             float p, uint64_t seed, uint64_t offset, uint64_t elem_base,
                             void* dx, void* dresidual, void* stream);

/* mfx_bias_dropout_add_bwd reading the bit mask of
 * mfx_bias_dropout_add_train_packed (keep_bits, required): dx and dresidual
 * are the same bits as with the byte mask.  Fastest when g, dx, dresidual
 * and keep_bits are 16-byte aligned and rows * cols is a multiple of 8. */
int mfx_bias_dropout_add_bwd_packed(int x_dt, int res_dt, int64_t rows, int64_t cols,
                                    const void* g, const uint8_t* keep_bits, float p,
                                    void* dx, void* dresidual, void* stream);

/* ------------------------------------------------------------------------ */
/* Fused bias gradients.  The fusions page's backward hands one gradient      */
/* tensor to the input and to the broadcast bias (§4.3, "both return tmp"),  */
/* and autograd sums it over the rows.  These variants of the backward calls */
/* also write that column sum, dbias[c] = sum_r grad[r, c] of the gradient as */
/* stored (rounded to its dtype), without reading the gradient back: each    */
/* thread adds the values it stores for its columns into a partial sum, the  */
/* partials land in a caller-provided fp32 workspace, and a second small     */
/* kernel adds them per column in a fixed order (same bits run to run on a   */
/* given GPU model) and rounds once to the bias dtype.                       */
/*                                                                           */
/* Workspace protocol: call with workspace == NULL to get the required size  */
/* in *workspace_bytes (nothing is launched; sizes and dtype must be the     */
/* real ones, the current device is assumed); then call with a 16-byte       */
/* aligned device buffer of at least that size and its size in               */
/* *workspace_bytes (else MFX_ERR_WORKSPACE).  The buffer is scratch: its    */
/* contents on entry do not matter.  dbias has the gradient's dtype; with    */
/* rows == 0 it is set to zero.                                              */
/* ------------------------------------------------------------------------ */

/* mfx_bias_gelu_bwd, plus dbias[c] = sum_r dy[r, c] (dbias: [cols]). */
int mfx_bias_gelu_bwd_dbias(int dt, int64_t rows, int64_t cols,
                            const void* g, const void* bias, const void* y, void* dy,
                            void* dbias, void* workspace, size_t* workspace_bytes, void* stream);

/* The same as mfx_bias_gelu_bwd_dbias, for callers that cannot hand the
 * library a workspace: code whose device memory is all owned by a pool that
 * does not give library calls scratch buffers, code on a path where a device
 * allocation (which can synchronise the device) is not acceptable, and C
 * callers with no device allocator of their own.  The fusions page has no
 * counterpart; this is a calling convention, not another operation.
 *   - It allocates nothing.  The partial sums go to a fixed 4 MiB array
 *     inside the library, which every GPU that loads the library holds until
 *     the process exits.
 *   - When the size mfx_bias_gelu_bwd_dbias would ask for fits in the array
 *     (on a GB300 its pipelined partials take about 2.5 MB whatever the
 *     shape), the call runs exactly what that entry point runs: dy and dbias
 *     are the same bits.  Otherwise (a device with more resident threads)
 *     it runs the plain backward and the row-interleaved partial layout,
 *     min(rows, 64) partial sums per column, which needs
 *     min(rows, 64) x cols x 4 bytes: dy is still the same bits, dbias is
 *     the same sum in another fixed order (it may differ in the last bits).
 *     Every width up to 16384 columns is therefore accepted.  A problem that
 *     fits neither way returns MFX_ERR_WORKSPACE and launches nothing; use
 *     mfx_bias_gelu_bwd_dbias then.
 *   - The first call on each device looks up that device's array address
 *     (with that device current) and keeps it for later calls.
 *   - Every call uses the same array, so calls whose kernels overlap on the
 *     GPU (different streams, different host threads) race and give wrong
 *     results; serialise them.  Nothing from an earlier call needs clearing:
 *     each call writes every slot it reads. */
int mfx_bias_gelu_bwd_dbias_noalloc(int dt, int64_t rows, int64_t cols,
                                    const void* g, const void* bias, const void* y, void* dy,
                                    void* dbias, void* stream);

/* mfx_bias_geglu_bwd, plus dbias[c] = sum_r dx[r, c] over the full width 2F
 * (dbias: [2F], the gradient of the bias added before the split). */
int mfx_bias_geglu_bwd_dbias(int dt, int64_t rows, int64_t F,
                             const void* g, const void* x, const void* bias, void* dx,
                             void* dbias, void* workspace, size_t* workspace_bytes, void* stream);

/* mfx_bias_swiglu_bwd, plus dbias[c] = sum_r dx[r, c] (dbias: [2F]).  With a
 * weight the backward owns rows, so the partial sums come from one extra
 * read of dx. */
int mfx_bias_swiglu_bwd_dbias(int dt, int64_t rows, int64_t F,
                              const void* g, const void* x, const void* bias,
                              const float* weight, void* dx, float* dweight,
                              void* dbias, void* workspace, size_t* workspace_bytes, void* stream);

/* mfx_bias_dropout_add_bwd, plus dbias[c] = sum_r dx[r, c] (dbias: [cols]). */
int mfx_bias_dropout_add_bwd_dbias(int x_dt, int res_dt, int64_t rows, int64_t cols,
                                   const void* g, const uint8_t* keep_mask,
                                   float p, uint64_t seed, uint64_t offset, uint64_t elem_base,
                                   void* dx, void* dresidual, void* dbias,
                                   void* workspace, size_t* workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Status helpers                                                            */
/* ------------------------------------------------------------------------ */

/* Static English description of a status code (never NULL). */
const char* mfx_status_string(int status);

/* cudaError_t of the last MFX_ERR_CUDA returned on this host thread (0 if
 * none). */
int mfx_last_cuda_error(void);

/* Kernels that stream through shared memory wait on barriers for their own
 * bulk copies; every such wait is bounded (a few seconds), and a kernel whose
 * wait runs out stops early, leaving its outputs unfinished, and records a
 * nonzero code in a per-device error word.  This call synchronises the
 * current device, copies the word into *code (if code is not NULL), clears it
 * and returns MFX_ERR_DEVICE if it was nonzero, else MFX_OK.  A correct
 * program never sees a nonzero word; the word is the library's only device
 * state besides the kernels. */
int mfx_device_error(unsigned* code);

/* Library ABI version, (major << 16) | minor. */
int mfx_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MFX_H */
