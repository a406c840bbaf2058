/*
 * forge.h -- C ABI of libforge.so: the weight-gradient GEMM dW = X^T dY with
 * the optimizer step fused into its tiled epilogue, for NVIDIA GB300
 * (compute capability 10.3, sm_103a).
 *
 * What the operations are (FORGE assessment PR, tessera#565, "docs(audit):
 * FORGE assessment + residency-aware epilogue-fusion track"):
 *   - The weight gradient of a linear layer is dW = X^T dY ("What's already
 *     in tree and easy to miss": dRhs = matmul(lhs, dy, transposeA=true)).
 *   - The optimizer step runs in the GEMM's tiled epilogue, so the gradient
 *     never reaches device memory (opening paragraph).  Each output tile is
 *     owned by one CTA and keeps the whole token dimension K (the full_k
 *     legality condition of FORGE Prop. 1, same section), so there is no
 *     split-K and no atomic accumulation; results are bitwise reproducible
 *     ("Math verified, not asserted", P1).
 *   - The fp32 accumulator feeds the optimizer state without truncation to
 *     bf16 (P6; the "truncf" item of "What's already in tree").
 *   - AdamW and SGD with momentum are the optimizers ("Claim hygiene on the
 *     source").  AdamW follows torch.optim.AdamW: W <- W (1 - lr wd);
 *     m <- b1 m + (1-b1) g; v <- b2 v + (1-b2) g^2;
 *     W <- W - lr (m / (1-b1^t)) / (sqrt(v / (1-b2^t)) + eps).
 *     SGD follows torch.optim.SGD (dampening 0, no Nesterov):
 *     g' = g + wd W; buf <- mu buf + g'; W <- W - lr buf.
 *   - The fused steps offer no gradient clipping: exact global-norm clipping
 *     cannot be fused ("Math verified, not asserted", P2).  The paths that
 *     hold gradients in memory clip them with forge_grad_norm and
 *     forge_clip_grads before the owner's step.
 *   - A routed (expert) weight whose expert received no tokens still takes
 *     the step with g = 0, i.e. m and v decay by b1, b2 and W by its weight
 *     decay (P5).
 *
 * Layouts (all row-major, element strides 1, no padding):
 *   X  [K, N]   activations, token-major (K tokens, N = d_in)
 *   dY [K, M]   output gradients, token-major (M = d_out)
 *   W, m, v, buf, dW  [N, M]   ([E, N, M] for the grouped call)
 *   dW[n][m] = sum_k X[k][n] * dY[k][m]  (times sX * sdY for e4m3 inputs)
 * An nn.Linear weight [d_out, d_in] is the transpose of W; pass it as its
 * [d_in, d_out] row-major view.
 *
 * Ownership and ordering: every pointer is caller-owned device memory of
 * the current device (cudaMalloc, a memory pool or a virtual-memory mapping;
 * host memory, managed memory and a peer GPU's memory are refused) and the
 * library keeps no pointer after the call returns.  Calls whose operands TMA
 * can address allocate nothing.  Four cases take stream-ordered scratch from
 * a memory pool the library creates per device (allocated and freed on
 * `stream`; the pool keeps what it has reserved, at most the largest scratch
 * in use at once, until the process ends):
 *   - an operand (X or dY; for dX, dY or Wb) whose base is not 16-byte
 *     aligned or whose row stride is not a multiple of 16 bytes (any odd
 *     bf16 width, any e4m3 width not divisible by 16) is first copied into
 *     rows padded to 16 bytes (one extra read and write of that operand).
 *     If that allocation fails, or the environment variable
 *     FORGE_MISALIGNED is "loader", an X or dY of the weight-gradient calls
 *     whose rows are a multiple of 4 bytes is fetched by the kernel itself
 *     with cp.async instead; other rows need the copy, and a failed
 *     allocation returns FORGE_ERR_CUDA.  forge_wgrad_adamw_noalloc stages
 *     into a fixed buffer instead;
 *   - forge_backward_adamw without a bf16 weight copy (see there);
 *   - forge_embedding_grad and forge_embedding_adamw (the order of the tokens);
 *   - forge_grad_norm (partial sums).
 * W, m, v, buf are updated in place.  Calls are asynchronous and ordered on
 * `stream`, and can be captured in a CUDA graph once a first call has run
 * on the device; the return value reports only host-side validation and
 * launch errors.  Errors detected on the device (a bounded wait that
 * ran out) are recorded in a device status word read by
 * forge_get_device_status().  The library resolves the device addresses of
 * its own device variables (that status word, the no-allocation staging
 * buffer) once per device ordinal and keeps them; they belong to the device's
 * primary context, so calls after cudaDeviceReset, or from a context other
 * than the primary one, are not supported.
 *
 * Environment (each read on every call unless noted; none is needed):
 *   FORGE_MISALIGNED = stage | loader  how X, dY rows TMA cannot address
 *                      reach the kernel (default stage, see above)
 *   FORGE_KERNEL = single | pair       the weight-gradient kernel form:
 *                      one CTA per 128 x 256 tile, or CTA pairs on 256 x 256
 *                      tiles (default: pairs when d_out > 128)
 *   FORGE_RASTER_BAND = n              d_out tiles per raster band of the
 *                      tile walk (default 8; 0 = whole rows); the results
 *                      do not depend on it
 *   FORGE_DGRAD_KERNEL = single | pair the dX kernel form (default: pairs
 *                      unless K fits one 128-token tile)
 *   FORGE_WAIT_TIMEOUT_MS = ms         limit of every device-side wait
 *                      (read once per process; default 10000)
 *
 * Caller preconditions (not checked):
 *   - X and dY do not overlap W, m, v, buf or dW.
 *   - dX = dY W^T has already consumed the old W (the in-place
 *     "dX-before-update" hazard, "Math verified, not asserted", P1).
 *   - W's whole gradient for this step is X^T dY: no tied or shared use
 *     (the single-use guard of P1).
 *
 * Host-side checks run before any launch, in this order: null pointers
 * (X and dY may be NULL only when K == 0), sizes (M >= 1, N >= 1, K >= 0,
 * E >= 1, step >= 1), dtypes, then the device (compute capability 10.3),
 * then residency (every pointer the call reads or writes is device memory
 * of the current device, else FORGE_ERR_INVALID_ARG), then alignment (X, dY:
 * bases aligned to their element size, rows of any length; W, dW: 4-byte
 * bases; m, v, buf: bases aligned to their element size; see
 * FORGE_ERR_MISALIGNED).  The checks up to the dtypes need no GPU.
 */
#ifndef FORGE_H
#define FORGE_H

#include <stdint.h>

#if defined(__GNUC__)
#define FORGE_API __attribute__((visibility("default")))
#else
#define FORGE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without including the CUDA headers (same underlying type). */
typedef struct CUstream_st* forge_stream_t;

typedef enum {
    FORGE_OK = 0,
    FORGE_ERR_INVALID_ARG = -1,       /* null pointer, bad size or hyperparameter, or a
                                         pointer that is not device memory of the
                                         current device */
    FORGE_ERR_UNSUPPORTED_DTYPE = -2, /* dtype outside the supported set */
    FORGE_ERR_UNSUPPORTED_DEVICE = -3,/* no device, or compute capability != 10.3 */
    FORGE_ERR_MISALIGNED = -4,        /* a base pointer not aligned to its element size */
    FORGE_ERR_CUDA = -5,              /* a CUDA runtime / driver call failed */
    FORGE_ERR_TIMEOUT = -6,           /* a device-side bounded wait ran out */
    FORGE_ERR_SCRATCH_TOO_SMALL = -7  /* forge_wgrad_adamw_noalloc: staging exceeds its buffer */
} forge_status;

typedef enum {
    FORGE_BF16 = 0, /* bfloat16 */
    FORGE_E4M3 = 1, /* OCP fp8 E4M3 ("fn": no infinities, max 448) */
    FORGE_F32 = 2,  /* IEEE binary32 */
    FORGE_I32 = 3,  /* token ids only: 32-bit signed integers */
    FORGE_I64 = 4   /* token ids only: 64-bit signed integers */
} forge_dtype;

/*
 * Fused dW = X^T dY and one AdamW step on W, m, v.
 *   X, dY        device, [K, N] and [K, M] of in_dtype (FORGE_BF16 or
 *                FORGE_E4M3).  K may be 0: the step then runs with g = 0.
 *   W            device fp32 [N, M], updated in place.
 *   m, v         device [N, M] of state_dtype (FORGE_F32 or FORGE_BF16),
 *                updated in place.  With bf16 state, W is updated from the
 *                unrounded fp32 m, v and then m, v are stored rounded to
 *                nearest even.
 *   lr, beta1, beta2, eps, wd   AdamW hyperparameters (0 < beta < 1,
 *                lr >= 0, eps >= 0, wd >= 0).
 *   step         1-based step count after incrementing (as torch's AdamW).
 *   scales       device fp32 [2] = {sX, sdY} for FORGE_E4M3 inputs (the
 *                gradient is sX * sdY * X^T dY); must be NULL for bf16.
 * Row strides: N * elemsize(in_dtype) and M * elemsize(in_dtype) bytes, of
 * any length (rows TMA cannot address are staged, see above).
 */
FORGE_API forge_status forge_wgrad_adamw(const void* X, const void* dY, float* W, void* m, void* v,
                               int64_t M, int64_t N, int64_t K, forge_dtype in_dtype,
                               forge_dtype state_dtype, float lr, float beta1, float beta2,
                               float eps, float wd, int64_t step, const float* scales,
                               forge_stream_t stream);

/*
 * forge_wgrad_adamw without any device allocation.  The FORGE pages have no
 * counterpart to this call: it is a library variant of forge_wgrad_adamw for
 * callers that must not allocate device memory during a step.  Arguments,
 * layouts, checks and results are those of forge_wgrad_adamw (the results
 * are bitwise identical); only the staging copy of an operand whose base or
 * row stride is not 16-byte aligned differs: it goes into a fixed 256 MiB
 * buffer per device, a file-scope device array inside the library, instead
 * of a stream-ordered allocation.
 *   - Oversize: a call whose staging copy needs more than the buffer
 *     ((rows of X, dY) x (row bytes rounded up to 16), summed over the
 *     operands that need staging) returns FORGE_ERR_SCRATCH_TOO_SMALL before
 *     any launch and changes nothing.  Aligned operands need no staging.
 *   - Races: the buffer is shared by every call of this function on the
 *     device.  Calls that stage must be ordered (one stream, or streams
 *     synchronised with each other); two overlapping calls on unordered
 *     streams overwrite each other's staging copy.  forge_wgrad_adamw and
 *     the other entry points never touch the buffer.
 *   - State: each call writes every byte of the buffer that its kernel then
 *     reads (the padding after each staged row lies outside the tensor maps),
 *     so nothing carries over from an earlier call.
 *   - First-call setup: the first call on a device resolves the buffer's
 *     address (cudaGetSymbolAddress) and caches it for that device ordinal.
 *     Under lazy module loading (the CUDA default) this first call loads the
 *     library module holding the buffer and reserves its 256 MiB there for
 *     the life of the process; with CUDA_MODULE_LOADING=EAGER every device
 *     reserves it as soon as the process creates its context there, whether
 *     or not this function is ever called.  Make that first call outside
 *     stream capture; later calls are capturable.  The cached address
 *     belongs to the device's primary context: calls after cudaDeviceReset,
 *     or from another context on the device, are not supported.
 *   - FORGE_MISALIGNED=loader selects the kernel's own cp.async loader here
 *     too for rows that are a multiple of 4 bytes (no staging, no buffer);
 *     other rows are still staged into the buffer.
 */
FORGE_API forge_status forge_wgrad_adamw_noalloc(const void* X, const void* dY, float* W, void* m,
                                                 void* v, int64_t M, int64_t N, int64_t K,
                                                 forge_dtype in_dtype, forge_dtype state_dtype,
                                                 float lr, float beta1, float beta2, float eps,
                                                 float wd, int64_t step, const float* scales,
                                                 forge_stream_t stream);

/*
 * Several AdamW weight-gradient steps that share X, in one launch: for each
 * problem j < P, dW_j = X^T dY_j and one AdamW step on W_j, m_j, v_j, exactly
 * as forge_wgrad_adamw(X, dY[j], W[j], m[j], v[j], M[j], N, K, ...) would
 * compute it (bitwise wherever that call runs on CTA pairs, M[j] > 128: the
 * same 256 x 256 tiles in the same K order).  For layers whose
 * projections read the same activations (an attention block's projections):
 * the problems' tiles form one list walked by one grid, so SMs that a small
 * problem alone would leave idle run the others' tiles.  The operation of
 * each problem is the one forge_wgrad_adamw states; the pages know no
 * batched form of it.
 *   X            device bf16 [K, N], shared by all problems.
 *   P            1 <= P <= 8 problems.
 *   dY, M, W, m, v   host arrays of P entries: device bf16 dY[j] [K, M[j]],
 *                device fp32 W[j] and state_dtype m[j], v[j] [N, M[j]]
 *                (pointers the caller owns; the arrays are read during the
 *                call only).  Problems must not share W, m or v.
 *   in_dtype     FORGE_BF16 only (else FORGE_ERR_UNSUPPORTED_DTYPE).
 *   state_dtype, lr, beta1, beta2, eps, wd, step: as forge_wgrad_adamw, the
 *                same for every problem.
 * Checks as forge_wgrad_adamw, per problem, before any launch; operands
 * whose rows TMA cannot address are staged into the library's memory pool
 * (one allocation per call), and a failed allocation returns FORGE_ERR_CUDA.
 */
FORGE_API forge_status forge_wgrad_adamw_multi(const void* X, int64_t N, int64_t K, int32_t P,
                                               const void* const* dY, const int64_t* M,
                                               float* const* W, void* const* m, void* const* v,
                                               forge_dtype in_dtype, forge_dtype state_dtype,
                                               float lr, float beta1, float beta2, float eps,
                                               float wd, int64_t step, forge_stream_t stream);

/*
 * Per-tensor e4m3 quantisation with an amax scale, the step in front of an
 * fp8 call (the fp8 rows of "Math verified, not asserted", P6; the recipe
 * s = amax / 448 of the fp8 workload):
 *   x       device [n] of x_dtype (FORGE_F32 or FORGE_BF16), read as a flat
 *           array (any tensor shape, row-major).
 *   codes   device [n] bytes: OCP e4m3fn codes, each the value nearest to
 *           x / s computed in fp32 (ties to even; magnitudes past 448 saturate).
 *   scale   device float[1]: receives s = amax|x| / 448 (an fp32 division),
 *           or 1 when amax is 0 (n == 0 included).  NaN entries of x are left
 *           out of the amax (their codes are NaN).
 * Pass codes and scale as X (or dY) and scales[0] (or scales[1]) of an e4m3
 * call.  Nothing is allocated: two passes over x, the first of which parks
 * one partial maximum per block (at most four blocks per SM) in an aligned
 * window of `codes`, which the second pass then overwrites with the codes.
 * codes must not overlap x or scale.  Errors: n < 0, scale NULL, or x / codes
 * NULL with n > 0 -> FORGE_ERR_INVALID_ARG; x_dtype -> FORGE_ERR_UNSUPPORTED_DTYPE;
 * x not aligned to its element size or scale not 4-byte aligned ->
 * FORGE_ERR_MISALIGNED; a pointer that is not device memory of the current
 * device -> FORGE_ERR_INVALID_ARG.
 */
FORGE_API forge_status forge_quantize_e4m3(const void* x, forge_dtype x_dtype, int64_t n,
                                           uint8_t* codes, float* scale, forge_stream_t stream);

/*
 * The input gradient dX = dY W^T (bf16 in, fp32 accumulation, bf16 out,
 * nearest even), the GEMM on the other side of the backward pass that must
 * read W before the fused update overwrites it ("Math verified, not
 * asserted", P1).
 *   dY  device [K, M] bf16 (the same tensor the weight gradient reads).
 *   Wb  device [N, M] bf16: the weight as the forward pass used it (for a
 *       fp32 master W, its bf16 copy).
 *   dX  device [K, N] bf16, written.
 * in_dtype must be FORGE_BF16; K may be 0 (nothing is written).  dY, Wb and
 * dX need bases aligned to their element size (else FORGE_ERR_MISALIGNED);
 * rows of any width are accepted: when dY's or Wb's base is not 16-byte
 * aligned or M * 2 is not a multiple of 16, that operand is first copied into
 * rows padded to 16 bytes in a stream-ordered scratch buffer from the
 * library's memory pool (freed on `stream` after the launch; a failed
 * allocation returns FORGE_ERR_CUDA).
 */
FORGE_API forge_status forge_dgrad(const void* dY, const void* Wb, void* dX, int64_t M, int64_t N,
                                   int64_t K, forge_dtype in_dtype, forge_stream_t stream);

/*
 * One backward-and-update step for a linear layer, in the order the in-place
 * update requires: dX = dY Wb^T first, then the fused dW = X^T dY + AdamW on
 * W, m, v (exactly forge_wgrad_adamw), both on `stream`, so dX always sees
 * the weights from before this step.  Wb is the bf16 copy of W the forward
 * pass used; with Wb == NULL the library first rounds W to bf16 (nearest
 * even) into a scratch copy (N rows of M * 2 bytes rounded up to 16) from its
 * memory pool, allocated and freed in stream order on `stream`, together with
 * any staging copy forge_dgrad would make.  bf16 inputs only.  Every argument
 * check of both halves runs before the first launch; the arguments are those
 * of forge_dgrad and forge_wgrad_adamw.
 */
FORGE_API forge_status forge_backward_adamw(const void* X, const void* dY, float* W, void* m,
                                            void* v, const void* Wb, void* dX, int64_t M,
                                            int64_t N, int64_t K, forge_dtype in_dtype,
                                            forge_dtype state_dtype, float lr, float beta1,
                                            float beta2, float eps, float wd, int64_t step,
                                            forge_stream_t stream);

/*
 * Fused dW = X^T dY and one SGD-momentum step on W and the momentum buffer
 * mom ([N, M] of state_dtype).  On the first step pass mom = 0 (then
 * mom' = g + wd W, as torch's SGD).  Other arguments as forge_wgrad_adamw.
 */
FORGE_API forge_status forge_wgrad_sgdm(const void* X, const void* dY, float* W, void* mom, int64_t M,
                              int64_t N, int64_t K, forge_dtype in_dtype, forge_dtype state_dtype,
                              float lr, float momentum, float wd, const float* scales,
                              forge_stream_t stream);

/*
 * dW = X^T dY alone, stored as fp32 [N, M] into dW (device).  This is the
 * only call that writes a gradient to device memory; it exists to check the
 * contraction by itself.
 */
FORGE_API forge_status forge_wgrad_only(const void* X, const void* dY, float* dW, int64_t M, int64_t N,
                              int64_t K, forge_dtype in_dtype, const float* scales,
                              forge_stream_t stream);

/*
 * Grouped (mixture-of-experts) form: E experts, each with its own W, m, v
 * block [N, M] (stacked as [E, N, M]) and its own token rows.  X [T, N] and
 * dY [T, M] hold the tokens packed by expert: expert e owns rows
 * [offsets[e], offsets[e+1]) (offsets: device int32 [E+1], non-decreasing,
 * offsets[0] >= 0, read on the device, so no host synchronisation).
 * The gradient of expert e is X_e^T dY_e over its own rows only.  An expert
 * with no rows still takes the AdamW step with g = 0 (P5).  `step` is the
 * same for every expert.  T_total = offsets[E] is bounded by `T_max`
 * (the number of rows of the X, dY allocations).  1 <= E <= 1024.
 */
FORGE_API forge_status forge_grouped_wgrad_adamw(const void* X, const void* dY, float* W, void* m, void* v,
                                       const int32_t* offsets, int32_t E, int64_t T_max,
                                       int64_t M, int64_t N, forge_dtype in_dtype,
                                       forge_dtype state_dtype, float lr, float beta1, float beta2,
                                       float eps, float wd, int64_t step, const float* scales,
                                       forge_stream_t stream);

/*
 * The owner's optimizer step behind a reduce-scatter (data parallelism with
 * the optimizer state sharded, ZeRO-2 style; "Math verified, not asserted",
 * P3: under a reduce-scatter every output tile has exactly one owner, which
 * alone applies the update).  Each rank contracts its own tokens into a
 * partial fp32 dW (forge_wgrad_only); a reduce-scatter sums the partials and
 * hands every rank the rows of W it owns; the owner then calls this on its
 * shard.  Unlike the fused calls this path reads a gradient from device
 * memory: the partial gradients exist because the collective exchanges them.
 *   G      device fp32 [n]: the summed gradient of the owner's shard.
 *   W      device fp32 [n], updated in place.
 *   m, v   device [n] of state_dtype (FORGE_F32 or FORGE_BF16), updated in place.
 *   n      elements in the shard (a row range [r0, r1) of a row-major [N, M]
 *          weight is the flat range [r0 M, r1 M)); n = 0 does nothing.
 *   lr, beta1, beta2, eps, wd, step: as forge_wgrad_adamw.
 * The update is the fused epilogue's arithmetic, operation for operation:
 * given the dW that forge_wgrad_only computes for (X, dY), the result equals
 * forge_wgrad_adamw's on (X, dY) bit for bit.  G must not overlap W, m, v.
 * Errors: n < 0 or a NULL pointer with n > 0, or a hyperparameter out of
 * range -> FORGE_ERR_INVALID_ARG; state_dtype -> FORGE_ERR_UNSUPPORTED_DTYPE;
 * pointers outside device memory of the current device ->
 * FORGE_ERR_INVALID_ARG; G, W not 4-byte aligned or m, v not aligned to
 * their element size -> FORGE_ERR_MISALIGNED.  Allocates nothing.
 */
FORGE_API forge_status forge_owner_adamw(const float* G, float* W, void* m, void* v, int64_t n,
                                         forge_dtype state_dtype, float lr, float beta1,
                                         float beta2, float eps, float wd, int64_t step,
                                         forge_stream_t stream);

/* The same for SGD with momentum (mom as forge_wgrad_sgdm's). */
FORGE_API forge_status forge_owner_sgdm(const float* G, float* W, void* mom, int64_t n,
                                        forge_dtype state_dtype, float lr, float momentum,
                                        float wd, forge_stream_t stream);

/*
 * Log-probabilities of given tokens under rows of logits, with entropy and the
 * top alternatives: the loss, the scoring of given answers and the answers of
 * a decode step, in one pass over the logits.  For row r, z = scale * logits[r],
 *   lse = ln sum_j exp z_j,   p_j = exp(z_j - lse),
 *   logprob = z_t - lse (t = targets[r]),   entropy = -sum_j p_j ln p_j.
 *   logits  device [R, V] of dtype (FORGE_BF16 or FORGE_F32), rows ld elements
 *           apart (ld >= V: a padded vocabulary).  Rows of any alignment.
 *   targets device [R] of id_dtype (FORGE_I32 or FORGE_I64), or NULL (then
 *           logprob is NULL too and every row counts).  A negative target
 *           marks padding: nothing of the row counts, its logprob, lse, entropy
 *           and top_logprob are 0 and its top_index -1.  A target >= V is recorded
 *           as FORGE_ERR_INVALID_ARG in the device status word and its row
 *           taken as padding.
 *   scale   the inverse temperature, 0 < scale <= 2e38.
 *   logprob, lse, entropy  device fp32 [R], written; each may be NULL.
 *   top_k   0 <= top_k <= min(V, 32); top_index (device int32) and top_logprob
 *           (device fp32), [R, top_k], receive the top_k largest logits' columns
 *           and log-probabilities, largest first; equal logits by the lower
 *           column.
 * Masked entries are -inf: their p is 0.  A row with no other entry has
 * lse = logprob = top_logprob = -inf and entropy 0.  A NaN or +inf among a
 * row's logits makes its logprob, lse, entropy and top_logprob NaN; NaN
 * ranks above every number in the top entries.  Maxima, sums and results are
 * held in fp32 or wider.  Allocates nothing.  R = 0 does nothing.
 */
FORGE_API forge_status forge_token_logprob(const void* logits, forge_dtype dtype, int64_t R,
                                           int64_t V, int64_t ld, const void* targets,
                                           forge_dtype id_dtype, float scale, float* logprob,
                                           float* lse, float* entropy, int32_t top_k,
                                           int32_t* top_index, float* top_logprob,
                                           forge_stream_t stream);

/*
 * The gradient of sum_r (grad_logprob[r] logprob[r] + grad_entropy[r] entropy[r])
 * by the logits of forge_token_logprob:
 *   dlogits[r][j] = scale (a (1[j = t] - p_j) - b p_j (ln p_j + entropy[r])),
 *   a = grad_logprob[r], b = grad_entropy[r], p_j = exp(scale logits[r][j] - lse[r]).
 * With a = -1 / (rows that count), dlogits is the gradient of the mean
 * cross-entropy: the bf16 dY of the head's forge_backward_adamw.
 *   logits, dtype, R, V, ld, targets, id_dtype, scale  as given to
 *           forge_token_logprob (targets not NULL); a row whose target is
 *           padding, or whose lse is -inf, gets zeros.
 *   lse     device fp32 [R], from forge_token_logprob.
 *   grad_logprob  device fp32 [R].
 *   entropy, grad_entropy  device fp32 [R]; grad_entropy may be NULL (no
 *           entropy term), then entropy is not read.
 *   dlogits device [R, V] of out_dtype (FORGE_BF16, rounded once to nearest
 *           even, or FORGE_F32), rows ld_out >= V elements apart, written.  It
 *           may be logits itself when out_dtype and ld_out equal dtype and ld;
 *           rows that share memory in any other way are refused
 *           (FORGE_ERR_INVALID_ARG).
 * Allocates nothing.
 */
FORGE_API forge_status forge_token_logprob_grad(
    const void* logits, forge_dtype dtype, int64_t R, int64_t V, int64_t ld, const void* targets,
    forge_dtype id_dtype, float scale, const float* lse, const float* grad_logprob,
    const float* entropy, const float* grad_entropy, void* dlogits, forge_dtype out_dtype,
    int64_t ld_out, forge_stream_t stream);

/*
 * The embedding lookup with scaling: Y[t] = scale * W[ids[t]].
 *   ids     device [T] of id_dtype (FORGE_I32 or FORGE_I64).  A negative id is
 *           padding: Y[t] = 0.  An id >= V is recorded as FORGE_ERR_INVALID_ARG
 *           in the device status word and taken as padding.
 *   W       device [V, D] of w_dtype (FORGE_BF16 or FORGE_F32).
 *   Y       device [T, D] of y_dtype (FORGE_BF16, the fp32 product rounded once
 *           to nearest even, or FORGE_F32), written.
 * W and Y of any width and alignment; T <= 2^30.  Allocates nothing.  T = 0
 * does nothing.
 */
FORGE_API forge_status forge_embedding(const void* ids, forge_dtype id_dtype, int64_t T,
                                       const void* W, forge_dtype w_dtype, int64_t V, int64_t D,
                                       float scale, void* Y, forge_dtype y_dtype,
                                       forge_stream_t stream);

/*
 * The gradient of forge_embedding by W, summed by tokens:
 *   dW[r] = scale * sum over {t : ids[t] = r} of dY[t]   (+ dW[r] if accumulate)
 *   dY      device [T, D] of dy_dtype (FORGE_BF16 or FORGE_F32); rows of padding
 *           tokens are not read.
 *   ids     as forge_embedding's; T <= 2^30.
 *   dW      device fp32 [V, D].  accumulate = 0: written whole, rows without a
 *           token as zeros.  accumulate != 0: added to; rows without a token are
 *           neither read nor written.
 * The tokens are first ordered by row on the device; a row's sum is taken in
 * fp32 in an order that the ids alone determine, so results are bitwise
 * reproducible.  The order, a table of the rows and the partial sums of rows
 * with many tokens take stream-ordered scratch from the library's memory pool;
 * a failed allocation returns FORGE_ERR_CUDA.
 */
FORGE_API forge_status forge_embedding_grad(const void* dY, forge_dtype dy_dtype, const void* ids,
                                            forge_dtype id_dtype, int64_t T, int64_t V, int64_t D,
                                            float scale, float* dW, int32_t accumulate,
                                            forge_stream_t stream);

/*
 * forge_embedding_grad fused with one AdamW step on W, m, v: the gradient of a
 * row is used where it is summed and never reaches device memory.  Rows
 * without a token take the step with g = 0, as an expert without tokens does
 * (P5).  W device fp32 [V, D]; m, v device [V, D] of state_dtype (FORGE_F32 or
 * FORGE_BF16); lr ... step as forge_wgrad_adamw; the other arguments, the order
 * of sums and the scratch as forge_embedding_grad.  W must not be read by
 * another operation of the same step afterwards (the single-use guard of P1:
 * an embedding tied to the head takes forge_embedding_grad).
 */
FORGE_API forge_status forge_embedding_adamw(const void* dY, forge_dtype dy_dtype, const void* ids,
                                             forge_dtype id_dtype, int64_t T, int64_t V, int64_t D,
                                             float scale, float* W, void* m, void* v,
                                             forge_dtype state_dtype, float lr, float beta1,
                                             float beta2, float eps, float wd, int64_t step,
                                             forge_stream_t stream);

/*
 * The global norm of P gradient tensors, norm[0] = sqrt(sum of all g^2), for
 * the paths that hold gradients in memory (forge_wgrad_only,
 * forge_embedding_grad, an owner's shard): exact clipping needs every gradient
 * before it may touch one, so the fused steps cannot offer it (P2).
 *   grads   host array of P device pointers (NULL only where n[j] = 0) to n[j]
 *           elements of dtype (FORGE_BF16 or FORGE_F32); read during the call only.
 *   norm    device fp32[1], written (0 for P = 0).
 * Squares are summed in fp32 over at most a few hundred elements (in fp64 where
 * such a sum leaves fp32's range or its terms lose digits at the range's lower
 * end) and in fp64 from there, in a fixed order: bitwise reproducible, and as
 * exact for gradients of any size that dtype holds.  NaN and infinities
 * propagate.  Takes a few KB of stream-ordered scratch from the library's
 * memory pool.
 */
FORGE_API forge_status forge_grad_norm(const void* const* grads, const int64_t* n, int32_t P,
                                       forge_dtype dtype, float* norm, forge_stream_t stream);

/*
 * Clipping by a global norm: out[j] = grads[j] * min(1, max_norm / (norm[0] + 1e-6)),
 * element by element, in fp32 and rounded once to out_dtype.
 *   grads, n, P, dtype  as forge_grad_norm.
 *   norm    device fp32[1]: forge_grad_norm's (under data parallelism, after
 *           its square was summed over the ranks).  A NaN norm makes every
 *           output NaN, as torch.nn.utils.clip_grad_norm_ does.
 *   max_norm  >= 0 (infinity: never clips, not even by an infinite norm, where
 *           torch.nn.utils.clip_grad_norm_ makes every output NaN).
 *   out     host array of P device pointers to n[j] elements of out_dtype.
 *           out[j] may be grads[j] (clipping in place) when out_dtype is dtype;
 *           a tensor clipped in place by a factor of exactly 1 is left as it is.
 *           Any other overlap of the two is refused (FORGE_ERR_INVALID_ARG);
 *           overlaps with another tensor of the lists are not supported.
 * Allocates nothing.
 */
FORGE_API forge_status forge_clip_grads(const void* const* grads, const int64_t* n, int32_t P,
                                        forge_dtype dtype, const float* norm, float max_norm,
                                        void* const* out, forge_dtype out_dtype,
                                        forge_stream_t stream);

/* Static description of a status code; never NULL. */
FORGE_API const char* forge_status_string(forge_status status);

/*
 * Read and clear the device status word of the current device: FORGE_OK, or
 * FORGE_ERR_TIMEOUT if a kernel's bounded wait ran out since the last read.
 * Synchronises the current device.
 */
FORGE_API forge_status forge_get_device_status(void);

/*
 * Failure-detection self-test: launches one CTA that waits on a barrier no
 * one arrives at, with a limit of timeout_us microseconds; the wait runs out,
 * the kernel records FORGE_ERR_TIMEOUT in the device status word and
 * returns normally (no trap, the context stays usable).
 */
FORGE_API forge_status forge_selftest_wait_timeout(uint32_t timeout_us, forge_stream_t stream);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
FORGE_API int32_t forge_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FORGE_H */
