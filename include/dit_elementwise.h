/*
 * dit_elementwise.h -- C ABI of libdit_elementwise.so, the GB300 (sm_103a)
 * kernels for the memory-bound elementwise hot path of LTX-2-style video
 * diffusion transformers.
 *
 * Operations, each one kernel launch on the caller's stream:
 *
 *   dit_residual_gate_add          out = hidden + update * gate
 *   dit_rmsnorm_modulate           out = rms_norm(x, eps) * (1 + scale) + shift
 *   dit_gate_add_rmsnorm_modulate  both in one pass: writes the new residual
 *                                  and the modulated input of the next site
 *   dit_*_fp8                      the modulation / fused op with an FP8
 *                                  (E4M3) modulated output
 *   dit_gelu_tanh                  the feed-forward's tanh-GELU, elementwise
 *   dit_grouped                    one of the first three over several
 *                                  problems (e.g. video and audio streams)
 *                                  in one launch
 *   dit_selfcheck                  bit-for-bit check of one runtime key
 *
 * and the same kind of operations for the token transformers beside it (the
 * language model that reads the prompt), with their gradients:
 *
 *   dit_rmsnorm, dit_add_rmsnorm   out = rms_norm(x, eps) * (offset + weight),
 *                                  x = hidden + update; *_fp8: E4M3 output
 *                                  with a scale per row or per 128 columns
 *   dit_rmsnorm_backward           gradients of x and of the weight
 *   dit_embedding                  rows of a table by token id, times a scale
 *   dit_embedding_backward         the table's gradient, by sorted tokens
 *   dit_grad_norm, dit_clip_grads  the 2-norm over many tensors; clipping
 *
 * and around attention:
 *
 *   dit_rotary_table               cos and sin of the positions' angles, over
 *                                  one or several axes
 *   dit_rope, dit_rmsnorm_rope     queries and keys turned by them, with the
 *                                  norm of each head in the same pass
 *   dit_rmsnorm_rope_backward      its gradients
 *   dit_cache_write, dit_cache_read  a paged cache of keys and values, E4M3
 *                                  with a scale per row or in the dtype
 *   dit_paged_attention            one new token per sequence over that cache
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Tensors.  Every tensor is contiguous, row-major [B, L, D] in device memory
 *   (or memory the device can address), all of one dtype.  A "row" is one
 *   (b, l) pair of D elements.  An operand of layout DIT_ROW_BCAST has shape
 *   [B, 1, D]: its row b is used for all L rows of batch b.
 * Arithmetic.  Every element is loaded exactly into fp32, computed with IEEE
 *   fp32 operations (round to nearest even, no fused multiply-add where the
 *   formula below writes two operations, no flush of subnormals) and rounded
 *   once to the output dtype (round to nearest even; overflow gives +-inf;
 *   NaN propagates).
 * Ownership.  The caller owns all memory.  The library allocates nothing,
 *   keeps no per-call state and never synchronises: each call validates its
 *   arguments on the host, enqueues one kernel on `stream` (0 = the legacy
 *   default stream; dit_grouped: one kernel, or one per problem as stated
 *   there) and returns.  Outputs are complete once the stream
 *   reaches that point.
 * Aliasing.  out == hidden (exactly the same pointer) is allowed, as is
 *   residual_out == hidden; any other overlap between an output and another
 *   tensor returns DIT_ERR_ALIAS.
 * Alignment.  Pointers must be aligned to the element size (2 bytes for
 *   bf16/fp16, 4 for fp32); otherwise DIT_ERR_MISALIGNED.  Any such pointer
 *   is accepted: the widest vector access that every pointer and the row
 *   pitch D * element_size allow is chosen per call (up to 32 bytes).  Rows
 *   whose pitch is not a multiple of 16 bytes, in tensors that start on
 *   16-byte boundaries, are still moved in 16-byte granules (the row-wise
 *   operations group the rows by their offset modulo 16 bytes); only
 *   sub-views that start off a 16-byte boundary fall back to narrower
 *   accesses.
 * Errors.  Argument errors are returned before any launch and leave outputs
 *   untouched.  B, L, D >= 0; a call with B * L * D == 0 returns DIT_OK and
 *   launches nothing.  A launch failure reported by the CUDA runtime returns
 *   DIT_ERR_LAUNCH; faults during execution surface at the caller's next
 *   synchronisation, as for any CUDA kernel.  There is no fallback path.
 * Threads.  Entry points may be called from several host threads; the only
 *   shared state is a per-device cache of launch limits, filled on first use.
 */
#ifndef DIT_ELEMENTWISE_H
#define DIT_ELEMENTWISE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The stream type of the CUDA runtime, without requiring its headers. */
typedef struct CUstream_st* dit_stream_t;

typedef enum { DIT_BF16 = 0, DIT_FP16 = 1, DIT_FP32 = 2 } dit_dtype;

typedef enum {
  DIT_FULL = 0,      /* [B, L, D]: one value per element            */
  DIT_ROW_BCAST = 1  /* [B, 1, D]: one vector per batch, reused over L */
} dit_layout;

typedef enum {
  DIT_OK = 0,
  DIT_ERR_NULL_PTR = 1,     /* a tensor pointer is NULL while B*L*D > 0      */
  DIT_ERR_BAD_SHAPE = 2,    /* B, L or D negative, or B*L*D overflows         */
  DIT_ERR_BAD_DTYPE = 3,    /* dtype is not a dit_dtype value                 */
  DIT_ERR_BAD_LAYOUT = 4,   /* layout is not a dit_layout value               */
  DIT_ERR_ALIAS = 5,        /* an output overlaps another tensor (other than
                               the allowed out == hidden)                     */
  DIT_ERR_BAD_EPS = 6,      /* eps is negative, infinite or NaN               */
  DIT_ERR_LAUNCH = 7,       /* the CUDA runtime rejected the launch           */
  DIT_ERR_MISALIGNED = 8,   /* a pointer is not aligned to the element size   */
  DIT_ERR_NO_DEVICE = 9,    /* no current CUDA device could be queried        */
  DIT_ERR_BAD_OP = 10,      /* op is not a dit_op value, or (dit_grouped) count
                               is outside [0, DIT_MAX_GROUP]                  */
  DIT_ERR_WORKSPACE = 11,   /* a workspace that is NULL, smaller than the call's
                               _workspace_bytes or not 256-byte aligned       */
  DIT_ERR_BAD_STATISTIC = 12, /* dit_set_statistic: not a dit_statistic value */
  DIT_ERR_BAD_SCALAR = 13,  /* a scale, weight_offset or max_norm is infinite or
                               NaN (max_norm: or negative)                    */
  DIT_ERR_BAD_FORMAT = 14,  /* an id type or a scale group that is not one of
                               the documented values                          */
  DIT_ERR_NO_MEMORY = 15    /* the host has no memory for the call's own list */
} dit_status;

/* Version of this interface; bumped on any incompatible change. */
#define DIT_ABI_VERSION 3
int dit_abi_version(void);

/* A static, human-readable name for a status code. */
const char* dit_status_string(dit_status status);

/*
 * The row statistic r = 1 / sqrt(mean(x^2) + eps) of the modulating
 * operations (dit_rmsnorm_modulate, dit_gate_add_rmsnorm_modulate, their
 * _strided, grouped and _fp8 forms), chosen for the whole process:
 *
 *   DIT_STATISTIC_FAST (default): the row's fp32 sum of squares, one FMA per
 *     element, merged in tree order; ms = S / D by a corrected quotient;
 *     r = rsqrtf(fl(ms + eps)) refined by one Newton-Raphson step.  r is
 *     within about seventeen fp32 ulps of the exact statistic's, so each
 *     output element is within one bf16/fp16 ulp of the exact definition's
 *     except where the final + shift cancels (|y| much smaller than
 *     |x r (1 + scale)|), where the difference stays below one dtype ulp of
 *     max(|t|, |y|), t = n (1 + scale); fp32 outputs within 2^-18 of
 *     max(|t|, |y|).  A row whose fp32 sum leaves [2^-100, 2^100] (a square
 *     that overflows fp32, infinities, squares below its normal range) is
 *     summed again with its elements scaled by 2^-64 or 2^64; a mean square
 *     in fp32's subnormal range with eps = 0 may then be one subnormal step
 *     off.
 *   DIT_STATISTIC_EXACT: ms = RN32(mean(x^2)), the exact mean of the row's
 *     squares rounded once to fp32, and r = RN32(1 / sqrt(fl(ms + eps))),
 *     correctly rounded: every output element equals the definition
 *     evaluated in fp32 with those values, bit for bit (NaN payloads aside),
 *     whatever kernel or launch shape computes it.  The squares are summed in
 *     compensated (TwoSum) pairs with a proven error bound and the rounding
 *     decided from it; rows the bound cannot decide (ties and near-ties) are
 *     summed exactly.  It costs time: on [1,32640,4096] bf16 the modulation
 *     takes about a third longer and the fused op an eighth (the compensated
 *     sum makes them issue-bound).
 *
 * Sources: the statistic is fp32 and the result is held to one bf16 ulp per
 * element (prhub summary of sglang PR #34172, "implementation breakdown"
 * item 2 and risks item 1).
 *
 * The mode is read when a call is made (host side) and selects the kernel
 * it launches -- a CUDA graph keeps the statistic its captured calls were
 * made with; set it before launching, not concurrently with calls from other
 * threads.  dit_set_statistic returns
 * DIT_ERR_BAD_STATISTIC for other values and leaves the mode unchanged.
 */
typedef enum {
  DIT_STATISTIC_FAST = 0,
  DIT_STATISTIC_EXACT = 1
} dit_statistic;
dit_status dit_set_statistic(dit_statistic statistic);
dit_statistic dit_get_statistic(void);

/*
 * Gated residual update:  out[b,l,d] = hidden[b,l,d] + update[b,l,d] * G
 * with G = gate[b,l,d] (gate_layout DIT_FULL) or gate[b,0,d] (DIT_ROW_BCAST),
 * evaluated as p = fl32(update * G), s = fl32(hidden + p), out = rnd(s).
 *
 * Source: sglang PR #29361 "Add diffusion residual-gate CUDA fast path for
 * LTX2", section Motivation (the hot pattern hidden + update * gate for
 * contiguous [B, L, D] tensors with a full gate or a [B, 1, D] gate) and
 * section Modifications (full and row-broadcast gates, dtype coverage, tail
 * shapes, rejection of unsupported inputs).
 *
 * out, hidden, update: [B, L, D].  gate: [B, L, D] or [B, 1, D].
 * out may be hidden (in-place update).
 */
dit_status dit_residual_gate_add(void* out, const void* hidden,
                                 const void* update, const void* gate,
                                 int64_t B, int64_t L, int64_t D,
                                 dit_dtype dtype, dit_layout gate_layout,
                                 dit_stream_t stream);

/*
 * adaLN modulation with a weightless RMSNorm over each row:
 *   r   = 1 / sqrt(mean_d(x[b,l,d]^2) + eps)     (fp32 statistic per row)
 *   out = rnd(fl32(fl32(fl32(x * r) * fl32(1 + S)) + H))
 * with S, H = scale, shift at [b,l,d] (mod_layout DIT_FULL) or [b,0,d]
 * (DIT_ROW_BCAST).  The statistic is computed as dit_set_statistic chose
 * (fast by default; exact: ms = RN32(mean(x^2)) and r = RN32(1/sqrt(fl(ms +
 * eps))), the same output bits whatever the launch shape).  A row holding a
 * NaN gives NaN; a row holding an infinity a zero statistic.
 *
 * Rows of at most 2^24 elements (D larger: DIT_ERR_BAD_SHAPE).
 *
 * Source: prhub summary of sglang PR #34172 (LTX-2 quality=high fused
 * RMSNorm+modulate), section "key source snippet" (the eager expression
 * rms_norm(x, eps) * (1 + scale) + shift of _ltx2_rms_norm_modulate, called
 * with the block's norm_eps) and section "implementation breakdown", item 2
 * (RMSNormNoWeight: the norm has no weight; one launch for the whole
 * expression).
 *
 * out, x: [B, L, D].  scale, shift: [B, L, D] or [B, 1, D].  eps >= 0.
 */
dit_status dit_rmsnorm_modulate(void* out, const void* x, const void* scale,
                                const void* shift, int64_t B, int64_t L,
                                int64_t D, float eps, dit_dtype dtype,
                                dit_layout mod_layout, dit_stream_t stream);

/*
 * Fused residual gate + modulation, one pass over the rows:
 *   residual_out = dit_residual_gate_add(hidden, update, gate)   (stored)
 *   modulated_out = dit_rmsnorm_modulate(residual_out, scale, shift, eps)
 * The statistic is taken over the residual as stored (rounded to the dtype),
 * so the two outputs are bitwise those of the two separate calls.  The
 * residual is never re-read from memory.  D at most 2^24.
 *
 * Source: the two operations above; the pages name the fused family member
 * (fused_gate_rmsnorm, prhub summary of sglang PR #34172, "implementation
 * breakdown" items 2 and 4) without describing it.
 *
 * residual_out, modulated_out, hidden, update: [B, L, D].
 * gate: per gate_layout.  scale, shift: per mod_layout.
 * residual_out may be hidden; modulated_out may not alias anything.
 */
dit_status dit_gate_add_rmsnorm_modulate(
    void* residual_out, void* modulated_out, const void* hidden,
    const void* update, const void* gate, const void* scale, const void* shift,
    int64_t B, int64_t L, int64_t D, float eps, dit_dtype dtype,
    dit_layout gate_layout, dit_layout mod_layout, dit_stream_t stream);

/*
 * Strided [B, 1, D] operands.  The same three operations, with one more
 * argument: vec_stride, the distance in elements between the vectors of
 * consecutive batches of every DIT_ROW_BCAST operand of the call (D for a
 * contiguous [B, 1, D] tensor).  It lets a caller pass rows of an adaLN
 * table directly: with a per-block table of shape [B, 9, D] (shift, scale,
 * gate for each of the block's three modulation sites -- self-attention,
 * prompt cross-attention, feed-forward: prhub summary of sglang PR #34172,
 * "implementation breakdown" item 3), the site's vectors are
 * table + i*D with vec_stride = 9*D, and no chunk is copied out.
 *
 * vec_stride must be >= D when B > 1 (DIT_ERR_BAD_SHAPE otherwise); it is
 * unused for DIT_FULL operands.  Aliasing is checked over the whole span
 * [p, p + ((B-1)*vec_stride + D) elements) of each strided operand.
 */
dit_status dit_residual_gate_add_strided(void* out, const void* hidden,
                                         const void* update, const void* gate,
                                         int64_t B, int64_t L, int64_t D,
                                         dit_dtype dtype, dit_layout gate_layout,
                                         int64_t vec_stride, dit_stream_t stream);

dit_status dit_rmsnorm_modulate_strided(void* out, const void* x,
                                        const void* scale, const void* shift,
                                        int64_t B, int64_t L, int64_t D,
                                        float eps, dit_dtype dtype,
                                        dit_layout mod_layout, int64_t vec_stride,
                                        dit_stream_t stream);

dit_status dit_gate_add_rmsnorm_modulate_strided(
    void* residual_out, void* modulated_out, const void* hidden,
    const void* update, const void* gate, const void* scale, const void* shift,
    int64_t B, int64_t L, int64_t D, float eps, dit_dtype dtype,
    dit_layout gate_layout, dit_layout mod_layout, int64_t vec_stride,
    dit_stream_t stream);

/*
 * tanh-approximated GELU, elementwise over n contiguous elements:
 *   out[i] = 0.5 * x[i] * (1 + tanh(z)),  z = sqrt(2/pi) * (x + 0.044715 x^3)
 * evaluated in fp32 as x * sigmoid(2z) (the same function: 1 + tanh(z) =
 * 2 / (1 + exp(-2z))), then rounded once to the dtype.  16-bit dtypes use
 * the hardware approximations of 2^v and 1/v (each within about 2^-22
 * relative); fp32 uses expf and an IEEE division.
 *
 * Source: prhub summary of sglang PR #34172, "implementation breakdown"
 * item 3 (LTX2FeedForward: proj_in, then the tanh-GELU act) and "functions
 * and motivation" (the FFN GELU is the second elementwise chain that
 * torch.compile fuses).
 *
 * out may be x (in place); any other overlap returns DIT_ERR_ALIAS.
 */
dit_status dit_gelu_tanh(void* out, const void* x, int64_t n, dit_dtype dtype,
                         dit_stream_t stream);

/*
 * Modulated output quantised to FP8 (OCP E4M3: 4 exponent bits, bias 7, 3
 * fraction bits, no infinities, largest finite 448), with a static
 * per-tensor scale:
 *   y   = the fp32 modulation value of dit_rmsnorm_modulate (before any
 *         rounding to the activation dtype)
 *   out = e4m3(fl32(y * fl32(1 / *quant_scale)))
 * rounded to nearest-even, saturating to +-448 (infinities included); NaN
 * stays NaN.  One byte per element, [B, L, D] row-major.
 *
 * Source: the prhub summary of sglang PR #34172 lists, among its related
 * PRs, the RMSNorm + FP8 quantisation fusion of the same fused-norm family;
 * the pages give neither the format nor the scaling, so the plainest
 * readings are taken: E4M3 (the activation FP8 format of such fusions), a
 * per-tensor scale that divides (applied as a multiplication by its
 * correctly rounded reciprocal), saturation instead of overflow.
 *
 * quant_scale: DEVICE pointer to one fp32 value, finite and > 0 (read by the
 * kernel, so it may change between graph replays; not checked on the host:
 * other values give defined but meaningless codes).  vec_stride: as in the
 * _strided calls.
 *
 * These calls take the staged row kernel only: every input pointer (and
 * residual_out) 16-byte aligned, D * element_size a multiple of 16 bytes (a
 * multiple of 16 elements is what FP8 GEMM inputs need anyway), the vector
 * stride in bytes a multiple of 16, and `out` aligned to 8 bytes (bf16/fp16)
 * or 4 (fp32) -- otherwise DIT_ERR_MISALIGNED; rows of at most 16 KB (D <=
 * 8192 for 16-bit, 4096 for fp32) -- otherwise DIT_ERR_BAD_SHAPE.  `out`
 * may not overlap any other tensor or *quant_scale.
 */
dit_status dit_rmsnorm_modulate_fp8(void* out, const void* x, const void* scale,
                                    const void* shift, int64_t B, int64_t L,
                                    int64_t D, float eps, dit_dtype dtype,
                                    dit_layout mod_layout, int64_t vec_stride,
                                    const float* quant_scale, dit_stream_t stream);

/* The fused op with its modulated output in E4M3 (residual_out keeps the
 * dtype, bitwise that of dit_residual_gate_add). */
dit_status dit_gate_add_rmsnorm_modulate_fp8(
    void* residual_out, void* out, const void* hidden, const void* update,
    const void* gate, const void* scale, const void* shift, int64_t B,
    int64_t L, int64_t D, float eps, dit_dtype dtype, dit_layout gate_layout,
    dit_layout mod_layout, int64_t vec_stride, const float* quant_scale,
    dit_stream_t stream);

/*
 * Grouped launches: one operation over up to DIT_MAX_GROUP independent
 * problems of one dtype and layout, each with its own pointers, B, L, D and
 * vec_stride.  An LTX-2 block applies each of its adaLN modulations to the
 * video stream (hidden size 4096) and to the audio stream (hidden size 2048)
 * -- prhub summary of sglang PR #34172, "implementation breakdown" item 3
 * (the six sites: video/audio self-attention, prompt cross-attention and
 * feed-forward) and the test section (hidden 4096 = video, 2048 = audio) --
 * so one grouped call covers both streams of a site.
 *
 * Each problem computes what the single call of the same operation
 * computes: the residual bit for bit; the modulated output bit for bit with
 * the exact statistic, and within the fast statistic's bound otherwise (its
 * sum may be taken in another tree order than a single call's).
 *
 * Launch: when every non-empty problem has 16-byte aligned pointers, pitch
 * and vec_stride and (for the modulating operations) rows of at most 8192
 * 16-bit or 4096 fp32 elements, the call enqueues ONE kernel on `stream`
 * that covers all of them, with the CTAs split in proportion to the
 * problems' sizes.  Otherwise, and for a DIT_FULL gate of the residual gate
 * (whose flat kernel has no rows), it enqueues one kernel per non-empty
 * problem, in order.  No problem may write memory that another problem
 * reads or writes (DIT_ERR_ALIAS), since they run concurrently.
 *
 * problems: a HOST array of `count` descriptors (0 <= count <= DIT_MAX_GROUP;
 * NULL allowed when count == 0), read during the call only.  Validation is
 * that of the single calls, per problem, before anything is launched; the
 * first failing problem's status is returned.
 */
#define DIT_MAX_GROUP 8

typedef enum {
  DIT_OP_RESIDUAL_GATE = 0,          /* out = hidden + update * gate */
  DIT_OP_RMSNORM_MODULATE = 1,       /* out = rms_norm(x) * (1 + scale) + shift */
  DIT_OP_GATE_ADD_RMSNORM_MODULATE = 2 /* both, fused */
} dit_op;

typedef struct {
  void* out;          /* residual gate: out; modulation: out; fused: residual_out */
  void* out2;         /* fused: modulated_out; NULL otherwise */
  const void* x;      /* residual gate, fused: hidden; modulation: x */
  const void* update; /* residual gate, fused */
  const void* gate;   /* residual gate, fused */
  const void* scale;  /* modulation, fused */
  const void* shift;  /* modulation, fused */
  int64_t B, L, D;
  int64_t vec_stride; /* as in the _strided calls (elements; D if contiguous) */
} dit_problem;

/* gate_layout is read by the residual gate and the fused op, mod_layout by
 * the modulation and the fused op; eps by the modulating operations. */
dit_status dit_grouped(dit_op op, const dit_problem* problems, int count,
                       float eps, dit_dtype dtype, dit_layout gate_layout,
                       dit_layout mod_layout, dit_stream_t stream);

/*
 * Self-check of one runtime key: (op, dtype, gate_layout, mod_layout, D).
 *
 * The pages' integration checks every runtime key of its pointwise fusions
 * bit for bit on first use and falls back to the model's math on a mismatch
 * or a launch failure (vllm-omni PR #7350, "[Kernel] Enable LTX DiffVAE
 * fusions on SM100 and SM103", section Purpose).  This library has no
 * fallback; dit_selfcheck gives the caller the check itself.  It enqueues on
 * `stream`, in order:
 *   1. seeded inputs of a [2, 7, D] problem, written into `workspace`;
 *   2. the operation, through the same validation and launch path as the
 *      public call of that op, dtype and layouts (so the kernel the library
 *      picks for 256-byte aligned tensors with rows of D elements);
 *   3. the expected outputs from plain one-thread-per-element kernels;
 *   4. the count of output words that differ from the expected ones, added
 *      to *mismatches after the call has set it to zero.
 * Every output has exactly one correct value: the residual gate is defined
 * to the bit, and the inputs of the modulating ops make the row statistic
 * exact in any summation order (every normalised value is +-1/2, eps = 3/4,
 * so r = 1).  Zero mismatches: the key's path computes the definition.
 *
 * workspace: device memory of at least dit_selfcheck_workspace_bytes(op,
 * dtype, D) bytes, 256-byte aligned, owned by the caller and free for the
 * call's duration; on return it holds, from offset 0, nine tensors of
 * N = 14 * D elements each starting on a 256-byte boundary -- x (hidden),
 * update, gate, scale, shift (a [2, 1, D] operand fills its first 2 * D
 * elements), out, out2, expected, expected2 -- then 14 fp32 row statistics.
 * mismatches: device pointer to one unsigned int (4-byte aligned).
 * eps is fixed (3/4) and not an argument.  The call does not synchronise:
 * read *mismatches after the stream has reached it.
 */
int64_t dit_selfcheck_workspace_bytes(dit_op op, dit_dtype dtype, int64_t D);

dit_status dit_selfcheck(dit_op op, dit_dtype dtype, dit_layout gate_layout,
                         dit_layout mod_layout, int64_t D, void* workspace,
                         int64_t workspace_bytes, unsigned int* mismatches,
                         dit_stream_t stream);

/*
 * dit_selfcheck_static: the same check, with no workspace argument and no
 * allocation.  The pages have no counterpart; this entry point exists for
 * callers that cannot allocate device memory when they want the check -- a
 * process whose device memory is all held by a framework's caching
 * allocator, or a latency-critical loop that must not call cudaMalloc or
 * cudaFree (both may synchronise the device).
 *
 * The workspace is a static device array of DIT_SELFCHECK_STATIC_BYTES
 * (4 MiB) inside the library, which every GPU that loads the library keeps
 * until the process exits.  That covers bf16/fp16 keys up to D = 16384 and
 * fp32 keys up to D = 8192; a key whose dit_selfcheck_workspace_bytes is
 * larger returns DIT_ERR_WORKSPACE.  The caller passes `mismatches` (device,
 * one unsigned int) as for dit_selfcheck; the call allocates nothing.
 *
 * Every call looks up the array's device address in the current context
 * (cudaGetSymbolAddress, a host-side runtime query that allocates nothing;
 * the first one per context may load the library's device code).  All calls
 * share the one array, and nothing in it needs to start at zero; calls whose
 * work overlaps on the GPU (other streams, other host threads) race on its
 * contents, so order them -- one stream, or a synchronisation between them.
 * After the check the array holds dit_selfcheck's workspace layout: nine
 * slots of round_up(2 * 7 * D * element size, 256) bytes -- inputs hidden/x,
 * update, gate, scale, shift, outputs out (residual), modulated, and the
 * plain kernels' expected out and modulated -- then the row statistics.
 */
#define DIT_SELFCHECK_STATIC_BYTES (4u << 20)

dit_status dit_selfcheck_static(dit_op op, dit_dtype dtype,
                                dit_layout gate_layout, dit_layout mod_layout,
                                int64_t D, unsigned int* mismatches,
                                dit_stream_t stream);

/*
 * dit_selfcheck_static_workspace: the device address (*workspace) and size
 * (*bytes, DIT_SELFCHECK_STATIC_BYTES) of dit_selfcheck_static's array in
 * the current context, for reading back what a check left there.  The array
 * belongs to the library: the caller may read it (after the check's stream
 * is synchronised) and must not free it.  DIT_ERR_NULL_PTR for a NULL
 * argument; DIT_ERR_NO_DEVICE (with *workspace = NULL, *bytes = 0) when no
 * device is current or the runtime cannot give the address.
 */
dit_status dit_selfcheck_static_workspace(void** workspace, int64_t* bytes);

/* ---------------------------------------------------------------------------
 * Token-transformer operators
 *
 * The conventions above hold, with these differences.
 *   Tensors are contiguous; rows = the product of all sizes but the last, D =
 *   the last.  A call whose output is empty returns DIT_OK and launches
 *   nothing (the gradients of weights and tables are written even when there are no
 *   rows: they are zero).  D is at most 2^24, rows and tokens at most 2^31 - 1.
 *   The row statistic is the fast one, whatever dit_set_statistic says.
 *   A call may enqueue several kernels, in order, on `stream`; every sum has
 *   one order for given sizes and alignment on one GPU model, so the same call gives
 *   the same bits.
 * Workspaces.  A call that needs memory of its own takes `workspace` (device,
 *   256-byte aligned, at least the size its _workspace_bytes function gives;
 *   that function returns -1 for sizes the call refuses).  It
 *   holds nothing between calls and needs no initial value; calls that may
 *   run at the same time, and graphs that may replay at the same time, need
 *   one each.
 * None of this has a counterpart in the pages: they are the memory-bound
 * operations of a language model's step, offered beside the diffusion
 * transformer's.
 * ------------------------------------------------------------------------- */

/*
 * Weighted RMSNorm, alone or with the residual's addition:
 *   s   = rnd(hidden + update)              -> residual_out (dit_add_rmsnorm)
 *   r   = 1 / sqrt(mean_d(s^2) + eps)       (the fast statistic)
 *   out = rnd(fl32(fl32(s * r) * fl32(weight_offset + weight[d])))
 * with s = x for dit_rmsnorm.  weight: [D], weight_offset 0 for a plain weight,
 * 1 for one stored as its difference from one.  The statistic is taken over
 * the residual as stored.  With eps = 0 a row whose mean square rounds to zero
 * in fp32 (below 2^-150) has r = +inf: infinities, and NaN where s is zero (E4M3: scales
 * that are not finite).
 * residual_out may be hidden; no other overlap of an
 * output with another tensor is allowed.  Any element-aligned pointer and any
 * D: tensors that start on 16-byte boundaries move in 16-byte accesses whatever D
 * (rows too long for registers only where D is a multiple of them), others
 * element by element.
 */
dit_status dit_rmsnorm(void* out, const void* x, const void* weight, int64_t rows, int64_t D,
                       float eps, float weight_offset, dit_dtype dtype, dit_stream_t stream);

dit_status dit_add_rmsnorm(void* residual_out, void* out, const void* hidden, const void* update,
                           const void* weight, int64_t rows, int64_t D, float eps,
                           float weight_offset, dit_dtype dtype, dit_stream_t stream);

/*
 * The same with the normed output in E4M3 (as dit_rmsnorm_modulate_fp8) and
 * dynamic scales: with y the fp32 value of out before its rounding and m the
 * maximum of |y| over the row (group 0) or over each 128 columns of it (group 128, the
 * last group holding what is left),
 *   scale = m / 448,  code = e4m3(y / scale),  y ~ code * scale,
 * evaluated as code = e4m3(fl32(t * (448 / max|t|))) with t = fl32(s *
 * fl32(weight_offset + weight)), which leaves r out of the codes, and the
 * quotient carried in two fp32 numbers; scale = fl32(fl32(max|t| * r) *
 * fl32(1 / 448)).  They are taken from y itself where a sum of squares
 * or a maximum leaves [2^-100, 2^100].  m = 0 gives scale 0 and codes 0; a NaN
 * or an infinity in s makes the scale of its row or group NaN, and the codes NaN.
 * out: [rows, D] bytes.  scales: fp32 [rows, 1], or [rows, ceil(D / 128)].
 * Other groups: DIT_ERR_BAD_FORMAT.  out and scales may overlap nothing.  Rows
 * of no columns (D = 0, group 0) have scale 0, written where scales is not NULL.
 */
dit_status dit_rmsnorm_fp8(void* out, float* scales, const void* x, const void* weight,
                           int64_t rows, int64_t D, int64_t group, float eps, float weight_offset,
                           dit_dtype dtype, dit_stream_t stream);

dit_status dit_add_rmsnorm_fp8(void* residual_out, void* out, float* scales, const void* hidden,
                               const void* update, const void* weight, int64_t rows, int64_t D,
                               int64_t group, float eps, float weight_offset, dit_dtype dtype,
                               dit_stream_t stream);

/*
 * Gradient of the weighted RMSNorm.  With n = x * r, t = grad_out *
 * (weight_offset + weight) and grad_residual the gradient that reaches x on
 * the skip path (NULL: none),
 *   grad_x      = rnd(r * (t - n * mean_d(t * n)) + grad_residual)
 *   grad_weight = rnd(sum over the rows of grad_out * n)
 * in fp32.  x is the norm's input: for dit_add_rmsnorm its residual_out, and
 * grad_x is then the gradient of hidden and of update alike.
 * grad_weight may be NULL (a frozen weight; the workspace may then be NULL too).
 * Up to 128 rows of at most 8189 columns need no workspace (its size is 0).
 * grad_x may be grad_out or grad_residual; no other overlap of an output with
 * another tensor or with the workspace is allowed.
 */
int64_t dit_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t D);

dit_status dit_rmsnorm_backward(void* grad_x, void* grad_weight, const void* grad_out,
                                const void* grad_residual, const void* x, const void* weight,
                                int64_t rows, int64_t D, float eps, float weight_offset,
                                dit_dtype dtype, void* workspace, int64_t workspace_bytes,
                                dit_stream_t stream);

/*
 * Embedding lookup:  out[t] = rnd(fl32(table[ids[t]] * scale)),
 * a row of zeros where ids[t] is outside [0, V) (a padded place).
 * out: [tokens, D], table: [V, D], V at most 2^31 - 1; ids: [tokens], aligned to their size.
 */
typedef enum { DIT_INT32 = 0, DIT_INT64 = 1 } dit_id_type;

dit_status dit_embedding(void* out, const void* ids, const void* table, int64_t tokens, int64_t V,
                         int64_t D, float scale, dit_dtype dtype, dit_id_type id_type,
                         dit_stream_t stream);

/*
 * Its gradient:  grad_table[v] = rnd(fl32(scale * sum of grad_out[t], ids[t] = v)),
 * every row of [V, D] written, zeros where no token names it; ids outside
 * [0, V) take no part.  The tokens are sorted by id (stably, so the rows of
 * an id are added in the order of their positions) and the sums are fp32.
 * grad_table may overlap neither the inputs nor the workspace.  Up to 256
 * tokens need no workspace (its size is 0, the pointer may be NULL).
 */
int64_t dit_embedding_backward_workspace_bytes(int64_t tokens, int64_t D);

dit_status dit_embedding_backward(void* grad_table, const void* grad_out, const void* ids,
                                  int64_t tokens, int64_t V, int64_t D, float scale,
                                  dit_dtype dtype, dit_id_type id_type, void* workspace,
                                  int64_t workspace_bytes, dit_stream_t stream);

/*
 * Global norm of many tensors, and clipping by it:
 *   norm   = sqrt(sum over all tensors and elements of g^2)
 *   out[i] = rnd(fl32(g[i] * c)),  c = fl32(min(1, max_norm / (norm + eps)))
 * The squares are summed in fp32 within a thread's few dozen elements and in
 * pairs of fp32 or in fp64 beyond (in fp64 throughout where such a sum leaves
 * [2^-100, 2^100]).
 * norm: device, one fp32 (the norm before clipping).  A NaN norm makes
 * c NaN; an infinite one makes c 0.
 *
 * tensors: a HOST array of `count` descriptions, read during the call only;
 * each tensor has its own size and dtype, and sizes of zero are
 * allowed.  dit_grad_norm ignores `out`.  out may be g itself; any other overlap
 * of an out with a g, an out, the norm or the workspace returns DIT_ERR_ALIAS.
 * Each tensor has at most 2^44 elements.
 */
typedef struct {
  const void* g;
  void* out;
  int64_t n;
  int64_t dtype; /* a dit_dtype value */
} dit_tensor;

int64_t dit_grad_norm_workspace_bytes(int64_t count);

dit_status dit_grad_norm(float* norm, const dit_tensor* tensors, int64_t count, void* workspace,
                         int64_t workspace_bytes, dit_stream_t stream);

dit_status dit_clip_grads(float* norm, const dit_tensor* tensors, int64_t count, float max_norm,
                          float eps, void* workspace, int64_t workspace_bytes,
                          dit_stream_t stream);

/* ---------------------------------------------------------------------------
 * Operators around attention
 *
 * What a transformer does between the projection of queries, keys and values and the
 * projection of attention's output, as far as it is bound by memory: the
 * rotation of queries and keys by their positions, with the norm of each head
 * in the same pass, its gradient, a paged cache of keys and values, and the attention
 * of one new token per sequence over it.  The conventions of the token-transformer
 * operators hold (workspaces, one order for every sum, several kernels a
 * call), with these differences.
 *   Tensors of heads may be views with any strides but the last: dit_heads.
 *   Strides are in elements and not negative; a stride of 0 repeats an input.
 *   An output's elements must lie apart from each other and from every other
 *   tensor of the call (DIT_ERR_ALIAS), which views that interleave without
 *   touching, such as the queries and keys of one packed projection, do; where an
 *   output may be an input, it is exactly that view.
 * ------------------------------------------------------------------------- */

/* Element (b, l, h, d) of a tensor [B, L, H, D] is p[b batch + l token + h head + d].
 * Operators over tokens alone ([tokens, H, D]) do not read `batch`. */
typedef struct {
  void* p; /* inputs are not written */
  int64_t batch, token, head;
} dit_heads;

/*
 * Rotary angles:  angle[t, j] = positions[axis(j), t] * freqs[j],
 *   cos[t, j] = rnd(cos(angle)),  sin[t, j] = rnd(sin(angle))
 * positions: [axes, tokens]; the first sections[0] columns belong to axis 0,
 * the next sections[1] to axis 1, and so on (one axis for text; time, height and width
 * for images and video).  sections: a HOST array of `axes` (1 to
 * DIT_MAX_AXES) counts, read during the call only; R is their sum, at most 512.  freqs:
 * [R], fp64, the angle per unit of position.  cos, sin: fp32 [tokens, R].
 * The frequency is taken in turns, in fp64 (within 2^-52 of it), and the angle reduced to a part of
 * a turn before it is rounded: for integer positions as a 64-bit fraction of a
 * turn (exact but for the frequency's 64-bit fraction, 2^-64 |position| turns), for fp32 ones as a sum of
 * fp32 products and their errors.  The part of a turn, its sine and its cosine are fp32.  A
 * position or frequency that is not finite, or an fp32 product that overflows, gives NaN.
 */
#define DIT_MAX_AXES 8
typedef enum { DIT_POS_INT32 = 0, DIT_POS_INT64 = 1, DIT_POS_FP32 = 2 } dit_position_type;

dit_status dit_rotary_table(float* cos, float* sin, const void* positions, const double* freqs,
                            int64_t tokens, const int64_t* sections, int64_t axes,
                            dit_position_type position_type, dit_stream_t stream);

/*
 * Rotation of queries and keys: with the pair (a, b) of columns (j, j + R), or
 * (2j, 2j + 1) where `interleaved`, for j < R, and the token's row of the table,
 *   a' = rnd(a cos - b sin),  b' = rnd(b cos + a sin)
 * (inverse: with -sin, which is the gradient); columns from 2R on are copied.
 * Each tensor is [B, L, H, D]: Hq heads of queries, Hk of keys, 2R <= D <= 1024,
 * H at most 65535.
 * cos, sin: fp32 [table_rows, R] with table_rows = B * L, or L (one table for
 * all batches).  k and k_out may be NULL (Hk = 0).  An output may be its input.
 */
dit_status dit_rope(const dit_heads* q_out, const dit_heads* k_out, const dit_heads* q,
                    const dit_heads* k, const float* cos, const float* sin, int64_t B, int64_t L,
                    int64_t Hq, int64_t Hk, int64_t D, int64_t R, int64_t table_rows,
                    int interleaved, int inverse, dit_dtype dtype, dit_stream_t stream);

/*
 * The same after a weighted RMSNorm of each head (its D columns), in one pass and
 * rounded once:  y = x * r * (weight_offset + weight),  r = 1 / sqrt(mean(x^2) + eps).
 * weight_q, weight_k: [D], shared by the heads.  The statistic is a
 * fp32 sum; r is within three fp32 ulps of that sum's (with eps = 0 a head of zeros gives NaN).  R may be
 * 0 (the norm alone; cos and sin may then be NULL).
 */
dit_status dit_rmsnorm_rope(const dit_heads* q_out, const dit_heads* k_out, const dit_heads* q,
                            const dit_heads* k, const void* weight_q, const void* weight_k,
                            const float* cos, const float* sin, int64_t B, int64_t L, int64_t Hq,
                            int64_t Hk, int64_t D, int64_t R, int64_t table_rows, float eps,
                            float weight_offset, int interleaved, dit_dtype dtype,
                            dit_stream_t stream);

/*
 * Its gradient.  With u the gradient of the output turned back, n = x * r and
 * t = u * (weight_offset + weight),
 *   grad_x      = rnd(r * (t - n * mean(t * n)))        (grad_q, grad_k)
 *   grad_weight = rnd(sum over tokens and heads of u * n)
 * in fp32.  grad_weight_q and grad_weight_k may each be NULL (a frozen weight).  q_grad
 * and k_grad, the outputs, may be the gradients they come from (q_out_grad,
 * k_out_grad).
 */
int64_t dit_rmsnorm_rope_backward_workspace_bytes(int64_t D);

dit_status dit_rmsnorm_rope_backward(const dit_heads* q_grad, const dit_heads* k_grad,
                                     void* grad_weight_q, void* grad_weight_k,
                                     const dit_heads* q_out_grad, const dit_heads* k_out_grad,
                                     const dit_heads* q, const dit_heads* k, const void* weight_q,
                                     const void* weight_k, const float* cos, const float* sin,
                                     int64_t B, int64_t L, int64_t Hq, int64_t Hk, int64_t D,
                                     int64_t R, int64_t table_rows, float eps, float weight_offset,
                                     int interleaved, dit_dtype dtype, void* workspace,
                                     int64_t workspace_bytes, dit_stream_t stream);

/*
 * A paged cache of keys and values.  Each of k and v is [pages, heads, page_size,
 * D], page p starting at p * page_stride elements (at least heads * page_size * D, so that
 * both may be halves of one allocation) and the rest contiguous.  format: a dit_dtype value, or
 * DIT_E4M3: codes with one scale per row of D, scales [pages, heads,
 * page_size] fp32, page p at p * scale_stride.  The value is code * scale, whatever the scale's sign.
 * page_size and pages * page_size are at most 2^31 - 1, D at most 1024, page_stride at most 2^40.
 * A place ("slot") is page * page_size + the token's place in the page.
 */
#define DIT_E4M3 3
typedef struct {
  void *k, *v;
  float *k_scales, *v_scales; /* DIT_E4M3 only */
  int64_t pages, heads, page_size, D;
  int64_t page_stride, scale_stride;
  int64_t format;
} dit_cache;

/*
 * Write the keys and values [tokens, heads, D] of dtype `dtype` (the cache's, where it is one) to
 * slots[t]; a token whose slot is outside [0, pages * page_size) is not
 * written.  The slots within that range must differ from each other: a slot that is named twice
 * gets some of the rows of both.  In E4M3, with m the maximum of |x| over the row,
 *   scale = fl32(m / 448),  code = e4m3(fl32(x * 448 / m)),
 * the quotient carried in two fp32 numbers.  m = 0 gives scale 0 and codes 0; a NaN or an
 * infinity makes the row's scale and codes NaN.  Nothing else of the cache changes.
 */
dit_status dit_cache_write(const dit_cache* cache, const dit_heads* k, const dit_heads* v,
                           int64_t tokens, const void* slots, dit_id_type id_type,
                           dit_dtype dtype, dit_stream_t stream);

/* The reverse:  k[t] = the row of slots[t], in E4M3 rnd(code * scale), a row of zeros where
 * the slot is outside the cache. */
dit_status dit_cache_read(const dit_cache* cache, const dit_heads* k, const dit_heads* v,
                          int64_t tokens, const void* slots, dit_id_type id_type, dit_dtype dtype,
                          dit_stream_t stream);

/*
 * Attention of one new token per sequence: for sequence b of n = lengths[b] tokens, query head
 * h and its key head h / (Hq / heads), over the tokens t from
 * max(0, n - window) (window 0: from 0) to n,
 *   s[t] = scale * sum_d q[b, h, d] k[t, d],  w[t] = exp(s[t] - max s),
 *   out[b, h] = rnd(sum w[t] v[t] / sum w[t]),  lse[b, h] = log(sum exp(s[t])).
 * Token t is at place t % page_size of page pages[b, t / page_size].  The new token's own
 * key and value are in the cache (write them first).
 *   q, out: [B, Hq, D] (dit_heads without `batch`); Hq a multiple of the cache's heads; D <= 512.
 *   pages: int32 [B, width], row b at b * pages_stride (0: one row for all).  lengths: [B], int32 or
 *   int64.  A length is cut to [0, width * page_size] (at most 2^31 - 4096).  A token whose page
 *   is outside the cache is left out.  A sequence with no token has out 0
 *   and lse -infinity.  What lies in the cache's pages behind a sequence does not matter, NaN included.
 *   lse: fp32 [B, Hq], or NULL.
 * Keys, values and weights of 16-bit types are multiplied on the tensor cores, with products and sums in fp32.  The
 * weights of bf16 and fp16 caches are rounded there to their type.  Over E4M3 they are rounded to fp16, after the value's
 * scale is taken in, or for fp16 queries taken in two parts, 22 bits of them.  For fp32 queries every number is
 * taken so, 22 bits and more of it (where an infinity among keys or values gives NaN).
 * The length is split over the GPU and the parts joined by a second kernel, in one order for
 * given lengths.
 */
int64_t dit_paged_attention_workspace_bytes(int64_t Hq, int64_t heads, int64_t D);

dit_status dit_paged_attention(const dit_heads* out, float* lse, const dit_heads* q,
                               const dit_cache* cache, const int32_t* pages, int64_t pages_stride,
                               int64_t width, const void* lengths, int64_t B, int64_t Hq,
                               float scale, int64_t window, dit_id_type id_type, dit_dtype dtype,
                               void* workspace, int64_t workspace_bytes, dit_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DIT_ELEMENTWISE_H */
