/*
 * fp8q.h -- C ABI of libfp8q: FP8 delayed-scaling quantization, microscaled
 * 4-bit operands, residual norms, FP8 products and 8-bit checkpoints on one GPU.
 *
 * Twenty operations, each one kernel launch on the caller's stream (those that
 * sum gradients over rows two; a 4-bit product with an empty k is a fill):
 *   fp8q_quantize_amax        bf16 -> FP8 bytes, fused with amax = max|x|
 *   fp8q_multi_quantize_amax  the same over a ragged list of tensors
 *   fp8q_dequantize           FP8 bytes -> bf16
 *   fp8q_amax_scale_update    amax-history roll + amax selection + scale and
 *                             scale_inv, for many FP8 metadata slots at once
 *   fp8q_qdq_amax             quantize then dequantize (bf16 -> bf16) + amax
 *   fp8q_amax_scale_update_ring  the update over a ring buffer (no roll)
 *   fp8q_gelu_quantize_amax   GELU producer fused with quantize + amax
 *   fp8q_layernorm_quantize_amax  LayerNorm producer fused with quantize + amax
 *   fp8q_amax_scale_update_ring_quantize  the ring update fused with the next
 *                             step's first quantize
 *   fp8q_fp4_quantize_amax    bf16 -> microscaled 4-bit operands (of a matrix,
 *                             its transpose, or both), fused with amax
 *   fp8q_fp4_dequantize       microscaled 4-bit -> bf16
 *   fp8q_fp4_matmul           the product of two microscaled 4-bit operands
 *   fp8q_residual_norm_quantize_amax  RMS norm after a block, gate, residual
 *                             add, RMS norm before the next block, quantize
 *   fp8q_residual_norm_backward  its gradients
 *   fp8q_matmul               the product of two FP8 operands, with bias, GELU,
 *                             residual, FP8 codes and a checkpoint in its epilogue
 *   fp8q_grouped_matmul       the same over rows grouped by expert
 *   fp8q_grouped_weight_gradient  the gradients of the experts' weights
 *   fp8q_checkpoint_quantize  bf16 -> an 8-bit checkpoint
 *   fp8q_checkpoint_dequantize  8-bit checkpoint -> bf16
 *   fp8q_gelu_backward_quantize_amax  back through a GELU from the checkpoint of
 *                             its input, quantize, the bias's gradient
 *
 * Sources (web pages, by title and section):
 *   "User Guide on Native XLA-FP8" (NVIDIA JAX-Toolbox): opening section
 *     (E4M3 / E5M2 formats, quantization Q and de-quantization DQ); section
 *     "JAX" (Q = cast(A / A_scale), DQ = cast(a_fp8) * a_scale, delayed
 *     scaling A_scale = max|A| / E4M3_MAX); section "Gradient accumulation of
 *     FP8 params" (FP8 meta accumulates with max, not add).
 *   "Fusion of Fp8 quantization and amax reduction kernels" (openxla/xla
 *     issue): quantization and the amax reduction are memory bound and
 *     belong in one pass over the tensor.
 *   "Implement fused kernel for FP8 scale update" (NVIDIA/TransformerEngine
 *     PR): amax_and_scale_update (history roll, amax selection, scale,
 *     scale_inv) as one in-place kernel in a framework-agnostic library,
 *     batched over all layers.
 *
 * Conventions shared by every call:
 *   - Data pointers are DEVICE memory of the calling thread's current CUDA
 *     device, owned by the caller.  The library allocates nothing, frees
 *     nothing and keeps no per-call state.  Inputs and outputs must not
 *     overlap unless a call says it works in place.
 *   - bf16 tensors are contiguous arrays of 16-bit patterns (any 2-byte
 *     aligned address); FP8 tensors are contiguous byte arrays.  Any
 *     alignment works; tensors whose bf16 and FP8 pointers are aligned alike
 *     (as allocators return them) take the vectorised path.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *     return once the kernel is enqueued; results are ready when the stream
 *     reaches that point.  The kernels of fp8q_fp4_* and of the calls behind it
 *     in the list above are launched so that their start overlaps the end of
 *     the kernel before them in the stream; they touch memory only when that
 *     has ended.
 *   - Errors are returned as fp8q_status, never raised or aborted.  Argument
 *     errors are detected before anything is launched.  FP8Q_ERR_CUDA means
 *     the launch itself failed; fp8q_last_cuda_error() (per thread) then
 *     describes it, and the error has been taken off the CUDA runtime's
 *     per-thread last error (cudaGetLastError) so that it is reported once.
 *     Each call checks only its own launch: a runtime error that an earlier,
 *     unrelated call left pending is neither reported nor cleared.
 *     A zero-sized call succeeds and launches nothing (but an output that is a
 *     sum over nothing is zeros, where a call says so).
 */
#ifndef FP8Q_H
#define FP8Q_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8Q_E4M3FN = 0, /* 1-4-3, bias 7, no inf, max 448 (forward pass) */
    FP8Q_E5M2 = 1,   /* 1-5-2, bias 15, IEEE inf/NaN, max 57344 (gradients) */
    /* microscaled 4-bit formats: e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and
     * their negatives) with a scale for each block of a row; taken by the
     * fp8q_fp4_* and fp8q_residual_norm_* calls only */
    FP8Q_MXFP4 = 2,  /* blocks of 32, scales are powers of two (ue8m0) */
    FP8Q_NVFP4 = 3   /* blocks of 16, e4m3 scales, and a binary32 tensor scale */
} fp8q_format;

typedef enum {
    FP8Q_OUT_BF16 = 0,
    FP8Q_OUT_F32 = 1
} fp8q_out_type;

typedef enum {
    FP8Q_ALGO_MAX = 0,        /* amax = max over the (rolled) history window */
    FP8Q_ALGO_MOST_RECENT = 1 /* amax = the newest entry */
} fp8q_amax_algo;

typedef enum {
    FP8Q_OK = 0,
    FP8Q_ERR_INVALID_ARG = 1,
    FP8Q_ERR_UNSUPPORTED = 2,
    FP8Q_ERR_CUDA = 3,
    FP8Q_ERR_TOO_MANY_TENSORS = 4
} fp8q_status;

/* Largest tensor count of one fp8q_multi_quantize_amax call (descriptors
 * travel inside the kernel's parameter block). */
#define FP8Q_MAX_TENSORS 512

/*
 * Fused quantize + amax of one bf16 tensor ("User Guide on Native XLA-FP8",
 * section "JAX", the quantization step; "Fusion of Fp8 quantization and amax
 * reduction kernels": amax fused into the same pass).
 *
 *   q[i]  = FP8(x[i] / *scale)   quotient in binary32, rounded to nearest even;
 *                                then rounded to the FP8 grid (nearest, ties
 *                                to even), saturating to +-448 / +-57344;
 *                                +-inf saturates; NaN gives a NaN code.
 *   *amax = max(*amax, max_i |x[i]|)   max-accumulated (not overwritten); a
 *                                NaN input makes it NaN; +-inf gives +inf.
 *
 * x_bf16: n bf16 values (device).  q: n bytes (device, written).
 * scale:  one float (device, read); any value, positive normal scales in
 *         [2^-60, 2^60] take the fast exact path.
 * amax:   one float (device, read-modify-write).  Start it at +0 (or any
 *         non-negative value) before the first tensor of a step.
 * Errors: INVALID_ARG for n < 0, an unknown fmt, a NULL pointer with n > 0
 *         or an odd x_bf16 address.
 */
fp8q_status fp8q_quantize_amax(const void* x_bf16, uint8_t* q, int64_t n, fp8q_format fmt,
                               const float* scale, float* amax, void* stream);

/* One tensor of a ragged list: its own size, scale and amax. */
typedef struct {
    const void* x_bf16; /* n bf16 values (device) */
    uint8_t* q;         /* n bytes (device, written) */
    int64_t n;          /* elements; 0 is allowed (pointers then unused) */
    const float* scale; /* one float (device) */
    float* amax;        /* one float (device), max-accumulated */
} fp8q_tensor;

/*
 * fp8q_quantize_amax over `count` tensors in ONE launch ("Fusion of Fp8
 * quantization and amax reduction kernels": weights and activations all need
 * Q + amax; "Implement fused kernel for FP8 scale update": batch the per-layer
 * work).  Each tensor gets exactly the result fp8q_quantize_amax would give.
 *
 * list:   `count` descriptors in HOST memory, read during the call only.
 * Errors: TOO_MANY_TENSORS for count > FP8Q_MAX_TENSORS; INVALID_ARG for
 *         count < 0, list == NULL with count > 0, or any descriptor that
 *         fp8q_quantize_amax would reject.  Two tensors may share an amax or
 *         a scale; outputs must not overlap.
 */
fp8q_status fp8q_multi_quantize_amax(const fp8q_tensor* list, int32_t count, fp8q_format fmt,
                                     void* stream);

/*
 * Dequantize ("User Guide on Native XLA-FP8", section "JAX": up-cast the FP8
 * value and multiply by the scale):
 *   y[i] = bf16_rne( float(q[i]) * *scale )   product in binary32 (RN), then
 *                                             rounded to nearest-even bf16;
 *                                             NaN codes give a NaN.
 * q: n bytes (device).  y_bf16: n bf16 (device, written).  scale: one float
 * (device).  Errors: INVALID_ARG for n < 0, unknown fmt, NULL with n > 0, odd
 * y_bf16 address.
 */
fp8q_status fp8q_dequantize(const uint8_t* q, void* y_bf16, int64_t n, fp8q_format fmt,
                            const float* scale, void* stream);

/*
 * amax_and_scale_update for `num_slots` FP8 metadata slots in ONE launch,
 * in place ("Implement fused kernel for FP8 scale update"; scale formula from
 * "User Guide on Native XLA-FP8", section "JAX", delayed scaling).  Per slot s:
 *   1. roll:   hist[h][s] <- hist[h-1][s] for h = H-1 .. 1 (oldest dropped);
 *              hist[0][s] <- amax_new[s]
 *   2. select: a = max_h hist[h][s] (ALGO_MAX; NaN wins) or hist[0][s]
 *              (ALGO_MOST_RECENT)
 *   3. scale:  if a is finite and > 0 and sc = RN(a / FP8_MAX) * 2^margin is
 *              a normal float: scale[s] = sc, scale_inv[s] = RN(1 / sc);
 *              otherwise scale[s] and scale_inv[s] are left unchanged.
 * FP8_MAX = 448 (e4m3fn) or 57344 (e5m2): from slot_format[s] when it is not
 * NULL (0 = e4m3fn, 1 = e5m2, any other code leaves that slot's scale alone),
 * else from fmt for every slot.
 *
 * amax_history: float[history_len][num_slots], row-major, row 0 newest
 * (device, updated in place).  amax_new: float[num_slots] (device, read).
 * scale, scale_inv: float[num_slots] (device, updated in place).
 * slot_format: uint8[num_slots] (device) or NULL.
 * Errors: INVALID_ARG for history_len < 1, num_slots < 1, a NULL or
 *         misaligned float pointer, unknown fmt or algo, margin outside
 *         [-64, 64].  amax_new must not overlap the history.
 */
fp8q_status fp8q_amax_scale_update(float* amax_history, int32_t history_len, int32_t num_slots,
                                   const float* amax_new, float* scale, float* scale_inv,
                                   const uint8_t* slot_format, fp8q_format fmt,
                                   fp8q_amax_algo algo, int32_t margin, void* stream);

/*
 * Fused quantize -> dequantize ("fake quant") with amax, in one pass
 * ("User Guide on Native XLA-FP8", section "Gradient accumulation of FP8
 * params": in_qdq passes a value through Q and DQ with its scale):
 *   y[i]  = bf16_rne( float(FP8(x[i] / *scale)) * *scale )   exactly
 *           fp8q_dequantize(fp8q_quantize_amax(x)), without the FP8 bytes
 *   *amax = max(*amax, max_i |x[i]|)
 * x_bf16: n bf16 (device).  y_bf16: n bf16 (device, written); y_bf16 may equal
 * x_bf16 (in place) but must not partially overlap it.  scale, amax: as for
 * fp8q_quantize_amax.  Errors: as for fp8q_quantize_amax, plus an odd y_bf16.
 */
fp8q_status fp8q_qdq_amax(const void* x_bf16, void* y_bf16, int64_t n, fp8q_format fmt,
                          const float* scale, float* amax, void* stream);

/*
 * amax_and_scale_update over a ring buffer: the same window, selection and
 * scale as fp8q_amax_scale_update, without moving the history.  Each slot's
 * oldest entry is overwritten in place instead of every entry shifting by one
 * row, so a call reads the history and writes one row.  (Window and scale:
 * "Implement fused kernel for FP8 scale update"; "User Guide on Native
 * XLA-FP8", section "JAX", delayed scaling.)  Per slot s, with h = head[s]:
 *   1. h' = (h + 1) mod H;  hist[h'][s] <- amax_new[s];  head[s] <- h'
 *   2. select: a = max over all H rows (ALGO_MAX; NaN wins) or amax_new[s]
 *   3. scale / scale_inv exactly as fp8q_amax_scale_update.
 * Logical row r (0 = newest) of slot s is physical row (head[s] - r) mod H,
 * so after any sequence of calls the window and the scales equal those of the
 * rolled form.  Start with head[s] = H - 1 to fill rows 0, 1, 2, ... in order.
 * A head outside [0, H) leaves that slot's history, head and scales untouched.
 *
 * amax_history: float[H][num_slots] row-major (device, one row per slot
 * written).  head: int32[num_slots] (device, read and advanced).  Other
 * arguments and errors: as for fp8q_amax_scale_update (head is checked like
 * the float pointers).
 */
fp8q_status fp8q_amax_scale_update_ring(float* amax_history, int32_t* head, int32_t history_len,
                                        int32_t num_slots, const float* amax_new, float* scale,
                                        float* scale_inv, const uint8_t* slot_format,
                                        fp8q_format fmt, fp8q_amax_algo algo, int32_t margin,
                                        void* stream);

/*
 * GELU producer fused with quantize + amax: the first MLP layer's output goes
 * through GELU and straight into FP8 for the next FP8 dense layer ("Fusion of
 * Fp8 quantization and amax reduction kernels": the reproducer's
 * dense -> gelu -> dense pattern, with quantization fused into what produces
 * its input), in one pass:
 *   y[i]  = bf16_rne(GELU(h[i]))        tanh form x / (1 + exp(-2u)),
 *                                        u = sqrt(2/pi)(x + 0.044715 x^3)
 *   q[i]  = FP8(y[i] / *scale)           exactly fp8q_quantize_amax of y
 *   *amax = max(*amax, max_i |y[i]|)
 * GELU is evaluated by a fixed sequence of correctly rounded binary32
 * operations (exp by additive range reduction and a degree-6 Taylor
 * polynomial), so it is reproducible bit for bit: y is the bf16 rounding of a
 * value within (6|v| + 10) 2^-24 relative of the exact tanh-form GELU, with
 * v = 2 sqrt(2/pi) x (1 + 0.044715 x^2) (and within 2^-122 absolute where
 * |GELU| < 2^-122).  The codes and the amax are exactly those of quantizing
 * the y returned.
 * h_bf16: n bf16 (device).  y_bf16: n bf16 (device, written) or NULL when only
 * the FP8 codes are wanted.  q, scale, amax: as for fp8q_quantize_amax.
 * Large tensors go through a table of every bf16 input built by thread-block
 * clusters; on a device where no such cluster can be resident (a partitioned
 * or shared GPU) the call takes the element-by-element kernel, with the same
 * results.  The first large call on a device queries how many clusters fit
 * (host-side calls, allowed during graph capture).
 * Errors: as for fp8q_quantize_amax, plus an odd y_bf16.
 */
fp8q_status fp8q_gelu_quantize_amax(const void* h_bf16, void* y_bf16, uint8_t* q, int64_t n,
                                    fp8q_format fmt, const float* scale, float* amax, void* stream);

/*
 * LayerNorm producer fused with quantize + amax: the transformer block of the
 * reproducer in "Fusion of Fp8 quantization and amax reduction kernels"
 * (test.py) normalises its input with a LayerNorm and feeds the MLP's first
 * FP8 dense layer; this computes that layer's FP8 input in one pass over x.
 * Row by row (rows x hidden, row-major), in binary32 with Flax's defaults:
 *   mean = S / H, var = max(0, Q / H - mean^2), rstd = 1 / sqrt(var + eps)
 *   y[i]  = bf16_rne((x[i] - mean) * (rstd * gamma[i]) + beta[i])
 *   q[i]  = FP8(y[i] / *scale)           exactly fp8q_quantize_amax of y
 *   *amax = max(*amax, max |y|)          over every row
 * with S = sum x and Q = sum x^2.  Precision: y is the bf16 rounding of a
 * value within a stated bound of the exact (float64) LayerNorm; the bound
 * follows binary32 error analysis with row sums whose longest chain of
 * additions is at most hidden / 128 + 32 (rows are summed in a fixed order, so
 * a call is reproducible bit for bit), and y is that exact value rounded once to bf16
 * unless it lies close to a bf16 rounding boundary.  The codes and the amax
 * are always exactly those of quantizing the y returned.  A NaN or infinite
 * x makes its row's y NaN.
 * The kernel stages rows of x in shared memory with asynchronous bulk copies
 * and waits for each copy at most one second.  Should a wait ever run out
 * (correct operation never gets there), the call stops early, leaving the
 * outputs incomplete and *amax holding the bit pattern 0x7FFFFFFF: a NaN that
 * no bf16 data can produce (a NaN input gives the canonical 0x7FC00000 or
 * another pattern below 0x7FFFFFFF).  A caller that must tell this apart reads
 * *amax's bits after the stream has reached the call.
 * x_bf16: rows * hidden bf16 (device).  y_bf16: the same (device, written)
 * or NULL when only the FP8 codes are wanted.  q: rows * hidden bytes
 * (device).  gamma, beta: hidden floats each (device).  These five must be
 * 16-byte aligned.  scale, amax: as for fp8q_quantize_amax.  hidden: a
 * multiple of 16 from 16 to 32768.  Rows longer than 4096 run on
 * thread-block clusters of ceil(hidden / 4096) CTAs, each CTA a column slice
 * (up to 96 KB of shared memory); where no cluster of that size fits on the
 * device, one CTA takes each batch of rows instead (rows longer than 16384
 * then take 4 * hidden bytes of shared memory, one CTA per SM).  Both give y
 * within the same bound, not always the same bits.
 * The first call on a device also sets the kernel's shared-memory limit
 * (cudaFuncSetAttribute) and reads its occupancy.  Those are host-side calls,
 * not stream work, so that first call may itself be captured in a CUDA graph.
 * Errors: FP8Q_ERR_INVALID_ARG for a bad fmt, rows < 0, hidden < 16 or not a
 * multiple of 16, a NULL pointer (other than y_bf16) with rows > 0, or a
 * misaligned scale/amax; FP8Q_ERR_UNSUPPORTED for hidden > 32768 or a
 * misaligned x_bf16, y_bf16, q, gamma or beta; FP8Q_ERR_CUDA if the launch
 * or its first-call set-up fails.  rows == 0 launches nothing.
 */
fp8q_status fp8q_layernorm_quantize_amax(const void* x_bf16, void* y_bf16, uint8_t* q, int64_t rows,
                                         int32_t hidden, const float* gamma, const float* beta,
                                         float eps, fp8q_format fmt, const float* scale, float* amax,
                                         void* stream);

/*
 * The ring-buffer update fused with the quantize that follows it, in one
 * launch: the update sits between one step's amax and the next step's casts
 * ("Implement fused kernel for FP8 scale update": one launch per update; the
 * next quantize then needs its new scale), so this call does both:
 *   fp8q_amax_scale_update_ring(history, heads, ...)   for every slot, then
 *   fp8q_quantize_amax(x, q, n, fmt, &scale[slot], amax)
 * with identical results.  The heads come in through head_in (read only) and
 * go out through head_out (written for every slot; swap the two arrays between
 * steps).  The quantizing CTAs compute slot `slot`'s new scale themselves from
 * its history column (without the row the update overwrites) and amax_new,
 * with the update's own arithmetic, so no CTA waits for another.
 * amax_history, history_len, num_slots, amax_new, scale, scale_inv,
 * slot_format, algo, margin: as fp8q_amax_scale_update_ring.  fmt: the FP8
 * format of q, and the format of slots without slot_format (give slot `slot`
 * the format of q).  x_bf16, q, n, amax: as fp8q_quantize_amax; amax must not
 * alias amax_new or the history.  slot: 0 <= slot < num_slots.
 * Errors: those of both calls, plus FP8Q_ERR_INVALID_ARG for a slot out of
 * range or head_out equal to head_in.  n == 0 runs only the update.
 */
fp8q_status fp8q_amax_scale_update_ring_quantize(float* amax_history, const int32_t* head_in,
                                                 int32_t* head_out, int32_t history_len, int32_t num_slots,
                                                 const float* amax_new, float* scale, float* scale_inv,
                                                 const uint8_t* slot_format, fp8q_format fmt,
                                                 fp8q_amax_algo algo, int32_t margin, const void* x_bf16,
                                                 uint8_t* q, int64_t n, int32_t slot, float* amax,
                                                 void* stream);

/*
 * Microscaled 4-bit operands.  A packed operand of an [rows, cols] matrix is
 *   codes   rows x fp8q_fp4_row_bytes(cols) bytes: two e2m1 codes a byte (the
 *           even column in the low four bits), each row filled up with zero
 *           codes to a multiple of 32 columns;
 *   scales  fp8q_fp4_scale_bytes(rows, cols, fmt) bytes: one for each block of
 *           32 (FP8Q_MXFP4) or 16 (FP8Q_NVFP4) columns, in tiles of 128 rows x
 *           4 blocks of 512 bytes, tiles row by row; within a tile the scale
 *           of (row, block) lies at (row % 32) * 16 + (row % 128) / 32 * 4 +
 *           block % 4.  A row's blocks are filled up to a multiple of 4 with
 *           zero scales; rows that fill up the last tile are neither written
 *           nor used.
 * Both arrays start on 16-byte boundaries.  The two functions give 0 for sizes
 * that the calls refuse.
 */
int64_t fp8q_fp4_row_bytes(int64_t cols);
int64_t fp8q_fp4_scale_bytes(int64_t rows, int64_t cols, fp8q_format fmt);

/*
 * bf16 -> microscaled 4 bits with amax, in one pass over x, which is [rows,
 * cols], row-major.  q, sf: the packed operand of x (blocks along a row).  qt,
 * sft: the packed operand of x's transpose, [cols, rows] (blocks down a
 * column): what the products of a backward pass read.  Either pair may be
 * NULL, not both.  With a = max|x| of a block:
 *   FP8Q_MXFP4  scale 2^e, e = max(-127, floor(log2 a) - 2); an infinite a
 *               counts as the largest finite bf16; a NaN in the block makes
 *               its scale NaN (0xFF).  code = e2m1(x / 2^e).
 *   FP8Q_NVFP4  with the tensor scale s: block scale sb = e4m3(RN(a / RN(6 s))),
 *               held at 448, d = RN(sb s), code = e2m1(RN(x / d)), signed zeros
 *               where d is 0; RN is a rounding to binary32.  A NaN in the
 *               block, or an s whose RN(6 s) is not positive and finite, makes
 *               sb NaN (0x7F), but a block of zeros always has scale and
 *               codes 0.
 * e2m1 rounds to nearest, ties to the even code, held at +-6; infinities become
 * +-6.  *amax = max(*amax, max|x|) as for fp8q_quantize_amax.
 * scale: one float (device), or NULL for 1; NULL for FP8Q_MXFP4.  amax / 2688
 * (the largest element 6 times the largest block scale 448) uses the whole
 * range.  amax: one float (device), or NULL where it is not wanted.
 * Errors: INVALID_ARG for another fmt, rows or cols < 0, a NULL x_bf16, no
 *         output or half a pair, a scale with FP8Q_MXFP4, or a misaligned
 *         x_bf16, scale or amax; UNSUPPORTED for q, sf, qt or sft off a
 *         16-byte boundary, or rows or cols above 2^31 - 1024.
 */
fp8q_status fp8q_fp4_quantize_amax(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* q, uint8_t* sf,
                                   uint8_t* qt, uint8_t* sft, fp8q_format fmt, const float* scale, float* amax,
                                   void* stream);

/*
 * Microscaled 4 bits -> bf16: y = bf16(RN(code * block scale * s)), y [rows,
 * cols] row-major; the product of code and block scale is exact.  scale: one
 * float (device), or NULL for 1; NULL for FP8Q_MXFP4.  Errors: as for
 * fp8q_fp4_quantize_amax.
 */
fp8q_status fp8q_fp4_dequantize(const uint8_t* q, const uint8_t* sf, void* y_bf16, int64_t rows, int64_t cols,
                                fp8q_format fmt, const float* scale, void* stream);

/*
 * The product of two microscaled 4-bit operands of the same format, both
 * packed along k:
 *   d[i][j] = RN_out( (sum_k a[i][k] b[j][k]) * RN(a_scale * b_scale) )
 * a is [m, k], b is [n, k], d is [m, n], row-major, bf16 or binary32.  A linear
 * layer's output is the product of its input and its weight; its input's
 * gradient that of the output's gradient and the weight's transpose; its
 * weight's gradient that of the output's gradient's and the input's
 * transposes.  Products are exact; sums are held in binary32.
 * a_scale, b_scale: the tensor scales, one float each (device), or NULL for 1;
 * NULL for FP8Q_MXFP4.  Calls with the same arguments give the same bits.
 * With k == 0, d is zeros (the operands may be NULL).
 * A wait inside the kernel that runs out, which only a fault elsewhere could
 * cause, ends the kernel and shows as NaN in d, with all the bits behind the
 * sign set.
 * Errors: INVALID_ARG for another fmt or out, m, n or k < 0, a NULL operand or
 *         d, a scale with FP8Q_MXFP4, or a misaligned d or scale; UNSUPPORTED
 *         for an operand off a 16-byte boundary or m, n or k above 2^31 -
 *         1024.  m == 0 or n == 0 launches nothing.
 */
fp8q_status fp8q_fp4_matmul(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, void* d,
                            int64_t m, int64_t n, int64_t k, fp8q_format fmt, fp8q_out_type out,
                            const float* a_scale, const float* b_scale, void* stream);

/*
 * The RMS norms after and before a transformer block, fused with the block's
 * gate, the residual scale and the quantization of the next block's input.
 * Row by row, in binary32:
 *   y  = b / sqrt(mean(b^2) + eps) * post_weight     (y = b without post_weight)
 *   r' = bf16(residual + alpha * gate * y)           (r' = residual without block)
 *   h  = bf16(r' / sqrt(mean(r'^2) + eps) * pre_weight)    of the rounded r'
 *   q  = the codes of h in fmt, exactly those of fp8q_quantize_amax or
 *        fp8q_fp4_quantize_amax;  *amax = max(*amax, max|h|)
 * A norm of a row that holds a NaN or an infinity, or whose sum of squares is
 * beyond binary32 (an element of 2^64 is enough), is NaN in every column: y, and
 * so r', for such a row of block (with post_weight); h for one of r'.  Any part
 * may be left out by NULL: block (then no post_weight and gate), post_weight,
 * gate (1), residual_out (without block only), pre_weight (then no h, q and
 * amax), h or q (one of them with pre_weight), sf (FP8 formats), scale (NULL
 * for FP8Q_MXFP4; 1 for FP8Q_NVFP4 without), amax, rstd_post, rstd_pre.
 */
typedef struct {
    int64_t rows;             /* tokens */
    int32_t hidden;           /* a multiple of 16 from 16 to 32768 */
    fp8q_format fmt;          /* of q */
    const void* residual;     /* [rows, hidden] bf16 */
    const void* block;        /* [rows, hidden] bf16: the block's output */
    const float* post_weight; /* [hidden] */
    const void* gate;         /* [ceil(rows / rows_per_gate), hidden] binary32 or bf16 */
    int64_t rows_per_gate;    /* consecutive rows that share a row of gate: 1, a sequence, or all */
    int32_t gate_is_bf16;
    float alpha;              /* the residual scale */
    float eps;
    const float* pre_weight;  /* [hidden] */
    void* residual_out;       /* [rows, hidden] bf16; may be residual */
    void* h;                  /* [rows, hidden] bf16 */
    uint8_t* q;               /* FP8: [rows, hidden] bytes; 4 bits: a packed operand's codes */
    uint8_t* sf;              /* 4 bits: its scales */
    const float* scale;       /* one float */
    float* amax;              /* one float, max-accumulated */
    float* rstd_post;         /* [rows]: 1 / sqrt(mean(b^2) + eps), for the backward pass */
    float* rstd_pre;          /* [rows]: 1 / sqrt(mean(r'^2) + eps) */
} fp8q_residual_norm;

/*
 * Errors: INVALID_ARG for a NULL args, another fmt, rows < 0, hidden < 16 or
 *         not a multiple of 16, rows_per_gate < 1 with gate, parts missing or
 *         left over as listed above, or a misaligned scale, amax or rstd;
 *         UNSUPPORTED for hidden > 32768, rows above 2^31 - 1024 or another
 *         pointer off a 16-byte boundary.  rows == 0 launches nothing.
 */
fp8q_status fp8q_residual_norm_quantize_amax(const fp8q_residual_norm* args, void* stream);

/*
 * Gradients of the call above (the quantization counts as the identity).  With
 * n1 = block * rstd_post (block without post_weight), n2 = r' * rstd_pre,
 * dn = d_h * pre_weight:
 *   D             = d_residual_out + rstd_pre (dn - n2 mean(dn n2))
 *   d_residual    = bf16(D)                      (d_residual_out's and d_h's share)
 *   e             = alpha * gate * D
 *   d_block       = bf16(rstd_post (e post_weight - n1 mean(e post_weight n1)))
 *                                                (bf16(e) without post_weight)
 *   d_pre_weight  = sum over rows of d_h n2
 *   d_post_weight = sum over rows of e n1
 *   d_gate        = sum over the rows of a gate's row of alpha D n1 post_weight
 * D is not rounded on the way to the others.  Sums are taken in binary32 in a
 * fixed order: the same arguments give the same bits.
 */
typedef struct {
    int64_t rows;
    int32_t hidden;
    int32_t gate_is_bf16;
    const void* d_residual_out; /* [rows, hidden] bf16, or NULL for zeros */
    const void* d_h;            /* [rows, hidden] bf16, or NULL without pre_weight */
    const void* residual_out;   /* r', [rows, hidden] bf16 (with d_h) */
    const float* rstd_pre;      /* [rows] (with d_h) */
    const float* pre_weight;    /* [hidden] (with d_h) */
    const void* block;          /* [rows, hidden] bf16, or NULL */
    const float* rstd_post;     /* [rows] (with post_weight) */
    const float* post_weight;   /* [hidden], or NULL */
    const void* gate;           /* as in the forward call, or NULL */
    int64_t rows_per_gate;
    float alpha;
    void* d_residual;           /* [rows, hidden] bf16, or NULL */
    void* d_block;              /* [rows, hidden] bf16, or NULL */
    float* d_pre_weight;        /* [hidden], or NULL */
    float* d_post_weight;       /* [hidden], or NULL */
    void* d_gate;               /* gate's shape and type, or NULL */
    void* workspace;            /* fp8q_residual_norm_backward_workspace bytes */
    int64_t workspace_bytes;
} fp8q_residual_norm_grad;

/* Bytes of workspace (16-byte aligned, contents irrelevant) for the gradients
 * of weights and of a gate that rows share; one call at a time may use it.
 * rows_per_gate: 0 without gate.  0 for sizes that the call refuses. */
int64_t fp8q_residual_norm_backward_workspace(int64_t rows, int32_t hidden, int64_t rows_per_gate);

/*
 * Errors: INVALID_ARG for a NULL args, rows < 0, hidden < 16 or not a multiple
 *         of 16, neither gradient given, parts missing or left over, too small
 *         a workspace, or a misaligned rstd; UNSUPPORTED for hidden > 32768,
 *         rows above 2^31 - 1024 or another pointer off a 16-byte boundary.
 *         With rows == 0 d_pre_weight and d_post_weight are zeros; nothing else
 *         is read or written.
 */
fp8q_status fp8q_residual_norm_backward(const fp8q_residual_norm_grad* args, void* stream);

/*
 * The product of two FP8 operands with what follows a linear layer:
 *   z = RN(a_scale * b_scale) * (sum_k a[i][k] b[j][k]) + bias[j]
 *   y = act(z) + residual[i][j]
 *   d = RN_out(y);   q = FP8(bf16(y) / *q_scale), exactly fp8q_quantize_amax of
 *   bf16(y);   *amax = max(*amax, max|bf16(y)|)
 *   (h, h_sf) = fp8q_checkpoint_quantize of bf16(z)
 * Parts may be left out by NULL: bias, residual, and of d, q, amax and h any but
 * the last one.  A is [m, k], or with a_trans stored as its transpose, [k, m]; B
 * is [n, k], or with b_trans [k, n]; each row starts lda (ldb) bytes behind the
 * one before.  So with x [m, k], w [n, k] and the gradient dy [m, n], a layer's
 * output is (x, w), its input's gradient (dy, w with b_trans) and its weight's
 * gradient (dy with a_trans, x with b_trans); no transposed copies are needed.
 * d, q, residual and h are contiguous [m, n].  residual has d's type (bf16
 * without d) and may be d.  (An operand's rows lie 16 bytes or a multiple
 * apart, so codes q of a width that is no multiple of 16 have to be laid out
 * anew before they are the next product's operand.)  Products are exact.  Sums
 * are held in binary32 by the tensor cores, which cut off, towards zero, what
 * lies below a sum's last place, once for 32 of k at most: measured, of the
 * results' root mean square, 3e-8 at k = 512, 1e-7 to 2.4e-7 at 4096 and 6e-7
 * to 1.5e-6 at 16384; a longer k goes by parts of 8192 whose sums are added
 * rounded to nearest, 6e-7 at any length.  The rest is binary32, rounded to
 * nearest, with the GELU (tanh form) within 2^-16 of its value (2^-18 from z =
 * -5 on; below z = -10, where it is near 0, within 2^-100; NaN at -infinity, as
 * in fp8q_gelu_quantize_amax, whose bits are its own: these are not those).
 * Calls with the same arguments give the same bits.  With k == 0 the sums are
 * zeros and a and b may be NULL.
 * A wait inside the kernel that runs out, which only a fault elsewhere could
 * cause (none has to last as long as a long k does), ends the kernel and shows
 * as NaN in what it had not finished.
 */
typedef enum {
    FP8Q_ACT_NONE = 0,
    FP8Q_ACT_GELU = 1
} fp8q_activation;

typedef struct {
    int64_t m, n, k;
    const uint8_t* a;     /* codes */
    const uint8_t* b;
    int64_t lda, ldb;     /* bytes from row to row as stored; multiples of 16 */
    fp8q_format a_fmt, b_fmt;
    int32_t a_trans, b_trans;
    const float* a_scale; /* tensor scales, one float each, or NULL for 1 */
    const float* b_scale;
    const void* bias;     /* [n] binary32 or bf16 */
    int32_t bias_is_bf16;
    fp8q_activation act;
    const void* residual; /* [m, n] */
    void* d;              /* [m, n] */
    fp8q_out_type out;    /* of d; FP8Q_OUT_BF16 with q or amax, or without d */
    fp8q_format q_fmt;
    uint8_t* q;           /* [m, n] */
    const float* q_scale; /* one float (with q) */
    float* amax;          /* one float, max-accumulated */
    uint8_t* h;           /* [m, n] */
    uint8_t* h_sf;        /* [m, ceil(n / 32)] (with h) */
} fp8q_product;

/*
 * Errors: INVALID_ARG for a NULL args, an unknown format, type or act, m, n or
 *         k < 0, parts missing or left over as said above, a row shorter than
 *         its elements, or a pointer that its elements' size does not divide;
 *         UNSUPPORTED for a, b, lda or ldb off 16 bytes, lda or ldb from 2^31
 *         on, or m, n or k above 2^31 - 1024.  m == 0 or n == 0 launches
 *         nothing.
 */
fp8q_status fp8q_matmul(const fp8q_product* args, void* stream);

/*
 * fp8q_matmul over rows grouped by expert: row i of A, of group g, is multiplied
 * by B's g-th matrix.  Group g is the rows offsets[g] to offsets[g + 1] - 1; it
 * may be empty.  args: A is [m, k] (never transposed), m the rows of all groups;
 * B is [groups, n, k] ([groups, k, n] with b_trans), the matrices one behind the
 * other; bias is [groups, n].  All groups share a_scale, b_scale and q_scale.
 * Rows before the first group and behind the last are not written and count for
 * nothing.
 * offsets: int32[groups + 1] (device), read by the kernel: they must not
 * decrease.  Any values are safe: one outside [0, m] counts as the bound, and a
 * group that would end before it starts is empty; rows that two groups hold
 * then get either's result (on a residual in place, possibly both's).
 * Errors: as for fp8q_matmul, and INVALID_ARG for groups < 0, NULL offsets or
 *         a_trans; UNSUPPORTED for groups > 512.  groups == 0 launches nothing.
 */
fp8q_status fp8q_grouped_matmul(const fp8q_product* args, const int32_t* offsets, int32_t groups, void* stream);

/*
 * The gradients of the experts' weights: for every group g
 *   d[g] = RN_out( RN(a_scale * b_scale) * sum over the group's rows t of a[t][i] b[t][j] + residual[g][i][j] )
 * args: a is [k, m] and b is [k, n], k the rows of all groups (a_trans and
 * b_trans are set); d and residual are [groups, m, n]; no bias, act, q, amax or
 * h.  An empty group's sums are zeros.  Codes of other groups' rows, NaN among
 * them, do not reach a group's sums.  offsets, groups, errors: as for
 * fp8q_grouped_matmul.
 */
fp8q_status fp8q_grouped_weight_gradient(const fp8q_product* args, const int32_t* offsets, int32_t groups, void* stream);

/*
 * The 8-bit checkpoint of an activation, for a backward pass: e4m3 codes under
 * a power of two for each block of 32 columns of a row.  With a = max|x| of the
 * block, its scale is 2^e with the least e >= -127 for which a <= 448 * 2^e, kept
 * as the byte e + 127; code = e4m3(x / 2^e), the quotient exact.  So a value is
 * off by at most 2^-4 of itself, or 2^(e - 10) where that is more.  An infinity
 * counts as the largest finite bf16 in a and comes back as an infinity, and so do
 * the eight finite bf16 from 248 * 2^120 on (0x7F78 to 0x7F7F, and their
 * negatives): their code is that of 256, and 256 * 2^120 is beyond binary32.  A
 * NaN in the block makes its scale NaN (0xFF).
 * q: [rows, cols] bytes, sf: fp8q_checkpoint_scale_bytes, [rows, ceil(cols / 32)]
 * bytes, both contiguous, from any address; on 16-byte and 4-byte boundaries, with
 * x_bf16 on a 32-byte one and cols a multiple of 16, they take the vectorised path.
 * Back: y = bf16(code * 2^e), the product exact.
 * Errors: INVALID_ARG for rows or cols < 0, a NULL or an odd bf16 pointer;
 *         UNSUPPORTED for rows or cols above 2^31 - 1024.
 */
int64_t fp8q_checkpoint_scale_bytes(int64_t rows, int64_t cols);
fp8q_status fp8q_checkpoint_quantize(const void* x_bf16, uint8_t* q, uint8_t* sf, int64_t rows, int64_t cols, void* stream);
fp8q_status fp8q_checkpoint_dequantize(const uint8_t* q, const uint8_t* sf, void* y_bf16, int64_t rows, int64_t cols, void* stream);

/*
 * Back through a GELU (tanh form), from the checkpoint (h, h_sf) of its input:
 *   D      = d_y * GELU'(h)                       in binary32 (d_y without h)
 *   d_x    = bf16(D),  q = FP8(d_x / *scale) exactly as fp8q_quantize_amax,
 *   *amax  = max(*amax, max|d_x|),  d_bias = sum over rows of D
 * h and h_sf may be NULL together (a layer without activation), and of q (with
 * scale), d_x, d_bias and amax any but the last one.  GELU' is within 2^-19 (1 +
 * |h|) of its value; a NaN in h or d_y gives NaN.  Sums are taken in binary32 in
 * a fixed order.
 */
typedef struct {
    int64_t rows, cols;
    fp8q_format fmt;      /* of q */
    const void* d_y;      /* [rows, cols] bf16 */
    const uint8_t* h;     /* [rows, cols] */
    const uint8_t* h_sf;  /* [rows, ceil(cols / 32)] */
    void* d_x;            /* [rows, cols] bf16 */
    uint8_t* q;           /* [rows, cols] */
    const float* scale;   /* one float */
    float* amax;          /* one float, max-accumulated */
    float* d_bias;        /* [cols] */
    void* workspace;      /* fp8q_gelu_backward_workspace bytes, with d_bias */
    int64_t workspace_bytes;
} fp8q_gelu_grad;

/* Bytes of workspace (4-byte aligned, contents irrelevant) for d_bias; one call
 * at a time may use it.  0 for sizes that the call refuses. */
int64_t fp8q_gelu_backward_workspace(int64_t rows, int64_t cols);

/*
 * Errors: INVALID_ARG for a NULL args or d_y, an unknown fmt, rows or cols < 0,
 *         parts missing or left over, too small a workspace, or a misaligned
 *         pointer; UNSUPPORTED for rows or cols above 2^31 - 1024.  With rows ==
 *         0 d_bias is zeros and nothing else is read or written.
 */
fp8q_status fp8q_gelu_backward_quantize_amax(const fp8q_gelu_grad* args, void* stream);

/* Static, human-readable name of a status. */
const char* fp8q_status_string(fp8q_status status);

/* Text of the calling thread's last FP8Q_ERR_CUDA ("" if none). */
const char* fp8q_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_H */
