/*
 * fp8amax.h -- C ABI of the GB300 (sm_103a) FP8 delayed-scaling linear layer.
 *
 * The operations follow three web pages on FP8 mixed-precision training:
 *  - "NVIDIA Transformer Engine and FP8 mixed precision: implementation guide"
 *    (ai-tool-zukan.com): section "What are Transformer Engine and FP8 mixed
 *    precision" (E4M3 = 4 exponent / 3 mantissa bits for the forward pass,
 *    E5M2 = 5 / 2 for the backward pass; dynamic scaling watches each
 *    tensor's range and adjusts its scale factor) and section "Dynamic
 *    scaling and the FP8 recipe" (DelayedScaling with margin, fp8_format,
 *    amax_history_len; Format.HYBRID = E4M3 forward / E5M2 backward; the
 *    amax history is part of the model state).
 *  - "FP8 quantization with NVIDIA TensorRT" (ai.warp-studio.com): explicit
 *    quantize / dequantize (Q/DQ) nodes and the Absolute-Max statistic.
 *  - "Mixed-precision training" wiki note (notes.yuuk.io): "Definition" table
 *    (E4M3 max 448, E5M2 max 57,344) and the bullets "extension to FP8"
 *    (only the GEMMs run in FP8) and "per-tensor scaling is the key"
 *    (delayed or just-in-time per-tensor scaling).
 *
 * Numerics (identical on every call):
 *  - amax(x) = max |x_i| over the tensor, NaN entries skipped, exact.
 *  - cast: v = fl32(x * scale) (one binary32 multiply), then round to the
 *    nearest FP8 value, ties to the even code; |v| above the largest finite
 *    value and +-inf saturate to +-448 (E4M3) / +-57344 (E5M2); NaN stays NaN;
 *    the sign of zero is kept.  E4M3 is the variant with no infinities whose
 *    only NaN code is S.1111.111 (largest finite 448); E5M2 is IEEE-style.
 *  - scale update: history <- [amax, history[0..L-2]]; m = max(history); if
 *    0 < m < inf then scale = fl32(fl32(fmax / m) * 2^-margin) (+inf clamped
 *    to FLT_MAX) and scale_inv = fl32(1 / scale); otherwise both unchanged.
 *  - GEMM: D[i][j] = bf16_rne(fl32(acc[i][j] * fl32(a_scale_inv * b_scale_inv)))
 *    with acc = sum_k A[i][k] * B[j][k] accumulated in fp32 by the tensor
 *    cores, and d_amax = max |D| over the emitted BF16 values.
 *
 * Conventions for every entry point:
 *  - Pointers named as DEVICE pointers must be device (or managed) memory of
 *    the current device; the caller allocates and owns every buffer.  The
 *    library allocates no device memory, never synchronizes the stream (except
 *    fp8_sync_status), and keeps no state beyond cached device properties,
 *    one device-side error flag, the diagnostic clock-probe pointer
 *    (fp8_set_clock_probe) and the fixed work array that
 *    fp8_linear_bwd_noalloc uses (described there).
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream).  All work is enqueued on it, in order; scales are read on the
 *    device, so a training step needs no host round trip.
 *  - Tensors are dense row-major (the block-scaled ones at the end of this
 *    file take row strides and any size).  Row and column counts must be multiples of
 *    16 and tensor pointers 16-byte aligned (else FP8_ERR_ALIGN), so that
 *    every row of every FP8 and BF16 tensor starts on a 16-byte boundary.
 *    Pointers to fp32 scalars and to the fp8_meta buffers need 4-byte
 *    alignment only.
 *  - Arguments are checked on the host before anything is enqueued; on any
 *    status other than FP8_OK nothing was enqueued, and fp8_last_error()
 *    gives a message (thread-local).  Errors reported by the CUDA runtime at
 *    launch give FP8_ERR_CUDA.
 *  - Bounded waits: every spin-wait in a kernel gives up after about two
 *    seconds, sets a device error flag and returns; fp8_sync_status() reports
 *    it as FP8_ERR_TIMEOUT.
 */
#ifndef FP8AMAX_H
#define FP8AMAX_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8AMAX_ABI_VERSION 4

typedef enum { FP8_E4M3 = 0, FP8_E5M2 = 1 } fp8_format;

typedef enum {
    FP8_OK = 0,
    FP8_ERR_ARG = 1,         /* bad size, NULL pointer, bad format / margin / history length */
    FP8_ERR_ALIGN = 2,       /* size not a multiple of 16 or a pointer misaligned */
    FP8_ERR_CUDA = 3,        /* the CUDA runtime reported an error */
    FP8_ERR_TIMEOUT = 4,     /* a kernel's bounded wait ran out (see fp8_sync_status) */
    FP8_ERR_UNSUPPORTED = 5  /* the current device is not an sm_103 GPU */
} fp8_status;

/* The five tensors of one linear layer whose scaling state is tracked. */
enum { FP8_SLOT_X = 0, FP8_SLOT_W = 1, FP8_SLOT_Y = 2, FP8_SLOT_DY = 3, FP8_SLOT_DX = 4,
       FP8_NUM_SLOTS = 5 };

/* Scaling state of one linear layer (the DelayedScaling state the
 * implementation guide says is saved with the model).  All DEVICE pointers,
 * caller-owned, fp32:
 *   history   [5][history_len]  row = slot; history[slot*L + 0] is the newest
 *   amax      [5]               this step's amax of each slot
 *   scale     [5]               multiplier applied before the FP8 cast (init 1)
 *   scale_inv [5]               1 / scale, applied in the GEMM epilogue (init 1)
 * A fresh state is history = 0, amax = 0, scale = scale_inv = 1. */
typedef struct {
    float *history;
    float *amax;
    float *scale;
    float *scale_inv;
    int32_t history_len;
} fp8_meta;

/* DelayedScaling recipe (implementation guide, "Dynamic scaling and the FP8
 * recipe"): margin (>= 0, default 0; larger = fewer overflows, more
 * underflow), amax_history_len (default 1024) and the format choice.
 * hybrid = 1: E4M3 for X, W, Y and E5M2 for dY, dX (Format.HYBRID);
 * hybrid = 0: E4M3 for all five.  The scale is updated every step.
 * scaling selects between the two per-tensor scalings the wiki note names
 * ("per-tensor scaling is the key": delayed or just-in-time):
 *   FP8_SCALING_DELAYED  the casts use the scales the previous step's
 *                        fp8_amax_scale_update derived from the history;
 *   FP8_SCALING_CURRENT  X, W and dY are cast with a scale derived from
 *                        their own amax in the same call (the formula with
 *                        a history of one), written to meta->scale /
 *                        scale_inv; the history update still runs. */
enum { FP8_SCALING_DELAYED = 0, FP8_SCALING_CURRENT = 1 };
typedef struct {
    int32_t margin;
    int32_t history_len;
    int32_t hybrid;
    int32_t scaling;
} fp8_recipe;

/* ABI version of the loaded library (FP8AMAX_ABI_VERSION). */
int32_t fp8_abi_version(void);

/* Message of the last non-OK status returned on this host thread. */
const char *fp8_last_error(void);

/* Synchronize `stream`, then report (and clear) the device error flag:
 * FP8_ERR_TIMEOUT if a kernel gave up a bounded wait since the last call,
 * FP8_ERR_CUDA if the stream reports an error, else FP8_OK. */
fp8_status fp8_sync_status(void *stream);

/* Diagnostic, not part of the method: launches one warp that waits with the
 * library's bounded wait on a barrier nothing ever signals, so the wait runs
 * out after limit_ns (1 .. 5e9) and the kernel records it in the device
 * error flag and returns -- the path every kernel takes when a wait runs out.
 * The next fp8_sync_status on the stream then returns FP8_ERR_TIMEOUT (and
 * clears the flag); the context stays usable. */
fp8_status fp8_selftest_wait_timeout(int64_t limit_ns, void *stream);

/* Diagnostic, not part of the method: a clock probe for measuring the SM
 * clock the GEMMs actually run at.  While acc is not NULL, the first CTA of
 * every GEMM launch (fp8_gemm_tn, fp8_gemm_tn_grouped and the GEMMs inside
 * the layer calls) adds the SM clock cycles (%clock64) and the nanoseconds
 * (%globaltimer) between its start and its end to acc[0] and acc[1] (atomic
 * adds); acc[0] / acc[1] is then the average SM clock during those launches
 * in GHz.  The kernels persist over all tiles, so that CTA lives as long as
 * the launch.  acc: DEVICE, 2 uint64, 8-byte aligned, caller-owned and
 * zeroed by the caller; NULL (the default) turns the probe off.  The
 * setting is process-wide and is read when a launch is enqueued (a CUDA
 * graph keeps the value it was captured with). */
fp8_status fp8_set_clock_probe(uint64_t *acc);

/* amax of a BF16 tensor (the implementation guide's range monitoring; the
 * TensorRT page's Absolute-Max statistic).
 *   x     DEVICE, n BF16 values (n >= 0, multiple of 16; n == 0 gives 0)
 *   amax  DEVICE, 1 float, overwritten with max |x_i| (NaN skipped). */
fp8_status fp8_amax(const void *x, int64_t n, float *amax, void *stream);

/* Fused scaled cast BF16 -> FP8 with transposed copy and amax (the Q node of
 * the TensorRT page; formats of the implementation guide / wiki table).
 *   x      DEVICE, [rows][cols] BF16
 *   scale  DEVICE, 1 float, read on the device
 *   fmt    FP8_E4M3 or FP8_E5M2
 *   out    DEVICE, [rows][cols] FP8 codes, or NULL
 *   out_t  DEVICE, [cols][rows] FP8 codes (the transpose of out), or NULL
 *   amax   DEVICE, 1 float overwritten with amax(x), or NULL
 * rows, cols >= 0 and multiples of 16.  At least one of out / out_t unless
 * the tensor is empty (then only the amax, 0, is written). */
fp8_status fp8_quantize_transpose(const void *x, int64_t rows, int64_t cols, const float *scale,
                                  int32_t fmt, uint8_t *out, uint8_t *out_t, float *amax,
                                  void *stream);

/* Scaled cast of an fp32 tensor to FP8 (the Q node of the TensorRT page on
 * fp32 values, such as the fp32 quantities that FP8-LM stores in FP8, wiki
 * note "extension to FP8"): q_i = satRNE_fmt(fl32(x_i * scale)) in element
 * order, with the same rounding, saturation and NaN rules as the BF16 cast.
 *   x      DEVICE, n fp32 values, 16-byte aligned (n >= 0, multiple of 16)
 *   scale  DEVICE, 1 float, read on the device
 *   fmt    FP8_E4M3 or FP8_E5M2
 *   out    DEVICE, n FP8 codes, 16-byte aligned (may be NULL when n == 0)
 *   amax   DEVICE, 1 float overwritten with max |x_i| (NaN skipped), or NULL */
fp8_status fp8_quantize_f32(const float *x, int64_t n, const float *scale, int32_t fmt,
                            uint8_t *out, float *amax, void *stream);

/* Just-in-time (current) scaling of one tensor (wiki note, "per-tensor
 * scaling is the key": the scale comes from the tensor itself): amax(x),
 * then scale = the recipe formula applied to that amax alone, then the fused
 * cast with that scale.  Two kernels, in stream order.
 *   x, rows, cols, fmt, out, out_t  as fp8_quantize_transpose
 *   margin     0 <= margin <= 64
 *   amax       DEVICE, 1 float, overwritten with amax(x)
 *   scale, scale_inv  DEVICE, 1 float each: replaced by the new scale and
 *              its inverse when 0 < amax < inf, left as they are otherwise
 *              (the cast then uses the given scale). */
fp8_status fp8_quantize_transpose_current(const void *x, int64_t rows, int64_t cols, int32_t fmt,
                                          int32_t margin, uint8_t *out, uint8_t *out_t,
                                          float *amax, float *scale, float *scale_inv,
                                          void *stream);

/* Delayed-scaling update of `num_tensors` independent scaling states (the
 * recipe section's margin and amax_history_len, with the scale formula in
 * the header comment).  All DEVICE:
 *   history    [num_tensors][history_len], shifted in place, [t][0] newest
 *   amax       [num_tensors], the value pushed into each history (read only)
 *   scale, scale_inv [num_tensors], updated in place
 * format_mask: bit t set = tensor t is E5M2 (fmax 57344), clear = E4M3 (448).
 * 1 <= num_tensors <= 32, 1 <= history_len <= 8192, 0 <= margin <= 64. */
fp8_status fp8_scale_update(float *history, const float *amax, float *scale, float *scale_inv,
                            int32_t num_tensors, int32_t history_len, uint32_t format_mask,
                            int32_t margin, void *stream);

/* The recipe's update of all five slots of one layer, run once per step
 * after fp8_linear_fwd and fp8_linear_bwd: fp8_scale_update over meta with
 * the recipe's formats (HYBRID: slots dY and dX are E5M2), after which the
 * five amax slots are cleared to 0 for the next step.
 * meta->history_len must equal recipe->history_len. */
fp8_status fp8_amax_scale_update(const fp8_meta *meta, const fp8_recipe *recipe, void *stream);

/* FP8 GEMM with both operands contiguous along K ("TN"), fp32 accumulation
 * in TMEM on the tcgen05 tensor cores, and the dequant epilogue (wiki note,
 * "extension to FP8"; the DQ node of the TensorRT page).
 *   A  DEVICE [M][K] FP8 codes of format fa;  B  DEVICE [N][K] of format fb
 *   a_scale_inv, b_scale_inv  DEVICE, 1 float each
 *   D  DEVICE [M][N] BF16 output
 *   d_amax  DEVICE, 1 float overwritten with max |D|, or NULL
 * M, N, K >= 16 and multiples of 16. */
fp8_status fp8_gemm_tn(const uint8_t *A, int32_t fa, const uint8_t *B, int32_t fb, int64_t M,
                       int64_t N, int64_t K, const float *a_scale_inv, const float *b_scale_inv,
                       void *D, float *d_amax, void *stream);

/* One GEMM of fp8_gemm_tn_grouped; fields as the arguments of fp8_gemm_tn. */
typedef struct {
    const uint8_t *A;
    int32_t fa;
    const uint8_t *B;
    int32_t fb;
    int64_t M, N, K;
    const float *a_scale_inv;
    const float *b_scale_inv;
    void *D;
    float *d_amax;
} fp8_gemm_desc;

/* One or two independent fp8_gemm_tn problems in a single persistent launch
 * (helper; the backward pass runs dgrad and wgrad this way): the tiles of
 * both form one list, so one GEMM's last partial wave is filled with the
 * other's tiles.  n is 1 or 2; each problem is checked as by fp8_gemm_tn,
 * and each d_amax (when not NULL) is overwritten with its own output amax. */
fp8_status fp8_gemm_tn_grouped(const fp8_gemm_desc *descs, int32_t n, void *stream);

/* One tensor of fp8_quantize_transpose_grouped; fields as the arguments of
 * fp8_quantize_transpose. */
typedef struct {
    const void *x;
    int64_t rows, cols;
    const float *scale;
    uint8_t *out;
    uint8_t *out_t;
    float *amax;
} fp8_cast_desc;

/* One or two fp8_quantize_transpose casts of the same format in a single
 * persistent launch (helper; the forward pass casts X and W this way).  Each
 * tensor is checked as by fp8_quantize_transpose; each amax (when not NULL)
 * is overwritten with its own tensor's amax. */
fp8_status fp8_quantize_transpose_grouped(const fp8_cast_desc *descs, int32_t n, int32_t fmt,
                                          void *stream);

/* LayerNorm fused with the scaled cast (te.LayerNorm in front of an FP8
 * linear; implementation guide, "Basic structure of FP8 training code"):
 *   mean[r] = sum_c x[r][c] / C,  var[r] = sum_c (x[r][c] - mean[r])^2 / C,
 *   rstd[r] = 1 / sqrt(var[r] + eps),
 *   y[r][c] = ((x[r][c] - mean[r]) * rstd[r]) * gamma[c] + beta[c]   (fp32),
 * then the cast of y exactly as fp8_quantize_transpose casts x (y is never
 * written out in BF16).  Rows of at most 4096 columns with out given: one
 * kernel computes the statistics and the row-major codes from one read of x,
 * and out_t (if given) is the byte transpose of those codes.  Otherwise two
 * kernels: row statistics, then LayerNorm + cast.  Both compute the same
 * statistics bit for bit.
 *   x      DEVICE [rows][cols] BF16;  gamma, beta  DEVICE [cols] BF16
 *   eps    >= 0;  scale  DEVICE, 1 float;  fmt, out, out_t as fp8_quantize_transpose
 *   amax   DEVICE, 1 float overwritten with max |y| (fp32 y, NaN skipped), or NULL
 *   mean, rstd  DEVICE [rows] fp32 outputs (kept for the LayerNorm backward)
 * rows, cols multiples of 16, cols >= 16.  Sums run in fp32 in a different
 * order from a sequential sum, so y matches an exact evaluation to about
 * 1e-6 relative, not bit for bit. */
fp8_status fp8_layernorm_quantize_transpose(const void *x, const void *gamma, const void *beta,
                                            int64_t rows, int64_t cols, float eps,
                                            const float *scale, int32_t fmt, uint8_t *out,
                                            uint8_t *out_t, float *amax, float *mean, float *rstd,
                                            void *stream);

/* LayerNorm row statistics alone (te.LayerNormLinear's LayerNorm; the same
 * page and section as fp8_layernorm_quantize_transpose): mean[r] and rstd[r]
 * exactly as that call computes them (bit for bit), which the LayerNorm
 * backward keeps, and, if amax is given, max |y| over y = LN(x) as defined
 * there: the amax that just-in-time scaling needs before any code is written.
 *   x      DEVICE [rows][cols] BF16
 *   gamma, beta  DEVICE [cols] BF16, read only when amax is given (else may be NULL)
 *   eps    >= 0
 *   mean, rstd  DEVICE [rows] fp32 outputs
 *   amax   DEVICE, 1 float overwritten with max |y| (fp32 y, NaN skipped; 0 for
 *          no rows), or NULL
 * rows, cols multiples of 16, cols >= 16; x, gamma, beta 16-byte aligned.
 * Rows of at most 4096 columns are held in registers (one HBM read of x);
 * wider rows are staged in shared memory or, past 8192 columns, read twice. */
fp8_status fp8_layernorm_stats(const void *x, const void *gamma, const void *beta, int64_t rows,
                               int64_t cols, float eps, float *mean, float *rstd, float *amax,
                               void *stream);

/* Forward of LayerNorm + FP8 linear (te.LayerNormLinear): Y = LN(X) W^T with
 * LN(X) cast to E4M3 as fp8_layernorm_quantize_transpose casts it (its amax
 * is slot X's; under delayed scaling X8t is the byte transpose of X8), W cast
 * as in fp8_linear_fwd, then fprop.  Arguments as fp8_linear_fwd plus gamma,
 * beta [K] (BF16), eps, and mean, rstd [M] (fp32 outputs).  X8 / X8t hold the
 * FP8 LayerNorm output, so fp8_linear_bwd follows unchanged. */
fp8_status fp8_layernorm_linear_fwd(const void *X, const void *gamma, const void *beta, float eps,
                                    const void *W, int64_t M, int64_t N, int64_t K,
                                    const fp8_meta *meta, const fp8_recipe *recipe, uint8_t *X8,
                                    uint8_t *X8t, uint8_t *W8, uint8_t *W8t, void *Y, float *mean,
                                    float *rstd, void *stream);

/* Forward of the FP8 linear layer Y = X W^T (te.Linear under fp8_autocast,
 * implementation guide "Basic structure of FP8 training code" and the
 * recipe section).  Uses this step's (delayed) scales of X and W, or under
 * FP8_SCALING_CURRENT derives them from X's and W's own amax first.
 *   X   DEVICE [M][K] BF16 input;   W  DEVICE [N][K] BF16 weight
 *   X8, X8t  DEVICE [M][K] and [K][M] FP8 (E4M3), written; X8t is kept for wgrad
 *   W8, W8t  DEVICE [N][K] and [K][N] FP8 (E4M3), written; W8t is kept for dgrad
 *   Y   DEVICE [M][N] BF16 output
 * Max-combines the amax of X, W and Y into meta->amax[X], [W], [Y]: the
 * slots hold the running max since the last fp8_amax_scale_update, which
 * clears them (a fresh meta has them at 0), so several forward calls before
 * one update (micro-batches) record the max over all of them.  Under
 * FP8_SCALING_CURRENT the X and W slots are overwritten with this call's
 * amax instead. */
fp8_status fp8_linear_fwd(const void *X, const void *W, int64_t M, int64_t N, int64_t K,
                          const fp8_meta *meta, const fp8_recipe *recipe, uint8_t *X8,
                          uint8_t *X8t, uint8_t *W8, uint8_t *W8t, void *Y, void *stream);

/* Backward of the FP8 linear layer: dX = dY W (dgrad), dW = dY^T X (wgrad),
 * with dY cast to E5M2 under HYBRID (E4M3 otherwise); under
 * FP8_SCALING_CURRENT dY's scale is derived from its own amax first.
 *   dY  DEVICE [M][N] BF16 output gradient
 *   X8t, W8t  DEVICE, the transposed copies written by fp8_linear_fwd
 *   dY8, dY8t DEVICE [M][N] and [N][M] FP8 work buffers, written
 *   dX  DEVICE [M][K] BF16;  dW  DEVICE [N][K] BF16
 * Max-combines the amax of dY and dX into meta->amax[dY], [dX] (as
 * fp8_linear_fwd does for its slots; under FP8_SCALING_CURRENT the dY slot is
 * overwritten with this call's amax). */
fp8_status fp8_linear_bwd(const void *dY, int64_t M, int64_t N, int64_t K, const fp8_meta *meta,
                          const fp8_recipe *recipe, const uint8_t *X8t, const uint8_t *W8t,
                          uint8_t *dY8, uint8_t *dY8t, void *dX, void *dW, void *stream);

/* Hyper-parameters of one Adam step (AdamW's decoupled weight decay).  The
 * bias corrections 1 - beta1^t and 1 - beta2^t are computed by the caller
 * for step t (>= 1) and passed as binary32. */
typedef struct {
    float lr, beta1, beta2, eps, weight_decay;
    float bias_correction1, bias_correction2;
    int32_t margin;   /* for the state scales, 0..64 */
} fp8_adam_hyper;

/* One Adam step on optimizer states of decoupled precision (wiki note,
 * bullet "precision decoupling": first moment FP8, second moment FP16,
 * master weights FP16 with tensor scaling: 5 bytes of state per parameter;
 * the note's 6 also counts an FP8 gradient, which this path keeps BF16).  In
 * binary32, one rounding per operation, for every element (Adam's textbook
 * bias correction m / (1 - b1^t), v / (1 - b2^t); AdamW's decoupled decay):
 *   m = b1*m + (1-b1)*g;  v = b2*v + (1-b2)*(g*g);
 *   u = (m / bc1) / (sqrt(v / bc2) + eps);  w = w - lr*(u + wd*w)
 * with m = E4M3 code * m1_scale_inv and w = FP16 code * w_scale_inv.  The new
 * states take just-in-time per-tensor scales: scale = (fmax / amax) /
 * 2^margin of the new values (fmax 448 for m, 65504 for w), kept when that
 * amax is 0 or not finite.  FP16 encodes round to nearest even and saturate
 * at +-65504.  Four kernels, in stream order.
 *   grad        DEVICE [n] BF16 gradient
 *   m1          DEVICE [n] E4M3 codes, updated in place
 *   m1_scale, m1_scale_inv   DEVICE 1 float each, updated
 *   m2          DEVICE [n] FP16 second moment, updated in place
 *   w16         DEVICE [n] FP16 master-weight codes, updated in place
 *   w_scale, w_scale_inv     DEVICE 1 float each, updated
 *   w_bf16      DEVICE [n] BF16 output: the weights for the next forward
 *   amax        DEVICE [2] output: amax of the new m and w (fp32)
 * n >= 0, a multiple of 16; arrays 16-byte aligned. */
fp8_status fp8_adam_step(const void *grad, int64_t n, uint8_t *m1, float *m1_scale,
                         float *m1_scale_inv, uint16_t *m2, uint16_t *w16, float *w_scale,
                         float *w_scale_inv, void *w_bf16, float *amax, const fp8_adam_hyper *hp,
                         void *stream);

/* Initial state for fp8_adam_step of one BF16 weight tensor (same bullet):
 * zero moments with first-moment scale and inverse 1, and the master weights
 * in FP16 under the just-in-time scale of w itself -- the recipe formula on
 * amax(w) alone with FP16's largest finite value:
 *   s_w = fl32(fl32(65504 / amax(w)) * 2^-margin)  (FLT_MAX if it overflows;
 *         1 when amax(w) is 0 or not finite),  w_scale_inv = fl32(1 / s_w),
 *   w16[i] = FP16 code of fl32(w[i] * s_w), nearest even, saturating.
 *   w       DEVICE [n] BF16 weights (read)
 *   margin  0..64
 *   m1 [n] E4M3 codes, m2 [n] FP16, w16 [n] FP16: DEVICE outputs
 *   m1_scale, m1_scale_inv, w_scale, w_scale_inv: DEVICE, 1 float each, written
 *   amax    DEVICE [2] output: {0, amax(w)}
 * n >= 0, a multiple of 16; arrays 16-byte aligned.  Three kernels (after a
 * one-word memset), in stream order. */
fp8_status fp8_adam_init(const void *w, int64_t n, int32_t margin, uint8_t *m1, float *m1_scale,
                         float *m1_scale_inv, uint16_t *m2, uint16_t *w16, float *w_scale,
                         float *w_scale_inv, float *amax, void *stream);

/* The summing half of an FP8 all-reduce with one shared scale (wiki note,
 * bullet "per-tensor scaling is the key": every rank casts with the one
 * scalar s'_g = min(s'_1, ..., s'_N), so the exchanged FP8 codes of all ranks
 * can be summed directly).  After this rank's shard of every rank's codes
 * has been exchanged:
 *   out[i] = bf16_rne( sum_r dec(parts[r][i]) * fl32(1 / scale) )
 * with the sum and the product exact, rounded once to BF16 (nearest, ties to
 * even; overflow to +-inf; gradual underflow, a nonzero result that rounds
 * to zero keeps its sign; an exact zero is +0).  Special codes follow IEEE
 * arithmetic: a NaN code, or +inf and -inf together, give NaN; one kind of
 * infinity gives that infinity times fl32(1 / scale) (NaN when that factor
 * is 0 or NaN).  The result does not depend on the order of the ranks.
 *   parts   DEVICE [nranks][n] FP8 codes of format fmt, 16-byte aligned
 *   scale   DEVICE, 1 float: the shared scale the parts were cast with
 *   out     DEVICE [n] BF16 output
 * 1 <= nranks <= 65536; n >= 0, a multiple of 16.  One kernel; it uses 96 KB
 * of shared memory per block and no global scratch memory. */
fp8_status fp8_dequant_sum(const uint8_t *parts, int32_t nranks, int64_t n, int32_t fmt,
                           const float *scale, void *out, void *stream);

/* fp8_linear_bwd for callers that cannot allocate device memory.  The pages
 * have no counterpart: this is a calling convenience, not part of the method.
 * It computes exactly what fp8_linear_bwd computes, but the two FP8 work
 * buffers (dY8, dY8t) are not passed in: they live in a fixed array in the
 * library's own device memory (64 MiB on every GPU that loads the library,
 * held until the process exits).  Callers that need it: a plugin handed only
 * its input and output tensors by a framework whose allocator owns the device
 * memory, or code that must not call cudaMalloc / cudaFree (cudaFree waits
 * for the whole device).
 *   Arguments as fp8_linear_bwd, without dY8 / dY8t.
 *   Limit: M * N <= 2^25 (33,554,432) elements; larger sizes return
 *   FP8_ERR_ARG ("exceeds the fixed work area") and nothing is enqueued.
 *   Other argument errors are those of fp8_linear_bwd.
 *   Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 *   Set-up: the first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.  The address belongs to the device's primary
 *   context: after cudaDeviceReset on a device, do not call this function on
 *   that device again in the same process.
 *   All calls share the one array: calls that overlap on the GPU (on
 *   different streams, or from different threads without ordering) race on
 *   it; calls ordered on one stream do not.  Every call overwrites the part it
 *   uses before reading it, so it never depends on what a previous call left
 *   there. */
fp8_status fp8_linear_bwd_noalloc(const void *dY, int64_t M, int64_t N, int64_t K,
                                  const fp8_meta *meta, const fp8_recipe *recipe,
                                  const uint8_t *X8t, const uint8_t *W8t, void *dX, void *dW,
                                  void *stream);

/* ------------------------------------------------------------------------
 * Block scaling: one scale for each block of 128
 *
 * Beside the per-tensor scales above, a tensor can carry one scale for each
 * 128 consecutive columns of a row (block_rows = 1: activations, gradients)
 * or for each 128 x 128 tile (block_rows = 128: weights).  An element stands
 * for code * scale of its block.  Blocks start at row 0 and column 0; the last
 * ones may be partly filled.  The quantizers choose powers of two, so that
 * dividing by a scale is exact and the only rounding is the code's own:
 *   amax  = the largest finite magnitude in the block
 *   scale = 2^e, e the smallest integer >= -127 with amax <= fmax * 2^e
 *           (fmax 448 or 57344), so the smallest scale for a block of zeros
 *   code  = x / scale rounded to nearest, ties to the even code; infinities
 *           saturate to +-fmax, NaN stays NaN, the sign of zero is kept.
 * Sizes are free (odd ones too; 0 rows or columns: nothing is done).
 * Everything is dense along the columns; `ld` is the distance between rows
 * in elements.  Rows, columns and strides are below 2^31. */

typedef enum { FP8_DTYPE_F32 = 0, FP8_DTYPE_BF16 = 1, FP8_DTYPE_F16 = 2 } fp8_dtype;

/* How a block's scale is stored: FP8_SCALE_E8M0, a byte b for 2^(b - 127)
 * (255: NaN), or FP8_SCALE_F32, the factor itself, any float. */
typedef enum { FP8_SCALE_E8M0 = 0, FP8_SCALE_F32 = 1 } fp8_scale_type;

/* A matrix in 32 or 16 bits: DEVICE data [rows][ld], ld >= cols, aligned to
 * its element.  16-byte aligned rows (data, and ld * element size) are faster. */
typedef struct {
    void *data;
    int64_t rows, cols, ld;
    int32_t dtype;
} fp8_matrix;

/* A block-scaled FP8 matrix, all DEVICE memory of the caller's:
 *   codes  [rows][ld] FP8 codes of format fmt; 16-byte aligned, ld >= cols a
 *          multiple of 16.  Columns from cols on are neither read as values
 *          nor written.
 *   scales [ceil(rows / block_rows)][ld_scales]; column j holds the scale of
 *          columns 128 j .. 128 j + 127; ld_scales >= ceil(cols / 128), for
 *          E8M0 a multiple of 4; 4-byte aligned. */
typedef struct {
    uint8_t *codes;
    int64_t rows, cols, ld;
    void *scales;
    int64_t ld_scales;
    int32_t fmt;
    int32_t block_rows;
    int32_t scale_type;
} fp8_block_tensor;

/* Quantizes x [rows][cols] into q and / or its transpose into qt [cols][rows]
 * (either may be NULL, not both).  q and qt have the same format, block_rows
 * and scale type.  With block_rows = 1, q's blocks run along x's rows and
 * qt's along its columns, the operands of products that sum over columns and
 * over rows; with 128 both hold the same tiles.  One kernel. */
fp8_status fp8_block_quantize(const fp8_matrix *x, const fp8_block_tensor *q,
                              const fp8_block_tensor *qt, void *stream);

/* out [rows][cols] = code * scale, rounded to out's type.  One kernel. */
fp8_status fp8_block_dequantize(const fp8_block_tensor *q, const fp8_matrix *out, void *stream);

/* D [M][N] (BF16) = A [M][K] . B [N][K]^T of two block-scaled matrices:
 *   D[i][j] = bf16_rne( sum over blocks k of sA(i, k) * sB(j, k) * dot_k ),
 *   dot_k = sum over the block's 128 columns of a[i][c] * b[j][c],
 * with the products summed in fp32.  A and B each E4M3 or E5M2, each with
 * block_rows 1 or 128, both with one scale type; a product sA * sB has to be
 * a normal fp32 number or zero.  M, N, K >= 0; K = 0 gives zeros. */
fp8_status fp8_block_gemm_tn(const fp8_block_tensor *A, const fp8_block_tensor *B,
                             const fp8_matrix *D, void *stream);

/* LayerNorm of x [rows][cols], in fp32:
 *   mean = sum x / cols, rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
 *   y = ((x - mean) * rstd) * gamma + beta.
 * Writes mean and rstd (fp32 [rows]) and any of: y (of x's type); y8, y block
 * quantized straight from fp32 (block_rows 1), the operand of a following
 * product; x8, x itself in 8 bits (block_rows 1), which
 * fp8_layernorm_bwd and fp8_layernorm_recompute take in x's place, so that
 * neither x nor y has to be kept until the backward pass.  gamma and beta
 * [cols] are of type wtype (fp8_dtype).  cols >= 1. */
fp8_status fp8_layernorm_fwd(const fp8_matrix *x, const void *gamma, const void *beta,
                             int32_t wtype, float eps, const fp8_matrix *y,
                             const fp8_block_tensor *y8, const fp8_block_tensor *x8, float *mean,
                             float *rstd, void *stream);

/* Backward of LayerNorm from dy [rows][cols] and the forward's input, either
 * x or its 8-bit copy x8 (the other NULL), with the forward's mean and rstd:
 *   xhat = (x - mean) * rstd,  u = dy * gamma,
 *   dx = rstd * (u - sum(u) / cols - xhat * sum(u * xhat) / cols)  (per row),
 *   dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy.
 * dy, x and dx are of one type; dgamma and dbeta are fp32 [cols], overwritten;
 * dx may be dy.  workspace: DEVICE, 16-byte aligned, of at least
 * fp8_layernorm_bwd_workspace(rows, cols) bytes, in use until the call's
 * kernels are done.  The sums' order is fixed: equal calls give equal bits. */
fp8_status fp8_layernorm_bwd(const fp8_matrix *dy, const fp8_matrix *x,
                             const fp8_block_tensor *x8, const void *gamma, int32_t wtype,
                             const float *mean, const float *rstd, const fp8_matrix *dx,
                             float *dgamma, float *dbeta, void *workspace, int64_t workspace_bytes,
                             void *stream);
int64_t fp8_layernorm_bwd_workspace(int64_t rows, int64_t cols);

/* LayerNorm's output again from the 8-bit copy of its input, transposed:
 * yt [cols][rows] (block_rows 1: blocks along the tokens), the operand of the
 * weight gradient of the product that follows the LayerNorm. */
fp8_status fp8_layernorm_recompute(const fp8_block_tensor *x8, const void *gamma,
                                   const void *beta, int32_t wtype, const float *mean,
                                   const float *rstd, const fp8_block_tensor *yt, void *stream);

/* Root-mean-square norm with the residual's addition, x [rows][cols], in fp32:
 *   s = x + residual, rounded to x's type (residual NULL: s = x),
 *   rstd = 1 / sqrt(sum s^2 / cols + eps),  y = (s * rstd) * gamma.
 * The norm is taken of s as it is stored.  Writes rstd (fp32 [rows]) and any of:
 * sum, s itself (with a residual only); y (both of x's type); y8, y block
 * quantized straight from fp32 (block_rows 1), the operand of a following product;
 * x8, s in 8 bits (block_rows 1), which fp8_rmsnorm_bwd and
 * fp8_rmsnorm_recompute take in s's place.  residual is of x's type; sum and y may
 * each be x's or the residual's own memory (same address and stride).  Outputs that
 * overlap each other, or an input in any other way, are refused (FP8_ERR_ARG), as in
 * the two calls below; rows may lie between another matrix's.  gamma [cols] is of
 * type wtype (fp8_dtype).  cols >= 1. */
fp8_status fp8_rmsnorm_fwd(const fp8_matrix *x, const fp8_matrix *residual, const void *gamma,
                           int32_t wtype, float eps, const fp8_matrix *sum, const fp8_matrix *y,
                           const fp8_block_tensor *y8, const fp8_block_tensor *x8, float *rstd,
                           void *stream);

/* Backward of fp8_rmsnorm_fwd from dy [rows][cols] and s, either x (the forward's
 * sum) or its 8-bit copy x8 (the other NULL), with the forward's rstd:
 *   xhat = s * rstd,  u = dy * gamma,
 *   dx = dsum + rstd * (u - xhat * sum(u * xhat) / cols)   (per row),
 *   dgamma = sum over rows of dy * xhat.
 * dsum: the gradient that reaches s by the residual's way (NULL: none).  dx is the
 * gradient of x and of the residual alike.  dy, x, dsum and dx are of one type;
 * dgamma is fp32 [cols], overwritten; dx may be dy, dsum or x (same address and
 * stride).  workspace: DEVICE, 16-byte aligned, of at least
 * fp8_rmsnorm_bwd_workspace(rows, cols) bytes, in use until the call's kernels
 * are done.  The sums' order is fixed: equal calls give equal bits. */
fp8_status fp8_rmsnorm_bwd(const fp8_matrix *dy, const fp8_matrix *x, const fp8_block_tensor *x8,
                           const void *gamma, int32_t wtype, const float *rstd,
                           const fp8_matrix *dsum, const fp8_matrix *dx, float *dgamma,
                           void *workspace, int64_t workspace_bytes, void *stream);
int64_t fp8_rmsnorm_bwd_workspace(int64_t rows, int64_t cols);

/* The RMS norm's output again from the 8-bit copy of s, transposed: yt
 * [cols][rows] (block_rows 1: blocks along the tokens), the operand of the weight
 * gradient of the product that follows the norm. */
fp8_status fp8_rmsnorm_recompute(const fp8_block_tensor *x8, const void *gamma, int32_t wtype,
                                 const float *rstd, const fp8_block_tensor *yt, void *stream);

/* SwiGLU of h [M][2F] = [gate | value]: a = gate / (1 + exp(-gate)) * value in
 * fp32, block quantized into a8 [M][F] (block_rows 1).  h8 (or NULL): h itself
 * in 8 bits [M][2F], for fp8_swiglu_bwd.  F a multiple of 128, so that no
 * block of h holds columns of both halves.  One kernel. */
fp8_status fp8_swiglu_fwd(const fp8_matrix *h, const fp8_block_tensor *a8,
                          const fp8_block_tensor *h8, void *stream);

/* Backward of SwiGLU from da [M][F] and the 8-bit h8 [M][2F].  With
 * s = 1 / (1 + exp(-gate)), in fp32:
 *   d gate = da * value * s * (1 + gate * (1 - s)),  d value = da * (gate * s)
 * block quantized into dh8 [M][2F] and dh8t [2F][M], the operands of the input
 * gradient's and the weight gradient's product, and the forward's output
 * again, gate * s * value, into a8t [F][M], the operand of the next layer's
 * weight gradient.  All block_rows 1; any of the three may be NULL, not all;
 * dh8 and dh8t have the same format.  One kernel. */
fp8_status fp8_swiglu_bwd(const fp8_matrix *da, const fp8_block_tensor *h8,
                          const fp8_block_tensor *dh8, const fp8_block_tensor *dh8t,
                          const fp8_block_tensor *a8t, void *stream);

/* The gated feed-forward product: both projections, SiLU and the product in one
 * kernel, and nothing of it in 16 bits on the way.  A [M][K] and B [2F][K] = [gate
 * rows | value rows], both with E8M0 scales, E4M3 or E5M2, block_rows 1 or 128:
 *   [g | u] = A . B^T as fp8_block_gemm_tn sums it, in fp32,
 *   a = g / (1 + exp(-g)) * u,
 * a block quantized into a8 [M][F], and [g | u] into h8 [M][2F] (or NULL) for
 * fp8_block_gemm_swiglu_bwd, both straight from fp32 (block_rows 1).  F a multiple
 * of 128, K >= 1, M >= 0.  What is written overlaps nothing else (FP8_ERR_ARG where
 * it does; rows may lie between another tensor's).  fp8_block_gemm_tn and fp8_swiglu_fwd do the same in two steps
 * with h in between, which serves float scales and one wanting h. */
fp8_status fp8_block_gemm_swiglu_fwd(const fp8_block_tensor *A, const fp8_block_tensor *B,
                                     const fp8_block_tensor *a8, const fp8_block_tensor *h8,
                                     void *stream);

/* Its backward: A = dy [M][K] and B [F][K] (the transpose of the matrix that takes
 * a back to the output), scales as above, and h8 [M][2F] = [g | u]:
 *   da = A . B^T in fp32,  s = 1 / (1 + exp(-g)),
 *   d g = da * u * s * (1 + g * (1 - s)),  d u = da * (g * s)
 * block quantized into dh8 [M][2F] and dh8t [2F][M], and a again, g * s * u, into
 * a8t [F][M]: what fp8_swiglu_bwd writes, from the product itself, in one kernel.
 * The outputs' block_rows and h8's are 1; any of the three may be NULL, not all; dh8
 * and dh8t have the same format.  dh8 may be h8's own memory (same addresses and
 * strides); otherwise what is written overlaps nothing else, as above. */
fp8_status fp8_block_gemm_swiglu_bwd(const fp8_block_tensor *A, const fp8_block_tensor *B,
                                     const fp8_block_tensor *h8, const fp8_block_tensor *dh8,
                                     const fp8_block_tensor *dh8t, const fp8_block_tensor *a8t,
                                     void *stream);

/* ------------------------------------------------------------------------
 * The norm of many gradients together, and clipping by it */

/* n consecutive elements of type dtype (fp8_dtype), DEVICE, aligned to the element
 * (16-byte aligned ones are faster); 0 <= n <= 2^40, and 2^44 in a list. */
typedef struct {
    void *data;
    int64_t n;
    int32_t dtype;
} fp8_vector;

/* norm[0] (DEVICE, fp32) = sqrt(sum over the vectors of the sum of their squares),
 * of any size: squares are summed in 32 bits with the additions' rounding errors
 * kept, or in 64 bits where they could leave 32 bits' range, and the sums are joined
 * in 64 bits.  A NaN or an infinity among the elements gives NaN or infinity, no
 * elements 0.  grads: HOST array of count vectors (count >= 0), read before the call
 * returns.  workspace: DEVICE, 8-byte aligned, of at least
 * fp8_grad_norm_workspace(count) bytes, in use until the call's kernels are done;
 * it overlaps neither norm nor a vector (FP8_ERR_ARG).
 * The sums' order is fixed: equal calls give equal bits.  One kernel for each 1000
 * vectors, and one that joins their sums; for few elements one alone. */
fp8_status fp8_grad_norm(const fp8_vector *grads, int32_t count, float *norm, void *workspace,
                         int64_t workspace_bytes, void *stream);
int64_t fp8_grad_norm_workspace(int32_t count);

/* outs[i] = grads[i] * c in fp32, rounded to the type of outs[i], with the norm
 * read on the device:
 *   c = max_norm / norm  where max_norm < norm < infinity, else 1,
 * so that gradients whose norm is not finite pass through as they are (the caller
 * sees it by the norm, and skips the step).  outs (NULL: grads, in place): HOST
 * array of count vectors of the grads' lengths; outs[i] may be grads[i] (same
 * address and type), and overlaps no other vector and not norm (FP8_ERR_ARG where
 * it does: a gradient is twice in the list).  max_norm >= 0.  One kernel for each 1000
 * vectors. */
fp8_status fp8_grad_clip(const fp8_vector *grads, const fp8_vector *outs, int32_t count,
                         const float *norm, float max_norm, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8AMAX_H */
