/*
 * qmx.h -- C ABI of libqmx.so: the steps of an MoE layer around the expert
 * products of qmv.h, on AMD Instinct MI355X (gfx950).
 *
 *   qmx_rmsnorm     residual addition and root-mean-square norm, written as
 *                   bf16 or directly in an activation format of the products
 *   qmx_router      a token's top_k experts and their weights: the
 *                   expert_ids and route_weights that the gathers read
 *   qmx_quantize    values -> MXFP4 or int8 blocks (activations or weights)
 *   qmx_dequantize  MXFP4 or int8 blocks -> values
 *
 * ------------------------------------------------------------------ formats
 * Blocks are 32 consecutive values of a row; codes and scales are separate
 * arrays in the layouts of qmv.h.
 *
 *   QMX_MXFP4  codes uint8 [rows][K/2] (two e2m1 nibbles per byte, the even
 *              value in the low nibble), scales uint8 [rows][K/32] (E8M0).
 *              Per block of finite values, with amax = max |v|:
 *                b     = exponent byte of (amax + a quarter of its own power
 *                        of two), that is floor(log2 amax) + 127, one more
 *                        where amax is 1.75 powers of two or above,
 *                byte  = max(b - 2, 0), the scale 2^(byte - 127),
 *                code  = v / 2^(byte - 127) rounded to the nearest e2m1
 *                        value, ties to the even code; v's sign is kept.
 *              b counts amax as rounded to e2m1's two significant bits
 *              (e2m1's largest value is 6 = 1.5 * 2^2), so no value is
 *              clamped by more than half a step of the grid.
 *              A block that holds a NaN or an infinity gets scale byte 255
 *              (NaN) and codes 0.
 *   QMX_Q8B32  codes int8 [rows][K], scales fp16 [rows][K/32]: the block
 *              quantizer of qmv.h (QMV_A_BF16_Q8) in fp32:
 *                d16 = fp16(amax / 127), code = clamp(rint(v * (1 / d16)),
 *                -127, 127), 0 where d16 is 0 or infinite.
 *              A block that holds a NaN or an infinity gets scale NaN and
 *              codes 0.
 *   QMX_BF16   bf16 [rows][K], no scales (the norm's output only).
 *
 * -------------------------------------------------------------- conventions
 * As in qmv.h: every pointer is a device pointer owned by the caller, arrays
 * are dense row-major, a call only enqueues one launch on `stream` (one per
 * 2^20 rows of the norm, per 2^22 tokens of the router), takes no memory of
 * its own and reads and writes only the extents given here.  The
 * stream's device must be the current one.  Arguments are checked on the
 * host before the launch.  Results are bitwise identical from run to run
 * (fixed reduction order, no atomics).
 *
 * Alignment: x, residual, residual_out, weight, y and codes 16 bytes when
 * K % 8 == 0; with another K (QMX_BF16 output only) each array's own element
 * size.  logits, ids, weights and scales: their element size.
 */
#ifndef QMX_H
#define QMX_H

#include "qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { QMX_T_F32 = 0, QMX_T_BF16 = 1, QMX_T_F16 = 2 } qmx_type_t;
typedef enum { QMX_BF16 = 0, QMX_Q8B32 = 1, QMX_MXFP4 = 2 } qmx_fmt_t;
typedef enum { QMX_SOFTMAX = 0, QMX_SIGMOID = 1 } qmx_scoring_t;

/*
 * Residual addition and root-mean-square norm, per row of K values:
 *   h = x + residual                (fp32; h = x without a residual)
 *   residual_out = h                (rounded to the residual's type)
 *   y = h / sqrt(mean(h^2) + eps) * weight
 * The norm is taken of the fp32 sum, before residual_out's rounding, and its
 * statistics and products are formed in fp64 and rounded once to fp32, so
 * that the quantized outputs hold the codes of the correctly rounded norm;
 * the fp32 value is then rounded or quantized to `fmt` as above.
 *   x          xtype [M][K]
 *   residual   rtype [M][K] or NULL;  residual_out likewise, NULL exactly
 *              when residual is; it may be the residual array itself.  The
 *              other outputs overlap no input.
 *   weight     wtype [K] or NULL (all ones)
 *   y, y_scales  the output in `fmt`; y_scales NULL exactly for QMX_BF16
 * 1 <= K <= 16384; QMX_Q8B32 and QMX_MXFP4 need K % 32 == 0.  eps >= 0.
 */
qmv_status_t qmx_rmsnorm(qmx_type_t xtype, const void *x, qmx_type_t rtype, const void *residual,
                         void *residual_out, qmx_type_t wtype, const void *weight, float eps,
                         qmx_fmt_t fmt, void *y, void *y_scales, int M, int K, hipStream_t stream);

/*
 * A token's top_k experts: the largest logits in falling order, the lower
 * index first among equals, and their weights:
 *   QMX_SOFTMAX  w_j = exp(l_j) / sum exp(l): over the chosen experts with
 *                normalize, over all E without
 *   QMX_SIGMOID  w_j = 1 / (1 + exp(-l_j)), divided by their sum over the
 *                chosen experts with normalize
 * times `scale`.  A logit of -infinity or NaN masks its expert: it is never
 * chosen and adds nothing to a sum; +infinity is chosen first, and makes the
 * softmax weights NaN.  A token with fewer than top_k unmasked
 * experts gets id -1 and weight 0 in its last slots (the gathers write zero
 * rows for such ids).
 *   logits  ltype (QMX_T_F32 or QMX_T_BF16) [M][E]
 *   ids     int32 [M][top_k],  weights  fp32 [M][top_k]
 * 1 <= E <= 1024, 1 <= top_k <= 16, top_k <= E.
 */
qmv_status_t qmx_router(qmx_type_t ltype, const void *logits, int M, int E, int top_k,
                        qmx_scoring_t scoring, int normalize, float scale, int32_t *ids,
                        float *weights, hipStream_t stream);

/*
 * Values -> blocks (QMX_MXFP4 or QMX_Q8B32); x is xtype [rows][K] with
 * K % 32 == 0.  rows * K may pass 2^32 (an expert projection of any size).
 */
qmv_status_t qmx_quantize(qmx_type_t xtype, const void *x, qmx_fmt_t fmt, void *codes,
                          void *scales, long long rows, int K, hipStream_t stream);

/*
 * Blocks -> values: code times scale in fp32, rounded to ytype
 * (y: ytype [rows][K]); a NaN scale gives NaN.
 */
qmv_status_t qmx_dequantize(qmx_fmt_t fmt, const void *codes, const void *scales,
                            qmx_type_t ytype, void *y, long long rows, int K,
                            hipStream_t stream);

/* Static English text for a status code of these calls (never NULL). */
const char *qmx_strerror(qmv_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* QMX_H */
