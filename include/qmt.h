/*
 * qmt.h -- C ABI of libqmt.so: the steps of a model around the 8-bit
 * floating-point products of qmv.h (QMV_W_F8B128 x QMV_A_F8B128), on AMD
 * Instinct MI355X (gfx950).
 *
 *   qmt_quantize_weights    values -> e4m3 codes with a scale per 128 x 128
 *                           block: the weights of those products
 *   qmt_dequantize_weights  the other way
 *   qmt_qk_norm_rope        norm of each query and key head and the rotation
 *                           by position, from the rows that a query/key/value
 *                           product writes
 *   qmt_logprobs            log probability of a given token, entropy and the
 *                           top alternatives, from the logits that a head's
 *                           product writes
 *
 * -------------------------------------------------------------- conventions
 * As in qmv.h and qmx.h: every pointer is a device pointer owned by the
 * caller, arrays are dense row-major, a call only enqueues launches on
 * `stream`, takes no memory of its own and reads and writes only the extents
 * given here.  The stream's device must be the current one.  Arguments are
 * checked on the host before the first launch.  Results are bitwise identical
 * from run to run (fixed reduction order, no atomics on results).
 */
#ifndef QMT_H
#define QMT_H

#include "qmx.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * E matrices of N rows of K values -> e4m3 codes uint8 [E][N][K] and scales
 * fp32 [E][ceil(N/128)][ceil(K/128)] (the weights of QMV_W_F8B128).  Blocks
 * start at each matrix's first row; the last of either direction may be short.
 * With amax = max |v| of a block:
 *   d    = max(amax / 448, 2^-126), the quotient rounded to fp32,
 *   code = v / d rounded to the nearest e4m3 value, ties to even
 * (of the exact quotient: no rounding before).  A block that holds a NaN or
 * an infinity gets scale NaN and codes 0.
 *   x  xtype [E][N][K], 16-byte aligned, as codes; scales 4-byte aligned.
 * K % 32 == 0, K < 2^24, N < 2^24, E * N * K <= 2^60.
 */
qmv_status_t qmt_quantize_weights(qmx_type_t xtype, const void *x, void *codes, float *scales, int E,
                                  int N, int K, hipStream_t stream);

/* Code times scale in fp32, rounded to ytype (y: ytype [E][N][K]). */
qmv_status_t qmt_dequantize_weights(const void *codes, const float *scales, qmx_type_t ytype, void *y,
                                    int E, int N, int K, hipStream_t stream);

typedef enum { QMT_HALF = 0, QMT_PAIRS = 1 } qmt_rotation_t;

/*
 * For each of M tokens and each of its heads h[0..D), with the queries' or the
 * keys' weights w:
 *   n[i] = h[i] / sqrt(mean(h^2) + eps) * w[i]
 * and, for i < R / 2, with position p = positions[m], cos = table[p][i] and
 * sin = table[p][R / 2 + i]:
 *   QMT_HALF   (a, b) = (n[i], n[i + R / 2])
 *   QMT_PAIRS  (a, b) = (n[2 i], n[2 i + 1])
 *   written in their places: a cos - b sin,  b cos + a sin
 * The values R .. D - 1 of a head are only normed.  The statistics and the
 * norm's products are formed in fp64 and rounded to fp32 once, the rotation in
 * fp32.
 *   x          xtype [M][row]: the query heads, then the key heads, D values
 *              each; what follows them (row >= (heads + kv_heads) * D, the
 *              values say) is not read
 *   table      fp32 [P][R]: R / 2 cosines, then R / 2 sines, for each position
 *   positions  int32 [M].  A position outside [0, P) is not an error: the
 *              token's queries and keys are zeros.
 *   q_weight, k_weight   wtype [D], or NULL (all ones)
 *   q          ytype [M][heads][D]
 *   k          ytype [M][kv_heads][D]; NULL exactly when kv_heads is 0
 * The outputs overlap no input.  D % 8 == 0, D <= 512, R % 8 == 0, 8 <= R
 * <= D, row % 4 == 0, 1 <= heads, 0 <= kv_heads, heads + kv_heads <= 4096, row < 2^24,
 * M * (heads + kv_heads) < 2^31.  Alignment: x, q, k and the weights four of
 * their elements, table 16 bytes, positions 4.
 */
qmv_status_t qmt_qk_norm_rope(qmx_type_t xtype, const void *x, int row, int heads, int kv_heads, int D,
                              const float *table, int P, int R, const int32_t *positions,
                              qmx_type_t wtype, const void *q_weight, const void *k_weight, float eps,
                              qmt_rotation_t rotation, qmx_type_t ytype, void *q, void *k, int M,
                              hipStream_t stream);

/*
 * For each of M rows l[0..V) of logits, with m = max l and s = sum exp(l - m):
 *   logprob      l[t] - m - log s               t = tokens[row]
 *   entropy      log s - sum exp(l - m) (l - m) / s
 *   top_ids, top_logprobs   the top_k largest logits in falling order, the
 *                lower index first among equals, and their log probabilities
 * A logit of -infinity or NaN is masked: it adds nothing, is never among the
 * top and has log probability -infinity.  Slots that no logit is left for get
 * id -1 and -infinity; a row with every logit masked has entropy 0.  +infinity
 * makes a row's log probabilities and entropy NaN.  A token outside [0, V) is
 * not an error: its log probability is 0.
 * Exponentials are fp32; sums are fp64, of terms or of up to eight fp32 terms
 * none of which is the largest logit's (so that a log probability next to 0 keeps
 * its digits); the rest of a row's arithmetic is fp64.
 *   logits     ltype [M][V]
 *   tokens     int32 [M], or NULL with logprobs NULL
 *   logprobs   fp32 [M], or NULL
 *   entropy    fp32 [M], or NULL
 *   top_ids    int32 [M][top_k], top_logprobs fp32 [M][top_k]; NULL exactly
 *              when top_k is 0
 *   workspace  qmt_logprobs_workspace(M, V, top_k) bytes (0: may be NULL),
 *              overwritten; calls that overlap need one each
 * 1 <= V < 2^30, 0 <= top_k <= 32, M < 2^24; M * V may pass 2^32.  Alignment:
 * workspace 16 bytes, the rest their element size.
 */
qmv_status_t qmt_logprobs(qmx_type_t ltype, const void *logits, int M, int V, const int32_t *tokens,
                          int top_k, float *logprobs, float *entropy, int32_t *top_ids,
                          float *top_logprobs, void *workspace, hipStream_t stream);

/* Bytes of workspace of such a call (0 for sizes that it refuses). */
long long qmt_logprobs_workspace(int M, int V, int top_k);

/* Static English text for a status code of these calls (never NULL). */
const char *qmt_strerror(qmv_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* QMT_H */
