// qmt_host.hpp -- argument checks and launch plans of libqmt.so (include/qmt.h).
// Plain C++17 without HIP calls, so that the host compiler's sanitizers can
// drive it.
#pragma once

#include <stdint.h>

#include "qmt.h"

namespace qmt_host {

constexpr int kMaxHead = 512;        // 64 lanes of 8 values
constexpr int kMaxHeads = 4096;
constexpr int kMaxTop = 32;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool type_ok(int t) { return t >= QMX_T_F32 && t <= QMX_T_F16; }
inline uintptr_t type_bytes(int t) { return t == QMX_T_F32 ? 4 : 2; }

inline qmv_status_t check_weights(int type, const void *values, const void *codes, const void *scales, int E, int N,
                                  int K)
{
    if (!values || !codes || !scales || E <= 0 || N <= 0 || K <= 0)
        return QMV_EINVAL;
    if (!type_ok(type) || K % 32 != 0 || K >= 1 << 24 || N >= 1 << 24 ||
        (long long)N * K > (1LL << 60) / E)
        return QMV_EUNSUPPORTED;
    if (!aligned(values, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return QMV_EINVAL;
    return QMV_OK;
}

inline qmv_status_t check_qk(int xtype, const void *x, int row, int heads, int kv_heads, int D, const void *table, int P,
                             int R, const void *positions, int wtype, const void *q_weight, const void *k_weight,
                             float eps, int rotation, int ytype, const void *q, const void *k, int M)
{
    if (!x || !table || !positions || !q || !k != (kv_heads == 0) || M <= 0 || heads <= 0 || kv_heads < 0 || D <= 0 ||
        P <= 0 || R <= 0 || row <= 0 || !(eps >= 0.0f))
        return QMV_EINVAL;
    if (!type_ok(xtype) || !type_ok(ytype) || ((q_weight || k_weight) && !type_ok(wtype)) ||
        (rotation != QMT_HALF && rotation != QMT_PAIRS) || D % 8 != 0 || D > kMaxHead || R % 8 != 0 || R > D ||
        heads > kMaxHeads || kv_heads > kMaxHeads - heads || row >= 1 << 24 ||
        (long long)M * (heads + kv_heads) >= 1LL << 31)
        return QMV_EUNSUPPORTED;
    if (row < (heads + kv_heads) * D || row % 4 != 0 || !aligned(x, 4 * type_bytes(xtype)) ||
        !aligned(q, 4 * type_bytes(ytype)) || (k && !aligned(k, 4 * type_bytes(ytype))) || !aligned(table, 16) ||
        !aligned(positions, 4) || (q_weight && !aligned(q_weight, 4 * type_bytes(wtype))) ||
        (k_weight && !aligned(k_weight, 4 * type_bytes(wtype))))
        return QMV_EINVAL;
    return QMV_OK;
}

inline qmv_status_t check_logprobs(int ltype, const void *logits, int M, int V, const void *tokens, int top_k,
                                   const void *logprobs, const void *entropy, const void *top_ids,
                                   const void *top_logprobs)
{
    if (!logits || !tokens != !logprobs || M <= 0 || V <= 0 || top_k < 0 || !top_ids != (top_k == 0) ||
        !top_logprobs != (top_k == 0) || (!logprobs && !entropy && top_k == 0))
        return QMV_EINVAL;
    if (!type_ok(ltype) || V >= 1 << 30 || M >= 1 << 24 || top_k > kMaxTop)
        return QMV_EUNSUPPORTED;
    if (!aligned(logits, type_bytes(ltype)) || !aligned(tokens, 4) || !aligned(logprobs, 4) || !aligned(entropy, 4) ||
        !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
        return QMV_EINVAL;
    return QMV_OK;
}

// A row of V logits is cut into `parts` (at most kMaxParts), a workgroup of
// `threads` each that takes `steps` times 8 logits a thread: one step where the
// call has no more than kMaxShort parts (part).  Unless one long part is the row
// (join), each part leaves its sums (kListSums bytes) and a list of 64 entries for
// a second launch, a workgroup a row.  (Top 20, us in short parts and in long
// ones: 201088 fp32 logits: 1 row 10 and 18, 16 16 and 20, 32 (3168 parts) 21 and
// 23, 64 30 and 27; 131071 bf16: 1 10 and 13, 32 (2048) 16 and 19, 64 (4096) 23 and
// 23, 128 36 and 28; 32000 fp32: 1 10 and 13, 128 (2048) 17 and 20.)
constexpr int kMaxShort = 4096;
constexpr int kMaxParts = 128, kJoinWaves = 8, kListSums = 32;
struct LogprobPlan {
    int parts, threads, steps;
    bool part, join;
};

inline LogprobPlan plan_logprobs(int M, int V)
{
    auto cut = [](int of, int n) { return n / of + (n % of != 0); };
    // (up to 14 logits before and behind whole groups of 8 go with the first part)
    const int shorts = cut(2048, V);
    if (shorts <= kMaxParts && (long long)shorts * M <= kMaxShort)
        return {shorts, 256, 1, true, true};
    const int steps = cut(4096, V);
    int parts = 512 / M;                              // two for each of 256 CUs, as far as the row goes
    parts = parts < 1 ? 1 : parts > kMaxParts ? kMaxParts : parts > steps ? steps : parts;
    const int each = cut(parts, steps);
    parts = cut(each, steps);
    return {parts, 512, each, false, parts > 1};
}

inline long long logprobs_workspace(int M, int V, int top_k)
{
    if (M <= 0 || V <= 0 || top_k < 0 || V >= 1 << 30 || M >= 1 << 24 || top_k > kMaxTop)
        return 0;
    const LogprobPlan p = plan_logprobs(M, V);
    return p.join ? (long long)M * p.parts * (kListSums + (top_k ? 512 : 0)) : 0;
}

inline const char *status_text(int status)
{
    switch (status) {
    case QMV_OK: return "success";
    case QMV_EINVAL: return "invalid argument (null or misaligned pointer, a size <= 0, a row shorter than its heads or "
                            "no multiple of 4, eps below zero, or an output that does not go with the others)";
    case QMV_EUNSUPPORTED: return "unsupported type or size (weights: K % 32 == 0; heads: D % 8 == 0, D <= 512, "
                                  "R % 8 == 0, 8 <= R <= D, at most 4096 heads; log probabilities: V < 2^30, top_k <= 32)";
    case QMV_EHIP: return "the HIP runtime rejected the kernel launch";
    }
    return "unknown status";
}

}  // namespace qmt_host
