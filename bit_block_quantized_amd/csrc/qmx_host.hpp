// qmx_host.hpp -- argument checks of libqmx.so (include/qmx.h).  Plain C++17
// without HIP calls, so that the host compiler's sanitizers can drive it.
#pragma once

#include <stdint.h>

#include "qmx.h"

namespace qmx_host {

constexpr int kMaxNormK = 16384;     // a row's values stay in one workgroup's registers
constexpr int kMaxExperts = 1024;    // 16 logits per lane of a wave
constexpr int kMaxTopK = 16;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool type_ok(int t) { return t >= QMX_T_F32 && t <= QMX_T_F16; }
inline uintptr_t type_bytes(int t) { return t == QMX_T_F32 ? 4 : 2; }

inline qmv_status_t check_rmsnorm(int xtype, const void *x, int rtype, const void *residual,
                                  const void *residual_out, int wtype, const void *weight, float eps, int fmt,
                                  const void *y, const void *y_scales, int M, int K)
{
    if (!x || !y || !residual != !residual_out || M <= 0 || K <= 0 || !(eps >= 0.0f))
        return QMV_EINVAL;
    if (!type_ok(xtype) || (residual && !type_ok(rtype)) || (weight && !type_ok(wtype)) || fmt < QMX_BF16 ||
        fmt > QMX_MXFP4 || K > kMaxNormK || (fmt != QMX_BF16 && K % 32 != 0))
        return QMV_EUNSUPPORTED;
    if ((fmt == QMX_BF16) != !y_scales)
        return QMV_EINVAL;
    const bool vec = K % 8 == 0;
    if (!aligned(x, vec ? 16 : type_bytes(xtype)) || !aligned(y, vec ? 16 : 2) ||
        (residual && (!aligned(residual, vec ? 16 : type_bytes(rtype)) ||
                      !aligned(residual_out, vec ? 16 : type_bytes(rtype)))) ||
        (weight && !aligned(weight, vec ? 16 : type_bytes(wtype))) || (fmt == QMX_Q8B32 && !aligned(y_scales, 2)))
        return QMV_EINVAL;
    return QMV_OK;
}

inline qmv_status_t check_router(int ltype, const void *logits, int M, int E, int top_k, int scoring,
                                 const void *ids, const void *weights)
{
    if (!logits || !ids || !weights || M <= 0 || E <= 0 || top_k <= 0)
        return QMV_EINVAL;
    if ((ltype != QMX_T_F32 && ltype != QMX_T_BF16) || (scoring != QMX_SOFTMAX && scoring != QMX_SIGMOID) ||
        E > kMaxExperts || top_k > kMaxTopK || top_k > E)
        return QMV_EUNSUPPORTED;
    if (!aligned(logits, type_bytes(ltype)) || !aligned(ids, 4) || !aligned(weights, 4))
        return QMV_EINVAL;
    return QMV_OK;
}

// qmx_quantize and qmx_dequantize: `values` is the xtype/ytype array.
inline qmv_status_t check_blocks(int type, const void *values, int fmt, const void *codes, const void *scales,
                                 long long rows, int K)
{
    if (!values || !codes || !scales || rows <= 0 || K <= 0)
        return QMV_EINVAL;
    // (rows bound: the byte count of 32-bit values stays below 2^62)
    if (!type_ok(type) || (fmt != QMX_Q8B32 && fmt != QMX_MXFP4) || K % 32 != 0 || rows > (1LL << 60) / K)
        return QMV_EUNSUPPORTED;
    if (!aligned(values, 16) || !aligned(codes, 16) || (fmt == QMX_Q8B32 && !aligned(scales, 2)))
        return QMV_EINVAL;
    return QMV_OK;
}

inline const char *status_text(int status)
{
    switch (status) {
    case QMV_OK: return "success";
    case QMV_EINVAL: return "invalid argument (null or misaligned pointer, a size <= 0, eps below zero, or an "
                            "output that does not go with the others)";
    case QMV_EUNSUPPORTED: return "unsupported type, format or size (norm: K <= 16384; blocks: K % 32 == 0; "
                                  "router: fp32 or bf16 logits, E <= 1024, top_k <= 16 and <= E)";
    case QMV_EHIP: return "the HIP runtime rejected the kernel launch";
    }
    return "unknown status";
}

}  // namespace qmx_host
