// qmx_values.hpp -- loads, stores and conversions of values that the kernels
// of libqmx.so and libqmt.so share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmx.h"

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------ 8 values a lane
// Eight consecutive values of a 32- or 16-bit type as loaded: 32 or 16 bytes.
struct Raw8 {
    uint4 a, b;
};

// (the type is the same for the whole launch: the branches are uniform)
__device__ __forceinline__ Raw8 load_raw8(const void *base, size_t i, int type)
{
    Raw8 r;
    r.b = make_uint4(0, 0, 0, 0);
    if (type == QMX_T_F32) {
        const uint4 *p = (const uint4 *)((const float *)base + i);
        r.a = p[0];
        r.b = p[1];
    } else {
        r.a = *(const uint4 *)((const uint16_t *)base + i);
    }
    return r;
}

__device__ __forceinline__ void raw_to_f32(const Raw8 &r, int type, float (&v)[8])
{
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (type == QMX_T_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    } else if (type == QMX_T_BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f16x2 h = __builtin_bit_cast(f16x2, w[j]);
            v[2 * j] = (float)h[0];
            v[2 * j + 1] = (float)h[1];
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const bf16x2 h = {(__bf16)a, (__bf16)b};                  // nearest, ties to even
    return __builtin_bit_cast(uint32_t, h);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    const f16x2 h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
}

__device__ __forceinline__ void store8(void *base, size_t i, int type, const float (&v)[8])
{
    if (type == QMX_T_F32) {
        float4 *p = (float4 *)((float *)base + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if (type == QMX_T_BF16) {
        *(uint4 *)((uint16_t *)base + i) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
        *(uint4 *)((uint16_t *)base + i) =
            make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7]));
    }
}

// Values first, first + step, ... of a row of K values of any type, the last
// one again past the end (P loads with no branch between them, all in flight
// at once); a value's bits to its value.
template <int P>
__device__ __forceinline__ void load_bits(const void *base, size_t row, int first, int step, int K, int type,
                                          uint32_t (&v)[P])
{
    if (type == QMX_T_F32) {
        const uint32_t *const p = (const uint32_t *)base + row;
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = p[min(first + i * step, K - 1)];
    } else {
        const uint16_t *const p = (const uint16_t *)base + row;
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = p[min(first + i * step, K - 1)];
    }
}

template <int P>
__device__ __forceinline__ void bits_to_f32(const uint32_t (&b)[P], int type, float (&v)[P])
{
    if (type == QMX_T_F16) {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)b[i]);
    } else {
        const int up = type == QMX_T_BF16 ? 16 : 0;
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = __uint_as_float(b[i] << up);
    }
}

__device__ __forceinline__ void store1(void *base, size_t i, int type, float v)
{
    if (type == QMX_T_F32)
        ((float *)base)[i] = v;
    else if (type == QMX_T_BF16)
        ((uint16_t *)base)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else
        ((uint16_t *)base)[i] = __builtin_bit_cast(uint16_t, (_Float16)v);
}

// ---------------------------------------------------------- blocks of 128
// The scale of an e4m3 block from its largest magnitude's bits.  The quotient by
// 448 is rounded as a division's: the product with the reciprocal's nearest is
// off by a last place at most, its remainder is exact, and a constant's nearest
// reciprocal then rounds right (Markstein's theorem).
__device__ __forceinline__ float f8_scale(uint32_t amax)
{
    if (amax >= 0x7F800000u) return __builtin_nanf("");
    const float a = __uint_as_float(amax), q = a * (1.0f / 448.0f);
    return fmaxf(__builtin_fmaf(__builtin_fmaf(-448.0f, q, a), 1.0f / 448.0f, q), 0x1p-126f);
}

// Eight e4m3 codes of v / d, value j in byte j: the nearest of the exact
// quotient, ties to even.  v times the reciprocal is off by at most 2^-22 of
// itself, so only a product that lies next to a border between two codes may
// round to the wrong one, and on which side the quotient lies is the sign of v -
// border d, which one multiply-add gives.  20 bits below e4m3's last one a border
// is a half, plus or minus 4; below the normal range, 2^-6, codes are as far apart
// as above it, so 2^-6 more has the same bits there (off by another half at
// most).  (The quotients in 64 bits of every group of 8 with such a value, with 8-bit
// values of 8-bit largest ones many: 92160 rows of 2880 from bf16 226 us, so 175;
// divisions rounded right for all of them bound the quantizers.)
__device__ __forceinline__ uint2 f8_codes(const float (&v)[8], float d)
{
    if (!(d < __builtin_inff())) return make_uint2(0, 0);
    const float r = __builtin_amdgcn_rcpf(d);                 // (off by 2^-23 of itself at most; d and r are normal)
    float t[8], low = __builtin_inff();
    uint32_t border = ~0u;                                    // the smallest distance to a border, plus 4, << 12
    auto test = [&](float f) {
        const uint32_t o = (__float_as_uint(f) << 12) + ((0x80000u + 4u) << 12);
        border = border < o ? border : o;
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        t[j] = v[j] * r;
        test(t[j]);
        low = __builtin_fminf(low, __builtin_fabsf(t[j]));
    }
    if (low < 0x1p-6f) {
        border = ~0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = __builtin_fabsf(t[j]);
            test(m < 0x1p-6f ? m + 0x1p-6f : m);
        }
    }
    if (border < 9u << 12) {
        // (scaled up where the difference could underflow)
        const float up = d < 0x1p-60f ? 0x1p60f : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = __builtin_fabsf(t[j]), more = m < 0x1p-6f ? 0x1p-6f : 0.0f;
            const uint32_t b = __float_as_uint(m + more);
            const float at = __uint_as_float((b & 0xFFF00000u) | 0x80000u) - more;
            const float side = __builtin_fmaf(-at, d * up, __builtin_fabsf(v[j]) * up);
            const uint32_t e = __float_as_uint(at) + (side > 0.0f ? 1u : side < 0.0f ? ~0u : 0u);
            if ((b << 12) + ((0x80000u + 4u) << 12) < 9u << 12) t[j] = __builtin_copysignf(__uint_as_float(e), v[j]);
        }
    }
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

__device__ __forceinline__ void f8_values(uint2 c, float d, float (&v)[8])
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        v[4 * i] = a[0] * d, v[4 * i + 1] = a[1] * d, v[4 * i + 2] = b[0] * d, v[4 * i + 3] = b[1] * d;
    }
}

// The largest magnitude of eight values as its bit pattern in fp32 (every NaN
// and infinity is at or above 0x7F800000), and of the 16 lanes of a row, which
// hold a block's 128.  All lanes of the row take part.
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        m = m > b ? m : b;
    }
    return m;
}

// The same of values as loaded: 16-bit patterns two at a time.
template <int T> __device__ __forceinline__ uint32_t amax_bits8(const Raw8 &r)
{
    if constexpr (T == QMX_T_F32) {
        float v[8];
        raw_to_f32(r, T, v);
        return amax_bits8(v);
    } else {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 h = {0, 0};
        for (const uint32_t w : {r.a.x, r.a.y, r.a.z, r.a.w})
            h = __builtin_elementwise_max(h, __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu));
        const uint16_t o = h[0] > h[1] ? h[0] : h[1];
        return T == QMX_T_BF16 ? (uint32_t)o << 16 : __float_as_uint((float)__builtin_bit_cast(_Float16, o));
    }
}

template <int CTRL> __device__ __forceinline__ uint32_t row_max_step(uint32_t m)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xF, 0xF, false);
    return m > o ? m : o;
}

__device__ __forceinline__ uint32_t row16_max(uint32_t m)
{
    m = row_max_step<0x128>(m);                               // row_ror 8, 4, 2, 1
    m = row_max_step<0x124>(m);
    m = row_max_step<0x122>(m);
    return row_max_step<0x121>(m);
}

}  // namespace
