// qmx.hip -- libqmx.so (include/qmx.h): residual + RMS norm, router, and the
// MXFP4 / int8 block quantizers, with their C ABI.
//
// Everything here is bound by the bytes it moves (or, for a few tokens, by a
// launch): one pass over the data, 16-byte accesses, rows held in registers
// between the reduction and the output.  Times are a kernel's own: its median in
// a trace of ten calls with three sets of inputs in turn.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmx_host.hpp"

namespace {

using namespace qmx_host;

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

// ------------------------------------------------------------ block formats
// Four neighbouring lanes hold a block (8 values each).  The largest
// magnitude as its bit pattern: magnitudes order like their bits, and every
// NaN and infinity is at or above 0x7F800000.
template <int CTRL> __device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, CTRL, 0xF, 0xF, true);
    return m > o ? m : o;
}

__device__ __forceinline__ uint32_t block_amax_bits(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        m = m > b ? m : b;
    }
    m = quad_max<0xB1>(m);                                    // lane ^ 1 (quad_perm 1,0,3,2)
    return quad_max<0x4E>(m);                                 // lane ^ 2 (quad_perm 2,3,0,1)
}

// Scale byte of an MXFP4 block: adding 1/4 of its power of two to amax (bit
// 21) carries into the exponent from 1.75 on, where amax rounds up to the
// next power of two at e2m1's two significant bits.
__device__ __forceinline__ uint32_t mxfp4_byte(uint32_t amax)
{
    if (amax >= 0x7F800000u) return 255u;
    const int e = (int)((amax + 0x00200000u) >> 23) - 2;
    return e > 0 ? (uint32_t)e : 0u;
}

// Eight e2m1 codes, value j in bits 4 j .. 4 j + 3.  The multiplication by
// the power of two is exact (or far below e2m1's smallest step); the convert
// rounds to nearest, ties to even, and keeps the sign.
__device__ __forceinline__ uint32_t mxfp4_codes(const float (&v)[8], uint32_t byte)
{
    if (byte == 255u) return 0u;
    const int e = 127 - (int)byte;
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = __builtin_ldexpf(v[j], e);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[0], t[1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[2], t[3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[4], t[5], 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[6], t[7], 1.0f, 3);
    return c;
}

// int8 block: the fp16 scale, and eight codes.  Division and reciprocal are
// the correctly rounded ones.
__device__ __forceinline__ _Float16 q8_scale(uint32_t amax)
{
    if (amax >= 0x7F800000u) return __builtin_bit_cast(_Float16, (uint16_t)0x7E00);
    return (_Float16)(__uint_as_float(amax) / 127.0f);
}

__device__ __forceinline__ uint2 q8_codes(const float (&v)[8], _Float16 d16)
{
    const float d = (float)d16;
    uint2 q = make_uint2(0, 0);
    if (d > 0.0f && d < __builtin_inff()) {
        const float r = 1.0f / d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = fminf(fmaxf(__builtin_rintf(v[j] * r), -127.0f), 127.0f);
            const float hi = fminf(fmaxf(__builtin_rintf(v[4 + j] * r), -127.0f), 127.0f);
            q.x |= ((uint32_t)(int)lo & 0xFFu) << (8 * j);
            q.y |= ((uint32_t)(int)hi & 0xFFu) << (8 * j);
        }
    }
    return q;
}

// Write eight values at flat index i (a multiple of 8) of an output in FMT;
// the four lanes of a block call it together.
template <int FMT>
__device__ __forceinline__ void put8(void *y, void *ys, size_t i, const float (&v)[8])
{
    if constexpr (FMT == QMX_BF16) {
        store8(y, i, QMX_T_BF16, v);
    } else {
        const uint32_t amax = block_amax_bits(v);
        if constexpr (FMT == QMX_MXFP4) {
            const uint32_t byte = mxfp4_byte(amax);
            *(uint32_t *)((uint8_t *)y + i / 2) = mxfp4_codes(v, byte);
            if ((i & 31) == 0) ((uint8_t *)ys)[i >> 5] = (uint8_t)byte;
        } else {
            const _Float16 d = q8_scale(amax);
            *(uint2 *)((uint8_t *)y + i) = q8_codes(v, d);
            if ((i & 31) == 0) ((_Float16 *)ys)[i >> 5] = d;
        }
    }
}

// ---------------------------------------------------------------- RMS norm
// One row per group of T threads (T = 64: four rows per workgroup, a wave
// each; else one row per workgroup), P steps of 8 values a thread, held in
// registers from the load to the output: x and the residual are read once.
// sum(h^2) and the products are formed in fp64: the quantizers round to a
// border-exact code, and an fp32 norm is off by 1e-7, which moves one code
// in 1e5 across a border.  The kernel waits for memory, not for the fp64
// rate: 2048 rows of 7168, to int8: bf16 with an fp32 residual 35 us for 162 MB,
// 4.6 TB/s, fp32 with a bf16 one 29 us for 133 MB (a copy reaches 5.1 TB/s).
struct NormArgs {
    const void *x, *res, *w;
    void *res_out, *y, *ys;
    float eps;
    int xt, rt, wt, M, K, row0;
};

template <int T>
__device__ __forceinline__ double row_sum(double s, double *part)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0.0;
#pragma unroll
        for (int i = 0; i < T / 64; ++i) s += part[i];        // the same order in every thread
    }
    return s;
}

template <int FMT, int T, int P>
__global__ __launch_bounds__(T == 64 ? 256 : T) void qmx_rmsnorm_kernel(const NormArgs a)
{
    __shared__ double part[16];
    constexpr int R = T == 64 ? 4 : 1;
    const int tid = T == 64 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
    const long long row = a.row0 + (long long)blockIdx.x * R + (T == 64 ? threadIdx.x >> 6 : 0);
    if (row >= a.M) return;                                   // whole waves; T > 64 has one row a group
    const size_t base = (size_t)row * a.K;
    Raw8 xr[P], rr[P], wr[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int k = 8 * (p * T + tid);
        if (k < a.K) {
            xr[p] = load_raw8(a.x, base + k, a.xt);
            if (a.res) rr[p] = load_raw8(a.res, base + k, a.rt);
            if (a.w) wr[p] = load_raw8(a.w, k, a.wt);
        }
    }
    float h[P][8];
    double s = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int k = 8 * (p * T + tid);
        if (k < a.K) {
            raw_to_f32(xr[p], a.xt, h[p]);
            if (a.res) {
                float r[8];
                raw_to_f32(rr[p], a.rt, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[p][j] += r[j];
                store8(a.res_out, base + k, a.rt, h[p]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s = __builtin_fma((double)h[p][j], (double)h[p][j], s);
        }
    }
    s = row_sum<T>(s, part);
    const double r = 1.0 / __builtin_sqrt(s / (double)a.K + (double)a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int k = 8 * (p * T + tid);
        if (k < a.K) {
            float o[8], w[8];
            if (a.w) {
                raw_to_f32(wr[p], a.wt, w);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = (float)((double)h[p][j] * r * (double)w[j]);
            put8<FMT>(a.y, a.ys, base + k, o);
        }
    }
}

// Rows whose length is no multiple of 8 (bf16 output): the same, with thread
// t of the group taking values t, t + T, ... one at a time, so that a wave's
// accesses are still consecutive.  All loads are given out before the first
// is used (777 rows of 2879: 7.2 us, 8.9 with a wait a value).
template <int T, int P>
__global__ __launch_bounds__(T == 64 ? 256 : T) void qmx_rmsnorm_odd_kernel(const NormArgs a)
{
    __shared__ double part[16];
    constexpr int R = T == 64 ? 4 : 1;
    const int tid = T == 64 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
    const long long row = a.row0 + (long long)blockIdx.x * R + (T == 64 ? threadIdx.x >> 6 : 0);
    if (row >= a.M) return;
    const size_t base = (size_t)row * a.K;
    uint32_t xb[P], rb[P], wb[P];
    load_bits<P>(a.x, base, tid, T, a.K, a.xt, xb);
    if (a.res) load_bits<P>(a.res, base, tid, T, a.K, a.rt, rb);
    if (a.w) load_bits<P>(a.w, 0, tid, T, a.K, a.wt, wb);
    float h[P], w[P];
    bits_to_f32<P>(xb, a.xt, h);
    if (a.res) {
        float rv[P];
        bits_to_f32<P>(rb, a.rt, rv);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            h[p] += rv[p];
            if (p * T + tid < a.K) store1(a.res_out, base + p * T + tid, a.rt, h[p]);
        }
    }
    double s = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p)
        if (p * T + tid < a.K) s = __builtin_fma((double)h[p], (double)h[p], s);
    s = row_sum<T>(s, part);
    const double r = 1.0 / __builtin_sqrt(s / (double)a.K + (double)a.eps);
    if (a.w) {
        bits_to_f32<P>(wb, a.wt, w);
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p) w[p] = 1.0f;
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
        if (p * T + tid < a.K)
            store1(a.y, base + p * T + tid, QMX_T_BF16, (float)((double)h[p] * r * (double)w[p]));
}

// Threads a row: a step of 8 values each keeps the most bytes in flight
// (2048 rows of 7168, us: 256 threads 38.7, 512 35.4, 1024 34.9; one row of
// 7168 5.6, 4.3, 4.0), except where a row of up to 4096 leaves many of 512
// threads idle and there are rows enough to fill the chip (rows of 2880: 2048
// of them 14.1 us with 256 threads, 15.7 with 512; 1024 10.5 and 10.2; 512 7.0
// and 6.8; one 3.6 and 3.1).
template <int FMT>
const void *norm_kernel(int M, int K, int &threads, int &rows)
{
    rows = 1;
    threads = 256;
    if (K <= 512) { rows = 4; return (const void *)&qmx_rmsnorm_kernel<FMT, 64, 1>; }
    if (K <= 2048) return (const void *)&qmx_rmsnorm_kernel<FMT, 256, 1>;
    if (K <= 4096 && M >= 1024) return (const void *)&qmx_rmsnorm_kernel<FMT, 256, 2>;
    if (K <= 4096) { threads = 512; return (const void *)&qmx_rmsnorm_kernel<FMT, 512, 1>; }
    threads = 1024;
    if (K <= 8192) return (const void *)&qmx_rmsnorm_kernel<FMT, 1024, 1>;
    return (const void *)&qmx_rmsnorm_kernel<FMT, 1024, 2>;
}

const void *norm_odd_kernel(int K, int &threads, int &rows)
{
    rows = 1;
    if (K <= 256) { threads = 256; rows = 4; return (const void *)&qmx_rmsnorm_odd_kernel<64, 4>; }
    if (K <= 4096) { threads = 256; return (const void *)&qmx_rmsnorm_odd_kernel<256, 16>; }
    threads = 1024;
    return (const void *)&qmx_rmsnorm_odd_kernel<1024, 16>;
}

// ---------------------------------------------------- quantize / dequantize
// A flat array of 8-value pieces: thread t of a workgroup takes pieces
// t, t + 256, ... (UN of them in flight) of the workgroup's run.  Bound by the
// bytes: 92160 rows of 2880 bf16 to MXFP4 124 us, back 129, to int8 145: 5.2 to
// 5.6 TB/s, the rate of a copy.
constexpr int kPieceUnroll = 4;

template <int FMT>
__global__ __launch_bounds__(256) void qmx_quantize_kernel(const void *x, int xt, void *y, void *ys,
                                                           long long pieces)
{
    constexpr int UN = kPieceUnroll;
    for (long long p0 = (long long)blockIdx.x * (256 * UN); p0 < pieces; p0 += (long long)gridDim.x * (256 * UN)) {
        Raw8 r[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const long long p = p0 + u * 256 + threadIdx.x;
            if (p < pieces) r[u] = load_raw8(x, 8 * (size_t)p, xt);
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const long long p = p0 + u * 256 + threadIdx.x;
            if (p < pieces) {                                 // pieces % 4 == 0: whole blocks
                float v[8];
                raw_to_f32(r[u], xt, v);
                put8<FMT>(y, ys, 8 * (size_t)p, v);
            }
        }
    }
}

__device__ __forceinline__ float e8m0(uint32_t s)
{
    if (s == 0u) return __uint_as_float(0x00400000u);         // 2^-127
    return s == 255u ? __builtin_nanf("") : __uint_as_float(s << 23);
}

template <int FMT>
__global__ __launch_bounds__(256) void qmx_dequantize_kernel(const void *c, const void *cs, int yt, void *y,
                                                             long long pieces)
{
    constexpr int UN = kPieceUnroll;
    for (long long p0 = (long long)blockIdx.x * (256 * UN); p0 < pieces; p0 += (long long)gridDim.x * (256 * UN)) {
        uint2 r[UN];
        uint32_t sc[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const long long p = p0 + u * 256 + threadIdx.x;
            if (p < pieces) {
                if constexpr (FMT == QMX_MXFP4) {
                    r[u].x = ((const uint32_t *)c)[p];
                    sc[u] = ((const uint8_t *)cs)[p >> 2];
                } else {
                    r[u] = ((const uint2 *)c)[p];
                    sc[u] = ((const uint16_t *)cs)[p >> 2];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const long long p = p0 + u * 256 + threadIdx.x;
            if (p < pieces) {
                float v[8];
                if constexpr (FMT == QMX_MXFP4) {
                    const float s = e8m0(sc[u]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        // e2m1: sign, two exponent bits, one mantissa bit
                        const uint32_t n = r[u].x >> (4 * j);
                        const uint32_t e = (n >> 1) & 3u, m = n & 1u;
                        const float a = e ? __uint_as_float(((126u + e) << 23) | (m << 22)) : 0.5f * (float)m;
                        v[j] = ((n & 8u) ? -a : a) * s;
                    }
                } else {
                    const float d = (float)__builtin_bit_cast(_Float16, (uint16_t)sc[u]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j] = (float)(int8_t)(r[u].x >> (8 * j)) * d;
                        v[4 + j] = (float)(int8_t)(r[u].y >> (8 * j)) * d;
                    }
                }
                store8(y, 8 * (size_t)p, yt, v);
            }
        }
    }
}

// ------------------------------------------------------------------- router
// One wave per token, L logits a lane (expert lane + 64 i), held in registers;
// top_k times the largest is taken out.  Logits order like these keys; NaN and
// -infinity get key 0 (masked).  The instructions of the selection bound it
// (8192 tokens of 256, top 8: 7.6 us, of which 0.43 a selection; the bytes
// alone take about 2): the maximum runs over the lanes with row shifts and
// broadcasts of the vector ALUs (12.4 us with shuffles through LDS), and the
// lowest expert that has it comes from ballots in scalar registers, with no
// second reduction.
__device__ __forceinline__ uint32_t logit_key(float l)
{
    const uint32_t b = __float_as_uint(l + 0.0f);             // -0 and 0 are equal
    if (!(l > -__builtin_inff())) return 0u;                  // -infinity and NaN
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;          // > 0: -FLT_MAX gives 0x00800000
}

__device__ __forceinline__ float key_logit(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

template <int CTRL> __device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;                                     // (lanes with no source: 0)
}

// The wave's largest value, the same in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = lanes_max<0x111>(v);                                  // from the lane 1, 2, 4, 8 below in the row of 16
    v = lanes_max<0x112>(v);
    v = lanes_max<0x114>(v);
    v = lanes_max<0x118>(v);
    v = lanes_max<0x142>(v);                                  // a row's last lane to the row after it
    v = lanes_max<0x143>(v);                                  // lane 31 to the upper half
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

struct RouterArgs {
    const void *logits;
    int32_t *ids;
    float *weights;
    float scale;
    int lt, M, E, top_k, scoring, normalize, row0;
};

template <int L>
__global__ __launch_bounds__(256) void qmx_router_kernel(const RouterArgs a)
{
    const int lane = threadIdx.x & 63;
    const long long t = a.row0 + (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.M) return;
    const size_t base = (size_t)t * a.E;
    uint32_t key[L];
    float l[L];
    load_bits<L>(a.logits, base, lane, 64, a.E, a.lt, key);
    bits_to_f32<L>(key, a.lt, l);
#pragma unroll
    for (int i = 0; i < L; ++i) key[i] = lane + 64 * i < a.E ? logit_key(l[i]) : 0u;
    // the j-th largest: the wave's largest key, then the lowest expert that
    // has it; lane j keeps it, its owner clears it.  (Once only masked experts
    // are left the key is 0, and clearing a 0 changes nothing.)
    uint32_t my_key = 0, first = 0;
    int my_id = -1;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < L; ++i) m = m > key[i] ? m : key[i];
        m = wave_max(m);
        first = j == 0 ? m : first;
        int lowest = 0;
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            const unsigned long long have = __ballot(key[i] == m);
            lowest = have ? 64 * i + __builtin_ctzll(have) : lowest;
        }
        my_key = lane == j ? m : my_key;
        my_id = lane == j ? lowest : my_id;
#pragma unroll
        for (int i = 0; i < L; ++i) key[i] = lane + 64 * i == lowest ? 0u : key[i];
    }
    const bool have = my_key != 0u;
    if (!have) my_id = -1;
    const float mine = have ? key_logit(my_key) : 0.0f, top = first ? key_logit(first) : 0.0f;
    float w = 0.0f;
    if (a.scoring == QMX_SOFTMAX) {
        const float e = have ? expf(mine - top) : 0.0f;
        float part = e;                                       // the chosen, and without normalize the rest
        if (!a.normalize) {
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (key[i]) part += expf(key_logit(key[i]) - top);
        }
        const float sum = wave_sum(part);
        w = have ? e / sum : 0.0f;
    } else if (a.normalize) {
        // both sides of the quotient times e^-top where top < 0, so that
        // logits far below zero do not divide 0 by 0
        float s = 0.0f;
        if (have) s = top < 0.0f ? expf(mine - top) / (1.0f + expf(mine)) : 1.0f / (1.0f + expf(-mine));
        const float sum = wave_sum(s);
        w = have ? s / sum : 0.0f;
    } else {
        // (e^-l passes fp32's largest where the quotient is still a subnormal number)
        const float e = expf(-fabsf(mine));
        w = have ? (mine < 0.0f ? e : 1.0f) / (1.0f + e) : 0.0f;
    }
    if (lane < a.top_k) {
        a.ids[(size_t)t * a.top_k + lane] = my_id;
        a.weights[(size_t)t * a.top_k + lane] = w * a.scale;
    }
}

const void *router_kernel(int E)
{
    if (E <= 64) return (const void *)&qmx_router_kernel<1>;
    if (E <= 128) return (const void *)&qmx_router_kernel<2>;
    if (E <= 256) return (const void *)&qmx_router_kernel<4>;
    if (E <= 512) return (const void *)&qmx_router_kernel<8>;
    return (const void *)&qmx_router_kernel<16>;
}

// HIP limits a launch to 2^32 threads: beyond this many workgroups the
// element-wise kernels loop and the row kernels are launched again.
constexpr long long kMaxGroups = 1LL << 20;

qmv_status_t go(const void *fn, long long groups, int threads, void **args, hipStream_t stream)
{
    return hipLaunchKernel(fn, dim3((unsigned)groups), dim3((unsigned)threads), args, 0, stream) == hipSuccess
               ? QMV_OK
               : QMV_EHIP;
}

// Rows 0 .. M - 1 of a kernel that takes `rows` a workgroup from a.row0 on.
template <class Args>
qmv_status_t go_rows(const void *fn, Args &a, int rows, int threads, hipStream_t stream)
{
    void *args[] = {&a};
    for (long long r = 0; r < a.M; r += kMaxGroups * rows) {
        const long long left = ((long long)a.M - r + rows - 1) / rows;
        a.row0 = (int)r;
        const qmv_status_t s = go(fn, left < kMaxGroups ? left : kMaxGroups, threads, args, stream);
        if (s != QMV_OK)
            return s;
    }
    return QMV_OK;
}

long long piece_groups(long long pieces)
{
    const long long g = (pieces + 256 * kPieceUnroll - 1) / (256 * kPieceUnroll);
    return g < kMaxGroups ? g : kMaxGroups;
}

}  // namespace

extern "C" {

#define QMX_API __attribute__((visibility("default")))

QMX_API qmv_status_t qmx_rmsnorm(qmx_type_t xtype, const void *x, qmx_type_t rtype, const void *residual,
                                 void *residual_out, qmx_type_t wtype, const void *weight, float eps,
                                 qmx_fmt_t fmt, void *y, void *y_scales, int M, int K, hipStream_t stream)
{
    const qmv_status_t s = check_rmsnorm(xtype, x, rtype, residual, residual_out, wtype, weight, eps, fmt, y,
                                         y_scales, M, K);
    if (s != QMV_OK)
        return s;
    NormArgs a = {x, residual, weight, residual_out, y, y_scales, eps, (int)xtype, (int)rtype, (int)wtype, M, K, 0};
    int threads, rows;
    const void *fn = K % 8 != 0          ? norm_odd_kernel(K, threads, rows)
                     : fmt == QMX_BF16   ? norm_kernel<QMX_BF16>(M, K, threads, rows)
                     : fmt == QMX_Q8B32  ? norm_kernel<QMX_Q8B32>(M, K, threads, rows)
                                         : norm_kernel<QMX_MXFP4>(M, K, threads, rows);
    return go_rows(fn, a, rows, threads, stream);
}

QMX_API qmv_status_t qmx_router(qmx_type_t ltype, const void *logits, int M, int E, int top_k,
                                qmx_scoring_t scoring, int normalize, float scale, int32_t *ids,
                                float *weights, hipStream_t stream)
{
    const qmv_status_t s = check_router(ltype, logits, M, E, top_k, scoring, ids, weights);
    if (s != QMV_OK)
        return s;
    RouterArgs a = {logits, ids, weights, scale, (int)ltype, M, E, top_k, (int)scoring, normalize ? 1 : 0, 0};
    return go_rows(router_kernel(E), a, 4, 256, stream);
}

QMX_API qmv_status_t qmx_quantize(qmx_type_t xtype, const void *x, qmx_fmt_t fmt, void *codes, void *scales,
                                  long long rows, int K, hipStream_t stream)
{
    const qmv_status_t s = check_blocks(xtype, x, fmt, codes, scales, rows, K);
    if (s != QMV_OK)
        return s;
    long long pieces = rows * (K / 8);
    int xt = (int)xtype;
    const void *fn = fmt == QMX_MXFP4 ? (const void *)&qmx_quantize_kernel<QMX_MXFP4>
                                      : (const void *)&qmx_quantize_kernel<QMX_Q8B32>;
    void *args[] = {&x, &xt, &codes, &scales, &pieces};
    return go(fn, piece_groups(pieces), 256, args, stream);
}

QMX_API qmv_status_t qmx_dequantize(qmx_fmt_t fmt, const void *codes, const void *scales, qmx_type_t ytype,
                                    void *y, long long rows, int K, hipStream_t stream)
{
    const qmv_status_t s = check_blocks(ytype, y, fmt, codes, scales, rows, K);
    if (s != QMV_OK)
        return s;
    long long pieces = rows * (K / 8);
    int yt = (int)ytype;
    const void *fn = fmt == QMX_MXFP4 ? (const void *)&qmx_dequantize_kernel<QMX_MXFP4>
                                      : (const void *)&qmx_dequantize_kernel<QMX_Q8B32>;
    void *args[] = {&codes, &scales, &yt, &y, &pieces};
    return go(fn, piece_groups(pieces), 256, args, stream);
}

QMX_API const char *qmx_strerror(qmv_status_t status) { return status_text(status); }

}  // extern "C"
