// qmt.hip -- libqmt.so (include/qmt.h): the weight quantizer of the 8-bit
// floating-point products, the norm and rotation of query and key heads, and
// log probabilities, with their C ABI.
//
// Everything here is bound by the bytes it moves (or, for a few tokens, by a
// launch): one pass over the data, 16-byte accesses.  Times are a kernel's own:
// its median in a trace of ten calls with three sets of inputs in turn.
#include "qmt_host.hpp"
#include "qmx_values.hpp"

namespace {

using namespace qmt_host;

// ----------------------------------------------------------- square blocks
// One workgroup takes a block of 128 x 128: 16 lanes a row, 16 rows at a time,
// the whole block in registers between the maximum and the codes.  (A kernel for
// each type: 16-bit values take half the registers, and twice the waves are
// there to wait for memory.)  32 matrices of 2880 x 2880 from bf16 (797 MB) 170
// us, 4.7 TB/s, and back 142, 5.6 TB/s (148 with neighbours on different XCDs);
// with one kernel for all types, a maximum in fp32 and 64-bit quotients of all
// values below the normal range 257.
struct SquareBlock {
    long long at;        // of the thread's first value
    int k, row, N, K;    // its column and row in the matrix
    long long scale;     // the block's scale

    __device__ __forceinline__ SquareBlock(long long b, int N, int K) : N(N), K(K)
    {
        const int NB = (N + 127) / 128, KB = (K + 127) / 128;
        const long long line = b / KB, e = line / NB;          // block row of all matrices; matrix
        k = (int)(b - line * KB) * 128 + 8 * (threadIdx.x & 15);
        row = (int)(line - e * NB) * 128 + (int)(threadIdx.x >> 4);
        at = (e * N + row) * K + k;
        scale = b;
    }
    __device__ __forceinline__ bool has(int p) const { return k < K && row + 16 * p < N; }
    __device__ __forceinline__ size_t index(int p) const { return (size_t)(at + (long long)(16 * p) * K); }
};

// Workgroup b runs on XCD b % 8: blocks that are neighbours in a row go to one XCD, whose L2 has the
// cache lines that rows of odd multiples of 32 have in common.  (The grid is a multiple of 8.)
__device__ __forceinline__ long long first_square()
{
    return (long long)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
}

template <int XT>
__global__ __launch_bounds__(256) void qmt_quantize_weights_kernel(const void *x, void *codes, float *scales,
                                                                   long long blocks, int N, int K)
{
    __shared__ uint32_t part[2][16];
    int turn = 0;
    for (long long b = first_square(); b < blocks; b += gridDim.x, turn ^= 1) {
        const SquareBlock s(b, N, K);
        Raw8 r[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            r[p].a = r[p].b = make_uint4(0, 0, 0, 0);
            if (s.has(p)) r[p] = load_raw8(x, s.index(p), XT);
        }
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const uint32_t o = amax_bits8<XT>(r[p]);
            m = m > o ? m : o;
        }
        m = row16_max(m);
        if ((threadIdx.x & 15) == 0) part[turn][threadIdx.x >> 4] = m;
        __syncthreads();                                       // (the other buffer is the next block's)
#pragma unroll
        for (int i = 0; i < 16; ++i) m = m > part[turn][i] ? m : part[turn][i];
        const float d = f8_scale(m);
        if (threadIdx.x == 0) scales[s.scale] = d;
#pragma unroll
        for (int p = 0; p < 8; ++p)
            if (s.has(p)) {
                float v[8];
                raw_to_f32(r[p], XT, v);
                *(uint2 *)((uint8_t *)codes + s.index(p)) = f8_codes(v, d);
            }
    }
}

__global__ __launch_bounds__(256) void qmt_dequantize_weights_kernel(const void *codes, const float *scales, int yt,
                                                                     void *y, long long blocks, int N, int K)
{
    for (long long b = first_square(); b < blocks; b += gridDim.x) {
        const SquareBlock s(b, N, K);
        const float d = scales[s.scale];
        uint2 c[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            c[p] = make_uint2(0, 0);
            if (s.has(p)) c[p] = *(const uint2 *)((const uint8_t *)codes + s.index(p));
        }
#pragma unroll
        for (int p = 0; p < 8; ++p)
            if (s.has(p)) {
                float v[8];
                f8_values(c[p], d, v);
                store8(y, s.index(p), yt, v);
            }
    }
}

// ------------------------------------------------------ values of other lanes
// The value of lane ^ J, by the vector ALUs (a sort of 64 by way of LDS took
// three times as long).
template <int J> __device__ __forceinline__ uint32_t lane_xor(uint32_t v)
{
    if constexpr (J == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);     // quad_perm
    if constexpr (J == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
    if constexpr (J == 4)                                     // a half row mirrored (^ 7), a quad mirrored (^ 3)
        return (uint32_t)__builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true), 0x1B, 0xF, 0xF, true);
    if constexpr (J == 8) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, true);    // row_ror
    if constexpr (J == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return threadIdx.x & 16 ? r[0] : r[1];
    }
    if constexpr (J == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return threadIdx.x & 32 ? r[0] : r[1];
    }
}
template <int J> __device__ __forceinline__ uint64_t lane_xor(uint64_t v)
{
    return (uint64_t)lane_xor<J>((uint32_t)(v >> 32)) << 32 | lane_xor<J>((uint32_t)v);
}
template <int J> __device__ __forceinline__ double lane_xor(double v)
{
    return __builtin_bit_cast(double, lane_xor<J>(__builtin_bit_cast(uint64_t, v)));
}

// ------------------------------------------------- norm and rotation of heads
// Four consecutive values of a 32- or 16-bit type.
__device__ __forceinline__ uint4 load_raw4(const void *base, size_t i, int type)
{
    if (type == QMX_T_F32) return *(const uint4 *)((const float *)base + i);
    const uint2 h = *(const uint2 *)((const uint16_t *)base + i);
    return make_uint4(h.x, h.y, 0, 0);
}

__device__ __forceinline__ void raw4_to_f32(uint4 r, int type, float (&v)[4])
{
    if (type == QMX_T_F32) {
        v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
    } else if (type == QMX_T_BF16) {
        v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xFFFF0000u);
        v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xFFFF0000u);
    } else {
        const f16x2 a = __builtin_bit_cast(f16x2, r.x), b = __builtin_bit_cast(f16x2, r.y);
        v[0] = (float)a[0], v[1] = (float)a[1], v[2] = (float)b[0], v[3] = (float)b[1];
    }
}

__device__ __forceinline__ void store4(void *base, size_t i, int type, const float (&v)[4])
{
    if (type == QMX_T_F32)
        *(float4 *)((float *)base + i) = make_float4(v[0], v[1], v[2], v[3]);
    else if (type == QMX_T_BF16)
        *(uint2 *)((uint16_t *)base + i) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else
        *(uint2 *)((uint16_t *)base + i) = make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
}

// 1 / sqrt(m) to 2^-45 of itself: the instruction's 2^-23 or better, and one step of
// Newton's method.  (A square root and a division in 64 bits took as many
// instructions as all the rest of a head.)  0 and infinity have no step.
__device__ __forceinline__ double inverse_root(double m)
{
    const double r = __builtin_amdgcn_rsq(m);
    const double e = __builtin_fma(-m * r, r, 1.0);
    return r > 0.0 && r < __builtin_inf() ? __builtin_fma(0.5 * r, e, r) : r;
}

struct QkArgs {
    const void *x, *qw, *kw;
    const float *table;
    const int32_t *positions;
    void *q, *k;
    float eps;
    int xt, wt, yt, row, heads, all_heads, D, P, R, pairs, M;
    int per_token;       // groups of lanes a token takes
    long long group0;
    double inv_d;        // 1 / D
};

// G lanes take a head, lane j of them its values a = A .. A + 3 and b = B ..
// B + 3 such that the rotation pairs a[i] with b[i] (QMT_HALF), or neighbours
// in a and in b (QMT_PAIRS): no value crosses lanes.  A group takes UN heads of
// its token, all their loads given out at once; the lane's cosines, sines and
// weights serve them all.
//
// 8192 tokens of 40 heads of 128, bf16 (168 MB): 42 us, 4.0 TB/s.  A SIMD issues 14100
// vector instructions, 176 for four heads (one a group), 33 of them additions and
// products in 64 bits; the vector ALUs have work in 70% of a CU's cycles.  A square
// root and a division in 64 bits, sums by way of LDS, and types looked up at every
// load took 52.  (XT, YT, PAIRS: the types and the rotation,
// or -1 for those of the arguments, which serve calls of few heads: a launch's
// time whatever they do.)
template <int G, int UN, int XT, int YT, int PAIRS>
__global__ __launch_bounds__(256) void qmt_qk_norm_rope_kernel(const QkArgs a)
{
    const int xt = XT < 0 ? a.xt : XT, yt = YT < 0 ? a.yt : YT;
    const bool pairs = PAIRS < 0 ? a.pairs != 0 : PAIRS != 0;
    const int j = threadIdx.x & (G - 1);
    const long long g = a.group0 + (long long)blockIdx.x * (256 / G) + threadIdx.x / G;
    const unsigned t = (unsigned)g / (unsigned)a.per_token, h0 = (unsigned)g - t * (unsigned)a.per_token;
    if (t >= (unsigned)a.M) return;                            // whole groups
    const bool mine = 8 * j < a.D, turned = 8 * j < a.R, halves = turned && !pairs;
    const int A = halves ? 4 * j : 8 * j, B = halves ? A + a.R / 2 : A + 4;
    const int xs = xt == QMX_T_F32 ? 4 : 2, ys = yt == QMX_T_F32 ? 4 : 2;
    const uint8_t *const xr = (const uint8_t *)a.x + (size_t)t * a.row * xs;
    uint8_t *const qr = (uint8_t *)a.q + (size_t)t * (a.heads * a.D) * ys;
    uint8_t *const kr = (uint8_t *)a.k + (size_t)t * ((a.all_heads - a.heads) * a.D) * ys;
    uint4 xa[UN], xb[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        const int h = h0 + u * a.per_token;
        xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
        if (mine && h < a.all_heads) {
            xa[u] = load_raw4(xr, (unsigned)(h * a.D + A), xt);
            xb[u] = load_raw4(xr, (unsigned)(h * a.D + B), xt);
        }
    }
    const int p = a.positions[t];
    const bool inside = (unsigned)p < (unsigned)a.P;
    float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (turned && inside) {
        const float4 c4 = *(const float4 *)(a.table + (size_t)p * a.R + 4 * j);
        const float4 s4 = *(const float4 *)(a.table + (size_t)p * a.R + a.R / 2 + 4 * j);
        cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
        sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
    }
    float w[2][2][4];                                          // [queries, keys][a, b]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const void *const base = i ? a.kw : a.qw;
#pragma unroll
        for (int n = 0; n < 4; ++n) w[i][0][n] = w[i][1][n] = 1.0f;
        if (base && mine) {
            raw4_to_f32(load_raw4(base, A, a.wt), a.wt, w[i][0]);
            raw4_to_f32(load_raw4(base, B, a.wt), a.wt, w[i][1]);
        }
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        const int h = h0 + u * a.per_token;
        if (h >= a.all_heads) break;                           // whole groups
        float va[4], vb[4];
        raw4_to_f32(xa[u], xt, va);
        raw4_to_f32(xb[u], xt, vb);
        double s = 0.0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            s = __builtin_fma((double)va[n], (double)va[n], s);
            s = __builtin_fma((double)vb[n], (double)vb[n], s);
        }
        s += lane_xor<1>(s);
        s += lane_xor<2>(s);
        if constexpr (G > 4) s += lane_xor<4>(s);
        if constexpr (G > 8) s += lane_xor<8>(s);
        if constexpr (G > 16) s += lane_xor<16>(s);
        if constexpr (G > 32) s += lane_xor<32>(s);
        const double r = inverse_root(__builtin_fma(s, a.inv_d, (double)a.eps));
        const bool key = h >= a.heads;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            // (one rounding; fp32 products with the weights would be a second, for 1.5 to 4% of the time)
            va[n] = (float)((double)va[n] * r * (double)(key ? w[1][0][n] : w[0][0][n]));
            vb[n] = (float)((double)vb[n] * r * (double)(key ? w[1][1][n] : w[0][1][n]));
        }
        auto turn = [&](float &x, float &y, int i) {
            const float u0 = __builtin_fmaf(x, cs[i], -(y * sn[i])), v0 = __builtin_fmaf(y, cs[i], x * sn[i]);
            x = u0, y = v0;
        };
        if (turned) {
            if (pairs) {
                turn(va[0], va[1], 0), turn(va[2], va[3], 1);
                turn(vb[0], vb[1], 2), turn(vb[2], vb[3], 3);
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) turn(va[n], vb[n], n);
            }
        }
        if (!inside) {
#pragma unroll
            for (int n = 0; n < 4; ++n) va[n] = vb[n] = 0.0f;
        }
        if (mine) {
            const unsigned at = (unsigned)((key ? h - a.heads : h) * a.D);
            store4(key ? kr : qr, at + A, yt, va);
            store4(key ? kr : qr, at + B, yt, vb);
        }
    }
}

// A head each of any types, or 4 of these.
template <int G, int XT, int YT>
const void *qk_kernel4(bool pairs)
{
    return pairs ? (const void *)&qmt_qk_norm_rope_kernel<G, 4, XT, YT, 1>
                 : (const void *)&qmt_qk_norm_rope_kernel<G, 4, XT, YT, 0>;
}
template <int G, int XT>
const void *qk_kernel4(int yt, bool pairs)
{
    return yt == QMX_T_F32    ? qk_kernel4<G, XT, QMX_T_F32>(pairs)
           : yt == QMX_T_BF16 ? qk_kernel4<G, XT, QMX_T_BF16>(pairs)
                              : qk_kernel4<G, XT, QMX_T_F16>(pairs);
}
template <int G>
const void *qk_kernel(bool many, int xt, int yt, bool pairs)
{
    if (!many) return (const void *)&qmt_qk_norm_rope_kernel<G, 1, -1, -1, -1>;
    return xt == QMX_T_F32    ? qk_kernel4<G, QMX_T_F32>(yt, pairs)
           : xt == QMX_T_BF16 ? qk_kernel4<G, QMX_T_BF16>(yt, pairs)
                              : qk_kernel4<G, QMX_T_F16>(yt, pairs);
}
const void *qk_kernel(int D, bool many, int xt, int yt, bool pairs, int &G)
{
    G = D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64;
    return G == 4    ? qk_kernel<4>(many, xt, yt, pairs)
           : G == 8  ? qk_kernel<8>(many, xt, yt, pairs)
           : G == 16 ? qk_kernel<16>(many, xt, yt, pairs)
           : G == 32 ? qk_kernel<32>(many, xt, yt, pairs)
                     : qk_kernel<64>(many, xt, yt, pairs);
}

// ------------------------------------------------------- log probabilities
// One pass over the row.  A wave keeps its largest logit so far, m, and each
// lane the sums of exp(l - m) and exp(l - m) (l - m), which move with it; and
// the wave keeps the top entries it has seen.
//
// An entry is 64 bits, the logit's ordered bits over the inverted index, so
// that entries are all different and the larger one comes first; 0 is none.
__device__ __forceinline__ uint32_t order_bits(float l)
{
    const uint32_t b = __float_as_uint(l + 0.0f);             // -0 and 0 are equal
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;          // -FLT_MAX gives 0x00800000
}
__device__ __forceinline__ float order_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
// The value below l (there is none of -0's bits).
__device__ __forceinline__ float below(uint32_t k) { return order_value(k - (k == 0x80000000u ? 2u : 1u)); }
__device__ __forceinline__ uint64_t entry(float l, int index)
{
    return (uint64_t)order_bits(l) << 32 | (uint32_t)~index;
}

template <class T> __device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }
template <class T> __device__ __forceinline__ T smaller(T a, T b) { return a > b ? b : a; }

// Steps of a bitonic sort: lanes L and L ^ J in order, for J, J / 2, .. 1; runs of
// K lanes alternate in direction.
template <int K, int J, bool FALLING, class T>
__device__ __forceinline__ T sort_steps(T v)
{
    const T o = lane_xor<J>(v);
    const bool first = ((threadIdx.x & J) == 0) == (K == 64 || (threadIdx.x & K) == 0);
    v = first == FALLING ? larger(v, o) : smaller(v, o);
    if constexpr (J > 1)
        return sort_steps<K, J / 2, FALLING>(v);
    else
        return v;
}

// The wave's 64 values in order over its lanes: falling, or rising.
template <bool FALLING, class T>
__device__ __forceinline__ T wave_sort(T v)
{
    v = sort_steps<2, 1, FALLING>(v);
    v = sort_steps<4, 2, FALLING>(v);
    v = sort_steps<8, 4, FALLING>(v);
    v = sort_steps<16, 8, FALLING>(v);
    v = sort_steps<32, 16, FALLING>(v);
    return sort_steps<64, 32, FALLING>(v);
}

// The larger 64 of two sorted lists (a falling, b rising), falling.
template <class T>
__device__ __forceinline__ T wave_merge(T a, T b)
{
    return sort_steps<64, 32, true>(larger(a, b));
}

template <class T, class F>
__device__ __forceinline__ T wave_reduce(T v, F f)
{
    v = f(v, lane_xor<1>(v));
    v = f(v, lane_xor<2>(v));
    v = f(v, lane_xor<4>(v));
    v = f(v, lane_xor<8>(v));
    v = f(v, lane_xor<16>(v));
    return f(v, lane_xor<32>(v));
}

__device__ __forceinline__ double add(double x, double y) { return x + y; }

template <class T> __device__ __forceinline__ T lane_value(T v, int lane);
template <> __device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
template <> __device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane)
{
    return (uint64_t)lane_value((uint32_t)(v >> 32), lane) << 32 | lane_value((uint32_t)v, lane);
}

// How many of the lanes below this one have their bit in m.
__device__ __forceinline__ int lanes_below(unsigned long long m)
{
    return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// A wave's top entries, falling over the lanes, and entries waiting (in LDS)
// to be merged with them 64 at a time.
struct TopList {
    uint64_t kept;
    volatile uint64_t *wait;
    int waiting;

    __device__ __forceinline__ TopList(uint64_t *lds) : kept(0), wait(lds), waiting(0) {}

    // (all lanes call these)
    __device__ __forceinline__ void add(bool have, uint64_t e)
    {
        const unsigned long long m = __ballot(have);
        if (m == 0) return;
        if (have) wait[waiting + lanes_below(m)] = e;
        waiting += (int)__popcll(m);
    }
    // Merges, 64 at a time or what there is, until less than `left` wait.
    __device__ __forceinline__ void merge(int left)
    {
        const int lane = threadIdx.x & 63;
        while (waiting >= left && waiting > 0) {
            asm volatile("" ::: "memory");
            const int from = waiting > 64 ? waiting - 64 : 0;
            const uint64_t v = from + lane < waiting ? wait[from + lane] : 0;
            kept = wave_merge(kept, wave_sort<false>(v));
            waiting = from;
            asm volatile("" ::: "memory");
        }
    }
};

// exp(z), z <= 0 (1 for 0).
__device__ __forceinline__ float exp_below(float z) { return __builtin_amdgcn_exp2f(z * 1.4426950408889634f); }

// exp(d), -200 <= d <= 0, for sums that move to another maximum.  A row that rises
// moves them at every step by nearly the same d, so what a factor is off adds up
// (in fp32 to 8e-6 of the sums over 512 steps).  But d n is the rise in n steps, and
// what was summed before it counts e^-dn only: an error of d^8 / 8! in a factor comes
// to d^7 / 8! of the sums, 1.5e-8 at most with |d| <= log(2) / 2, so seven terms of the
// series do, of what is left of d without a power of two.  (1024 rows of 131071 bf16
// logits, top 5: a call 65.2 us, with the library's function 66.3; fp32 factors 65.8,
// without a top 44.7 for 46.8.)
__device__ __forceinline__ double factor(double d)
{
    const double n = __builtin_rint(d * 1.4426950408889634), r = __builtin_fma(n, -0.6931471805599453, d);
    double p = 1.0 / 5040.0;
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// The largest logit and the sums relative to it.
struct Sums {
    float m;
    double s, u;

    __device__ __forceinline__ void move(double d, double c)
    {
        u = c * (u + s * d);
        s *= c;
    }
    // relative to a larger (or equal) maximum.  (Sums of nothing are 0; below -200
    // nothing of them is left, and the difference may be infinite, or NaN.)
    __device__ __forceinline__ void rise(float to)
    {
        const double d = fmax((double)m - (double)to, -200.0);
        move(d, factor(d));
        m = to;
    }
};

// The sums of all lanes, relative to the largest of their maxima.  (A lane's N move
// there at once, each with one factor of its own, rounded as the terms' exponentials are.)
template <int N>
__device__ __forceinline__ Sums wave_join(Sums (&of)[N])
{
    float to = of[0].m;
#pragma unroll
    for (int i = 1; i < N; ++i) to = fmaxf(to, of[i].m);
    Sums all = {order_value(wave_reduce(order_bits(to), larger<uint32_t>)), 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = fmaxf(of[i].m - all.m, -200.0f);
        of[i].move((double)d, (double)exp_below(d));
        all.s += of[i].s;
        all.u += of[i].u;
    }
    all.s = wave_reduce(all.s, add);
    all.u = wave_reduce(all.u, add);
    return all;
}

struct LogArgs {
    const void *logits;
    const int32_t *tokens;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *top_ids;
    uint8_t *work;
    int lt, M, V, top_k, parts, steps;
    long long first;     // workgroup 0's place in the call
};

__device__ __forceinline__ float logit_at(const void *base, size_t i, int type)
{
    if (type == QMX_T_F32) return ((const float *)base)[i];
    const uint32_t h = ((const uint16_t *)base)[i];
    return type == QMX_T_BF16 ? __uint_as_float(h << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// The row's token and its logit, both on their way long before they are needed.
struct Given {
    bool inside;
    float l;

    __device__ __forceinline__ Given(const LogArgs &a, int row) : inside(false), l(0.0f)
    {
        if (a.logprobs) {
            const int t = a.tokens[row];
            inside = (unsigned)t < (unsigned)a.V;
            l = logit_at(a.logits, (size_t)row * a.V + (inside ? t : 0), a.lt);
        }
    }
};

// Row `row`'s outputs from its sums and list (one wave).
__device__ __forceinline__ void put_row(const LogArgs &a, int row, const Given &g, const Sums &s, uint64_t kept)
{
    const int lane = threadIdx.x & 63;
    const bool none = !(s.m > -__builtin_inff());
    const double logs = none ? 0.0 : s.m == __builtin_inff() ? __builtin_nan("") : log(s.s);
    auto logprob = [&](float l) { return l > -__builtin_inff() ? (float)((double)l - (double)s.m - logs) : -__builtin_inff(); };
    if (lane < a.top_k) {
        const uint32_t k = (uint32_t)(kept >> 32);
        a.top_ids[(size_t)row * a.top_k + lane] = kept ? (int)~(uint32_t)kept : -1;
        a.top_logprobs[(size_t)row * a.top_k + lane] = kept ? logprob(order_value(k)) : -__builtin_inff();
    }
    if (lane == 0) {
        if (a.entropy) a.entropy[row] = none ? 0.0f : (float)(logs - s.u / s.s);
        if (a.logprobs) a.logprobs[row] = g.inside ? logprob(g.l) : 0.0f;
    }
}

// A row's logits of a type: `groups` of 8 from its first whole 16 bytes on, and up
// to 7 before and 7 behind them, the rest.
template <int TYPE>
struct LogRow {
    static constexpr int SIZE = TYPE == QMX_T_F32 ? 4 : 2;
    const uint8_t *base;
    int head, groups, V;

    __device__ __forceinline__ LogRow(const LogArgs &a, int row) : V(a.V)
    {
        base = (const uint8_t *)a.logits + (size_t)row * a.V * SIZE;
        head = min((int)((16 - ((uintptr_t)base & 15)) & 15) / SIZE, V);
        groups = (V - head) / 8;
    }
    // index of group g's first logit
    __device__ __forceinline__ int at(int g) const { return head + 8 * g; }
    // group g's logits; masked ones behind the last
    __device__ __forceinline__ Raw8 load(int g) const
    {
        constexpr uint32_t masked = TYPE == QMX_T_F32 ? 0xFF800000u : TYPE == QMX_T_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
        Raw8 r;
        r.a = r.b = make_uint4(masked, masked, masked, masked);
        if (g < groups) {
            const uint4 *const p = (const uint4 *)(base + (long long)at(g) * SIZE);
            r.a = p[0];
            if constexpr (SIZE == 4) r.b = p[1];
        }
        return r;
    }
    // lane i < 14 of a wave: the i-th of the rest, and its index
    __device__ __forceinline__ float rest(int i, int &index) const
    {
        index = i < head ? i : at(groups) + i - head;
        return i < 14 && index < V ? logit_at(base, index, TYPE) : -__builtin_inff();
    }
};

// What a workgroup leaves of a part for the join: its sums (wave 0, any lane) and 64 entries.
template <bool TOP>
__device__ __forceinline__ void put_part(const LogArgs &a, long long place, const Sums &s, uint64_t e)
{
    const int lane = threadIdx.x & 63;
    if (lane == 0) {
        double *const out = (double *)(a.work + place * kListSums);
        out[0] = s.s;
        out[1] = s.u;
        *(float *)(out + 2) = s.m;
    }
    if constexpr (TOP) ((uint64_t *)(a.work + (long long)a.M * a.parts * kListSums))[place * 64 + lane] = e;
}

// A short part of a row, a group of 8 for each lane of 4 waves at most: first the
// largest logit of the workgroup and a bound of its top entries -- of the waves'
// 16 largest lanes the top_k-th: as many logits are at least that -- then the
// sums and what is no smaller than the bound, hardly more than top_k entries.
// (201088 logits, top 20, in 99 parts: 4.8 us, and 3.0 without a top.)
template <int TYPE, bool TOP>
__global__ __launch_bounds__(256) void qmt_logprobs_part_kernel(const LogArgs a)
{
    constexpr int NW = 4;
    __shared__ uint64_t few[64], wait[NW][128];
    __shared__ uint32_t lanes[64];
    __shared__ double part_s[NW], part_u[NW];
    __shared__ int count;
    const float low = -__builtin_inff();
    const long long place = a.first + blockIdx.x;
    const int row = (int)(place / a.parts), part = (int)(place - (long long)row * a.parts);
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const LogRow<TYPE> r(a, row);
    // (as many for each part, and for each of its waves: with all of a part's few in one wave the bound
    // would be that wave's 16 lanes only, or none)
    const int per = (r.groups + a.parts - 1) / a.parts, each = (per + NW - 1) / NW;
    const int g = lane < each && w * each + lane < per ? part * per + w * each + lane : r.groups;
    const Raw8 raw = r.load(g);
    // (the rest: with the last wave of the first part)
    int rest_at = 0;
    const float rest = part == 0 && w == NW - 1 ? r.rest(lane, rest_at) : low;
    if (tid == 0) count = 0;
    float l[8], big = rest > low ? rest : low;
    raw_to_f32(raw, TYPE, l);
#pragma unroll
    for (int j = 0; j < 8; ++j) big = l[j] > big ? l[j] : big;                 // (NaN is no maximum)
    const uint32_t mine = big > low ? order_bits(big) : 0u;
    if constexpr (TOP) {
        const uint32_t order = wave_sort<true>(mine);
        if (lane < 16) lanes[16 * w + lane] = order;
    } else {
        const uint32_t m = wave_reduce(mine, larger<uint32_t>);
        if (lane < 16) lanes[16 * w + lane] = m;
    }
    __syncthreads();
    const uint32_t sorted = TOP ? wave_sort<true>(lanes[lane]) : wave_reduce(lanes[lane], larger<uint32_t>);
    const uint32_t top = lane_value(sorted, 0);
    const float m = top ? order_value(top) : low;
    double s = 0.0;
    float u = 0.0f;
    auto term = [&](float v) {
        // (below -200 the exponential is 0 in fp32; NaN, both -infinity among it, gives -200 too)
        const float z = __builtin_amdgcn_fmed3f(v - m, -200.0f, 0.0f), e = exp_below(z);
        s += (double)e;                                       // (a largest logit's 1 would take the digits of an fp32 sum)
        u = __builtin_fmaf(e, z, u);
    };
    term(rest);
#pragma unroll
    for (int j = 0; j < 8; ++j) term(l[j]);
    s = wave_reduce(s, add);
    const double su = wave_reduce((double)u, add);
    if (lane == 0) part_s[w] = s, part_u[w] = su;
    uint64_t mine64 = 0;
    float tau = low;
    if constexpr (TOP) {
        const uint32_t bound = lane_value(sorted, a.top_k - 1);
        tau = bound ? order_value(bound) : -__FLT_MAX__;
        auto put = [&](float v, int index) {
            const bool have = v >= tau;
            const unsigned long long b = __ballot(have);
            if (b != 0) {
                int at = 0;
                if (lane == 0) at = atomicAdd(&count, (int)__popcll(b));
                at = __builtin_amdgcn_readfirstlane(at) + lanes_below(b);
                if (have && at < 64) few[at] = entry(v, index);
            }
        };
        put(rest, rest_at);
#pragma unroll
        for (int j = 0; j < 8; ++j) put(l[j], r.at(g) + j);
    }
    __syncthreads();
    if constexpr (TOP) {
        const int n = count;
        if (n > 64) {
            // (many logits that are all alike)
            TopList list(wait[w]);
            list.add(rest >= tau, entry(rest, rest_at));
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                float v = l[0];
#pragma unroll
                for (int q = 1; q < 8; ++q) v = q == j ? l[q] : v;
                list.add(v >= tau, entry(v, r.at(g) + j));
                list.merge(64);
            }
            list.merge(1);
            wait[w][lane] = list.kept;
            __syncthreads();
            if (w == 0) {
                mine64 = list.kept;
                for (int i = 1; i < NW; ++i) mine64 = wave_merge(mine64, wait[i][63 - lane]);
            }
        } else if (w == 0) {
            mine64 = lane < n ? few[lane] : 0;
        }
    }
    if (w == 0) {
        Sums all = {m, 0.0, 0.0};
        for (int i = 0; i < NW; ++i) all.s += part_s[i], all.u += part_u[i];
        put_part<TOP>(a, place, all, mine64);
    }
}

// A row, or a long part of one: 8 waves, `steps` groups of 8 logits a lane of
// them, two always on their way; the rest of the row is one more step, the last,
// of the first part's first wave.  (A part may have one step only: the second load
// is of masked logits then.)  1024 rows of 131071 bf16 logits, top 5 (268 MB): 74 us,
// 3.6 TB/s.  The vector ALUs bound it, at work in every cycle of a CU's, with 17
// instructions a logit; without a top list it takes two thirds.
template <int TYPE, bool TOP>
__global__ __launch_bounds__(512) void qmt_logprobs_kernel(const LogArgs a)
{
    constexpr int NW = 8;
    __shared__ uint64_t wait[NW][64 + 4 * 64];
    __shared__ uint32_t first_top[NW * 8];
    __shared__ Sums part_sums[NW];
    const float low = -__builtin_inff();
    const long long place = a.first + blockIdx.x;
    const int row = (int)(place / a.parts), part = (int)(place - (long long)row * a.parts);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const LogRow<TYPE> r(a, row);
    const Given given(a, row);
    auto uniform = [](float v) { return __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane(__float_as_uint(v))); };
    Sums sums = {low, 0.0, 0.0};                               // m is the wave's
    TopList top(wait[w]);
    float tau = low;                                           // only logits above it can be among the top
    auto biggest = [&](const float (&l)[8]) {                  // (NaN is no maximum)
        float big = low;
#pragma unroll
        for (int j = 0; j < 8; ++j) big = l[j] > big ? l[j] : big;
        return big;
    };
    auto largest = [&](const float (&l)[8]) {
        const float big = biggest(l);
        return big > low ? order_bits(big) : 0u;
    };
    auto step = [&](const float (&l)[8], int index) {
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = l[j] - sums.m;
        const float top_z = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
        if (__any(top_z >= 0.0f)) {
            // a logit as large as the largest so far: its 1 would take the digits
            // of the others in an fp32 sum, so it is added here and the others
            // as ever
            const uint32_t k = wave_reduce(largest(l), larger<uint32_t>);
            sums.rise(uniform(larger(sums.m, order_value(k))));
            int ones = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                z[j] = l[j] - sums.m;
                ones += z[j] == 0.0f;
                z[j] = z[j] == 0.0f ? low : z[j];
            }
            sums.s += (double)ones;
        }
        float e[8], u = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // (below -200 the exponential is 0 in fp32; NaN gives -200 too)
            z[j] = __builtin_amdgcn_fmed3f(z[j], -200.0f, 0.0f);
            e[j] = exp_below(z[j]);
            u = __builtin_fmaf(e[j], z[j], u);
        }
        sums.s += (double)(((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
        sums.u += (double)u;
        if constexpr (TOP) {
            // (rounded differences keep the order, equal ones may stand for unequal
            // logits; where the bound's is -infinity -- no bound yet, a logit of
            // +infinity, a difference past fp32's range -- the logits themselves say)
            const float zz = top_z < 0.0f ? top_z : 0.0f, bound = tau - sums.m;
            if (bound > low ? __any(zz >= bound) : __any(biggest(l) > tau)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) top.add(l[j] > tau, entry(l[j], index + j));
                if (top.waiting >= 64) top.merge(64);
#pragma unroll
                for (int j = 4; j < 8; ++j) top.add(l[j] > tau, entry(l[j], index + j));
                if (top.waiting >= 32) {
                    top.merge(32);
                    // (not within a step: the same logit at a lower index may come after)
                    const uint32_t k = (uint32_t)(lane_value(top.kept, a.top_k - 1) >> 32);
                    if (k) tau = uniform(fmaxf(tau, order_value(k)));
                }
            }
        }
    };
    const int s0 = part * a.steps, s1 = s0 + a.steps;
    auto load = [&](int s) { return r.load(s < s1 ? s * (NW * 64) + tid : r.groups); };
    auto at = [&](int s) { return r.at(s * (NW * 64) + tid); };
    Raw8 raw0 = load(s0), raw1 = load(s0 + 1);
    if constexpr (TOP) {
        // the top_k-th largest of the waves' 8 largest lanes of the first step:
        // as many logits of the row are at least that
        float l[8];
        raw_to_f32(raw0, TYPE, l);
        const uint32_t order = wave_sort<true>(largest(l));
        if (lane < 8) first_top[8 * w + lane] = order;
        __syncthreads();
        const uint32_t k = lane_value(wave_sort<true>(first_top[lane]), a.top_k - 1);
        tau = k == 0u ? low : uniform(below(k));
    }
    for (int s = s0; s < s1; s += 2) {
        float l[8];
        raw_to_f32(raw0, TYPE, l);
        raw0 = load(s + 2);
        step(l, at(s));
        raw_to_f32(raw1, TYPE, l);
        raw1 = load(s + 3);
        if (s + 1 < s1) step(l, at(s + 1));
    }
    if (part == 0 && w == 0) {
        int index = 0;
        const float odd = r.rest(lane, index);
        const float l[8] = {odd, low, low, low, low, low, low, low};
        // (these may have the same logit at a lower index)
        if (TOP && tau > low) tau = uniform(below(order_bits(tau)));
        step(l, index);
    }
    sums.s = wave_reduce(sums.s, add);
    sums.u = wave_reduce(sums.u, add);
    if (lane == 0) part_sums[w] = sums;
    uint64_t kept = 0;
    if constexpr (TOP) {
        top.merge(1);
        kept = top.kept;
        wait[w][lane] = kept;
    }
    __syncthreads();
    if (w != 0) return;
    Sums each[1] = {lane < NW ? part_sums[lane] : Sums{low, 0.0, 0.0}};
    const Sums all = wave_join(each);
    if constexpr (TOP)
        for (int i = 1; i < NW; ++i) kept = wave_merge(kept, wait[i][63 - lane]);
    if (a.parts == 1)
        put_row(a, row, given, all, kept);
    else
        put_part<TOP>(a, place, all, kept);
}

// The parts of a row joined: one workgroup a row, all entries in registers.  The
// top_k-th largest of the parts' maxima (of fewer parts, of the waves' 8 largest
// lanes, or of a wave's lanes) bounds the row's top_k-th logit from below, and
// what is no smaller is hardly more than top_k entries, which one wave sorts: 5.0
// us for 99 parts and top 20.  (With each wave's own bound only, 11.4.)
template <bool TOP>
__global__ __launch_bounds__(64 * kJoinWaves) void qmt_logprobs_join_kernel(const LogArgs a)
{
    constexpr int NW = kJoinWaves, PER = kMaxParts / NW;       // lists a wave takes at most
    __shared__ uint64_t few[64], wait[TOP ? NW : 1][128];
    __shared__ uint32_t bound[NW], lanes[64];
    __shared__ int count;
    const int row = (int)(a.first + blockIdx.x), tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const long long list0 = (long long)row * a.parts;
    uint64_t e[PER];
    if constexpr (TOP) {
        const uint64_t *const in = (const uint64_t *)(a.work + (long long)a.M * a.parts * kListSums) + list0 * 64;
#pragma unroll
        for (int i = 0; i < PER; ++i) e[i] = w + NW * i < a.parts ? in[(w + NW * i) * 64 + lane] : 0;
    }
    // (the sums are wave 0's, the maxima every wave's, for its bound; loaded here, before anything is waited for)
    Sums half[kMaxParts / 64];                                 // lane l's parts l, l + 64, ..
#pragma unroll
    for (int i = 0; i < kMaxParts / 64; ++i) {
        const int p = min(lane + 64 * i, a.parts - 1);
        const double *const at = (const double *)(a.work + (list0 + p) * kListSums);
        half[i] = Sums{*(const float *)(at + 2), at[0], at[1]};
    }
    const Given given(a, row);
    if (tid == 0) count = 0;
    uint64_t kept = 0;
    if constexpr (TOP) {
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) big = larger(big, (uint32_t)(e[i] >> 32));
        if (a.parts >= a.top_k) {
            float m = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < kMaxParts / 64; ++i)
                if (lane + 64 * i < a.parts) m = fmaxf(m, half[i].m);
            big = m > -__builtin_inff() ? order_bits(m) : 0u;
        }
        big = wave_sort<true>(big);
        if (lane == a.top_k - 1) bound[w] = big;
        if (lane < 64 / NW) lanes[64 / NW * w + lane] = big;
        __syncthreads();
        uint32_t tau = 1;                                      // (0 is no entry)
        if (a.parts < a.top_k) tau = larger(tau, lane_value(wave_sort<true>(lanes[lane]), a.top_k - 1));
#pragma unroll
        for (int i = 0; i < NW; ++i) tau = larger(tau, bound[i]);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool have = (uint32_t)(e[i] >> 32) >= tau;
            const unsigned long long m = __ballot(have);
            if (m != 0) {
                int at = 0;
                if (lane == 0) at = atomicAdd(&count, (int)__popcll(m));
                at = __builtin_amdgcn_readfirstlane(at) + lanes_below(m);
                if (have && at < 64) few[at] = e[i];
            }
        }
        __syncthreads();
        const int n = count;
        if (n <= 64) {
            if (w == 0) kept = wave_sort<true>(lane < n ? few[lane] : 0);
        } else {
            // (many logits that are all alike, or the top ones all in one lane's)
            TopList top(wait[w]);
#pragma unroll 1
            for (int i = 0; i < PER; ++i) {
                uint64_t v = e[0];
#pragma unroll
                for (int q = 1; q < PER; ++q) v = q == i ? e[q] : v;
                top.add((uint32_t)(v >> 32) >= tau, v);
                top.merge(64);
            }
            top.merge(1);
            kept = top.kept;
            wait[w][lane] = kept;
            __syncthreads();
            if (w == 0)
                for (int i = 1; i < NW; ++i) kept = wave_merge(kept, wait[i][63 - lane]);
        }
    }
    if (w != 0) return;
#pragma unroll
    for (int i = 0; i < kMaxParts / 64; ++i)
        if (lane + 64 * i >= a.parts) half[i] = Sums{-__builtin_inff(), 0.0, 0.0};
    const Sums sums = wave_join(half);
    put_row(a, row, given, sums, kept);
}

template <int TYPE, bool TOP>
const void *logprobs_kernel(const LogprobPlan &p)
{
    return p.part ? (const void *)&qmt_logprobs_part_kernel<TYPE, TOP> : (const void *)&qmt_logprobs_kernel<TYPE, TOP>;
}

template <bool TOP>
const void *logprobs_kernel(int type, const LogprobPlan &p)
{
    return type == QMX_T_F32    ? logprobs_kernel<QMX_T_F32, TOP>(p)
           : type == QMX_T_BF16 ? logprobs_kernel<QMX_T_BF16, TOP>(p)
                                : logprobs_kernel<QMX_T_F16, TOP>(p);
}

// HIP limits a launch to 2^32 threads: beyond this many workgroups a kernel
// loops or is launched again.
constexpr long long kMaxGroups = 1LL << 20;

qmv_status_t go(const void *fn, long long groups, void **args, hipStream_t stream, int threads = 256)
{
    return hipLaunchKernel(fn, dim3((unsigned)groups), dim3((unsigned)threads), args, 0, stream) == hipSuccess
               ? QMV_OK
               : QMV_EHIP;
}

// Workgroups 0 .. n - 1 of a kernel whose first one's number is a.*FIRST times `unit`.
template <class Args>
qmv_status_t go_all(const void *fn, Args &a, long long Args::*first, long long unit, long long n, hipStream_t stream,
                    int threads = 256)
{
    void *args[] = {&a};
    for (long long g = 0; g < n; g += kMaxGroups) {
        a.*first = g * unit;
        const qmv_status_t s = go(fn, n - g < kMaxGroups ? n - g : kMaxGroups, args, stream, threads);
        if (s != QMV_OK)
            return s;
    }
    return QMV_OK;
}

long long square_groups(long long blocks) { return blocks < kMaxGroups ? (blocks + 7) / 8 * 8 : kMaxGroups; }

}  // namespace

extern "C" {

#define QMT_API __attribute__((visibility("default")))

QMT_API qmv_status_t qmt_quantize_weights(qmx_type_t xtype, const void *x, void *codes, float *scales, int E, int N,
                                          int K, hipStream_t stream)
{
    const qmv_status_t s = check_weights(xtype, x, codes, scales, E, N, K);
    if (s != QMV_OK)
        return s;
    long long blocks = (long long)E * ((N + 127) / 128) * ((K + 127) / 128);
    void *args[] = {&x, &codes, &scales, &blocks, &N, &K};
    const void *const fn = xtype == QMX_T_F32 ? (const void *)&qmt_quantize_weights_kernel<QMX_T_F32>
                           : xtype == QMX_T_BF16 ? (const void *)&qmt_quantize_weights_kernel<QMX_T_BF16>
                                                 : (const void *)&qmt_quantize_weights_kernel<QMX_T_F16>;
    return go(fn, square_groups(blocks), args, stream);
}

QMT_API qmv_status_t qmt_dequantize_weights(const void *codes, const float *scales, qmx_type_t ytype, void *y, int E,
                                            int N, int K, hipStream_t stream)
{
    const qmv_status_t s = check_weights(ytype, y, codes, scales, E, N, K);
    if (s != QMV_OK)
        return s;
    long long blocks = (long long)E * ((N + 127) / 128) * ((K + 127) / 128);
    int yt = (int)ytype;
    void *args[] = {&codes, &scales, &yt, &y, &blocks, &N, &K};
    return go((const void *)&qmt_dequantize_weights_kernel, square_groups(blocks), args, stream);
}

QMT_API qmv_status_t qmt_qk_norm_rope(qmx_type_t xtype, const void *x, int row, int heads, int kv_heads, int D,
                                      const float *table, int P, int R, const int32_t *positions, qmx_type_t wtype,
                                      const void *q_weight, const void *k_weight, float eps, qmt_rotation_t rotation,
                                      qmx_type_t ytype, void *q, void *k, int M, hipStream_t stream)
{
    const qmv_status_t s = check_qk(xtype, x, row, heads, kv_heads, D, table, P, R, positions, wtype, q_weight,
                                    k_weight, eps, rotation, ytype, q, k, M);
    if (s != QMV_OK)
        return s;
    const int all = heads + kv_heads;
    QkArgs a = {x, q_weight, k_weight, table, positions, q, k, eps, (int)xtype, (int)wtype, (int)ytype, row, heads, all,
                D, P, R, rotation == QMT_PAIRS ? 1 : 0, M, all, 0, 1.0 / D};
    int G;
    // (one head a group and four, us: 40 heads of 128, bf16: 512 tokens 6.0 and 6.3, 1024 10.4 and 8.9)
    const bool many = (long long)M * all >= 32768;
    const void *fn = qk_kernel(D, many, (int)xtype, (int)ytype, rotation == QMT_PAIRS, G);
    if (many) a.per_token = (all + 3) / 4;
    return go_all(fn, a, &QkArgs::group0, 256 / G, ((long long)M * a.per_token * G + 255) / 256, stream);
}

QMT_API long long qmt_logprobs_workspace(int M, int V, int top_k) { return logprobs_workspace(M, V, top_k); }

QMT_API qmv_status_t qmt_logprobs(qmx_type_t ltype, const void *logits, int M, int V, const int32_t *tokens, int top_k,
                                  float *logprobs, float *entropy, int32_t *top_ids, float *top_logprobs,
                                  void *workspace, hipStream_t stream)
{
    const qmv_status_t s = check_logprobs(ltype, logits, M, V, tokens, top_k, logprobs, entropy, top_ids, top_logprobs);
    if (s != QMV_OK)
        return s;
    const LogprobPlan p = plan_logprobs(M, V);
    if (p.join && (!workspace || !aligned(workspace, 16)))
        return QMV_EINVAL;
    LogArgs a = {logits, tokens, logprobs, entropy, top_logprobs, top_ids, (uint8_t *)workspace, (int)ltype, M, V,
                 top_k, p.parts, p.steps, 0};
    const void *fn = top_k ? logprobs_kernel<true>(ltype, p) : logprobs_kernel<false>(ltype, p);
    const void *join = top_k ? (const void *)&qmt_logprobs_join_kernel<true>
                             : (const void *)&qmt_logprobs_join_kernel<false>;
    const qmv_status_t st = go_all(fn, a, &LogArgs::first, 1, (long long)M * p.parts, stream, p.threads);
    if (st != QMV_OK || !p.join)
        return st;
    return go_all(join, a, &LogArgs::first, 1, M, stream, 64 * kJoinWaves);
}

QMT_API const char *qmt_strerror(qmv_status_t status) { return status_text(status); }

}  // extern "C"
