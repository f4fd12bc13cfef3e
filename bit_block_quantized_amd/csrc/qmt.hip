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
// the whole block in registers between the maximum and the codes.
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

__global__ __launch_bounds__(256) void qmt_quantize_weights_kernel(const void *x, int xt, void *codes, float *scales,
                                                                   long long blocks, int N, int K)
{
    __shared__ uint32_t part[2][16];
    int turn = 0;
    for (long long b = blockIdx.x; b < blocks; b += gridDim.x, turn ^= 1) {
        const SquareBlock s(b, N, K);
        Raw8 r[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            r[p].a = r[p].b = make_uint4(0, 0, 0, 0);
            if (s.has(p)) r[p] = load_raw8(x, s.index(p), xt);
        }
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            raw_to_f32(r[p], xt, v);
            const uint32_t o = amax_bits8(v);
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
                raw_to_f32(r[p], xt, v);
                *(uint2 *)((uint8_t *)codes + s.index(p)) = f8_codes(v, d);
            }
    }
}

__global__ __launch_bounds__(256) void qmt_dequantize_weights_kernel(const void *codes, const float *scales, int yt,
                                                                     void *y, long long blocks, int N, int K)
{
    for (long long b = blockIdx.x; b < blocks; b += gridDim.x) {
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

struct QkArgs {
    const void *x, *qw, *kw;
    const float *table;
    const int32_t *positions;
    void *q, *k;
    float eps;
    int xt, wt, yt, row, heads, all_heads, D, P, R, pairs, M;
    int per_token;       // groups of lanes a token takes
    long long group0;
};

// G lanes take a head, lane j of them its values a = A .. A + 3 and b = B ..
// B + 3 such that the rotation pairs a[i] with b[i] (QMT_HALF), or neighbours
// in a and in b (QMT_PAIRS): no value crosses lanes.  A group takes UN heads of
// its token, all their loads given out at once; the lane's cosines, sines and
// weights serve them all.
template <int G, int UN>
__global__ __launch_bounds__(256) void qmt_qk_norm_rope_kernel(const QkArgs a)
{
    const int j = threadIdx.x & (G - 1);
    const long long g = a.group0 + (long long)blockIdx.x * (256 / G) + threadIdx.x / G;
    const unsigned t = (unsigned)g / (unsigned)a.per_token, h0 = (unsigned)g - t * (unsigned)a.per_token;
    if (t >= (unsigned)a.M) return;                            // whole groups
    const bool mine = 8 * j < a.D, turned = 8 * j < a.R, halves = turned && !a.pairs;
    const int A = halves ? 4 * j : 8 * j, B = halves ? A + a.R / 2 : A + 4;
    uint4 xa[UN], xb[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        const int h = h0 + u * a.per_token;
        xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
        if (mine && h < a.all_heads) {
            const size_t at = (size_t)t * a.row + (size_t)h * a.D;
            xa[u] = load_raw4(a.x, at + A, a.xt);
            xb[u] = load_raw4(a.x, at + B, a.xt);
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
        raw4_to_f32(xa[u], a.xt, va);
        raw4_to_f32(xb[u], a.xt, vb);
        double s = 0.0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            s = __builtin_fma((double)va[n], (double)va[n], s);
            s = __builtin_fma((double)vb[n], (double)vb[n], s);
        }
#pragma unroll
        for (int d = G / 2; d >= 1; d >>= 1) s += __shfl_xor(s, d);
        const double r = 1.0 / __builtin_sqrt(s / (double)a.D + (double)a.eps);
        const bool key = h >= a.heads;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            va[n] = (float)((double)va[n] * r * (double)(key ? w[1][0][n] : w[0][0][n]));
            vb[n] = (float)((double)vb[n] * r * (double)(key ? w[1][1][n] : w[0][1][n]));
        }
        auto turn = [&](float &x, float &y, int i) {
            const float u0 = __builtin_fmaf(x, cs[i], -(y * sn[i])), v0 = __builtin_fmaf(y, cs[i], x * sn[i]);
            x = u0, y = v0;
        };
        if (turned) {
            if (a.pairs) {
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
            void *const base = key ? a.k : a.q;
            const int H = key ? a.all_heads - a.heads : a.heads;
            const size_t at = ((size_t)t * H + (key ? h - a.heads : h)) * a.D;
            store4(base, at + A, a.yt, va);
            store4(base, at + B, a.yt, vb);
        }
    }
}

template <int UN>
const void *qk_kernel(int D, int &G)
{
    if (D <= 32) { G = 4; return (const void *)&qmt_qk_norm_rope_kernel<4, UN>; }
    if (D <= 64) { G = 8; return (const void *)&qmt_qk_norm_rope_kernel<8, UN>; }
    if (D <= 128) { G = 16; return (const void *)&qmt_qk_norm_rope_kernel<16, UN>; }
    if (D <= 256) { G = 32; return (const void *)&qmt_qk_norm_rope_kernel<32, UN>; }
    G = 64;
    return (const void *)&qmt_qk_norm_rope_kernel<64, UN>;
}

// ------------------------------------------------------- log probabilities
// One pass over the row: a thread keeps the largest of its logits, m, and the
// sums of exp(l - m) and exp(l - m) (l - m), which move with it; a wave keeps
// the top entries it has seen.
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
__device__ __forceinline__ uint64_t entry(float l, int index)
{
    return (uint64_t)order_bits(l) << 32 | (uint32_t)~index;
}

template <class T> __device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }
template <class T> __device__ __forceinline__ T smaller(T a, T b) { return a > b ? b : a; }

// The wave's 64 values in order over its lanes: falling, or rising.
template <bool FALLING, class T>
__device__ __forceinline__ T wave_sort(T v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j >= 1; j >>= 1) {
            const T o = __shfl_xor(v, j);
            const bool first = ((lane & j) == 0) == ((lane & k) == 0 || k == 64);
            v = first == FALLING ? larger(v, o) : smaller(v, o);
        }
    return v;
}

// The larger 64 of two sorted lists (a falling, b rising), falling.
template <class T>
__device__ __forceinline__ T wave_merge(T a, T b)
{
    const int lane = threadIdx.x & 63;
    T v = larger(a, b);
#pragma unroll
    for (int j = 32; j >= 1; j >>= 1) {
        const T o = __shfl_xor(v, j);
        v = (lane & j) == 0 ? larger(v, o) : smaller(v, o);
    }
    return v;
}

// A wave's top entries, falling over the lanes, and entries waiting (in LDS,
// less than 64 between calls) to be merged with them 64 at a time.
struct TopList {
    uint64_t kept;
    volatile uint64_t *wait;     // [128]
    int waiting;

    __device__ __forceinline__ TopList(uint64_t *lds) : kept(0), wait(lds), waiting(0) {}

    __device__ __forceinline__ void merge()
    {
        const int lane = threadIdx.x & 63;
        asm volatile("" ::: "memory");
        const uint64_t v = lane < waiting ? wait[lane] : 0;
        kept = wave_merge(kept, wave_sort<false>(v));
        waiting -= 64;
        if (waiting > 0) {
            const uint64_t rest = wait[64 + lane];
            if (lane < waiting) wait[lane] = rest;
        } else {
            waiting = 0;
        }
        asm volatile("" ::: "memory");
    }
    // (all lanes call it)
    __device__ __forceinline__ void add(bool have, uint64_t e)
    {
        const unsigned long long m = __ballot(have);
        if (m == 0) return;
        const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
        if (have) wait[waiting + before] = e;
        waiting += (int)__popcll(m);
        if (waiting >= 64) merge();
    }
    __device__ __forceinline__ void finish()
    {
        if (waiting > 0) merge();
    }
};

// The largest logit and the sums relative to it.
struct Sums {
    float m;
    double s, u;

    // relative to a larger (or equal) maximum
    __device__ __forceinline__ void move(float to)
    {
        const float d = m > -__builtin_inff() ? m - to : 0.0f;        // (nothing so far: sums are 0)
        const double c = m > -__builtin_inff() ? (double)exp2f(d * 1.4426950408889634f) : 0.0;
        u = c * (u + s * (double)d);
        s *= c;
        m = to;
    }
};

__device__ __forceinline__ Sums wave_sums(Sums a)
{
    float m = a.m;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    a.move(m);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        a.s += __shfl_xor(a.s, d);
        a.u += __shfl_xor(a.u, d);
    }
    return a;
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

constexpr int kLogWaves = 4;

struct LogShared {
    uint64_t wait[kLogWaves][128];
    uint64_t lists[kLogWaves][64];
    Sums sums[kLogWaves];
};

// The waves' sums and lists -> the workgroup's, in wave 0.
template <bool TOP>
__device__ __forceinline__ void join_waves(LogShared &sh, Sums &a, uint64_t &kept)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    if (lane == 0) sh.sums[w] = a;
    if constexpr (TOP) sh.lists[w][lane] = kept;
    __syncthreads();
    if (w != 0) return;
    a = sh.sums[0];
    float m = a.m;
#pragma unroll
    for (int i = 1; i < kLogWaves; ++i) m = fmaxf(m, sh.sums[i].m);
    a.move(m);
#pragma unroll
    for (int i = 1; i < kLogWaves; ++i) {
        Sums o = sh.sums[i];
        o.move(m);
        a.s += o.s;
        a.u += o.u;
    }
    if constexpr (TOP) {
#pragma unroll
        for (int i = 1; i < kLogWaves; ++i) kept = wave_merge(kept, sh.lists[i][63 - lane]);
    }
}

__device__ __forceinline__ float logit_at(const void *base, size_t i, int type)
{
    if (type == QMX_T_F32) return ((const float *)base)[i];
    const uint32_t h = ((const uint16_t *)base)[i];
    return type == QMX_T_BF16 ? __uint_as_float(h << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// Row `row`'s outputs from its sums and list (wave 0).
__device__ __forceinline__ void put_row(const LogArgs &a, int row, const Sums &s, uint64_t kept)
{
    const int lane = threadIdx.x & 63;
    const double inf = __builtin_inf();
    const bool none = !(s.m > -__builtin_inff());
    const double logs = none ? 0.0 : s.m == __builtin_inff() ? __builtin_nan("") : log(s.s);
    auto logprob = [&](float l) { return l > -__builtin_inff() ? (float)((double)l - (double)s.m - logs) : -__builtin_inff(); };
    if (lane < a.top_k) {
        const uint32_t k = (uint32_t)(kept >> 32);
        a.top_ids[(size_t)row * a.top_k + lane] = kept ? (int)~(uint32_t)kept : -1;
        a.top_logprobs[(size_t)row * a.top_k + lane] = kept ? logprob(order_value(k)) : (float)-inf;
    }
    if (lane == 0) {
        if (a.entropy) a.entropy[row] = none ? 0.0f : (float)(logs - s.u / s.s);
        if (a.logprobs) {
            const int t = a.tokens[row];
            a.logprobs[row] = (unsigned)t < (unsigned)a.V ? logprob(logit_at(a.logits, (size_t)row * a.V + t, a.lt)) : 0.0f;
        }
    }
}

template <bool TOP>
__global__ __launch_bounds__(64 * kLogWaves) void qmt_logprobs_kernel(const LogArgs a)
{
    __shared__ LogShared sh;
    constexpr int UN = 4;
    const float low = -__builtin_inff();
    const long long place = a.first + blockIdx.x;
    const int row = (int)(place / a.parts), part = (int)(place - (long long)row * a.parts);
    const int size = a.lt == QMX_T_F32 ? 4 : 2;
    const uint8_t *const base = (const uint8_t *)a.logits + (size_t)row * a.V * size;
    // groups of 8 start at whole 16 bytes, the first one up to 7 logits before the row
    const int head = (int)((uintptr_t)base & 15) / size;
    const int tid = threadIdx.x, w = tid >> 6;
    const int s0 = part * a.steps, s1 = s0 + a.steps;
    auto load = [&](int i, Raw8 &r) {
        r.b = make_uint4(0, 0, 0, 0);
        if (i >= 0 && i + 8 <= a.V) {
            const uint4 *const p = (const uint4 *)(base + (long long)i * size);
            r.a = p[0];
            if (size == 4) r.b = p[1];
        } else {
            // a group over the row's border: its logits one at a time, the others masked
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = i + j >= 0 && i + j < a.V;
                const uint32_t masked = a.lt == QMX_T_F32 ? 0xFF800000u : a.lt == QMX_T_BF16 ? 0xFF80u : 0xFC00u;
                v[j] = !in ? masked : size == 4 ? ((const uint32_t *)base)[i + j] : ((const uint16_t *)base)[i + j];
            }
            if (size == 4) {
                r.a = make_uint4(v[0], v[1], v[2], v[3]);
                r.b = make_uint4(v[4], v[5], v[6], v[7]);
            } else {
                r.a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
            }
        }
    };
    Sums sums = {low, 0.0, 0.0};
    TopList top(sh.wait[w]);
    float tau = low;                                           // only logits above it can be among the top
    bool first = true;
    for (int s = s0; s < s1; s += UN) {
        Raw8 raw[UN];
#pragma unroll
        for (int n = 0; n < UN; ++n) load(s + n < s1 ? (s + n) * kStep - head + 8 * tid : a.V, raw[n]);
#pragma unroll
        for (int n = 0; n < UN; ++n) {
            float l[8];
            raw_to_f32(raw[n], a.lt, l);
#pragma unroll
            for (int j = 0; j < 8; ++j) l[j] = l[j] > low ? l[j] : low;      // NaN too
            const float big = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
            if (big > sums.m) sums.move(big);
            double e[8];
            float u = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // (below -200 the exponential is 0 in fp32; both -infinity: NaN, which gives -200)
                const float z = fmaxf(l[j] - sums.m, -200.0f);
                const float x = exp2f(z * 1.4426950408889634f);
                u = __builtin_fmaf(x, z, u);
                e[j] = (double)x;
            }
            sums.s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            sums.u += (double)u;
            if constexpr (TOP) {
                if (first) {
                    // the top_k-th largest of the lanes' largest: as many logits are at least that
                    first = false;
                    const uint32_t k = __shfl(wave_sort<true>(big > low ? order_bits(big) : 0u), a.top_k - 1);
                    // the value below it (there is none of -0's bits)
                    tau = k == 0u ? low : order_value(k - (k == 0x80000000u ? 2u : 1u));
                }
                if (__any(big > tau)) {
                    const int i = (s + n) * kStep - head + 8 * tid;
#pragma unroll 1
                    for (int j = 0; j < 8; ++j) {
                        float v = l[0];
#pragma unroll
                        for (int q = 1; q < 8; ++q) v = q == j ? l[q] : v;
                        top.add(v > tau, entry(v, i + j));
                    }
                    // (not within a step: the same logit at a lower index may come after)
                    const uint32_t k = (uint32_t)(__shfl(top.kept, a.top_k - 1) >> 32);
                    if (k) tau = fmaxf(tau, order_value(k));
                }
            }
        }
    }
    if constexpr (TOP) top.finish();
    Sums all = wave_sums(sums);
    uint64_t kept = top.kept;
    join_waves<TOP>(sh, all, kept);
    if (w != 0) return;
    if (a.parts == 1) {
        put_row(a, row, all, kept);
        return;
    }
    uint8_t *const out = a.work + place * part_bytes(a.top_k);
    if (tid == 0) {
        *(double *)out = all.s;
        *(double *)(out + 8) = all.u;
        *(float *)(out + 16) = all.m;
    }
    if (TOP && tid < a.top_k) *(uint64_t *)(out + 32 + 8 * tid) = kept;
}

// The parts of a row joined: one workgroup a row.
template <bool TOP>
__global__ __launch_bounds__(64 * kLogWaves) void qmt_logprobs_join_kernel(const LogArgs a)
{
    __shared__ LogShared sh;
    const float low = -__builtin_inff();
    const int row = (int)(a.first + blockIdx.x), tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const long long bytes = part_bytes(a.top_k);
    const uint8_t *const work = a.work + (long long)row * a.parts * bytes;
    Sums sums = {low, 0.0, 0.0};
    for (int p = tid; p < a.parts; p += 64 * kLogWaves) {
        const uint8_t *const at = work + p * bytes;
        Sums o = {*(const float *)(at + 16), *(const double *)at, *(const double *)(at + 8)};
        const float m = fmaxf(sums.m, o.m);
        sums.move(m);
        o.move(m);
        sums.s += o.s;
        sums.u += o.u;
    }
    TopList top(sh.wait[w]);
    if constexpr (TOP) {
        // at least top_k entries are no smaller than the top_k-th largest of 64 lanes' largest
        uint64_t big = 0;
        for (int p = lane; p < a.parts; p += 64) big = larger(big, *(const uint64_t *)(work + p * bytes + 32));
        const uint64_t tau = __shfl(wave_sort<true>(big), a.top_k - 1);
        const int n = a.parts * a.top_k;
        for (int i0 = w * 64; i0 < n; i0 += 64 * kLogWaves) {
            const int i = i0 + lane, p = i / a.top_k;
            const uint64_t e = i < n ? *(const uint64_t *)(work + p * bytes + 32 + 8 * (i - p * a.top_k)) : 0;
            top.add(e != 0 && e >= tau, e);
        }
        top.finish();
    }
    Sums all = wave_sums(sums);
    uint64_t kept = top.kept;
    join_waves<TOP>(sh, all, kept);
    if (w == 0) put_row(a, row, all, kept);
}

// HIP limits a launch to 2^32 threads: beyond this many workgroups a kernel
// loops or is launched again.
constexpr long long kMaxGroups = 1LL << 20;

qmv_status_t go(const void *fn, long long groups, void **args, hipStream_t stream)
{
    return hipLaunchKernel(fn, dim3((unsigned)groups), dim3(256), args, 0, stream) == hipSuccess ? QMV_OK : QMV_EHIP;
}

// Workgroups 0 .. n - 1 of a kernel whose first one's number is a.*FIRST times `unit`.
template <class Args>
qmv_status_t go_all(const void *fn, Args &a, long long Args::*first, long long unit, long long n, hipStream_t stream)
{
    void *args[] = {&a};
    for (long long g = 0; g < n; g += kMaxGroups) {
        a.*first = g * unit;
        const qmv_status_t s = go(fn, n - g < kMaxGroups ? n - g : kMaxGroups, args, stream);
        if (s != QMV_OK)
            return s;
    }
    return QMV_OK;
}

long long square_groups(long long blocks) { return blocks < kMaxGroups ? blocks : kMaxGroups; }

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
    int xt = (int)xtype;
    void *args[] = {&x, &xt, &codes, &scales, &blocks, &N, &K};
    return go((const void *)&qmt_quantize_weights_kernel, square_groups(blocks), args, stream);
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
                D, P, R, rotation == QMT_PAIRS ? 1 : 0, M, all, 0};
    int G;
    const bool many = (long long)M * all >= 16384;
    const void *fn = many ? qk_kernel<4>(D, G) : qk_kernel<1>(D, G);
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
    if (p.parts > 1 && (!workspace || !aligned(workspace, 16)))
        return QMV_EINVAL;
    LogArgs a = {logits, tokens, logprobs, entropy, top_logprobs, top_ids, (uint8_t *)workspace, (int)ltype, M, V,
                 top_k, p.parts, p.steps, 0};
    const void *fn = top_k ? (const void *)&qmt_logprobs_kernel<true> : (const void *)&qmt_logprobs_kernel<false>;
    const void *join = top_k ? (const void *)&qmt_logprobs_join_kernel<true>
                             : (const void *)&qmt_logprobs_join_kernel<false>;
    const qmv_status_t st = go_all(fn, a, &LogArgs::first, 1, (long long)M * p.parts, stream);
    if (st != QMV_OK || p.parts == 1)
        return st;
    return go_all(join, a, &LogArgs::first, 1, M, stream);
}

QMT_API const char *qmt_strerror(qmv_status_t status) { return status_text(status); }

}  // extern "C"
