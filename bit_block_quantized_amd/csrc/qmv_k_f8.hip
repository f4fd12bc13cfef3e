// qmv_k_f8.hip -- e4m3 weights with an fp32 scale per 128 x 128 block x e4m3
// activations with an fp32 scale per 128, on the matrix cores' bf16 products:
// dense, gather, gate/up with SwiGLU, and the combine of up to 4 tokens.
//
//     y = sum over blocks b of (sw_b * sx_b) * sum_128 e4m3 * e4m3
//
// Codes stay e4m3 in memory and LDS and are widened to bf16 (which holds every
// e4m3 value) in registers.  The f8f6f4 instructions would take them as they
// are at twice the rate, but they add products eight at a time to 14 bits of
// the largest: blocks of normal values' codes came out 1.8e-6 of the sum of their
// magnitudes off (root mean square of 200; 7.5e-6 at most; 1e-5 of the result), with
// bf16 operands 2.3e-9 (1.8e-8).
//
// The products of a block form its whole sum in fp32 from zero, which one
// multiply-add per output adds to the result with the product of the block's two
// scales: four 16 x 16 x 32 instructions, or eight of 32 x 32 x 16.  With the
// former a lane holds 32 bytes of its row (column): lane (c, q) = lane 16 q + c
// takes chunks q and q + 4 (16 bytes each) of row c's 128.  (A sum does not care
// which k a lane holds, as long as both operands agree.)
//
// Times here and at the choices between these kernels are of a call among others
// in a graph, with three sets of weights and vectors in turn.
#include "qmv_routed.hpp"

#include <type_traits>
#include <utility>

namespace qmv {

constexpr int kF8Few = 16;           // vectors of a few-vector workgroup
constexpr int kF8Waves = kRoutedWaves;
constexpr int kF8Chunk = 96;         // vectors of a tile at most (also in qmv.hip)
constexpr int kF8Block = 128;        // weights of a block, and code bytes

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A lane's 32 codes as operands: two chunks, four instructions' values.
struct Wide {
    bf16x8 v[4];
};

__device__ __forceinline__ Wide widen(const u32x4 (&c)[2])
{
    Wide r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u32x4 h;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w = c[i >> 1][2 * (i & 1) + j];
            h[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
            h[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
        }
        r.v[i] = __builtin_bit_cast(bf16x8, h);
    }
    return r;
}

// The block sums of 16 rows x 16 columns.
__device__ __forceinline__ f32x4 block_sum(const Wide &a, const Wide &b)
{
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], s, 0, 0, 0);
    return s;
}

__device__ __forceinline__ void add_scaled(f32x4 &acc, f32x4 part, float s)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(part[k], s, acc[k]);
}

// The 32 x 32 instruction: lane (n, k) = lane 32 k + n holds chunks k, k + 2, k +
// 4, k + 6 of row (column) n's 128 bytes, eight instructions' values, and of
// the products rows 8 i + 4 k .. of column n in registers 4 i .. .
typedef float f32x16 __attribute__((ext_vector_type(16)));

// A chunk's 16 codes: two instructions' values.
__device__ __forceinline__ void widen_chunk(u32x4 c, bf16x8 &lo, bf16x8 &hi)
{
    u32x4 h[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false));
        h[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true));
    }
    lo = __builtin_bit_cast(bf16x8, h[0]);
    hi = __builtin_bit_cast(bf16x8, h[1]);
}

// Keeps what forms x here: without it the compiler moves products, conversions
// and additions to their results' first use, with all their operands held.
template <class T> __device__ __forceinline__ void pin(T &x) { asm volatile("" : "+v"(x)); }

__device__ __forceinline__ f32x16 mfma32(const bf16x8 &x, const bf16x8 &y, const f32x16 &z)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, z, 0, 0, 0);
}

// Waits until at most N of the wave's loads (and stores) are on their way and
// its reads of LDS are done, then for the workgroup.  (A barrier of the
// compiler's waits for every load into LDS.)
template <int N> __device__ __forceinline__ void wait_loads_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

typedef __attribute__((address_space(3))) void lds_t;

template <int... I, class Part>
__device__ __forceinline__ void parts(std::integer_sequence<int, I...>, Part part)
{
    (part(std::integral_constant<int, I>{}), ...);
}

// The sums to add after product k of eight: from the third on, when the last product before has them.
constexpr __host__ __device__ int from_k(int k) { return k < 2 ? 0 : k == 8 ? 16 : 3 * k - 6; }

// ------------------------------------------------------------- many vectors
// A tile is (expert, 128 weight rows; gate/up: 64 of each) against a chunk of
// its vectors (up to 32 CF): 4 waves of 32 rows -- gate/up has the gate's 16 in
// registers 0 .. 7 of the products and the up projection's in 8 .. 15 -- for
// all of K, two such workgroups a CU, or for each of two halves of K (HV), the
// even and the odd blocks, where there are no more tiles than CUs.
//
// Codes go from memory into LDS without passing registers, 8 rows of 128 bytes
// a load, and the place of a lane's 16 bytes (byte 16 l of the piece) is that
// of chunk l % 8 ^ (row / 2 % 8) of its row, so that 16 lanes that read a chunk of
// 16 rows touch 16 different bank groups.  While a block is multiplied, the
// rows' codes of a half's next two are on their way and the vectors' of the
// next.  A wave's rows are its own; a half's vectors are staged by its four waves,
// one barrier a block.
//
// Bound by the weight bytes (gate/up of 32 experts top 4, 2880 -> 2880, 531 MB, experts
// drawn evenly: 64 tokens 114 us, 4.7 TB/s; with rows of 2816 106, 4.9 TB/s: their
// blocks do not straddle cache lines; gather of 1024 tokens top 8 of 256, 7168 -> 2048,
// 3.7 GB: 715, 5.2 TB/s).  With many vectors a tile less so: 512 tokens 149 us, and 170
// to 175 with popular and unpopular experts (1 to 385 pairs, in 41 chunks for 32).  Of
// the 149, as copies of the kernel without one of its parts show, its start and end,
// without any block, take 36, and the vectors' loads 14; without any load of the rows it
// takes 109, without products 133, without widening the later fragments 136.
//
// Tried: 16 x 16 fragments staged through registers, 64 vectors a tile: 512 tokens of
// popular and unpopular experts 185 us, so 171 to 179; 7168 -> 7168, 1024 vectors
// 156, so 147.  All tiles in two halves: 227 and 153.  Runs of row tiles that share
// the counting of the pairs: 2 187 us, 3 215.  Row tiles dealt to the XCDs in turn,
// the next block's first operands widened beside the last products: no faster.
constexpr int kF8Ring = 3;           // blocks of the rows' codes in LDS

// Row tile rt of expert e against nv vectors: pairs vecs[0..nv) of a routed
// call, vectors vstart .. of a dense one (vecs null).
template <int MODE, int HV, int CF>
__device__ __forceinline__ void f8_tile(const Args &a, uint8_t *lds, int e, int rt, const uint16_t *vecs, int vstart, int nv)
{
    constexpr int R = kF8Ring;
    constexpr int TR = MODE == 1 ? 64 : 128;         // output rows of a tile
    constexpr int PX = CF;                           // pieces of the vectors a wave stages
    constexpr int HALF = 2 * CF * 4096 + 2 * CF * 128 + 4 * R * 4096;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));                    // (keeps the offsets below out of the caller's registers)
    const int lane = tid & 63;
    const int half = HV == 2 ? __builtin_amdgcn_readfirstlane(tid >> 8) : 0, w = __builtin_amdgcn_readfirstlane(tid >> 6 & 3);
    const int n = lane & 31, hk = lane >> 5;
    const int lr = lane >> 3, lc = (lane & 7) ^ (lr >> 1);           // row and chunk of a load's even pieces; odd: ^ 4
    const bool gather = vecs != nullptr;
    const int N = a.N;
    const int KB = a.units, U = a.K >> 4;            // blocks, 16-byte chunks of a row
    uint8_t *const lx = lds + half * HALF;                            // [2][CF][32 vectors x 128 bytes]
    float *const ls = (float *)(lx + 2 * CF * 4096);                  // [2][32 CF]
    uint8_t *const lw = lx + 2 * CF * 4096 + 2 * CF * 128 + w * (R * 4096);   // this wave's: [R][32 rows x 128 bytes]

    // rows past N repeat the last one and are not stored
    const __amdgpu_buffer_rsrc_t rc0 = buffer_rsrc(a.codes + e * a.expert_cb, a.expert_cb);
    const __amdgpu_buffer_rsrc_t rc1 = buffer_rsrc((MODE == 1 ? a.codes2 : a.codes) + e * a.expert_cb, a.expert_cb);
    uint32_t oc[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int row = rt * TR + (MODE == 1 ? 16 * w + 8 * (p & 1) : 32 * w + 8 * p) + lr;
        oc[p] = (uint32_t)min(row, N - 1) * (uint32_t)a.rcb + 16u * (lc ^ (4 * (p & 1)));
    }
    const int top_k = a.top_k;
    const bool by_token = gather && !a.x_per_slot;
    auto vec_row = [&](int v) -> uint32_t {
        const int i = gather ? (int)vecs[v] : vstart + v;
        return (uint32_t)(by_token ? i / top_k : i);
    };
    const int x_rows = gather && a.x_per_slot ? a.M * a.top_k : a.M;
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x, (long long)x_rows * a.x_vec_bytes);
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(a.xs, (long long)x_rows * KB * 4);
    uint32_t ox[PX];                                 // wave w stages pieces w, w + 4: vectors 8 w .. of a fragment
#pragma unroll
    for (int k = 0; k < PX; ++k) {
        const int v = 32 * k + 8 * w + lr;
        ox[k] = v < nv ? vec_row(v) * (uint32_t)a.x_vec_bytes + 16u * (lc ^ (4 * (w & 1))) : kXPast;
    }
    const int sv = 64 * w + lane;                    // the vector whose scale this lane stages
    const uint32_t os = sv < nv ? vec_row(sv) * (uint32_t)KB * 4u : kXPast;
    // The blocks that are loaded next, rows' and vectors': number, place.  A block
    // is the loads' scalar offset, past every buffer's end behind the last block:
    // as many loads, of zeros.  (Chunks past the row's end read zeros too: the
    // bytes there are another row's.)
    const bool cut0 = lc >= U - 8 * (KB - 1), cut1 = (lc ^ 4) >= U - 8 * (KB - 1);
    constexpr int PAST = 0x7FFFFFF0, PIECES = PX + 5;
    int u_l = half, at_l = 0, u_x = half, at_x = 0;
    // Piece q: the vectors' codes, their scales, the rows' codes last.
    auto load = [&](int q) {
        if (q < PX) {
            const bool out = u_x == KB - 1 && (w & 1 ? cut1 : cut0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_t *)(lx + at_x * (CF * 4096) + q * 4096 + w * 1024), 16,
                                                     out ? kXPast : ox[q], u_x < KB ? 128 * u_x : PAST, 0, 0);
        } else if (q == PX) {
            if (w < (CF + 1) / 2 && sv < 32 * CF)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_t *)(ls + at_x * (32 * CF) + 64 * w), 4, os,
                                                         u_x < KB ? 4 * u_x : PAST, 0, 0);
            at_x ^= 1;
            u_x += HV;
        } else {
            const int p = q - PX - 1;
            const bool out = u_l == KB - 1 && (p & 1 ? cut1 : cut0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(MODE == 1 && p >= 2 ? rc1 : rc0, (lds_t *)(lw + at_l * 4096 + p * 1024), 16,
                                                     out ? kXPast : oc[p], u_l < KB ? 128 * u_l : PAST, 0, 0);
            if (p == 3) {
                at_l = at_l == R - 1 ? 0 : at_l + 1;
                u_l += HV;
            }
        }
    };
    // the tile's rows lie in one block row of the scales
    typedef const __attribute__((address_space(4))) float scalar_float;
    auto row_scale = [&](const uint8_t *base, int u) {
        const long long at = (long long)(rt * TR / kF8Block) * KB + min(u, KB - 1);
        const float s = *(scalar_float *)(uintptr_t)(base + e * a.expert_sb + 4 * at);
        return u < KB ? s : 0.0f;
    };
    const int rd = n * 128 + 16 * (hk ^ (n >> 1 & 7));

    float acc[CF][16];
    f32x16 sum[CF];
    float by0[CF], by1[CF];                          // the scales that the sums take: registers 0 .. 7, 8 .. 15
#pragma unroll
    for (int g = 0; g < CF; ++g) {
        by0[g] = by1[g] = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[g][i] = sum[g][i] = 0.0f;
    }
    static_assert(PIECES <= 8, "one with each product of the first fragment");
    auto scale = [&](int g, int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            acc[g][i] = __builtin_fmaf(sum[g][i], MODE == 1 && i >= 8 ? by1[g] : by0[g], acc[g][i]);
            pin(acc[g][i]);
        }
    };
    const f32x16 zero = {};

#pragma unroll
    for (int q = PX + 1; q < PIECES; ++q) load(q);
#pragma unroll
    for (int q = 0; q < PIECES; ++q) load(q);
    float sw0 = row_scale(a.scales, half), sw1 = MODE == 1 ? row_scale(a.scales2, half) : 0.0f;
    int at = 0, ax = 0;
    for (int u = half; u < KB + half; u += HV) {     // (both halves as often)
        // this block's codes are here (the last loads are the next one's
        // rows), and the places of the one before are free
        wait_loads_barrier<4>();
        const uint8_t *const pa = lw + at * 4096, *const pb = lx + ax * (CF * 4096);
        auto chunk = [&](const uint8_t *base, int j) { return *(const u32x4 *)(base + (rd ^ (32 * j))); };
        u32x4 ra[4], rb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) ra[j] = chunk(pa, j), rb[j] = chunk(pb, j);
        float sx[CF];
#pragma unroll
        for (int g = 0; g < CF; ++g) sx[g] = ls[ax * (32 * CF) + 32 * g + n];
        const float sn0 = row_scale(a.scales, u + HV), sn1 = MODE == 1 ? row_scale(a.scales2, u + HV) : 0.0f;
        bf16x8 W[8], B[8];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            widen_chunk(ra[j], W[2 * j], W[2 * j + 1]);
            widen_chunk(rb[j], B[2 * j], B[2 * j + 1]);
        }
        if constexpr (CF == 1) scale(0, 0, 16);
#pragma unroll
        for (int g = 0; g < CF; ++g) {
            if (g + 1 < CF) {
#pragma unroll
                for (int j = 0; j < 4; ++j) rb[j] = chunk(pb + (g + 1) * 4096, j);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum[g] = mfma32(W[k], B[k], k ? sum[g] : zero);
                pin(sum[g]);
                // (the sums of the fragment before, of the block before)
                if constexpr (CF > 1) scale(g ? g - 1 : CF - 1, from_k(k), from_k(k + 1));
                // (given out together, the loads would hold up the products behind them)
                if (g == 0 && k < PIECES) load(k);
                if (g + 1 < CF && (k & 1)) {
                    widen_chunk(rb[k >> 1], B[k - 1], B[k]);
                    pin(B[k - 1]);
                    pin(B[k]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            by0[g] = sw0 * sx[g];
            by1[g] = sw1 * sx[g];
        }
        sw0 = sn0, sw1 = sn1;
        at = at == R - 1 ? 0 : at + 1;
        ax ^= 1;
    }
    scale(CF - 1, 0, 16);

    const bool vec4 = (N & 3) == 0 && ((uintptr_t)a.y & 15) == 0;
    const int row0 = (MODE == 1 ? 16 : 32) * w + 4 * hk;   // registers 4 i ..: rows row0 + 8 i .. of the tile
    auto y_row = [&](int v) { return a.y + (size_t)(gather ? (int)vecs[v] : vstart + v) * N + rt * TR; };
    const int rows = min(TR, N - rt * TR);
    wait_loads_barrier<0>();                         // (nothing on its way into LDS; all its codes are read)
    if constexpr (HV == 1) {
        // by way of LDS, a vector's rows together (in 16-byte pieces, 32 vectors a store: 156 us for the 512 tokens' 149)
        constexpr int PITCH = TR + 4;
        float *const out = (float *)lds;
#pragma unroll
        for (int g = 0; g < CF; ++g)
#pragma unroll
            for (int i = 0; i < (MODE == 1 ? 2 : 4); ++i) {
                float q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    q[k] = MODE == 1 ? swiglu(acc[g][4 * i + k], acc[g][(4 * i + 8 + k) & 15]) : acc[g][4 * i + k];
                *(float4 *)(out + (32 * g + n) * PITCH + row0 + 8 * i) = make_float4(q[0], q[1], q[2], q[3]);
            }
        __syncthreads();
        if (vec4) {
            for (int t = tid; t < nv * (TR / 4); t += 64 * kF8Waves) {
                const int v = t / (TR / 4), r = 4 * (t % (TR / 4));
                if (r < rows) *(float4 *)(y_row(v) + r) = *(const float4 *)(out + v * PITCH + r);
            }
        } else {
            for (int t = tid; t < nv * TR; t += 64 * kF8Waves) {
                const int v = t / TR, r = t % TR;
                if (r < rows) y_row(v)[r] = out[v * PITCH + r];
            }
        }
        return;
    }
    auto store = [&](int v, int r0, const float (&r)[4]) {
        if (v < nv && r0 < rows) {
            float *const yr = y_row(v) + r0;
            if (vec4) {
                *(float4 *)yr = make_float4(r[0], r[1], r[2], r[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r0 + k < rows) yr[k] = r[k];
            }
        }
    };
    // Each half gives the other one half of its registers (gate/up: of the
    // gate's and of the up projection's), and stores the rest.
    float *const give = (float *)lds + (4 * half + w) * (CF * 512) + lane;
    const float *const take = (const float *)lds + (4 * (half ^ 1) + w) * (CF * 512) + lane;
    // registers of the part that half h keeps
    auto reg = [](int h, int i) { return MODE == 1 ? 8 * (i >> 2) + 4 * h + (i & 3) : 8 * h + i; };
#pragma unroll
    for (int g = 0; g < CF; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) give[(8 * g + i) * 64] = half ? acc[g][reg(0, i)] : acc[g][reg(1, i)];
    __syncthreads();
#pragma unroll
    for (int g = 0; g < CF; ++g) {
        float r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)                  // (two terms: the same sum in either order)
            r[i] = (half ? acc[g][reg(1, i)] : acc[g][reg(0, i)]) + take[(8 * g + i) * 64];
#pragma unroll
        for (int i = 0; i < (MODE == 1 ? 1 : 2); ++i) {
            float q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) q[k] = MODE == 1 ? swiglu(r[k], r[4 + k]) : r[4 * i + k];
            store(32 * g + n, row0 + (MODE == 1 ? 8 * half : 16 * half + 8 * i), q);
        }
    }
}

// Workgroup b runs on XCD b % 8; the tiles are dealt to the XCDs in contiguous
// parts, expert by expert, row tile by row tile, so that an XCD's L2 holds the
// vectors of a few experts, and a row tile's codes for all of the expert's chunks
// (512 tokens, top 4 of 32, 2880 -> 2880, chunk by chunk: 702 MB for 531 of codes).
template <int MODE, int HV>
__global__ __launch_bounds__(64 * kF8Waves * HV, 2) void qmv_f8_tile_kernel(const Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int CHUNK = kF8Chunk, TR = MODE == 1 ? 64 : 128;
    uint16_t *const list = (uint16_t *)lds;           // [CHUNK]
    uint8_t *const buf = lds + 2 * CHUNK;             // (16-byte aligned)
    int item = -1, rt = 0, place = 0;
    auto pick = [&](int items) {
        const int all = items * a.bt_row_tiles, per_xcd = (all + 7) / 8, i = blockIdx.x >> 3;
        const int r = i < per_xcd ? (int)(blockIdx.x & 7) * per_xcd + i : all;
        if (r < all) {
            item = r / a.bt_row_tiles;
            rt = r - item * a.bt_row_tiles;
            place = r;
        }
        return item;
    };
    // the same places of all chunks first .. first + n - 1, row tile by row tile
    auto order = [&](int, int first, int n) {
        const int at = place - first * a.bt_row_tiles;
        rt = at / n;
        const int chunk = at - rt * n;
        item = first + chunk;
        return chunk;
    };
    int e = 0, nv, vstart = 0;
    const bool gather = a.ids != nullptr;
    if (gather) {
        // (a call without any id in [0, E) still has its zero rows: one item.
        // The first half counts; the other has no pairs)
        const int P = threadIdx.x < 64 * kRoutedWaves ? a.M * a.top_k : 0;
        const RoutedItem it = routed_item<CHUNK>(a.ids, P, a.E, (int *)buf, list, [&](int items) { return pick(max(items, 1)); },
                                                  order);
        if (item < 0) return;
        e = it.e;
        nv = it.nv;
        if (threadIdx.x < 64 * kRoutedWaves) routed_zero_rows(a, item, max(it.items, 1), rt * TR, min(rt * TR + TR, a.N));
        if (nv == 0) return;
    } else {
        const int chunks = (a.M + CHUNK - 1) / CHUNK, cs = (a.M + chunks - 1) / chunks;   // equal chunks
        if (pick(chunks) < 0) return;
        vstart = order(item, 0, chunks) * cs;
        nv = min(cs, a.M - vstart);
    }
    const uint16_t *const vecs = gather ? list : nullptr;
    if (nv > 64)
        f8_tile<MODE, HV, 3>(a, buf, e, rt, vecs, vstart, nv);
    else if (nv > 32)
        f8_tile<MODE, HV, 2>(a, buf, e, rt, vecs, vstart, nv);
    else
        f8_tile<MODE, HV, 1>(a, buf, e, rt, vecs, vstart, nv);
}

// -------------------------------------------------------------- few vectors
// Up to 16 vectors of an expert (a dense matrix), or (MODE 2, the combine) a
// token's slots, each with its expert, against one tile of 16 rows.  The call
// waits for its weight bytes, so the 4 waves of a workgroup split K -- wave w
// takes blocks w, w + 4, ... -- and each has up to kF8Ahead blocks of its rows
// on their way from the start; the vectors and the scales are staged in LDS
// once.  The waves' partial tiles are summed in wave order.  Columns past the
// last vector repeat one (nothing of them is stored).
//
// Bound by the weight bytes where there are many: gate/up of one token, top 8 of
// 256, 7168 -> 2048 (235 MB) 42 us, 5.6 TB/s; combine of 4 tokens, 2048 -> 7168 (470
// MB) 94 us; 7168 -> 40960 (294 MB) 51 us; by one trip to memory after another
// where there are few: 7168 -> 2048 (15 MB) 8.2 us.
constexpr int kF8Ahead = 4;

// Bytes from vector to vector of the staged codes (whole blocks, and 16 more
// so that the 16 vectors of a read lie in different bank groups), and floats
// from vector to vector of the staged scales.
__host__ __device__ constexpr int f8_x_pitch(int KB) { return KB * 128 + 16; }
__host__ __device__ constexpr int f8_s_pitch(int KB) { return KB | 1; }

template <int MODE>
__global__ __launch_bounds__(64 * kF8Waves) void qmv_f8_few_kernel(const Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int NW = kF8Waves, H = MODE == 1 ? 2 : 1, D = kF8Ahead;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4, lr = lane >> 3, lc = lane & 7;
    const int KB = a.units, U = a.K >> 4;
    const int XP = f8_x_pitch(KB), SP = f8_s_pitch(KB);
    const int N = a.N;
    const bool gather = MODE != 2 && a.ids != nullptr;
    const int P = gather ? a.M * a.top_k : a.M;

    uint16_t *const list = (uint16_t *)lds;                    // [kF8Few]
    uint8_t *const la = lds + 64 + w * (H * 2048);             // this wave's weight pieces; its partial sums
    uint8_t *const lx = lds + 64 + NW * H * 2048;              // [vectors] x XP
    float *const lxs = (float *)(lx + a.bt_vmax * XP);         // [vectors] x SP
    float *const ls = lxs + a.bt_vmax * SP;                    // [H or slots] x SP

    // ---- which expert, vectors and row tiles
    int e = 0, nv = 1, v0 = 0, rt = blockIdx.x;
    int ids_lane = 0;
    float rw_lane = 0.0f;
    if constexpr (MODE == 2) {
        // lane j holds slot j's expert and weight
        if (lane < a.top_k) {
            ids_lane = a.ids[blockIdx.y * a.top_k + lane];
            rw_lane = a.route_w[blockIdx.y * a.top_k + lane];
        }
    } else if (!gather) {
        v0 = blockIdx.y * kF8Few;
        nv = min(kF8Few, a.M - v0);
    } else if (P <= 64) {
        // workgroup row blockIdx.y: pair blockIdx.y's expert, if no earlier
        // pair has it (up to 64 pairs: one lane each)
        const int id = lane < P ? a.ids[lane] : -1, y = blockIdx.y % P;
        const int chunk = blockIdx.y / P;                      // of bt_vmax pairs of the expert
        e = __builtin_amdgcn_readlane(id, y);
        if ((unsigned)e >= (unsigned)a.E) {
            if (chunk == 0)
                for (int n = rt * 16 + tid; n < min(rt * 16 + 16, N); n += 64 * NW) a.y[(size_t)y * N + n] = 0.0f;
            return;
        }
        const unsigned long long m = __ballot(id == e);
        if (__ffsll((long long)m) - 1 != y) return;
        // (bit counts are unsigned: as int before anything is subtracted)
        const int r = (int)__popcll(m & ((1ull << lane) - 1ull)) - chunk * a.bt_vmax;
        const int left = (int)__popcll(m) - chunk * a.bt_vmax;
        if (left <= 0) return;
        nv = min(left, a.bt_vmax);
        if ((m >> lane & 1) && r >= 0 && r < a.bt_vmax) list[r] = (uint16_t)lane;    // (every wave the same)
    } else {
        int item = -1;
        const RoutedItem it = routed_item<kF8Few>(a.ids, P, a.E, (int *)(lds + 64), list, [&](int items) {
            const int all = max(items, 1) * a.bt_row_tiles, per_xcd = (all + 7) / 8, i = blockIdx.x >> 3;
            const int r = i < per_xcd ? (int)(blockIdx.x & 7) * per_xcd + i : all;
            if (r < all) {
                item = r / a.bt_row_tiles;
                rt = r - item * a.bt_row_tiles;
            }
            return item;
        });
        if (item < 0) return;
        e = it.e;
        nv = it.nv;
        routed_zero_rows(a, item, max(it.items, 1), rt * 16, min(rt * 16 + 16, N));
        if (nv == 0) return;
        __syncthreads();                                       // (the counts lie where the staging goes)
    }
    const bool routed = MODE == 2 || gather;
    const int top_k = a.top_k;
    const int x_rows = routed && a.x_per_slot ? a.M * top_k : a.M;
    auto pair_of = [&](int v) { return MODE == 2 ? (int)blockIdx.y * top_k + v : gather ? (int)list[v] : v0 + v; };
    auto vec_row = [&](int v) -> uint32_t {
        const int p = pair_of(v);
        return (uint32_t)(routed && !a.x_per_slot ? p / top_k : p);
    };

    // ---- groups of slots (MODE 2: bt_vmax at a time; else one pass)
    const int slots = MODE == 2 ? top_k : 1, per = MODE == 2 ? a.bt_vmax : 1;
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x, (long long)x_rows * a.x_vec_bytes);
    f32x4 tot = {0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 A[D][H][2];
    const int row0 = rt * 16;
    uint32_t oc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) oc[i] = (uint32_t)min(row0 + 8 * i + lr, N - 1) * (uint32_t)a.rcb + 16u * lc;
    for (int s0 = 0; s0 < slots; s0 += per) {
        const int ns = min(per, slots - s0), total = ns * KB;
        auto load_a = [&](int i, u32x4 (&R)[H][2]) {
            const int g = w + NW * i;
            const int slot = MODE == 2 ? g / KB : 0, u = g - slot * KB;
            int ee = e;
            long long size = a.expert_cb;
            if constexpr (MODE == 2) {
                ee = __builtin_amdgcn_readlane(ids_lane, g < total ? s0 + slot : 0);
                if ((unsigned)ee >= (unsigned)a.E) ee = 0, size = 0;           // reads zeros
            }
            const uint32_t so = g < total && 8 * u + lc < U ? 128u * u : kXPast;
#pragma unroll
            for (int h = 0; h < H; ++h) {                                      // (nt: read once)
                const __amdgpu_buffer_rsrc_t rc = buffer_rsrc((h ? a.codes2 : a.codes) + ee * a.expert_cb, size);
#pragma unroll
                for (int k = 0; k < 2; ++k) R[h][k] = __builtin_amdgcn_raw_buffer_load_b128(rc, oc[k] + so, 0, 2);
            }
        };
#pragma unroll
        for (int i = 0; i < D; ++i) load_a(i, A[i]);
        // the vectors (MODE 2: those of the group's slots), and all scales
        const int vecs = MODE == 2 ? (a.x_per_slot ? ns : 1) : nv;
        for (int t = tid; t < vecs * 8 * KB; t += 64 * NW) {
            const int v = t / (8 * KB), b = t - v * 8 * KB;
            const uint32_t o = vec_row(MODE == 2 ? s0 + v : v) * (uint32_t)a.x_vec_bytes + 16u * b;
            *(u32x4 *)(lx + v * XP + 16 * b) =
                __builtin_amdgcn_raw_buffer_load_b128(rx, b < U ? o : kXPast, 0, 0);
        }
        for (int t = tid; t < vecs * KB; t += 64 * NW) {
            const int v = t / KB, u = t - v * KB;
            lxs[v * SP + u] = ((const float *)a.xs)[(size_t)vec_row(MODE == 2 ? s0 + v : v) * KB + u];
        }
        const size_t block_row = (size_t)(row0 / kF8Block) * KB;
        for (int k = 0; k < (MODE == 2 ? ns : H); ++k) {
            int ee = e;
            if constexpr (MODE == 2) {
                ee = __builtin_amdgcn_readlane(ids_lane, s0 + k);
                if ((unsigned)ee >= (unsigned)a.E) ee = 0;                     // (unused)
            }
            const uint8_t *const base = MODE == 1 && k == 1 ? a.scales2 : a.scales;
            if (tid < KB) ls[k * SP + tid] = ((const float *)(base + ee * a.expert_sb))[block_row + tid];
        }
        __syncthreads();

        f32x4 acc[H];
#pragma unroll
        for (int h = 0; h < H; ++h) acc[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int wst = swz_chunk(lr, lc), rd = c * 128 + 16 * (q ^ ((c >> 1) & 7));
        const int vc = MODE == 2 ? 0 : (c < nv ? c : nv - 1);                  // columns past nv repeat
        const int mine = total > w ? (total - w + NW - 1) / NW : 0;            // this wave's blocks
        for (int i0 = 0; i0 < mine; i0 += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int i = i0 + d;
                if (i < mine) {
                    const int g = w + NW * i;
                    const int slot = MODE == 2 ? g / KB : 0, u = g - slot * KB;
                    const int v = MODE == 2 ? (a.x_per_slot ? slot : 0) : vc;
                    const float sx = lxs[v * SP + u];
                    u32x4 B[2];
                    B[0] = *(const u32x4 *)(lx + v * XP + 128 * u + 16 * q);
                    B[1] = *(const u32x4 *)(lx + v * XP + 128 * u + 64 + 16 * q);
                    const Wide b = widen(B);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        *(u32x4 *)(la + h * 2048 + wst) = A[d][h][0];
                        *(u32x4 *)(la + h * 2048 + 1024 + (wst ^ 64)) = A[d][h][1];
                    }
                    asm volatile("" ::: "memory");                             // (written before read: one wave's LDS)
                    load_a(i + D, A[d]);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const float sw = ls[(MODE == 2 ? slot : h) * SP + u];
                        u32x4 F[2];
                        F[0] = *(const u32x4 *)(la + h * 2048 + rd);
                        F[1] = *(const u32x4 *)(la + h * 2048 + (rd ^ 64));
                        add_scaled(acc[h], block_sum(widen(F), b), sw * sx);
                    }
                    asm volatile("" ::: "memory");
                    if constexpr (MODE == 2) {
                        if ((g + NW) / KB != slot || i + 1 == mine) {          // this wave's last block of the slot
                            const float rw = __uint_as_float(
                                __builtin_amdgcn_readlane(__float_as_uint(rw_lane), s0 + slot));
                            // (a slot without an expert is 0 whatever its vector holds)
                            const bool have = (unsigned)__builtin_amdgcn_readlane(ids_lane, s0 + slot) < (unsigned)a.E;
#pragma unroll
                            for (int k = 0; k < 4; ++k) tot[k] = __builtin_fmaf(rw, have ? acc[0][k] : 0.0f, tot[k]);
                            acc[0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                        }
                    }
                }
            }
        }
        if constexpr (MODE == 2) {
            if (s0 + per < slots) {
                __syncthreads();                           // (the next group's staging)
                continue;
            }
            acc[0] = tot;
        }
#pragma unroll
        for (int h = 0; h < H; ++h) *(f32x4 *)(la + h * 2048 + 16 * lane) = acc[h];
        __syncthreads();
        // lane (c, q): rows 4 q .. 4 q + 3 of vector c, summed over the waves
        if (w == 0 && c < nv) {
            f32x4 r[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                r[h] = acc[h];
#pragma unroll
                for (int i = 1; i < NW; ++i) r[h] += *(const f32x4 *)(la + (i * H + h) * 2048 + 16 * lane);
            }
            float *const yr = a.y + (size_t)(MODE == 2 ? (int)blockIdx.y : pair_of(c)) * N;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = row0 + 4 * q + k;
                if (n < N) yr[n] = MODE == 1 ? swiglu(r[0][k], r[H - 1][k]) : r[0][k];
            }
        }
    }
}

// ------------------------------------------------------------- wide dense
// A dense matrix against many vectors is bound by the matrix cores, beside them
// by the vector ALUs, which widen the operands and scale the block sums, and by
// the chip's power.  The two units run side by side with the 32 x 32
// instruction (a product and six vector instructions: 41 cycles of a SIMD with
// two waves, the product alone 33), hardly with the 16 x 16 one (27 and 17 for
// half the product and three).  So tiles of 256 rows x 128 vectors, 4 x 2 waves
// of 64 x 64, in fragments of 32 x 32: lane (n, k) = lane 32 k + n holds
// chunks k, k + 2, k + 4, k + 6 of row (column) n's 128 bytes, eight
// instructions' values, and after them rows 8 i + 4 k .. of column n in
// registers 4 i .. .
//
// Both operands' codes go from memory into LDS without passing registers, a
// block ahead, one load for every second product: given out together they hold
// up the products behind them (833 us, 903 together, for the 8192 vectors
// below).  A fragment is widened chunk by chunk into the registers that the one
// before has left, and its sums are scaled and added while the next one's
// products run.  One barrier a block, where the last of its codes is read.
//
// 8192 vectors, 7168 -> 7168: 713 us a call, 1.18 PFLOP/s, in calls one after
// another up to 833 (at 1.6 GHz: the power limit); a library's product of bf16
// matrices of these sizes takes 640, of f16 677.  16 x 16 fragments staged
// through registers, 256 x 192 tiles: 910; 64 x 96 a wave: 919.
constexpr int kF8WideRows = 256;
constexpr int kF8WideCF = 2;         // 32-vector fragments per wave
constexpr int kF8WideVecs = 64 * kF8WideCF;

__device__ __forceinline__ void f8_wide_tile(const Args &a, uint8_t *lds, int row0, int vec0)
{
    constexpr int NWC = 2, NW = 8, RF = 2, CF = kF8WideCF;
    constexpr int BR = kF8WideRows, BC = kF8WideVecs;   // tile: rows, vectors
    constexpr int AB = BR * 128, XB = BC * 128;             // bytes of a block's codes
    constexpr int PA = BR / 8 / NW, PX = BC / 8 / NW;       // staged pieces (8 rows x 128 bytes) a wave
    uint8_t *const lx = lds + 2 * AB;                       // [2][XB], behind [2][AB]
    float *const ls = (float *)(lds + 2 * (AB + XB));       // [2][BC]

    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = w / NWC, wc = w % NWC;
    const int n = lane & 31, hk = lane >> 5;
    const int KB = a.units, U = a.K >> 4;

    float acc[RF][CF][16];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int g = 0; g < CF; ++g)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[f][g][i] = 0.0f;

    // wave w stages pieces w, w + NW, ... of each operand; lane l's 16 bytes go
    // to byte 16 l of the piece, which is the place of chunk l % 8 ^ (row / 2 %
    // 8) of its row; rows past N and vectors past M lie past the buffers'
    // ends and read zeros, and so do chunks past the row's end
    const __amdgpu_buffer_rsrc_t rc = buffer_rsrc(a.codes, a.expert_cb);
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x, (long long)a.M * a.x_vec_bytes);
    const int lr = 8 * w + (lane >> 3), lc = (lane & 7) ^ (lr >> 1 & 7);
    const uint32_t oa = (uint32_t)(row0 + lr) * (uint32_t)a.rcb + 16u * lc;
    const uint32_t ox = (uint32_t)(vec0 + lr) * (uint32_t)a.x_vec_bytes + 16u * lc;
    const uint32_t step = 8u * NW * (uint32_t)a.rcb;         // (rcb and x_vec_bytes are both K)
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(a.xs, (long long)a.M * KB * 4);
    const uint32_t os = (uint32_t)(vec0 + tid) * (uint32_t)KB * 4u;
    uint32_t ta = 0, tx = 0;
    // piece p of block u: PA of the rows, PX of the vectors, one of these' scales, one a lane
    auto stage = [&](int u, int h, int p) {
        if (p == 0) ta = 8 * u + lc < U ? oa + 128u * u : kXPast;
        if (p == PA) tx = 8 * u + lc < U ? ox + 128u * u : kXPast;
        if (p < PA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_t *)(lds + h * AB + (w + NW * p) * 1024), 16, ta, p * step, 0, 0);
        else if (p < PA + PX)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_t *)(lx + h * XB + (w + NW * (p - PA)) * 1024), 16, tx,
                                                     (p - PA) * step, 0, 0);
        else if (p == PA + PX && w < BC / 64)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_t *)(ls + h * BC + 64 * w), 4, u < KB ? os + 4u * u : kXPast, 0, 0, 0);
    };
    auto stage_all = [&](int u, int h) {
#pragma unroll
        for (int p = 0; p <= PA + PX; ++p) stage(u, h, p);
    };
    // (the wave's rows lie in one block row)
    const float *const swp = (const float *)a.scales + (size_t)(min(row0 + 64 * wr, a.N - 1) / kF8Block) * KB;

    const int rd = n * 128 + 16 * (hk ^ (n >> 1 & 7));
    const int ra = wr * RF * 4096 + rd, rb = 2 * AB + wc * CF * 4096 + rd;
    // chunk 2 j + hk of the lane's row, of its column
    auto read_a = [&](int h, int f, int j) { return *(const u32x4 *)(lds + (ra ^ (32 * j)) + h * AB + f * 4096); };
    auto read_b = [&](int h, int g, int j) { return *(const u32x4 *)(lds + (rb ^ (32 * j)) + h * XB + g * 4096); };
    const float *const lsn = ls + 32 * CF * wc + n;

    bf16x8 W[RF][8], B[8];
    stage_all(0, 0);
    float sw = swp[0];
    __builtin_amdgcn_s_waitcnt(0x0F70);                     // vmcnt(0)
    __syncthreads();
    stage_all(1, 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int f = 0; f < RF; ++f) widen_chunk(read_a(0, f, j), W[f][2 * j], W[f][2 * j + 1]);
        widen_chunk(read_b(0, 0, j), B[2 * j], B[2 * j + 1]);
    }
    f32x16 sum[RF];
    float sc = 0.0f, sp = 0.0f;                             // the scales that the sums of this and the last group take
    u32x4 nb[2], na[2];                                     // chunks on their way: columns, rows

    auto scale = [&](float (&to)[16], const f32x16 &from, float by, int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            to[i] = __builtin_fmaf(from[i], by, to[i]);
            pin(to[i]);
        }
    };
    auto widen_to = [](u32x4 c, bf16x8 &lo, bf16x8 &hi) {
        widen_chunk(c, lo, hi);
        pin(lo);
        pin(hi);
    };
    const f32x16 zero = {};

    // Pass (g, 0) multiplies rows 0 .. 31 and adds the sums of the pass before;
    // pass (g, 1) rows 32 .. 63, and widens the next group's columns.
    auto block = [&](int u, auto BUF, auto FIRST) {
        constexpr int h = decltype(BUF)::value;
        constexpr bool first = decltype(FIRST)::value;
        const float swn = swp[min(u + 1, KB - 1)];
        auto group = [&](auto G) {
            constexpr int g = decltype(G)::value;
            constexpr bool last = g == CF - 1;
            sp = sc;
            sc = sw * lsn[h * BC + 32 * g];
            if constexpr (last) {
                // the next block's codes are in LDS, and all of this one's are read
                __builtin_amdgcn_s_waitcnt(0x0F70);
                __syncthreads();
            }
            constexpr int hb = last ? h ^ 1 : h, gb = last ? 0 : g + 1;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum[0] = mfma32(W[0][k], B[k], k ? sum[0] : zero);
                pin(sum[0]);
                if constexpr (g > 0) scale(acc[1][g - 1], sum[1], sp, from_k(k), from_k(k + 1));
                if constexpr (g == 0 && !first) scale(acc[1][CF - 1], sum[1], sp, from_k(k), from_k(k + 1));
                if (k == 4) nb[0] = read_b(hb, gb, 0);
                if (k == 6) nb[1] = read_b(hb, gb, 1);
                if constexpr (last) {
                    // (given out together, the loads would hold up the products behind them)
                    if (!(k & 1)) stage(u + 2, h, k >> 1);
                    if (k == 5) na[0] = read_a(h ^ 1, 0, 0);
                    if (k == 7) na[1] = read_a(h ^ 1, 0, 1);
                }
                if constexpr (g == 0 && !first) {
                    if (k & 1) {
                        const int j = k >> 1;
                        widen_to(na[j & 1], W[1][2 * j], W[1][2 * j + 1]);
                        if (j + 2 < 4) na[j & 1] = read_a(h, 1, j + 2);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum[1] = mfma32(W[1][k], B[k], k ? sum[1] : zero);
                pin(sum[1]);
                scale(acc[0][g], sum[0], sc, from_k(k), from_k(k + 1));
                if (k & 1) {
                    const int j = k >> 1;
                    widen_to(nb[j & 1], B[2 * j], B[2 * j + 1]);
                    if (j + 2 < 4) nb[j & 1] = read_b(hb, gb, j + 2);
                    if constexpr (last) {
                        widen_to(na[j & 1], W[0][2 * j], W[0][2 * j + 1]);
                        na[j & 1] = j + 2 < 4 ? read_a(h ^ 1, 0, j + 2) : read_a(h ^ 1, 1, j - 2);
                    }
                }
                if constexpr (last) {
                    if (!(k & 1)) stage(u + 2, h, 4 + (k >> 1));
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        parts(std::make_integer_sequence<int, CF>{}, group);
        sw = swn;
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    block(0, I0{}, std::true_type{});
    int u = 1;
    for (; u + 1 < KB; u += 2) {
        block(u, I1{}, std::false_type{});
        block(u + 1, I0{}, std::false_type{});
    }
    if (u < KB) block(u, I1{}, std::false_type{});
    scale(acc[1][CF - 1], sum[1], sc, 0, 16);
    __builtin_amdgcn_s_waitcnt(0x0F70);                     // (nothing on its way into LDS when the workgroup ends)

    const bool vec4 = (a.N & 3) == 0 && ((uintptr_t)a.y & 15) == 0;
#pragma unroll
    for (int g = 0; g < CF; ++g) {
        const int v = vec0 + 32 * (wc * CF + g) + n;
        if (v < a.M) {
            float *const yr = a.y + (size_t)v * a.N;
#pragma unroll
            for (int f = 0; f < RF; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n0 = row0 + 64 * wr + 32 * f + 8 * i + 4 * hk;
                    const float(&r)[16] = acc[f][g];
                    if (n0 < a.N) {
                        if (vec4) {
                            *(float4 *)(yr + n0) = make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (n0 + k < a.N) yr[n0 + k] = r[4 * i + k];
                        }
                    }
                }
        }
    }
}

// The tiles lie in groups of bt_vmax vector chunks, chunk-fastest inside, and
// are dealt to the XCDs in contiguous parts: the tiles an XCD runs at a time
// share both operands.
__global__ __launch_bounds__(512, 2) void qmv_f8_wide_kernel(const Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int BC = kF8WideVecs;
    const int tile = (blockIdx.x & 7) * a.bt_per_xcd + (blockIdx.x >> 3);
    if (tile >= a.bt_tiles) return;
    const int chunks = (a.M + BC - 1) / BC, group = a.bt_vmax * a.bt_row_tiles;
    const int gi = tile / group, in = tile - gi * group, gw = min(a.bt_vmax, chunks - gi * a.bt_vmax);
    f8_wide_tile(a, lds, in / gw * kF8WideRows, (gi * a.bt_vmax + in % gw) * BC);
}

extern const void *const kTableF8Wide[1];
const void *const kTableF8Wide[1] = {
    (const void *)&qmv_f8_wide_kernel,
};

// [plain, gate/up, combine]
extern const void *const kTableF8Few[3];
const void *const kTableF8Few[3] = {
    (const void *)&qmv_f8_few_kernel<0>,
    (const void *)&qmv_f8_few_kernel<1>,
    (const void *)&qmv_f8_few_kernel<2>,
};

// [whole K, halves][plain, gate/up]
extern const void *const kTableF8Tile[2][2];
const void *const kTableF8Tile[2][2] = {
    {(const void *)&qmv_f8_tile_kernel<0, 1>, (const void *)&qmv_f8_tile_kernel<1, 1>},
    {(const void *)&qmv_f8_tile_kernel<0, 2>, (const void *)&qmv_f8_tile_kernel<1, 2>},
};

}  // namespace qmv
