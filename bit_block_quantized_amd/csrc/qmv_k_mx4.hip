// qmv_k_mx4.hip -- MXFP4 weights x MXFP4 activations on the block-scaled
// matrix cores (v_mfma_scale_f32_16x16x128_f8f6f4): dense, gather, gate/up
// with SwiGLU, and the combine of up to 4 tokens.
//
//     y = sum over blocks b of 2^(sw_b - 127 + sx_b - 127) * sum_32 e2m1 * e2m1
//
// The instruction takes 16 rows x 128 k of A, 128 k x 16 columns of B, and
// one E8M0 byte per row (column) and 32 k; lane (c, q) = lane 16 q + c holds
// the 32 e2m1 values of row (column) c's block q: 16 bytes exactly as they
// lie in memory.  So codes go from memory into the operands unchanged, and
// the sums are formed in fp32.
#include "qmv_device.hpp"

#include <type_traits>

namespace qmv {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kXPast = 0x80000000u;       // >= every buffer size: reads zeros

// The product with the lane's scale bytes in byte OP of sa and of sb.
template <int OP>
__device__ __forceinline__ f32x4 mfma_mx4_op(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb)
{
    const i32x8 A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, OP, (int)sa, OP, (int)sb);
}

// One 16 x 128 x 16 product; sa, sb: the lane's scale bytes in bits 0-7.
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb)
{
    const i32x8 A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Items: 16 rows of one expert (a dense matrix, a token of a combine) and 16
// of its vectors; the NW waves of a workgroup split K, wave w taking the
// 128-weight steps w, w + NW, ..., and the waves' partial tiles are summed
// in wave order.
template <int MODE, int NW>
__global__ __launch_bounds__(64 * NW) void qmv_mx4_few_kernel(const Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int H = MODE == 1 ? 2 : 1;            // weight tensors
    constexpr int D = 4;                            // steps in flight
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int row0 = blockIdx.x * 16;
    const int U = a.units;
    const int S = (U + 3) >> 2;
    const bool gather = a.ids != nullptr;
    const int P = gather ? a.M * a.top_k : a.M;
    f32x4 *const part = (f32x4 *)lds;               // [NW][H][64]
    PairList L;
    L.cnt = (int *)(lds + NW * H * 1024);
    L.perm = (uint16_t *)(L.cnt + kMaxCounts + 4);

    int e = 0, count = P, slots = 1;
    int ids_lane = 0;                               // combine: lane j holds the id of slot j
    if constexpr (MODE == 2) {
        slots = a.top_k;
        count = 1;
        if (lane < a.top_k) ids_lane = a.ids[blockIdx.y * a.top_k + lane];
    } else if (gather) {
        // grid.y: one per expert, or with fewer pairs than experts one per
        // pair (the first pair of an expert takes it)
        const Ids8 id0 = load_ids8<64 * NW>(a.ids, P, a.E, 0);
        const bool by_pair = P < a.E;
        if (by_pair ? (unsigned)a.ids[blockIdx.y] >= (unsigned)a.E : blockIdx.y == 0) {
            // the rows of ids outside [0, E) are zeros (by pair: this one's)
            const int ci = by_pair ? 1 : list_pairs<64 * NW>(a.ids, P, a.E, -1, L, id0);
            for (int o = threadIdx.x; o < ci * 16; o += 64 * NW) {
                const int pz = by_pair ? (int)blockIdx.y : (int)L.perm[o >> 4];
                if (row0 + (o & 15) < a.N) a.y[(size_t)pz * a.N + row0 + (o & 15)] = 0.0f;
            }
            if (by_pair) return;
            __syncthreads();
        }
        e = by_pair ? a.ids[blockIdx.y] : (int)blockIdx.y;
        count = list_pairs<64 * NW>(a.ids, P, a.E, e, L, id0);
        if (count == 0 || (by_pair && (int)L.perm[0] != (int)blockIdx.y)) return;
    }
    const int rowc = row0 + c;
    const int x_bytes = (MODE == 2 || gather ? (a.x_per_slot ? a.M * a.top_k : a.M) : a.M) * a.x_vec_bytes;
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x, x_bytes);
    const __amdgpu_buffer_rsrc_t rxs = buffer_rsrc(a.xs, x_bytes / 16);
    const int vfirst = MODE == 2 || gather ? 0 : blockIdx.y * 16;
    const int vlast = MODE == 2 || gather ? count : min(P, vfirst + 16);
    for (int v0 = vfirst; v0 < vlast; v0 += 16) {
        const int nv = min(16, vlast - v0);
        // this lane's column: a vector of the chunk (columns past nv repeat the first)
        const int vi = c < nv ? v0 + c : v0;
        const int pair = MODE == 2 ? blockIdx.y * a.top_k : gather ? (int)L.perm[vi] : vi;
        int vec = pair;
        if (MODE == 2 || gather) vec = a.x_per_slot ? pair : pair / a.top_k;
        f32x4 acc[H], tot = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < H; ++h) acc[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // (slot, step) of this wave: slot-major, every NW-th one
        const int total = slots * S;
        for (int g0 = w; g0 < total; g0 += NW * D) {
            u32x4 A[D][H], B[D];
            uint32_t sa[D][H], sb[D];
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int g = g0 + NW * d;
                const int slot = MODE == 2 ? g / S : 0;
                const int s = g - slot * S;
                const int blk = 4 * s + q;
                const bool in = g < total && blk < U;
                int ee = e;
                bool ok = in && rowc < a.N;
                if constexpr (MODE == 2) {
                    ee = __builtin_amdgcn_readlane(ids_lane, slot < slots ? slot : 0);
                    ok = ok && (unsigned)ee < (unsigned)a.E;
                    if ((unsigned)ee >= (unsigned)a.E) ee = 0;
                }
                const uint32_t oc = ok ? (uint32_t)rowc * (uint32_t)a.rcb + 16u * blk : kXPast;
                const uint32_t os = ok ? (uint32_t)rowc * (uint32_t)a.rsb + blk : kXPast;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const __amdgpu_buffer_rsrc_t rc =
                        buffer_rsrc((h ? a.codes2 : a.codes) + (long long)ee * a.expert_cb, a.expert_cb);
                    const __amdgpu_buffer_rsrc_t rs =
                        buffer_rsrc((h ? a.scales2 : a.scales) + (long long)ee * a.expert_sb, a.expert_sb);
                    A[d][h] = __builtin_amdgcn_raw_buffer_load_b128(rc, oc, 0, 0);
                    sa[d][h] = __builtin_amdgcn_raw_buffer_load_b8(rs, os, 0, 0);
                }
                const int xv = vec + (MODE == 2 && a.x_per_slot ? slot : 0);
                B[d] = __builtin_amdgcn_raw_buffer_load_b128(
                    rx, in ? (uint32_t)xv * (uint32_t)a.x_vec_bytes + 16u * blk : kXPast, 0, 0);
                sb[d] = __builtin_amdgcn_raw_buffer_load_b8(
                    rxs, in ? (uint32_t)xv * (uint32_t)a.rsb + blk : kXPast, 0, 0);
            }
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int g = g0 + NW * d;
#pragma unroll
                for (int h = 0; h < H; ++h) acc[h] = mfma_mx4(A[d][h], B[d], acc[h], sa[d][h], sb[d]);
                if constexpr (MODE == 2) {
                    if (g < total && (g + NW) / S != g / S) {
                        const float rw = a.route_w[blockIdx.y * a.top_k + g / S];
#pragma unroll
                        for (int k = 0; k < 4; ++k) tot[k] = __builtin_fmaf(rw, acc[0][k], tot[k]);
                        acc[0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                }
            }
        }
        if constexpr (MODE == 2) acc[0] = tot;
#pragma unroll
        for (int h = 0; h < H; ++h) part[(w * H + h) * 64 + lane] = acc[h];
        __syncthreads();
        if (threadIdx.x < 64 && c < nv) {
            f32x4 r[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                r[h] = part[h * 64 + lane];
                for (int i = 1; i < NW; ++i) r[h] += part[(i * H + h) * 64 + lane];
            }
            float *const yr = a.y + (size_t)(MODE == 2 ? blockIdx.y : pair) * a.N;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = row0 + 4 * q + k;
                if (n < a.N) yr[n] = MODE == 1 ? swiglu(r[0][k], r[H - 1][k]) : r[0][k];
            }
        }
        __syncthreads();
    }
}

extern const void *const kTableMx4Few[3];
const void *const kTableMx4Few[3] = {
    (const void *)&qmv_mx4_few_kernel<0, 4>,
    (const void *)&qmv_mx4_few_kernel<1, 4>,
    (const void *)&qmv_mx4_few_kernel<2, 4>,
};

// ------------------------------------------------------------- many vectors
// A tile is (expert, 16 RF NWR weight rows) against a chunk of its vectors,
// NWR x NWC waves of RF x CF fragments each.  K goes in slabs of 512 weights
// (4 MFMA steps):
//   codes of the rows   straight from memory into the A operands, one slab
//                       ahead (lane (c, q): row c's block q of a step -- 16
//                       rows x 64 bytes a load, which streams within 3% of
//                       contiguous reads on MI355X)
//   codes of the vectors  staged in LDS in operand order (a fragment of a
//                       step is 64 lanes x 16 bytes, read without bank
//                       conflicts), double-buffered, loaded one slab ahead
//   scale bytes         staged in LDS per slab as 16 bytes a row, transposed
//                       so that lane (c, q) reads its four steps' bytes as one
//                       dword, which the instruction indexes itself
// One barrier per slab.
// A row's 16 scale bytes of a slab as loaded: five whole dwords around them.
struct ScaleSeg {
    u32x4 d;
    uint32_t last;
};

// o: byte offset of the segment from the 4-byte aligned buffer start.  ENDS:
// the segment may reach the buffer's end, so every dword is checked alone.
template <bool ENDS>
__device__ __forceinline__ ScaleSeg load_seg(__amdgpu_buffer_rsrc_t r, uint32_t o)
{
    ScaleSeg s;
    const uint32_t a = o & ~3u;
    if constexpr (ENDS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s.d[i] = __builtin_amdgcn_raw_buffer_load_b32(r, a + 4u * i, 0, 0);
    } else {
        s.d = __builtin_amdgcn_raw_buffer_load_b128(r, a, 0, 0);
    }
    s.last = __builtin_amdgcn_raw_buffer_load_b32(r, a + 16u, 0, 0);
    return s;
}

// The segment's bytes in lane order: dword q holds block 4 s + q of steps
// s = 0..3 in byte s.  ENDS: only the first n bytes belong to the row, the
// rest become 0.
template <bool ENDS>
__device__ __forceinline__ u32x4 seg_order(const ScaleSeg &s, uint32_t o, int n)
{
    const uint32_t w[5] = {s.d[0], s.d[1], s.d[2], s.d[3], s.last};
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        d[i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], o & 3u);
        if constexpr (ENDS) {
            const int k = min(max(n - 4 * i, 0), 4);  // bytes of this dword inside the row
            d[i] &= (uint32_t)((1ull << (8 * k)) - 1ull);
        }
    }
    const uint32_t l01 = perm(d[1], d[0], 0x05010400u), h01 = perm(d[1], d[0], 0x07030602u);
    const uint32_t l23 = perm(d[3], d[2], 0x05010400u), h23 = perm(d[3], d[2], 0x07030602u);
    return u32x4{perm(l23, l01, 0x05040100u), perm(l23, l01, 0x07060302u), perm(h23, h01, 0x05040100u),
                 perm(h23, h01, 0x07060302u)};
}

template <int MODE, bool DENSE, int RF, int CF, int NWR, int NWC, int AD>
__device__ __forceinline__ void mx4_tile_chunk(const Args &a, uint8_t *lds, int e, int row_base,
                                               const uint16_t *vecs, int vstart, int nv)
{
    constexpr int NW = NWR * NWC;
    constexpr int CT = CF * NWC;                     // column fragments of the chunk
    constexpr int BR = 16 * RF * NWR;                // weight rows of the tile (gate/up: of both)
    constexpr int RH = MODE == 1 ? RF / 2 : RF;      // output row fragments per wave
    constexpr int XU = (4 * CT + NW - 1) / NW;       // staged fragments per wave and slab
    constexpr int NP = XU > 4 ? 4 : 1;               // staged in this many portions
    constexpr int XP = XU / NP;
    constexpr int XG = CT > NW ? CT / NW : 1;        // distinct column fragments a wave stages
    constexpr int GB = CF > 4 ? 4 : CF;              // column fragments read from LDS at a time
    constexpr int NS = 64 * NW;                      // staged scale segments (one per thread)
    static_assert(BR + 16 * CT <= NS && (MODE == 1 ? BR / 2 : BR) % 64 == 0, "one thread per staged scale row");
    static_assert(4 * CT % NW == 0 || 4 * CT < NW, "staging split");
    uint8_t *const lx = lds;
    uint8_t *const ls = lx + 2 * 4 * CT * 1024;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));                    // (keeps the offsets below inside the chunk loop)
    const int lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = NWC == 1 ? w : w / NWC, wc = NWC == 1 ? 0 : w % NWC;
    const int c = lane & 15, q = lane >> 4;
    const bool gather = !DENSE && a.ids != nullptr;
    const int U = a.units;
    const int S = (U + 3) >> 2;                      // steps
    const int J = (S + 3) >> 2;                      // slabs

    f32x4 acc[RF][CF];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int g = 0; g < CF; ++g) acc[f][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // rows past N repeat the last one and are not stored
    const long long eo = e;
    const __amdgpu_buffer_rsrc_t rc0 = buffer_rsrc(a.codes + eo * a.expert_cb, a.expert_cb);
    const __amdgpu_buffer_rsrc_t rc1 = buffer_rsrc((MODE == 1 ? a.codes2 : a.codes) + eo * a.expert_cb, a.expert_cb);
    uint32_t oc[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) {
        const int n = min(row_base + 16 * RH * wr + 16 * (MODE == 1 ? f % RH : f) + c, a.N - 1);
        oc[f] = (uint32_t)n * (uint32_t)a.rcb + 16u * q;
    }
    auto load_a = [&](int s, u32x4 (&A)[RF]) {
        const uint32_t so = s < S ? 64u * s : kXPast;           // (oc < 2^31: the sum does not wrap)
#pragma unroll
        for (int f = 0; f < RF; ++f)
            A[f] = __builtin_amdgcn_raw_buffer_load_b128(MODE == 1 && f >= RH ? rc1 : rc0, oc[f] + so, 0, 0);
    };

    // staged vectors: fragment (step s, column fragment g) = unit s CT + g,
    // wave w takes units w, w + NW, ...
    const int top_k = a.top_k;
    const bool by_token = gather && !a.x_per_slot;
    auto vec_row = [&](int v) -> uint32_t {
        const int i = gather ? (int)vecs[v] : vstart + v;
        return (uint32_t)(by_token ? i / top_k : i);
    };
    const int x_rows = gather && a.x_per_slot ? a.M * a.top_k : a.M;
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x, (long long)x_rows * a.x_vec_bytes);
    uint32_t ox[XG];
#pragma unroll
    for (int k = 0; k < XG; ++k) {
        const int v = 16 * ((w + NW * k) % CT) + c;
        ox[k] = v < nv && w < 4 * CT ? vec_row(v) * (uint32_t)a.x_vec_bytes + 16u * q : kXPast;
    }
    auto load_x = [&](int j, int p, u32x4 (&X)[XP]) {
#pragma unroll
        for (int k = 0; k < XP; ++k) {
            const int u = w + NW * (p * XP + k);
            const int s = 4 * j + u / CT;
            const uint32_t o = ox[XG == 1 ? 0 : (p * XP + k) % XG];
            const bool ok = 4 * s + q < U && o != kXPast;
            X[k] = __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? o + 64u * s : kXPast, 0, 0);
        }
    };
    auto store_x = [&](int j, int p, const u32x4 (&X)[XP]) {
#pragma unroll
        for (int k = 0; k < XP; ++k) {
            const int u = w + NW * (p * XP + k);
            if (4 * CT >= NW || w < 4 * CT) *(u32x4 *)(lx + ((j & 1) * 4 * CT + u) * 1024 + 16 * lane) = X[k];
        }
    };

    // staged scales: one row's 16 bytes a thread -- first the tile's rows
    // (gate/up: the gate's, then the up's), then the chunk's vectors.  Which
    // of the three a wave reads is the same for all its lanes.
    const int role = w < (MODE == 1 ? BR / 2 : BR) / 64 ? 0 : w < BR / 64 ? 1 : 2;
    const uintptr_t ps = role == 2 ? (uintptr_t)a.xs
                                   : (uintptr_t)((MODE == 1 && role == 1 ? a.scales2 : a.scales) + eo * a.expert_sb);
    const long long zs = (long long)(ps & 3) + (role == 2 ? (long long)x_rows * a.rsb : a.expert_sb);
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc((const void *)(ps & ~(uintptr_t)3), (zs + 3) & ~3ll);
    uint32_t os;
    {
        const int t = MODE == 1 ? tid & (BR / 2 - 1) : tid;
        const uint32_t row = role == 2 ? vec_row(tid - BR < nv ? tid - BR : 0)
                                       : (uint32_t)min(row_base + t, a.N - 1);
        os = (uint32_t)(ps & 3) + row * (uint32_t)a.rsb;
    }
    // where the wave's fragments' scales stand
    auto seg_of_row = [&](int f) { return MODE == 1 ? (f >= RH ? BR / 2 : 0) + 16 * (wr * RH + f % RH) : 16 * (wr * RF + f); };

    u32x4 A[AD][RF];
    {
        const ScaleSeg sg = load_seg<true>(rs, os);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            u32x4 X[XP];
            load_x(0, p, X);
            if (p == NP - 1) {
#pragma unroll
                for (int s = 0; s < AD; ++s) load_a(s, A[s]);
            }
            store_x(0, p, X);
        }
        *(u32x4 *)(ls + tid * 16) = seg_order<true>(sg, os, U);
    }
    __syncthreads();
    // LAST 0: slabs j and j + 1 are not the last; 1: slab j + 1 is; 2: slab j is
    auto slab = [&](int j, auto LAST) {
        constexpr int last = decltype(LAST)::value;
        const uint8_t *const xb = lx + (j & 1) * (4 * CT * 1024) + 16 * lane;
        const uint8_t *const sc = ls + (j & 1) * (NS * 16) + c * 16 + 4 * q;
        ScaleSeg sg;
        u32x4 X[XP];
        if constexpr (last < 2) {
            sg = load_seg<last == 1>(rs, os + 16u * (j + 1));
            load_x(j + 1, 0, X);
        }
        uint32_t ta[RF], tb[CF];
#pragma unroll
        for (int f = 0; f < RF; ++f) ta[f] = *(const uint32_t *)(sc + seg_of_row(f) * 16);
#pragma unroll
        for (int g = 0; g < CF; ++g) tb[g] = *(const uint32_t *)(sc + (BR + 16 * (wc * CF + g)) * 16);
        // (step, GB column fragments) at a time; the next ones are read from
        // LDS while these multiply
        constexpr int H = CF / GB;
        u32x4 B[2][GB];
        auto read_b = [&](int i, u32x4 (&b)[GB]) {
#pragma unroll
            for (int g = 0; g < GB; ++g)
                b[g] = *(const u32x4 *)(xb + ((i / H) * CT + wc * CF + (i % H) * GB + g) * 1024);
        };
        read_b(0, B[0]);
        auto part = [&](auto IDX) {
            constexpr int i = decltype(IDX)::value;
            constexpr int s = i / H, g0 = (i % H) * GB;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (i + 1 < 4 * H) read_b(i + 1, B[(i + 1) & 1]);
#pragma unroll
            for (int g = 0; g < GB; ++g)
#pragma unroll
                for (int f = 0; f < RF; ++f)
                    acc[f][g0 + g] = mfma_mx4_op<s>(A[s % AD][f], B[i & 1][g], acc[f][g0 + g], ta[f], tb[g0 + g]);
            // (the compiler would move the products past the barrier to their
            // last use, with all their operands held until then)
#pragma unroll
            for (int g = 0; g < GB; ++g)
#pragma unroll
                for (int f = 0; f < RF; ++f) asm volatile("" : "+v"(acc[f][g0 + g]));
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (i % H == H - 1 && last < 2) load_a(4 * j + s + AD, A[s % AD]);
            if constexpr (i % H == H - 1 && last == 2 && s + AD < 4) load_a(4 * j + s + AD, A[s % AD]);
        };
        auto step = [&](auto SIDX) {
            constexpr int s = decltype(SIDX)::value;
            part(std::integral_constant<int, s * H>{});
            if constexpr (H > 1) part(std::integral_constant<int, s * H + 1>{});
        };
        // with four portions each is loaded before a step and stored after it
        auto next = [&](int p) {
            if constexpr (NP == 4 && last < 2) {
                store_x(j + 1, p - 1, X);
                load_x(j + 1, p, X);
            }
        };
        step(std::integral_constant<int, 0>{});
        next(1);
        step(std::integral_constant<int, 1>{});
        next(2);
        step(std::integral_constant<int, 2>{});
        next(3);
        step(std::integral_constant<int, 3>{});
        if constexpr (last < 2) {
            store_x(j + 1, NP - 1, X);
            *(u32x4 *)(ls + ((j + 1) & 1) * (NS * 16) + tid * 16) = seg_order<last == 1>(sg, os, U - 16 * (j + 1));
        }
        __syncthreads();
    };
    int j = 0;
    for (; j + 2 < J; ++j) slab(j, std::integral_constant<int, 0>{});
    if (j + 1 < J) slab(j++, std::integral_constant<int, 1>{});
    slab(j, std::integral_constant<int, 2>{});

    // lane (c, q) holds rows 4 q .. 4 q + 3 of vector c of each fragment
    const bool vec4 = (a.N & 3) == 0 && ((uintptr_t)a.y & 15) == 0;
#pragma unroll
    for (int g = 0; g < CF; ++g) {
        const int v = 16 * (wc * CF + g) + c;
        if (v < nv) {
            float *const yr = a.y + (size_t)(gather ? (int)vecs[v] : vstart + v) * a.N;
#pragma unroll
            for (int f = 0; f < RH; ++f) {
                const int n0 = row_base + 16 * RH * wr + 16 * f + 4 * q;
                float r[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    r[k] = MODE == 1 ? swiglu(acc[f][g][k], acc[f + RF - RH][g][k]) : acc[f][g][k];
                if (n0 < a.N) {
                    if (vec4) {
                        *(float4 *)(yr + n0) = make_float4(r[0], r[1], r[2], r[3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (n0 + k < a.N) yr[n0 + k] = r[k];
                    }
                }
            }
        }
    }
}

// The tile's expert and vectors, then its chunks.  CMAX: column fragments per
// wave of the largest chunk.
// DENSE: no routed calls.
template <int MODE, bool DENSE, int RF, int NWR, int NWC, int AD, int CMIN, int CMAX, int WPE>
__global__ __launch_bounds__(64 * NWR * NWC, WPE) void qmv_mx4_tile_kernel(const Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int THREADS = 64 * NWR * NWC;
    constexpr int TR = 16 * RF * NWR / (MODE == 1 ? 2 : 1);
    constexpr int VCAP = 16 * CMAX * NWC;
    const int b = blockIdx.x;
    const int t = (b & 7) * a.bt_per_xcd + (b >> 3);
    if (t >= a.bt_tiles) return;
    const bool gather = !DENSE && a.ids != nullptr;
    int e = 0, cnt = 0, vstart = 0, rt;
    const uint16_t *vecs = nullptr;
    if (gather) {
        const int bucket = t / a.bt_row_tiles;
        rt = t - bucket * a.bt_row_tiles;
        const int row_base = rt * TR;
        PairList L;
        L.cnt = (int *)(lds + a.lds_vec_bytes);       // behind the staging buffers
        L.perm = (uint16_t *)(L.cnt + kMaxCounts + 4);
        const Ids8 id0 = load_ids8<THREADS>(a.ids, a.M * a.top_k, a.E, 0);
        if (bucket == 0) {
            // the tiles of expert 0 also write the zero rows of ids outside [0, E)
            const int ci = list_pairs<THREADS>(a.ids, a.M * a.top_k, a.E, -1, L, id0);
            const int rows = min(TR, a.N - row_base);
            for (int o = threadIdx.x; o < ci * rows; o += THREADS)
                a.y[(size_t)L.perm[o / rows] * a.N + row_base + o % rows] = 0.0f;
            __syncthreads();
        }
        e = bucket;
        cnt = list_pairs<THREADS>(a.ids, a.M * a.top_k, a.E, bucket, L, id0);
        if (cnt == 0) return;
        vecs = L.perm;
    } else {
        // dense: groups of bt_vmax vector chunks, chunk-fastest inside, so that
        // the tiles an XCD runs at a time share both operands
        const int chunks = (a.M + VCAP - 1) / VCAP;
        const int per = a.bt_vmax * a.bt_row_tiles;
        const int grp = t / per;
        const int in = t - grp * per;
        const int gw = min(a.bt_vmax, chunks - grp * a.bt_vmax);
        rt = in / gw;
        vstart = (grp * a.bt_vmax + in - rt * gw) * VCAP;
        cnt = min(VCAP, a.M - vstart);
    }
    const int row_base = rt * TR;
    const int nch = (cnt + VCAP - 1) / VCAP;
    const int cs = (cnt + nch - 1) / nch;             // equal chunks
    for (int ch = 0; ch < nch; ++ch) {
        const int nv = min(cs, cnt - ch * cs);
        const uint16_t *const cv = vecs ? vecs + ch * cs : nullptr;
        const int vs = vstart + ch * cs;
        if (CMIN <= 1 && nv <= 16 * NWC)
            mx4_tile_chunk<MODE, DENSE, RF, CMIN <= 1 ? 1 : CMAX, NWR, NWC, AD>(a, lds, e, row_base, cv, vs, nv);
        else if (CMIN <= 2 && CMAX >= 2 && nv <= 32 * NWC)
            mx4_tile_chunk<MODE, DENSE, RF, CMIN <= 2 && CMAX >= 2 ? 2 : CMAX, NWR, NWC, AD>(a, lds, e, row_base, cv, vs, nv);
        else if (CMIN <= 4 && CMAX >= 4 && nv <= 64 * NWC)
            mx4_tile_chunk<MODE, DENSE, RF, CMIN <= 4 && CMAX >= 4 ? 4 : CMAX, NWR, NWC, AD>(a, lds, e, row_base, cv, vs, nv);
        else
            mx4_tile_chunk<MODE, DENSE, RF, CMAX, NWR, NWC, AD>(a, lds, e, row_base, cv, vs, nv);
        __syncthreads();                              // (the next chunk stages over this one's buffers)
    }
}

// [plain, gate/up], then [plain] for wide dense calls
extern const void *const kTableMx4Tile[3];
const void *const kTableMx4Tile[3] = {
    (const void *)&qmv_mx4_tile_kernel<0, false, 2, 8, 1, 2, 1, 4, 4>,
    (const void *)&qmv_mx4_tile_kernel<1, false, 2, 8, 1, 2, 1, 4, 4>,
    (const void *)&qmv_mx4_tile_kernel<0, true, 4, 4, 2, 2, 8, 8, 2>,
};

}  // namespace qmv
