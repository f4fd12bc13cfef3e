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
//
// Times here are a kernel's own: its median in a trace of ten calls with three
// sets of weights and vectors in turn.
#include "qmv_routed.hpp"

#include <type_traits>

namespace qmv {

// The product with the lane's scale bytes in byte OP of sa and of sb.
template <int OP>
__device__ __forceinline__ f32x4 mfma_mx4_op(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb)
{
    const i32x8 A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, OP, (int)sa, OP, (int)sb);
}

// ------------------------------------------------------------- many vectors
// A tile is (expert, 128 weight rows; gate/up: 64 of each) against a chunk of
// its vectors (up to 64 or 128), 4 waves of 2 x CF fragments each (RF = 2).  K goes in slabs of 512 weights (4 MFMA
// steps) of two units (2 steps, 128 code bytes a row).
//
// The MFMA wants lane (c, q) = lane 16 q + c to hold 16 bytes of row c, but a
// load whose neighbouring lanes lie in different rows costs the address unit
// a cycle per lane (16 bytes per cycle and CU -- hardly more than the CU's
// share of HBM).  So codes are loaded as they lie -- 8 lanes take a row's 128
// bytes, 8 rows a load -- and turned into operand order by a pass through
// LDS: chunk k (16 bytes) of row r stands at 128 r + 16 (k ^ (r/2 % 8)), so
// that the 16 lanes of a write and of a read each touch 16 different bank
// groups.
//   codes of the rows   through a piece of LDS of the wave's own (LDS keeps a
//                       wave's accesses in order: no barrier), two units ahead
//                       in registers
//   codes of the vectors  staged by all waves, double-buffered, one unit ahead
//   scale bytes         staged for the whole tile, 16 bytes (a slab) at a time
//                       transposed so that lane (c, q) reads its four steps'
//                       bytes as one dword, which the instruction indexes
// One barrier per unit; two workgroups of 4 waves share a CU.
//
// Bound by the weight stream: 1024 tokens x top-8 of 256, 7168 -> 2048, moves
// 2.07 GB in 404 to 414 us (5.1 TB/s of the 6.3 that default-policy loads reach).  Short
// rows leave more of a tile's time to its start (the ids' counts, the vector
// list, the scales): 512 tokens x top-4 of 32, gate/up 2880 -> 2880, 282 MB in
// 93 us, 3.0 TB/s (nontemporal loads of the codes took an eighth more).

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

constexpr int kMx4Few = 16;          // few kernel
constexpr int kMx4Waves = 4;
constexpr int kMx4RF = 2;            // 16-row fragments per wave of a tile

// Bytes from row to row of the staged scales of J slabs.
__host__ __device__ constexpr int mx4_scale_pitch(int J) { return 16 * (J | 1); }

// Row tiles rt0 .. rt1 - 1 of expert e against nv vectors: pairs vecs[0..nv)
// of a routed call, vectors vstart .. of a dense one (vecs null).
// XR: vectors that the LDS layout has room for.
template <int MODE, int CF, int XR>
__device__ __forceinline__ void mx4_tile_run(const Args &a, uint8_t *lds, int e, int rt0, int rt1,
                                             const uint16_t *vecs, int vstart, int nv)
{
    constexpr int NW = kMx4Waves, RF = kMx4RF;
    constexpr int BR = 16 * RF * NW;                 // weight rows of a tile (gate/up: of both)
    constexpr int RH = MODE == 1 ? RF / 2 : RF;      // output row fragments per wave
    constexpr int TR = 16 * RH * NW;                 // output rows of a tile
    constexpr int XU = (2 * CF + NW - 1) / NW;       // staged pieces (8 vectors x 128 bytes) per wave and unit
    constexpr int XB = CF * 2048;                    // bytes of one vector buffer
    constexpr int GB = CF < 4 ? CF : 4, HG = CF / GB; // vector fragments read at a time; groups of them
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));                    // (keeps the offsets below out of the caller's loop head)
    const int lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint8_t *const lx = lds;                                      // [2][CF][16 vectors x 128 bytes]
    uint8_t *const la = lds + 2 * XR * 128 + w * (RF * 2048);        // [RF][16 rows x 128 bytes], this wave's
    uint8_t *const ls = lds + 2 * XR * 128 + NW * RF * 2048;        // [BR + 16 CF] rows of SP bytes
    const int c = lane & 15, q = lane >> 4;
    const int lr = lane >> 3, lc = lane & 7;         // row and chunk of a load
    const bool gather = vecs != nullptr;
    const int N = a.N;
    const int U = a.units;
    const int S = (U + 3) >> 2;                      // steps
    const int J = (S + 3) >> 2;                      // slabs
    const int SP = mx4_scale_pitch(J);
    const uint32_t rsb = (uint32_t)a.rsb;

    const __amdgpu_buffer_rsrc_t rc0 = buffer_rsrc(a.codes + e * a.expert_cb, a.expert_cb);
    const __amdgpu_buffer_rsrc_t rc1 = buffer_rsrc((MODE == 1 ? a.codes2 : a.codes) + e * a.expert_cb, a.expert_cb);
    // rows past N repeat the last one and are not stored
    uint32_t oc[RF][2];
    auto set_rows = [&](int row_base) {
#pragma unroll
        for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = min(row_base + 16 * RH * w + 16 * (MODE == 1 ? f % RH : f) + 8 * i + lr, N - 1);
                oc[f][i] = (uint32_t)n * (uint32_t)a.rcb + 16u * lc;
            }
    };
    auto load_a = [&](int u, u32x4 (&A)[RF][2]) {
        const uint32_t so = 2 * u < S ? 128u * u : kXPast;      // (oc < 2^31: the sum does not wrap)
#pragma unroll
        for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                A[f][i] = __builtin_amdgcn_raw_buffer_load_b128(MODE == 1 && f >= RH ? rc1 : rc0, oc[f][i] + so, 0, 0);
    };
    const int wst = swz_chunk(lr, lc);               // rows 8 further: + 1024, ^ 64
    auto store_a = [&](const u32x4 (&A)[RF][2]) {
#pragma unroll
        for (int f = 0; f < RF; ++f) {
            *(u32x4 *)(la + f * 2048 + wst) = A[f][0];
            *(u32x4 *)(la + f * 2048 + 1024 + (wst ^ 64)) = A[f][1];
        }
    };

    // staged vectors: piece p = vectors 8 p .. 8 p + 7; wave w takes pieces w, w + NW, ...
    const int top_k = a.top_k;
    const bool by_token = gather && !a.x_per_slot;
    auto vec_row = [&](int v) -> uint32_t {
        const int i = gather ? (int)vecs[v] : vstart + v;
        return (uint32_t)(by_token ? i / top_k : i);
    };
    const int x_rows = gather && a.x_per_slot ? a.M * a.top_k : a.M;
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x, (long long)x_rows * a.x_vec_bytes);
    uint32_t ox[XU];
#pragma unroll
    for (int k = 0; k < XU; ++k) {
        const int v = 8 * (w + NW * k) + lr;
        ox[k] = v < nv ? vec_row(v) * (uint32_t)a.x_vec_bytes + 16u * lc : kXPast;
    }
    auto load_x = [&](int u, u32x4 (&X)[XU]) {
#pragma unroll
        for (int k = 0; k < XU; ++k) {
            const bool ok = 8 * u + lc < U && ox[k] != kXPast;
            X[k] = __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? ox[k] + 128u * u : kXPast, 0, 0);
        }
    };
    auto store_x = [&](int buf, const u32x4 (&X)[XU]) {
#pragma unroll
        for (int k = 0; k < XU; ++k) {
            const int p = w + NW * k;
            if (2 * CF >= NW || w < 2 * CF)
                *(u32x4 *)(lx + buf * XB + p * 1024 + (wst ^ ((p & 1) << 6))) = X[k];
        }
    };

    // Scales: whole rows at once -- a row's 16 bytes of a slab alone would
    // fetch their 128-byte line anew for every slab.  Neighbouring lanes take
    // neighbouring slabs of a row; an odd number of 16-byte segments from row
    // to row (bank conflicts).
    auto scale_rsrc = [&](const uint8_t *base, long long bytes) {
        const uintptr_t p0 = (uintptr_t)base;
        return buffer_rsrc((const void *)(p0 & ~(uintptr_t)3), ((long long)(p0 & 3) + bytes + 3) & ~3ll);
    };
    // segments t0, t0 + 256, ... of `rows` rows (the last one again past the end)
    auto load_s = [&](const uint8_t *base, __amdgpu_buffer_rsrc_t r, int rows, int t0, auto row_of, auto &sg) {
        constexpr int SB = sizeof(sg) / sizeof(sg[0]);
#pragma unroll
        for (int k = 0; k < SB; ++k) {
            const int t = min(t0 + k * 64 * NW, rows * J - 1), row = t / J, j = t - row * J;
            sg[k].o = (uint32_t)((uintptr_t)base & 3) + row_of(row) * rsb + 16u * j;
            sg[k].at = row * SP + 16 * j;
            sg[k].n = U - 16 * j;
            sg[k].s = load_seg<true>(r, sg[k].o);
        }
    };
    auto store_s = [&](uint8_t *dst, const auto &sg) {
        constexpr int SB = sizeof(sg) / sizeof(sg[0]);
#pragma unroll
        for (int k = 0; k < SB; ++k) *(u32x4 *)(dst + sg[k].at) = seg_order<true>(sg[k].s, sg[k].o, sg[k].n);
    };
    struct Seg { ScaleSeg s; uint32_t o; int at, n; };
    // A tile's scale rows, and (VECS) the vectors' before them: the first
    // segments of all of them are on their way before one is waited for.
    auto stage_scales = [&](int row_base, auto VECS) {
        constexpr bool vecs_too = decltype(VECS)::value;
        int t0 = tid;
        asm volatile("" : "+v"(t0));
        auto tile_row = [&](int row) { return (uint32_t)min(row_base + row, N - 1); };
        auto vec = [&](int v) { return vec_row(v < nv ? v : 0); };
        const uint8_t *const b0 = a.scales + e * a.expert_sb, *const b1 = (MODE == 1 ? a.scales2 : a.scales) + e * a.expert_sb;
        const uint8_t *const bx = (const uint8_t *)a.xs;
        const __amdgpu_buffer_rsrc_t r0 = scale_rsrc(b0, a.expert_sb), r1 = scale_rsrc(b1, a.expert_sb),
                                     rv = scale_rsrc(bx, (long long)x_rows * rsb);
        constexpr int SR = MODE == 1 ? 2 : 4, SV = 4;
        Seg g0[SR], g1[SR], gv[SV];
        load_s(b0, r0, TR, t0, tile_row, g0);
        if constexpr (MODE == 1) load_s(b1, r1, TR, t0, tile_row, g1);
        if constexpr (vecs_too) load_s(bx, rv, 16 * CF, t0, vec, gv);
        store_s(ls, g0);
        if constexpr (MODE == 1) store_s(ls + TR * SP, g1);
        if constexpr (vecs_too) store_s(ls + BR * SP, gv);
#pragma unroll 1
        for (int t = t0 + SR * 64 * NW; t < TR * J; t += SR * 64 * NW) {
            load_s(b0, r0, TR, t, tile_row, g0);
            if constexpr (MODE == 1) load_s(b1, r1, TR, t, tile_row, g1);
            store_s(ls, g0);
            if constexpr (MODE == 1) store_s(ls + TR * SP, g1);
        }
        if constexpr (vecs_too) {
#pragma unroll 1
            for (int t = t0 + SV * 64 * NW; t < 16 * CF * J; t += SV * 64 * NW) {
                load_s(bx, rv, 16 * CF, t, vec, gv);
                store_s(ls + BR * SP, gv);
            }
        }
    };
    // where the wave's fragments' scales stand
    auto seg_of_row = [&](int f) { return MODE == 1 ? (f >= RH ? TR : 0) + 16 * (w * RH + f % RH) : 16 * (w * RF + f); };
    const int rd = c * 128 + 16 * (q ^ ((c >> 1) & 7));         // step 0's chunk of lane (c, q); step 1: ^ 64
    const bool vec4 = (N & 3) == 0 && ((uintptr_t)a.y & 15) == 0;

    // While unit u multiplies, its codes stand in LDS and those of units u + 1
    // and u + 2 are on their way to A[(u + 1) % 2], A[u % 2] and X likewise:
    // every load has a whole unit's time before its registers are needed.
    // (Loads return in the order of issue: a wait for the vectors alone, one
    // unit ahead, would wait for the weights issued before them too.)
    u32x4 A0[RF][2], A[2][RF][2], X[2][XU];
    auto first_loads = [&](int row_base) {
        set_rows(row_base);
        load_a(0, A0);
        load_x(0, X[0]);
        load_x(1, X[1]);
        load_a(1, A[1]);
        load_a(2, A[0]);
    };
    first_loads(rt0 * TR);
    for (int rt = rt0; rt < rt1; ++rt) {
        const int row_base = rt * TR;
        if (rt == rt0)
            stage_scales(row_base, std::true_type{});
        else
            stage_scales(row_base, std::false_type{});
        store_a(A0);
        store_x(0, X[0]);
        f32x4 acc[RF][CF];
#pragma unroll
        for (int f = 0; f < RF; ++f)
#pragma unroll
            for (int g = 0; g < CF; ++g) acc[f][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        __syncthreads();
        auto slab = [&](int j, auto LAST) {
            constexpr bool last = decltype(LAST)::value;
            const uint8_t *const sc = ls + c * SP + 16 * j + 4 * q;
            uint32_t ta[RF], tb[CF];
            auto unit = [&](auto HALF) {
                constexpr int h = decltype(HALF)::value;            // the unit's vector buffer too
                constexpr bool more = !last || h == 0;              // another unit follows
                const int u = 2 * j + h;
                u32x4 F[2][RF], B[2][GB];
                // group i of the unit: step i / HG's vectors i % HG * GB ..
                auto read_b = [&](int i, u32x4 (&b)[GB]) {
#pragma unroll
                    for (int g = 0; g < GB; ++g)
                        b[g] = *(const u32x4 *)(lx + h * XB + (i % HG * GB + g) * 2048 + (rd ^ (64 * (i / HG))));
                };
                if constexpr (h == 0) {
#pragma unroll
                    for (int f = 0; f < RF; ++f) ta[f] = *(const uint32_t *)(sc + seg_of_row(f) * SP);
#pragma unroll
                    for (int g = 0; g < CF; ++g) tb[g] = *(const uint32_t *)(sc + (BR + 16 * g) * SP);
                }
#pragma unroll
                for (int f = 0; f < RF; ++f) F[0][f] = *(const u32x4 *)(la + f * 2048 + rd);
                read_b(0, B[0]);
#pragma unroll
                for (int f = 0; f < RF; ++f) F[1][f] = *(const u32x4 *)(la + f * 2048 + (rd ^ 64));
                if constexpr (!last) load_x(u + 2, X[h]);
                asm volatile("" ::: "memory");                      // (the next unit's codes go where these were)
                if constexpr (more) {
                    store_a(A[h ^ 1]);
                    if constexpr (!last) load_a(u + 3, A[h ^ 1]);
                }
                auto part = [&](auto IDX) {
                    constexpr int i = decltype(IDX)::value, s = i / HG, g0 = i % HG * GB;
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (i + 1 < 2 * HG) read_b(i + 1, B[(i + 1) & 1]);
#pragma unroll
                    for (int g = 0; g < GB; ++g)
#pragma unroll
                        for (int f = 0; f < RF; ++f)
                            acc[f][g0 + g] = mfma_mx4_op<2 * h + s>(F[s][f], B[i & 1][g], acc[f][g0 + g], ta[f], tb[g0 + g]);
                    // (the compiler would move the products past the barrier to
                    // their last use, with all their operands held until then)
#pragma unroll
                    for (int g = 0; g < GB; ++g)
#pragma unroll
                        for (int f = 0; f < RF; ++f) asm volatile("" : "+v"(acc[f][g0 + g]));
                };
                part(std::integral_constant<int, 0>{});
                part(std::integral_constant<int, 1>{});
                if constexpr (HG > 1) {
                    part(std::integral_constant<int, 2>{});
                    part(std::integral_constant<int, 3>{});
                }
                if constexpr (more) store_x(h ^ 1, X[h ^ 1]);
                __syncthreads();
            };
            unit(std::integral_constant<int, 0>{});
            unit(std::integral_constant<int, 1>{});
        };
        for (int j = 0; j + 1 < J; ++j) slab(j, std::false_type{});
        slab(J - 1, std::true_type{});

        // the next tile's first loads go out before this tile's results
        if (rt + 1 < rt1) first_loads(row_base + TR);
        // lane (c, q) holds rows 4 q .. 4 q + 3 of vector c of each fragment
        int vc = c;
        asm volatile("" : "+v"(vc));                                // (the rows' addresses are formed here, not kept)
#pragma unroll
        for (int g = 0; g < CF; ++g) {
            const int v = 16 * g + vc;
            if (v < nv) {
                float *const yr = a.y + (size_t)(gather ? (int)vecs[v] : vstart + v) * N;
#pragma unroll
                for (int f = 0; f < RH; ++f) {
                    const int n0 = row_base + 16 * RH * w + 16 * f + 4 * q;
                    float r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        r[k] = MODE == 1 ? swiglu(acc[f][g][k], acc[f + RF - RH][g][k]) : acc[f][g][k];
                    if (n0 < N) {
                        if (vec4) {
                            *(float4 *)(yr + n0) = make_float4(r[0], r[1], r[2], r[3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (n0 + k < N) yr[n0 + k] = r[k];
                        }
                    }
                }
            }
        }
    }
}

// A workgroup takes a run of up to bt_chunk row tiles of one item.  Workgroup
// b runs on XCD b % 8; the runs (item-major) are dealt to the XCDs in
// contiguous parts, so that an XCD's L2 holds the vectors of a few experts,
// and an expert's second chunk finds its weights there.
template <int MODE, int CHUNK>
__global__ __launch_bounds__(64 * kMx4Waves, 2) void qmv_mx4_tile_kernel(const Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int TR = 16 * kMx4RF * kMx4Waves / (MODE == 1 ? 2 : 1);
    uint16_t *const list = (uint16_t *)lds;           // [CHUNK]
    uint8_t *const buf = lds + 2 * CHUNK;
    const int runs = (a.bt_row_tiles + a.bt_chunk - 1) / a.bt_chunk;   // per item
    int item = -1, rt0 = 0, rt1 = 0;
    auto pick = [&](int items) {
        const int all = items * runs, per_xcd = (all + 7) / 8, i = blockIdx.x >> 3;
        const int r = i < per_xcd ? (int)(blockIdx.x & 7) * per_xcd + i : all;
        if (r < all) {
            item = r / runs;
            rt0 = (r - item * runs) * a.bt_chunk;
            rt1 = min(rt0 + a.bt_chunk, a.bt_row_tiles);
        }
        return item;
    };
    int e = 0, nv, vstart = 0;
    const bool gather = a.ids != nullptr;
    if (gather) {
        // (a call without any id in [0, E) still has its zero rows: one item)
        const int P = a.M * a.top_k;
        const RoutedItem it = routed_item<CHUNK>(a.ids, P, a.E, (int *)buf, list, [&](int items) { return pick(max(items, 1)); });
        if (item < 0) return;
        e = it.e;
        nv = it.nv;
        routed_zero_rows(a, item, max(it.items, 1), rt0 * TR, min(rt1 * TR, a.N));
        if (nv == 0) return;
    } else {
        if (pick((a.M + CHUNK - 1) / CHUNK) < 0) return;
        vstart = item * CHUNK;
        nv = min(CHUNK, a.M - vstart);
    }
    const uint16_t *const vecs = gather ? list : nullptr;
    if (CHUNK > 64 && nv > 64)
        mx4_tile_run<MODE, CHUNK / 16, CHUNK>(a, buf, e, rt0, rt1, vecs, vstart, nv);
    else if (nv > 32)
        mx4_tile_run<MODE, 4, CHUNK>(a, buf, e, rt0, rt1, vecs, vstart, nv);
    else if (nv > 16)
        mx4_tile_run<MODE, 2, CHUNK>(a, buf, e, rt0, rt1, vecs, vstart, nv);
    else
        mx4_tile_run<MODE, 1, CHUNK>(a, buf, e, rt0, rt1, vecs, vstart, nv);
}

// -------------------------------------------------------------- few vectors
// Up to 16 vectors of an expert (a dense matrix), or (MODE 2, the combine) a
// token's slots, each with its expert, against one tile of 16 rows.  The call waits for its weight bytes, so the 4
// waves of a workgroup split K -- wave w takes units (256 weights) w, w + 4,
// ... -- and each has up to kFewAhead units of its rows on their way from the
// start; the vectors and the scale bytes are staged in LDS once.  The waves'
// partial tiles are summed in wave order.  Columns past the last vector
// repeat one (nothing of them is stored).  One token's top-4 of 32, 2880 ->
// 2880: 7.2 us for 18 MB (2.5 TB/s: 720 workgroups of a few loads each, most
// of it the way from the ids to the first codes), gate/up 12.1 us for 35 MB;
// 7168 -> 7168 with 4 vectors 9 us for 27 MB; the combine of 4 tokens x 8,
// 2048 -> 7168: 51 us for 250 MB, 4.9 TB/s.
constexpr int kFewAhead = 4;

// Bytes from vector to vector of the staged codes: whole units, and 16 more
// so that the 16 vectors of a read lie in different bank groups.
__host__ __device__ constexpr int mx4_x_pitch(int U) { return (U + 7) / 8 * 128 + 16; }

template <int MODE>
__global__ __launch_bounds__(64 * kMx4Waves) void qmv_mx4_few_kernel(const Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int NW = kMx4Waves, H = MODE == 1 ? 2 : 1, D = kFewAhead;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4, lr = lane >> 3, lc = lane & 7;
    const int U = a.units, J = (U + 15) >> 4, NU = (U + 7) >> 3;
    const int SP = mx4_scale_pitch(J), XP = mx4_x_pitch(U);
    const int N = a.N;
    const uint32_t rsb = (uint32_t)a.rsb;
    const bool gather = MODE != 2 && a.ids != nullptr;
    const int P = gather ? a.M * a.top_k : a.M;

    uint16_t *const list = (uint16_t *)lds;                    // [kMx4Few]
    uint8_t *const la = lds + 64 + w * (H * 2048);             // this wave's weight pieces; its partial sums
    uint8_t *const lx = lds + 64 + NW * H * 2048;              // [vectors] x XP
    uint8_t *const lxs = lx + a.bt_vmax * XP;                  // [vectors] x SP
    uint8_t *const ls = lxs + a.bt_vmax * SP;                  // [H or slots][16 rows] x SP

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
        v0 = blockIdx.y * kMx4Few;
        nv = min(kMx4Few, a.M - v0);
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
        const RoutedItem it = routed_item<kMx4Few>(a.ids, P, a.E, (int *)(lds + 64), list, [&](int items) {
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
    const int vmask = nv - 1;                                  // columns past nv repeat
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
        const int ns = min(per, slots - s0), total = ns * NU;
        auto load_a = [&](int i, u32x4 (&R)[H][2]) {
            const int g = w + NW * i;
            const int slot = MODE == 2 ? g / NU : 0, u = g - slot * NU;
            int ee = e;
            long long size = a.expert_cb;
            if constexpr (MODE == 2) {
                ee = __builtin_amdgcn_readlane(ids_lane, g < total ? s0 + slot : 0);
                if ((unsigned)ee >= (unsigned)a.E) ee = 0, size = 0;           // reads zeros
            }
            const uint32_t so = g < total ? 128u * u : kXPast;
#pragma unroll
            for (int h = 0; h < H; ++h) {                                      // (nt: read once)
                const __amdgpu_buffer_rsrc_t rc = buffer_rsrc((h ? a.codes2 : a.codes) + ee * a.expert_cb, size);
#pragma unroll
                for (int k = 0; k < 2; ++k) R[h][k] = __builtin_amdgcn_raw_buffer_load_b128(rc, oc[k] + so, 0, 2);
            }
        };
        auto stage_s = [&](const uint8_t *base, long long bytes, int rows, auto row_of, uint8_t *dst) {
            const uintptr_t p0 = (uintptr_t)base;
            const __amdgpu_buffer_rsrc_t r =
                buffer_rsrc((const void *)(p0 & ~(uintptr_t)3), ((long long)(p0 & 3) + bytes + 3) & ~3ll);
            for (int t = tid; t < rows * J; t += 64 * NW) {
                const int row = t / J, j = t - row * J;
                const uint32_t o = (uint32_t)(p0 & 3) + row_of(row) * rsb + 16u * j;
                *(u32x4 *)(dst + row * SP + 16 * j) = seg_order<true>(load_seg<true>(r, o), o, U - 16 * j);
            }
        };
        auto tile_row = [&](int row) { return (uint32_t)min(row0 + row, N - 1); };
#pragma unroll
        for (int i = 0; i < D; ++i) load_a(i, A[i]);
        // the vectors (MODE 2: those of the group's slots)
        const int vecs = MODE == 2 ? (a.x_per_slot ? ns : 1) : nv;
        for (int t = tid; t < vecs * 8 * NU; t += 64 * NW) {
            const int v = t / (8 * NU), b = t - v * 8 * NU;
            const uint32_t o = vec_row(MODE == 2 ? s0 + v : v) * (uint32_t)a.x_vec_bytes + 16u * b;
            *(u32x4 *)(lx + v * XP + 16 * b) =
                __builtin_amdgcn_raw_buffer_load_b128(rx, b < U ? o : kXPast, 0, 0);
        }
        stage_s((const uint8_t *)a.xs, (long long)x_rows * rsb, vecs,
                [&](int v) { return vec_row(MODE == 2 ? s0 + v : v); }, lxs);
        if constexpr (MODE == 2) {
            for (int k = 0; k < ns; ++k) {
                int ee = __builtin_amdgcn_readlane(ids_lane, s0 + k);
                if ((unsigned)ee >= (unsigned)a.E) ee = 0;                     // (unused)
                stage_s(a.scales + ee * a.expert_sb, a.expert_sb, 16, tile_row, ls + k * 16 * SP);
            }
        } else {
            stage_s(a.scales + e * a.expert_sb, a.expert_sb, 16, tile_row, ls);
            if constexpr (H == 2) stage_s(a.scales2 + e * a.expert_sb, a.expert_sb, 16, tile_row, ls + 16 * SP);
        }
        __syncthreads();

        f32x4 acc[H];
#pragma unroll
        for (int h = 0; h < H; ++h) acc[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int wst = swz_chunk(lr, lc), rd = c * 128 + 16 * (q ^ ((c >> 1) & 7));
        const int vc = MODE == 2 ? 0 : (c < nv ? c : vmask);
        const int mine = total > w ? (total - w + NW - 1) / NW : 0;            // this wave's units
        for (int i0 = 0; i0 < mine; i0 += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int i = i0 + d;
                if (i < mine) {
                    const int g = w + NW * i;
                    const int slot = MODE == 2 ? g / NU : 0, u = g - slot * NU;
                    const int v = MODE == 2 ? (a.x_per_slot ? slot : 0) : vc;
                    // slab u / 2's bytes of this unit's two steps in bits 0-15
                    const int sh = 16 * (u & 1), so = 16 * (u >> 1) + 4 * q;
                    const uint32_t tb = *(const uint32_t *)(lxs + v * SP + so) >> sh;
                    const u32x4 B0 = *(const u32x4 *)(lx + v * XP + 128 * u + 16 * q);
                    const u32x4 B1 = *(const u32x4 *)(lx + v * XP + 128 * u + 64 + 16 * q);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        *(u32x4 *)(la + h * 2048 + wst) = A[d][h][0];
                        *(u32x4 *)(la + h * 2048 + 1024 + (wst ^ 64)) = A[d][h][1];
                    }
                    asm volatile("" ::: "memory");                             // (written before read: one wave's LDS)
                    load_a(i + D, A[d]);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const uint32_t ta =
                            *(const uint32_t *)(ls + ((MODE == 2 ? slot : h) * 16 + c) * SP + so) >> sh;
                        const u32x4 F0 = *(const u32x4 *)(la + h * 2048 + rd);
                        const u32x4 F1 = *(const u32x4 *)(la + h * 2048 + (rd ^ 64));
                        acc[h] = mfma_mx4_op<0>(F0, B0, acc[h], ta, tb);
                        acc[h] = mfma_mx4_op<1>(F1, B1, acc[h], ta, tb);
                    }
                    asm volatile("" ::: "memory");
                    if constexpr (MODE == 2) {
                        if ((g + NW) / NU != slot || i + 1 == mine) {          // this wave's last unit of the slot
                            const float rw = __uint_as_float(
                                __builtin_amdgcn_readlane(__float_as_uint(rw_lane), s0 + slot));
                            // (a slot without an expert is 0 whatever scales
                            // its vector has; zero codes times NaN are not)
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
// A dense matrix against thousands of vectors is bound by the matrix cores
// and by LDS.  256 x 256 tiles, 4 x 2 waves of 64 rows x 128 vectors: a wave's
// step reads 12 fragments from LDS for 32 products.  Both operands are staged
// for a unit (256 weights, 2 steps) at a time, double-buffered, half of a
// unit's loads in flight during each step.  The vectors' fragments are read in
// two groups of 4, each group while the other is multiplied, and a row's
// fragment as soon as its last product of the step is given out, so a step
// enters with its operands read.  One barrier a unit, in the middle of its
// second step, where every fragment of the unit is read.
// 8192 vectors, 7168 -> 7168: 266 to 296 us from card to card, 2.8 to 3.2
// PFLOP/s (531 in the tile kernel's 128 x 64).  With one set of inputs again and
// again, before the last round's halves: 270, in 128 x 128 tiles of 4 waves 398;
// all-zero operands 227, which the chip's power limit explains (2.1 GHz against
// 2.4); of those the products alone take 145, LDS reads add 20, the staging stores
// 30, the loads 30; loads two steps ahead, or written between other products,
// change nothing.
//
// RF: 16-row fragments per wave; the tile starts at row0 and vec0.
template <int RF>
__device__ __forceinline__ void mx4_wide_tile(const Args &a, uint8_t *lds, int row0, int vec0)
{
    constexpr int CF = 8, NWR = 4, NWC = 2, NW = NWR * NWC;
    constexpr int BR = 16 * RF * NWR, BC = 16 * CF * NWC;   // tile: rows, vectors
    constexpr int AB = BR * 128, XB = BC * 128;       // bytes of a unit's codes
    constexpr int NS = BR + BC;                       // staged scale rows, at most one a thread
    constexpr int KA = BR / 8 / NW, KX = BC / 8 / NW; // staged pieces (8 rows x 128 bytes) per wave and unit
    constexpr int GB = CF / 2;                        // column fragments read at a time
    static_assert(NS <= 64 * NW && BR % 64 == 0 && KA % 2 == 0 && KX % 2 == 0 && NW % 2 == 0, "staging split");
    uint8_t *const ld = lds;                          // [2][AB + XB]
    uint8_t *const ls = lds + 2 * (AB + XB);          // [2][NS] x 16 bytes

    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = w / NWC, wc = w % NWC;
    const int c = lane & 15, q = lane >> 4, lr = lane >> 3, lc = lane & 7;
    const int U = a.units, J = (U + 15) >> 4;

    f32x4 acc[RF][CF];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int g = 0; g < CF; ++g) acc[f][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // wave w stages pieces w, w + NW, ... of each operand; rows past N and
    // vectors past M lie past the buffers' ends and read zeros
    const __amdgpu_buffer_rsrc_t rc = buffer_rsrc(a.codes, a.expert_cb);
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.x, (long long)a.M * a.x_vec_bytes);
    const uint32_t oa = (uint32_t)(row0 + 8 * w + lr) * (uint32_t)a.rcb + 16u * lc;
    const uint32_t ox = (uint32_t)(vec0 + 8 * w + lr) * (uint32_t)a.x_vec_bytes + 16u * lc;
    const uint32_t pa = 8u * NW * (uint32_t)a.rcb, px = 8u * NW * (uint32_t)a.x_vec_bytes;
    u32x4 ga[KA / 2], gx[KX / 2];                     // half a unit's pieces
    auto load_half = [&](int u, int half) {
        // (a row's blocks past its end: zeros; the pieces' offsets are built
        // anew each time: registers are scarcer than additions)
        const bool ok = 8 * u + lc < U;
        uint32_t ta = oa, tx = ox;
        asm volatile("" : "+v"(ta), "+v"(tx));
#pragma unroll
        for (int k = 0; k < KA / 2; ++k)
            ga[k] = __builtin_amdgcn_raw_buffer_load_b128(rc, ok ? ta + ((half * (KA / 2) + k) * pa + 128u * u) : kXPast, 0, 0);
#pragma unroll
        for (int k = 0; k < KX / 2; ++k)
            gx[k] = __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? tx + ((half * (KX / 2) + k) * px + 128u * u) : kXPast, 0, 0);
    };
    // piece p stands in fragment p / 2, rows 8 (p % 2) ..; p has the wave's parity
    const int wst = (w >> 1) * 2048 + (w & 1) * 1024 + (swz_chunk(lr, lc) ^ ((w & 1) << 6));
    auto store_half = [&](int buf, int half) {
        uint8_t *const d = ld + buf * (AB + XB) + wst;
#pragma unroll
        for (int k = 0; k < KA / 2; ++k) *(u32x4 *)(d + (half * (KA / 2) + k) * (NW * 1024)) = ga[k];
#pragma unroll
        for (int k = 0; k < KX / 2; ++k) *(u32x4 *)(d + AB + (half * (KX / 2) + k) * (NW * 1024)) = gx[k];
    };

    // scale bytes: thread t takes 16 bytes (a slab, two units) of row t of the
    // tile or of vector t - BR, the same tensor for a whole wave
    const bool vecs = w >= BR / 64;
    const uintptr_t p0 = (uintptr_t)(vecs ? (const uint8_t *)a.xs : a.scales);
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(
        (const void *)(p0 & ~(uintptr_t)3), ((long long)(p0 & 3) + (long long)(vecs ? a.M : a.N) * a.rsb + 3) & ~3ll);
    const uint32_t os = (uint32_t)(p0 & 3) +
                        (uint32_t)(vecs ? min(vec0 + tid - BR, a.M - 1) : min(row0 + tid, a.N - 1)) * (uint32_t)a.rsb;
    auto put_s = [&](int j, u32x4 v) {
        if (NS == 64 * NW || tid < NS) *(u32x4 *)(ls + (j & 1) * (NS * 16) + tid * 16) = v;
    };
    const int rd = c * 128 + 16 * (q ^ ((c >> 1) & 7));

    u32x4 F[RF], B[2][GB];                            // fragments: rows; two groups of vectors
    uint32_t ta[RF], tb[2][GB];                       // their scale bytes, a slab's dword each
    const uint8_t *const fa = ld + wr * RF * 2048, *const fb = ld + AB + wc * CF * 2048;
    // step s of the unit in buffer h
    auto read_f = [&](int h, int s, int f) {
        uint32_t o = rd ^ (64 * s);
        asm volatile("" : "+v"(o));
        F[f] = *(const u32x4 *)(fa + h * (AB + XB) + f * 2048 + o);
    };
    auto read_b = [&](int h, int s, int grp) {
        uint32_t o = rd ^ (64 * s);
        asm volatile("" : "+v"(o));
#pragma unroll
        for (int g = 0; g < GB; ++g) B[grp][g] = *(const u32x4 *)(fb + h * (AB + XB) + (grp * GB + g) * 2048 + o);
    };
    const uint8_t *const fs = ls + c * 16 + 4 * q;
    auto read_ta = [&](int j, int f) { ta[f] = *(const uint32_t *)(fs + (j & 1) * (NS * 16) + 256 * (wr * RF + f)); };
    auto read_tb = [&](int j, int grp) {
#pragma unroll
        for (int g = 0; g < GB; ++g)
            tb[grp][g] = *(const uint32_t *)(fs + (j & 1) * (NS * 16) + BR * 16 + 256 * (wc * CF + grp * GB + g));
    };

    {
        const ScaleSeg sg = load_seg<true>(rs, os);
        load_half(0, 0);
        store_half(0, 0);
        load_half(0, 1);
        store_half(0, 1);
        load_half(1, 0);
        put_s(0, seg_order<true>(sg, os, U));
    }
    __syncthreads();
    read_b(0, 0, 0);
    read_tb(0, 0);
#pragma unroll
    for (int f = 0; f < RF; ++f) {
        read_f(0, 0, f);
        read_ta(0, f);
    }
    // a slab: LAST 0: two more follow; 1: one more; 2: none
    auto slab = [&](int j, auto LAST) {
        constexpr int last = decltype(LAST)::value;
        ScaleSeg sg;
        read_tb(j, 1);
        auto step = [&](auto HALF, auto SIDX) {
            constexpr int h = decltype(HALF)::value;  // the unit's buffer too
            constexpr int s = decltype(SIDX)::value;
            constexpr bool more = last < 2 || h == 0; // another unit follows
            if constexpr (h == 1 && s == 0 && last < 2) sg = load_seg<last == 1>(rs, os + 16u * (j + 1));
            read_b(h, s, 1);
            __builtin_amdgcn_s_setprio(1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int g = 0; g < GB; ++g)
#pragma unroll
                for (int f = 0; f < RF; ++f)
                    acc[f][g] = mfma_mx4_op<2 * h + s>(F[f], B[0][g], acc[f][g], ta[f], tb[0][g]);
            // (keeps the products here)
#pragma unroll
            for (int g = 0; g < GB; ++g)
#pragma unroll
                for (int f = 0; f < RF; ++f) asm volatile("" : "+v"(acc[f][g]));
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(0);
            if constexpr (more) store_half(h ^ 1, s);
            if constexpr (h == 1 && s == 1 && last < 2) put_s(j + 1, seg_order<last == 1>(sg, os, U - 16 * (j + 1)));
            // every fragment of this unit is read, and the next unit is staged
            if constexpr (s == 1 && more) __syncthreads();
            if constexpr (s == 0 && more) load_half(2 * j + h + 1, 1);
            if constexpr (s == 1 && last < 2) load_half(2 * j + h + 2, 0);
            if constexpr (s == 0 || more) read_b(s ? h ^ 1 : h, s ^ 1, 0);
            if constexpr (h == 1 && s == 1 && last < 2) read_tb(j + 1, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int f = 0; f < RF; ++f) {
#pragma unroll
                for (int g = 0; g < GB; ++g)
                    acc[f][GB + g] = mfma_mx4_op<2 * h + s>(F[f], B[1][g], acc[f][GB + g], ta[f], tb[1][g]);
#pragma unroll
                for (int g = 0; g < GB; ++g) asm volatile("" : "+v"(acc[f][GB + g]));
                if constexpr (s == 0 || more) read_f(s ? h ^ 1 : h, s ^ 1, f);
                if constexpr (h == 1 && s == 1 && last < 2) read_ta(j + 1, f);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        step(std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 1>{}, std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    };
    int j = 0;
    for (; j + 2 < J; ++j) slab(j, std::integral_constant<int, 0>{});
    if (j + 1 < J) slab(j++, std::integral_constant<int, 1>{});
    slab(j, std::integral_constant<int, 2>{});

    const bool vec4 = (a.N & 3) == 0 && ((uintptr_t)a.y & 15) == 0;
#pragma unroll
    for (int g = 0; g < CF; ++g) {
        const int v = vec0 + 16 * (wc * CF + g) + c;
        if (v < a.M) {
            float *const yr = a.y + (size_t)v * a.N;
#pragma unroll
            for (int f = 0; f < RF; ++f) {
                const int n0 = row0 + 16 * (wr * RF + f) + 4 * q;
                if (n0 < a.N) {
                    if (vec4) {
                        *(float4 *)(yr + n0) = make_float4(acc[f][g][0], acc[f][g][1], acc[f][g][2], acc[f][g][3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (n0 + k < a.N) yr[n0 + k] = acc[f][g][k];
                    }
                }
            }
        }
    }
}

// The tiles lie in groups of bt_vmax vector chunks, chunk-fastest inside, and
// are dealt to the XCDs in contiguous parts: the tiles an XCD runs at a time
// share both operands.  Of an XCD's bt_per_xcd tiles all from bt_chunk on are
// done as two halves of 128 rows.
__global__ __launch_bounds__(512, 2) void qmv_mx4_wide_kernel(const Args a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int i = blockIdx.x >> 3, half = i - a.bt_chunk;
    const int tile = (blockIdx.x & 7) * a.bt_per_xcd + (half < 0 ? i : a.bt_chunk + half / 2);
    if (tile >= a.bt_tiles) return;
    const int chunks = (a.M + 255) / 256, group = a.bt_vmax * a.bt_row_tiles;
    const int gi = tile / group, in = tile - gi * group, gw = min(a.bt_vmax, chunks - gi * a.bt_vmax);
    const int row0 = in / gw * 256, vec0 = (gi * a.bt_vmax + in % gw) * 256;
    if (half < 0)
        mx4_wide_tile<4>(a, lds, row0, vec0);
    else if (row0 + 128 * (half & 1) < a.N)
        mx4_wide_tile<2>(a, lds, row0 + 128 * (half & 1), vec0);
}

extern const void *const kTableMx4Wide[1];
const void *const kTableMx4Wide[1] = {
    (const void *)&qmv_mx4_wide_kernel,
};

extern const void *const kTableMx4Few[3];
const void *const kTableMx4Few[3] = {
    (const void *)&qmv_mx4_few_kernel<0>,
    (const void *)&qmv_mx4_few_kernel<1>,
    (const void *)&qmv_mx4_few_kernel<2>,
};

// [chunks of 64 or 128 vectors][plain, gate/up]
extern const void *const kTableMx4Tile[4];
const void *const kTableMx4Tile[4] = {
    (const void *)&qmv_mx4_tile_kernel<0, 64>,
    (const void *)&qmv_mx4_tile_kernel<1, 64>,
    (const void *)&qmv_mx4_tile_kernel<0, 128>,
    (const void *)&qmv_mx4_tile_kernel<1, 128>,
};

}  // namespace qmv
