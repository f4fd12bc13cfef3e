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

namespace qmv {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kXPast = 0x80000000u;       // >= every buffer size: reads zeros

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

}  // namespace qmv
