// qmv_routed.hpp -- what the matrix-core kernels of MXFP4 and e4m3 activations
// share: their operand types, the order of a piece of codes in LDS, and the
// routed calls' work.
#pragma once

#include "qmv_device.hpp"

namespace qmv {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kXPast = 0x80000000u;       // >= every buffer size: reads zeros

// A piece of 16-byte chunks in LDS: chunk k of row r (128 bytes) stands so that
// 16 lanes that write or read the same chunk of 16 rows, or 8 chunks of 2 rows,
// touch 16 different bank groups.
__device__ __forceinline__ int swz_chunk(int row, int chunk) { return row * 128 + 16 * (chunk ^ ((row >> 1) & 7)); }

// The routed calls' work: an expert's pairs in chunks of at most CHUNK.
// Every workgroup counts the pairs per expert itself (LDS atomics on whole
// numbers: the same counts everywhere), so the grid needs no device-wide
// knowledge: item i is the i-th (expert, chunk) of the experts in order.
constexpr int kRoutedWaves = 4;       // wave64s of a workgroup

struct RoutedItem {
    int e;               // expert
    int nv;              // vectors of the chunk (0: no pair has an id in [0, E))
    int items;           // items of the call
};

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8: within 16 lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // lane 15 of rows 0, 2 to rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // lane 31 to rows 2, 3
    return v;
}

// cnt: 1024 + 8 words of LDS.  `pick` maps the number of items to this
// workgroup's item (or -1), and `order` that, the first item of its expert and
// how many it has to the workgroup's chunk of the expert; the chunk's pairs go to
// list.  ids: thread t looks at ids t, t + 256, ...  Every wave finds the item by
// itself.
template <int CHUNK, class Pick, class Order>
__device__ __forceinline__ RoutedItem routed_item(const int32_t *ids, int P, int E, int *cnt, uint16_t *list, Pick pick, Order order)
{
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, w = tid >> 6;
    int *const info = cnt + 1024;
    int idv[32];
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j * 256 < P) idv[j] = ids[min(tid + j * 256, P - 1)];
    *(int4 *)(cnt + 4 * tid) = make_int4(0, 0, 0, 0);
    if (tid == 0) info[4] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j * 256 < P) {
            if (tid + j * 256 < P && (unsigned)idv[j] < (unsigned)E) atomicAdd(&cnt[idv[j]], 1);
        }
    __syncthreads();
    // lane l: experts 16 l .. 16 l + 15 (those past E have no pairs)
    int c[16], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int4 v = *(const int4 *)(cnt + 16 * lane + 4 * i);
        c[4 * i] = v.x, c[4 * i + 1] = v.y, c[4 * i + 2] = v.z, c[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) n += (c[i] + CHUNK - 1) / CHUNK;
    int before = wave_scan(n);
    const int items = __builtin_amdgcn_readlane(before, 63);
    before -= n;
    const int item = pick(items);
    RoutedItem it = {0, 0, items};
    if (item < 0 || item >= items) return it;
    const unsigned long long owner = __ballot(item >= before && item < before + n);
    int e = 0, first = 0, total = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int k = (c[i] + CHUNK - 1) / CHUNK;
        if (item >= before && item < before + k) e = 16 * lane + i, first = before, total = c[i];
        before += k;
    }
    const int o = __ffsll((long long)owner) - 1;
    it.e = __builtin_amdgcn_readlane(e, o);
    first = __builtin_amdgcn_readlane(first, o);
    total = __builtin_amdgcn_readlane(total, o);
    const int nch = (total + CHUNK - 1) / CHUNK, chunk = order(item, first, nch);
    const int cs = (total + nch - 1) / nch;           // equal chunks
    it.nv = min(cs, total - chunk * cs);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j * 256 < P) m |= (uint32_t)(idv[j] == it.e && tid + j * 256 < P) << j;
    if (nch == 1) {
        // one chunk: the order of its pairs changes no result
        for (; m; m &= m - 1) list[atomicAdd(&info[4], 1)] = (uint16_t)(tid + 256 * (__ffs(m) - 1));
    } else {
        // the pairs of e in (thread, round) order, the same in every
        // workgroup: this chunk's ranks
        n = (int)__popc(m);
        int rank = wave_scan(n);
        if (lane == 63) info[w] = rank;
        __syncthreads();
        for (int i = 0; i < 4; ++i)
            if (i < w) rank += info[i];
        rank -= n + chunk * cs;
        for (; m; m &= m - 1, ++rank)
            if (rank >= 0 && rank < it.nv) list[rank] = (uint16_t)(tid + 256 * (__ffs(m) - 1));
    }
    __syncthreads();
    return it;
}

// The chunks of an expert in order.
template <int CHUNK, class Pick>
__device__ __forceinline__ RoutedItem routed_item(const int32_t *ids, int P, int E, int *cnt, uint16_t *list, Pick pick)
{
    return routed_item<CHUNK>(ids, P, E, cnt, list, pick, [](int item, int first, int) { return item - first; });
}

// The rows [n0, n1) of pairs whose id is outside [0, E) are zeros: of `items`
// items, item i takes the pairs i, i + items, ...
__device__ __forceinline__ void routed_zero_rows(const Args &a, int item, int items, int n0, int n1)
{
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, w = tid >> 6, P = a.M * a.top_k;
    for (int p0 = item + items * 16 * w; p0 < P; p0 += items * 16 * kRoutedWaves) {
        const int p = p0 + items * (lane & 15);
        const bool bad = lane < 16 && p < P && (unsigned)a.ids[min(p, P - 1)] >= (unsigned)a.E;
        for (unsigned long long m = __ballot(bad); m; m &= m - 1) {
            float *const yr = a.y + (size_t)(p0 + items * (__ffsll((long long)m) - 1)) * a.N;
            for (int n = n0 + lane; n < n1; n += 64) yr[n] = 0.0f;
        }
    }
}

}  // namespace qmv
