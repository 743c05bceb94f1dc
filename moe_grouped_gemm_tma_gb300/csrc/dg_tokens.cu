// Tokens by expert and back, around the grouped products: where every routed slot goes (dg_moe_sort_contiguous,
// dg_moe_sort_masked), the tokens' rows there (dg_moe_gather), the weighted sum of the experts' rows back to the tokens
// (dg_moe_combine), and that sum's gradient (dg_moe_combine_backward). The gather's own gradient is the sum without
// weights.
//
// Sort. A counting sort by expert that keeps the slots' order, so that its result does not depend on timing: a warp takes
// consecutive slots, 32 at a time; ballots over the bits of the expert give each lane the others with its own, whose number
// below it is its place among the 32. Up to SORT_ALONE slots are sorted by one launch, whose CTAs each count all slots and
// place 512 of them; more are cut into chunks, whose counts a first launch writes, a second adds up and a third uses. It is
// bound by the latency of its steps: 512 slots of 256 experts take 4.3 us in a CUDA graph, 65512 7.2, 262144 17.
//
// The rows are moved token by token: a token's row is read once, however many experts it goes to. Rows without a token inside an
// expert's block of 128 are zeroed by warps of their own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "dg.h"
#include "dg_host.cuh"
#include "dg_ptx.cuh"
#include "dg_quant.cuh"

namespace dg {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// ------------------------------------------------------------------------------------ sort
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ALONE = 16384;                 // slots that one launch sorts
constexpr int SORT_CHUNKS = 608;                  // chunks at most: four CTAs an SM
constexpr int64_t SORT_MAX_SLOTS = 1 << 23;       // (a chunk's counts fit 16 bits: it has 13824 slots then)

struct SortParams {
    const int32_t* ids;
    int32_t* rows;
    int32_t* counts;
    int32_t* m_indices;   // null: masked layout
    int32_t* totals;      // [E], then, by expert, the chunks' counts, which become those of the chunks before
    int32_t* chunk_counts;
    int slots, experts, bits, blocks, max_m, groups, chunks;
};

__device__ __forceinline__ unsigned lanes_below() {
    unsigned m;
    asm("mov.u32 %0, %%lanemask_lt;" : "=r"(m));
    return m;
}

// A slot's expert, `experts` where there is none.
__device__ __forceinline__ int slot_expert(const SortParams& p, int slot) {
    const int id = slot < p.slots ? ld_input(p.ids + slot) : -1;
    return static_cast<unsigned>(id) < static_cast<unsigned>(p.experts) ? id : p.experts;
}

// The lanes that have the same e, of `bits` bits. (match.any goes through the values one by one: a group of 32 slots took
// 1 us.)
__device__ __forceinline__ unsigned same_lanes(int e, int bits) {
    unsigned same = FULL;
    for (int i = 0; i < bits; ++i) {
        const unsigned ones = __ballot_sync(FULL, e >> i & 1);
        same &= e >> i & 1 ? ones : ~ones;
    }
    return same;
}

// ALONE: the only launch; each CTA counts all slots, and places its own chunk. COUNT: the first of three launches, which
// writes the chunks' counts; PLACE: the last, when they have been added up.
enum SortStep { SORT_STEP_ALONE, SORT_STEP_COUNT, SORT_STEP_PLACE };

template <SortStep STEP>
__global__ void __launch_bounds__(SORT_THREADS) sort_kernel(const SortParams p) {
    __shared__ uint32_t s_warp[SORT_WARPS][MAX_ROUTE_EXPERTS / 2];   // 16 bits each: a warp's slots of an expert, then those of the warps before it
    __shared__ int s_total[MAX_ROUTE_EXPERTS + 1];               // an expert's slots
    __shared__ int s_before[MAX_ROUTE_EXPERTS];                  // those of the chunks before this one
    __shared__ int s_base[MAX_ROUTE_EXPERTS];                    // the expert's first row
    __shared__ int s_sum[SORT_WARPS];

    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.experts, chunk = static_cast<int>(blockIdx.x);
    const int first = (chunk * SORT_WARPS + warp) * p.groups * 32 + lane;
    for (int i = threadIdx.x; i < (E + 1) / 2; i += SORT_THREADS) {
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) s_warp[w][i] = 0;
    }
    if (STEP == SORT_STEP_ALONE)
        for (int i = threadIdx.x; i <= E; i += SORT_THREADS) s_total[i] = 0;
    __syncthreads();

    // ---- counts (whole numbers: in any order)
    if (STEP == SORT_STEP_ALONE) {
        // a total in the lower 16 bits, what of it lies before this chunk in the upper ones
        const int start = chunk * SORT_THREADS;
#pragma unroll 4
        for (int slot = threadIdx.x; slot < p.slots; slot += SORT_THREADS) {
            const int e = slot_expert(p, slot);
            atomicAdd(&s_total[e], slot < start ? 0x10001 : 1);
            if (slot == first && e < E) atomicAdd(&s_warp[warp][e >> 1], 1u << (16 * (e & 1)));
        }
    } else {
#pragma unroll 4
        for (int g = 0; g < p.groups; ++g) {
            const int e = slot_expert(p, first + g * 32);
            if (e < E) atomicAdd(&s_warp[warp][e >> 1], 1u << (16 * (e & 1)));
        }
    }
    __syncthreads();
    if (STEP == SORT_STEP_ALONE) {
        for (int e = threadIdx.x; e < E; e += SORT_THREADS) {
            const int both = s_total[e];
            s_total[e] = both & 0xffff;
            s_before[e] = both >> 16;
        }
    }
    // ---- over the warps, two experts a thread
    for (int i = threadIdx.x; i < (E + 1) / 2; i += SORT_THREADS) {
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            const uint32_t c = s_warp[w][i];
            s_warp[w][i] = sum;
            sum += c;
        }
        if (STEP == SORT_STEP_COUNT) {
            int32_t* dst = p.chunk_counts + 2 * i * p.chunks + chunk;
            dst[0] = static_cast<int>(sum & 0xffff);
            if (2 * i + 1 < E) dst[p.chunks] = static_cast<int>(sum >> 16);
        }
    }
    if (STEP == SORT_STEP_COUNT) return;

    if (STEP == SORT_STEP_PLACE) {
        for (int e = threadIdx.x; e < E; e += SORT_THREADS) {
            s_total[e] = __ldcg(p.totals + e);
            s_before[e] = __ldcg(p.chunk_counts + e * p.chunks + chunk);
        }
    }
    __syncthreads();

    // ---- the experts' first rows
    if (p.max_m > 0) {
        for (int e = threadIdx.x; e < E; e += SORT_THREADS) s_base[e] = e * p.max_m;
    } else {
        constexpr int PER = MAX_ROUTE_EXPERTS / SORT_THREADS;
        int room[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = static_cast<int>(threadIdx.x) * PER + i;
            room[i] = e < E ? (s_total[e] + 127) / 128 * 128 : 0;
            sum += room[i];
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
        int base = upto - sum;
        for (int w = 0; w < warp; ++w) base += s_sum[w];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = static_cast<int>(threadIdx.x) * PER + i;
            if (e < E) s_base[e] = base;
            base += room[i];
        }
    }
    __syncthreads();

    // ---- the slots' rows
    if (chunk < p.chunks) {
        for (int g = 0; g < p.groups; ++g) {
            const int slot = first + g * 32;
            const int e = slot_expert(p, slot);
            const unsigned same = same_lanes(e, p.bits), below = same & lanes_below();
            int row = -1;
            if (e < E) {
                const int place = s_before[e] + static_cast<int>(s_warp[warp][e >> 1] >> (16 * (e & 1)) & 0xffff) + __popc(below);
                if (p.max_m == 0 || place < p.max_m) row = s_base[e] + place;
            }
            if (p.groups > 1) {
                __syncwarp();
                if (e < E && below == 0) atomicAdd(&s_warp[warp][e >> 1], static_cast<uint32_t>(__popc(same)) << (16 * (e & 1)));
                __syncwarp();
            }
            if (slot < p.slots) p.rows[slot] = row;
        }
    }
    if (chunk == 0)
        for (int e = threadIdx.x; e < E; e += SORT_THREADS) p.counts[e] = s_total[e];

    // ---- the expert of every row: a block of 128 rows is one expert's, the last whose first row is not behind it
    if (p.m_indices != nullptr) {
        for (int b = chunk * SORT_WARPS + warp; b < p.blocks; b += static_cast<int>(gridDim.x) * SORT_WARPS) {
            int e = 0;
            for (int lo = 1, hi = E; lo < hi;) {
                const int mid = (lo + hi) >> 1;
                if (s_base[mid] <= b * 128) {
                    e = mid;
                    lo = mid + 1;
                } else {
                    hi = mid;
                }
            }
            const int left = s_total[e] - (b * 128 - s_base[e]) - lane * 4;   // rows from this lane's first on
            reinterpret_cast<int4*>(p.m_indices)[static_cast<size_t>(b) * 32 + lane] =
                make_int4(left > 0 ? e : -1, left > 1 ? e : -1, left > 2 ? e : -1, left > 3 ? e : -1);
        }
    }
}

// The chunks' counts of an expert added up, a warp an expert.
__global__ void __launch_bounds__(SORT_THREADS) sort_scan_kernel(int32_t* totals, int32_t* chunk_counts, int experts, int chunks) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, e = static_cast<int>(blockIdx.x) * SORT_WARPS + (threadIdx.x >> 5);
    if (e >= experts) return;
    constexpr int PER = SORT_CHUNKS / 32;
    int32_t* mine = chunk_counts + e * chunks + lane * PER;   // the lane's chunks are consecutive
    int n[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n[i] = lane * PER + i < chunks ? __ldcg(mine + i) : 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += n[i];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) totals[e] = upto;
    int before = upto - sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (lane * PER + i < chunks) mine[i] = before;
        before += n[i];
    }
}

// ------------------------------------------------------------------------------------ rows
constexpr int MOVE_WARPS = 8;                     // of a CTA of the weighted sum
constexpr int GATHER_WARPS = 2;                   // ... and of the gather, which the copies out of an SM limit where there are few

// Rows that a warp looks at for zeros, a power of two: fewer the longer they are. (With 8 for every length and 8 warps a CTA, 45
// tokens of 6528 codes to 5 of 6 experts took 11.5 us with their sort instead of 4.9, 8189 of 7168 to 8 of 256 115.6 instead of 105.2;
// with 2 for every length 8189 of 1024 took 38.8 instead of 24.2.)
int pad_rows(int64_t row_bytes) { return row_bytes <= 2048 ? 8 : row_bytes <= 4096 ? 4 : 2; }

__device__ __forceinline__ int slot_row(const int32_t* rows, size_t at, int Mt) {
    const int r = ld_input(rows + at);
    return static_cast<unsigned>(r) < static_cast<unsigned>(Mt) ? r : -1;
}

// The rows without a token of a block that has some, as bits, of the item's `rows`.
__device__ __forceinline__ unsigned pads_of(unsigned item, int rows, const int32_t* m_indices, int lane) {
    const unsigned first = item * rows;
    if (ld_input(m_indices + first / 128 * 128) < 0) return 0;
    return __ballot_sync(FULL, lane < rows && ld_input(m_indices + first + (lane & (rows - 1))) < 0);
}

struct GatherParams {
    const uint4* x;
    const float* sf;
    const int32_t* rows;
    const int32_t* m_indices;
    uint4* out;
    float* out_sf;
    int k, vectors, scales, Mt, pieces, pad_rows; // 16-byte vectors, scales and pieces of a row
    unsigned tokens_items, items;
};

// A warp has a piece of a token's row in shared memory, from where lane j has it copied to the row of slot j: the copies
// are what the kernel is about, and each is one instruction, whatever its length. What bounds it is memory, nearly all written:
// 8189 tokens of 7168 codes to 8 experts each, with the zeros, take 98 us without their sort (6.8 TB/s; a memset of the 702 MB that they lie in takes 173).
constexpr int GATHER_VECTORS = 256;               // a piece: 4096 bytes, with 32 scales of codes

__global__ void __launch_bounds__(32 * GATHER_WARPS) gather_kernel(const GatherParams p) {
    __shared__ __align__(128) uint4 s_piece[GATHER_WARPS][GATHER_VECTORS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned item = blockIdx.x * GATHER_WARPS + warp;
    if (item >= p.items) return;
    uint4* piece = s_piece[warp];
    if (item >= p.tokens_items) {
        const unsigned first = (item - p.tokens_items) * p.pad_rows, pads = pads_of(item - p.tokens_items, p.pad_rows, p.m_indices, lane);
        if (pads == 0) return;
#pragma unroll
        for (int i = 0; i < GATHER_VECTORS / 32; ++i) piece[i * 32 + lane] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        for (int i = lane; i < p.pad_rows * p.pieces; i += 32) {
            const int r = i & (p.pad_rows - 1), at = i / p.pad_rows * GATHER_VECTORS, left = p.vectors - at;
            if (pads >> r & 1) bulk_store(p.out + static_cast<size_t>(first + r) * p.vectors + at, piece, 16u * static_cast<uint32_t>(left < GATHER_VECTORS ? left : GATHER_VECTORS));
        }
        bulk_commit();
        if (p.out_sf != nullptr) {
            const float lowest = block_scale(0).s;
            for (unsigned which = pads; which; which &= which - 1)
                for (int b = lane; b < p.scales; b += 32) p.out_sf[static_cast<size_t>(first + __ffs(which) - 1) * p.scales + b] = lowest;
        }
        bulk_wait_read();
        return;
    }
    const unsigned t = item / p.pieces;
    const int at = static_cast<int>(item - t * p.pieces) * GATHER_VECTORS;
    const int here = p.vectors - at < GATHER_VECTORS ? p.vectors - at : GATHER_VECTORS;
    const int mine = lane < p.k ? slot_row(p.rows, static_cast<size_t>(t) * p.k + lane, p.Mt) : -1;
    const uint4* src = p.x + static_cast<size_t>(t) * p.vectors + at;
#pragma unroll
    for (int i = 0; i < GATHER_VECTORS / 32; ++i)
        if (i * 32 + lane < here) cp_async_16(piece + i * 32 + lane, src + i * 32 + lane);
    const int b = at / 8 + lane;                  // (a scale for each 8 vectors)
    const bool scaled = p.sf != nullptr && b < p.scales;
    const float s = scaled ? ld_input(p.sf + static_cast<size_t>(t) * p.scales + b) : 0.f;
    const unsigned open = __ballot_sync(FULL, mine >= 0);
    cp_async_wait_all();
    fence_proxy_async_smem();
    __syncwarp();
    if (mine >= 0) bulk_store(p.out + static_cast<size_t>(mine) * p.vectors + at, piece, 16u * static_cast<uint32_t>(here));
    bulk_commit();
    if (p.sf != nullptr)
        for (unsigned left = open; left; left &= left - 1) {
            const size_t row = static_cast<size_t>(__shfl_sync(FULL, mine, __ffs(left) - 1));
            if (scaled) p.out_sf[row * p.scales + b] = s;
        }
    bulk_wait_read();
}

// ------------------------------------------------------------------------------------ weighted sum
struct CombineParams {
    const uint4* y;
    const int32_t* rows;
    const float* weights;
    const uint4* residual;
    uint4* out;
    int k, vectors, Mt, pieces;
    unsigned items;
};

__device__ __forceinline__ void add_scaled(float2 (&a)[4], const uint4& v, float w) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __ffma2_rn(make_float2(w, w), make_float2(bf16_lo(u[i]), bf16_hi(u[i])), a[i]);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint4 pack_bf16(const float2 (&a)[4]) {
    return make_uint4(pack_bf16(a[0].x, a[0].y), pack_bf16(a[1].x, a[1].y), pack_bf16(a[2].x, a[2].y), pack_bf16(a[3].x, a[3].y));
}

// A warp a piece of 1024 bytes of a token's row, two experts' rows in flight at a time. FP32 sums, in the slots' order from
// zero on, the residual last. What bounds it is memory: 4099 tokens of 7168, a quarter of 8 slots each, 39.1 us (6.0 TB/s), all
// slots 86.8 us (6.8). Pieces of 512 bytes with 2 or 4 rows take 42.2 and 50.3 us, 1024 with 4 rows 42.3, 2048 with 2 42.7: the
// registers of more loads cost more warps than the loads bring.
constexpr int COMBINE_VECTORS = 2, COMBINE_ROWS = 2;

__global__ void __launch_bounds__(32 * MOVE_WARPS) combine_kernel(const CombineParams p) {
    constexpr int VECTORS = COMBINE_VECTORS, BATCH = COMBINE_ROWS;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const unsigned item = blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    if (item >= p.items) return;
    const unsigned t = item / p.pieces, piece = item - t * p.pieces;
    const size_t slot = static_cast<size_t>(t) * p.k + lane;
    const int mine = lane < p.k ? slot_row(p.rows, slot, p.Mt) : -1;
    const float weight = lane < p.k && p.weights != nullptr ? ld_input(p.weights + slot) : 1.f;
    unsigned open = __ballot_sync(FULL, mine >= 0);
    const int v = static_cast<int>(piece) * 32 * VECTORS + lane;
    const size_t at = static_cast<size_t>(t) * p.vectors + v;
    uint4 res[VECTORS];
    float2 a[VECTORS][4];
#pragma unroll
    for (int u = 0; u < VECTORS; ++u) {
        res[u] = make_uint4(0, 0, 0, 0);
        if (p.residual != nullptr && v + 32 * u < p.vectors) res[u] = ld_input(p.residual + at + 32 * u);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[u][i] = make_float2(0.f, 0.f);
    }
    for (; open != 0;) {
        uint4 y[BATCH][VECTORS];
        float w[BATCH];
        const int n = __popc(open);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int j = i < n ? __ffs(open) - 1 : 0;
            open &= open - 1;
            const int row = __shfl_sync(FULL, mine, j);
            w[i] = __shfl_sync(FULL, weight, j);
#pragma unroll
            for (int u = 0; u < VECTORS; ++u)
                if (i < n && v + 32 * u < p.vectors) y[i][u] = ld_input(p.y + static_cast<size_t>(row) * p.vectors + v + 32 * u);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
#pragma unroll
            for (int u = 0; u < VECTORS; ++u)
                if (i < n && v + 32 * u < p.vectors) add_scaled(a[u], y[i][u], w[i]);
    }
#pragma unroll
    for (int u = 0; u < VECTORS; ++u) {
        if (v + 32 * u >= p.vectors) break;
        if (p.residual != nullptr) add_scaled(a[u], res[u], 1.f);
        p.out[at + 32 * u] = pack_bf16(a[u]);
    }
}

// ------------------------------------------------------------------------------------ its gradient
struct CombineBackwardParams {
    const uint4* dout;
    const uint4* y;
    const int32_t* rows;
    const float* weights;
    const int32_t* m_indices;
    uint4* dy;
    float* dweights;
    int T, k, vectors, Mt, pad_rows;
    unsigned token_ctas, pads;
};

constexpr int CB_NARROW = 4;                      // tokens of a CTA, a warp each
constexpr int CB_WARPS = 8;                       // warps of a token at most
constexpr int CB_VECTORS = 4;                     // a lane's vectors at a time

// WIDE: a CTA a token; else a warp a token. A lane keeps its piece of dout while it goes through the token's experts; the
// products with their rows are added up over the lanes, and over the warps in order. What bounds it is memory, half of it
// written: 4096 tokens of 8 x 7168 take 164 us, 6.4 TB/s.
template <bool WIDE>
__global__ void __launch_bounds__(32 * (WIDE ? CB_WARPS : CB_NARROW)) combine_backward_kernel(const CombineBackwardParams p) {
    __shared__ float s_dot[CB_WARPS][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x / 32;
    if (blockIdx.x >= p.token_ctas) {
        const unsigned item = (blockIdx.x - p.token_ctas) * warps + warp;
        if (item >= p.pads) return;
        for (unsigned which = pads_of(item, p.pad_rows, p.m_indices, lane); which; which &= which - 1) {
            uint4* row = p.dy + (static_cast<size_t>(item) * p.pad_rows + __ffs(which) - 1) * p.vectors;
            for (int v = lane; v < p.vectors; v += 32) row[v] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const int t = static_cast<int>(WIDE ? blockIdx.x : blockIdx.x * CB_NARROW + warp);
    if (!WIDE && t >= p.T) return;
    const size_t slot = static_cast<size_t>(t) * p.k + lane;
    const int mine = lane < p.k ? slot_row(p.rows, slot, p.Mt) : -1;
    const float weight = lane < p.k && p.weights != nullptr ? ld_input(p.weights + slot) : 1.f;
    const unsigned open = __ballot_sync(FULL, mine >= 0);
    const int first = WIDE ? warp * 32 + lane : lane, step = WIDE ? static_cast<int>(blockDim.x) : 32;
    float dot = 0.f;                              // of slot `lane`
    for (int v0 = first; v0 - lane < p.vectors; v0 += step * CB_VECTORS) {
        uint4 d[CB_VECTORS];
#pragma unroll
        for (int i = 0; i < CB_VECTORS; ++i) {
            d[i] = make_uint4(0, 0, 0, 0);
            if (v0 + i * step < p.vectors) d[i] = ld_input(p.dout + static_cast<size_t>(t) * p.vectors + v0 + i * step);
        }
        for (unsigned left = open; left; left &= left - 1) {
            const int j = __ffs(left) - 1;
            const size_t at = static_cast<size_t>(__shfl_sync(FULL, mine, j)) * p.vectors + v0;
            uint4 y[CB_VECTORS];
#pragma unroll
            for (int i = 0; i < CB_VECTORS; ++i) {
                y[i] = make_uint4(0, 0, 0, 0);
                if (p.dweights != nullptr && v0 + i * step < p.vectors) y[i] = ld_input(p.y + at + i * step);
            }
            if (p.dy != nullptr) {
                const float w = __shfl_sync(FULL, weight, j);
#pragma unroll
                for (int i = 0; i < CB_VECTORS; ++i) {
                    if (v0 + i * step < p.vectors) {
                        const uint32_t dw[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
                        uint32_t o[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float2 v = __fmul2_rn(make_float2(w, w), make_float2(bf16_lo(dw[c]), bf16_hi(dw[c])));
                            o[c] = pack_bf16(v.x, v.y);
                        }
                        p.dy[at + i * step] = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            if (p.dweights != nullptr) {
                float2 a = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < CB_VECTORS; ++i) {
                    const uint32_t yw[4] = {y[i].x, y[i].y, y[i].z, y[i].w}, dw[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        a = __ffma2_rn(make_float2(bf16_lo(yw[c]), bf16_hi(yw[c])), make_float2(bf16_lo(dw[c]), bf16_hi(dw[c])), a);
                }
                float sum = a.x + a.y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
                if (lane == j) dot += sum;
            }
        }
    }
    if (p.dweights == nullptr) return;
    if (!WIDE) {
        if (lane < p.k) p.dweights[slot] = dot;
        return;
    }
    s_dot[warp][lane] = dot;
    __syncthreads();
    if (warp == 0 && lane < p.k) {
        float sum = s_dot[0][lane];
        for (int w = 1; w < warps; ++w) sum += s_dot[w][lane];
        p.dweights[slot] = sum;
    }
}

// Chunks of the slots and groups of 32 a warp; several launches' worth of chunks have their counts in the workspace.
void sort_plan(int64_t slots, int* groups, int* chunks) {
    *groups = 1;
    if (slots > SORT_ALONE) *groups = cdiv(slots, static_cast<int64_t>(SORT_THREADS) * SORT_CHUNKS);
    *chunks = cdiv(slots, static_cast<int64_t>(SORT_THREADS) * *groups);
}

dg_status sort_check(const int32_t* ids, int32_t* rows, int32_t* counts, int T, int k, int E) {
    if (T < 0 || k < 0 || E < 1) return DG_INVALID_ARG;
    if (k > MAX_ROUTE_K || E > MAX_ROUTE_EXPERTS || static_cast<int64_t>(T) * k > SORT_MAX_SLOTS) return DG_UNSUPPORTED_SHAPE;
    if (!counts || (static_cast<int64_t>(T) * k > 0 && (!ids || !rows))) return DG_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(rows, 4) || !aligned(counts, 4)) return DG_MISALIGNED;
    return DG_OK;
}

dg_status sort(const int32_t* ids, int32_t* rows, int32_t* counts, int32_t* m_indices, void* workspace, int64_t workspace_bytes, int T, int k,
               int E, int Mt, int max_m, cudaStream_t stream) {
    const int64_t need = dg_moe_sort_workspace(T, k, E);
    if (need > 0 && (!workspace || workspace_bytes < need)) return DG_INVALID_ARG;
    if (!aligned(workspace, 16)) return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status st = device_info(&dev);
    if (st != DG_OK) return st;
    SortParams p;
    p.ids = ids;
    p.rows = rows;
    p.counts = counts;
    p.m_indices = Mt > 0 ? m_indices : nullptr;
    p.totals = static_cast<int32_t*>(workspace);
    p.chunk_counts = need > 0 ? p.totals + E : nullptr;
    p.slots = T * k;
    p.experts = E;
    p.blocks = Mt / 128;
    p.max_m = max_m;
    sort_plan(p.slots, &p.groups, &p.chunks);
    for (p.bits = 0; E >> p.bits != 0;) ++p.bits;         // of 0 .. E
    cudaError_t e = cudaSuccess;
    const dim3 block(SORT_THREADS);
    if (p.slots <= SORT_ALONE) {
        // (CTAs without slots help to write m_indices, four blocks of rows a warp)
        const int most = p.m_indices != nullptr ? cdiv(p.blocks, 4 * SORT_WARPS) : 1;
        const int ctas = p.chunks > most ? p.chunks : most < SORT_CHUNKS ? most : SORT_CHUNKS;
        e = launch_overlapped(sort_kernel<SORT_STEP_ALONE>, dim3(static_cast<unsigned>(ctas)), block, stream, p);
    } else {
        const dim3 grid(static_cast<unsigned>(p.chunks));
        e = launch_overlapped(sort_kernel<SORT_STEP_COUNT>, grid, block, stream, p);
        if (e == cudaSuccess)
            e = launch_overlapped(sort_scan_kernel, dim3(static_cast<unsigned>(cdiv(E, SORT_WARPS))), block, stream, p.totals, p.chunk_counts, E, p.chunks);
        if (e == cudaSuccess) e = launch_overlapped(sort_kernel<SORT_STEP_PLACE>, grid, block, stream, p);
    }
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

// Common checks of the calls that move rows: sizes, and that 32 bits number the warps' pieces, a few past the last too.
dg_status rows_check(const int32_t* rows, int T, int k, int H, int Mt, int granule) {
    if (T < 0 || k < 0 || H < 0 || Mt < 0) return DG_INVALID_ARG;
    if (k > MAX_ROUTE_K || H % granule != 0) return DG_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(T) * (1 + H / 256) + Mt > INT32_MAX - 65536) return DG_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(T) * k > 0 && !rows) return DG_INVALID_ARG;
    return aligned(rows, 4) ? DG_OK : DG_MISALIGNED;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

int64_t dg_moe_sort_rows(int T, int k, int E) {
    if (T < 0 || k < 0 || E < 1 || k > MAX_ROUTE_K || E > MAX_ROUTE_EXPERTS) return -1;
    const int64_t slots = static_cast<int64_t>(T) * k;
    if (slots > SORT_MAX_SLOTS) return -1;
    return (slots + 127 * (slots < E ? slots : E)) / 128 * 128;
}

int64_t dg_moe_sort_workspace(int T, int k, int E) {
    if (T < 0 || k < 0 || E < 1 || k > MAX_ROUTE_K || E > MAX_ROUTE_EXPERTS) return -1;
    const int64_t slots = static_cast<int64_t>(T) * k;
    if (slots > SORT_MAX_SLOTS) return -1;
    if (slots <= SORT_ALONE) return 0;
    // (the most chunks that any number of slots up to this has: a workspace is for smaller calls too)
    const int64_t chunks = cdiv(slots, SORT_THREADS) < SORT_CHUNKS ? cdiv(slots, SORT_THREADS) : SORT_CHUNKS;
    return (chunks + 1) * E * 4;
}

dg_status dg_moe_sort_contiguous(const int32_t* ids, int32_t* rows, int32_t* counts, int32_t* m_indices, void* workspace,
                                 int64_t workspace_bytes, int T, int k, int E, int Mt, cudaStream_t stream) {
    const dg_status st = sort_check(ids, rows, counts, T, k, E);
    if (st != DG_OK) return st;
    if (Mt < 0) return DG_INVALID_ARG;
    if (Mt % 128 != 0 || Mt < dg_moe_sort_rows(T, k, E)) return DG_UNSUPPORTED_SHAPE;
    if (Mt > 0 && !m_indices) return DG_INVALID_ARG;
    if (!aligned(m_indices, 16)) return DG_MISALIGNED;
    return sort(ids, rows, counts, m_indices, workspace, workspace_bytes, T, k, E, Mt, 0, stream);
}

dg_status dg_moe_sort_masked(const int32_t* ids, int32_t* rows, int32_t* masked_m, void* workspace, int64_t workspace_bytes, int T,
                             int k, int E, int max_m, cudaStream_t stream) {
    const dg_status st = sort_check(ids, rows, masked_m, T, k, E);
    if (st != DG_OK) return st;
    if (max_m < 1) return DG_INVALID_ARG;
    if (static_cast<int64_t>(E) * max_m > INT32_MAX) return DG_UNSUPPORTED_SHAPE;
    return sort(ids, rows, masked_m, nullptr, workspace, workspace_bytes, T, k, E, 0, max_m, stream);
}

dg_status dg_moe_gather(const void* x, const float* sf, int x_type, const int32_t* rows, const int32_t* m_indices, void* out, float* out_sf,
                        int T, int k, int H, int Mt, cudaStream_t stream) {
    if (x_type != DG_TYPE_E4M3 && x_type != DG_TYPE_BF16) return DG_INVALID_ARG;
    const bool codes = x_type == DG_TYPE_E4M3;
    const dg_status st = rows_check(rows, T, k, H, Mt, codes ? 128 : 8);
    if (st != DG_OK) return st;
    if (m_indices && Mt % 128 != 0) return DG_UNSUPPORTED_SHAPE;
    if (H == 0 || Mt == 0 || (static_cast<int64_t>(T) * k == 0 && !m_indices)) return DG_OK;
    if (!out || (T > 0 && k > 0 && !x)) return DG_INVALID_ARG;
    if (codes ? (!out_sf || (T > 0 && k > 0 && !sf)) : (sf || out_sf)) return DG_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(sf, 4) || !aligned(out_sf, 4) || !aligned(m_indices, 4)) return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status ds = device_info(&dev);
    if (ds != DG_OK) return ds;
    GatherParams p;
    p.x = static_cast<const uint4*>(x);
    p.sf = sf;
    p.rows = rows;
    p.m_indices = m_indices;
    p.out = static_cast<uint4*>(out);
    p.out_sf = out_sf;
    p.k = k;
    p.vectors = codes ? H / 16 : H / 8;
    p.scales = codes ? H / 128 : 0;
    p.Mt = Mt;
    p.pieces = cdiv(p.vectors, GATHER_VECTORS);
    p.tokens_items = k > 0 ? static_cast<unsigned>(T) * static_cast<unsigned>(p.pieces) : 0u;
    p.pad_rows = pad_rows(16 * static_cast<int64_t>(p.vectors));
    p.items = p.tokens_items + (m_indices ? static_cast<unsigned>(Mt / p.pad_rows) : 0u);
    const cudaError_t e = launch_overlapped(gather_kernel, dim3((p.items + GATHER_WARPS - 1) / GATHER_WARPS), dim3(32 * GATHER_WARPS), stream, p);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

dg_status dg_moe_combine(const void* y, const int32_t* rows, const float* weights, const void* residual, void* out, int T, int k, int H,
                         int Mt, cudaStream_t stream) {
    const dg_status st = rows_check(rows, T, k, H, Mt, 8);
    if (st != DG_OK) return st;
    if (T == 0 || H == 0) return DG_OK;
    if (!out || (k > 0 && Mt > 0 && !y)) return DG_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(weights, 4)) return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status ds = device_info(&dev);
    if (ds != DG_OK) return ds;
    CombineParams p;
    p.y = static_cast<const uint4*>(y);
    p.rows = rows;
    p.weights = weights;
    p.residual = static_cast<const uint4*>(residual);
    p.out = static_cast<uint4*>(out);
    p.k = k;
    p.vectors = H / 8;
    p.Mt = Mt;
    p.pieces = cdiv(p.vectors, 32 * COMBINE_VECTORS);
    p.items = static_cast<unsigned>(T) * static_cast<unsigned>(p.pieces);
    const cudaError_t e = launch_overlapped(combine_kernel, dim3((p.items + MOVE_WARPS - 1) / MOVE_WARPS), dim3(32 * MOVE_WARPS), stream, p);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

dg_status dg_moe_combine_backward(const void* dout, const void* y, const int32_t* rows, const float* weights, const int32_t* m_indices, void* dy,
                                  float* dweights, int T, int k, int H, int Mt, cudaStream_t stream) {
    const dg_status st = rows_check(rows, T, k, H, Mt, 8);
    if (st != DG_OK) return st;
    if (m_indices && Mt % 128 != 0) return DG_UNSUPPORTED_SHAPE;
    if (!dy && !dweights) return DG_OK;
    const bool slots = T > 0 && k > 0, pads = dy && m_indices && Mt > 0 && H > 0;
    if (!slots && !pads) return DG_OK;
    if (slots && H > 0 && (!dout || (dweights && Mt > 0 && !y))) return DG_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(dweights, 4) || !aligned(weights, 4) || !aligned(m_indices, 4))
        return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status ds = device_info(&dev);
    if (ds != DG_OK) return ds;
    CombineBackwardParams p;
    p.dout = static_cast<const uint4*>(dout);
    p.y = static_cast<const uint4*>(y);
    p.rows = rows;
    p.weights = weights;
    p.m_indices = m_indices;
    p.dy = static_cast<uint4*>(dy);
    p.dweights = dweights;
    p.T = T;
    p.k = k;
    p.vectors = H / 8;
    p.Mt = Mt;
    // Few tokens get as many warps each as they have pieces for, up to eight, many get four. Rows of 7168, us with 8, 4 and 2 warps:
    //   tokens of 8    16: 19.1, 26.3, 38.0    256: 27.6, 32.0, 43.2    1024: 53.6, 57.9, 56.2    1536: 72.5, 70.1, 73.8    2048: 92.6, 92.7, 103.2
    //                  4096: 170.5, 163.9, 171.4    8192: 324.4, 312.4, 313.8
    //   tokens of 2    16: 11.2, 11.3, 14.6    256: 21.4, 21.3, 24.1    1024: 30.8, 28.8, 29.6    2048: 42.3, 38.1, 40.5
    //                  4096: 66.1, 60.4, 60.5    8192: 114.8, 106.2, 102.2
    // (Four would be best from somewhere between 1024 and 1536 tokens of 8 on, and from 256 of 2; with rows of 2048 all take the
    // same.) By the sizes alone, and so is the order of the sums.
    const bool wide = H > 32 * CB_VECTORS * 8;
    const int most = T < 2048 ? CB_WARPS : 4, pieces = cdiv(p.vectors, 32 * CB_VECTORS);
    const int warps = !wide ? CB_NARROW : pieces < most ? pieces : most;
    p.token_ctas = !slots ? 0u : (wide ? static_cast<unsigned>(T) : static_cast<unsigned>(cdiv(T, CB_NARROW)));
    p.pad_rows = pad_rows(16 * static_cast<int64_t>(p.vectors));
    p.pads = pads ? static_cast<unsigned>(Mt / p.pad_rows) : 0u;
    const dim3 grid(p.token_ctas + static_cast<unsigned>(cdiv(p.pads, warps))), block(32u * static_cast<unsigned>(warps));
    const cudaError_t e = launch_overlapped(wide ? combine_backward_kernel<true> : combine_backward_kernel<false>, grid, block, stream, p);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

}  // extern "C"
