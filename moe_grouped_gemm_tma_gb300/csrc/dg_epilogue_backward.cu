// Backward pass of the product with an epilogue (dg_epilogue_backward): from dD and the kept pre-activation
// Z, the gradient dZ = dD * act'(Z) in the three forms that the rest of the backward pass reads -- e4m3
// codes with 1x128 scales along N (the A operand of dX = dZ . B), codes of the transpose with 1x128 scales
// along M (the B operand of the weight gradient), and the bias gradient, the sum of dZ's rows in FP32.
//
// One pass: a CTA owns a 128 x 128 tile, which is one scaling block in either direction, so dZ is computed
// once, stays in registers, and is quantised twice. A thread holds 4 x 8 values (4 consecutive rows x 8
// consecutive columns): a half warp reads 256 contiguous bytes of a row, a row's largest magnitude is found
// over 16 lanes by shuffles, a column's over the tile's 16 warps through shared memory. The transposed codes
// go through 16 KB of shared memory, four rows of one column in a word, words XOR-ed by the column group so
// that neither side conflicts, and leave as 128-byte rows.
//
// The bias gradient is summed in a fixed order whatever the timing: each tile writes its column sums, and these
// are added up, every fourth tile's in turn, then the four sums: by the CTA that finishes a column strip last, or,
// where there are more tiles than run at once, by a kernel of its own. Telling which CTA is last costs every
// tile a fence behind its stores: 44.3 us for 4096 x 7168 with silu and 37.3 without an activation, where the
// second launch gives 42.0 and 31.1; at 333 x 2048 it gives 5.4 for 5.8 us, less than the launch costs the host.
//
// Floor: 4 bytes read and 2 written per element (2 read without an activation), 26.6 us for 4096 x 7168 at the
// measured copy bandwidth. It takes 39.3 us: 67% of the issue slots, loads whose latency two CTAs an SM hide only
// in part, and two barriers a tile, because the two scalings need the whole tile's maxima between the loads and the
// stores. (A persistent form with the next tile's operands in shared memory by TMA was 7 us slower; without the exact
// divisions of the codes it would be 1 us faster.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg.h"
#include "dg_host.cuh"
#include "dg_ptx.cuh"
#include "dg_quant.cuh"

namespace dg {
namespace {

constexpr int EB_THREADS = 512;
constexpr int EB_WARPS = EB_THREADS / 32;
constexpr int EB_TILE = 128;

struct EbParams {
    const __nv_bfloat16* dd;
    const __nv_bfloat16* z;
    uint8_t* q;
    float* sf;
    uint8_t* qt;
    float* sft;
    float* dbias;
    float* sums;          // [m_tiles][N] column sums of each tile
    unsigned* done;       // [N / 128] tiles of a strip that have written theirs; null: a second kernel adds them up
    int m, n, m_tiles;
    int ahead;            // tiles between a CTA's own and the one that it asks L2 for; 0: none
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// (STRIPS: the last CTA of a strip adds its tiles' sums)
template <int ACT, bool STRIPS>
__global__ void __launch_bounds__(EB_THREADS, 2) epilogue_backward_kernel(const EbParams p) {
    __shared__ __align__(16) uint32_t s_codes[EB_TILE * EB_TILE / 4];
    __shared__ __align__(16) float s_amax[EB_WARPS][EB_TILE];
    __shared__ __align__(16) float s_sum[EB_WARPS][EB_TILE];
    __shared__ __align__(16) float s_divisor[EB_TILE], s_reciprocal[EB_TILE];   // (divisors negative)
    __shared__ int s_last;

    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = lane >> 4, l16 = lane & 15;
    const int m0 = static_cast<int>(blockIdx.x) * EB_TILE, n0 = static_cast<int>(blockIdx.y) * EB_TILE;
    const int r0 = warp * 8 + half * 4;                // first of this thread's 4 rows of the tile
    const int c0 = l16 * 8;                            // first of its 8 columns
    const size_t base = static_cast<size_t>(m0 + r0) * p.n + n0 + c0;
    const int valid = p.m - (m0 + r0);                 // rows of the thread's 4 that exist (may be <= 0)

    float2 dz[4][4];                                   // [row][pair of columns]
    {
        uint4 d[4], z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] = make_uint4(0, 0, 0, 0);
            z[i] = make_uint4(0, 0, 0, 0);
            if (i < valid) {
                d[i] = ld_input(reinterpret_cast<const uint4*>(p.dd + base + static_cast<size_t>(i) * p.n));
                if (ACT != DG_ACT_NONE) z[i] = ld_input(reinterpret_cast<const uint4*>(p.z + base + static_cast<size_t>(i) * p.n));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t dw[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
            const uint32_t zw[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dz[i][j] = make_float2(bf16_lo(dw[j]), bf16_hi(dw[j]));
                // (rows past M stay zero: every slope at 0 is finite)
                if (ACT != DG_ACT_NONE) dz[i][j] = __fmul2_rn(dz[i][j], act_slope2<ACT>(make_float2(bf16_lo(zw[j]), bf16_hi(zw[j]))));
            }
        }
    }

    // ---- the tile that is `ahead` further on, into L2: a CTA's loads are what it waits for most. (Not for GELU, which
    // it made slower, 45.7 against 47.4 us at 4096 x 7168: its arithmetic needs the registers.)
    if (!STRIPS && ACT != DG_ACT_GELU && p.ahead > 0 && (l16 & 7) == 0) {
        const unsigned tile = blockIdx.y * gridDim.x + blockIdx.x + static_cast<unsigned>(p.ahead);
        const unsigned ny = tile / gridDim.x, nx = tile - ny * gridDim.x;
        if (ny < gridDim.y) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = static_cast<int>(nx) * EB_TILE + r0 + i;
                if (row < p.m) {
                    const size_t at = static_cast<size_t>(row) * p.n + ny * EB_TILE + c0;
                    prefetch_l2(p.dd + at);
                    if (ACT != DG_ACT_NONE) prefetch_l2(p.z + at);
                }
            }
        }
    }

    // ---- the columns' largest magnitudes and sums over this warp's rows, to shared memory
    if (p.qt != nullptr) {
        float a[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[2 * j] = abs_max(dz[0][j].x, dz[1][j].x, dz[2][j].x);
            a[2 * j + 1] = abs_max(dz[0][j].y, dz[1][j].y, dz[2][j].y);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = abs_max(a[j], j & 1 ? dz[3][j >> 1].y : dz[3][j >> 1].x);
            a[j] = abs_max(a[j], __shfl_xor_sync(0xffffffffu, a[j], 16));
        }
        if (half == 0) {
            float4* dst = reinterpret_cast<float4*>(&s_amax[warp][c0]);
            dst[0] = make_float4(a[0], a[1], a[2], a[3]);
            dst[1] = make_float4(a[4], a[5], a[6], a[7]);
        }
    }
    if (p.dbias != nullptr) {
        float2 a[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = __fadd2_rn(__fadd2_rn(dz[0][j], dz[1][j]), __fadd2_rn(dz[2][j], dz[3][j]));
            a[j].x += __shfl_xor_sync(0xffffffffu, a[j].x, 16);
            a[j].y += __shfl_xor_sync(0xffffffffu, a[j].y, 16);
        }
        if (half == 0) {
            float4* dst = reinterpret_cast<float4*>(&s_sum[warp][c0]);
            dst[0] = make_float4(a[0].x, a[0].y, a[1].x, a[1].y);
            dst[1] = make_float4(a[2].x, a[2].y, a[3].x, a[3].y);
        }
    }
    // ---- codes along the rows
    if (p.q != nullptr) {
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a[i] = abs_max(abs_max(dz[i][0].x, dz[i][0].y, dz[i][1].x), abs_max(dz[i][1].y, dz[i][2].x, dz[i][2].y), abs_max(dz[i][3].x, dz[i][3].y));
        // over the 16 lanes, giving away rows on the way: lane l ends with that of row l / 4, and makes its scale
        const bool up8 = (l16 & 8) != 0, up4 = (l16 & 4) != 0;
        const float b0 = abs_max(up8 ? a[2] : a[0], __shfl_xor_sync(0xffffffffu, up8 ? a[0] : a[2], 8));
        const float b1 = abs_max(up8 ? a[3] : a[1], __shfl_xor_sync(0xffffffffu, up8 ? a[1] : a[3], 8));
        float most = abs_max(up4 ? b1 : b0, __shfl_xor_sync(0xffffffffu, up4 ? b0 : b1, 4));
        most = abs_max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        most = abs_max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        const BlockScale mine = block_scale(abs_bits(most));
        if ((l16 & 3) == 0 && (l16 >> 2) < valid) p.sf[static_cast<size_t>(m0 + r0 + (l16 >> 2)) * (p.n / 128) + blockIdx.y] = mine.s;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            BlockScale k;
            k.d = __shfl_sync(0xffffffffu, mine.d, i * 4, 16);
            k.r = __shfl_sync(0xffffffffu, mine.r, i * 4, 16);
            const uint32_t w0 = quantise4(dz[i][0], dz[i][1], k), w1 = quantise4(dz[i][2], dz[i][3], k);
            if (i < valid) *reinterpret_cast<uint2*>(p.q + base + static_cast<size_t>(i) * p.n) = make_uint2(w0, w1);
        }
    }
    if (p.qt == nullptr && p.dbias == nullptr) return;
    __syncthreads();

    const int mt = p.m_tiles;                          // scale blocks along the transpose's rows
    if (threadIdx.x < EB_TILE) {
        if (p.qt != nullptr) {
            const int c = threadIdx.x;
            float a = 0.f;
#pragma unroll
            for (int g = 0; g < EB_WARPS; ++g) a = abs_max(a, s_amax[g][c]);
            const BlockScale k = block_scale(abs_bits(a));
            s_divisor[c] = -k.d;
            s_reciprocal[c] = k.r;
            p.sft[static_cast<size_t>(n0 + c) * mt + blockIdx.x] = k.s;
        }
    } else if (threadIdx.x < 2 * EB_TILE && p.dbias != nullptr) {
        const int c = threadIdx.x - EB_TILE;
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < EB_WARPS; ++w) a += s_sum[w][c];
        if (mt == 1) p.dbias[n0 + c] = a;              // the strip's only tile
        else __stcg(p.sums + static_cast<size_t>(blockIdx.x) * p.n + n0 + c, a);
    }
    __syncthreads();
    const bool strip = STRIPS && p.dbias != nullptr && mt > 1;
    if (strip && threadIdx.x == 0) {
        // (releases the sums, which the barrier has ordered before it, to the strip's last CTA)
        __threadfence();
        s_last = atomicAdd(p.done + blockIdx.y, 1u) == static_cast<unsigned>(mt - 1);
    }

    // ---- codes along the columns: rows 4w .. 4w + 3 of column n in word w ^ 2 (n / 8) of its 32
    if (p.qt != nullptr) {
        const int word = (warp * 2 + half) ^ (2 * l16);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const float4 d = *reinterpret_cast<const float4*>(&s_divisor[c0 + 2 * j]);
            const float4 r = *reinterpret_cast<const float4*>(&s_reciprocal[c0 + 2 * j]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 nd = x ? make_float2(d.z, d.w) : make_float2(d.x, d.y), rr = x ? make_float2(r.z, r.w) : make_float2(r.x, r.y);
                float2 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = quotient2(dz[i][j + x], nd, rr);
                uint32_t* dst = s_codes + (c0 + 2 * (j + x)) * 32 + word;
                dst[0] = pack_e4m3x2(v[0].x, v[1].x) | (pack_e4m3x2(v[2].x, v[3].x) << 16);
                dst[32] = pack_e4m3x2(v[0].y, v[1].y) | (pack_e4m3x2(v[2].y, v[3].y) << 16);
            }
        }
    }
    __syncthreads();
    if (p.qt != nullptr) {
        const size_t pitch = static_cast<size_t>(mt) * EB_TILE;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = i * 32 + warp * 2 + half;
            const uint2 w = *reinterpret_cast<const uint2*>(s_codes + c * 32 + 2 * (l16 ^ (c >> 3)));
            *reinterpret_cast<uint2*>(p.qt + static_cast<size_t>(n0 + c) * pitch + m0 + l16 * 8) = w;
        }
    }
    if (strip && s_last) {
        // every fourth tile's sums by each quarter of the threads, then the four in order
        __threadfence();
        const int c = threadIdx.x % EB_TILE, part = threadIdx.x / EB_TILE;
        constexpr int PARTS = EB_THREADS / EB_TILE;
        const float* src = p.sums + n0 + c;
        float a = 0.f;
#pragma unroll 8
        for (int i = part; i < mt; i += PARTS) a += __ldcg(src + static_cast<size_t>(i) * p.n);
        s_sum[part][c] = a;
        __syncthreads();
        if (threadIdx.x < EB_TILE) p.dbias[n0 + c] = (s_sum[0][c] + s_sum[1][c]) + (s_sum[2][c] + s_sum[3][c]);
        if (threadIdx.x == 0) p.done[blockIdx.y] = 0;  // the workspace is as the next call expects it
    }
}

// The bias gradient from the tiles' column sums: 32 columns a CTA, every fourth tile a warp.
__global__ void __launch_bounds__(128) add_strips_kernel(const float* sums, float* dbias, int n, int m_tiles) {
    __shared__ float s_part[4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const float* src = sums + static_cast<int>(blockIdx.x) * 32 + lane;
    float a = 0.f;
#pragma unroll 8
    for (int i = warp; i < m_tiles; i += 4) a += __ldcg(src + static_cast<size_t>(i) * n);
    s_part[warp][lane] = a;
    __syncthreads();
    if (warp == 0) dbias[static_cast<int>(blockIdx.x) * 32 + lane] = (s_part[0][lane] + s_part[1][lane]) + (s_part[2][lane] + s_part[3][lane]);
}

template <int ACT>
cudaError_t launch_eb(const EbParams& p, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.m_tiles), static_cast<unsigned>(p.n / EB_TILE));
    const cudaError_t e = p.done != nullptr ? launch_overlapped(epilogue_backward_kernel<ACT, true>, grid, dim3(EB_THREADS), stream, p)
                                            : launch_overlapped(epilogue_backward_kernel<ACT, false>, grid, dim3(EB_THREADS), stream, p);
    if (e != cudaSuccess || p.dbias == nullptr || p.m_tiles == 1 || p.done != nullptr) return e;
    return launch_overlapped(add_strips_kernel, dim3(static_cast<unsigned>(p.n / 32)), dim3(128), stream, static_cast<const float*>(p.sums), p.dbias, p.n, p.m_tiles);
}

// The workspace: the strips' counters, in the same place whatever the size (no size's sums may lie where another's
// counters do), then the column sums.
constexpr int EB_STRIPS = 256;
constexpr int64_t EB_DONE_BYTES = 4 * EB_STRIPS;
static_assert(EB_DONE_BYTES == DG_EPILOGUE_BACKWARD_ZEROED, "the sums need no zeros");

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

int64_t dg_epilogue_backward_workspace(int M, int N) {
    if (M <= 0 || N <= 0) return 0;
    return EB_DONE_BYTES + static_cast<int64_t>(cdiv(M, EB_TILE)) * N * 4;
}

dg_status dg_epilogue_backward(const void* dD, const void* Z, int act, uint8_t* q, float* sf, uint8_t* qt, float* sft,
                               float* dbias, void* workspace, int64_t workspace_bytes, int M, int N, cudaStream_t stream) {
    if (M < 0 || N < 0 || act < DG_ACT_NONE || act > DG_ACT_SILU) return DG_INVALID_ARG;
    if ((q == nullptr) != (sf == nullptr) || (qt == nullptr) != (sft == nullptr)) return DG_INVALID_ARG;
    if (N == 0 || (!q && !qt && !dbias)) return DG_OK;
    if (N % 128 != 0) return DG_UNSUPPORTED_SHAPE;
    if (cdiv(N, EB_TILE) > 65535 || M > INT32_MAX - EB_TILE) return DG_UNSUPPORTED_SHAPE;
    if (!aligned(dD, 16) || !aligned(Z, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(sf, 4) || !aligned(sft, 4) ||
        !aligned(dbias, 4) || !aligned(workspace, 16))
        return DG_MISALIGNED;
    if (M == 0) {
        if (!dbias) return DG_OK;
        DeviceInfo dev;
        const dg_status st = device_info(&dev);
        if (st != DG_OK) return st;
        return cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 4, stream) == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
    }
    if (!dD || (act != DG_ACT_NONE && !Z)) return DG_INVALID_ARG;
    if (dbias && (!workspace || workspace_bytes < dg_epilogue_backward_workspace(M, N))) return DG_INVALID_ARG;
    DeviceInfo dev;
    const dg_status st = device_info(&dev);
    if (st != DG_OK) return st;
    EbParams p;
    p.dd = static_cast<const __nv_bfloat16*>(dD);
    p.z = static_cast<const __nv_bfloat16*>(Z);
    p.q = q;
    p.sf = sf;
    p.qt = qt;
    p.sft = sft;
    p.dbias = dbias;
    p.sums = dbias ? reinterpret_cast<float*>(static_cast<char*>(workspace) + EB_DONE_BYTES) : nullptr;
    p.m = M;
    p.n = N;
    p.m_tiles = cdiv(M, EB_TILE);
    const int strips = N / EB_TILE;
    const bool one_round = static_cast<int64_t>(p.m_tiles) * strips <= 2 * dev.sms && strips <= EB_STRIPS;   // two CTAs fit an SM
    // one and a half tiles an SM ahead, from six on (4096 x 7168 with silu 39.8 -> 38.4 us, gelu_tanh 45.0 -> 44.4;
    // 4096 x 4096 24.0 -> 23.5; 4096 x 2048, 3.4 tiles an SM, 13.9 -> 14.4)
    p.ahead = static_cast<int64_t>(p.m_tiles) * strips >= 6 * dev.sms ? dev.sms * 3 / 2 : 0;
    p.done = one_round ? static_cast<unsigned*>(workspace) : nullptr;
    cudaError_t e = cudaErrorInvalidValue;
    switch (act) {
        case DG_ACT_NONE: e = launch_eb<DG_ACT_NONE>(p, stream); break;
        case DG_ACT_RELU: e = launch_eb<DG_ACT_RELU>(p, stream); break;
        case DG_ACT_GELU: e = launch_eb<DG_ACT_GELU>(p, stream); break;
        case DG_ACT_GELU_TANH: e = launch_eb<DG_ACT_GELU_TANH>(p, stream); break;
        case DG_ACT_SILU: e = launch_eb<DG_ACT_SILU>(p, stream); break;
    }
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

}  // extern "C"
