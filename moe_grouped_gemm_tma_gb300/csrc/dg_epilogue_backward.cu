// Backward pass of the product with an epilogue (dg_epilogue_backward): from dD and the kept pre-activation
// Z, the gradient dZ = dD * act'(Z) in the three forms that the rest of the backward pass reads -- e4m3
// codes with 1x128 scales along N (the A operand of dX = dZ . B), codes of the transpose with 1x128 scales
// along M (the B operand of the weight gradient), and the bias gradient, the sum of dZ's rows in FP32.
//
// One pass: a CTA owns a 128 x 128 tile, which is one scaling block in either direction, so dZ is computed
// once, stays in registers, and is quantised twice. A thread holds 8 x 8 values (8 consecutive rows x 8
// consecutive columns): a half warp reads 256 contiguous bytes of a row, a row's largest magnitude is found
// over 16 lanes by shuffles, a column's over the tile's 16 row groups through shared memory. The transposed
// codes go through 16 KB of shared memory, eight rows of one column in one 8-byte chunk, chunks XOR-ed by
// the column group so that neither side conflicts, and leave as 128-byte rows.
//
// The bias gradient is summed in a fixed order whatever the timing: each tile writes its column sums, and
// the CTA that finishes a column strip last adds the strip's tiles from the first to the last.
//
// Floor: 4 bytes read and 2 written per element (2 read without an activation).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg.h"
#include "dg_host.cuh"
#include "dg_quant.cuh"

namespace dg {
namespace {

constexpr int EB_THREADS = 256;
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
    unsigned* done;       // [N / 128] tiles of a strip that have written theirs
    int m, n, m_tiles;
    int act;
};

template <int ACT>
__global__ void __launch_bounds__(EB_THREADS, 2) epilogue_backward_kernel(const EbParams p) {
    __shared__ __align__(16) uint8_t s_codes[EB_TILE * EB_TILE];
    __shared__ __align__(16) uint32_t s_amax[16][EB_TILE];
    __shared__ __align__(16) float s_sum[8][EB_TILE];
    __shared__ float2 s_scale[EB_TILE];
    __shared__ int s_last;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = lane >> 4, l16 = lane & 15;
    const int m0 = static_cast<int>(blockIdx.x) * EB_TILE, n0 = static_cast<int>(blockIdx.y) * EB_TILE;
    const int r0 = warp * 16 + half * 8;               // first of this thread's 8 rows of the tile
    const int c0 = l16 * 8;                            // first of its 8 columns
    const size_t base = static_cast<size_t>(m0 + r0) * p.n + n0 + c0;
    const int valid = p.m - (m0 + r0);                 // rows of the thread's 8 that exist (may be <= 0)

    float dz[8][8];
    {
        uint4 d[8], z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            d[i] = make_uint4(0, 0, 0, 0);
            if (ACT != DG_ACT_NONE) z[i] = make_uint4(0, 0, 0, 0);
            if (i < valid) {
                d[i] = __ldcs(reinterpret_cast<const uint4*>(p.dd + base + static_cast<size_t>(i) * p.n));
                if (ACT != DG_ACT_NONE) z[i] = __ldcs(reinterpret_cast<const uint4*>(p.z + base + static_cast<size_t>(i) * p.n));
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t dw[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
            const uint32_t zw[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dz[i][2 * j] = bf16_lo(dw[j]);
                dz[i][2 * j + 1] = bf16_hi(dw[j]);
                if (ACT != DG_ACT_NONE) {
                    dz[i][2 * j] *= act_slope<ACT>(bf16_lo(zw[j]));
                    dz[i][2 * j + 1] *= act_slope<ACT>(bf16_hi(zw[j]));
                    // rows past M stay zero (0 * slope(0) is 0)
                }
            }
        }
    }

    // ---- the columns' largest magnitudes and sums over this thread's rows, to shared memory
    if (p.qt != nullptr) {
        uint32_t a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) a[j] = max(a[j], abs_bits(dz[i][j]));
        }
        uint4* dst = reinterpret_cast<uint4*>(&s_amax[warp * 2 + half][c0]);
        dst[0] = make_uint4(a[0], a[1], a[2], a[3]);
        dst[1] = make_uint4(a[4], a[5], a[6], a[7]);
    }
    if (p.dbias != nullptr) {
        float a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) a[j] += dz[i][j];
            a[j] += __shfl_xor_sync(0xffffffffu, a[j], 16);
        }
        if (half == 0) {
            float4* dst = reinterpret_cast<float4*>(&s_sum[warp][c0]);
            dst[0] = make_float4(a[0], a[1], a[2], a[3]);
            dst[1] = make_float4(a[4], a[5], a[6], a[7]);
        }
    }
    // ---- codes along the rows
    if (p.q != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t a = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) a = max(a, abs_bits(dz[i][j]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
            const BlockScale k = block_scale(a);
            if (i < valid) {
                const uint32_t w0 = quantise4(dz[i][0], dz[i][1], dz[i][2], dz[i][3], k);
                const uint32_t w1 = quantise4(dz[i][4], dz[i][5], dz[i][6], dz[i][7], k);
                *reinterpret_cast<uint2*>(p.q + base + static_cast<size_t>(i) * p.n) = make_uint2(w0, w1);
                if (l16 == 0) p.sf[static_cast<size_t>(m0 + r0 + i) * (p.n / 128) + blockIdx.y] = k.s;
            }
        }
    }
    if (p.qt == nullptr && p.dbias == nullptr) return;
    __syncthreads();

    const int mt = p.m_tiles;                          // scale blocks along the transpose's rows
    if (threadIdx.x < EB_TILE) {
        const int c = threadIdx.x;
        if (p.qt != nullptr) {
            uint32_t a = 0;
#pragma unroll
            for (int g = 0; g < 16; ++g) a = max(a, s_amax[g][c]);
            const BlockScale k = block_scale(a);
            s_scale[c] = make_float2(k.d, k.r);
            p.sft[static_cast<size_t>(n0 + c) * mt + blockIdx.x] = k.s;
        }
    } else if (p.dbias != nullptr) {
        const int c = threadIdx.x - EB_TILE;
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) a += s_sum[w][c];
        __stcg(p.sums + static_cast<size_t>(blockIdx.x) * p.n + n0 + c, a);
        __threadfence();                               // the strip's last CTA reads it
    }
    __syncthreads();
    if (p.dbias != nullptr && threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(p.done + blockIdx.y, 1u) == static_cast<unsigned>(mt - 1);
    }

    // ---- codes along the columns: chunk (m / 8) of column n at 8-byte slot (m / 8) ^ (n / 8)
    if (p.qt != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const BlockScale k{0.f, s_scale[c0 + j].x, s_scale[c0 + j].y};
            const uint32_t w0 = quantise4(dz[0][j], dz[1][j], dz[2][j], dz[3][j], k);
            const uint32_t w1 = quantise4(dz[4][j], dz[5][j], dz[6][j], dz[7][j], k);
            const int slot = (warp * 2 + half) ^ l16;
            *reinterpret_cast<uint2*>(s_codes + (c0 + j) * EB_TILE + slot * 8) = make_uint2(w0, w1);
        }
    }
    __syncthreads();
    if (p.qt != nullptr) {
        const size_t pitch = static_cast<size_t>(mt) * EB_TILE;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = i * 16 + warp * 2 + half;
            const uint2 w = *reinterpret_cast<const uint2*>(s_codes + c * EB_TILE + ((l16 ^ (c >> 3)) * 8));
            *reinterpret_cast<uint2*>(p.qt + static_cast<size_t>(n0 + c) * pitch + m0 + l16 * 8) = w;
        }
    }
    if (p.dbias != nullptr && s_last && threadIdx.x < EB_TILE) {
        __threadfence();
        const float* src = p.sums + n0 + threadIdx.x;
        float a = 0.f;
#pragma unroll 8
        for (int i = 0; i < mt; ++i) a += __ldcg(src + static_cast<size_t>(i) * p.n);
        p.dbias[n0 + threadIdx.x] = a;
        if (threadIdx.x == 0) p.done[blockIdx.y] = 0;  // the workspace is as the next call expects it
    }
}

template <int ACT>
cudaError_t launch_eb(const EbParams& p, cudaStream_t stream) {
    epilogue_backward_kernel<ACT><<<dim3(static_cast<unsigned>(p.m_tiles), static_cast<unsigned>(p.n / EB_TILE)), EB_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

// The counters come first, on their own 128-byte lines' worth of space, then the column sums.
int64_t done_bytes(int n) { return (static_cast<int64_t>(cdiv(n, EB_TILE)) * 4 + 255) / 256 * 256; }

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

int64_t dg_epilogue_backward_workspace(int M, int N) {
    if (M <= 0 || N <= 0) return 0;
    return done_bytes(N) + static_cast<int64_t>(cdiv(M, EB_TILE)) * N * 4;
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
    p.done = static_cast<unsigned*>(workspace);
    p.sums = dbias ? reinterpret_cast<float*>(static_cast<char*>(workspace) + done_bytes(N)) : nullptr;
    p.m = M;
    p.n = N;
    p.m_tiles = cdiv(M, EB_TILE);
    p.act = act;
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
