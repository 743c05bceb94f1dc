// The gated activation between two grouped products (dg_glu), its pre-activations kept in 8 bits on request, its backward
// pass from them (dg_glu_backward), and the values of 8-bit codes quantised along the other axis (dg_transpose_fp8), which
// makes the operand of a weight gradient from the codes that the forward product read.
//
//   h = act(g) u,  (q, sf) = Q(h),  (kept, kept_sf) = Q(g; u)
//   dg = dh u act'(g),  du = dh act(g): Q(dg; du) along rows and along columns, Q(h) along columns
//
// Forward: a half warp has the 128 values of a scaling block of 4 rows, 8 columns a lane, and both halves of Z's rows there.
// Backward and transposition: tiles of 128 x 128 (dg_tile.cuh).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "dg.h"
#include "dg_host.cuh"
#include "dg_ptx.cuh"
#include "dg_quant.cuh"
#include "dg_tile.cuh"

namespace dg {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int GLU_WARPS = 4;
constexpr int GLU_ROWS = 8 * GLU_WARPS;           // rows of a CTA

struct GluParams {
    const __nv_bfloat16* z;
    uint8_t* q;
    float* sf;
    uint8_t* kept;
    float* kept_sf;
    const int32_t* m_indices;
    const int32_t* masked_m;
    int m, inner, max_m, pow2;
};

// Four lines' largest magnitudes over 16 lanes, giving away lines on the way: lane l ends with that of line l / 4.
__device__ __forceinline__ float four_maxima(const float (&a)[4], int l16) {
    const bool up8 = (l16 & 8) != 0, up4 = (l16 & 4) != 0;
    const float b0 = abs_max(up8 ? a[2] : a[0], __shfl_xor_sync(FULL, up8 ? a[0] : a[2], 8));
    const float b1 = abs_max(up8 ? a[3] : a[1], __shfl_xor_sync(FULL, up8 ? a[1] : a[3], 8));
    float most = abs_max(up4 ? b1 : b0, __shfl_xor_sync(FULL, up4 ? b0 : b1, 4));
    most = abs_max(most, __shfl_xor_sync(FULL, most, 2));
    return abs_max(most, __shfl_xor_sync(FULL, most, 1));
}

__device__ __forceinline__ float abs_max8(const float2 (&a)[4]) {
    return abs_max(abs_max(a[0].x, a[0].y, a[1].x), abs_max(a[1].y, a[2].x, a[2].y), abs_max(a[3].x, a[3].y));
}

__device__ __forceinline__ void unpack_bf16(const uint4& v, float2 (&a)[4]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
}

// Codes of 4 rows of a block of 128 and their scales; `rows` has a bit for each row that is written.
__device__ __forceinline__ void quantise_rows(const float2 (&v)[4][4], uint8_t* q, size_t pitch, float* sf, size_t scales, bool pow2, unsigned rows,
                                              int l16) {
    const float a[4] = {abs_max8(v[0]), abs_max8(v[1]), abs_max8(v[2]), abs_max8(v[3])};
    const uint32_t most = abs_bits(four_maxima(a, l16));
    const BlockScale mine = pow2 ? block_scale_pow2(most) : block_scale(most);
    if ((l16 & 3) == 0 && (rows >> (l16 >> 2) & 1)) sf[static_cast<size_t>(l16 >> 2) * scales] = mine.s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        BlockScale k;
        k.d = __shfl_sync(FULL, mine.d, i * 4, 16);
        k.r = __shfl_sync(FULL, mine.r, i * 4, 16);
        const uint2 w = make_uint2(quantise4(v[i][0], v[i][1], k), quantise4(v[i][2], v[i][3], k));
        if (rows >> i & 1) *reinterpret_cast<uint2*>(q + static_cast<size_t>(i) * pitch) = w;
    }
}

template <int ACT>
__global__ void __launch_bounds__(32 * GLU_WARPS) glu_kernel(const GluParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, l16 = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
    const int r0 = static_cast<int>(blockIdx.x) * GLU_ROWS + warp * 8 + half * 4;
    const int c0 = static_cast<int>(blockIdx.y) * 128 + l16 * 8;
    unsigned rows = 0;
    if (p.m_indices != nullptr) {
        // (4 rows are of one block of 128, which is computed if its first row has an expert)
        if (r0 < p.m && ld_input(p.m_indices + r0 / 128 * 128) >= 0) rows = 15;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r0 + i < p.m && (p.masked_m == nullptr || (r0 + i) % p.max_m < ld_input(p.masked_m + (r0 + i) / p.max_m))) rows |= 1u << i;
    }
    if (__all_sync(FULL, rows == 0)) return;

    const size_t base = static_cast<size_t>(r0) * (2 * p.inner) + c0;
    uint4 gw[4], uw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        gw[i] = uw[i] = make_uint4(0, 0, 0, 0);
        if (rows >> i & 1) {
            gw[i] = ld_input(reinterpret_cast<const uint4*>(p.z + base + static_cast<size_t>(i) * (2 * p.inner)));
            uw[i] = ld_input(reinterpret_cast<const uint4*>(p.z + base + static_cast<size_t>(i) * (2 * p.inner) + p.inner));
        }
    }
    const size_t blocks = p.inner / 128;
    float2 v[4][4];
    if (p.kept != nullptr) {
        float* sf = p.kept_sf + static_cast<size_t>(r0) * (2 * blocks) + blockIdx.y;
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack_bf16(gw[i], v[i]);
        quantise_rows(v, p.kept + base, 2 * static_cast<size_t>(p.inner), sf, 2 * blocks, false, rows, l16);
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack_bf16(uw[i], v[i]);
        quantise_rows(v, p.kept + base + p.inner, 2 * static_cast<size_t>(p.inner), sf + blocks, 2 * blocks, false, rows, l16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 g[4], u[4];
        unpack_bf16(gw[i], g);
        unpack_bf16(uw[i], u);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] = __fmul2_rn(act_value2<ACT>(g[c]), u[c]);
    }
    quantise_rows(v, p.q + static_cast<size_t>(r0) * p.inner + c0, p.inner, p.sf + static_cast<size_t>(r0) * blocks + blockIdx.y, blocks, p.pow2 != 0, rows, l16);
}

// ------------------------------------------------------------------------------------ backward
// Eight codes times their scale.
__device__ __forceinline__ void code_values(uint2 w, float s, float2 (&a)[4]) {
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        a[i] = __fmul2_rn(__half22float2(__half2(h)), make_float2(s, s));
    }
}

struct GluBackwardParams {
    const __nv_bfloat16* dh;
    const __nv_bfloat16* z;
    const uint8_t* kept;
    const float* kept_sf;
    uint8_t* q;
    float* sf;
    uint8_t* qt;
    float* sft;
    uint8_t* ht;
    float* hsft;
    int m, inner, m_tiles;
};

// blockIdx.z: what of the tile this CTA makes: dg, du or h.
template <int ACT, bool KEPT>
__global__ void __launch_bounds__(TILE_THREADS, 2) glu_backward_kernel(const GluBackwardParams p) {
    __shared__ TileShared s;
    grid_dependency_wait();
    grid_launch_dependents();
    const TileThread me;
    const int part = static_cast<int>(blockIdx.z);
    const int m0 = static_cast<int>(blockIdx.x) * TILE, n0 = static_cast<int>(blockIdx.y) * TILE;
    const int valid = p.m - (m0 + me.row);
    const size_t row = m0 + me.row, inner = p.inner, blocks = inner / 128;

    float2 v[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 d[4], g[4], u[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) d[c] = g[c] = u[c] = make_float2(0.f, 0.f);
        if (i < valid) {
            if (part != 2) unpack_bf16(ld_input(reinterpret_cast<const uint4*>(p.dh + (row + i) * inner + n0 + me.column)), d);
            const size_t at = (row + i) * (2 * inner) + n0 + me.column;
            if (KEPT) {
                const float* sf = p.kept_sf + (row + i) * (2 * blocks) + blockIdx.y;
                code_values(ld_input(reinterpret_cast<const uint2*>(p.kept + at)), ld_input(sf), g);
                code_values(ld_input(reinterpret_cast<const uint2*>(p.kept + at + inner)), ld_input(sf + blocks), u);
            } else {
                unpack_bf16(ld_input(reinterpret_cast<const uint4*>(p.z + at)), g);
                unpack_bf16(ld_input(reinterpret_cast<const uint4*>(p.z + at + inner)), u);
            }
        }
        // (rows past M are 0: so are the activations there, and their slopes are finite)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (part == 0) v[i][c] = __fmul2_rn(__fmul2_rn(d[c], u[c]), act_slope2<ACT>(g[c]));
            else v[i][c] = __fmul2_rn(act_value2<ACT>(g[c]), part == 1 ? d[c] : u[c]);
        }
    }
    const size_t column = part == 1 ? inner + n0 : n0, pitch = static_cast<size_t>(p.m_tiles) * TILE;
    if (part != 2) {
        if (p.q != nullptr)
            tile_rows(v, p.q + row * (2 * inner) + column + me.column, 2 * inner, p.sf + row * (2 * blocks) + column / 128, 2 * blocks, valid, me.l16);
        if (p.qt != nullptr)
            tile_columns(v, s, p.qt + column * pitch + m0, pitch, p.sft + column * p.m_tiles + blockIdx.x, p.m_tiles, me);
    } else {
        tile_columns(v, s, p.ht + column * pitch + m0, pitch, p.hsft + column * p.m_tiles + blockIdx.x, p.m_tiles, me);
    }
}

struct TransposeParams {
    const uint8_t* q;
    const float* sf;
    uint8_t* qt;
    float* sft;
    int m, n, m_tiles;
};

__global__ void __launch_bounds__(TILE_THREADS, 2) transpose_kernel(const TransposeParams p) {
    __shared__ TileShared s;
    grid_dependency_wait();
    grid_launch_dependents();
    const TileThread me;
    const int m0 = static_cast<int>(blockIdx.x) * TILE, n0 = static_cast<int>(blockIdx.y) * TILE;
    const int valid = p.m - (m0 + me.row);
    float2 v[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t row = m0 + me.row + i;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] = make_float2(0.f, 0.f);
        if (i < valid) code_values(ld_input(reinterpret_cast<const uint2*>(p.q + row * p.n + n0 + me.column)), ld_input(p.sf + row * (p.n / 128) + blockIdx.y), v[i]);
    }
    const size_t pitch = static_cast<size_t>(p.m_tiles) * TILE;
    tile_columns(v, s, p.qt + n0 * pitch + m0, pitch, p.sft + static_cast<size_t>(n0) * p.m_tiles + blockIdx.x, p.m_tiles, me);
}

template <bool KEPT>
cudaError_t launch_backward(const GluBackwardParams& p, int act, int parts, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.m_tiles), static_cast<unsigned>(p.inner / TILE), static_cast<unsigned>(parts)), block(TILE_THREADS);
    switch (act) {
        case DG_ACT_RELU: return launch_overlapped(glu_backward_kernel<DG_ACT_RELU, KEPT>, grid, block, stream, p);
        case DG_ACT_GELU: return launch_overlapped(glu_backward_kernel<DG_ACT_GELU, KEPT>, grid, block, stream, p);
        case DG_ACT_GELU_TANH: return launch_overlapped(glu_backward_kernel<DG_ACT_GELU_TANH, KEPT>, grid, block, stream, p);
        case DG_ACT_SILU: return launch_overlapped(glu_backward_kernel<DG_ACT_SILU, KEPT>, grid, block, stream, p);
        default: return launch_overlapped(glu_backward_kernel<DG_ACT_NONE, KEPT>, grid, block, stream, p);
    }
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_glu(const void* Z, uint8_t* q, float* sf, uint8_t* kept, float* kept_sf, const int32_t* m_indices, const int32_t* masked_m, int G,
                 int act, int pow2, int M, int I, cudaStream_t stream) {
    if (M < 0 || I < 0 || G < 0 || act < DG_ACT_NONE || act > DG_ACT_SILU) return DG_INVALID_ARG;
    if ((kept == nullptr) != (kept_sf == nullptr) || (m_indices && masked_m)) return DG_INVALID_ARG;
    if (I % 128 != 0 || I / 128 > 65535) return DG_UNSUPPORTED_SHAPE;
    if (m_indices && M % 128 != 0) return DG_UNSUPPORTED_SHAPE;
    if (masked_m && (G < 1 || M % G != 0)) return DG_INVALID_ARG;
    if (M == 0 || I == 0) return DG_OK;
    if (M > INT32_MAX - GLU_ROWS) return DG_UNSUPPORTED_SHAPE;
    if (!Z || !q || !sf) return DG_INVALID_ARG;
    if (!aligned(Z, 16) || !aligned(q, 16) || !aligned(kept, 16) || !aligned(sf, 4) || !aligned(kept_sf, 4) || !aligned(m_indices, 4) || !aligned(masked_m, 4))
        return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status st = device_info(&dev);
    if (st != DG_OK) return st;
    GluParams p;
    p.z = static_cast<const __nv_bfloat16*>(Z);
    p.q = q;
    p.sf = sf;
    p.kept = kept;
    p.kept_sf = kept_sf;
    p.m_indices = m_indices;
    p.masked_m = masked_m;
    p.m = M;
    p.inner = I;
    p.max_m = masked_m ? M / G : M;
    p.pow2 = pow2;
    const dim3 grid(static_cast<unsigned>(cdiv(M, GLU_ROWS)), static_cast<unsigned>(I / 128)), block(32 * GLU_WARPS);
    cudaError_t e = cudaErrorInvalidValue;
    switch (act) {
        case DG_ACT_NONE: e = launch_overlapped(glu_kernel<DG_ACT_NONE>, grid, block, stream, p); break;
        case DG_ACT_RELU: e = launch_overlapped(glu_kernel<DG_ACT_RELU>, grid, block, stream, p); break;
        case DG_ACT_GELU: e = launch_overlapped(glu_kernel<DG_ACT_GELU>, grid, block, stream, p); break;
        case DG_ACT_GELU_TANH: e = launch_overlapped(glu_kernel<DG_ACT_GELU_TANH>, grid, block, stream, p); break;
        case DG_ACT_SILU: e = launch_overlapped(glu_kernel<DG_ACT_SILU>, grid, block, stream, p); break;
    }
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

dg_status dg_glu_backward(const void* dH, const void* Z, const uint8_t* kept, const float* kept_sf, int act, uint8_t* q, float* sf, uint8_t* qt,
                          float* sft, uint8_t* ht, float* hsft, int M, int I, cudaStream_t stream) {
    if (M < 0 || I < 0 || act < DG_ACT_NONE || act > DG_ACT_SILU) return DG_INVALID_ARG;
    if ((q == nullptr) != (sf == nullptr) || (qt == nullptr) != (sft == nullptr) || (ht == nullptr) != (hsft == nullptr)) return DG_INVALID_ARG;
    if ((kept == nullptr) != (kept_sf == nullptr) || (Z && kept)) return DG_INVALID_ARG;
    if (I % 128 != 0 || I / 128 > 65535) return DG_UNSUPPORTED_SHAPE;
    if (M == 0 || I == 0 || (!q && !qt && !ht)) return DG_OK;
    if (M > INT32_MAX - TILE) return DG_UNSUPPORTED_SHAPE;
    if ((!Z && !kept) || ((q || qt) && !dH)) return DG_INVALID_ARG;
    if (!aligned(dH, 16) || !aligned(Z, 16) || !aligned(kept, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(ht, 16) || !aligned(kept_sf, 4) ||
        !aligned(sf, 4) || !aligned(sft, 4) || !aligned(hsft, 4))
        return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status st = device_info(&dev);
    if (st != DG_OK) return st;
    GluBackwardParams p;
    p.dh = static_cast<const __nv_bfloat16*>(dH);
    p.z = static_cast<const __nv_bfloat16*>(Z);
    p.kept = kept;
    p.kept_sf = kept_sf;
    p.q = q;
    p.sf = sf;
    p.qt = qt;
    p.sft = sft;
    p.ht = ht;
    p.hsft = hsft;
    p.m = M;
    p.inner = I;
    p.m_tiles = cdiv(M, TILE);
    const int parts = ht ? 3 : 2;
    const cudaError_t e = kept ? launch_backward<true>(p, act, parts, stream) : launch_backward<false>(p, act, parts, stream);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

dg_status dg_transpose_fp8(const uint8_t* q, const float* sf, uint8_t* qt, float* sft, int M, int N, cudaStream_t stream) {
    if (M < 0 || N < 0) return DG_INVALID_ARG;
    if (N % 128 != 0 || N / 128 > 65535) return DG_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return DG_OK;
    if (M > INT32_MAX - TILE) return DG_UNSUPPORTED_SHAPE;
    if (!q || !sf || !qt || !sft) return DG_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(qt, 16) || !aligned(sf, 4) || !aligned(sft, 4)) return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status st = device_info(&dev);
    if (st != DG_OK) return st;
    const TransposeParams p = {q, sf, qt, sft, M, N, cdiv(M, TILE)};
    const cudaError_t e = launch_overlapped(transpose_kernel, dim3(static_cast<unsigned>(p.m_tiles), static_cast<unsigned>(N / TILE)), dim3(TILE_THREADS), stream, p);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

}  // extern "C"
