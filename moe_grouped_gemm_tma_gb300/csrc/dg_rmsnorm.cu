// Root-mean-square norm with the residual's addition (dg_rmsnorm), its output quantised for the FP8 products, and its
// gradient (dg_rmsnorm_backward).
//
//   s = bf16(x + residual),  r = rsqrt(mean(s^2) + eps),  y = s r g
//   dx = r (g dy - s r^2 mean(g dy s)) + dsum,  dg = sum over rows of dy s r
//
// What bounds them is memory: 16381 x 7168 with residual, sum and both outputs takes 153 us (6.9 TB/s), its gradient at 8192 x 7168
// 74.1 (6.3 TB/s, the second launch for the weight gradient included); one row of 7168 takes 3.0 us in a CUDA graph.
//
// A row is in registers from its load to its stores: up to 1024 values a warp has a row of its own, above that a CTA with
// up to 32 values a thread. A thread's vectors of 8 values are a whole CTA (warp) apart, so that every load covers
// consecutive memory, and 16 consecutive lanes hold the 128 values of a scaling block.
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
constexpr int NORM_VECTORS = 4;                   // vectors of 8 values a thread at most
constexpr int NORM_MAX_WARPS = 16;
constexpr int NORM_MAX_H = NORM_MAX_WARPS * 32 * NORM_VECTORS * 8;
constexpr int NORM_WARP_H = 32 * NORM_VECTORS * 8;   // rows up to this are a warp's
constexpr int NORM_MAX_T = INT32_MAX - 65536;     // (rows are numbered in 32 bits, a few thousand past the last too)
constexpr int NORM_ROWS = 4;                      // rows of a CTA then
constexpr int NORM_BACK_ROWS = 8;                 // ... and of the gradient's

struct NormParams {
    const uint4* x;
    const uint4* residual;
    const void* weight;
    uint4* sum;
    uint4* y;
    uint2* q;
    float* sf;
    int rows, vectors, pow2;
    float inverse, eps;                           // 1 / H
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float2 a) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(a.y), "f"(a.x));
    return d;
}

__device__ __forceinline__ uint4 pack_bf16(const float2 (&a)[4]) {
    return make_uint4(pack_bf16(a[0]), pack_bf16(a[1]), pack_bf16(a[2]), pack_bf16(a[3]));
}

__device__ __forceinline__ void unpack_bf16(const uint4& v, float2 (&a)[4]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
}

// Eight of the norm's weights.
template <typename W>
__device__ __forceinline__ void load_weights(const void* weight, int v, float2 (&g)[4]) {
    if constexpr (sizeof(W) == 2) {
        unpack_bf16(ld_input(static_cast<const uint4*>(weight) + v), g);
    } else {
        const float4 a = ld_input(static_cast<const float4*>(weight) + 2 * v), b = ld_input(static_cast<const float4*>(weight) + 2 * v + 1);
        g[0] = make_float2(a.x, a.y);
        g[1] = make_float2(a.z, a.w);
        g[2] = make_float2(b.x, b.y);
        g[3] = make_float2(b.z, b.w);
    }
}

// The largest magnitude of a lane's eight values.
__device__ __forceinline__ float abs_max8(const float2 (&a)[4]) {
    return abs_max(abs_max(a[0].x, a[0].y, a[1].x), abs_max(a[1].y, a[2].x, a[2].y), abs_max(a[3].x, a[3].y));
}

// ROW_CTA: a row a CTA, else a row a warp; N vectors a thread.
template <typename W, bool ROW_CTA, int N>
__global__ void __launch_bounds__(ROW_CTA ? 32 * NORM_MAX_WARPS : 32 * NORM_ROWS) rmsnorm_kernel(const NormParams p) {
    __shared__ float s_part[NORM_MAX_WARPS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = static_cast<int>(ROW_CTA ? blockIdx.x : blockIdx.x * NORM_ROWS + warp);
    if (!ROW_CTA && row >= p.rows) return;
    const int first = ROW_CTA ? threadIdx.x : lane, step = ROW_CTA ? blockDim.x : 32;
    const size_t base = static_cast<size_t>(row) * p.vectors;

    uint4 x[N], r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int v = first + i * step;
        x[i] = make_uint4(0, 0, 0, 0);
        r[i] = make_uint4(0, 0, 0, 0);
        if (v < p.vectors) {
            x[i] = ld_input(p.x + base + v);
            if (p.residual != nullptr) r[i] = ld_input(p.residual + base + v);
        }
    }
    float2 squares = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int v = first + i * step;
        float2 a[4];
        unpack_bf16(x[i], a);
        if (p.residual != nullptr) {
            float2 b[4];
            unpack_bf16(r[i], b);
#pragma unroll
            for (int c = 0; c < 4; ++c) a[c] = __fadd2_rn(a[c], b[c]);
            x[i] = pack_bf16(a);                  // the sum as it is kept: the norm is of that
            unpack_bf16(x[i], a);
        }
        if (p.sum != nullptr && v < p.vectors) p.sum[base + v] = x[i];
#pragma unroll
        for (int c = 0; c < 4; ++c) squares = __ffma2_rn(a[c], a[c], squares);
    }
    float total = warp_sum(squares.x + squares.y);
    if (ROW_CTA) {
        if (lane == 0) s_part[warp] = total;
        __syncthreads();
        total = 0.f;
        for (int w = 0; w < step / 32; ++w) total += s_part[w];
    }
    const float rs = __frsqrt_rn(fmaf(total, p.inverse, p.eps));

    float2 a[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int v = first + i * step;
        float2 g[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) g[c] = make_float2(0.f, 0.f);
        if (v < p.vectors) load_weights<W>(p.weight, v, g);
        unpack_bf16(x[i], a[i]);
#pragma unroll
        for (int c = 0; c < 4; ++c) a[i][c] = __fmul2_rn(__fmul2_rn(a[i][c], make_float2(rs, rs)), g[c]);
        if (p.y != nullptr && v < p.vectors) p.y[base + v] = pack_bf16(a[i]);
    }
    if (p.q == nullptr) return;
    // (a scaling block's 16 lanes are inside the row, or none of them is)
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int v = first + i * step;
        float m = v < p.vectors ? abs_max8(a[i]) : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = abs_max(m, __shfl_xor_sync(FULL, m, o));
        const BlockScale k = p.pow2 ? block_scale_pow2(abs_bits(m)) : block_scale(abs_bits(m));
        if (v < p.vectors) {
            p.q[base + v] = make_uint2(quantise4(a[i][0], a[i][1], k), quantise4(a[i][2], a[i][3], k));
            if ((lane & 15) == 0) p.sf[static_cast<size_t>(row) * (p.vectors / 16) + v / 16] = k.s;
        }
    }
}

// ------------------------------------------------------------------------------------ gradient
struct NormBackwardParams {
    const uint4* dy;
    const uint4* x;
    const void* weight;
    const uint4* dsum;
    uint4* dx;
    float* partial;                               // [ctas][H] weight gradients of a CTA's rows
    int rows, vectors, ctas;
    float inverse, eps;
};

// A group (a CTA, or a warp of 8 in a CTA) takes every groups-th row and keeps its columns' weight gradient in registers. The rows come
// by asynchronous copies into shared memory, NORM_STAGES rows ahead, each thread's vectors to places of its own, so that no
// thread waits for another's copies; the row's two sums cost the only barrier. (By loads into registers, 8192 x 7168 took 118 us.)
constexpr int NORM_STAGES = 2;

template <typename W, bool ROW_CTA, int N>
__global__ void __launch_bounds__(ROW_CTA ? 32 * NORM_MAX_WARPS : 32 * NORM_BACK_ROWS, ROW_CTA ? (N == 4 ? 1 : 2) : (N == 4 ? 2 : 4)) rmsnorm_backward_kernel(const NormBackwardParams p) {
    extern __shared__ __align__(16) uint4 s_rows[];   // [stage][x, dy, dsum][N][thread]
    __shared__ float2 s_part[2][NORM_MAX_WARPS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = static_cast<int>(ROW_CTA ? blockIdx.x : blockIdx.x * NORM_BACK_ROWS + warp);
    const int groups = static_cast<int>(ROW_CTA ? gridDim.x : gridDim.x * NORM_BACK_ROWS);
    const int first = ROW_CTA ? threadIdx.x : lane, step = ROW_CTA ? blockDim.x : 32;
    const int threads = blockDim.x, arrays = p.dsum != nullptr ? 3 : 2;
    uint4* mine = s_rows + threadIdx.x;
    const auto place = [&](int stage, int array, int i) { return mine + ((stage * arrays + array) * N + i) * threads; };
    const auto fetch = [&](int row, int stage) {
        if (row < p.rows) {
            const size_t base = static_cast<size_t>(row) * p.vectors;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int v = first + i * step;
                if (v < p.vectors) {
                    cp_async_16(place(stage, 0, i), p.x + base + v);
                    cp_async_16(place(stage, 1, i), p.dy + base + v);
                    if (arrays == 3) cp_async_16(place(stage, 2, i), p.dsum + base + v);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NORM_STAGES; ++i) fetch(group + i * groups, i);

    float2 g[N][4], dg[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int c = 0; c < 4; ++c) g[i][c] = dg[i][c] = make_float2(0.f, 0.f);
        if (first + i * step < p.vectors) load_weights<W>(p.weight, first + i * step, g[i]);
    }
    int turn = 0, stage = 0;
    for (int row = group; row < p.rows; row += groups, turn ^= 1, stage = stage + 1 == NORM_STAGES ? 0 : stage + 1) {
        const size_t base = static_cast<size_t>(row) * p.vectors;
        cp_async_wait_group<NORM_STAGES - 1>();
        float2 squares = make_float2(0.f, 0.f), products = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (first + i * step >= p.vectors) break;
            float2 a[4], b[4];
            unpack_bf16(*place(stage, 0, i), a);
            unpack_bf16(*place(stage, 1, i), b);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                squares = __ffma2_rn(a[c], a[c], squares);
                products = __ffma2_rn(__fmul2_rn(b[c], g[i][c]), a[c], products);
            }
        }
        float2 total = make_float2(warp_sum(squares.x + squares.y), warp_sum(products.x + products.y));
        if (ROW_CTA) {
            if (lane == 0) s_part[turn][warp] = total;
            __syncthreads();
            total = make_float2(0.f, 0.f);
            for (int w = 0; w < step / 32; ++w) total = __fadd2_rn(total, s_part[turn][w]);
        }
        const float rs = __frsqrt_rn(fmaf(total.x, p.inverse, p.eps));
        const float mean = rs * rs * (total.y * p.inverse);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int v = first + i * step;
            if (v >= p.vectors) break;
            float2 a[4], b[4], z[4];
            unpack_bf16(*place(stage, 0, i), a);
            unpack_bf16(*place(stage, 1, i), b);
            unpack_bf16(arrays == 3 ? *place(stage, 2, i) : make_uint4(0, 0, 0, 0), z);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                dg[i][c] = __ffma2_rn(__fmul2_rn(b[c], a[c]), make_float2(rs, rs), dg[i][c]);
                const float2 t = __ffma2_rn(a[c], make_float2(-mean, -mean), __fmul2_rn(b[c], g[i][c]));
                z[c] = __ffma2_rn(t, make_float2(rs, rs), z[c]);
            }
            p.dx[base + v] = pack_bf16(z);
        }
        fetch(row + NORM_STAGES * groups, stage);
    }
    if (p.partial == nullptr) return;
    if (!ROW_CTA) {
        // the warps' sums, in order, by way of the rows' places
        cp_async_wait_all();
        __syncthreads();
        float4* s_sums = reinterpret_cast<float4*>(s_rows);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (first + i * step >= p.vectors) break;
            float4* dst = s_sums + (warp * p.vectors + first + i * step) * 2;
            dst[0] = make_float4(dg[i][0].x, dg[i][0].y, dg[i][1].x, dg[i][1].y);
            dst[1] = make_float4(dg[i][2].x, dg[i][2].y, dg[i][3].x, dg[i][3].y);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * p.vectors; i += threads) {
            float4 a = s_sums[i];
#pragma unroll
            for (int w = 1; w < NORM_BACK_ROWS; ++w) {
                const float4 b = s_sums[w * 2 * p.vectors + i];
                a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
            }
            __stcg(reinterpret_cast<float4*>(p.partial) + static_cast<size_t>(blockIdx.x) * 2 * p.vectors + i, a);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int v = first + i * step;
            if (v < p.vectors) {
                float4* dst = reinterpret_cast<float4*>(p.partial + (static_cast<size_t>(group) * p.vectors + v) * 8);
                __stcg(dst, make_float4(dg[i][0].x, dg[i][0].y, dg[i][1].x, dg[i][1].y));
                __stcg(dst + 1, make_float4(dg[i][2].x, dg[i][2].y, dg[i][3].x, dg[i][3].y));
            }
        }
    }
}

// The weight gradient from the groups' sums: 32 columns a CTA, every ADD_WARPS-th group a warp, then the warps in order.
constexpr int ADD_WARPS = 16;
__global__ void __launch_bounds__(32 * ADD_WARPS) add_groups_kernel(const float* partial, float* dweight, int H, int groups) {
    __shared__ float s_sum[ADD_WARPS][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = static_cast<int>(blockIdx.x) * 32 + lane;
    float a = 0.f;
    if (c < H) {
#pragma unroll 8
        for (int i = warp; i < groups; i += ADD_WARPS) a += __ldcg(partial + static_cast<size_t>(i) * H + c);
    }
    s_sum[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < H) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < ADD_WARPS; ++w) sum += s_sum[w][lane];
        dweight[c] = sum;
    }
}

template <typename W>
cudaError_t launch_norm(const NormParams& p, int H, cudaStream_t stream) {
    const auto go = [&](auto kernel, bool cta) {
        const unsigned grid = static_cast<unsigned>(cta ? p.rows : cdiv(p.rows, NORM_ROWS));
        const unsigned block = static_cast<unsigned>(cta ? 32 * cdiv(H, NORM_WARP_H) : 32 * NORM_ROWS);
        return launch_overlapped(kernel, dim3(grid), dim3(block), stream, p);
    };
    if (H > NORM_WARP_H) return go(rmsnorm_kernel<W, true, NORM_VECTORS>, true);
    if (H > 512) return go(rmsnorm_kernel<W, false, 4>, false);
    if (H > 256) return go(rmsnorm_kernel<W, false, 2>, false);
    return go(rmsnorm_kernel<W, false, 1>, false);
}

template <typename W, bool ROW_CTA, int N>
cudaError_t launch_norm_backward_as(const NormBackwardParams& p, int H, cudaStream_t stream) {
    constexpr auto kernel = rmsnorm_backward_kernel<W, ROW_CTA, N>;
    constexpr int STAGE = 3 * N * 16 * (ROW_CTA ? 32 * NORM_MAX_WARPS : 32 * NORM_BACK_ROWS);      // of the largest CTA
    const unsigned grid = static_cast<unsigned>(p.ctas);
    const unsigned block = static_cast<unsigned>(ROW_CTA ? 32 * cdiv(H, 32 * 8 * N) : 32 * NORM_BACK_ROWS);
    const cudaError_t e = allow_smem<kernel>(NORM_STAGES * STAGE);
    if (e != cudaSuccess) return e;
    return launch_overlapped_smem(kernel, dim3(grid), dim3(block), static_cast<size_t>(NORM_STAGES) * (p.dsum != nullptr ? 3 : 2) * N * block * 16, stream, p);
}

template <typename W>
cudaError_t launch_norm_backward(const NormBackwardParams& p, int H, cudaStream_t stream) {
    if (H > NORM_MAX_H / 2) return launch_norm_backward_as<W, true, 4>(p, H, stream);
    if (H > NORM_WARP_H) return launch_norm_backward_as<W, true, 2>(p, H, stream);
    if (H > 512) return launch_norm_backward_as<W, false, 4>(p, H, stream);
    if (H > 256) return launch_norm_backward_as<W, false, 2>(p, H, stream);
    return launch_norm_backward_as<W, false, 1>(p, H, stream);
}

// CTAs of the gradient: about what fits the GPU at once, but rather one an SM than fewer than 8 rows for a CTA (4 for a warp),
// whose sums would be as many as its rows (900 x 3792: 9.4 us, with a row or two for each of 608 CTAs 15.2). By the sizes alone, so that
// sums do not depend on the GPU.
int norm_ctas(int T, int H) {
    const bool warp_rows = H <= NORM_WARP_H;
    const int most = warp_rows ? 304 : H <= 4096 ? 608 : H <= NORM_MAX_H / 2 ? 304 : 152;
    const int one = warp_rows ? cdiv(T, NORM_BACK_ROWS) : T;      // a row a warp, or a CTA
    const int few = warp_rows ? cdiv(T, 4 * NORM_BACK_ROWS) : cdiv(T, 8);
    const int least = one < 152 ? one : 152;
    return few > most ? most : few > least ? few : least;
}

dg_status norm_check(int weight_type, int T, int H, float eps) {
    if (T < 0 || H < 0 || !(eps >= 0.f)) return DG_INVALID_ARG;
    if (weight_type != DG_TYPE_BF16 && weight_type != DG_TYPE_F32) return DG_INVALID_ARG;
    if (H % 8 != 0 || H > NORM_MAX_H || T > NORM_MAX_T) return DG_UNSUPPORTED_SHAPE;
    return DG_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_rmsnorm(const void* x, const void* residual, const void* weight, int weight_type, void* sum, void* y, uint8_t* q, float* sf,
                     int pow2, int T, int H, float eps, cudaStream_t stream) {
    const dg_status st = norm_check(weight_type, T, H, eps);
    if (st != DG_OK) return st;
    if ((q == nullptr) != (sf == nullptr)) return DG_INVALID_ARG;
    if (q && H % 128 != 0) return DG_UNSUPPORTED_SHAPE;
    if (T == 0 || H == 0 || (!sum && !y && !q)) return DG_OK;
    if (!x || !weight) return DG_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) || !aligned(y, 16) || !aligned(q, 16) || !aligned(sf, 4))
        return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status ds = device_info(&dev);
    if (ds != DG_OK) return ds;
    NormParams p;
    p.x = static_cast<const uint4*>(x);
    p.residual = static_cast<const uint4*>(residual);
    p.weight = weight;
    p.sum = static_cast<uint4*>(sum);
    p.y = static_cast<uint4*>(y);
    p.q = reinterpret_cast<uint2*>(q);
    p.sf = sf;
    p.rows = T;
    p.vectors = H / 8;
    p.pow2 = pow2;
    p.inverse = 1.f / static_cast<float>(H);
    p.eps = eps;
    const cudaError_t e = weight_type == DG_TYPE_F32 ? launch_norm<float>(p, H, stream) : launch_norm<__nv_bfloat16>(p, H, stream);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

int64_t dg_rmsnorm_backward_workspace(int T, int H) {
    if (T < 0 || H < 0 || H % 8 != 0 || H > NORM_MAX_H || T > NORM_MAX_T) return -1;
    return static_cast<int64_t>(norm_ctas(T, H)) * H * 4;
}

dg_status dg_rmsnorm_backward(const void* dy, const void* x, const void* weight, int weight_type, const void* dsum, void* dx, float* dweight,
                              void* workspace, int64_t workspace_bytes, int T, int H, float eps, cudaStream_t stream) {
    const dg_status st = norm_check(weight_type, T, H, eps);
    if (st != DG_OK) return st;
    if (H == 0 || (T == 0 && !dweight)) return DG_OK;
    if (T > 0 && (!dy || !x || !weight || !dx)) return DG_INVALID_ARG;
    const int64_t need = dweight ? dg_rmsnorm_backward_workspace(T, H) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return DG_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(weight, 16) || !aligned(dsum, 16) || !aligned(dx, 16) || !aligned(dweight, 4) || !aligned(workspace, 16))
        return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status ds = device_info(&dev);
    if (ds != DG_OK) return ds;
    if (T == 0) return cudaMemsetAsync(dweight, 0, static_cast<size_t>(H) * 4, stream) == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
    NormBackwardParams p;
    p.dy = static_cast<const uint4*>(dy);
    p.x = static_cast<const uint4*>(x);
    p.weight = weight;
    p.dsum = static_cast<const uint4*>(dsum);
    p.dx = static_cast<uint4*>(dx);
    p.partial = dweight ? static_cast<float*>(workspace) : nullptr;
    p.rows = T;
    p.vectors = H / 8;
    p.ctas = norm_ctas(T, H);
    p.inverse = 1.f / static_cast<float>(H);
    p.eps = eps;
    cudaError_t e = weight_type == DG_TYPE_F32 ? launch_norm_backward<float>(p, H, stream) : launch_norm_backward<__nv_bfloat16>(p, H, stream);
    if (e == cudaSuccess && dweight)
        e = launch_overlapped(add_groups_kernel, dim3(static_cast<unsigned>(cdiv(H, 32))), dim3(32 * ADD_WARPS), stream, static_cast<const float*>(p.partial), dweight, H, p.ctas);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

}  // extern "C"
