// The router around the experts' products: top-k selection with its weights (dg_moe_route) and their
// gradient (dg_moe_route_backward), one warp a row.
//
// Selection. A lane holds VPL experts of the row: consecutive ones where the rows can be read in vectors, else
// every 32nd, so that a load or store of the warp still covers one piece of the row (E = 510, FP32, 25052 rows:
// the gradient took 52.8 us with consecutive experts and single loads, 13.0 so). k whole-warp maxima over the lanes' best values give a bound below which no selected value can lie (k lanes
// hold one at least as large); the few values at or above it -- k and a handful in practice -- are compacted
// through shared memory, one a lane, and each counts those that precede it (larger, or equal with a lower
// expert), which is its place in the order. More than 32 candidates (many equal values) take k rounds of
// find-and-remove instead.
//
// With a bias the selection values are sums of a sigmoid, and which of two close ones is larger has to be
// right: they are defined with an accurate exponential and a rounded reciprocal. Only the candidates pay for
// that: the bound is found with the hardware's approximations, lowered by more than they can be off.
//
// What bounds it is instruction issue: a row of 256 BF16 logits is 512 bytes, or 1.5 instructions' time on
// the whole GPU, and 250 instructions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>

#include "dg.h"
#include "dg_host.cuh"
#include "dg_ptx.cuh"
#include "dg_quant.cuh"

namespace dg {
namespace {

constexpr int ROUTE_WARPS = 8;
constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// The lane's VPL logits of a row, -inf past the row's end: consecutive ones by vector loads where the rows allow
// that (`vec`: VPL divides E, and rows and base are aligned to the lane's whole vector), else every 32nd.
template <int VPL, typename T>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, bool vec, float (&v)[VPL]) {
    const int e0 = lane * VPL;
    constexpr int BYTES = VPL * static_cast<int>(sizeof(T));
    if constexpr (BYTES >= 8) {
        if (vec) {
            if (e0 >= E) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) v[i] = -INFINITY;
                return;
            }
            constexpr int W = BYTES >= 16 ? 16 : 8;
            constexpr int PER = W / static_cast<int>(sizeof(T));
#pragma unroll
            for (int c = 0; c < BYTES / W; ++c) {
                uint32_t w[W / 4];
                if constexpr (W == 16) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + e0) + c);
                    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                } else {
                    const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + e0) + c);
                    w[0] = u.x; w[1] = u.y;
                }
#pragma unroll
                for (int j = 0; j < W / 4; ++j) {
                    if constexpr (sizeof(T) == 4) {
                        v[c * PER + j] = __uint_as_float(w[j]);
                    } else {
                        v[c * PER + 2 * j] = bf16_lo(w[j]);
                        v[c * PER + 2 * j + 1] = bf16_hi(w[j]);
                    }
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = lane + 32 * i < E ? to_f32(row[lane + 32 * i]) : -INFINITY;
}

__device__ __forceinline__ float warp_max(float v) {
    float d;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// the accurate form: the selection with a bias compares these values
__device__ __forceinline__ float sigmoid(float l) { return __frcp_rn(1.f + expf(-l)); }

// How far a sum of the approximate sigmoid and a bias may be from that of the accurate one: 2^-19 of the
// sigmoid's range covers the exponential (2 ulp and, for arguments whose sigmoid is not tiny, the rounding of
// its argument) and the reciprocal ten times over; the sums are rounded to 2^-24 of themselves on either side.
__device__ __forceinline__ float selection_margin(float sum) { return 1.9073486e-6f + 2.4e-7f * fabsf(sum); }

// The VPL biases of a lane's experts e0, e0 + step, ... (0 past the row's end).
template <int VPL>
__device__ __forceinline__ void load_bias(const float* bias, int E, int e0, int step, bool vec, float (&v)[VPL]) {
    if constexpr (VPL >= 4) {
        if (vec) {
#pragma unroll
            for (int c = 0; c < VPL / 4; ++c) {
                float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
                if (e0 < E) u = __ldg(reinterpret_cast<const float4*>(bias + e0) + c);
                v[4 * c] = u.x; v[4 * c + 1] = u.y; v[4 * c + 2] = u.z; v[4 * c + 3] = u.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = e0 + i * step < E ? __ldg(bias + e0 + i * step) : 0.f;
}

// +inf counts as the largest finite value, so that no score is a quotient of infinities
__device__ __forceinline__ float finite_top(float l) { return fminf(l, FLT_MAX); }

template <int VPL, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
route_kernel(const T* __restrict__ logits, const float* __restrict__ bias, int32_t* __restrict__ ids,
             float* __restrict__ weights, int rows, int E, int k, int sigmoid_scores, int renorm, float scale, int vec) {
    __shared__ __align__(16) float s_value[ROUTE_WARPS][32];
    __shared__ int s_cand[ROUTE_WARPS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (One row a warp: persistent warps with the next row and the bias in registers take 61 registers and were
    // slower at every grid size, 18.8 to 24 us against 14 to 16: the chain of exchanges within a row is hidden by other
    // warps, which need the registers.)
    const int t = static_cast<int>(blockIdx.x) * ROUTE_WARPS + warp;
    grid_dependency_wait();
    grid_launch_dependents();
    if (t >= rows) return;
    const T* row = logits + static_cast<size_t>(t) * E;
    const int e0 = (vec & 1) ? lane * VPL : lane, step = (vec & 1) ? 1 : 32;     // the lane's experts
    // selection values: the logits, or the approximate sums; -inf where an expert cannot be selected (NaN too)
    float v[VPL];
    load_row<VPL, T>(row, E, lane, (vec & 1) != 0, v);
    if (bias != nullptr) {
        float b[VPL];
        load_bias<VPL>(bias, E, e0, step, vec == 3, b);
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = v[i] > -INFINITY ? fast_sigmoid(v[i]) + b[i] : -INFINITY;
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = v[i] > -INFINITY ? finite_top(v[i]) : -INFINITY;
    }
    float head = -INFINITY;                        // (fmaxf drops NaN)
#pragma unroll
    for (int i = 0; i < VPL; ++i) head = fmaxf(head, v[i]);

    // softmax: the largest logit, and the sum where all scores count
    float top = 0.f, total = 1.f;
    if (!sigmoid_scores) {
        top = warp_max(head);
        if (!renorm) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum += v[i] > -INFINITY ? __expf(v[i] - top) : 0.f;
            total = warp_sum(sum);
        }
    }

    // the bound: the k-th whole-warp maximum of the lanes' best values
    float h = head, bound = -INFINITY;
    for (int j = 0; j < k; ++j) {
        bound = warp_max(h);
        if (h == bound) h = -INFINITY;
    }
    if (bias != nullptr && bound < INFINITY) bound -= 2.f * selection_margin(bound);
    bound = fmaxf(bound, -FLT_MAX);                // -inf is never a candidate
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (v[i] >= bound) mask |= 1u << i;
    const int mine = __popc(mask);
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(FULL, before, o);
        if (lane >= o) before += u;
    }
    const int found = __shfl_sync(FULL, before, 31);
    before -= mine;

    int place = -1, expert = -1;     // this lane's selected expert, and where it comes in the row
    float value = -INFINITY;         // its logit
    const int picked = min(found, k);
    if (found <= 32) {
        // the candidates one a lane, which reads its logit again (it knows where from only now)
        int at = before;
        for (uint32_t m = mask; m != 0; m &= m - 1) s_cand[warp][at++] = e0 + (__ffs(m) - 1) * step;
        __syncwarp();
        float me = -INFINITY;
        if (lane < found) {
            expert = s_cand[warp][lane];
            value = finite_top(to_f32(row[expert]));
            me = bias != nullptr ? sigmoid(value) + __ldg(bias + expert) : value;
        }
        s_value[warp][lane] = me;
        __syncwarp();
        // candidates that are at least as large, four a turn; without equal values the lanes' counts are
        // 1 .. found, and where they are not, equal ones are counted by their experts' order
        int ahead = -1;
        for (int c = 0; c < found; c += 4) {
            const float4 o = *reinterpret_cast<const float4*>(&s_value[warp][c]);
            ahead += (o.x >= me ? 1 : 0) + (o.y >= me ? 1 : 0) + (o.z >= me ? 1 : 0) + (o.w >= me ? 1 : 0);
        }
        const unsigned counts = __reduce_or_sync(FULL, lane < found ? 1u << ahead : 0u);
        if (__popc(counts) != found) {
            ahead = 0;
            for (int c = 0; c < found; ++c) {
                const float other = __shfl_sync(FULL, me, c);
                const int oe = __shfl_sync(FULL, expert, c);
                if (oe < expert ? other >= me : other > me) ++ahead;
            }
        }
        if (lane < found && ahead < k) place = ahead;
        else expert = -1;
    } else {
        // many equal values: k rounds of find-and-remove
        if (bias != nullptr) {
#pragma unroll 1
            for (int i = 0; i < VPL; ++i) {
                const int e = e0 + i * step;
                float exact = -INFINITY;
                if (e < E) {
                    const float l = to_f32(row[e]);
                    if (l > -INFINITY) exact = sigmoid(finite_top(l)) + __ldg(bias + e);
                }
#pragma unroll
                for (int x = 0; x < VPL; ++x)
                    if (x == i) v[x] = exact;
            }
        }
        for (int j = 0; j < k; ++j) {
            float best = -INFINITY;
            int bi = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (v[i] > best) { best = v[i]; bi = i; }
            const float most = warp_max(best);
            const int own = e0 + bi * step;
            const int e = __reduce_min_sync(FULL, best == most ? own : INT_MAX);
            if (own == e) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (i == bi) v[i] = -INFINITY;
            }
            if (lane == j) { place = j; expert = e; }
        }
        if (place >= 0) value = finite_top(to_f32(row[expert]));
    }

    float score = 0.f;
    if (place >= 0) score = sigmoid_scores ? sigmoid(value) : __expf(value - top);
    if (renorm) total = warp_sum(score);
    const float w = total > 0.f ? score * __frcp_rn(total) : 0.f;
    const size_t out = static_cast<size_t>(t) * k;
    if (place >= 0) {
        ids[out + place] = expert;
        weights[out + place] = w * scale;
    }
    if (lane >= picked && lane < k) {
        ids[out + lane] = -1;
        weights[out + lane] = 0.f;
    }
}

__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int VPL, typename T>
__device__ __forceinline__ void store_row(T* row, int E, int lane, bool vec, const float (&v)[VPL]) {
    const int e0 = lane * VPL;
    constexpr int BYTES = VPL * static_cast<int>(sizeof(T));
    if constexpr (BYTES >= 8) {
        if (vec) {
            if (e0 >= E) return;
            uint32_t w[BYTES / 4];
#pragma unroll
            for (int j = 0; j < BYTES / 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    w[j] = __float_as_uint(v[j]);
                } else {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t*>(&b);
                }
            }
            if constexpr (BYTES >= 16) {
#pragma unroll
                for (int c = 0; c < BYTES / 16; ++c)
                    reinterpret_cast<uint4*>(row + e0)[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            } else {
                *reinterpret_cast<uint2*>(row + e0) = make_uint2(w[0], w[1]);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < E) store_one(row + lane + 32 * i, v[i]);
}

// The gradient of the row's k weights with respect to its logits. With p the scores of the selected
// experts, r = p / sum p and s the scale:
//   softmax, renormalised   dl_j = s r_j (dw_j - sum_i r_i dw_i) for the selected, 0 elsewhere
//   softmax                 dl_e = p_e (s dw_e [selected] - sum_i s p_i dw_i) for every expert
//   sigmoid, renormalised   dl_j = s (1 - p_j) r_j (dw_j - sum_i r_i dw_i)
//   sigmoid                 dl_j = s p_j (1 - p_j) dw_j
// (the selection itself, and a bias that only moves it, have no gradient). Only the plain softmax reads
// the whole row; every form writes it. Bound by those bytes.
template <int VPL, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
route_backward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ dweights,
                      T* __restrict__ dlogits, int rows, int E, int k, int sigmoid_scores, int renorm, float scale, int vec) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = static_cast<int>(blockIdx.x) * ROUTE_WARPS + warp;
    grid_dependency_wait();
    grid_launch_dependents();
    if (t >= rows) return;
    const T* row = logits + static_cast<size_t>(t) * E;
    int e = lane < k ? __ldg(ids + static_cast<size_t>(t) * k + lane) : -1;
    const bool open = e >= 0 && e < E;
    const float dw = open ? __ldg(dweights + static_cast<size_t>(t) * k + lane) * scale : 0.f;
    float mine = open ? to_f32(row[e]) : -INFINITY;
    if (!(mine > -INFINITY)) mine = -INFINITY;            // NaN is not selectable either
    mine = finite_top(mine);

    float grad, out[VPL];
    if (!sigmoid_scores && !renorm) {
        float l[VPL];
        load_row<VPL, T>(row, E, lane, vec != 0, l);
        float top = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            l[i] = l[i] > -INFINITY ? finite_top(l[i]) : -INFINITY;
            top = fmaxf(top, l[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            out[i] = l[i] > -INFINITY ? __expf(l[i] - top) : 0.f;
            sum += out[i];
        }
        sum = warp_sum(sum);
        const float inv = sum > 0.f ? __frcp_rn(sum) : 0.f;
        const float p = mine > -INFINITY ? __expf(mine - top) * inv : 0.f;
        const float dot = warp_sum(p * dw);
        // duplicates of an expert in one row add up: every lane that names it ends with the same total
        float add = 0.f;
        for (int j = 0; j < k; ++j) {
            const int oe = __shfl_sync(FULL, open ? e : -1, j);
            const float od = __shfl_sync(FULL, dw, j);
            if (oe == e) add += od;
        }
        grad = p * (add - dot);
#pragma unroll
        for (int i = 0; i < VPL; ++i) out[i] = -(out[i] * inv) * dot;
    } else {
        float p, top = 0.f;
        if (sigmoid_scores) {
            p = mine > -INFINITY ? sigmoid(mine) : 0.f;
        } else {
            top = mine;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
            p = mine > -INFINITY ? __expf(mine - top) : 0.f;
        }
        float g;
        if (renorm) {
            const float sum = warp_sum(p);
            const float r = sum > 0.f ? __fdiv_rn(p, sum) : 0.f;
            g = r * (dw - warp_sum(r * dw));
            if (sigmoid_scores) g *= 1.f - p;
        } else {
            g = p * (1.f - p) * dw;
        }
        grad = 0.f;
        for (int j = 0; j < k; ++j) {
            const int oe = __shfl_sync(FULL, open ? e : -1, j);
            const float og = __shfl_sync(FULL, g, j);
            if (oe == e) grad += og;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) out[i] = 0.f;
    }
    T* drow = dlogits + static_cast<size_t>(t) * E;
    store_row<VPL, T>(drow, E, lane, vec != 0, out);
    __syncwarp();                                         // the selected experts' values come last
    if (open) store_one(drow + e, grad);
}

template <int VPL, typename T>
bool vector_rows(const void* a, const void* b, int E) {
    constexpr int BYTES = VPL * static_cast<int>(sizeof(T));
    constexpr int W = BYTES >= 16 ? 16 : BYTES;
    return BYTES >= 8 && E % VPL == 0 && (static_cast<int64_t>(E) * sizeof(T)) % W == 0 && aligned(a, W) && aligned(b, W);
}

template <int VPL, typename T>
cudaError_t launch_route(const void* logits, const float* bias, int32_t* ids, float* weights, int rows, int E, int k,
                         int scoring, int renorm, float scale, cudaStream_t stream) {
    return launch_overlapped(route_kernel<VPL, T>, dim3(cdiv(rows, ROUTE_WARPS)), dim3(32 * ROUTE_WARPS), stream,
                             static_cast<const T*>(logits), bias, ids, weights, rows, E, k, scoring, renorm, scale,
                             (vector_rows<VPL, T>(logits, logits, E) ? 1 : 0) | (E % VPL == 0 && aligned(bias, 16) ? 2 : 0));
}

template <int VPL, typename T>
cudaError_t launch_route_backward(const void* logits, const int32_t* ids, const float* dweights, void* dlogits, int rows,
                                  int E, int k, int scoring, int renorm, float scale, cudaStream_t stream) {
    return launch_overlapped(route_backward_kernel<VPL, T>, dim3(cdiv(rows, ROUTE_WARPS)), dim3(32 * ROUTE_WARPS), stream,
                             static_cast<const T*>(logits), ids, dweights, static_cast<T*>(dlogits), rows, E, k, scoring,
                             renorm, scale, vector_rows<VPL, T>(logits, dlogits, E) ? 1 : 0);
}

// Arguments that both directions share. `need` collects what must not be null.
dg_status check_route(int type, int T, int E, int k, int scoring) {
    if (T < 0 || E < 0 || k < 0) return DG_INVALID_ARG;
    if (type != DG_TYPE_BF16 && type != DG_TYPE_F32) return DG_INVALID_ARG;
    if (scoring != DG_SCORE_SOFTMAX && scoring != DG_SCORE_SIGMOID) return DG_INVALID_ARG;
    if (E > MAX_ROUTE_EXPERTS || k > MAX_ROUTE_K || k > E) return DG_UNSUPPORTED_SHAPE;
    return DG_OK;
}

#define DG_ROUTE_VPL(CALL)                                    \
    if (E <= 32) return CALL(1);                              \
    if (E <= 64) return CALL(2);                              \
    if (E <= 128) return CALL(4);                             \
    if (E <= 256) return CALL(8);                             \
    if (E <= 512) return CALL(16);                            \
    return CALL(32);

template <typename T>
cudaError_t route_any(const void* logits, const float* bias, int32_t* ids, float* weights, int rows, int E, int k,
                      int scoring, int renorm, float scale, cudaStream_t stream) {
#define DG_CALL(V) (launch_route<V, T>(logits, bias, ids, weights, rows, E, k, scoring, renorm, scale, stream))
    DG_ROUTE_VPL(DG_CALL)
#undef DG_CALL
}

template <typename T>
cudaError_t route_backward_any(const void* logits, const int32_t* ids, const float* dweights, void* dlogits, int rows,
                               int E, int k, int scoring, int renorm, float scale, cudaStream_t stream) {
#define DG_CALL(V) (launch_route_backward<V, T>(logits, ids, dweights, dlogits, rows, E, k, scoring, renorm, scale, stream))
    DG_ROUTE_VPL(DG_CALL)
#undef DG_CALL
}
#undef DG_ROUTE_VPL

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_moe_route(const void* logits, int logits_type, const float* bias, int32_t* ids, float* weights, int T, int E,
                       int k, int scoring, int renormalize, float scale, cudaStream_t stream) {
    dg_status st = check_route(logits_type, T, E, k, scoring);
    if (st != DG_OK) return st;
    if (bias && scoring != DG_SCORE_SIGMOID) return DG_INVALID_ARG;
    if (T == 0 || k == 0) return DG_OK;
    if (!logits || !ids || !weights) return DG_INVALID_ARG;
    if (!aligned(logits, logits_type == DG_TYPE_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return DG_MISALIGNED;
    DeviceInfo dev;
    st = device_info(&dev);
    if (st != DG_OK) return st;
    const int renorm = renormalize ? 1 : 0;
    const cudaError_t e = logits_type == DG_TYPE_BF16
        ? route_any<__nv_bfloat16>(logits, bias, ids, weights, T, E, k, scoring, renorm, scale, stream)
        : route_any<float>(logits, bias, ids, weights, T, E, k, scoring, renorm, scale, stream);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

dg_status dg_moe_route_backward(const void* logits, int logits_type, const int32_t* ids, const float* dweights,
                                void* dlogits, int T, int E, int k, int scoring, int renormalize, float scale,
                                cudaStream_t stream) {
    dg_status st = check_route(logits_type, T, E, k, scoring);
    if (st != DG_OK) return st;
    if (T == 0 || E == 0) return DG_OK;
    if (!logits || !dlogits || (k > 0 && (!ids || !dweights))) return DG_INVALID_ARG;
    const int a = logits_type == DG_TYPE_BF16 ? 2 : 4;
    if (!aligned(logits, a) || !aligned(dlogits, a) || !aligned(ids, 4) || !aligned(dweights, 4)) return DG_MISALIGNED;
    DeviceInfo dev;
    st = device_info(&dev);
    if (st != DG_OK) return st;
    const int renorm = renormalize ? 1 : 0;
    const cudaError_t e = logits_type == DG_TYPE_BF16
        ? route_backward_any<__nv_bfloat16>(logits, ids, dweights, dlogits, T, E, k, scoring, renorm, scale, stream)
        : route_backward_any<float>(logits, ids, dweights, dlogits, T, E, k, scoring, renorm, scale, stream);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

}  // extern "C"
