// The router around the experts' products: top-k selection with its weights (dg_moe_route) and their
// gradient (dg_moe_route_backward). The general way is a row a warp; up to 32 experts take an expert a lane, and
// many rows of up to 16 four rows a warp (below).
//
// Selection. A lane holds VPL experts of the row: consecutive ones where the rows can be read in vectors, else
// every 32nd, so that a load or store of the warp still covers one piece of the row (E = 510, FP32, 25052 rows:
// the gradient took 52.8 us with consecutive experts and single loads, 13.0 so). k whole-warp maxima over the
// lanes' best values give a bound below which no selected value can lie (k lanes hold one at least as large); the
// few values at or above it -- k and a handful in practice -- are compacted through shared memory, one a lane, and
// each counts those that precede it (larger, or equal with a lower expert), which is its place in the order. More
// than 32 candidates (many equal values) take k rounds of find-and-remove instead.
//
// With a bias the selection values are sums of a sigmoid, and which of two close ones is larger has to be
// right: they are defined with an accurate exponential and a rounded reciprocal. Only the candidates pay for
// that: the bound is found with the hardware's approximations, lowered by more than they can be off.
//
// What bounds it is instruction issue: 32749 rows of 256 BF16 logits are 18.9 MB, 2.8 us of HBM, and 456
// instructions a row with sigmoid scores, a bias and k = 8, which at 83% of the issue slots take 14.4 us.
// Few rows are bound by one row's latency (1.7 us in a CUDA graph).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
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
                    const uint4 u = ld_input(reinterpret_cast<const uint4*>(row + e0) + c);
                    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                } else {
                    const uint2 u = ld_input(reinterpret_cast<const uint2*>(row + e0) + c);
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
                if (e0 < E) u = ld_input(reinterpret_cast<const float4*>(bias + e0) + c);
                v[4 * c] = u.x; v[4 * c + 1] = u.y; v[4 * c + 2] = u.z; v[4 * c + 3] = u.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = e0 + i * step < E ? ld_input(bias + e0 + i * step) : 0.f;
}

// v = the fast sigmoid of v + b; -inf where v is that or NaN.
template <int VPL>
__device__ __forceinline__ void approximate_sums(float (&v)[VPL], const float (&b)[VPL]) {
#pragma unroll
    for (int i = 0; i < VPL; i += 2) {
        const float2 y = __fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(-LOG2_E, -LOG2_E));
        const float2 d = __fadd2_rn(make_float2(exp2_approx(y.x), exp2_approx(y.y)), make_float2(1.f, 1.f));
        const float2 s = __fadd2_rn(make_float2(reciprocal_approx(d.x), reciprocal_approx(d.y)), make_float2(b[i], b[i + 1]));
        v[i] = v[i] > -INFINITY ? s.x : -INFINITY;
        v[i + 1] = v[i + 1] > -INFINITY ? s.y : -INFINITY;
    }
}

// +inf counts as the largest finite value, so that no score is a quotient of infinities
__device__ __forceinline__ float finite_top(float l) { return fminf(l, FLT_MAX); }

template <int VPL, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, VPL <= 8 ? 8 : (VPL == 16 ? 5 : 3))
route_kernel(const T* logits, const float* bias, int32_t* ids,
             float* weights, int rows, int E, int k, int sigmoid_scores, int renorm, float scale, int vec) {
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
        approximate_sums<VPL>(v, b);
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
            for (int i = 0; i < VPL; ++i) sum += v[i] > -INFINITY ? expf(v[i] - top) : 0.f;
            total = warp_sum(sum);
        }
    }

    // the bound: the k-th whole-warp maximum of the lanes' best values
    float h = head, bound = -INFINITY;
#pragma unroll 4
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
    float value = -INFINITY;         // its logit, or (sigmoid) its score
    const int picked = min(found, k);
    if (found <= 32) {
        // the candidates one a lane, which reads its logit again (it knows where from only now)
        int at = before;
        for (uint32_t m = mask; m != 0; m &= m - 1) s_cand[warp][at++] = e0 + (__ffs(m) - 1) * step;
        __syncwarp();
        float me = -INFINITY;
        if (lane < found) {
            expert = s_cand[warp][lane];
            me = value = finite_top(to_f32(row[expert]));
            if (sigmoid_scores) value = sigmoid(value);
            if (bias != nullptr) me = value + ld_input(bias + expert);
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
                    if (l > -INFINITY) exact = sigmoid(finite_top(l)) + ld_input(bias + e);
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
        if (place >= 0) {
            value = finite_top(to_f32(row[expert]));
            if (sigmoid_scores) value = sigmoid(value);
        }
    }

    float score = 0.f;
    if (place >= 0) score = sigmoid_scores ? value : expf(value - top);
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
route_backward_kernel(const T* logits, const int32_t* ids, const float* dweights,
                      T* dlogits, int rows, int E, int k, int sigmoid_scores, int renorm, float scale, int vec) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = static_cast<int>(blockIdx.x) * ROUTE_WARPS + warp;
    grid_dependency_wait();
    grid_launch_dependents();
    if (t >= rows) return;
    const T* row = logits + static_cast<size_t>(t) * E;
    int e = lane < k ? ld_input(ids + static_cast<size_t>(t) * k + lane) : -1;
    const bool open = e >= 0 && e < E;
    const float dw = open ? ld_input(dweights + static_cast<size_t>(t) * k + lane) * scale : 0.f;
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
            out[i] = l[i] > -INFINITY ? expf(l[i] - top) : 0.f;
            sum += out[i];
        }
        sum = warp_sum(sum);
        const float inv = sum > 0.f ? __frcp_rn(sum) : 0.f;
        const float p = mine > -INFINITY ? expf(mine - top) * inv : 0.f;
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
            p = mine > -INFINITY ? expf(mine - top) : 0.f;
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

// ---- few experts: four rows a warp
//
// With at most 16 experts most of a warp would hold nothing of its row. Here eight lanes hold a row, VPL consecutive
// experts each, and a warp works on four rows with the same instructions. (A row a lane was measured too: 5 us for
// 2048 rows as for 32768 with 16 experts, one warp's latency.)
constexpr int GROUP = 8;                           // lanes a row
constexpr int GROUP_ROWS = 32 / GROUP;             // rows a warp

__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = GROUP / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = GROUP / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// The lane's VPL logits of a row, from expert e0; -inf past its end, for NaN, and for a row that does not exist.
template <int VPL, typename T>
__device__ __forceinline__ void load_group(const T* row, int E, int e0, bool there, float (&l)[VPL]) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const float x = there && e0 + i < E ? to_f32(row[e0 + i]) : -INFINITY;
        l[i] = x > -INFINITY ? finite_top(x) : -INFINITY;
    }
}

template <int VPL, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
route_few_kernel(const T* logits, const float* bias, int32_t* ids,
                 float* weights, int rows, int E, int k, int sigmoid_scores, int renorm, float scale) {
    __shared__ float s_logit[ROUTE_WARPS][GROUP_ROWS][32];       // of the selected experts, in order
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane / GROUP, l8 = lane % GROUP;
    const int t = (static_cast<int>(blockIdx.x) * ROUTE_WARPS + warp) * GROUP_ROWS + g;
    grid_dependency_wait();
    grid_launch_dependents();
    if (t - g >= rows) return;
    const bool there = t < rows;
    const int e0 = l8 * VPL;
    float l[VPL], v[VPL];                          // logits, selection values
    load_group<VPL, T>(logits + static_cast<size_t>(t) * E, E, e0, there, l);
    float top = 0.f, sum = 0.f;
    if (!sigmoid_scores) {
        top = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) top = fmaxf(top, l[i]);
        top = group_max(top);
        if (!renorm) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum += l[i] > -INFINITY ? expf(l[i] - top) : 0.f;
            sum = group_sum(sum);
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        v[i] = bias != nullptr && l[i] > -INFINITY ? sigmoid(l[i]) + ld_input(bias + e0 + i) : l[i];
        if (!(v[i] > -INFINITY)) v[i] = -INFINITY;          // a NaN of the bias
    }

    const size_t out = static_cast<size_t>(t) * k;
    for (int j = 0; j < k; ++j) {
        float best = v[0], own = l[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < VPL; ++i)
            if (v[i] > best) { best = v[i]; own = l[i]; at = i; }
        const float most = group_max(best);        // (fmaxf drops NaN, which equals nothing either)
        // the lowest lane that holds it holds the lowest expert
        const unsigned equal = __ballot_sync(FULL, best == most) & (((1u << GROUP) - 1) << (g * GROUP));
        const bool open = most > -INFINITY;
        if (open ? lane == __ffs(equal) - 1 : l8 == 0) {
            s_logit[warp][g][j] = open ? own : -INFINITY;
            if (there) ids[out + j] = open ? e0 + at : -1;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i == at) v[i] = -INFINITY;
        }
    }
    __syncwarp();
    float score[32 / GROUP];
#pragma unroll
    for (int m = 0; m < 32 / GROUP; ++m) {
        score[m] = 0.f;
        if (m * GROUP + l8 < k) {
            const float x = s_logit[warp][g][m * GROUP + l8];
            if (x > -INFINITY) score[m] = sigmoid_scores ? sigmoid(x) : expf(x - top);
        }
    }
    if (renorm) sum = group_sum((score[0] + score[1]) + (score[2] + score[3]));
    const float inv = sigmoid_scores && !renorm ? 1.f : (sum > 0.f ? __frcp_rn(sum) : 0.f);
#pragma unroll
    for (int m = 0; m < 32 / GROUP; ++m)
        if (there && m * GROUP + l8 < k) weights[out + m * GROUP + l8] = score[m] * inv * scale;
}

// The gradient by expert: add = the weights' gradients of the slots that name it, times the scale, and `named` how
// many they are. With p the scores, r = p / sum(named p):
//   renormalised   r (add - named dot), dot = sum(r add), times 1 - p for the sigmoid
//   softmax        p (add - dot), dot = sum(p add)      sigmoid   p (1 - p) add
template <int VPL, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
route_few_backward_kernel(const T* logits, const int32_t* ids, const float* dweights,
                          T* dlogits, int rows, int E, int k, int sigmoid_scores, int renorm, float scale) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane / GROUP, l8 = lane % GROUP;
    const int t = (static_cast<int>(blockIdx.x) * ROUTE_WARPS + warp) * GROUP_ROWS + g;
    grid_dependency_wait();
    grid_launch_dependents();
    if (t - g >= rows) return;
    const bool there = t < rows;
    const int e0 = l8 * VPL;
    float l[VPL], add[VPL], named[VPL];
    load_group<VPL, T>(logits + static_cast<size_t>(t) * E, E, e0, there, l);
#pragma unroll
    for (int i = 0; i < VPL; ++i) add[i] = named[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += GROUP) {
        int e = -1;
        float dw = 0.f;
        if (there && j0 + l8 < k) {
            e = ld_input(ids + static_cast<size_t>(t) * k + j0 + l8);
            dw = ld_input(dweights + static_cast<size_t>(t) * k + j0 + l8) * scale;
        }
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
            const int oe = __shfl_sync(FULL, e, j, GROUP) - e0;
            const float od = __shfl_sync(FULL, dw, j, GROUP);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (oe == i) {
                    add[i] += od;
                    named[i] += 1.f;
                }
        }
    }
    // scores: of the named experts where they are renormalised, else of all
    float p[VPL], top = 0.f, sum = 0.f, dot = 0.f;
    if (!sigmoid_scores) {
        top = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (!renorm || named[i] > 0.f) top = fmaxf(top, l[i]);
        top = group_max(top);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool counts = l[i] > -INFINITY && (!renorm || named[i] > 0.f);
        p[i] = !counts ? 0.f : (sigmoid_scores ? sigmoid(l[i]) : expf(l[i] - top));
        sum = fmaf(renorm ? named[i] : 1.f, p[i], sum);
    }
    const bool quotient = renorm || !sigmoid_scores;
    if (quotient) sum = group_sum(sum);
    const float inv = !quotient ? 1.f : (sum > 0.f ? __frcp_rn(sum) : 0.f);
    float out[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        out[i] = p[i] * inv;
        dot = fmaf(out[i], add[i], dot);
    }
    if (quotient) dot = group_sum(dot);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (quotient) out[i] *= add[i] - (renorm ? named[i] : 1.f) * dot;
        else out[i] *= add[i];
        if (sigmoid_scores) out[i] *= 1.f - p[i];
        if (there && e0 + i < E) store_one(dlogits + static_cast<size_t>(t) * E + e0 + i, out[i]);
    }
}

// ---- an expert a lane
//
// Up to 32 experts: the k largest by k turns of find-and-remove, the lowest lane that holds the largest value
// winning, and every lane keeps the turn that it won (32 experts, k = 8: 1.7 us for 64 rows and 8.0 for 32768, where
// the general way takes 2.0 and 10.0). Warps take several rows, the next one's logits on their way.

// Whether a warp that has taken row t has another one, `stride` further on. (t + stride may be past 2^31.)
__host__ __device__ constexpr bool another_row(int t, int stride, int rows) { return rows - t > stride; }
static_assert(another_row(0, 8, 9) && !another_row(0, 8, 8) && !another_row(INT_MAX - 8, 32 * 1024, INT_MAX), "next row");

template <typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, 8)
route_lane_kernel(const T* logits, const float* bias, int32_t* ids,
                  float* weights, int rows, int E, int k, int sigmoid_scores, int renorm, float scale) {
    const int lane = threadIdx.x & 31, stride = static_cast<int>(gridDim.x) * ROUTE_WARPS;
    int t = static_cast<int>(blockIdx.x) * ROUTE_WARPS + static_cast<int>(threadIdx.x >> 5);
    grid_dependency_wait();
    grid_launch_dependents();
    if (t >= rows) return;
    const bool mine = lane < E;
    const float b = bias != nullptr && mine ? ld_input(bias + lane) : 0.f;
    float next = mine ? to_f32(logits[static_cast<size_t>(t) * E + lane]) : -INFINITY;
    for (bool more = true; more; t += more ? stride : 0) {
        const float l = next > -INFINITY ? finite_top(next) : -INFINITY;        // (NaN cannot be selected either)
        more = another_row(t, stride, rows);
        if (more && mine) next = to_f32(logits[static_cast<size_t>(t + stride) * E + lane]);
        float score = 0.f, total = 1.f, me = l;
        if (sigmoid_scores) {
            if (l > -INFINITY) score = sigmoid(l);
            if (bias != nullptr && l > -INFINITY) me = score + b;
        } else {
            const float top = warp_max(l);
            if (l > -INFINITY) score = expf(l - top);
            if (!renorm) total = warp_sum(score);
        }
        int place = -1;
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const float most = warp_max(me);
            if (lane == __ffs(__ballot_sync(FULL, me == most && me > -INFINITY)) - 1) {
                place = j;
                me = -INFINITY;
            }
        }
        const int picked = __popc(__ballot_sync(FULL, place >= 0));
        if (renorm) total = warp_sum(place >= 0 ? score : 0.f);
        const float w = total > 0.f ? score * __frcp_rn(total) : 0.f;
        const size_t out = static_cast<size_t>(t) * k;
        if (place >= 0) {
            ids[out + place] = lane;
            weights[out + place] = w * scale;
        }
        if (lane >= picked && lane < k) {
            ids[out + lane] = -1;
            weights[out + lane] = 0.f;
        }
    }
}

// The gradient by expert, as route_few_backward_kernel's.
template <typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, 8)
route_lane_backward_kernel(const T* logits, const int32_t* ids, const float* dweights,
                           T* dlogits, int rows, int E, int k, int sigmoid_scores, int renorm, float scale) {
    const int lane = threadIdx.x & 31, stride = static_cast<int>(gridDim.x) * ROUTE_WARPS;
    int t = static_cast<int>(blockIdx.x) * ROUTE_WARPS + static_cast<int>(threadIdx.x >> 5);
    grid_dependency_wait();
    grid_launch_dependents();
    if (t >= rows) return;
    const bool quotient = renorm || !sigmoid_scores;
    for (bool more = true; more; t += more ? stride : 0) {
        more = another_row(t, stride, rows);
        const float x = lane < E ? to_f32(logits[static_cast<size_t>(t) * E + lane]) : -INFINITY;
        int e = -1;
        float dw = 0.f;
        if (lane < k) {
            e = ld_input(ids + static_cast<size_t>(t) * k + lane);
            dw = ld_input(dweights + static_cast<size_t>(t) * k + lane) * scale;
        }
        const float l = x > -INFINITY ? finite_top(x) : -INFINITY;
        float add = 0.f, named = 0.f;
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const float od = __shfl_sync(FULL, dw, j);
            if (__shfl_sync(FULL, e, j) == lane) {
                add += od;
                named += 1.f;
            }
        }
        const bool counts = l > -INFINITY && (!renorm || named > 0.f);
        float p = 0.f, inv = 1.f;
        if (sigmoid_scores) {
            if (counts) p = sigmoid(l);
        } else {
            const float top = warp_max(counts ? l : -FLT_MAX);
            if (counts) p = expf(l - top);
        }
        const float times = renorm ? named : 1.f;
        if (quotient) {
            const float sum = warp_sum(times * p);
            inv = sum > 0.f ? __frcp_rn(sum) : 0.f;
        }
        float out = p * inv;
        if (quotient) out *= add - times * warp_sum(out * add);
        else out *= add;
        if (sigmoid_scores) out *= 1.f - p;
        if (lane < E) store_one(dlogits + static_cast<size_t>(t) * E + lane, out);
    }
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

// CTAs for rows that warps take several of: the eight that fit an SM, twice (32768 rows of 32 experts: 8.0 us, with
// half as many 8.4, with a row a warp 8.5).
int lane_grid(int rows) {
    DeviceInfo dev;
    const int most = device_info(&dev) == DG_OK ? 16 * dev.sms : 1 << 20;
    return std::min(cdiv(rows, ROUTE_WARPS), most);
}

template <typename T>
cudaError_t launch_route_lane(const void* logits, const float* bias, int32_t* ids, float* weights, int rows, int E, int k,
                              int scoring, int renorm, float scale, cudaStream_t stream) {
    return launch_overlapped(route_lane_kernel<T>, dim3(lane_grid(rows)), dim3(32 * ROUTE_WARPS), stream,
                             static_cast<const T*>(logits), bias, ids, weights, rows, E, k, scoring, renorm, scale);
}

template <typename T>
cudaError_t launch_route_lane_backward(const void* logits, const int32_t* ids, const float* dweights, void* dlogits, int rows,
                                       int E, int k, int scoring, int renorm, float scale, cudaStream_t stream) {
    return launch_overlapped(route_lane_backward_kernel<T>, dim3(lane_grid(rows)), dim3(32 * ROUTE_WARPS), stream,
                             static_cast<const T*>(logits), ids, dweights, static_cast<T*>(dlogits), rows, E, k, scoring,
                             renorm, scale);
}

template <int VPL, typename T>
cudaError_t launch_route_few(const void* logits, const float* bias, int32_t* ids, float* weights, int rows, int E, int k,
                             int scoring, int renorm, float scale, cudaStream_t stream) {
    return launch_overlapped(route_few_kernel<VPL, T>, dim3(cdiv(rows, GROUP_ROWS * ROUTE_WARPS)), dim3(32 * ROUTE_WARPS), stream,
                             static_cast<const T*>(logits), bias, ids, weights, rows, E, k, scoring, renorm, scale);
}

template <int VPL, typename T>
cudaError_t launch_route_few_backward(const void* logits, const int32_t* ids, const float* dweights, void* dlogits, int rows,
                                      int E, int k, int scoring, int renorm, float scale, cudaStream_t stream) {
    return launch_overlapped(route_few_backward_kernel<VPL, T>, dim3(cdiv(rows, GROUP_ROWS * ROUTE_WARPS)), dim3(32 * ROUTE_WARPS),
                             stream, static_cast<const T*>(logits), ids, dweights, static_cast<T*>(dlogits), rows, E, k, scoring,
                             renorm, scale);
}

// Four rows a warp for up to 16 experts from this many rows on, against an expert a lane (softmax, 8 experts, k = 2:
// 1.9 against 1.8 us for 4096 rows, 2.0 against 2.6 for 8192, 3.3 against 5.6 for 32768; 16 experts, k = 4: 2.4
// against 2.0, 2.4 against 2.8, 4.5 against 6.4). With more experts a row's k turns over eight lanes take longer
// than a whole warp's (32 experts, k = 8: 4.1 against 3.4 us for 8192; the gradient 10.2 against 7.2 for 32768).
constexpr int FEW_FROM = 6144;

// Arguments that both directions share. `need` collects what must not be null.
dg_status check_route(int type, int T, int E, int k, int scoring) {
    if (T < 0 || E < 0 || k < 0) return DG_INVALID_ARG;
    if (type != DG_TYPE_BF16 && type != DG_TYPE_F32) return DG_INVALID_ARG;
    if (scoring != DG_SCORE_SOFTMAX && scoring != DG_SCORE_SIGMOID) return DG_INVALID_ARG;
    if (E > MAX_ROUTE_EXPERTS || k > MAX_ROUTE_K || k > E) return DG_UNSUPPORTED_SHAPE;
    return DG_OK;
}

#define DG_ROUTE_VPL(CALL)                                    \
    if (E <= 64) return CALL(2);                              \
    if (E <= 128) return CALL(4);                             \
    if (E <= 256) return CALL(8);                             \
    if (E <= 512) return CALL(16);                            \
    return CALL(32);
#define DG_ROUTE_FEW(CALL)                                    \
    if (rows >= FEW_FROM) {                                   \
        if (E <= GROUP) return CALL(1);                       \
        if (E <= 2 * GROUP) return CALL(2);                   \
    }

template <typename T>
cudaError_t route_any(const void* logits, const float* bias, int32_t* ids, float* weights, int rows, int E, int k,
                      int scoring, int renorm, float scale, cudaStream_t stream) {
#define DG_FEW(V) (launch_route_few<V, T>(logits, bias, ids, weights, rows, E, k, scoring, renorm, scale, stream))
    DG_ROUTE_FEW(DG_FEW)
#undef DG_FEW
    if (E <= 32) return launch_route_lane<T>(logits, bias, ids, weights, rows, E, k, scoring, renorm, scale, stream);
#define DG_CALL(V) (launch_route<V, T>(logits, bias, ids, weights, rows, E, k, scoring, renorm, scale, stream))
    DG_ROUTE_VPL(DG_CALL)
#undef DG_CALL
}

template <typename T>
cudaError_t route_backward_any(const void* logits, const int32_t* ids, const float* dweights, void* dlogits, int rows,
                               int E, int k, int scoring, int renorm, float scale, cudaStream_t stream) {
#define DG_FEW(V) (launch_route_few_backward<V, T>(logits, ids, dweights, dlogits, rows, E, k, scoring, renorm, scale, stream))
    DG_ROUTE_FEW(DG_FEW)
#undef DG_FEW
    if (E <= 32) return launch_route_lane_backward<T>(logits, ids, dweights, dlogits, rows, E, k, scoring, renorm, scale, stream);
#define DG_CALL(V) (launch_route_backward<V, T>(logits, ids, dweights, dlogits, rows, E, k, scoring, renorm, scale, stream))
    DG_ROUTE_VPL(DG_CALL)
#undef DG_CALL
}
#undef DG_ROUTE_VPL
#undef DG_ROUTE_FEW

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
