// Device helpers shared by the operators around the products: the 1x128 quantisation to e4m3 and the
// activations with their slopes.
//
// Quantisation (the same recipe as inputs.quantize_1x128): s = max(amax, 1e-4) / 448 over a block of 128
// values, code = e4m3(v / s), both quotients rounded to FP32 and the code to nearest, ties to even,
// saturating. A NaN in a block makes its scale and all its codes NaN, an infinity makes the scale
// infinite (finite values become 0, infinities NaN), as the recipe itself gives.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "dg.h"

namespace dg {

constexpr float E4M3_TOP = 448.f;
constexpr float AMAX_FLOOR = 1e-4f;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// 1 / s to nearest: the hardware's approximation and one Newton step.
__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return fmaf(fmaf(-s, r, 1.f), r, r);
}

// v / s correctly rounded, with r = 1 / s to nearest: q = v r is within an ulp of the quotient and
// q + (v - q s) r, each step fused, rounds to it (Markstein's division). Three instructions where the general
// division takes a dozen and a call, which counts here: the quantisation is bound by instruction issue.
__device__ __forceinline__ float quotient(float v, float s, float r) {
    const float q = v * r;
    return fmaf(fmaf(-q, s, v), r, q);
}

// The scale of a block, and what its values are divided by. The largest magnitude comes as the bits of |v|:
// as unsigned integers these order like the magnitudes, with the infinity above every finite value and NaN
// above that, so integer maxima carry NaN through (fmaxf would drop it). For a scale that is not finite the
// divisor's pair is (0, 0) or (0, NaN), for which quotient() gives what the division would: 0 for finite
// values over an infinite scale, NaN for infinite ones and wherever the scale is NaN.
struct BlockScale {
    float s;               // the scale
    float d, r;            // divisor and its reciprocal for quotient()
};

__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits);
    const bool finite = amax_bits < 0x7f800000u;
    BlockScale b;
    b.s = finite ? quotient(a < AMAX_FLOOR ? AMAX_FLOOR : a, E4M3_TOP, 1.f / E4M3_TOP) : a;
    b.d = finite ? b.s : 0.f;
    b.r = finite ? reciprocal(b.s) : (amax_bits == 0x7f800000u ? 0.f : a);
    return b;
}

// Two values to e4m3 codes, `lo` in the low byte (to nearest even, saturating, NaN kept).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Four values of a block to codes, in order from the lowest byte.
__device__ __forceinline__ uint32_t quantise4(float a, float b, float c, float d, const BlockScale& k) {
    return pack_e4m3x2(quotient(a, k.d, k.r), quotient(b, k.d, k.r)) |
           (pack_e4m3x2(quotient(c, k.d, k.r), quotient(d, k.d, k.r)) << 16);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 1 / (1 + exp(-z)) with the fast exponential and reciprocal: both are good to a few ulp of FP32, and
// every use ends in BF16 or e4m3. Saturates to 0 and 1 without NaN; NaN stays.
__device__ __forceinline__ float fast_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// sqrt(2 / pi) and the cubic coefficient of the tanh form of GELU, z (1 + tanh(y)) / 2 with
// y = GELU_A (z + GELU_B z^3); (1 + tanh(y)) / 2 = sigmoid(2 y).
constexpr float GELU_A = 0.7978845608028654f;
constexpr float GELU_B = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == DG_ACT_RELU) return z < 0.f ? 0.f : z;                     // NaN stays
    if (ACT == DG_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    if (ACT == DG_ACT_GELU_TANH) return z * fast_sigmoid(2.f * GELU_A * (z + GELU_B * z * z * z));
    // (the quotient form keeps what the definition gives at the infinities)
    if (ACT == DG_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if (ACT == DG_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (ACT == DG_ACT_GELU)
        return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * 0.3989422804014327f * __expf(-0.5f * z * z);
    if (ACT == DG_ACT_GELU_TANH) {
        const float p = fast_sigmoid(2.f * GELU_A * (z + GELU_B * z * z * z));
        return p + 2.f * GELU_A * z * p * (1.f - p) * (1.f + 3.f * GELU_B * z * z);
    }
    if (ACT == DG_ACT_SILU) {
        const float p = fast_sigmoid(z);
        return p * (1.f + z * (1.f - p));
    }
    return 1.f;
}

// act over an array in registers, with one branch on the (uniform) choice around the whole loop.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    switch (act) {
        case DG_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<DG_ACT_RELU>(v[i]);
            break;
        case DG_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<DG_ACT_GELU>(v[i]);
            break;
        case DG_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<DG_ACT_GELU_TANH>(v[i]);
            break;
        case DG_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<DG_ACT_SILU>(v[i]);
            break;
        default: break;
    }
}

}  // namespace dg
