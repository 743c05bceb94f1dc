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

// The same for two values in packed arithmetic; `nd` are the divisors' negatives.
__device__ __forceinline__ float2 quotient2(float2 v, float2 nd, float2 r) {
    const float2 q = __fmul2_rn(v, r);
    return __ffma2_rn(__ffma2_rn(q, nd, v), r, q);
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
__device__ __forceinline__ uint32_t quantise4(float2 a, float2 b, const BlockScale& k) {
    const float2 nd = make_float2(-k.d, -k.d), r = make_float2(k.r, k.r);
    a = quotient2(a, nd, r);
    b = quotient2(b, nd, r);
    return pack_e4m3x2(a.x, a.y) | (pack_e4m3x2(b.x, b.y) << 16);
}
__device__ __forceinline__ uint32_t quantise4(float a, float b, float c, float d, const BlockScale& k) {
    return quantise4(make_float2(a, b), make_float2(c, d), k);
}

// The largest of two or three magnitudes; NaN wins. (Of two, the result's sign is of no meaning.)
__device__ __forceinline__ float abs_max(float a, float b) {
    float d;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float abs_max(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The hardware's base-2 exponential and reciprocal, good to an ulp or two of FP32.
__device__ __forceinline__ float exp2_approx(float t) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return e;
}

__device__ __forceinline__ float reciprocal_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// -1 / (1 + e) for two values: the approximation r and one Newton step, whose rest 1 + r (1 + e) is taken as
// (1 + r) + r e, so that the rounding of 1 + e does not stay. (Negative, because a negation is an instruction here.)
__device__ __forceinline__ float2 minus_one_over_one_plus2(float2 e) {
    const float2 one = make_float2(1.f, 1.f), minus = make_float2(-1.f, -1.f), s = __ffma2_rn(e, minus, minus);
    const float2 r = make_float2(reciprocal_approx(s.x), reciprocal_approx(s.y));
    return __ffma2_rn(__ffma2_rn(r, e, __fadd2_rn(r, one)), r, r);
}

constexpr float LOG2_E = 1.4426950408889634f;
constexpr float LOG2_E_REST = 1.925963e-8f;       // log2(e) - float(log2(e))

// sqrt(2 / pi) and the cubic coefficient of the tanh form of GELU, z (1 + tanh(y)) / 2 with
// y = GELU_A (z + GELU_B z^3); (1 + tanh(y)) / 2 = sigmoid(2 y).
constexpr float GELU_A = 0.7978845608028654f;
constexpr float GELU_B = 0.044715f;

// max(v, floor), NaN staying NaN
__device__ __forceinline__ float at_least(float v, float floor) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(v), "f"(floor));
    return d;
}

// ... and min(v, ceiling)
__device__ __forceinline__ float at_most(float v, float ceiling) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(v), "f"(ceiling));
    return d;
}

// GELU, z Phi(z), by the normal distribution's upper tail: 1 - Phi(m) = P(t) exp(-m^2 / 2), t = 1 / (1 + 0.4 m),
// for 0 <= m <= GELU_END; beyond it the tail is 0 to FP32. P was fitted to that quotient for the smallest largest
// relative error, which is 3.4e-7 in FP32 arithmetic (the form is Hastings' for the error function, whose published
// coefficients have 1.5e-7 of 1, not of the tail). The two reciprocals of a pair are one.
constexpr float GELU_END = 14.f;
__device__ __forceinline__ float2 upper_tail2(float2 m) {
    const float2 u = __ffma2_rn(m, make_float2(0.4f, 0.4f), make_float2(1.f, 1.f));
    const float r = reciprocal_approx(u.x * u.y);
    const float2 t = make_float2(r * u.y, r * u.x);
    constexpr float P[9] = {-1.1998804438917432e-05f, 0.15990442037582397f, 0.15578454732894897f, 0.15842628479003906f, -0.012412778101861477f,
                            0.2510190010070801f, -0.37372907996177673f, 0.20062635838985443f, -0.039606764912605286f};
    float2 s = make_float2(P[8], P[8]);
#pragma unroll
    for (int i = 7; i >= 0; --i) s = __ffma2_rn(s, t, make_float2(P[i], P[i]));
    return s;
}

// The same tail for the slope, which needs it right to a rounding of 1 where the value, m times it, does not: the
// polynomial is in w = 1 - t = 0.4 m t, which is small where the tail is near 1/2, so that what t is off does not count
// there (largest error of Phi 8e-8 against 2.3e-7, for two more products; far out the relative error is 4e-6).
__device__ __forceinline__ float2 upper_tail_slope2(float2 m) {
    const float2 a = __fmul2_rn(m, make_float2(0.4f, 0.4f)), u = __fadd2_rn(a, make_float2(1.f, 1.f));
    const float r = reciprocal_approx(u.x * u.y);
    const float2 w = __fmul2_rn(a, __fmul2_rn(make_float2(r, r), make_float2(u.y, u.x)));
    constexpr float P[9] = {0.5f, -0.9973523616790771f, 0.5650054216384888f, 0.05166908726096153f, -0.1137925535440445f,
                            -0.0038454888854175806f, -0.07830164581537247f, 0.11620645970106125f, -0.03960096091032028f};
    float2 s = make_float2(P[8], P[8]);
#pragma unroll
    for (int i = 7; i >= 0; --i) s = __ffma2_rn(s, w, make_float2(P[i], P[i]));
    return s;
}

// below zero g, from zero on 1 - g; NaN stays
__device__ __forceinline__ float slope_of(float z, float g) { return z < 0.f ? g : (z >= 0.f ? 1.f - g : z); }

// The slopes of an activation at two BF16 pre-activations, in packed arithmetic where it has a form for that.
//
// SILU: p (1 + z (1 - p)) with p = 1 / (1 + e), e = exp(-z), and 1 - p = e p, which does not cancel where p is near
// 1. z has eight significant bits, so its product with the upper 16 bits of log2(e) is exact and the rest goes
// in as a factor: the exponential's error is that of the base-2 one alone. It is held under 2^110 to keep
// everything finite; the slopes beyond that are under 1e-31.
//
// A slope that is off by a last bit moves some quotient of dZ across a midpoint between two codes, so these are as
// good as FP32 operations that round once each make them: over every BF16 pre-activation within 30 the largest error is
// 1.4e-7 (SILU) and 1.2e-7 (both GELUs), and of 134 M codes 336, 372 and 359 (SILU, GELU_TANH, GELU) differ from the
// definition in 64 bits, where the definition in FP32 has 318, 623 and 389. Without the Newton steps and with the tail
// of act_value2 the errors are 1.6e-7 to 2.0e-7, and 4096 x 7168 takes 37.9, 44.4 and 45.7 us for 39.3, 47.6 and 46.7.
template <int ACT>
__device__ __forceinline__ float2 act_slope2(float2 z) {
    const float2 one = make_float2(1.f, 1.f), minus = make_float2(-1.f, -1.f);
    if (ACT == DG_ACT_SILU) {
        constexpr float HI = 1.44268798828125f, LO = 7.0526075e-6f * 0.6931471805599453f;   // log2(e), 16 bits; the rest, times ln 2
        z = make_float2(at_least(z.x, -100.f), at_least(z.y, -100.f));       // (0 to FP32 below)
        const float2 t = __fmul2_rn(z, make_float2(-HI, -HI));
        float2 e = make_float2(exp2_approx(fminf(t.x, 110.f)), exp2_approx(fminf(t.y, 110.f)));
        e = __ffma2_rn(e, __fmul2_rn(z, make_float2(-LO, -LO)), e);
        const float2 p = minus_one_over_one_plus2(e);                    // (negative)
        return __fmul2_rn(p, __ffma2_rn(__fmul2_rn(z, e), p, minus));
    }
    if (ACT == DG_ACT_GELU_TANH) {
        // p + z p (1 - p) y', with y = 2 a z (1 + b z^2), p its sigmoid and 1 - p = e p; beyond 16 that is 0 or 1 to FP32
        z = make_float2(at_most(at_least(z.x, -16.f), 16.f), at_most(at_least(z.y, -16.f), 16.f));
        const float2 z2 = __fmul2_rn(z, z);
        const float2 y = __fmul2_rn(z, __ffma2_rn(z2, make_float2(2.f * GELU_A * GELU_B, 2.f * GELU_A * GELU_B), make_float2(2.f * GELU_A, 2.f * GELU_A)));
        const float2 dy = __ffma2_rn(z2, make_float2(6.f * GELU_A * GELU_B, 6.f * GELU_A * GELU_B), make_float2(2.f * GELU_A, 2.f * GELU_A));
        // the rounding of y log2(e), and what log2(e) has beyond FP32, go in as a factor too
        constexpr float LN2 = 0.6931471805599453f;
        const float2 l = make_float2(-LOG2_E, -LOG2_E), t = __fmul2_rn(y, l);
        float2 e = make_float2(exp2_approx(fminf(t.x, 126.f)), exp2_approx(fminf(t.y, 126.f)));
        const float2 low = __ffma2_rn(y, make_float2(-LOG2_E_REST, -LOG2_E_REST), __ffma2_rn(y, l, __fmul2_rn(t, minus)));
        e = __ffma2_rn(e, __fmul2_rn(low, make_float2(LN2, LN2)), e);
        const float2 p = minus_one_over_one_plus2(e);                    // (negative)
        return __ffma2_rn(__fmul2_rn(p, __fmul2_rn(e, p)), __fmul2_rn(z, dy), __fmul2_rn(p, minus));
    }
    if (ACT == DG_ACT_GELU) {
        // Phi(z) + z phi(z): with m = |z| that is g = (P(t) - m / sqrt(2 pi)) exp(-z^2 / 2) below zero, 1 - g above.
        // (z^2 is exact, and the rounding of its product with log2(e) / 2 counts only where g is small.)
        const float2 m = make_float2(fminf(fabsf(z.x), GELU_END), fminf(fabsf(z.y), GELU_END));
        const float2 x = __fmul2_rn(__fmul2_rn(m, m), make_float2(-0.5f * LOG2_E, -0.5f * LOG2_E));
        const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
        const float2 g = __fmul2_rn(e, __ffma2_rn(m, make_float2(-0.3989422804014327f, -0.3989422804014327f), upper_tail_slope2(m)));
        return make_float2(slope_of(z.x, g.x), slope_of(z.y, g.y));
    }
    if (ACT == DG_ACT_RELU) return make_float2(z.x > 0.f ? 1.f : 0.f, z.y > 0.f ? 1.f : 0.f);
    return one;
}

// Two products z sigmoid(y) with one reciprocal: with a = 1 + exp(-y0) and b = 1 + exp(-y1), 1 / a = b / (a b).
// The special-function unit takes eight cycles a warp for each exponential and reciprocal and is what bounds
// an epilogue of these, so three per pair instead of four count. The exponentials are held under 2^63 (a NaN
// counts as that) to keep a b finite, so that neither value of the pair can spoil the other; z is held at the
// value where its sigmoid is 2^-63, below which the product is under 5e-18.
//
// The rounding of y log2(e) stays, and the reciprocal is the approximate one: the product is within 5 ulp of FP32 for
// |y| up to 4 (0.8 rms, where FP32 operations one by one have 0.5) and within 2^-18 of itself at y = -40, where it is under
// 2e-16. It is rounded to the eight bits of a BF16 or, times another number, to the four of a code next, and the
// outputs' errors against 64 bits are those of FP32 operations to two digits (SILU and GELU_TANH, products and layers).
__device__ __forceinline__ float2 times_sigmoid2(float2 z, float2 y) {
    const float2 t = __fmul2_rn(y, make_float2(-LOG2_E, -LOG2_E));
    const float2 a = __fadd2_rn(make_float2(exp2_approx(fminf(t.x, 63.f)), exp2_approx(fminf(t.y, 63.f))), make_float2(1.f, 1.f));
    const float r = reciprocal_approx(a.x * a.y);
    return __fmul2_rn(make_float2(at_least(z.x, -43.668f), at_least(z.y, -43.668f)), make_float2(r * a.y, r * a.x));
}

template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 z) {
    if (ACT == DG_ACT_RELU) return make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);     // NaN stays
    if (ACT == DG_ACT_GELU) {
        const float2 m = make_float2(fminf(fabsf(z.x), GELU_END), fminf(fabsf(z.y), GELU_END));
        const float2 x = __fmul2_rn(__fmul2_rn(m, m), make_float2(-0.5f * LOG2_E, -0.5f * LOG2_E));
        const float2 tail = __fmul2_rn(upper_tail2(m), make_float2(exp2_approx(x.x), exp2_approx(x.y)));
        return __ffma2_rn(__fmul2_rn(m, make_float2(-1.f, -1.f)), tail, make_float2(at_least(z.x, 0.f), at_least(z.y, 0.f)));
    }
    if (ACT == DG_ACT_GELU_TANH) {
        const float2 c = __ffma2_rn(__fmul2_rn(z, z), make_float2(2.f * GELU_A * GELU_B, 2.f * GELU_A * GELU_B), make_float2(2.f * GELU_A, 2.f * GELU_A));
        return times_sigmoid2(z, __fmul2_rn(z, c));
    }
    if (ACT == DG_ACT_SILU) return times_sigmoid2(z, z);
    return z;
}

template <int ACT, int N>
__device__ __forceinline__ void act_pairs(float (&v)[N]) {
    static_assert(N % 2 == 0, "pairs");
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 a = act_value2<ACT>(make_float2(v[i], v[i + 1]));
        v[i] = a.x;
        v[i + 1] = a.y;
    }
}

// act over an array in registers, with one branch on the (uniform) choice around the whole loop.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    switch (act) {
        case DG_ACT_RELU: act_pairs<DG_ACT_RELU>(v); break;
        case DG_ACT_GELU: act_pairs<DG_ACT_GELU>(v); break;
        case DG_ACT_GELU_TANH: act_pairs<DG_ACT_GELU_TANH>(v); break;
        case DG_ACT_SILU: act_pairs<DG_ACT_SILU>(v); break;
        default: break;
    }
}

}  // namespace dg
