// A 128 x 128 tile of FP32 values in registers, quantised along its rows and along its columns: one scaling block in either
// direction. A warp has R whole rows and a lane 4 columns of each, v[row][pair of columns]: a row's largest magnitude is one
// reduction of the warp, and a column's needs no exchange inside a warp, only one over the 128 / R warps through shared memory.
#pragma once

#include <cstdint>

#include "dg_ptx.cuh"
#include "dg_quant.cuh"

namespace dg {

constexpr int TILE = 128;

// The largest magnitude over a warp, in all lanes; NaN wins.
__device__ __forceinline__ float warp_abs_max(float v) {
    float d;
    asm("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}

// Codes along the rows of two tiles' values at once: q points at the lane's first value of each, rows `pitch` apart, sf at the
// warp's first row's scale, `scales` apart; `valid` of the R rows exist. Lane l makes the scale of row l / (16 / R) of the first
// tile, or, from lane 16 on, of the second, and hands round its reciprocal.
template <int R>
__device__ __forceinline__ void tile_rows2(const float2 (&v)[R][2], const float2 (&u)[R][2], uint8_t* qv, uint8_t* qu, size_t pitch, float* sfv, float* sfu,
                                           size_t scales, int valid, int lane) {
    constexpr int SHARE = 16 / R;
    float a[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        a[i] = warp_abs_max(abs_max(abs_max(v[i][0].x, v[i][0].y, v[i][1].x), v[i][1].y));
        a[R + i] = warp_abs_max(abs_max(abs_max(u[i][0].x, u[i][0].y, u[i][1].x), u[i][1].y));
    }
#pragma unroll
    for (int half = R; half >= 1; half /= 2) {        // a[lane / SHARE], by the bits of the lane
        const bool up = (lane & half * SHARE) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) a[i] = up ? a[half + i] : a[i];
    }
    const float most = a[0];
    const BlockScale mine = block_scale(abs_bits(most));
    const int row = lane / SHARE & (R - 1);
    if (lane % SHARE == 0 && row < valid) (lane < 16 ? sfv : sfu)[row * scales] = mine.s;
#pragma unroll
    for (int i = 0; i < R; ++i, qv += pitch, qu += pitch) {
        const float rv = __shfl_sync(0xffffffffu, mine.r, i * SHARE), ru = __shfl_sync(0xffffffffu, mine.r, 16 + i * SHARE);
        const uint32_t a = quantise4_by(v[i][0], v[i][1], rv), b = quantise4_by(u[i][0], u[i][1], ru);
        if (i < valid) {
            *reinterpret_cast<uint32_t*>(qv) = a;
            *reinterpret_cast<uint32_t*>(qu) = b;
        }
    }
}

// Codes along the columns, in three steps with a barrier of the CTA behind each: every warp's maxima, the columns' scales,
// the codes, which then leave as the rows of the transpose. EXACT: by the rounded quotient, else by the reciprocal.
template <int R, bool EXACT>
struct TileColumns {
    static constexpr int WARPS = TILE / R;
    __align__(16) float amax[WARPS][TILE];
    __align__(16) float divisor[TILE];            // negative
    __align__(16) float reciprocal[TILE];
    __align__(16) uint32_t codes[TILE * TILE / 4];

    __device__ __forceinline__ void maxima(const float2 (&v)[R][2], int warp, int lane) {
        float a[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const auto at = [&](int i) { return c & 1 ? v[i][c >> 1].y : v[i][c >> 1].x; };
            a[c] = abs_max(at(0), at(1), at(2));
#pragma unroll
            for (int i = 3; i + 1 < R; i += 2) a[c] = abs_max(a[c], at(i), at(i + 1));
            if (R % 2 == 0) a[c] = abs_max(a[c], at(R - 1));
        }
        *reinterpret_cast<float4*>(&amax[warp][lane * 4]) = make_float4(a[0], a[1], a[2], a[3]);
    }

    // by 128 threads, one a column; sft: the column's scale
    __device__ __forceinline__ void scale(int c, float* sft) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WARPS; w += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = abs_max(a[j], amax[w + j][c], amax[w + j + 4][c]);
        const BlockScale k = block_scale(abs_bits(abs_max(abs_max(a[0], a[1], a[2]), a[3])));
        divisor[c] = -k.d;
        reciprocal[c] = k.r;
        *sft = k.s;
    }

    // Rows 4w .. 4w + 3 of column c are word w of its 32, at w ^ (R / 4) ((c / 4) % WARPS): neither these stores nor the loads
    // below meet in a bank.
    __device__ __forceinline__ void quantise(const float2 (&v)[R][2], int warp, int lane) {
        const float4 d = *reinterpret_cast<const float4*>(&divisor[lane * 4]), r = *reinterpret_cast<const float4*>(&reciprocal[lane * 4]);
        const int slot = warp ^ (lane & (WARPS - 1));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float2 nd = x ? make_float2(d.z, d.w) : make_float2(d.x, d.y), rr = x ? make_float2(r.z, r.w) : make_float2(r.x, r.y);
            uint32_t lo[R / 4], hi[R / 4];
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                float2 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = EXACT ? quotient2(v[i + j][x], nd, rr) : __fmul2_rn(v[i + j][x], rr);
                lo[i / 4] = pack_e4m3x2(w[0].x, w[1].x) | (pack_e4m3x2(w[2].x, w[3].x) << 16);
                hi[i / 4] = pack_e4m3x2(w[0].y, w[1].y) | (pack_e4m3x2(w[2].y, w[3].y) << 16);
            }
            uint32_t* dst = codes + (lane * 4 + 2 * x) * 32 + slot * (R / 4);
            if constexpr (R == 8) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(lo[0], lo[1]);
                *reinterpret_cast<uint2*>(dst + 32) = make_uint2(hi[0], hi[1]);
            } else {
                dst[0] = lo[0];
                dst[32] = hi[0];
            }
        }
    }

    // 128 bytes a column, R = 8: 16 lanes, R = 4: the warp; qt points at the tile's first column's codes, columns `pitch` apart.
    __device__ __forceinline__ void store(uint8_t* qt, size_t pitch, int warp, int lane) const {
        if constexpr (R == 8) {
            const int l16 = lane & 15, c0 = warp * 2 + (lane >> 4);
            uint8_t* dst = qt + static_cast<size_t>(c0) * pitch + l16 * 8;
            const uint32_t* src = codes + c0 * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i, dst += 32 * pitch)        // ((c >> 2) & 15 = c0 >> 2 ^ 8 (i & 1) for c = c0 + 32 i)
                *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src + i * 1024 + 2 * (l16 ^ (c0 >> 2) ^ (8 * (i & 1))));
        } else {
            uint8_t* dst = qt + static_cast<size_t>(warp) * pitch + lane * 4;
            const uint32_t* src = codes + warp * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i, dst += 32 * pitch)        // (c >> 2 = warp >> 2 ^ 8 i for c = warp + 32 i)
                *reinterpret_cast<uint32_t*>(dst) = src[i * 1024 + (lane ^ (warp >> 2) ^ (8 * i))];
        }
    }
};

// The tiles that a CTA takes: every gridDim.x-th, along the rows of tiles first, so that what runs at the same time reads whole
// rows. The steps are worked out once: a division for each tile would be a tenth of its instructions.
struct TileWalk {
    int m, n, step_m, step_n, m_tiles, n_tiles;
    __device__ __forceinline__ TileWalk(int m_tiles, int n_tiles) : m_tiles(m_tiles), n_tiles(n_tiles) {
        m = static_cast<int>(blockIdx.x) / n_tiles;
        n = static_cast<int>(blockIdx.x) - m * n_tiles;
        step_m = static_cast<int>(gridDim.x) / n_tiles;
        step_n = static_cast<int>(gridDim.x) - step_m * n_tiles;
    }
    __device__ __forceinline__ bool more() const { return m < m_tiles; }
    __device__ __forceinline__ void next() {
        m += step_m;
        n += step_n;
        if (n >= n_tiles) {
            n -= n_tiles;
            ++m;
        }
    }
};

}  // namespace dg
