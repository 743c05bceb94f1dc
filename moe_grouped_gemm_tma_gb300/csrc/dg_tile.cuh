// A 128 x 128 tile of FP32 values in the registers of 512 threads, quantised along its rows and along its columns: one
// scaling block in either direction. A thread holds 4 consecutive rows x 8 consecutive columns; a half warp has 4 whole
// rows, so that a row's largest magnitude is found over 16 lanes and a column's over the 16 warps.
#pragma once

#include <cstdint>

#include "dg_quant.cuh"

namespace dg {

constexpr int TILE = 128;
constexpr int TILE_THREADS = 512;
constexpr int TILE_WARPS = TILE_THREADS / 32;

struct TileShared {
    __align__(16) uint32_t codes[TILE * TILE / 4];
    __align__(16) float amax[TILE_WARPS][TILE];
    __align__(16) float divisor[TILE], reciprocal[TILE];    // (divisors negative)
};

// Where a thread is in its tile.
struct TileThread {
    int warp, half, l16, row, column;             // first of its rows and columns
    __device__ TileThread() {
        warp = threadIdx.x >> 5;
        half = (threadIdx.x >> 4) & 1;
        l16 = threadIdx.x & 15;
        row = warp * 8 + half * 4;
        column = l16 * 8;
    }
};

// Codes along the rows: q points at the thread's first value, rows `pitch` apart, sf at its first row's scale, `scales`
// apart; `valid` of its 4 rows exist.
__device__ __forceinline__ void tile_rows(const float2 (&v)[4][4], uint8_t* q, size_t pitch, float* sf, size_t scales, int valid, int l16) {
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = abs_max(abs_max(v[i][0].x, v[i][0].y, v[i][1].x), abs_max(v[i][1].y, v[i][2].x, v[i][2].y), abs_max(v[i][3].x, v[i][3].y));
    // over the 16 lanes, giving away rows on the way: lane l ends with that of row l / 4, and makes its scale
    const bool up8 = (l16 & 8) != 0, up4 = (l16 & 4) != 0;
    const float b0 = abs_max(up8 ? a[2] : a[0], __shfl_xor_sync(0xffffffffu, up8 ? a[0] : a[2], 8));
    const float b1 = abs_max(up8 ? a[3] : a[1], __shfl_xor_sync(0xffffffffu, up8 ? a[1] : a[3], 8));
    float most = abs_max(up4 ? b1 : b0, __shfl_xor_sync(0xffffffffu, up4 ? b0 : b1, 4));
    most = abs_max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    most = abs_max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    const BlockScale mine = block_scale(abs_bits(most));
    if ((l16 & 3) == 0 && (l16 >> 2) < valid) sf[static_cast<size_t>(l16 >> 2) * scales] = mine.s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        BlockScale k;
        k.d = __shfl_sync(0xffffffffu, mine.d, i * 4, 16);
        k.r = __shfl_sync(0xffffffffu, mine.r, i * 4, 16);
        const uint32_t w0 = quantise4(v[i][0], v[i][1], k), w1 = quantise4(v[i][2], v[i][3], k);
        if (i < valid) *reinterpret_cast<uint2*>(q + static_cast<size_t>(i) * pitch) = make_uint2(w0, w1);
    }
}

// Codes along the columns, by the whole CTA: qt points at the tile's first column's codes, columns `pitch` apart, sft at
// its scale, `scales` apart. `v` is 0 in rows that do not exist. The tile's shared memory may be used again at once.
__device__ __forceinline__ void tile_columns(const float2 (&v)[4][4], TileShared& s, uint8_t* qt, size_t pitch, float* sft, size_t scales,
                                             const TileThread& me) {
    float a[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a[2 * j] = abs_max(v[0][j].x, v[1][j].x, v[2][j].x);
        a[2 * j + 1] = abs_max(v[0][j].y, v[1][j].y, v[2][j].y);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        a[j] = abs_max(a[j], j & 1 ? v[3][j >> 1].y : v[3][j >> 1].x);
        a[j] = abs_max(a[j], __shfl_xor_sync(0xffffffffu, a[j], 16));
    }
    if (me.half == 0) {
        float4* dst = reinterpret_cast<float4*>(&s.amax[me.warp][me.column]);
        dst[0] = make_float4(a[0], a[1], a[2], a[3]);
        dst[1] = make_float4(a[4], a[5], a[6], a[7]);
    }
    __syncthreads();
    if (threadIdx.x < TILE) {
        const int c = threadIdx.x;
        float most = 0.f;
#pragma unroll
        for (int g = 0; g < TILE_WARPS; ++g) most = abs_max(most, s.amax[g][c]);
        const BlockScale k = block_scale(abs_bits(most));
        s.divisor[c] = -k.d;
        s.reciprocal[c] = k.r;
        sft[static_cast<size_t>(c) * scales] = k.s;
    }
    __syncthreads();
    // rows 4w .. 4w + 3 of column n in word w ^ 2 (n / 8) of its 32
    const int word = (me.warp * 2 + me.half) ^ (2 * me.l16);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const float4 d = *reinterpret_cast<const float4*>(&s.divisor[me.column + 2 * j]);
        const float4 r = *reinterpret_cast<const float4*>(&s.reciprocal[me.column + 2 * j]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float2 nd = x ? make_float2(d.z, d.w) : make_float2(d.x, d.y), rr = x ? make_float2(r.z, r.w) : make_float2(r.x, r.y);
            float2 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = quotient2(v[i][j + x], nd, rr);
            uint32_t* dst = s.codes + (me.column + 2 * (j + x)) * 32 + word;
            dst[0] = pack_e4m3x2(w[0].x, w[1].x) | (pack_e4m3x2(w[2].x, w[3].x) << 16);
            dst[32] = pack_e4m3x2(w[0].y, w[1].y) | (pack_e4m3x2(w[2].y, w[3].y) << 16);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = i * 32 + me.warp * 2 + me.half;
        const uint2 w = *reinterpret_cast<const uint2*>(s.codes + c * 32 + 2 * (me.l16 ^ (c >> 3)));
        *reinterpret_cast<uint2*>(qt + static_cast<size_t>(c) * pitch + me.l16 * 8) = w;
    }
}

}  // namespace dg
