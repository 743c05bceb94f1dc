// A tile of FP32 values in registers, 128 rows of 128 columns (a scaling block in either direction) or fewer, quantised along its
// columns and, with 128 of them, along its rows. A warp (or half of one) has R whole rows and a lane 4 columns of each, v[row][pair
// of columns]: a row's largest magnitude is one reduction of the warp, and a column's needs no exchange inside a warp, only
// one over the 128 / R groups of rows through shared memory.
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
// tile, or, from lane 16 on, of the second, and hands round its reciprocal and the reciprocal's rest.
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
    const float rest = reciprocal_rest(mine.d, mine.r);
    const int row = lane / SHARE & (R - 1);
    if (lane % SHARE == 0 && row < valid) (lane < 16 ? sfv : sfu)[row * scales] = mine.s;
#pragma unroll
    for (int i = 0; i < R; ++i, qv += pitch, qu += pitch) {
        const float rv = __shfl_sync(0xffffffffu, mine.r, i * SHARE), ru = __shfl_sync(0xffffffffu, mine.r, 16 + i * SHARE);
        const float lv = __shfl_sync(0xffffffffu, rest, i * SHARE), lu = __shfl_sync(0xffffffffu, rest, 16 + i * SHARE);
        const uint32_t a = quantise4_by(v[i][0], v[i][1], rv, lv), b = quantise4_by(u[i][0], u[i][1], ru, lu);
        if (i < valid) {
            *reinterpret_cast<uint32_t*>(qv) = a;
            *reinterpret_cast<uint32_t*>(qu) = b;
        }
    }
}

// Codes along the columns of a tile of 128 rows and COLUMNS columns, in three steps with a barrier of the CTA behind each: the
// largest magnitudes of every group of R rows, the columns' scales, the codes, which then leave as the rows of the transpose.
// A group of R rows is COLUMNS / 4 lanes', a warp's or half a warp's; `lane` is the one of these.
template <int R, int COLUMNS = TILE>
struct TileColumns {
    static_assert(R == 8 || R == 16, "two or four words of codes a lane and column");
    static constexpr int GROUPS = TILE / R;
    static constexpr int THREADS = GROUPS * COLUMNS / 4;
    __align__(16) float amax[GROUPS][COLUMNS];
    __align__(16) float reciprocal[COLUMNS];
    __align__(16) float rest[COLUMNS];            // of the reciprocal
    __align__(16) uint32_t codes[TILE * COLUMNS / 4];

    __device__ __forceinline__ void maxima(const float2 (&v)[R][2], int group, int lane) {
        float a[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const auto at = [&](int i) { return c & 1 ? v[i][c >> 1].y : v[i][c >> 1].x; };
            a[c] = abs_max(at(0), at(1), at(2));
#pragma unroll
            for (int i = 3; i + 1 < R; i += 2) a[c] = abs_max(a[c], at(i), at(i + 1));
            a[c] = abs_max(a[c], at(R - 1));
        }
        *reinterpret_cast<float4*>(&amax[group][lane * 4]) = make_float4(a[0], a[1], a[2], a[3]);
    }

    // by one thread a column; sft: the column's scale
    __device__ __forceinline__ void scale(int c, float* sft) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < GROUPS; w += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = abs_max(a[j], amax[w + j][c], amax[w + j + 4][c]);
        const BlockScale k = block_scale(abs_bits(abs_max(abs_max(a[0], a[1], a[2]), a[3])));
        reciprocal[c] = k.r;
        rest[c] = reciprocal_rest(k.d, k.r);
        *sft = k.s;
    }

    // Rows 4w .. 4w + 3 of column c are word w of its 32. A group's words are at group ^ (c / 4 % GROUPS): neither these stores nor
    // the loads below meet in a bank.
    __device__ __forceinline__ void quantise(const float2 (&v)[R][2], int group, int lane) {
        const float4 r = *reinterpret_cast<const float4*>(&reciprocal[lane * 4]);
        const float4 d = *reinterpret_cast<const float4*>(&rest[lane * 4]);
        const int slot = group ^ (lane & (GROUPS - 1));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float2 rest2 = x ? make_float2(d.z, d.w) : make_float2(d.x, d.y), rr = x ? make_float2(r.z, r.w) : make_float2(r.x, r.y);
            uint32_t lo[R / 4], hi[R / 4];
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                float2 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = quotient2_by(v[i + j][x], rr, rest2);
                lo[i / 4] = pack_e4m3x2(w[0].x, w[1].x) | (pack_e4m3x2(w[2].x, w[3].x) << 16);
                hi[i / 4] = pack_e4m3x2(w[0].y, w[1].y) | (pack_e4m3x2(w[2].y, w[3].y) << 16);
            }
            uint32_t* dst = codes + (lane * 4 + 2 * x) * 32 + slot * (R / 4);
            if constexpr (R == 16) {
                *reinterpret_cast<uint4*>(dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                *reinterpret_cast<uint4*>(dst + 32) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            } else {
                *reinterpret_cast<uint2*>(dst) = make_uint2(lo[0], lo[1]);
                *reinterpret_cast<uint2*>(dst + 32) = make_uint2(hi[0], hi[1]);
            }
        }
    }

    // 128 bytes a column by GROUPS lanes; qt points at the tile's first column's codes, columns `pitch` apart.
    __device__ __forceinline__ void store(uint8_t* qt, size_t pitch) const {
        constexpr int PASS = THREADS / GROUPS;    // columns at a time
        const int l = static_cast<int>(threadIdx.x) % GROUPS, c0 = static_cast<int>(threadIdx.x) / GROUPS;
        uint8_t* dst = qt + static_cast<size_t>(c0) * pitch + l * R;
        const uint32_t* src = codes + c0 * 32;
#pragma unroll
        for (int i = 0; i < COLUMNS / PASS; ++i, dst += PASS * pitch) {
            const int at = i * PASS * 32 + (l ^ (c0 >> 2) ^ (i * (PASS / 4) & (GROUPS - 1))) * (R / 4);      // (c0 >> 2 is below PASS / 4)
            if constexpr (R == 16) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src + at);
            else *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src + at);
        }
    }
};

// The tiles that a CTA (or a warp) takes: every gridDim.x-th, the inner index first. The steps are worked out once: a division for each tile
// would be a tenth of its instructions.
struct TileWalk {
    int outer, inner, step_outer, step_inner, outers, inners;
    __device__ __forceinline__ TileWalk(int outers, int inners, int first, int every) : outers(outers), inners(inners) {
        outer = first / inners;
        inner = first - outer * inners;
        step_outer = every / inners;
        step_inner = every - step_outer * inners;
    }
    __device__ __forceinline__ TileWalk(int outers, int inners) : TileWalk(outers, inners, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x)) {}
    __device__ __forceinline__ bool more() const { return outer < outers; }
    // To the next tile; whether the inner index has begun again.
    __device__ __forceinline__ bool next() {
        outer += step_outer;
        inner += step_inner;
        if (inner < inners) return false;
        inner -= inners;
        ++outer;
        return true;
    }
};

// A place in an array that moves with the tiles, by so much for each step of the outer and the inner index.
struct TileOffset {
    int64_t at, step, wrap;
    __device__ __forceinline__ TileOffset(const TileWalk& w, int64_t of_outer, int64_t of_inner)
        : at(w.outer * of_outer + w.inner * of_inner), step(w.step_outer * of_outer + w.step_inner * of_inner), wrap(of_outer - w.inners * of_inner) {}
    __device__ __forceinline__ void next(bool wrapped) { at += wrapped ? step + wrap : step; }
};

}  // namespace dg
