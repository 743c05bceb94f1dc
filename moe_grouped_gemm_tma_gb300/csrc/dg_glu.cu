// The gated activation between two grouped products (dg_glu), its pre-activations kept in 8 bits on request, its backward
// pass from them (dg_glu_backward), and the values of 8-bit codes quantised along the other axis (dg_transpose_fp8), which
// makes the operand of a weight gradient from the codes that the forward product read.
//
//   h = act(g) u,  (q, sf) = Q(h),  (kept, kept_sf) = Q(g; u)
//   dg = dh u act'(g),  du = dh act(g): Q(dg; du) along rows and along columns, Q(h) along columns
//
// Forward: a half warp has the 128 values of a scaling block of 4 rows, 8 columns a lane, and both halves of Z's rows there.
// Backward and transposition: tiles of 128 rows (dg_tile.cuh). All three are memory's by their bytes; the backward pass and the
// transposition are held up by instructions and barriers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>

#include "dg.h"
#include "dg_host.cuh"
#include "dg_ptx.cuh"
#include "dg_quant.cuh"
#include "dg_tile.cuh"

namespace dg {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int64_t TILES_MAX = INT32_MAX / 2;        // (tiles are numbered in 32 bits)
constexpr int GLU_WARPS = 4;
constexpr int GLU_LANE_ROWS = 4;                  // rows of a half warp
__host__ __device__ constexpr int glu_ctas(bool keep) { return keep ? 4 : 5; }    // of an SM: what the registers hold

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

__device__ __forceinline__ float abs_max8(const float2 (&a)[4]) {
    return abs_max(abs_max(a[0].x, a[0].y, a[1].x), abs_max(a[1].y, a[2].x, a[2].y), abs_max(a[3].x, a[3].y));
}

__device__ __forceinline__ void unpack_bf16(const uint4& v, float2 (&a)[4]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
}

// The largest magnitudes of N lines (a power of two up to 16), each spread over 16 lanes, giving away lines on the way: lane l
// ends with that of line l / (16 / N).
template <int N>
__device__ __forceinline__ float line_maxima(float (&a)[N], int l16) {
    int step = 8;
#pragma unroll
    for (int n = N; n > 1; n /= 2, step /= 2) {
        const bool up = (l16 & step) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float give = up ? a[i] : a[n / 2 + i], keep = up ? a[n / 2 + i] : a[i];
            a[i] = abs_max(keep, __shfl_xor_sync(FULL, give, step));
        }
    }
    float most = a[0];
#pragma unroll
    for (; step > 0; step /= 2) most = abs_max(most, __shfl_xor_sync(FULL, most, step));
    return most;
}

// Codes of a lane's 8 values of a line whose scale lane `from` has.
__device__ __forceinline__ uint2 line_codes(const float2 (&v)[4], const BlockScale& mine, float rest, int from) {
    const float r = __shfl_sync(FULL, mine.r, from, 16), l = __shfl_sync(FULL, rest, from, 16);
    return make_uint2(quantise4_by(v[0], v[1], r, l), quantise4_by(v[2], v[3], r, l));
}

// A half warp has the 128 values of a scaling block of 4 rows, a lane 8 columns of each, in both halves of Z. The largest
// magnitudes of all its lines (h's, with KEEP g's and u's) are found together, and each line's scale is made by one lane. A warp
// takes piece after piece, and the next one's values come by asynchronous copies into places that only their lane reads: with
// loads into registers 36.8 k rows of 2 x 2048 took 94.4 us (two rows a lane, 8 CTAs an SM) with codes kept and 58.9 without; so
// they take 86.6 (6.2 TB/s) and 56.6 (6.7), of which h's codes by the rounded quotient, where the reciprocal alone would move some
// twenty in a million by a step, are 1.9 and 0.7. With masked_m the walk goes over the room of all experts: 32 experts of 16 rows each
// take 4.4 us with max_m = 64 and 29 with 4096.
template <int ACT, bool KEEP>
__global__ void __launch_bounds__(32 * GLU_WARPS, glu_ctas(KEEP)) glu_kernel(const GluParams p) {
    constexpr int R = GLU_LANE_ROWS, LINES = KEEP ? 4 * R : R, SHARE = 16 / LINES;
    constexpr unsigned ALL = (1u << R) - 1;
    __shared__ __align__(16) uint4 s_z[2][2 * R][32 * GLU_WARPS];     // [stage][row of g, row of u][thread]
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, l16 = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
    const size_t inner = p.inner, blocks = inner / 128;
    TileWalk walk((p.m + 2 * R - 1) / (2 * R), p.inner / 128, static_cast<int>(blockIdx.x) * GLU_WARPS + warp, static_cast<int>(gridDim.x) * GLU_WARPS);

    // Asks for the next piece that has rows to compute: their mask, 0 where there is no such piece.
    unsigned rows = 0;
    int r0 = 0, block = 0;
    const auto fetch = [&](int stage) {
        for (rows = 0; walk.more(); walk.next()) {
            r0 = (walk.outer * 2 + half) * R;
            block = walk.inner;
            if (p.m_indices != nullptr) {
                // (the rows are of one block of 128, which is computed if its first row has an expert)
                if (r0 < p.m && ld_input(p.m_indices + r0 / 128 * 128) >= 0) rows = ALL;
            } else if (p.masked_m != nullptr) {
                int g = r0 / p.max_m, at = r0 - g * p.max_m;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (r0 + i < p.m && at < ld_input(p.masked_m + g)) rows |= 1u << i;
                    if (++at == p.max_m) {
                        at = 0;
                        ++g;
                    }
                }
            } else {
                const int left = p.m - r0;
                rows = left >= R ? ALL : left > 0 ? (1u << left) - 1 : 0;
            }
            if (__any_sync(FULL, rows != 0)) {
                walk.next();
                break;
            }
        }
        const __nv_bfloat16* src = p.z + static_cast<size_t>(r0) * (2 * inner) + block * 128 + l16 * 8;
#pragma unroll
        for (int i = 0; i < R; ++i, src += 2 * inner) {
            if (rows >> i & 1) {
                cp_async_16(&s_z[stage][i][threadIdx.x], src);
                cp_async_16(&s_z[stage][R + i][threadIdx.x], src + inner);
            } else {
                s_z[stage][i][threadIdx.x] = s_z[stage][R + i][threadIdx.x] = make_uint4(0, 0, 0, 0);
            }
        }
        cp_async_commit();
        return __any_sync(FULL, rows != 0);
    };
    int stage = 0;
    for (bool more = fetch(0); more; stage ^= 1) {
        const unsigned mask = rows;
        const int row0 = r0, column = block;
        more = fetch(stage ^ 1);
        cp_async_wait_group<1>();
        float2 h[R][4];
        float most[LINES];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float2 g[4], u[4];
            unpack_bf16(s_z[stage][i][threadIdx.x], g);
            unpack_bf16(s_z[stage][R + i][threadIdx.x], u);
            if (KEEP) {
                most[R + i] = abs_max8(g);
                most[2 * R + i] = abs_max8(u);
                most[3 * R + i] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) h[i][c] = __fmul2_rn(act_fine2<ACT>(g[c]), u[c]);
            most[i] = abs_max8(h[i]);
        }
        const uint32_t bits = abs_bits(line_maxima(most, l16));
        const int line = l16 / SHARE, row = line & (R - 1), which = line / R;
        const BlockScale mine = p.pow2 && which == 0 ? block_scale_pow2(bits) : block_scale(bits);
        const float rest = reciprocal_rest(mine.d, mine.r);
        if (l16 % SHARE == 0 && (mask >> row & 1)) {
            const size_t at = static_cast<size_t>(row0 + row) * blocks;
            if (which == 0) p.sf[at + column] = mine.s;
            if (KEEP && (which == 1 || which == 2)) p.kept_sf[2 * at + (which - 1) * blocks + column] = mine.s;
        }
        uint8_t* q = p.q + static_cast<size_t>(row0) * inner + column * 128 + l16 * 8;
        uint8_t* kept = KEEP ? p.kept + static_cast<size_t>(row0) * (2 * inner) + column * 128 + l16 * 8 : nullptr;
#pragma unroll
        for (int i = 0; i < R; ++i, q += inner) {
            const uint2 w = line_codes(h[i], mine, rest, i * SHARE);
            if (mask >> i & 1) *reinterpret_cast<uint2*>(q) = w;
        }
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < R; ++i, kept += 2 * inner) {
                float2 v[4];
                unpack_bf16(s_z[stage][i][threadIdx.x], v);
                const uint2 gq = line_codes(v, mine, rest, (R + i) * SHARE);
                unpack_bf16(s_z[stage][R + i][threadIdx.x], v);
                const uint2 uq = line_codes(v, mine, rest, (2 * R + i) * SHARE);
                if (mask >> i & 1) {
                    *reinterpret_cast<uint2*>(kept) = gq;
                    *reinterpret_cast<uint2*>(kept + inner) = uq;
                }
            }
        }
    }
}

// ------------------------------------------------------------------------------------ backward
// Four codes times their scale.
__device__ __forceinline__ void code_values(uint32_t w, float s, float2 (&a)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
        a[i] = __fmul2_rn(__half22float2(__half2(h)), make_float2(s, s));
    }
}

__device__ __forceinline__ void bf16_values(uint2 w, float2 (&a)[2]) {
    a[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
    a[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
}

struct GluBackwardParams {
    const __nv_bfloat16* dh;
    const __nv_bfloat16* z;
    const uint8_t* kept;
    const float* kept_sf;
    const void* any;      // an address to name where nothing is read
    uint8_t* q;
    float* sf;
    uint8_t* qt;
    float* sft;
    uint8_t* ht;
    float* hsft;
    int m, inner;
    int m_tiles, n_tiles;
};

constexpr int GB_ROWS = 8;                        // rows of a warp
constexpr int GB_THREADS = 32 * TILE / GB_ROWS;
template <bool KEPT>
struct GluBackwardShared {
    TileColumns<GB_ROWS> dg, du, h;
    __align__(16) uint2 dh[TILE][32];             // the tile's inputs, as they are in global memory
    __align__(16) uint32_t g[TILE][KEPT ? 32 : 64], u[TILE][KEPT ? 32 : 64];
    __align__(16) float scale[2][TILE];           // of g's and u's codes
};

// A CTA makes all three outputs of a tile, so that what they share is computed once: 96 values a thread, which is what the
// registers hold with one CTA of 512 threads an SM. Its barriers are hidden by nothing else, therefore: the next tile's
// inputs come while this one's are in use, and the rows' codes are made while some warps make the columns' scales.
//
// Floor: 9.25 bytes an element of dH from codes, 45.6 us for 16384 x 2048. It takes 82.3 us (SILU; GELU 91.1, its tanh form 85.3;
// from BF16 80.7), with codes by the reciprocal alone, some twenty in a million off by a step, 77.7. What bounds it is latency:
// 49 instructions an element at 53% of the issue slots, with the FP32 pipe 40% busy, the integer one 41% and DRAM 28%;
// four warps a scheduler that wait together at three barriers a tile leave the rest empty.
// With codes by the reciprocal a CTA for each of the three outputs took 153 us; all three in one with 1024 threads and 4 rows
// a lane 87.3 (one sigmoid for value and slope, the next inputs asked into L2), 84.1 with them copied to shared memory, 77.7 with 512
// threads; two CTAs an SM with half a tile's columns each, a pair of them exchanging the rows' maxima, took 83.7.
template <int ACT, bool KEPT>
__global__ void __launch_bounds__(GB_THREADS, 1) glu_backward_kernel(const GluBackwardParams p) {
    extern __shared__ __align__(16) uint8_t s_raw[];
    GluBackwardShared<KEPT>& s = *reinterpret_cast<GluBackwardShared<KEPT>*>(s_raw);
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t inner = p.inner, blocks = inner / 128, pitch = static_cast<size_t>(p.m_tiles) * TILE;
    // (rows past M are zeros: so are the activations there, and their slopes are finite)
    const auto fetch = [&](const TileWalk& at) {
        const int t = threadIdx.x, m0 = at.outer * TILE, n0 = at.inner * TILE;
#pragma unroll
        for (int i = 0; i < TILE * 16 / GB_THREADS; ++i) {
            const int r = i * (GB_THREADS / 16) + t / 16;
            const size_t row = m0 + r;
            const bool there = m0 + r < p.m;
            cp_async_16_or_zero(&s.dh[r][t % 16 * 2], there && p.dh != nullptr ? p.dh + row * inner + n0 + t % 16 * 8 : p.any, there && p.dh != nullptr);
            if (!KEPT) {
                const __nv_bfloat16* src = there ? p.z + row * (2 * inner) + n0 + t % 16 * 8 : static_cast<const __nv_bfloat16*>(p.any);
                cp_async_16_or_zero(&s.g[r][t % 16 * 4], src, there);
                cp_async_16_or_zero(&s.u[r][t % 16 * 4], there ? src + inner : src, there);
            }
        }
        if (KEPT) {
#pragma unroll
            for (int i = 0; i < TILE * 8 / GB_THREADS; ++i) {
                const int r = i * (GB_THREADS / 8) + t / 8;
                const size_t row = m0 + r;
                const bool there = m0 + r < p.m;
                const uint8_t* src = there ? p.kept + row * (2 * inner) + n0 + t % 8 * 16 : static_cast<const uint8_t*>(p.any);
                cp_async_16_or_zero(&s.g[r][t % 8 * 4], src, there);
                cp_async_16_or_zero(&s.u[r][t % 8 * 4], there ? src + inner : src, there);
            }
            if (t < 2 * TILE) {
                const int which = t / TILE, rs = t % TILE;
                if (m0 + rs < p.m) cp_async_4(&s.scale[which][rs], p.kept_sf + static_cast<size_t>(m0 + rs) * (2 * blocks) + which * blocks + at.inner);
                else s.scale[which][rs] = 0.f;
            }
        }
    };
    TileWalk walk(p.m_tiles, p.n_tiles);
    if (walk.more()) fetch(walk);
    cp_async_wait_all();
    __syncthreads();
    for (bool more = walk.more(); more;) {
        const int tm = walk.outer, tn = walk.inner;
        const int r0 = tm * TILE + warp * GB_ROWS, c0 = tn * TILE + lane * 4, valid = p.m - r0;
        float2 dg[GB_ROWS][2], du[GB_ROWS][2], h[GB_ROWS][2];
#pragma unroll
        for (int i = 0; i < GB_ROWS; ++i) {
            const int r = warp * GB_ROWS + i;
            float2 dv[2], gv[2], uv[2];
            bf16_values(s.dh[r][lane], dv);
            if (KEPT) {
                code_values(s.g[r][lane], s.scale[0][r], gv);
                code_values(s.u[r][lane], s.scale[1][r], uv);
            } else {
                bf16_values(*reinterpret_cast<const uint2*>(&s.g[r][lane * 2]), gv);
                bf16_values(*reinterpret_cast<const uint2*>(&s.u[r][lane * 2]), uv);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float2 a, slope;
                act_both2<ACT>(gv[c], a, slope);
                dg[i][c] = __fmul2_rn(__fmul2_rn(dv[c], uv[c]), slope);
                du[i][c] = __fmul2_rn(dv[c], a);
                h[i][c] = __fmul2_rn(a, uv[c]);
            }
        }
        if (p.qt != nullptr) {
            s.dg.maxima(dg, warp, lane);
            s.du.maxima(du, warp, lane);
        }
        if (p.ht != nullptr) s.h.maxima(h, warp, lane);
        __syncthreads();
        walk.next();
        more = walk.more();
        if (more) fetch(walk);
        const int part = static_cast<int>(threadIdx.x) / TILE, column = static_cast<int>(threadIdx.x) % TILE;
        if (p.qt != nullptr) {
            if (part == 0) s.dg.scale(column, p.sft + (static_cast<size_t>(tn) * TILE + column) * p.m_tiles + tm);
            else if (part == 1) s.du.scale(column, p.sft + (inner + static_cast<size_t>(tn) * TILE + column) * p.m_tiles + tm);
        }
        if (p.ht != nullptr && part == 2) s.h.scale(column, p.hsft + (static_cast<size_t>(tn) * TILE + column) * p.m_tiles + tm);
        if (p.q != nullptr) {
            uint8_t* q = p.q + static_cast<size_t>(r0) * (2 * inner) + c0;
            float* sf = p.sf + static_cast<size_t>(r0) * (2 * blocks) + tn;
            tile_rows2(dg, du, q, q + inner, 2 * inner, sf, sf + blocks, 2 * blocks, valid, lane);
        }
        __syncthreads();
        if (p.qt != nullptr) {
            s.dg.quantise(dg, warp, lane);
            s.du.quantise(du, warp, lane);
        }
        if (p.ht != nullptr) s.h.quantise(h, warp, lane);
        cp_async_wait_all();
        __syncthreads();
        const size_t first = static_cast<size_t>(tn) * TILE * pitch + static_cast<size_t>(tm) * TILE;
        if (p.qt != nullptr) {
            s.dg.store(p.qt + first, pitch);
            s.du.store(p.qt + inner * pitch + first, pitch);
        }
        if (p.ht != nullptr) s.h.store(p.ht + first, pitch);
    }
}

struct TransposeParams {
    const uint8_t* q;
    const float* sf;
    uint8_t* qt;
    float* sft;
    int m, n;
    int m_tiles, n_tiles;
};

// Tiles of 128 rows and 64 columns, 16 rows a lane, four CTAs of 128 threads an SM: three barriers a tile leave a CTA's warps
// waiting together, which more and smaller CTAs fill, and what a lane does once a tile is spread over more codes. 32768 x 7168
// takes 93.2 us (5.2 TB/s); with 128 columns and two CTAs 95.3, with 8 rows a lane 99.3 (128 columns 102.5, 32 columns 117.6). A CTA
// takes every gridDim.x-th tile; the next one's codes are asked for as soon as this one's are in use (two tiles ahead into
// shared memory was no faster). What bounds it is instruction issue between the barriers, a fifth of it the codes' way to
// FP32, and the pieces: copies of as many bytes in the same pieces take 82 us.
constexpr int TR_ROWS = 16;                       // rows of a half warp
constexpr int TR_COLUMNS = 64;
constexpr int TR_CTAS = 4;
using TransposeTile = TileColumns<TR_ROWS, TR_COLUMNS>;
static_assert(TR_ROWS <= TR_COLUMNS / 4, "a lane loads the scale of one of its group's rows");

__global__ void __launch_bounds__(TransposeTile::THREADS, TR_CTAS) transpose_kernel(const TransposeParams p) {
    __shared__ TransposeTile s;
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int LANES = TR_COLUMNS / 4;         // of a group of rows
    const int group = static_cast<int>(threadIdx.x) / LANES, lane = static_cast<int>(threadIdx.x) % LANES;
    const int64_t n = p.n, blocks = n / TILE, pitch = static_cast<int64_t>(p.m_tiles) * TILE;
    uint32_t codes[TR_ROWS];
    float scale = 0.f;                            // of the group's row `lane`
    TileWalk walk(p.m_tiles, p.n_tiles);
    const uint8_t* q = p.q + group * TR_ROWS * n + lane * 4;
    const float* sf = p.sf + (group * TR_ROWS + lane) * blocks;
    TileOffset from(walk, TILE * n, TR_COLUMNS), to(walk, TILE, TR_COLUMNS * pitch), scales(walk, 1, static_cast<int64_t>(TR_COLUMNS) * p.m_tiles);
    const auto load = [&]() {
        const int valid = p.m - walk.outer * TILE - group * TR_ROWS;
        const uint8_t* src = q + from.at;
        const float* ssf = sf + (walk.outer * TILE * blocks + walk.inner * TR_COLUMNS / TILE);
        if (valid >= TR_ROWS) {
            if (lane < TR_ROWS) scale = ld_input(ssf);
#pragma unroll
            for (int i = 0; i < TR_ROWS; ++i, src += n) codes[i] = ld_input(reinterpret_cast<const uint32_t*>(src));
        } else {
            scale = lane < TR_ROWS && lane < valid ? ld_input(ssf) : 0.f;
#pragma unroll
            for (int i = 0; i < TR_ROWS; ++i, src += n) codes[i] = i < valid ? ld_input(reinterpret_cast<const uint32_t*>(src)) : 0u;
        }
    };
    if (walk.more()) load();
    for (bool more = walk.more(); more;) {
        float2 v[TR_ROWS][2];
#pragma unroll
        for (int i = 0; i < TR_ROWS; ++i) code_values(codes[i], __shfl_sync(FULL, scale, i, LANES), v[i]);
        const bool wrapped = walk.next();
        from.next(wrapped);
        more = walk.more();
        if (more) load();
        s.maxima(v, group, lane);
        __syncthreads();
        if (threadIdx.x < TR_COLUMNS) s.scale(threadIdx.x, p.sft + scales.at + static_cast<int>(threadIdx.x) * p.m_tiles);
        scales.next(wrapped);
        __syncthreads();
        s.quantise(v, group, lane);
        __syncthreads();
        s.store(p.qt + to.at, pitch);
        to.next(wrapped);
    }
}

template <bool KEEP>
cudaError_t launch_glu(const GluParams& p, int act, int sms, cudaStream_t stream) {
    const int64_t pieces = static_cast<int64_t>(cdiv(p.m, 2 * GLU_LANE_ROWS)) * (p.inner / 128), ctas = (pieces + GLU_WARPS - 1) / GLU_WARPS;
    const dim3 grid(static_cast<unsigned>(ctas < glu_ctas(KEEP) * sms ? ctas : glu_ctas(KEEP) * sms)), block(32 * GLU_WARPS);
    switch (act) {
        case DG_ACT_RELU: return launch_overlapped(glu_kernel<DG_ACT_RELU, KEEP>, grid, block, stream, p);
        case DG_ACT_GELU: return launch_overlapped(glu_kernel<DG_ACT_GELU, KEEP>, grid, block, stream, p);
        case DG_ACT_GELU_TANH: return launch_overlapped(glu_kernel<DG_ACT_GELU_TANH, KEEP>, grid, block, stream, p);
        case DG_ACT_SILU: return launch_overlapped(glu_kernel<DG_ACT_SILU, KEEP>, grid, block, stream, p);
        default: return launch_overlapped(glu_kernel<DG_ACT_NONE, KEEP>, grid, block, stream, p);
    }
}

template <int ACT, bool KEPT>
cudaError_t launch_backward_as(const GluBackwardParams& p, int sms, cudaStream_t stream) {
    constexpr int BYTES = sizeof(GluBackwardShared<KEPT>);
    const cudaError_t e = allow_smem<glu_backward_kernel<ACT, KEPT>>(BYTES);
    if (e != cudaSuccess) return e;
    const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
    return launch_overlapped_smem(glu_backward_kernel<ACT, KEPT>, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(GB_THREADS), BYTES, stream, p);
}

template <bool KEPT>
cudaError_t launch_backward(const GluBackwardParams& p, int act, int sms, cudaStream_t stream) {
    switch (act) {
        case DG_ACT_RELU: return launch_backward_as<DG_ACT_RELU, KEPT>(p, sms, stream);
        case DG_ACT_GELU: return launch_backward_as<DG_ACT_GELU, KEPT>(p, sms, stream);
        case DG_ACT_GELU_TANH: return launch_backward_as<DG_ACT_GELU_TANH, KEPT>(p, sms, stream);
        case DG_ACT_SILU: return launch_backward_as<DG_ACT_SILU, KEPT>(p, sms, stream);
        default: return launch_backward_as<DG_ACT_NONE, KEPT>(p, sms, stream);
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
    if (M > INT32_MAX - TILE || static_cast<int64_t>(cdiv(M, 2 * GLU_LANE_ROWS)) * (I / 128) > TILES_MAX) return DG_UNSUPPORTED_SHAPE;
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
    const cudaError_t e = kept ? launch_glu<true>(p, act, dev.sms, stream) : launch_glu<false>(p, act, dev.sms, stream);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

dg_status dg_glu_backward(const void* dH, const void* Z, const uint8_t* kept, const float* kept_sf, int act, uint8_t* q, float* sf, uint8_t* qt,
                          float* sft, uint8_t* ht, float* hsft, int M, int I, cudaStream_t stream) {
    if (M < 0 || I < 0 || act < DG_ACT_NONE || act > DG_ACT_SILU) return DG_INVALID_ARG;
    if ((q == nullptr) != (sf == nullptr) || (qt == nullptr) != (sft == nullptr) || (ht == nullptr) != (hsft == nullptr)) return DG_INVALID_ARG;
    if ((kept == nullptr) != (kept_sf == nullptr) || (Z && kept)) return DG_INVALID_ARG;
    if (I % 128 != 0 || I / 128 > 65535) return DG_UNSUPPORTED_SHAPE;
    if (M == 0 || I == 0 || (!q && !qt && !ht)) return DG_OK;
    if (M > INT32_MAX - TILE || static_cast<int64_t>(cdiv(M, TILE)) * (I / TILE) > TILES_MAX) return DG_UNSUPPORTED_SHAPE;
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
    p.any = kept ? static_cast<const void*>(kept) : Z;
    p.q = q;
    p.sf = sf;
    p.qt = qt;
    p.sft = sft;
    p.ht = ht;
    p.hsft = hsft;
    p.m = M;
    p.inner = I;
    p.m_tiles = cdiv(M, TILE);
    p.n_tiles = I / TILE;
    const cudaError_t e = kept ? launch_backward<true>(p, act, dev.sms, stream) : launch_backward<false>(p, act, dev.sms, stream);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

dg_status dg_transpose_fp8(const uint8_t* q, const float* sf, uint8_t* qt, float* sft, int M, int N, cudaStream_t stream) {
    if (M < 0 || N < 0) return DG_INVALID_ARG;
    if (N % 128 != 0 || N / 128 > 65535) return DG_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return DG_OK;
    if (M > INT32_MAX - TILE || static_cast<int64_t>(cdiv(M, TILE)) * (N / TILE) > TILES_MAX) return DG_UNSUPPORTED_SHAPE;
    if (!q || !sf || !qt || !sft) return DG_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(qt, 16) || !aligned(sf, 4) || !aligned(sft, 4)) return DG_MISALIGNED;
    DeviceInfo dev;
    const dg_status st = device_info(&dev);
    if (st != DG_OK) return st;
    const TransposeParams p = {q, sf, qt, sft, M, N, cdiv(M, TILE), N / TR_COLUMNS};
    const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles, most = static_cast<int64_t>(TR_CTAS) * dev.sms;
    const cudaError_t e = launch_overlapped(transpose_kernel, dim3(static_cast<unsigned>(tiles < most ? tiles : most)), dim3(TransposeTile::THREADS), stream, p);
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

}  // extern "C"
