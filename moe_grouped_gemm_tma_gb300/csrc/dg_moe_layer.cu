// A whole mixture-of-experts layer for a few tokens in one launch (dg_moe_layer):
//
//   out[t] = residual[t] + sum_j w[t,j] W2[e] . Q(act(g) * u),   (g; u) = W13[e] . Q(x[t]),   e = ids[t,j]
//
// What bounds it is streaming the met experts' weights, 3 H I bytes each, from HBM; the tokens, the hidden
// activations and every partial sum stay in L2. So the whole layer is one persistent kernel of one CTA per
// SM whose weight stream stops for nothing but a full ring:
//
//   * Split. A stage is 256 weight rows x one 128-wide K block, 32 KB. The stages of a phase (phase 1: W13,
//     phase 2: W2) form a line, unit after unit. With more units than CTAs, CTA c of G takes the c-th G-th of it, whatever
//     the number of met experts: every SM streams the same bytes, to one stage. With fewer units each is for a whole number
//     of CTAs, and the CTAs left over stream nothing, as long as the others' shares stay within six stages of an even one
//     (make_line). Parts of a unit that the cuts divide are summed in the order of the CTAs, so the result does not depend
//     on timing.
//   * Order. The met experts' chunks are halved, and the lines are: phase 1 of the first half, phase 1 of the
//     second, phase 2 of the first, phase 2 of the second. The hidden activations of one half are finished
//     (a grid barrier) while the weights of the other half stream.
//   * The products run transposed, weights as the MMA's 128 rows, a chunk of an expert's tokens (up to NT) as
//     its N, so the tensor cores see whole tiles for a single token. TMEM lane = weight row, column = token;
//     the promotion acc[token] += P * sx[token] * sb reads the 128x128 weight scale once per tile.
//   * The tokens are quantised once, into rows gathered by expert, while the rings fill with weights. (Doing it
//     on the way into shared memory, in every CTA, saves that barrier but not time: four warps take 1.2 us a
//     stage for one token and 2.5 us for 32, where the weights take 0.74.)
//   * A phase-1 unit is 128 gate rows with their 128 up rows; whoever completes it applies the activation and
//     quantises 128 hidden values per token. Four warps of their own do that, from the sums that the promoting
//     warps leave in L2: a round trip through L2 takes 2 us beside the weight stream, and a divided unit takes
//     four of them. A phase-2 unit is 256 output rows of one expert, written as FP32
//     per gathered row; after the last grid barrier all CTAs sum each token's experts, weighted, in order.
//
// Measured (hidden 7168, intermediate 2048): 64 tokens on 16 experts, 705 MB of weights, 147 us where the weights
// alone are 105; 1 token on 8 experts 62 us of 52.5. What is left: 9 us until the tokens are quantised (the
// ring fills meanwhile), 3 us for each grid barrier, 7 us for the output of 64 tokens, and HBM at 86% between. A
// small layer (5 tokens, 8 experts of 1024 x 384) takes 17.5 us for 1.4 of weights: tables 2 us, three grid
// barriers of 2.2, and two products' and one finisher's latency of 2 each.
//
// Warp roles: warp 0 streams weights, warp 2 tokens and their scales, warp 1 issues MMAs, warp 3 crosses the grid
// barriers, warps 4..7 finish phase-1 units, warps 8..15 promote; those twelve quantise the tokens at the start and
// sum the output at the end. Every wait is bounded as in dg_gemm_kernel; a CTA that gives up still arrives at the grid
// barriers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "dg.h"
#include "dg_host.cuh"
#include "dg_kernel.cuh"
#include "dg_launch.cuh"

namespace dg {
namespace {

constexpr int ML_MAX_T = 64;
constexpr int ML_MAX_A = 1024;                 // assignments, T * k
constexpr int ML_MAX_E = 1024;
constexpr int ML_MAX_CTAS = 160;               // CTAs (workspace slots) at most; one per SM
constexpr int ML_W_BYTES = 2 * 128 * BK;       // weights of a stage
constexpr int ML_FIXED = DG_MOE_LAYER_ZEROED;  // workspace: barrier word and counters (all that is read before it is written)
constexpr int ML_THREADS = 512;
constexpr int ML_FIN_WARP0 = 4, ML_EPI_WARP0 = 8, ML_WORKERS = 12;
constexpr int ML_CTRL_REGS = 56, ML_FIN_REGS = 104, ML_EPI_REGS = 176;  // 128 * (56 + 104) + 256 * 176 = 512 * 128
constexpr int ML_PARTS = 4;                    // segments between the promoting and the finishing warps
constexpr int ML_SLOTS = 4 + ML_PARTS;         // sums in L2 per CTA: first and last unit of either line, whole units
constexpr int ML_BARRIERS = 4;                 // grid barriers: tokens, hidden of either half, products
constexpr unsigned FULL_MASK = 0xffffffffu;
constexpr uint32_t NO_ROW = 0xffffffffu;

struct MoeParams {
    const __nv_bfloat16* x;
    const int32_t* ids;
    const float* weights;
    const float* s13;
    const float* s2;
    const __nv_bfloat16* residual;
    __nv_bfloat16* out;
    uint8_t* xg;           // [rows_cap][H] codes of the tokens, by gathered row
    float* sx;             // [H / 128][rows_cap]
    uint8_t* hg;           // [rows_cap][I] codes of the hidden activations, by gathered row
    float* sh;             // [I / 128][rows_cap]
    float* parts;          // [CTA][ML_SLOTS][NT][256]: sums of phase-1 units and of parts of them
    float* y;              // [gathered row][part][pairs * 256] weighted by nothing yet
    unsigned* barrier;     // grid barrier word
    unsigned* count;       // [phase-1 line][CTA]: parts of the unit that the CTA's share ends in
    int* status;
    int T, k, E, H, I, rows_cap, act;
    unsigned long long wait_limit_ns;   // bound of every wait (0 = WAIT_LIMIT_NS); tests shorten it
    int fault;                          // test only (0 in every product call): DG_FAULT_*, what is left out so that a wait runs out
};

template <int NT>
struct MlCfg {
    static_assert(NT == 16 || NT == 32 || NT == 64, "tokens per chunk");
    static constexpr int T_BYTES = NT * BK;
    static constexpr int STAGE_BYTES = ML_W_BYTES + T_BYTES;
    static constexpr int NACC = (TMEM_COLS / (2 * NT)) > 8 ? 8 : TMEM_COLS / (2 * NT);
    // The token scales of a stage live until it is promoted: the ring and the accumulators can hold that
    // many stages between the two, so with two more no slot is rewritten before it has been read.
    static constexpr int SLOTS = 6 + NACC + 2;
    static constexpr int TABLES = 4 * ML_MAX_A + 4 * ML_MAX_A + 4 * 4 * (ML_MAX_CTAS + 1) + 128;
    static constexpr int STATIC_RESERVE = TABLES + SLOTS * NT * 4 + 768;
    static constexpr int STAGES_FIT = ring_stages(STAGE_BYTES, 0, 0, STATIC_RESERVE);
    static constexpr int STAGES = STAGES_FIT > 6 ? 6 : STAGES_FIT;
    static constexpr int DYN_SMEM = 1024 + STAGES * STAGE_BYTES;
    static constexpr int FLIGHT = 3;            // weight stages in flight at once
    static constexpr int NG = NT / 16;          // 8-column groups per epilogue warpgroup
    static_assert(DYN_SMEM + STATIC_RESERVE <= SMEM_LIMIT && STAGES >= 4, "ring");
};

// 32 lanes x 8 consecutive 32-bit columns: thread t of the warp receives lane (base lane + t).
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// `bytes` (a multiple of 16, as the addresses) from global to shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ unsigned atom_add_acq_rel(unsigned* p, unsigned v) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

__device__ __forceinline__ void red_add_release(unsigned* p, unsigned v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__device__ __forceinline__ void finishers_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void add4(float4& a, const float4& b) { a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w; }

// One thread's arrival at the barrier of all CTAs, and its wait. CTA 0 adds what carries the others' ones
// into the top bit, so the bit flips when the last one arrives and the low bits are back at zero: the word
// needs no reset between barriers or launches. `top` is the top bit before this barrier (it cannot flip before
// this CTA has arrived), so the arrival itself has nothing to wait for. The CTAs are co-resident (cooperative
// launch); the wait ends by itself all the same. (`arrive` false: it only waits, for the test of that.)
__device__ __forceinline__ bool grid_barrier(unsigned* word, unsigned top, bool arrive, volatile int* abort_flag, int* status, uint64_t limit_ns) {
    const unsigned add = blockIdx.x == 0 ? 0x80000000u - (gridDim.x - 1) : 1u;
    if (arrive) red_add_release(word, add);
    const uint64_t t0 = global_timer_ns();
    const uint64_t limit = limit_ns ? limit_ns : WAIT_LIMIT_NS;
    for (int i = 0; i < (1 << 26); ++i) {
        if ((ld_acquire(word) ^ top) & 0x80000000u) return true;
        if ((i & 63) == 63 && global_timer_ns() - t0 > limit) break;
    }
    *abort_flag = 1;
    record_status(status, STATUS_TIMEOUT);
    return false;
}

// A thread's wait until all parts of a unit that its CTAs finish together are there: `arrivals` in the low 16 bits of
// the count (the high ones count the CTAs that are done with them).
__device__ __forceinline__ bool wait_parts(const unsigned* count, unsigned arrivals, volatile int* abort_flag, int* status, uint64_t limit_ns) {
    const uint64_t t0 = global_timer_ns();
    const uint64_t limit = limit_ns ? limit_ns : WAIT_LIMIT_NS;
    for (int i = 0; i < (1 << 26); ++i) {
        if ((ld_acquire(count) & 0xffffu) == arrivals) return true;
        if (*abort_flag) return false;
        if ((i & 63) == 63 && global_timer_ns() - t0 > limit) break;
    }
    *abort_flag = 1;
    record_status(status, STATUS_TIMEOUT);
    return false;
}

// A chunk: expert (10 bits), first gathered row (12 bits), rows - 1 (6 bits).
__device__ __forceinline__ uint32_t pack_chunk(int e, int off, int n) {
    return static_cast<uint32_t>(e) | (static_cast<uint32_t>(off) << 10) | (static_cast<uint32_t>(n - 1) << 22);
}

// The lines: phase 1 of the first half of the chunks, of the second half; phase 2 of the first, of the second.
struct Line {
    int c0, nc;            // chunks
    int kbs, blocks;       // K blocks of a unit; units per chunk
    int total;             // stages
    int sharers;           // CTAs that share them
};

template <int NT>
struct Shared {
    uint64_t full_w[MlCfg<NT>::STAGES], full_t[MlCfg<NT>::STAGES], empty[MlCfg<NT>::STAGES];   // weights, tokens
    uint64_t acc_full[MlCfg<NT>::NACC], acc_empty[MlCfg<NT>::NACC];
    uint64_t scale_full[MlCfg<NT>::SLOTS];
    uint64_t part_full[ML_PARTS], part_empty[ML_PARTS];
    uint64_t done[ML_BARRIERS], go[ML_BARRIERS];                   // this CTA's work before a grid barrier is done; it is crossed
    uint32_t tmem;
    int abort, chunks, rows, last;
    __align__(16) float scales[MlCfg<NT>::SLOTS][NT];
    uint32_t chunk[ML_MAX_A];
    uint32_t row_of[ML_MAX_A];                  // gathered row of an assignment (t * k + j) | chunk << 16, or NO_ROW
    uint32_t share[4][ML_MAX_CTAS + 1];         // first stage of each CTA's share of each line
    Line line[4];
};

// Chunks of the first "half", five eighths: the second's phase 1 has to hide the finishing of the first's units,
// and the first's phase 2, which is half as long per chunk, that of the second's. Where half of phase 1 streams for
// less than the 8 us that its units take to be finished and seen by all (11 stages a CTA), one half is all: a second
// one only adds a barrier (5 tokens, 8 experts of 1024 x 384: 25 us with halves, 21 without; 1 token, 8 experts of
// 7168 x 2048: 70 and 76).
__device__ __forceinline__ int first_half(const MoeParams& p, int chunks) {
    const int stages = chunks * (p.I / 128) * (p.H / 128);
    return stages >= 22 * static_cast<int>(gridDim.x) ? (chunks * 5 + 7) / 8 : chunks;
}

// a / b for 0 <= a < 2^20, 0 < b: half a unit above a is further from the next quotient than the rounding reaches
__device__ __forceinline__ int small_quotient(int a, int b) { return static_cast<int>((static_cast<float>(a) + 0.5f) * reciprocal_approx(static_cast<float>(b))); }

// A line and the CTAs that share it. Where there are at least as many CTAs as units, a whole number of them takes each
// unit, so that a CTA has one segment and a unit as few parts as may be, unless that leaves so many CTAs out that the
// others stream six stages more than an even share (44 tokens, 5 experts of 1536 x 768: 36.5 -> 28.8 us, 64 tokens, 8
// of 2048 x 1024: 36.9 -> 29.8, one token, 8 of 7168 x 2048: 63.1 -> 62.2). With many rows a phase-2 unit is for two
// CTAs at most: every part is written and read again, in FP32 (as many as there are: 29.8 us for the first of these).
__device__ __forceinline__ Line make_line(const MoeParams& p, int chunks, int l) {
    Line n;
    const int half = first_half(p, chunks);
    n.c0 = (l & 1) ? half : 0;
    n.nc = (l & 1) ? chunks - half : half;
    n.kbs = (l < 2 ? p.H : p.I) / 128;
    n.blocks = l < 2 ? p.I / 128 : (p.H + 255) / 256;
    n.total = n.nc * n.blocks * n.kbs;
    n.sharers = min(n.total, static_cast<int>(gridDim.x));
    const int units = n.nc * n.blocks, ctas = static_cast<int>(gridDim.x);
    if (units > 0 && units <= ctas) {
        int m = min(n.kbs, small_quotient(ctas, units));
        if (l >= 2 && p.T * p.k >= 64) m = min(m, 2);
        if ((small_quotient(n.kbs + m - 1, m) - 6) * ctas <= n.total) n.sharers = units * m;
    }
    return n;
}

// Where a CTA's share of a line starts, and whose share a stage is in. Every sharer has at least one stage, so no CTA
// between two parts of a unit is empty. The host keeps total * CTAs in 32 bits.
__device__ __forceinline__ unsigned share_start(const Line& n, unsigned cta) {
    const unsigned s = static_cast<unsigned>(n.sharers);
    return cta >= s ? n.total : static_cast<unsigned>(n.total) * cta / s;
}
__device__ __forceinline__ int cta_of(unsigned pos, const Line& n) {
    return static_cast<int>(((pos + 1) * static_cast<unsigned>(n.sharers) - 1) / static_cast<unsigned>(n.total));
}
// Parts that a unit of the line can have at most.
__device__ __forceinline__ int most_parts(const Line& n) {
    if (n.total == 0) return 1;
    const int least = static_cast<int>(static_cast<unsigned>(n.total) / static_cast<unsigned>(n.sharers));
    return (n.kbs - 1 + least - 1) / least + 1;
}

// Whether the CTAs of a divided phase-1 unit of n columns finish it together: with three parts or more, and more
// columns than four warps take at once, if the line's shares are shorter than a unit, so that no CTA has more than
// two segments of it. (55 tokens, 8 experts of 1152 x 128, nine parts and 28 columns a unit: the last CTA alone takes
// 13 us for them, the layer 33.6 us; together 4, and 23.9.) The promoting warps count their parts themselves, so that no CTA waits for another's finishers.
__device__ __forceinline__ bool finished_together(const Line& ln, int n, int parts) {
    return parts > 2 && n > 4 && ln.total < ln.sharers * ln.kbs;
}

// What a CTA does of one unit: stages [kb0, kb0 + nkb) of unit `unit`, for one chunk of an expert's tokens.
struct Seg {
    int unit;              // phase 1: chunk of the line * blocks + row block; phase 2: row pair * chunks + chunk
    int kb0, nkb;
    int e, off, n;         // expert, first gathered row, rows (1 .. NT)
    int blk;               // phase 1: 128-row block of I; phase 2: pair of 128-row blocks of H
    int row0, row1;        // rows of the weight matrix (all experts stacked) of the stage's two tiles
    bool two;              // the second tile exists (phase 2: an odd number of row blocks ends in half a pair)
};

template <int PHASE>
__device__ __forceinline__ Seg make_seg(const MoeParams& p, const Line& ln, const uint32_t* chunk, int pos, int hi) {
    Seg s;
    s.unit = pos / ln.kbs;
    s.kb0 = pos - s.unit * ln.kbs;
    s.nkb = min(ln.kbs - s.kb0, hi - pos);
    const int per = PHASE == 1 ? ln.blocks : ln.nc;
    const int a = s.unit / per, b = s.unit - a * per;
    s.blk = PHASE == 1 ? b : a;
    const uint32_t c = chunk[ln.c0 + (PHASE == 1 ? a : b)];
    s.e = static_cast<int>(c & 0x3ffu);
    s.off = static_cast<int>((c >> 10) & 0xfffu);
    s.n = static_cast<int>(c >> 22) + 1;
    if (PHASE == 1) {
        s.row0 = s.e * 2 * p.I + s.blk * 128;
        s.row1 = s.row0 + p.I;
        s.two = true;
    } else {
        s.row0 = s.e * p.H + s.blk * 256;
        s.row1 = s.row0 + 128;
        s.two = s.blk * 256 + 128 < p.H;
    }
    return s;
}

// Running positions in a ring.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++stage == n) { stage = 0; phase ^= 1u; }
    }
};

// The four lines in order, each segment of this CTA's share: f(phase tag, line number, line, segment). It
// stops when f returns false; `enter` (line number) runs before a line and may stop it too.
template <int NT, class Enter, class F>
__device__ __forceinline__ bool for_segments(const MoeParams& p, const Shared<NT>& s, Enter&& enter, F&& f) {
    const int cta = static_cast<int>(blockIdx.x);
#pragma unroll 1
    for (int l = 0; l < 2; ++l) {
        if (!enter(l)) return false;
        const Line& ln = s.line[l];
        const int hi = static_cast<int>(s.share[l][cta + 1]);
        for (int pos = static_cast<int>(s.share[l][cta]); pos < hi;) {
            const Seg g = make_seg<1>(p, ln, s.chunk, pos, hi);
            pos += g.nkb;
            if (!f(std::integral_constant<int, 1>{}, l, ln, g)) return false;
        }
    }
#pragma unroll 1
    for (int l = 2; l < 4; ++l) {
        if (!enter(l)) return false;
        const Line& ln = s.line[l];
        const int hi = static_cast<int>(s.share[l][cta + 1]);
        for (int pos = static_cast<int>(s.share[l][cta]); pos < hi;) {
            const Seg g = make_seg<2>(p, ln, s.chunk, pos, hi);
            pos += g.nkb;
            if (!f(std::integral_constant<int, 2>{}, l, ln, g)) return false;
        }
    }
    return true;
}

// ---- routing: chunks of at most NT tokens of one expert, their rows, and each assignment's row (its rank among
// the assignments of its expert, in order). Every CTA makes the same tables from the same ids: every warp ranks
// 32 assignments among themselves and counts their experts, the counts are summed over the warps' turns per
// expert, then over the experts. `scratch`: 72 KB.
template <int NT>
__device__ void make_tables(const MoeParams& p, Shared<NT>& s, uint8_t* scratch) {
    uint32_t* offset = reinterpret_cast<uint32_t*>(scratch);            // rows of an expert, then its first row
    uint32_t* first_chunk = offset + ML_MAX_E;
    uint16_t* counts = reinterpret_cast<uint16_t*>(first_chunk + ML_MAX_E);   // [group of 32 assignments][expert]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int A = p.T * p.k, groups = (A + 31) / 32;
    const int pitch = (p.E + 7) & ~7;
    constexpr int TURNS = ML_MAX_A / ML_THREADS;
    int expert[TURNS], rank[TURNS];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int a = i * ML_THREADS + tid;
        expert[i] = a < A ? __ldg(p.ids + a) : -1;
        if (expert[i] >= p.E) expert[i] = -1;
    }
    for (int i = tid; i < groups * pitch / 8; i += ML_THREADS) reinterpret_cast<uint4*>(counts)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int g = i * (ML_THREADS / 32) + warp;
        if (g >= groups) continue;
        const int e = expert[i] < 0 ? -1 : expert[i];
        const unsigned same = __match_any_sync(FULL_MASK, e);
        rank[i] = __popc(same & ((1u << lane) - 1u));
        if (e >= 0 && rank[i] == 0) counts[g * pitch + e] = static_cast<uint16_t>(__popc(same));
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += ML_THREADS) {
        uint32_t sum = 0;
        for (int g = 0; g < groups; ++g) {
            const uint32_t n = counts[g * pitch + e];
            counts[g * pitch + e] = static_cast<uint16_t>(sum);
            sum += n;
        }
        offset[e] = sum;
    }
    __syncthreads();
    if (warp == ML_FIN_WARP0) {
        // exclusive sums over the experts: rows rounded up to 4, and chunks
        int rows = 0, chunks = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            const int n = e < p.E ? static_cast<int>(offset[e]) : 0;
            int r = (n + 3) & ~3, c = (n + NT - 1) / NT;
            const int r_own = r, c_own = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int ur = __shfl_up_sync(FULL_MASK, r, o), uc = __shfl_up_sync(FULL_MASK, c, o);
                if (lane >= o) { r += ur; c += uc; }
            }
            const int r0 = rows + r - r_own, c0 = chunks + c - c_own;
            if (e < p.E) {
                offset[e] = static_cast<uint32_t>(r0);
                first_chunk[e] = static_cast<uint32_t>(c0);
            }
            for (int i = 0; i < c_own; ++i) s.chunk[c0 + i] = pack_chunk(e, r0 + i * NT, min(NT, n - i * NT));
            rows += __shfl_sync(FULL_MASK, r, 31);
            chunks += __shfl_sync(FULL_MASK, c, 31);
        }
        if (lane < 4) s.line[lane] = make_line(p, chunks, lane);
        if (lane == 0) {
            s.chunks = chunks;
            s.rows = rows;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int a = i * ML_THREADS + tid;
        if (a >= A) continue;
        const int e = expert[i];
        uint32_t where = NO_ROW;
        if (e >= 0) {
            const uint32_t n = counts[(a >> 5) * pitch + e] + static_cast<uint32_t>(rank[i]);   // of the expert's rows
            where = (offset[e] + n) | ((first_chunk[e] + n / NT) << 16);
        }
        s.row_of[a] = where;
    }
    for (int i = tid; i < 4 * static_cast<int>(gridDim.x + 1); i += ML_THREADS) {
        const int l = i / static_cast<int>(gridDim.x + 1), c = i - l * static_cast<int>(gridDim.x + 1);
        const Line& n = s.line[l];
        s.share[l][c] = n.total ? share_start(n, static_cast<unsigned>(c)) : 0u;
    }
}

// ---- output: a warp takes 128 columns of a token and adds up the parts of its experts' sums, weighted, from task
// `first` on. Eight lanes hold the columns, 16 each; the warp's four groups of eight take every fourth part, three
// at a time, and their sums are added at the end: a fixed order. The loop is short on purpose: this code is
// new to the SM when the last grid barrier opens, and unrolled over the parts it waited for its instructions
// longer than for its loads (6 us for one token). The sources are worked out before that barrier.
template <int NT>
__device__ __forceinline__ void sum_output(const MoeParams& p, const Shared<NT>& s, int first, bool ok, volatile int* abort_flag, int lane) {
    const Line &la = s.line[2], &lb = s.line[3];
    const int pa = most_parts(la), pb = most_parts(lb);
    const int base_b = lb.nc ? static_cast<int>((s.chunk[la.nc] >> 10) & 0xfffu) : s.rows;
    const size_t width = static_cast<size_t>(la.blocks) * 256;
    const int blocks = p.H / 128, tasks = p.T * blocks, stride = static_cast<int>(gridDim.x) * ML_WORKERS;
    const int group = lane >> 3, l8 = lane & 7;
    bool crossed = false;
    for (int w = first; w < tasks && ok; w += stride) {
        const int t = w / blocks, blk = w - t * blocks;
        float sum[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] = 0.f;
#pragma unroll 1
        for (int j0 = 0; j0 < p.k; j0 += 32) {
            // lane j: where assignment j's sums of this block lie (in rows of `width`), of how many parts they
            // are (0: no expert), and its weight
            int at = 0, parts = 0;
            float weight = 0.f;
            const int here = min(32, p.k - j0);
            const uint32_t where = lane < here ? s.row_of[t * p.k + j0 + lane] : NO_ROW;
            if (where != NO_ROW) {
                weight = __ldg(p.weights + t * p.k + j0 + lane);
                const int row = static_cast<int>(where & 0xffffu), chunk = static_cast<int>(where >> 16);
                const bool b = chunk >= la.nc;
                const Line& ln = b ? lb : la;
                const unsigned u0 = static_cast<unsigned>((blk >> 1) * ln.nc + chunk - (b ? la.nc : 0)) * la.kbs;
                parts = cta_of(u0 + la.kbs - 1, ln) - cta_of(u0, ln) + 1;
                at = b ? base_b * pa + (row - base_b) * pb : row * pa;
            }
            const int most = static_cast<int>(__reduce_max_sync(FULL_MASK, static_cast<unsigned>(parts))) * here;
            if (!crossed) {
                const bool got = wait_bounded(const_cast<uint64_t*>(&s.go[3]), 0, abort_flag, p.status, p.wait_limit_ns);
                ok = __all_sync(FULL_MASK, got) != 0;
                crossed = true;
            }
#pragma unroll 1
            for (int n0 = 0; n0 < most; n0 += 12) {
                float4 v[3][4];
                float u[3];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int n = n0 + 4 * i + group, c = n / here, j = n - c * here;
                    const int f = __shfl_sync(FULL_MASK, at, j);
                    const bool there = c < __shfl_sync(FULL_MASK, parts, j);
                    u[i] = __shfl_sync(FULL_MASK, weight, j);
                    u[i] = there ? u[i] : 0.f;
                    const float4* src = reinterpret_cast<const float4*>(p.y + static_cast<size_t>(f + c) * width + blk * 128 + l8 * 16);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        v[i][x] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (there) v[i][x] = __ldcg(src + x);
                    }
                }
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        sum[4 * x + 0] = fmaf(u[i], v[i][x].x, sum[4 * x + 0]);
                        sum[4 * x + 1] = fmaf(u[i], v[i][x].y, sum[4 * x + 1]);
                        sum[4 * x + 2] = fmaf(u[i], v[i][x].z, sum[4 * x + 2]);
                        sum[4 * x + 3] = fmaf(u[i], v[i][x].w, sum[4 * x + 3]);
                    }
            }
        }
        // the groups' sums: groups g and g ^ 2 exchange halves of the columns, then g and g ^ 1 quarters, so that
        // a lane ends with four columns, 4 * group' of its 16
        float half[8], four[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float give = group & 2 ? sum[i] : sum[8 + i], keep = group & 2 ? sum[8 + i] : sum[i];
            half[i] = keep + __shfl_xor_sync(FULL_MASK, give, 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float give = group & 1 ? half[i] : half[4 + i], keep = group & 1 ? half[4 + i] : half[i];
            four[i] = keep + __shfl_xor_sync(FULL_MASK, give, 8);
        }
        const size_t at = static_cast<size_t>(t) * p.H + blk * 128 + l8 * 16 + group * 4;
        if (p.residual != nullptr) {
            const uint2 res = *reinterpret_cast<const uint2*>(p.residual + at);
            four[0] += bf16_lo(res.x); four[1] += bf16_hi(res.x); four[2] += bf16_lo(res.y); four[3] += bf16_hi(res.y);
        }
        if (ok) st_global_v2(p.out + at, pack_bf16x2(four[0], four[1]), pack_bf16x2(four[2], four[3]));
    }
}

template <int NT>
__global__ void __launch_bounds__(ML_THREADS, 1)
moe_layer_kernel(const __grid_constant__ CUtensorMap map_w13, const __grid_constant__ CUtensorMap map_w2,
                 const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_h,
                 const __grid_constant__ MoeParams p) {
    using C = MlCfg<NT>;
    constexpr int STAGES = C::STAGES, NACC = C::NACC, NG = C::NG, SLOTS = C::SLOTS, FLIGHT = C::FLIGHT;
    static_assert(sizeof(Shared<NT>) <= C::STATIC_RESERVE, "static shared memory");
    static_assert(SLOTS >= STAGES + NACC + 2, "a scale slot is rewritten only after it has been read");

    extern __shared__ uint8_t dyn_smem[];
    __shared__ Shared<NT> s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = static_cast<int>(blockIdx.x);

    const uint32_t raw = smem_u32(dyn_smem);
    uint8_t* smem = dyn_smem + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* smem_t = smem + STAGES * ML_W_BYTES;

    if (threadIdx.x == 0) {
        prefetch_tmap(&map_w13);
        prefetch_tmap(&map_w2);
        prefetch_tmap(&map_x);
        prefetch_tmap(&map_h);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s.full_w[i], 1);
            mbar_init(&s.full_t[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < NACC; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], EPI_WARPS);
        }
        for (int i = 0; i < SLOTS; ++i) mbar_init(&s.scale_full[i], 1);
        for (int i = 0; i < ML_PARTS; ++i) {
            mbar_init(&s.part_full[i], EPI_WARPS);
            mbar_init(&s.part_empty[i], 4);
        }
        for (int i = 0; i < ML_BARRIERS; ++i) {
            mbar_init(&s.done[i], i == 0 ? ML_WORKERS : (i < 3 ? 4 : EPI_WARPS));
            mbar_init(&s.go[i], 1);
        }
        s.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem, TMEM_COLS);
        tmem_relinquish();
    }
    // the tokens' values that this warp quantises (blocks w, w + stride, ...; the first ones are loaded while
    // the tables are made)
    constexpr int AHEAD = 2;
    const int kbs_x = p.H / 128, blocks_x = p.T * kbs_x, stride_x = static_cast<int>(gridDim.x) * ML_WORKERS;
    const int first_x = cta + (warp - ML_FIN_WARP0) * static_cast<int>(gridDim.x);
    uint2 ahead[AHEAD];
    if (warp >= ML_FIN_WARP0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int w = first_x + i * stride_x;
            if (w < blocks_x) ahead[i] = *reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(w) * 128 + lane * 4);
        }
    }
    make_tables<NT>(p, s, smem);   // before the ring is in use
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s.tmem;
    volatile int* abort_flag = &s.abort;
    const auto nothing = [](int) { return true; };

    if (warp < ML_FIN_WARP0) {
        regs_dec<ML_CTRL_REGS>();
        const bool issuer = elect_one();
        if (warp == 0) {
            // ---------------------------------------------------------------- weights
            // At most FLIGHT stages are on their way at once: what the whole GPU has asked of HBM is the latency
            // of every other access (all the rings' 29 MB are 4.4 us of HBM), and half of that already keeps
            // HBM busy. The rest of the ring fills up while the consumers wait for something. One at a time until
            // the tokens are there, whose stores and barrier nothing can hide.
            const uint64_t once = policy_evict_first();   // L2 is for the sums and activations
            Ring ring, landed;
            int flying = 0, limit = 1;
            bool skip_fill = p.fault == DG_FAULT_FIRST_FILL;   // test only: leave the first stage empty
            uint32_t issued = 0, issued_parity = 0;
            bool ok = for_segments<NT>(p, s, nothing, [&](auto tag, int, const Line&, const Seg& g) {
                const CUtensorMap* map = decltype(tag)::value == 1 ? &map_w13 : &map_w2;
                for (int kb = g.kb0; kb < g.kb0 + g.nkb; ++kb) {
                    bool got = wait_bounded(&s.empty[ring.stage], ring.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns);
                    if (limit == 1 && mbar_test_wait(&s.go[0], 0)) limit = FLIGHT;
                    limit = __shfl_sync(FULL_MASK, limit, 0);
                    if (flying == limit) {
                        got = got && wait_bounded(&s.full_w[landed.stage], landed.phase, abort_flag, p.status, p.wait_limit_ns);
                        landed.next(STAGES);
                    } else {
                        ++flying;
                    }
                    if (!__all_sync(FULL_MASK, got)) return false;
                    if (skip_fill) {
                        skip_fill = false;
                        ring.next(STAGES);
                        continue;
                    }
                    if (issuer) {
                        uint8_t* dst = smem + ring.stage * ML_W_BYTES;
                        mbar_arrive_expect_tx(&s.full_w[ring.stage], g.two ? ML_W_BYTES : ML_W_BYTES / 2);
                        tma_load_2d_hint(map, &s.full_w[ring.stage], dst, kb * BK, g.row0, once);
                        if (g.two) tma_load_2d_hint(map, &s.full_w[ring.stage], dst + 128 * BK, kb * BK, g.row1, once);
                    }
                    issued |= 1u << ring.stage;
                    issued_parity = (issued_parity & ~(1u << ring.stage)) | (ring.phase << ring.stage);
                    ring.next(STAGES);
                    __syncwarp();
                }
                return true;
            });
            // every stage has been consumed: no MMA-completion arrival is on its way when the CTA exits
            for (int i = 0; i < STAGES && ok; ++i) {
                const bool got = wait_bounded(&s.empty[ring.stage], ring.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns);
                if (!__all_sync(FULL_MASK, got)) ok = false;
                ring.next(STAGES);
            }
            if (!ok && issuer) {
                for (int i = 0; i < STAGES; ++i)
                    if (issued & (1u << i)) drain_wait(&s.full_w[i], (issued_parity >> i) & 1u);
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA issue
            Ring ring, acc, last_ring, last_acc;
            bool any = false;
            const uint32_t w_base = smem_u32(smem), t_base = smem_u32(smem_t);
            for_segments<NT>(p, s, nothing, [&](auto, int, const Line&, const Seg& g) {
                const uint32_t idesc = idesc_e4m3_f32(128, (g.n + 15) & ~15);
                for (int kb = 0; kb < g.nkb; ++kb) {
                    const bool got = wait_bounded(&s.acc_empty[acc.stage], acc.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns) &&
                                     wait_bounded(&s.full_w[ring.stage], ring.phase, abort_flag, p.status, p.wait_limit_ns) &&
                                     wait_bounded(&s.full_t[ring.stage], ring.phase, abort_flag, p.status, p.wait_limit_ns);
                    if (!__all_sync(FULL_MASK, got)) return false;
                    tc_fence_after();
                    if (issuer) {
                        const uint64_t td = sw128_kmajor_desc(t_base + ring.stage * C::T_BYTES);
                        const uint64_t wd = sw128_kmajor_desc(w_base + ring.stage * ML_W_BYTES);
                        const uint32_t d = tmem_base + static_cast<uint32_t>(acc.stage * 2 * NT);
#pragma unroll
                        for (int k = 0; k < BK / UMMA_K; ++k)
                            mma_f8f6f4(d, wd + static_cast<uint64_t>(k * (UMMA_K >> 4)), td + static_cast<uint64_t>(k * (UMMA_K >> 4)), idesc, k > 0 ? 1u : 0u);
                        if (g.two) {
#pragma unroll
                            for (int k = 0; k < BK / UMMA_K; ++k)
                                mma_f8f6f4(d + NT, wd + static_cast<uint64_t>(((128 * BK) >> 4) + k * (UMMA_K >> 4)),
                                           td + static_cast<uint64_t>(k * (UMMA_K >> 4)), idesc, k > 0 ? 1u : 0u);
                        }
                        mma_commit(&s.empty[ring.stage]);
                        mma_commit(&s.acc_full[acc.stage]);
                    }
                    any = true;
                    last_ring = ring;
                    last_acc = acc;
                    ring.next(STAGES);
                    acc.next(NACC);
                    __syncwarp();
                }
                return true;
            });
            // the last MMAs and their arrivals end before the shared and the tensor memory are given up, whichever
            // warp of the CTA it is that gave up (else they have ended already, or do presently)
            if (any && issuer) {
                drain_wait(&s.empty[last_ring.stage], last_ring.phase);
                drain_wait(&s.acc_full[last_acc.stage], last_acc.phase);
            }
        } else if (warp == 2) {
            // ---------------------------------------------------------------- tokens
            Ring ring, slot;
            uint32_t issued = 0, issued_parity = 0, scaled = 0, scaled_parity = 0;   // stages, scale slots: bits, for the drain
            static_assert(SLOTS <= 32, "a bit a slot");
            bool skip_scales = p.fault == DG_FAULT_TOKEN_SCALES;   // test only: leave the first scales out
            for_segments<NT>(p, s, [&](int l) {
                if (l == 1) return true;
                if (l == 3 && s.line[1].nc == 0) return true;
                const bool got = wait_bounded(&s.go[l == 0 ? 0 : l - 1], 0, abort_flag, p.status, p.wait_limit_ns);
                fence_proxy_async_all();        // what other CTAs wrote before the barrier is read by TMA
                return __all_sync(FULL_MASK, got) != 0;
            }, [&](auto tag, int, const Line&, const Seg& g) {
                constexpr bool ONE = decltype(tag)::value == 1;
                const CUtensorMap* map = ONE ? &map_x : &map_h;
                const float* scales = (ONE ? p.sx : p.sh) + g.off;
                const int boxes = (g.n + 15) / 16;
                const uint32_t scale_bytes = static_cast<uint32_t>((g.n + 3) / 4 * 16);
                for (int kb = g.kb0; kb < g.kb0 + g.nkb; ++kb) {
                    const bool got = wait_bounded(&s.empty[ring.stage], ring.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns);
                    if (!__all_sync(FULL_MASK, got)) return false;
                    if (issuer) {
                        uint8_t* dst = smem_t + ring.stage * C::T_BYTES;
                        mbar_arrive_expect_tx(&s.full_t[ring.stage], static_cast<uint32_t>(boxes * 16 * BK));
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(map, &s.full_t[ring.stage], dst + b * 16 * BK, kb * BK, g.off + b * 16);
                        mbar_arrive_expect_tx(&s.scale_full[slot.stage], scale_bytes);
                        if (!skip_scales)
                            bulk_load(s.scales[slot.stage], scales + static_cast<size_t>(kb) * p.rows_cap, scale_bytes, &s.scale_full[slot.stage]);
                    }
                    skip_scales = false;
                    issued |= 1u << ring.stage;
                    issued_parity = (issued_parity & ~(1u << ring.stage)) | (ring.phase << ring.stage);
                    scaled |= 1u << slot.stage;
                    scaled_parity = (scaled_parity & ~(1u << slot.stage)) | (slot.phase << slot.stage);
                    ring.next(STAGES);
                    slot.next(SLOTS);
                    __syncwarp();
                }
                return true;
            });
            // copies still in flight, of codes and of scales, land before the shared memory is given up: also where this
            // warp has issued all of its own and another one gave up. (Without that the consumers have waited for
            // each, and nothing is waited for here.)
            if (issuer) {
                for (int i = 0; i < STAGES; ++i)
                    if (issued & (1u << i)) drain_wait(&s.full_t[i], (issued_parity >> i) & 1u);
                for (int i = 0; i < SLOTS; ++i)
                    if (scaled & (1u << i)) drain_wait(&s.scale_full[i], (scaled_parity >> i) & 1u);
            }
        } else if (warp == 3) {
            // ---------------------------------------------------------------- grid barriers
            if (lane == 0) {
                unsigned top = ld_acquire(p.barrier) & 0x80000000u;
#pragma unroll 1
                for (int b = 0; b < ML_BARRIERS; ++b) {
                    if (b == 2 && s.line[1].nc == 0) continue;   // no second half
                    wait_bounded(&s.done[b], 0, abort_flag, p.status, p.wait_limit_ns);
                    const bool arrive = p.fault != DG_FAULT_GRID_BARRIER || b > 0 || blockIdx.x != gridDim.x - 1;
                    const bool got = grid_barrier(p.barrier, top, arrive, abort_flag, p.status, p.wait_limit_ns);
                    top ^= 0x80000000u;
                    fence_proxy_async_all();
                    if (got) mbar_arrive(&s.go[b]);
                }
            }
        }
        __syncwarp();
    } else {
        // Where a segment's sums lie: the first and the last unit of the CTA's share of a line may be divided
        // (the unit is the first of every CTA but the one in whose share it starts); whole units take turns.
        auto slot_at = [&](int c, int which) { return p.parts + static_cast<size_t>(c * ML_SLOTS + which) * (NT * 256); };
        auto divided_slot = [&](int c, int l, unsigned u0) { return slot_at(c, l * 2 + (u0 < s.share[l][c] ? 0 : 1)); };
        auto line_done = [&](int b) {
            // (codes and scales are read by TMA; the grid barrier's arrival releases the CTA's writes)
            fence_proxy_async_all();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.done[b]);
        };
        // ---- the tokens' codes and scales, to every row that they are gathered to
        auto quantise = [&](int w, uint2 u) {
            const int t = w / kbs_x, kb = w - t * kbs_x;
            const float a = bf16_lo(u.x), b = bf16_hi(u.x), c = bf16_lo(u.y), d = bf16_hi(u.y);
            const BlockScale sc = block_scale(__reduce_max_sync(FULL_MASK, max(max(abs_bits(a), abs_bits(b)), max(abs_bits(c), abs_bits(d)))));
            const uint32_t code = quantise4(a, b, c, d, sc);
            uint8_t* dst = p.xg + kb * 128 + lane * 4;
            for (int j0 = 0; j0 < p.k; j0 += 32) {
                const uint32_t row = j0 + lane < p.k ? s.row_of[t * p.k + j0 + lane] : NO_ROW;
                if (row != NO_ROW) p.sx[static_cast<size_t>(kb) * p.rows_cap + (row & 0xffffu)] = sc.s;
                const int here = min(32, p.k - j0);
#pragma unroll 4
                for (int j = 0; j < here; ++j) {
                    const uint32_t to = __shfl_sync(FULL_MASK, row, j);
                    if (to != NO_ROW) *reinterpret_cast<uint32_t*>(dst + static_cast<size_t>(to & 0xffffu) * p.H) = code;
                }
            }
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (first_x + i * stride_x < blocks_x) quantise(first_x + i * stride_x, ahead[i]);
        for (int w = first_x + AHEAD * stride_x; w < blocks_x; w += stride_x)
            quantise(w, *reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(w) * 128 + lane * 4));
        line_done(0);
        bool ok = true;
        if (warp < ML_EPI_WARP0) {
            // ---------------------------------------------------------------- finishing phase-1 units
            regs_dec<ML_FIN_REGS>();
            const int q = warp & 3;
            Ring part;
            // a CTA is done with a unit that is finished together; the last one leaves the count as the next launch
            // expects it
            auto leave = [](unsigned* count, int parts) {
                if ((atom_add_acq_rel(count, 0x10000u) >> 16) == static_cast<unsigned>(parts - 1)) *count = 0;
            };
            for_segments<NT>(p, s, [&](int l) {
                if (l > 0) line_done(l);
                return l < 2;
            }, [&](auto, int l, const Line& ln, const Seg& g) {
                if (ok) {
                    const bool got = wait_bounded(&s.part_full[part.stage], part.phase, abort_flag, p.status, p.wait_limit_ns);
                    ok = __all_sync(FULL_MASK, got) != 0;
                }
                const unsigned u0 = static_cast<unsigned>(g.unit) * ln.kbs;
                const bool divided = g.nkb < ln.kbs;
                const int c_lo = divided ? cta_of(u0, ln) : cta, c_hi = divided ? cta_of(u0 + ln.kbs - 1, ln) : cta;
                const int parts = c_hi - c_lo + 1;
                // A divided unit is finished by the CTA whose part comes last, adding the parts in order, or by all of
                // them together, each a share of the columns.
                const bool shared = finished_together(ln, g.n, parts);
                const int c_first = shared ? 4 * (cta - c_lo) : 0, c_step = shared ? 4 * parts : 4;
                unsigned* count = p.count + l * ML_MAX_CTAS + c_lo;
                bool mine = true;
                if (divided) {
                    finishers_barrier();
                    if (q == 0 && lane == 0) {
                        // (releases what part_full has gathered from this CTA, acquires the others' parts)
                        bool here;
                        if (shared) {
                            here = c_first < g.n && wait_parts(count, static_cast<unsigned>(EPI_WARPS * parts), abort_flag, p.status, p.wait_limit_ns);
                            if (!here) leave(count, parts);
                        } else {
                            here = atom_add_acq_rel(count, 1u) == static_cast<unsigned>(parts - 1);
                            if (here) *count = 0;   // as the next launch expects it
                        }
                        s.last = here ? 1 : 0;
                    }
                    finishers_barrier();
                    mine = s.last != 0;
                }
                if (mine) {
                    // A warp takes whole columns (tokens), four rows a lane. Eight pairs of loads are in flight: up
                    // to two parts of four columns, or the first eight parts of one.
                    const float* mine_at = p.parts + lane * 4;
                    auto part_at = [&](int pt) {    // in floats from there
                        return static_cast<size_t>((divided ? divided_slot(c_lo + pt, l, u0) : slot_at(cta, 4 + part.stage)) - p.parts);
                    };
                    auto finish = [&](const float4& gate, const float4& upv, int col) {
                        float v[4] = {gate.x, gate.y, gate.z, gate.w};
                        act_values<4>(p.act, v);
                        v[0] *= upv.x; v[1] *= upv.y; v[2] *= upv.z; v[3] *= upv.w;
                        const BlockScale k = block_scale(__reduce_max_sync(FULL_MASK, max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])))));
                        const uint32_t code = quantise4(v[0], v[1], v[2], v[3], k);
                        const int row = g.off + col;
                        if (col < g.n) {
                            *reinterpret_cast<uint32_t*>(p.hg + static_cast<size_t>(row) * p.I + g.blk * 128 + lane * 4) = code;
                            if (lane == 0) p.sh[static_cast<size_t>(g.blk) * p.rows_cap + row] = k.s;
                        }
                    };
                    // (adding the zeros of parts that do not exist changes no sum)
                    if (parts <= 2) {
                        const float* at0 = mine_at + part_at(0);
                        const float* at1 = parts == 2 ? mine_at + part_at(1) : at0;
#pragma unroll 1
                        for (int c0 = q * 4; c0 < g.n; c0 += 16) {
                            float4 gate[4], upv[4], gate1[4], upv1[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                gate[j] = upv[j] = gate1[j] = upv1[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (c0 + j < g.n) {
                                    gate[j] = __ldcg(reinterpret_cast<const float4*>(at0 + (c0 + j) * 256));
                                    upv[j] = __ldcg(reinterpret_cast<const float4*>(at0 + (c0 + j) * 256 + 128));
                                    if (parts == 2) {
                                        gate1[j] = __ldcg(reinterpret_cast<const float4*>(at1 + (c0 + j) * 256));
                                        upv1[j] = __ldcg(reinterpret_cast<const float4*>(at1 + (c0 + j) * 256 + 128));
                                    }
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                add4(gate[j], gate1[j]);
                                add4(upv[j], upv1[j]);
                                finish(gate[j], upv[j], c0 + j);
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int c0 = c_first + q; c0 < g.n; c0 += c_step) {
                            float4 gate = make_float4(0.f, 0.f, 0.f, 0.f), upv = gate;
#pragma unroll 1
                            for (int p0 = 0; p0 < parts; p0 += 8) {
                                float4 vg[8], vu[8];
                                const unsigned from = static_cast<unsigned>(part_at(min(p0 + (lane & 7), parts - 1)));
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const unsigned at = __shfl_sync(FULL_MASK, from, i);
                                    vg[i] = vu[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                                    if (p0 + i < parts) {
                                        const float* src = mine_at + at + c0 * 256;
                                        vg[i] = __ldcg(reinterpret_cast<const float4*>(src));
                                        vu[i] = __ldcg(reinterpret_cast<const float4*>(src + 128));
                                    }
                                }
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    add4(gate, vg[i]);
                                    add4(upv, vu[i]);
                                }
                            }
                            finish(gate, upv, c0);
                        }
                    }
                    if (shared) {
                        finishers_barrier();
                        if (q == 0 && lane == 0) leave(count, parts);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.part_empty[part.stage]);
                part.next(ML_PARTS);
                return true;
            });
            sum_output<NT>(p, s, (8 + warp - ML_FIN_WARP0) * static_cast<int>(gridDim.x) + cta, ok, abort_flag, lane);
        } else {
            // ---------------------------------------------------------------- promotion
            regs_inc<ML_EPI_REGS>();
            const int ew = warp - ML_EPI_WARP0;
            const int q = warp & 3;             // TMEM lane quarter
            const int h = ew >> 2;              // warpgroup: 8-column groups h, h + 2, ...
            const int r = q * 32 + lane;        // row of each 128-row tile
            const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(8 * h);
            Ring acc, slot, part;

            float a0[NG][8], a1[NG][8];
            auto clear = [&] {
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) a0[i][j] = a1[i][j] = 0.f;
            };
            // Promotion over a segment: sb0 / sb1 the two tiles' weight scales (by K block), 32 of them a load.
            auto promote = [&](const Seg& g, const float* sb0, const float* sb1) {
                float b0n = 0.f, b1n = 0.f;
                for (int kb = g.kb0; kb < g.kb0 + g.nkb; ++kb) {
                    const int k32 = (kb - g.kb0) & 31;
                    if (k32 == 0 && kb + lane < g.kb0 + g.nkb) {
                        b0n = __ldg(sb0 + kb + lane);
                        b1n = __ldg(sb1 + kb + lane);
                    }
                    bool got = (static_cast<unsigned>(mbar_try_wait(&s.acc_full[acc.stage], acc.phase)) &
                                static_cast<unsigned>(mbar_try_wait(&s.scale_full[slot.stage], slot.phase))) != 0u;
                    if (!got)
                        got = wait_bounded(&s.acc_full[acc.stage], acc.phase, abort_flag, p.status, p.wait_limit_ns) &&
                              wait_bounded(&s.scale_full[slot.stage], slot.phase, abort_flag, p.status, p.wait_limit_ns);
                    if (!__all_sync(FULL_MASK, got)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t taddr = lane_addr + static_cast<uint32_t>(acc.stage * 2 * NT);
                    // (columns past the chunk's tokens are loaded too, and not used: a branch between the loads and
                    // their wait would let the compiler move registers that the loads have yet to write)
                    uint32_t p0[NG][8], p1[NG][8];
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        tmem_ld_x8(taddr + 16 * i, p0[i]);
                        tmem_ld_x8(taddr + NT + 16 * i, p1[i]);
                    }
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.acc_empty[acc.stage]);
                    acc.next(NACC);
                    const float b0 = __shfl_sync(FULL_MASK, b0n, k32), b1 = __shfl_sync(FULL_MASK, b1n, k32);
                    const float* sx = s.scales[slot.stage];
                    slot.next(SLOTS);
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        if ((2 * i + h) * 8 < g.n) {
                            const float4 u = *reinterpret_cast<const float4*>(sx + (2 * i + h) * 8);
                            const float4 w = *reinterpret_cast<const float4*>(sx + (2 * i + h) * 8 + 4);
                            const float v[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                a0[i][j] = fmaf(__uint_as_float(p0[i][j]), v[j] * b0, a0[i][j]);
                                a1[i][j] = fmaf(__uint_as_float(p1[i][j]), v[j] * b1, a1[i][j]);
                            }
                        }
                    }
                }
            };
            // f(column of the chunk, accumulators) for this thread's valid columns
            auto columns = [&](int n, auto&& f) {
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if ((2 * i + h) * 8 + j < n) f((2 * i + h) * 8 + j, a0[i][j], a1[i][j]);
            };

            for_segments<NT>(p, s, nothing, [&](auto tag, int l, const Line& ln, const Seg& g) {
                clear();
                if constexpr (decltype(tag)::value == 1) {
                    const float* sb = p.s13 + (static_cast<size_t>(g.e) * 2 * ln.blocks + g.blk) * ln.kbs;
                    if (ok) promote(g, sb, sb + static_cast<size_t>(ln.blocks) * ln.kbs);
                    if (ok) {
                        const bool got = wait_bounded(&s.part_empty[part.stage], part.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns);
                        ok = __all_sync(FULL_MASK, got) != 0;
                    }
                    float* dst = g.nkb < ln.kbs ? divided_slot(cta, l, static_cast<unsigned>(g.unit) * ln.kbs) : slot_at(cta, 4 + part.stage);
                    columns(g.n, [&](int col, float& x0, float& x1) {
                        __stcg(dst + col * 256 + r, x0);
                        __stcg(dst + col * 256 + 128 + r, x1);
                    });
                    __syncwarp();
                    if (lane == 0) {
                        if (g.nkb < ln.kbs) {
                            const unsigned u0 = static_cast<unsigned>(g.unit) * ln.kbs;
                            const int c_lo = cta_of(u0, ln);
                            if (finished_together(ln, g.n, cta_of(u0 + ln.kbs - 1, ln) - c_lo + 1)) red_add_release(p.count + l * ML_MAX_CTAS + c_lo, 1u);
                        }
                        mbar_arrive(&s.part_full[part.stage]);
                    }
                    part.next(ML_PARTS);
                } else {
                    const float* sb = p.s2 + (static_cast<size_t>(g.e) * (p.H / 128) + 2 * g.blk) * ln.kbs;
                    if (ok) promote(g, sb, g.two ? sb + ln.kbs : sb);
                    // the unit's (part of the) products, by gathered row
                    const int parts = most_parts(ln);
                    const int at = g.kb0 == 0 ? 0 : cta - cta_of(static_cast<unsigned>(g.unit) * ln.kbs, ln);
                    const Line& first = s.line[2];
                    const int base = l == 2 ? 0 : static_cast<int>((s.chunk[first.nc] >> 10) & 0xfffu);
                    const int before = l == 2 ? 0 : base * most_parts(first);
                    const size_t width = static_cast<size_t>(ln.blocks) * 256;
                    float* y = p.y + (static_cast<size_t>(before) + (g.off - base) * parts + at) * width + g.blk * 256 + r;
                    columns(g.n, [&](int col, float& x0, float& x1) {
                        __stcg(y + static_cast<size_t>(col) * parts * width, x0);
                        if (g.two) __stcg(y + static_cast<size_t>(col) * parts * width + 128, x1);
                    });
                }
                return true;
            });
            line_done(3);

            sum_output<NT>(p, s, (warp - ML_EPI_WARP0) * static_cast<int>(gridDim.x) + cta, ok, abort_flag, lane);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// Gathered rows at most: every assignment, and every met expert's rows rounded up to 4.
int rows_cap(int T, int k, int E) {
    const int a = T * k;
    return (a + 3 * (a < E ? a : E) + 3) / 4 * 4;
}

int tokens_per_chunk(int T) { return T <= 16 ? 16 : (T <= 32 ? 32 : 64); }

// most_parts() of a phase-2 line of `nc` chunks over at most ML_MAX_CTAS CTAs.
int64_t parts_bound(int nc, int H, int I) {
    const int64_t kbs = I / 128, total = static_cast<int64_t>(nc) * ((H + 255) / 256) * kbs;
    if (total == 0) return 1;
    const int64_t least = total / std::min<int64_t>(total, ML_MAX_CTAS);
    return (kbs - 1 + least - 1) / least + 1;
}

// Rows of y that any routing of these sizes can need: for every number of chunks, the halves' rows (at most NT a
// chunk, rows_cap together) times their parts, the half of more parts filled first. Every call asks for it, so the
// search ends at the number of chunks whose smaller half can hold every row: from there on a half has all rows times
// its parts, and more chunks have no more parts. (All numbers of chunks took 22 us for 64 tokens of 16 experts.)
int64_t y_rows(int T, int k, int E, int H, int I) {
    const int nt = tokens_per_chunk(T), a = T * k;
    const int64_t cap = rows_cap(T, k, E);
    int64_t most = 0;
    bool full = false;
    for (int i = 0; i < 2 * a && !(full && i % 2 == 0); ++i) {
        const int chunks = i / 2 + 1, ca = i % 2 ? chunks : (chunks * 5 + 7) / 8, cb = chunks - ca;
        full = full || static_cast<int64_t>(cb) * nt >= cap;
        const int64_t pa = parts_bound(ca, H, I), pb = cb ? parts_bound(cb, H, I) : 1;
        const int64_t ra = std::min<int64_t>(cap, static_cast<int64_t>(ca) * nt), rb = std::min<int64_t>(cap, static_cast<int64_t>(cb) * nt);
        const int64_t rows = pb >= pa ? rb * pb + std::min(ra, cap - rb) * pa : ra * pa + std::min(rb, cap - ra) * pb;
        most = std::max(most, rows);
    }
    return most;
}

struct Layout {
    int64_t xg, sx, hg, sh, parts, y, bytes;
};

int64_t up(int64_t v) { return (v + 1023) / 1024 * 1024; }

Layout layout(int T, int k, int E, int H, int I) {
    const int64_t rows = rows_cap(T, k, E);
    Layout l;
    l.xg = ML_FIXED;
    l.sx = l.xg + up(rows * H);
    l.hg = l.sx + up(rows * (H / 128) * 4);
    l.sh = l.hg + up(rows * I);
    l.parts = l.sh + up(rows * (I / 128) * 4);
    l.y = l.parts + static_cast<int64_t>(ML_MAX_CTAS) * ML_SLOTS * tokens_per_chunk(T) * 256 * 4;
    l.bytes = l.y + y_rows(T, k, E, H, I) * ((H + 255) / 256) * 256 * 4;
    return l;
}

bool sizes_ok(int T, int k, int E, int H, int I) {
    if (T < 1 || T > ML_MAX_T || k < 1 || static_cast<int64_t>(T) * k > ML_MAX_A || E < 1 || E > ML_MAX_E || H < 128 || I < 128 || H % 128 || I % 128)
        return false;
    // rows of the stacked weights, and a line's stages times the CTAs, in 32 bits
    const int64_t chunks = T * k;
    return static_cast<int64_t>(E) * 2 * I <= INT32_MAX && static_cast<int64_t>(E) * H <= INT32_MAX &&
           chunks * (I / 128) * (H / 128) <= (int64_t{1} << 32) / ML_MAX_CTAS - 1;
}

template <int NT>
cudaError_t launch_moe(const CUtensorMap& w13, const CUtensorMap& w2, const CUtensorMap& x, const CUtensorMap& h, const MoeParams& p,
                       int ctas, cudaStream_t stream) {
    using C = MlCfg<NT>;
    auto kern = moe_layer_kernel<NT>;
    static std::mutex mu;
    static int ready[kMaxDevices] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::DYN_SMEM);
            if (e != cudaSuccess) return e;
            // as in dg_launch.cuh: the setmaxnreg split must equal what the kernel launches with
            cudaFuncAttributes fa;
            e = cudaFuncGetAttributes(&fa, kern);
            if (e != cudaSuccess) return e;
            if (fa.numRegs * ML_THREADS != (ML_CTRL_REGS + ML_FIN_REGS) * 128 + ML_EPI_REGS * 256) return cudaErrorInvalidConfiguration;
            ready[dev] = 1;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(ML_THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::DYN_SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, w13, w2, x, h, p);
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

int64_t dg_moe_layer_workspace(int T, int k, int E, int H, int I) {
    if (T == 0) return 0;
    return sizes_ok(T, k, E, H, I) ? layout(T, k, E, H, I).bytes : -1;
}

dg_status dg_moe_layer(const void* x, const int32_t* ids, const float* weights, const uint8_t* W13, const float* s13,
                       const uint8_t* W2, const float* s2, const void* residual, void* out, void* workspace,
                       int64_t workspace_bytes, int T, int k, int E, int H, int I, int act, cudaStream_t stream) {
    if (T < 0 || k < 0 || E < 0 || H < 0 || I < 0 || act < DG_ACT_NONE || act > DG_ACT_SILU) return DG_INVALID_ARG;
    if (T == 0) return DG_OK;
    if (!sizes_ok(T, k, E, H, I)) return DG_UNSUPPORTED_SHAPE;
    if (!x || !ids || !weights || !W13 || !s13 || !W2 || !s2 || !out || !workspace) return DG_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(W13, 16) || !aligned(W2, 16) || !aligned(residual, 16) || !aligned(out, 16) ||
        !aligned(ids, 4) || !aligned(weights, 4) || !aligned(s13, 4) || !aligned(s2, 4) || !aligned(workspace, 256))
        return DG_MISALIGNED;
    const Layout l = layout(T, k, E, H, I);
    if (workspace_bytes < l.bytes) return DG_INVALID_ARG;
    DeviceInfo dev;
    const dg_status st = common_prologue(&dev);
    if (st != DG_OK) return st;

    char* ws = static_cast<char*>(workspace);
    MoeParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.ids = ids;
    p.weights = weights;
    p.s13 = s13;
    p.s2 = s2;
    p.residual = static_cast<const __nv_bfloat16*>(residual);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.barrier = reinterpret_cast<unsigned*>(ws);
    p.count = reinterpret_cast<unsigned*>(ws + 1024);
    p.xg = reinterpret_cast<uint8_t*>(ws + l.xg);
    p.sx = reinterpret_cast<float*>(ws + l.sx);
    p.hg = reinterpret_cast<uint8_t*>(ws + l.hg);
    p.sh = reinterpret_cast<float*>(ws + l.sh);
    p.parts = reinterpret_cast<float*>(ws + l.parts);
    p.y = reinterpret_cast<float*>(ws + l.y);
    p.status = dev.status;
    p.T = T;
    p.k = k;
    p.E = E;
    p.H = H;
    p.I = I;
    p.rows_cap = rows_cap(T, k, E);
    p.act = act;
    const ArmedFault armed = take_armed_fault();
    p.wait_limit_ns = armed.wait_limit_ns;
    p.fault = armed.fault;
    CUtensorMap w13, w2, mx, mh;
    if (make_operand_map(&w13, W13, static_cast<int64_t>(E) * 2 * I, H, 128) != DG_OK ||
        make_operand_map(&w2, W2, static_cast<int64_t>(E) * H, I, 128) != DG_OK ||
        make_operand_map(&mx, p.xg, p.rows_cap, H, 16) != DG_OK || make_operand_map(&mh, p.hg, p.rows_cap, I, 16) != DG_OK)
        return DG_CUDA_ERROR;
    const int ctas = dev.sms < ML_MAX_CTAS ? dev.sms : ML_MAX_CTAS;
    cudaError_t e;
    switch (tokens_per_chunk(T)) {
        case 16: e = launch_moe<16>(w13, w2, mx, mh, p, ctas, stream); break;
        case 32: e = launch_moe<32>(w13, w2, mx, mh, p, ctas, stream); break;
        default: e = launch_moe<64>(w13, w2, mx, mh, p, ctas, stream); break;
    }
    return e == cudaSuccess ? DG_OK : DG_CUDA_ERROR;
}

}  // extern "C"
