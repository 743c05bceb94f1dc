// A whole mixture-of-experts layer for a few tokens in one launch (dg_moe_layer):
//
//   out[t] = residual[t] + sum_j w[t,j] W2[e] . Q(act(g) * u),   (g; u) = W13[e] . Q(x[t]),   e = ids[t,j]
//
// What bounds it is streaming the met experts' weights, 3 H I bytes each, from HBM; the tokens, the hidden
// activations and every partial sum stay in L2. So the whole layer is one persistent kernel of one CTA per
// SM whose weight stream stops for nothing but a full ring:
//
//   * Split. A stage is 256 weight rows x one 128-wide K block, 32 KB. The stages of a phase (phase 1: W13,
//     phase 2: W2) form a line, unit after unit, and CTA c of G takes the c-th G-th of it, whatever the
//     number of met experts: every SM streams the same bytes, to one stage. Parts of a unit that the cuts
//     divide are summed in the order of the CTAs, so the result does not depend on timing.
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
//     quantises 128 hidden values per token. A phase-2 unit is 256 output rows of one expert, written as FP32
//     per gathered row; after the last grid barrier all CTAs sum each token's experts, weighted, in order.
//
// Warp roles: warp 0 streams weights, warp 2 tokens and their scales, warp 1 issues MMAs, warp 3 crosses the grid
// barriers, warps 4..11 quantise the tokens, promote and finish units. Every wait is bounded as in dg_gemm_kernel; a CTA that gives up still arrives at the grid
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
constexpr int ML_MAX_CTAS = 192;               // CTAs (workspace slots) at most; one per SM
constexpr int ML_MAX_ROWS = ML_MAX_A + 3 * ML_MAX_A;   // gathered rows: every expert's start on a multiple of 4
constexpr int ML_W_BYTES = 2 * 128 * BK;       // weights of a stage
constexpr int ML_FIXED = 4096;                 // workspace: barrier word and counters
constexpr int ML_BARRIERS = 4;                 // grid barriers: tokens, hidden of either half, products
constexpr unsigned FULL_MASK = 0xffffffffu;

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
    float* parts;          // [CTA][phase-1 line][2][NT][256]: parts of divided phase-1 units
    float* y;              // [gathered row][part][pairs * 256] weighted by nothing yet
    unsigned* barrier;     // grid barrier word
    unsigned* count;       // [phase-1 line][CTA]: parts written of the unit that the CTA's share ends in
    int* status;
    int T, k, E, H, I, rows_cap, act;
    unsigned long long wait_limit_ns;
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
    static constexpr int TABLES = 4 * ML_MAX_A + 2 * ML_MAX_A + ML_MAX_ROWS + 4 * 4 * (ML_MAX_CTAS + 1);
    static constexpr int STATIC_RESERVE = TABLES + SLOTS * NT * 4 + 2 * 32 * 4 * 6 + 640;
    static constexpr int STAGES_FIT = ring_stages(STAGE_BYTES, 0, 0, STATIC_RESERVE);
    static constexpr int STAGES = STAGES_FIT > 6 ? 6 : STAGES_FIT;
    static constexpr int DYN_SMEM = 1024 + STAGES * STAGE_BYTES;
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

__device__ __forceinline__ void epi_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// One thread's arrival at the barrier of all CTAs, and its wait. CTA 0 adds what carries the others' ones
// into the top bit, so the bit flips when the last one arrives and the low bits are back at zero: the word
// needs no reset between barriers or launches. The CTAs are co-resident (cooperative launch); the wait ends
// by itself all the same.
__device__ __forceinline__ bool grid_barrier(unsigned* word, volatile int* abort_flag, int* status, uint64_t limit_ns) {
    const unsigned add = blockIdx.x == 0 ? 0x80000000u - (gridDim.x - 1) : 1u;
    const unsigned old = atom_add_acq_rel(word, add);
    const uint64_t t0 = global_timer_ns();
    const uint64_t limit = limit_ns ? limit_ns : WAIT_LIMIT_NS;
    for (int i = 0; i < (1 << 26); ++i) {
        if ((ld_acquire(word) ^ old) & 0x80000000u) return true;
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

template <int NT>
struct Shared {
    uint64_t full[MlCfg<NT>::STAGES], empty[MlCfg<NT>::STAGES];
    uint64_t acc_full[MlCfg<NT>::NACC], acc_empty[MlCfg<NT>::NACC];
    uint64_t scale_full[MlCfg<NT>::SLOTS];
    uint64_t done[ML_BARRIERS], go[ML_BARRIERS];                   // this CTA's work before a grid barrier is done; it is crossed
    uint32_t tmem;
    int abort, chunks, rows, last;
    __align__(16) float scales[MlCfg<NT>::SLOTS][NT];
    uint32_t amax[2][4][32];                    // [warpgroup][warp][column] of a unit being finished
    float unit_scale[2][2][32];                 // [warpgroup]: each column's divisor and its reciprocal
    uint32_t chunk[ML_MAX_A];
    uint16_t row_of[ML_MAX_A];                  // gathered row of an assignment (t * k + j); 0xffff: no expert
    uint8_t token[ML_MAX_ROWS];                 // token of a gathered row
    uint32_t share[4][ML_MAX_CTAS + 1];         // first stage of each CTA's share of each line
};

// The lines: phase 1 of the first half of the chunks, of the second half; phase 2 of the first, of the second.
struct Line {
    int c0, nc;            // chunks
    int kbs, blocks;       // K blocks of a unit; units per chunk
    int total;             // stages
};

__device__ __forceinline__ Line line_of(const MoeParams& p, int chunks, int l) {
    Line n;
    const int half = (chunks + 1) / 2;
    n.c0 = (l & 1) ? half : 0;
    n.nc = (l & 1) ? chunks - half : half;
    n.kbs = (l < 2 ? p.H : p.I) / 128;
    n.blocks = l < 2 ? p.I / 128 : (p.H + 255) / 256;
    n.total = n.nc * n.blocks * n.kbs;
    return n;
}

// CTAs that share a line (every one of them at least one stage, so that no CTA between two parts of a unit is
// empty), where a CTA's share starts, and whose share a stage is in. The host keeps total * CTAs in 32 bits.
__device__ __forceinline__ unsigned sharers(int total) { return min(static_cast<unsigned>(total), gridDim.x); }
__device__ __forceinline__ unsigned share_start(int total, unsigned cta) {
    const unsigned n = sharers(total);
    return cta >= n ? total : static_cast<unsigned>(total) * cta / n;
}
__device__ __forceinline__ int cta_of(unsigned pos, int total) {
    return static_cast<int>(((pos + 1) * sharers(total) - 1) / static_cast<unsigned>(total));
}
// Parts that a unit of the line can have at most.
__device__ __forceinline__ int most_parts(const Line& n) {
    if (n.total == 0) return 1;
    const int least = static_cast<int>(static_cast<unsigned>(n.total) / sharers(n.total));
    return (n.kbs - 1 + least - 1) / least + 1;
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
        const Line ln = line_of(p, s.chunks, l);
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
        const Line ln = line_of(p, s.chunks, l);
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
// the assignments of its expert, in order). Every CTA makes the same tables from the same ids. `scratch`: 8 KB.
template <int NT>
__device__ void make_tables(const MoeParams& p, Shared<NT>& s, uint32_t* scratch) {
    uint32_t* offset = scratch;                                          // rows of an expert, then its first row
    int32_t* ids = reinterpret_cast<int32_t*>(scratch + ML_MAX_E);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int A = p.T * p.k;
    for (int a = tid; a < A; a += THREADS) {
        const int e = __ldg(p.ids + a);
        ids[a] = e >= 0 && e < p.E ? e : -1;
    }
    for (int e = tid; e < p.E; e += THREADS) offset[e] = 0;
    __syncthreads();
    if (warp == EPI_WARP0) {
        for (int base = 0; base < A; base += 32) {
            const int a = base + lane;
            const int e = a < A ? ids[a] : -1;
            const unsigned same = __match_any_sync(FULL_MASK, e);
            const int rank = __popc(same & ((1u << lane) - 1u));
            const uint32_t before = e >= 0 ? offset[e] : 0u;
            __syncwarp();
            if (a < A) s.row_of[a] = e >= 0 ? static_cast<uint16_t>(before + rank) : 0xffffu;
            if (e >= 0 && rank == 0) offset[e] = before + __popc(same);
            __syncwarp();
        }
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
            if (e < p.E) offset[e] = static_cast<uint32_t>(r0);
            for (int i = 0; i < c_own; ++i) s.chunk[c0 + i] = pack_chunk(e, r0 + i * NT, min(NT, n - i * NT));
            rows += __shfl_sync(FULL_MASK, r, 31);
            chunks += __shfl_sync(FULL_MASK, c, 31);
        }
        if (lane == 0) {
            s.chunks = chunks;
            s.rows = rows;
        }
    }
    __syncthreads();
    for (int a = tid; a < A; a += THREADS) {
        if (s.row_of[a] != 0xffffu) {
            const uint32_t r = offset[ids[a]] + s.row_of[a];
            s.row_of[a] = static_cast<uint16_t>(r);
            s.token[r] = static_cast<uint8_t>(a / p.k);
        }
    }
    for (int i = tid; i < 4 * static_cast<int>(gridDim.x + 1); i += THREADS) {
        const int l = i / static_cast<int>(gridDim.x + 1), c = i - l * static_cast<int>(gridDim.x + 1);
        const Line n = line_of(p, s.chunks, l);
        s.share[l][c] = n.total ? share_start(n.total, static_cast<unsigned>(c)) : 0u;
    }
}

template <int NT>
__global__ void __launch_bounds__(THREADS, 1)
moe_layer_kernel(const __grid_constant__ CUtensorMap map_w13, const __grid_constant__ CUtensorMap map_w2,
                 const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_h,
                 const __grid_constant__ MoeParams p) {
    using C = MlCfg<NT>;
    constexpr int STAGES = C::STAGES, NACC = C::NACC, NG = C::NG, SLOTS = C::SLOTS;
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
            mbar_init(&s.full[i], 2);           // the weight and the token producer
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < NACC; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], EPI_WARPS);
        }
        for (int i = 0; i < SLOTS; ++i) mbar_init(&s.scale_full[i], 1);
        for (int i = 0; i < ML_BARRIERS; ++i) {
            mbar_init(&s.done[i], EPI_WARPS);
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
    constexpr int AHEAD = 3;
    const int kbs_x = p.H / 128, blocks_x = p.T * kbs_x, stride_x = static_cast<int>(gridDim.x) * EPI_WARPS;
    const int first_x = cta + (warp - EPI_WARP0) * static_cast<int>(gridDim.x);
    uint2 ahead[AHEAD];
    if (warp >= EPI_WARP0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int w = first_x + i * stride_x;
            if (w < blocks_x) ahead[i] = *reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(w) * 128 + lane * 4);
        }
    }
    make_tables<NT>(p, s, reinterpret_cast<uint32_t*>(smem));   // before the ring is in use
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s.tmem;
    volatile int* abort_flag = &s.abort;
    const auto nothing = [](int) { return true; };

    if (warp < EPI_WARP0) {
        regs_dec<CTRL_REGS>();
        const bool issuer = elect_one();
        if (warp == 0) {
            // ---------------------------------------------------------------- weights
            Ring ring;
            uint32_t issued = 0, issued_parity = 0;
            bool ok = for_segments<NT>(p, s, nothing, [&](auto tag, int, const Line&, const Seg& g) {
                const CUtensorMap* map = decltype(tag)::value == 1 ? &map_w13 : &map_w2;
                for (int kb = g.kb0; kb < g.kb0 + g.nkb; ++kb) {
                    const bool got = wait_bounded(&s.empty[ring.stage], ring.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns);
                    if (!__all_sync(FULL_MASK, got)) return false;
                    if (issuer) {
                        uint8_t* dst = smem + ring.stage * ML_W_BYTES;
                        mbar_arrive_expect_tx(&s.full[ring.stage], g.two ? ML_W_BYTES : ML_W_BYTES / 2);
                        tma_load_2d(map, &s.full[ring.stage], dst, kb * BK, g.row0);
                        if (g.two) tma_load_2d(map, &s.full[ring.stage], dst + 128 * BK, kb * BK, g.row1);
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
                    if (issued & (1u << i)) drain_wait(&s.full[i], (issued_parity >> i) & 1u);
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA issue
            Ring ring, acc;
            int last = -1;
            uint32_t last_parity = 0;
            const uint32_t w_base = smem_u32(smem), t_base = smem_u32(smem_t);
            const bool ok = for_segments<NT>(p, s, nothing, [&](auto, int, const Line&, const Seg& g) {
                const uint32_t idesc = idesc_e4m3_f32(128, (g.n + 15) & ~15);
                for (int kb = 0; kb < g.nkb; ++kb) {
                    const bool got = wait_bounded(&s.acc_empty[acc.stage], acc.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns) &&
                                     wait_bounded(&s.full[ring.stage], ring.phase, abort_flag, p.status, p.wait_limit_ns);
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
                    last = acc.stage;
                    last_parity = acc.phase;
                    ring.next(STAGES);
                    acc.next(NACC);
                    __syncwarp();
                }
                return true;
            });
            if (!ok && last >= 0 && issuer) drain_wait(&s.acc_full[last], last_parity);
        } else if (warp == 2) {
            // ---------------------------------------------------------------- tokens
            Ring ring, slot;
            for_segments<NT>(p, s, [&](int l) {
                if (l == 1) return true;
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
                        mbar_arrive_expect_tx(&s.full[ring.stage], static_cast<uint32_t>(boxes * 16 * BK));
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(map, &s.full[ring.stage], dst + b * 16 * BK, kb * BK, g.off + b * 16);
                        mbar_arrive_expect_tx(&s.scale_full[slot.stage], scale_bytes);
                        bulk_load(s.scales[slot.stage], scales + static_cast<size_t>(kb) * p.rows_cap, scale_bytes, &s.scale_full[slot.stage]);
                    }
                    ring.next(STAGES);
                    slot.next(SLOTS);
                    __syncwarp();
                }
                return true;
            });
        } else if (warp == 3) {
            // ---------------------------------------------------------------- grid barriers
            if (lane == 0) {
#pragma unroll 1
                for (int b = 0; b < ML_BARRIERS; ++b) {
                    wait_bounded(&s.done[b], 0, abort_flag, p.status, p.wait_limit_ns);
                    const bool got = grid_barrier(p.barrier, abort_flag, p.status, p.wait_limit_ns);
                    fence_proxy_async_all();
                    if (got) mbar_arrive(&s.go[b]);
                }
            }
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------------- promotion, units, output
        regs_inc<EPI_REGS>();
        // ---- the tokens' codes and scales, to every row that they are gathered to
        auto quantise = [&](int w, uint2 u) {
            const int t = w / kbs_x, kb = w - t * kbs_x;
            const float a = bf16_lo(u.x), b = bf16_hi(u.x), c = bf16_lo(u.y), d = bf16_hi(u.y);
            const BlockScale sc = block_scale(__reduce_max_sync(FULL_MASK, max(max(abs_bits(a), abs_bits(b)), max(abs_bits(c), abs_bits(d)))));
            const uint32_t code = quantise4(a, b, c, d, sc);
#pragma unroll 4
            for (int j = 0; j < p.k; ++j) {
                const uint32_t row = s.row_of[t * p.k + j];
                if (row == 0xffffu) continue;
                *reinterpret_cast<uint32_t*>(p.xg + static_cast<size_t>(row) * p.H + kb * 128 + lane * 4) = code;
                if (lane == 0) p.sx[static_cast<size_t>(kb) * p.rows_cap + row] = sc.s;
            }
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (first_x + i * stride_x < blocks_x) quantise(first_x + i * stride_x, ahead[i]);
        for (int w = first_x + AHEAD * stride_x; w < blocks_x; w += stride_x)
            quantise(w, *reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(w) * 128 + lane * 4));
        const int tid = static_cast<int>(threadIdx.x) - EPI_WARP0 * 32;   // 0 .. 255
        const int ew = warp - EPI_WARP0;
        const int q = warp & 3;                 // TMEM lane quarter
        const int h = ew >> 2;                  // warpgroup: 8-column groups h, h + 2, ...
        const int r = q * 32 + lane;            // row of each 128-row tile
        const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(8 * h);
        bool ok = true;
        Ring acc, slot;

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
                uint32_t p0[NG][8], p1[NG][8];
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if ((2 * i + h) * 8 < g.n) {
                        tmem_ld_x8(taddr + 16 * i, p0[i]);
                        tmem_ld_x8(taddr + NT + 16 * i, p1[i]);
                    }
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
        auto part_of = [&](int c, int l, int which) { return p.parts + static_cast<size_t>((c * 2 + l) * 2 + which) * (NT * 256); };
        auto line_done = [&](int b) {
            // (codes and scales are read by TMA; the grid barrier's arrival releases the CTA's writes)
            fence_proxy_async_all();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.done[b]);
        };
        // The sum of a divided unit's parts in the order of its CTAs, if this CTA's came last: every thread's
        // writes of the part are visible to whoever sees the full count.
        auto whole = [&](int l, const Line& ln, const Seg& g) {
            const unsigned u0 = static_cast<unsigned>(g.unit) * ln.kbs;
            const int c_lo = cta_of(u0, ln.total), c_hi = cta_of(u0 + ln.kbs - 1, ln.total);
            // the unit is the first of every CTA but the one in whose share it starts
            float* mine = part_of(cta, l, u0 < s.share[l][cta] ? 0 : 1);
            columns(g.n, [&](int col, float& x0, float& x1) {
                __stcg(mine + col * 256 + r, x0);
                __stcg(mine + col * 256 + 128 + r, x1);
            });
            epi_barrier();
            if (tid == 0) {
                // (releases what the barrier has gathered from the CTA's threads, acquires the others' parts)
                unsigned* count = p.count + l * ML_MAX_CTAS + c_lo;
                const bool last = atom_add_acq_rel(count, 1u) == static_cast<unsigned>(c_hi - c_lo);
                if (last) *count = 0;           // as the next launch expects it
                s.last = last ? 1 : 0;
            }
            epi_barrier();
            if (s.last == 0) return false;
            clear();
            for (int c = c_lo; c <= c_hi; ++c) {
                const float* part = part_of(c, l, u0 < s.share[l][c] ? 0 : 1);
                columns(g.n, [&](int col, float& x0, float& x1) {
                    x0 += __ldcg(part + col * 256 + r);
                    x1 += __ldcg(part + col * 256 + 128 + r);
                });
            }
            return true;
        };

        line_done(0);
        for_segments<NT>(p, s, [&](int l) {
            if (l == 1 || l == 2) line_done(l);
            return true;
        }, [&](auto tag, int l, const Line& ln, const Seg& g) {
            clear();
            if constexpr (decltype(tag)::value == 1) {
                const int blocks = ln.blocks;
                const float* sb = p.s13 + (static_cast<size_t>(g.e) * 2 * blocks + g.blk) * ln.kbs;
                if (ok) promote(g, sb, sb + static_cast<size_t>(blocks) * ln.kbs);
                if (g.nkb < ln.kbs && !whole(l, ln, g)) return true;
                // hidden activations of 128 rows of I: act(gate) * up, then codes by the largest of the 128
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if ((2 * i + h) * 8 < g.n) {
                        act_values<8>(p.act, a0[i]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            a0[i][j] *= a1[i][j];
                            const uint32_t top = __reduce_max_sync(FULL_MASK, abs_bits(a0[i][j]));
                            if (lane == 0) s.amax[h][q][i * 8 + j] = top;
                        }
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(2 + h) : "memory");
                if (q == 0) {                   // one lane a column (NT / 2 of them)
                    const int col = (2 * (lane >> 3) + h) * 8 + (lane & 7);
                    if (lane < 8 * NG && col < g.n) {
                        const BlockScale k = block_scale(max(max(s.amax[h][0][lane], s.amax[h][1][lane]), max(s.amax[h][2][lane], s.amax[h][3][lane])));
                        s.unit_scale[h][0][lane] = k.d;
                        s.unit_scale[h][1][lane] = k.r;
                        p.sh[static_cast<size_t>(g.blk) * p.rows_cap + g.off + col] = k.s;
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(2 + h) : "memory");
#pragma unroll
                for (int i = 0; i < NG; ++i) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int col = (2 * i + h) * 8 + j;
                        if (col < g.n) {
                            const float v = quotient(a0[i][j], s.unit_scale[h][0][i * 8 + j], s.unit_scale[h][1][i * 8 + j]);
                            p.hg[static_cast<size_t>(g.off + col) * p.I + g.blk * 128 + r] = static_cast<uint8_t>(pack_e4m3x2(v, 0.f) & 0xffu);
                        }
                    }
                }
                // (the next unit's first barrier keeps its scales from these reads)
            } else {
                const float* sb = p.s2 + (static_cast<size_t>(g.e) * (p.H / 128) + 2 * g.blk) * ln.kbs;
                if (ok) promote(g, sb, g.two ? sb + ln.kbs : sb);
                // the unit's (part of the) products, by gathered row
                const int parts = most_parts(ln);
                const int part = g.kb0 == 0 ? 0 : cta - cta_of(static_cast<unsigned>(g.unit) * ln.kbs, ln.total);
                const Line first = line_of(p, s.chunks, 2);
                const int base = l == 2 ? 0 : static_cast<int>((s.chunk[first.nc] >> 10) & 0xfffu);
                const int before = l == 2 ? 0 : base * most_parts(first);
                const size_t width = static_cast<size_t>(ln.blocks) * 256;
                float* y = p.y + (static_cast<size_t>(before) + (g.off - base) * parts + part) * width + g.blk * 256 + r;
                columns(g.n, [&](int col, float& x0, float& x1) {
                    __stcg(y + static_cast<size_t>(col) * parts * width, x0);
                    if (g.two) __stcg(y + static_cast<size_t>(col) * parts * width + 128, x1);
                });
            }
            return true;
        });
        line_done(3);
        {
            const bool got = wait_bounded(&s.go[3], 0, abort_flag, p.status, p.wait_limit_ns);
            ok = __all_sync(FULL_MASK, got) != 0;
        }
        // ---- output: a warp takes 128 columns of a token and adds up its experts in the order of its slots
        if (ok) {
            const Line la = line_of(p, s.chunks, 2), lb = line_of(p, s.chunks, 3);
            const int pa = most_parts(la), pb = most_parts(lb);
            const int base_b = lb.nc ? static_cast<int>((s.chunk[la.nc] >> 10) & 0xfffu) : s.rows;
            const int blocks = p.H / 128;
            const size_t width = static_cast<size_t>(la.blocks) * 256;
            for (int w = ew * static_cast<int>(gridDim.x) + cta; w < p.T * blocks; w += static_cast<int>(gridDim.x) * 8) {
                const int t = w / blocks, blk = w - t * blocks;
                const int col = blk * 128 + lane * 4;
                const size_t at = static_cast<size_t>(t) * p.H + col;
                uint2 res = make_uint2(0u, 0u);
                if (p.residual != nullptr) res = *reinterpret_cast<const uint2*>(p.residual + at);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int j0 = 0; j0 < p.k; j0 += 32) {
                    // lane j: where assignment j's sums lie (in rows of `width`), of how many parts, its weight
                    const int j = j0 + lane;
                    int first = 0, parts = 0;
                    float wt = 0.f;
                    const int row = j < p.k ? s.row_of[t * p.k + j] : 0xffff;
                    if (row != 0xffff) {
                        wt = __ldg(p.weights + t * p.k + j);
                        const bool b = row >= base_b;
                        const Line& ln = b ? lb : la;
                        // the row's chunk in its line: the last one that starts at or before it
                        int lo = ln.c0, hi = ln.c0 + ln.nc;
                        while (hi - lo > 1) {
                            const int mid = (lo + hi) >> 1;
                            if (static_cast<int>((s.chunk[mid] >> 10) & 0xfffu) <= row) lo = mid; else hi = mid;
                        }
                        const unsigned u0 = static_cast<unsigned>((blk >> 1) * ln.nc + lo - ln.c0) * ln.kbs;
                        parts = cta_of(u0 + ln.kbs - 1, ln.total) - cta_of(u0, ln.total) + 1;
                        first = b ? base_b * pa + (row - base_b) * pb : row * pa;
                    }
                    const int here = min(32, p.k - j0);
                    // eight assignments' first two parts are loaded together (a unit has more parts only where
                    // there are few stages in all)
                    for (int i0 = 0; i0 < here; i0 += 8) {
                        float4 v[8][2];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int f = __shfl_sync(FULL_MASK, first, (i0 + i) & 31), held = __shfl_sync(FULL_MASK, parts, (i0 + i) & 31);
                            const int n = i0 + i < here ? held : 0;
                            const float* src = p.y + static_cast<size_t>(f) * width + col;
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (c < n) v[i][c] = __ldcg(reinterpret_cast<const float4*>(src + c * width));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int f = __shfl_sync(FULL_MASK, first, (i0 + i) & 31), n = __shfl_sync(FULL_MASK, parts, (i0 + i) & 31);
                            const float u = __shfl_sync(FULL_MASK, wt, (i0 + i) & 31);
                            if (i0 + i >= here || n == 0) continue;
                            float4 d = make_float4(v[i][0].x + v[i][1].x, v[i][0].y + v[i][1].y, v[i][0].z + v[i][1].z, v[i][0].w + v[i][1].w);
                            const float* src = p.y + static_cast<size_t>(f) * width + col;
                            for (int c = 2; c < n; ++c) {
                                const float4 e = __ldcg(reinterpret_cast<const float4*>(src + static_cast<size_t>(c) * width));
                                d.x += e.x; d.y += e.y; d.z += e.z; d.w += e.w;
                            }
                            sum.x = fmaf(u, d.x, sum.x); sum.y = fmaf(u, d.y, sum.y);
                            sum.z = fmaf(u, d.z, sum.z); sum.w = fmaf(u, d.w, sum.w);
                        }
                    }
                }
                sum.x += bf16_lo(res.x); sum.y += bf16_hi(res.x); sum.z += bf16_lo(res.y); sum.w += bf16_hi(res.y);
                st_global_v2(p.out + at, pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
            }
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
// chunk, rows_cap together) times their parts, the half of more parts filled first.
int64_t y_rows(int T, int k, int E, int H, int I) {
    const int nt = tokens_per_chunk(T), a = T * k;
    const int64_t cap = rows_cap(T, k, E);
    int64_t most = 0;
    for (int chunks = 1; chunks <= a; ++chunks) {
        const int ca = (chunks + 1) / 2, cb = chunks - ca;
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
    l.y = l.parts + static_cast<int64_t>(ML_MAX_CTAS) * 4 * tokens_per_chunk(T) * 256 * 4;
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
            if (fa.numRegs * THREADS != CTRL_REGS * 128 + EPI_REGS * (THREADS - 128)) return cudaErrorInvalidConfiguration;
            ready[dev] = 1;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
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
