// A whole mixture-of-experts layer for a few tokens in one launch (dg_moe_layer):
//
//   out[t] = residual[t] + sum_j w[t,j] W2[e] . Q(act(g) * u),   (g; u) = W13[e] . Q(x[t]),   e = ids[t,j]
//
// What bounds it is streaming the met experts' weights, 3 H I bytes each, from HBM; the tokens, the hidden
// activations and every partial sum stay in L2. So the whole layer is one persistent kernel of one CTA per
// SM whose weight stream never stops for anything but a full ring:
//
//   * Split. The stages of a phase (phase 1: W13, phase 2: W2; a stage is 256 weight rows x one 128-wide K
//     block, 32 KB) form one line, unit after unit, and CTA c of G takes the c-th G-th of it, whatever the
//     number of met experts: every SM streams the same bytes, to one stage. A unit (phase 1: 128 gate rows
//     and their 128 up rows of one expert; phase 2: 256 rows of the output) that the cuts divide is summed
//     from the FP32 parts of its CTAs by whichever finishes last, always in the order of the CTAs, so that
//     the result does not depend on timing and nobody waits.
//   * Order. Phase 2 walks the output rows outermost and the experts within, so a CTA adds up its experts
//     for its rows on the spot and an output row block is finished by a handful of CTAs.
//   * Two grid barriers (the tokens are quantised; the hidden activations are complete) hold back only the
//     loads that depend on them: the weight producer runs ahead through both, its ring being 4 us of HBM.
//   * The products run transposed, weights as the MMA's 128 rows, a chunk of an expert's tokens (up to NT) as
//     its N, so the tensor cores see whole tiles for a single token. TMEM lane = weight row, column = token;
//     the promotion acc[token] += P * sx[token] * sb reads the 128x128 weight scale once per tile.
//
// Warp roles: warp 0 streams weights, warp 2 tokens (rows gathered per expert by phase 0), warp 1 issues MMAs,
// warp 3 crosses the grid barriers, warps 4..11 quantise the tokens (phase 0), promote, and finish units.
// Every wait is bounded as in dg_gemm_kernel; a CTA that gives up still arrives at the grid barriers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

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
constexpr unsigned FULL_MASK = 0xffffffffu;

struct MoeParams {
    const __nv_bfloat16* x;
    const int32_t* ids;
    const float* weights;
    const float* s13;
    const float* s2;
    const __nv_bfloat16* residual;
    __nv_bfloat16* out;
    uint8_t* xg;           // [rows_cap][H] codes of the gathered tokens
    float* sx;             // [H / 128][rows_cap]
    uint8_t* hg;           // [rows_cap][I] codes of the hidden activations
    float* sh;             // [I / 128][rows_cap]
    float* parts;          // [CTA][3][NT][256]
    unsigned* barrier;     // grid barrier word
    unsigned* count1;      // parts of a divided unit that are written, by the unit's first CTA
    unsigned* count2;
    int* status;
    int T, k, E, H, I, rows_cap, act;
    unsigned long long wait_limit_ns;
};

template <int NT>
struct MlCfg {
    static_assert(NT == 16 || NT == 32 || NT == 64, "tokens per chunk");
    static constexpr int T_BYTES = NT * BK;
    static constexpr int STAGE_BYTES = ML_W_BYTES + T_BYTES;
    static constexpr int TABLES = 4 * ML_MAX_E + 4 * ML_MAX_A + 2 * ML_MAX_A + 2 * ML_MAX_ROWS + 4 * ML_MAX_CTAS;
    static constexpr int STATIC_RESERVE = TABLES + 2 * 4 * 32 * 4 + 512;
    static constexpr int STAGES = ring_stages(STAGE_BYTES, 0, 0, STATIC_RESERVE);
    static constexpr int DYN_SMEM = 1024 + STAGES * STAGE_BYTES;
    static constexpr int NACC = (TMEM_COLS / (2 * NT)) > 8 ? 8 : TMEM_COLS / (2 * NT);
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

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void epi_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// One thread's arrival at the barrier of all CTAs, and its wait. CTA 0 adds what carries the others' ones
// into the top bit, so the bit flips when the last one arrives and the low bits are back at zero: the word
// needs no reset between barriers or launches. The CTAs are co-resident (cooperative launch); the wait ends
// by itself all the same.
__device__ __forceinline__ bool grid_barrier(unsigned* word, volatile int* abort_flag, int* status, uint64_t limit_ns) {
    __threadfence();
    const unsigned add = blockIdx.x == 0 ? 0x80000000u - (gridDim.x - 1) : 1u;
    const unsigned old = atomicAdd(word, add);
    const uint64_t t0 = global_timer_ns();
    const uint64_t limit = limit_ns ? limit_ns : WAIT_LIMIT_NS;
    for (int i = 0; i < (1 << 26); ++i) {
        if ((ld_acquire(word) ^ old) & 0x80000000u) {
            __threadfence();
            return true;
        }
        if ((i & 63) == 63 && global_timer_ns() - t0 > limit) break;
    }
    *abort_flag = 1;
    record_status(status, STATUS_TIMEOUT);
    return false;
}

// What a CTA does of one unit: stages [kb0, kb0 + nkb) of unit `unit`, for one chunk of an expert's tokens.
struct Seg {
    int unit;              // phase 1: chunk * (I / 128) + row block; phase 2: row pair * chunks + chunk
    int kb0, nkb;
    int e, off, n;         // expert, first gathered row, rows (1 .. NT)
    int blk;               // phase 1: 128-row block of I; phase 2: pair of 128-row blocks of H
    int row0, row1;        // rows of the weight matrix (all experts stacked) of the stage's two tiles
    bool two;              // the second tile exists (phase 2: an odd number of row blocks ends in half a pair)
};

// A chunk: expert (10 bits), first gathered row (12 bits), rows - 1 (6 bits).
__device__ __forceinline__ uint32_t pack_chunk(int e, int off, int n) {
    return static_cast<uint32_t>(e) | (static_cast<uint32_t>(off) << 10) | (static_cast<uint32_t>(n - 1) << 22);
}

struct Tables {
    const uint32_t* chunk;
    int chunks;
};

template <int PHASE>
__device__ __forceinline__ Seg make_seg(const MoeParams& p, const Tables& tb, int64_t pos, int64_t hi) {
    const int kbs = (PHASE == 1 ? p.H : p.I) / 128;
    Seg s;
    s.unit = static_cast<int>(pos / kbs);
    s.kb0 = static_cast<int>(pos - static_cast<int64_t>(s.unit) * kbs);
    s.nkb = static_cast<int>(min(static_cast<int64_t>(kbs - s.kb0), hi - pos));
    const int per = PHASE == 1 ? p.I / 128 : tb.chunks;
    const int a = s.unit / per, b = s.unit - a * per;
    const int ch = PHASE == 1 ? a : b;
    s.blk = PHASE == 1 ? b : a;
    const uint32_t c = tb.chunk[ch];
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

// Stages of a phase, the CTA's share of them, and the CTA that holds a stage.
__device__ __forceinline__ int64_t phase_stages(const MoeParams& p, int chunks, int phase) {
    return phase == 1 ? static_cast<int64_t>(chunks) * (p.I / 128) * (p.H / 128)
                      : static_cast<int64_t>((p.H + 255) / 256) * chunks * (p.I / 128);
}
// (fewer stages than CTAs: the first CTAs take one each, so that no CTA between two parts of a unit is empty)
__device__ __forceinline__ int sharers(int64_t total) { return static_cast<int>(min(total, static_cast<int64_t>(gridDim.x))); }
__device__ __forceinline__ int64_t share_start(int64_t total, int cta) {
    const int n = sharers(total);
    return cta >= n ? total : total * cta / n;
}
__device__ __forceinline__ int cta_of(int64_t pos, int64_t total) {
    return static_cast<int>(((pos + 1) * sharers(total) - 1) / total);
}

// Running positions in the stage ring.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++stage == n) { stage = 0; phase ^= 1u; }
    }
};

template <int NT>
struct Shared {
    uint64_t full[MlCfg<NT>::STAGES], empty[MlCfg<NT>::STAGES];
    uint64_t acc_full[MlCfg<NT>::NACC], acc_empty[MlCfg<NT>::NACC];
    uint64_t done, go[2];
    uint32_t tmem;
    int abort, chunks, last, twice;
    uint32_t amax[2][4][32];                    // [warpgroup][warp][column] of a unit being finished
    uint32_t offset[ML_MAX_E];                  // rows of an expert, then its first row
    uint32_t chunk[ML_MAX_A];
    uint32_t slot[ML_MAX_CTAS];                 // where the parts of a unit being summed lie
    uint16_t row_of[ML_MAX_A];                  // gathered row of an assignment (t * k + j); 0xffff: no expert
    uint16_t rows[ML_MAX_ROWS];                 // assignment of a gathered row
};

// ---- routing: chunks of at most NT tokens of one expert, their rows, and each assignment's row (its rank among
// the assignments of its expert, in order). Every CTA makes the same tables from the same ids.
template <int NT>
__device__ void make_tables(const MoeParams& p, Shared<NT>& s) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int A = p.T * p.k;
    for (int e = tid; e < p.E; e += THREADS) s.offset[e] = 0;
    __syncthreads();
    if (warp == 4) {
        for (int base = 0; base < A; base += 32) {
            const int a = base + lane;
            int e = a < A ? __ldg(p.ids + a) : -1;
            if (e < 0 || e >= p.E) e = -1;
            const unsigned same = __match_any_sync(FULL_MASK, e);
            const int rank = __popc(same & ((1u << lane) - 1u));
            const uint32_t before = e >= 0 ? s.offset[e] : 0u;
            __syncwarp();
            if (a < A) s.row_of[a] = e >= 0 ? static_cast<uint16_t>(before + rank) : 0xffffu;
            if (e >= 0 && rank == 0) s.offset[e] = before + __popc(same);
            __syncwarp();
        }
        // exclusive sums over the experts: rows rounded up to 4, and chunks
        int rows = 0, chunks = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            const int n = e < p.E ? static_cast<int>(s.offset[e]) : 0;
            int r = (n + 3) & ~3, c = (n + NT - 1) / NT;
            const int r_own = r, c_own = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int ur = __shfl_up_sync(FULL_MASK, r, o), uc = __shfl_up_sync(FULL_MASK, c, o);
                if (lane >= o) { r += ur; c += uc; }
            }
            const int r0 = rows + r - r_own, c0 = chunks + c - c_own;
            if (e < p.E) s.offset[e] = static_cast<uint32_t>(r0);
            for (int i = 0; i < c_own; ++i) s.chunk[c0 + i] = pack_chunk(e, r0 + i * NT, min(NT, n - i * NT));
            rows += __shfl_sync(FULL_MASK, r, 31);
            chunks += __shfl_sync(FULL_MASK, c, 31);
        }
        if (lane == 0) {
            s.chunks = chunks;
            s.twice = 0;
        }
    }
    __syncthreads();
    for (int a = tid; a < A; a += THREADS) {
        if (s.row_of[a] != 0xffffu) {
            const uint32_t r = s.offset[__ldg(p.ids + a)] + s.row_of[a];
            s.row_of[a] = static_cast<uint16_t>(r);
            s.rows[r] = static_cast<uint16_t>(a);
        }
    }
    __syncthreads();
    // a token that names an expert twice has neighbouring rows there
    for (int a = tid; a < A; a += THREADS) {
        const uint32_t r = s.row_of[a];
        if (r != 0xffffu && r > s.offset[__ldg(p.ids + a)] && s.rows[r - 1] / p.k == a / p.k) s.twice = 1;
    }
}

// ---- phase 0: the tokens' codes and scales, written to every row that they are gathered to
__device__ void quantise_tokens(const MoeParams& p, const uint16_t* row_of, int ew, int lane) {
    const int kbs = p.H / 128;
    const int total = p.T * kbs;
    for (int w = static_cast<int>(blockIdx.x) * EPI_WARPS + ew; w < total; w += static_cast<int>(gridDim.x) * EPI_WARPS) {
        const int t = w / kbs, kb = w - t * kbs;
        const uint2 u = *reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(t) * p.H + kb * 128 + lane * 4);
        const float a = bf16_lo(u.x), b = bf16_hi(u.x), c = bf16_lo(u.y), d = bf16_hi(u.y);
        const uint32_t top = __reduce_max_sync(FULL_MASK, max(max(abs_bits(a), abs_bits(b)), max(abs_bits(c), abs_bits(d))));
        const float s = block_scale(top);
        const uint32_t q = quantise4(a, b, c, d, s, __frcp_rn(s));
        for (int j = 0; j < p.k; ++j) {
            const uint32_t r = row_of[t * p.k + j];
            if (r == 0xffffu) continue;
            *reinterpret_cast<uint32_t*>(p.xg + static_cast<size_t>(r) * p.H + kb * 128 + lane * 4) = q;
            if (lane == 0) p.sx[static_cast<size_t>(kb) * p.rows_cap + r] = s;
        }
    }
}

template <int NT>
__global__ void __launch_bounds__(THREADS, 1)
moe_layer_kernel(const __grid_constant__ CUtensorMap map_w13, const __grid_constant__ CUtensorMap map_w2,
                 const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_h,
                 const __grid_constant__ MoeParams p) {
    using C = MlCfg<NT>;
    constexpr int STAGES = C::STAGES, NACC = C::NACC, NG = C::NG;
    static_assert(sizeof(Shared<NT>) <= C::STATIC_RESERVE, "static shared memory");

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
        mbar_init(&s.done, EPI_WARPS);
        mbar_init(&s.go[0], 1);
        mbar_init(&s.go[1], 1);
        s.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem, TMEM_COLS);
        tmem_relinquish();
    }
    make_tables<NT>(p, s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s.tmem;
    volatile int* abort_flag = &s.abort;
    const Tables tb{s.chunk, s.chunks};

    if (warp < EPI_WARP0) {
        regs_dec<CTRL_REGS>();
        const bool issuer = elect_one();
        Ring ring;
        bool ok = true;
        if (warp == 0) {
            // ---------------------------------------------------------------- weights
            uint32_t issued = 0, issued_parity = 0;
            auto stream = [&](auto phase_tag, const CUtensorMap* map) {
                constexpr int PHASE = decltype(phase_tag)::value;
                const int64_t total = phase_stages(p, tb.chunks, PHASE);
                const int64_t hi = share_start(total, cta + 1);
                for (int64_t pos = share_start(total, cta); pos < hi && ok;) {
                    const Seg g = make_seg<PHASE>(p, tb, pos, hi);
                    pos += g.nkb;
                    for (int kb = g.kb0; kb < g.kb0 + g.nkb; ++kb) {
                        const bool got = wait_bounded(&s.empty[ring.stage], ring.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns);
                        if (!__all_sync(FULL_MASK, got)) { ok = false; break; }
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
                }
            };
            stream(std::integral_constant<int, 1>{}, &map_w13);
            stream(std::integral_constant<int, 2>{}, &map_w2);
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
        } else if (warp == 2) {
            // ---------------------------------------------------------------- tokens
            auto stream = [&](auto phase_tag, const CUtensorMap* map) {
                constexpr int PHASE = decltype(phase_tag)::value;
                const int64_t total = phase_stages(p, tb.chunks, PHASE);
                const int64_t hi = share_start(total, cta + 1);
                if (ok) {
                    const bool got = wait_bounded(&s.go[PHASE - 1], 0, abort_flag, p.status, p.wait_limit_ns);
                    if (!__all_sync(FULL_MASK, got)) ok = false;
                    fence_proxy_async_all();    // what other CTAs wrote before the barrier is read by TMA
                }
                for (int64_t pos = share_start(total, cta); pos < hi && ok;) {
                    const Seg g = make_seg<PHASE>(p, tb, pos, hi);
                    pos += g.nkb;
                    const int boxes = (g.n + 15) / 16;
                    for (int kb = g.kb0; kb < g.kb0 + g.nkb; ++kb) {
                        const bool got = wait_bounded(&s.empty[ring.stage], ring.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns);
                        if (!__all_sync(FULL_MASK, got)) { ok = false; break; }
                        if (issuer) {
                            uint8_t* dst = smem_t + ring.stage * C::T_BYTES;
                            mbar_arrive_expect_tx(&s.full[ring.stage], static_cast<uint32_t>(boxes * 16 * BK));
                            for (int b = 0; b < boxes; ++b)
                                tma_load_2d(map, &s.full[ring.stage], dst + b * 16 * BK, kb * BK, g.off + b * 16);
                        }
                        ring.next(STAGES);
                        __syncwarp();
                    }
                }
            };
            stream(std::integral_constant<int, 1>{}, &map_x);
            stream(std::integral_constant<int, 2>{}, &map_h);
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA issue
            Ring acc;
            int last = -1;
            uint32_t last_parity = 0;
            const uint32_t w_base = smem_u32(smem), t_base = smem_u32(smem_t);
            auto run = [&](auto phase_tag) {
                constexpr int PHASE = decltype(phase_tag)::value;
                const int64_t total = phase_stages(p, tb.chunks, PHASE);
                const int64_t hi = share_start(total, cta + 1);
                for (int64_t pos = share_start(total, cta); pos < hi && ok;) {
                    const Seg g = make_seg<PHASE>(p, tb, pos, hi);
                    pos += g.nkb;
                    const uint32_t idesc = idesc_e4m3_f32(128, (g.n + 15) & ~15);
                    for (int kb = 0; kb < g.nkb; ++kb) {
                        const bool got = wait_bounded(&s.acc_empty[acc.stage], acc.phase ^ 1u, abort_flag, p.status, p.wait_limit_ns) &&
                                         wait_bounded(&s.full[ring.stage], ring.phase, abort_flag, p.status, p.wait_limit_ns);
                        if (!__all_sync(FULL_MASK, got)) { ok = false; break; }
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
                }
            };
            run(std::integral_constant<int, 1>{});
            run(std::integral_constant<int, 2>{});
            if (!ok && last >= 0 && issuer) drain_wait(&s.acc_full[last], last_parity);
        } else {
            // ---------------------------------------------------------------- grid barriers
            if (lane == 0) {
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    wait_bounded(&s.done, static_cast<uint32_t>(b), abort_flag, p.status, p.wait_limit_ns);
                    const bool got = grid_barrier(p.barrier, abort_flag, p.status, p.wait_limit_ns);
                    fence_proxy_async_all();
                    if (got) mbar_arrive(&s.go[b]);
                }
            }
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------------- epilogue warps
        regs_inc<EPI_REGS>();
        const int tid = static_cast<int>(threadIdx.x) - EPI_WARP0 * 32;   // 0 .. 255
        const int ew = warp - EPI_WARP0;
        const int q = warp & 3;                 // TMEM lane quarter
        const int h = ew >> 2;                  // warpgroup: 8-column groups h, h + 2, ...
        const int r = q * 32 + lane;            // row of each 128-row tile
        const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(8 * h);
        bool ok = true;
        Ring acc;

        quantise_tokens(p, s.row_of, ew, lane);
        fence_proxy_async_all();
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.done);

        float a0[NG][8], a1[NG][8];
        auto clear = [&] {
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) a0[i][j] = a1[i][j] = 0.f;
        };
        // Promotion over a segment: sx the token scales ([kb][rows_cap]), sb0 / sb1 the two tiles' weight
        // scales (by K block), all read one K block ahead.
        auto promote = [&](const Seg& g, const float* sx, const float* sb0, const float* sb1) {
            float4 sn[NG][2];
            auto scales = [&](int kb) {
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if ((2 * i + h) * 8 < g.n) {
                        const float4* src = reinterpret_cast<const float4*>(sx + static_cast<size_t>(kb) * p.rows_cap + g.off + (2 * i + h) * 8);
                        sn[i][0] = __ldcg(src);
                        sn[i][1] = __ldcg(src + 1);
                    }
                }
            };
            float b0n = __ldg(sb0 + g.kb0), b1n = __ldg(sb1 + g.kb0);
            scales(g.kb0);
            for (int kb = g.kb0; kb < g.kb0 + g.nkb; ++kb) {
                bool got = mbar_try_wait(&s.acc_full[acc.stage], acc.phase);
                if (!got) got = wait_bounded(&s.acc_full[acc.stage], acc.phase, abort_flag, p.status, p.wait_limit_ns);
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
                const float b0 = b0n, b1 = b1n;
                float4 sc[NG][2];
#pragma unroll
                for (int i = 0; i < NG; ++i) { sc[i][0] = sn[i][0]; sc[i][1] = sn[i][1]; }
                if (kb + 1 < g.kb0 + g.nkb) {
                    scales(kb + 1);
                    b0n = __ldg(sb0 + kb + 1);
                    b1n = __ldg(sb1 + kb + 1);
                }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if ((2 * i + h) * 8 < g.n) {
                        const float v[8] = {sc[i][0].x, sc[i][0].y, sc[i][0].z, sc[i][0].w, sc[i][1].x, sc[i][1].y, sc[i][1].z, sc[i][1].w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            a0[i][j] = fmaf(__uint_as_float(p0[i][j]), v[j] * b0, a0[i][j]);
                            a1[i][j] = fmaf(__uint_as_float(p1[i][j]), v[j] * b1, a1[i][j]);
                        }
                    }
                }
            }
        };
        auto slot_of = [&](int c, int which) { return p.parts + static_cast<size_t>(c * 3 + which) * (NT * 256); };
        // Whether this CTA's part of a divided unit came last (`count` of the unit's first CTA); every
        // thread's writes of the part are visible to whoever sees the full count.
        auto came_last = [&](unsigned* count, int parts) {
            __threadfence();
            epi_barrier();
            // (a unit of one CTA has no count: its first CTA's may be in use for the next unit already)
            if (parts == 1) return true;
            if (tid == 0) {
                const bool last = atomicAdd(count, 1u) == static_cast<unsigned>(parts - 1);
                if (last) *count = 0;           // as the next launch expects it
                __threadfence();
                s.last = last ? 1 : 0;
            }
            epi_barrier();
            return s.last != 0;
        };
        // The other CTAs' writes before a grid barrier may be read from here on, and this CTA's slots written.
        auto crossed = [&](int b) {
            const bool got = ok && wait_bounded(&s.go[b], 0, abort_flag, p.status, p.wait_limit_ns);
            ok = __all_sync(FULL_MASK, got) != 0;
        };

        // ---------------------------------------------------------------- phase 1
        crossed(0);
        {
            const int kbs = p.H / 128, blocks = p.I / 128;
            const int64_t total = phase_stages(p, tb.chunks, 1);
            const int64_t lo = share_start(total, cta), hi = share_start(total, cta + 1);
            for (int64_t pos = lo; pos < hi;) {
                const Seg g = make_seg<1>(p, tb, pos, hi);
                pos += g.nkb;
                clear();
                const float* sb = p.s13 + (static_cast<size_t>(g.e) * 2 * blocks + g.blk) * kbs;
                if (ok) promote(g, p.sx, sb, sb + static_cast<size_t>(blocks) * kbs);
                if (g.nkb < kbs) {
                    // part of a unit: whoever comes last adds up the parts in the order of the CTAs
                    const int64_t u0 = static_cast<int64_t>(g.unit) * kbs;
                    const int c_lo = cta_of(u0, total), c_hi = cta_of(u0 + kbs - 1, total);
                    float* mine = slot_of(cta, u0 < lo ? 0 : 1);
#pragma unroll
                    for (int i = 0; i < NG; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int col = (2 * i + h) * 8 + j;
                            if (col < g.n) {
                                __stcg(mine + col * 256 + r, a0[i][j]);
                                __stcg(mine + col * 256 + 128 + r, a1[i][j]);
                            }
                        }
                    if (!came_last(p.count1 + c_lo, c_hi - c_lo + 1)) continue;
                    clear();
                    for (int c = c_lo; c <= c_hi; ++c) {
                        // the unit is the first of every CTA but the one in whose share it starts
                        const float* part = slot_of(c, u0 < share_start(total, c) ? 0 : 1);
#pragma unroll
                        for (int i = 0; i < NG; ++i)
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int col = (2 * i + h) * 8 + j;
                                if (col < g.n) {
                                    a0[i][j] += __ldcg(part + col * 256 + r);
                                    a1[i][j] += __ldcg(part + col * 256 + 128 + r);
                                }
                            }
                    }
                }
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
#pragma unroll
                for (int i = 0; i < NG; ++i) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int col = (2 * i + h) * 8 + j;
                        if (col < g.n) {
                            const int c = i * 8 + j;
                            const float sc = block_scale(max(max(s.amax[h][0][c], s.amax[h][1][c]), max(s.amax[h][2][c], s.amax[h][3][c])));
                            const float v = finite_scale(sc) ? block_quotient(a0[i][j], sc, __frcp_rn(sc)) : __fdiv_rn(a0[i][j], sc);
                            p.hg[static_cast<size_t>(g.off + col) * p.I + g.blk * 128 + r] = static_cast<uint8_t>(pack_e4m3x2(v, 0.f) & 0xffu);
                            if (r == 0) p.sh[static_cast<size_t>(g.blk) * p.rows_cap + g.off + col] = sc;
                        }
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(2 + h) : "memory");   // the maxima may be overwritten
            }
            fence_proxy_async_all();
            __threadfence();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.done);
        }

        // ---------------------------------------------------------------- phase 2
        crossed(1);
        {
            const int kbs = p.I / 128;
            const int64_t total = phase_stages(p, tb.chunks, 2);
            const int64_t per_pair = static_cast<int64_t>(tb.chunks) * kbs;
            const int64_t lo = share_start(total, cta), hi = share_start(total, cta + 1);
            int pair = -1;
            float* mine = nullptr;
            // the pair's part of this CTA is complete: write it down, and finish the pair if it came last
            auto close = [&](int pr) {
                const int64_t u0 = pr * per_pair;
                const int c_lo = cta_of(u0, total), c_hi = cta_of(u0 + per_pair - 1, total);
                if (!came_last(p.count2 + c_lo, c_hi - c_lo + 1)) return;
                const int parts = c_hi - c_lo + 1;
                if (tid < parts) {
                    const int which = share_start(total, c_lo + tid) >= u0 ? 0 : (share_start(total, c_lo + tid + 1) <= u0 + per_pair ? 1 : 2);
                    s.slot[tid] = static_cast<uint32_t>((c_lo + tid) * 3 + which) * (NT * 256);
                }
                epi_barrier();
                for (int f = tid; f < p.T * 64; f += EPI_WARPS * 32) {
                    const int t = f >> 6, c4 = (f & 63) * 4;
                    const int col = pr * 256 + c4;
                    if (col >= p.H) continue;
                    const size_t at = static_cast<size_t>(t) * p.H + col;
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int c = 0; c < parts; ++c) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.parts + s.slot[c] + t * 256 + c4));
                        sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
                    }
                    if (p.residual != nullptr) {
                        const uint2 u = *reinterpret_cast<const uint2*>(p.residual + at);
                        sum.x += bf16_lo(u.x); sum.y += bf16_hi(u.x); sum.z += bf16_lo(u.y); sum.w += bf16_hi(u.y);
                    }
                    st_global_v2(p.out + at, pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
                }
                epi_barrier();                  // the slot may be used for the next pair
            };
            for (int64_t pos = lo; pos < hi;) {
                const Seg g = make_seg<2>(p, tb, pos, hi);
                pos += g.nkb;
                if (g.blk != pair) {
                    if (pair >= 0) close(pair);
                    pair = g.blk;
                    // slot 0: the pair that the CTA starts in, 1: the one it ends in, 2: any between
                    const int64_t u0 = pair * per_pair;
                    mine = slot_of(cta, lo >= u0 ? 0 : (hi <= u0 + per_pair ? 1 : 2));
                    for (int f = tid; f < p.T * 64; f += EPI_WARPS * 32)
                        __stcg(reinterpret_cast<float4*>(mine) + f, make_float4(0.f, 0.f, 0.f, 0.f));
                }
                clear();
                const float* sb = p.s2 + (static_cast<size_t>(g.e) * (p.H / 128) + 2 * g.blk) * kbs;
                if (ok) promote(g, p.sh, sb, g.two ? sb + kbs : sb);
                epi_barrier();                  // the zeros, or the previous expert's sums, are written
                // (the warpgroups take turns where a token has two columns of the chunk: they may be one's
                // and the other's)
                for (int turn = 0; turn < (s.twice ? 2 : 1); ++turn) {
                    if (turn) epi_barrier();
                    if (s.twice && turn != h) continue;
#pragma unroll
                    for (int i = 0; i < NG; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int col = (2 * i + h) * 8 + j;
                            if (col < g.n) {
                                const int a = s.rows[g.off + col];
                                const float w = __ldg(p.weights + a);
                                float* dst = mine + (a / p.k) * 256 + r;
                                __stcg(dst, fmaf(w, a0[i][j], __ldcg(dst)));
                                if (g.two) __stcg(dst + 128, fmaf(w, a1[i][j], __ldcg(dst + 128)));
                            }
                        }
                }
            }
            if (pair >= 0) close(pair);
            if (total == 0) {
                // no token met an expert
                for (size_t f = static_cast<size_t>(cta) * 256 + tid; f < static_cast<size_t>(p.T) * p.H / 4; f += static_cast<size_t>(gridDim.x) * 256)
                    reinterpret_cast<uint2*>(p.out)[f] = p.residual != nullptr ? reinterpret_cast<const uint2*>(p.residual)[f] : make_uint2(0u, 0u);
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

struct Layout {
    int64_t xg, sx, hg, sh, parts, bytes;
};

int64_t up(int64_t v) { return (v + 1023) / 1024 * 1024; }

Layout layout(int T, int k, int E, int H, int I) {
    const int64_t rows = rows_cap(T, k, E);
    Layout l;
    l.xg = ML_FIXED;
    l.sx = l.xg + up(rows * H);
    l.hg = l.sx + up((rows * (H / 128) + 16) * 4);     // scales are read 8 at a time, past the last row
    l.sh = l.hg + up(rows * I);
    l.parts = l.sh + up((rows * (I / 128) + 16) * 4);
    l.bytes = l.parts + static_cast<int64_t>(ML_MAX_CTAS) * 3 * tokens_per_chunk(T) * 256 * 4;
    return l;
}

bool sizes_ok(int T, int k, int E, int H, int I) {
    return T >= 1 && T <= ML_MAX_T && k >= 1 && static_cast<int64_t>(T) * k <= ML_MAX_A && E >= 1 && E <= ML_MAX_E && H >= 128 && I >= 128 &&
           H % 128 == 0 && I % 128 == 0 && static_cast<int64_t>(E) * 2 * I <= INT32_MAX && static_cast<int64_t>(E) * H <= INT32_MAX;
}

template <int NT>
cudaError_t launch_moe(const CUtensorMap& w13, const CUtensorMap& w2, const CUtensorMap& x, const CUtensorMap& h,
                       const MoeParams& p, int ctas, cudaStream_t stream) {
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
    p.count1 = reinterpret_cast<unsigned*>(ws + 1024);
    p.count2 = reinterpret_cast<unsigned*>(ws + 2048);
    p.xg = reinterpret_cast<uint8_t*>(ws + l.xg);
    p.sx = reinterpret_cast<float*>(ws + l.sx);
    p.hg = reinterpret_cast<uint8_t*>(ws + l.hg);
    p.sh = reinterpret_cast<float*>(ws + l.sh);
    p.parts = reinterpret_cast<float*>(ws + l.parts);
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
