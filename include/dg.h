/*
 * dg — block-scaled FP8 GEMM and MoE grouped GEMM for GB300 (sm_103a): the C ABI.
 *
 * The operation (DeepGEMM pages: "DeepSeek DeepGEMM" feature list and usage example;
 * "DeepSeek Open Source Week - Dia 3", technical features):
 *
 *   D[m,n] = sum_kb  sfa[m,kb] * sfb[n/128,kb] * sum_{k in block kb} A[m,k] * B[n,k]
 *
 * A and B hold float8 e4m3 codes ("fn" variant), K-contiguous ("NT": A is [M,K], B is [N,K]).
 * Fine-grained scaling gives one FP32 scale per 1x128 row block of A and per 128x128 block of B;
 * every 128-wide K block is contracted on the tensor cores and then promoted, scaled by its two
 * scales, into an FP32 running sum ("two-level accumulation"). Results are rounded to BF16
 * (round to nearest even) for the normal and m-grouped GEMMs; the k-grouped weight gradient
 * accumulates into FP32.
 *
 * Conventions shared by every entry point:
 *   - All tensors are caller-owned DEVICE memory, row-major and densely packed, unless stated
 *     otherwise. The library keeps no pointer after a call returns and allocates no memory.
 *   - Calls are asynchronous on `stream` (0 = the legacy default stream). Argument errors are
 *     returned synchronously before anything is launched; launch errors return DG_CUDA_ERROR.
 *   - K (and every k-grouped ks[g]) must be a multiple of 128, the scaling block ("K dimension
 *     aligned to 128" in the pages' requirements). N must be a multiple of 8 (16-byte output rows).
 *   - A and B must be 16-byte aligned (TMA), D 16-byte aligned, scales 4-byte aligned.
 *   - Zero-sized problems (M = 0, Mt = 0, G = 0) are valid and launch nothing.
 *   - The library runs on compute capability 10.3 only (sm_103a code); other devices get
 *     DG_NO_DEVICE_SUPPORT.
 *   - Device-side waits are bounded; a kernel that gives up records DG_DEVICE_TIMEOUT, which
 *     dg_device_status() reports. Tuning overrides and a test hook for this path: dg_tuning.h.
 *   - Distinct streams may call concurrently (no mutable host state after first use per device). Calls
 *     that take a workspace need one each: a workspace serves one call at a time.
 */
#ifndef DG_H
#define DG_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int dg_status;
enum {
    DG_OK = 0,
    DG_INVALID_ARG = 1,        /* null pointer with a non-empty shape, negative size, G out of range */
    DG_UNSUPPORTED_SHAPE = 2,  /* K % 128, N % 8, ks[g] % 128, or a size beyond the supported range */
    DG_MISALIGNED = 3,         /* a pointer not aligned as stated above */
    DG_CUDA_ERROR = 4,         /* a CUDA runtime/driver call or launch failed */
    DG_NO_DEVICE_SUPPORT = 5,  /* current device is not compute capability 10.3 */
    DG_DEVICE_TIMEOUT = 6,     /* a kernel's bounded wait expired (reported by dg_device_status) */
    DG_SCALE_NOT_UE8M0 = 7     /* a UE8M0-path scale was not a power of two (reported by dg_device_status) */
};

/*
 * Normal GEMM (pages: gemm_fp8_fp8_bf16_nt).
 *   A   [M, K]            e4m3 codes          sfa [M, K/128]            fp32
 *   B   [N, K]            e4m3 codes          sfb [ceil(N/128), K/128]  fp32
 *   D   [M, N]            bf16, overwritten
 * The usage example on the pages (M=4096, K=7168, N=2112) has sfa [4096, 56] and sfb [17, 56]:
 * sfb has ceil(N/128) rows, row j scaling B rows [128j, 128j+128).
 */
dg_status dg_gemm_fp8_nt(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb,
                         void* D, int M, int N, int K, cudaStream_t stream);

/*
 * The normal GEMM for the other operand layouts (the pages list NT, TN, NN and TT for SM100): the same
 * product D = A . B^T with the same scales, but A may be stored transposed, [K, M] with M contiguous
 * (a_mn_major != 0), and B transposed, [K, N] with N contiguous (b_mn_major != 0). sfa stays
 * [M, K/128] and sfb [ceil(N/128), K/128]. An MN-major operand needs its contiguous extent (M or N)
 * to be a multiple of 16 (DG_UNSUPPORTED_SHAPE otherwise). dg_gemm_fp8(..., 0, 0, ...) is
 * dg_gemm_fp8_nt.
 */
dg_status dg_gemm_fp8(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb, void* D,
                      int M, int N, int K, int a_mn_major, int b_mn_major, cudaStream_t stream);

/*
 * The normal GEMM for power-of-two scales, on the block-scaled tensor-core path (pages: the SM100
 * UE8M0 scale format): same arguments and result as dg_gemm_fp8_nt, but every sfa and sfb entry must
 * be a positive power of two in [2^-126, 2^127]. The tensor core applies the scales as 8-bit exponents
 * while it accumulates, so no per-128-K promotion runs. A scale that is not a power of two is
 * reported by dg_device_status as DG_SCALE_NOT_UE8M0 (its result is then unspecified).
 */
dg_status dg_gemm_fp8_nt_ue8m0(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb, void* D,
                               int M, int N, int K, cudaStream_t stream);

/*
 * The same block-scaled GEMM with the scales already in the packed UE8M0 format (pages: the SM100
 * scale layout, four UE8M0 values in one int32):
 *   sfa  [M, ceil(K/512)] int32          sfb  [ceil(N/128), ceil(K/512)] int32
 * Byte j (least significant first) of word w of a row is the biased exponent e of K block 4w + j; the
 * scale it stands for is 2^(e - 127). Bytes past the last K block are ignored. The exponents are used
 * as they are (no check; e = 255 is not a number). Result as dg_gemm_fp8_nt with those scales.
 * Device pointers, 4-byte aligned; errors as dg_gemm_fp8_nt.
 */
dg_status dg_gemm_fp8_nt_ue8m0_packed(const uint8_t* A, const int32_t* sfa, const uint8_t* B, const int32_t* sfb,
                                      void* D, int M, int N, int K, cudaStream_t stream);

/*
 * m-grouped GEMM, contiguous layout (pages: m_grouped_gemm_fp8_fp8_bf16_nt_contiguous; for training
 * forward and inference prefill). The experts' token rows are stacked along M; each expert's segment
 * starts on a multiple of 128 rows (segments padded to 128).
 *   A         [Mt, K]                 sfa [Mt, K/128]
 *   B         [G, N, K]               sfb [G, ceil(N/128), K/128]
 *   m_indices [Mt] int32 (device)     expert of each row, -1 on padding rows
 *   D         [Mt, N] bf16
 * Row r gets D[r] = A[r] . B[m_indices[r]]^T. The expert of a 128-row block is read from its first
 * row; a block whose first row is -1 (or >= G) is skipped and its D rows are left untouched. Rows
 * tagged -1 inside a computed block receive that block's expert's product (their content is
 * unspecified). Mt must be a multiple of 128.
 */
dg_status dg_m_grouped_contiguous(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb,
                                  const int32_t* m_indices, void* D, int Mt, int N, int K, int G,
                                  cudaStream_t stream);

/*
 * m-grouped GEMM, masked layout (pages: m_grouped_gemm_fp8_fp8_bf16_nt_masked; for decode, including
 * under CUDA graphs, since every shape argument is static and the per-expert counts stay on device).
 *   A        [G, max_m, K]            sfa [G, max_m, K/128]
 *   B        [G, N, K]                sfb [G, ceil(N/128), K/128]
 *   masked_m [G] int32 (device)       valid rows per expert, clamped to [0, max_m] on device
 *   D        [G, max_m, N] bf16
 * For r < masked_m[g]: D[g,r] = A[g,r] . B[g]^T. Rows r >= masked_m[g] are never written.
 * expected_m is a performance hint (typical masked_m); <= 0 means unknown. 1 <= G <= 1024.
 */
dg_status dg_m_grouped_masked(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb,
                              const int32_t* masked_m, void* D, int G, int max_m, int N, int K,
                              int expected_m, cudaStream_t stream);

/*
 * k-grouped weight-gradient GEMM with FP32 output (pages: k_grouped_wgrad_gemm_fp8_fp8_fp32_nt; the
 * MoE backward dW = X^T . dY per expert). Each expert g owns a window of ks[g] columns of the
 * token dimension, windows laid out in order:
 *   A  = X^T  [M, sumK]   e4m3        sfa [M, sumK/128]   (1x128 scales along K)
 *   B  = dY^T [N, sumK]   e4m3        sfb [N, sumK/128]   (1x128 scales along K, per row)
 *   ks_host [G] int32, HOST memory, each a multiple of 128 (0 allowed), sumK = sum(ks)
 *   D  [G, M, N] fp32, accumulated: D[g] += A[:, win_g] . B[:, win_g]^T
 * 1 <= G <= 128.
 */
dg_status dg_k_grouped_wgrad(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb,
                             const int32_t* ks_host, float* D, int G, int M, int N,
                             cudaStream_t stream);

/*
 * Dense weight-gradient GEMM with FP32 output (pages: wgrad_gemm_fp8_fp8_fp32_nt; dW = X^T . dY of a
 * dense layer in the backward pass). The single-expert case of dg_k_grouped_wgrad, plus an
 * overwriting form:
 *   A = X^T  [M, K]   e4m3        sfa [M, K/128]   (1x128 scales along K)
 *   B = dY^T [N, K]   e4m3        sfb [N, K/128]   (1x128 scales along K, per row)
 *   D        [M, N]   fp32: D += A . B^T if accumulate != 0, else D = A . B^T (old contents ignored)
 * K must be a multiple of 128. K == 0 leaves D unchanged when accumulating and zeroes it otherwise.
 */
dg_status dg_wgrad_fp8_nt(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb,
                          float* D, int M, int N, int K, int accumulate, cudaStream_t stream);

/* ---------------------------------------------------------------------- around the products */

/* Activations of dg_gemm_fp8_nt_epilogue, dg_epilogue_backward and dg_moe_layer. GELU is z Phi(z) (with erf),
 * GELU_TANH its tanh form, SILU z / (1 + exp(-z)). */
enum { DG_ACT_NONE = 0, DG_ACT_RELU = 1, DG_ACT_GELU = 2, DG_ACT_GELU_TANH = 3, DG_ACT_SILU = 4 };

/* Element types: of the router's logits and a norm's weights (BF16, F32), of the rows of dg_moe_gather (BF16, E4M3). */
enum { DG_TYPE_BF16 = 0, DG_TYPE_F32 = 1, DG_TYPE_E4M3 = 2 };

/* Router scores. */
enum { DG_SCORE_SOFTMAX = 0, DG_SCORE_SIGMOID = 1 };

/*
 * The normal GEMM with bias, activation and residual in its epilogue:
 *   Z = A . B^T + bias,   D = act(Z) + residual
 *   A, sfa, B, sfb, D     as dg_gemm_fp8_nt
 *   bias     [N] fp32, or null
 *   residual [M, N] bf16, or null; may be D itself (added in place), must not overlap it otherwise
 *   Z        [M, N] bf16, or null: the pre-activation kept for dg_epilogue_backward
 * Everything up to the two BF16 outputs stays in FP32. bias 4-byte, residual and Z 16-byte aligned. K = 0
 * is DG_UNSUPPORTED_SHAPE.
 */
dg_status dg_gemm_fp8_nt_epilogue(const uint8_t* A, const float* sfa, const uint8_t* B, const float* sfb, void* D,
                                  const float* bias, int act, const void* residual, void* Z, int M, int N, int K,
                                  cudaStream_t stream);

/*
 * Its backward pass up to the two products: dZ = dD * act'(Z), quantised in both directions, and the bias
 * gradient. (The residual's gradient is dD itself.)
 *   dD    [M, N] bf16        Z [M, N] bf16 (not read, and may be null, for DG_ACT_NONE)
 *   q     [M, N] e4m3        sf  [M, N/128]       dZ, 1x128 scales along N: A of dX = dZ . B, which is
 *                                                 dg_gemm_fp8 with b_mn_major and sfb transposed
 *   qt    [N, Mp] e4m3       sft [N, Mp/128]      dZ^T, 1x128 scales along M, Mp = M rounded up to 128, zeros
 *                                                 past M: an operand of dg_wgrad_fp8_nt / dg_k_grouped_wgrad
 *   dbias [N] fp32                                sum of dZ's rows (before quantisation), in a fixed order
 * q with sf, qt with sft, and dbias may each be null. Quantisation: s = max(amax, 1e-4) / 448 per block,
 * code = e4m3(v / s), both quotients rounded to FP32. With DG_ACT_NONE this quantises a BF16 matrix in one
 * or both directions. N must be a multiple of 128; M is free. dD, Z, q, qt 16-byte aligned.
 * workspace: device memory of dg_epilogue_backward_workspace(M, N) bytes, 16-byte aligned, needed for dbias
 * (else it may be null), its first DG_EPILOGUE_BACKWARD_ZEROED bytes zero before its first use; every call
 * leaves it ready for the next one, of any size that it is large enough for.
 */
enum { DG_EPILOGUE_BACKWARD_ZEROED = 1024 };
dg_status dg_epilogue_backward(const void* dD, const void* Z, int act, uint8_t* q, float* sf, uint8_t* qt, float* sft,
                               float* dbias, void* workspace, int64_t workspace_bytes, int M, int N,
                               cudaStream_t stream);
int64_t dg_epilogue_backward_workspace(int M, int N);

/*
 * The router: the k experts of each row with the largest selection values, largest first, ties to the lower
 * expert, and their weights.
 *   logits  [T, E] bf16 or fp32 (logits_type)
 *   bias    [E] fp32, or null; only with DG_SCORE_SIGMOID
 *   ids     [T, k] int32      weights [T, k] fp32
 * Selection value: the logit, or with a bias sigmoid(logit) + bias. Weight: scale times the score, softmax
 * over the row or sigmoid(logit) (never the bias), divided by the sum of the k scores with renormalize.
 * Logits of -inf and NaN cannot be selected and are no part of a softmax; +inf counts as the largest
 * finite value. Where fewer than k experts can be selected the slots left over get id -1 and weight 0; a
 * sum of scores that is 0 gives weights 0. E <= 1024, k <= 32, k <= E.
 */
dg_status dg_moe_route(const void* logits, int logits_type, const float* bias, int32_t* ids, float* weights, int T, int E,
                       int k, int scoring, int renormalize, float scale, cudaStream_t stream);

/*
 * The gradient of dg_moe_route's weights with respect to the logits: dlogits [T, E], of the logits' type,
 * from dweights [T, k] fp32 and the ids of the forward pass (ids outside [0, E) are empty slots). Every
 * logit is written, 0 where the weights do not depend on it. dlogits must not overlap logits.
 */
dg_status dg_moe_route_backward(const void* logits, int logits_type, const int32_t* ids, const float* dweights,
                                void* dlogits, int T, int E, int k, int scoring, int renormalize, float scale,
                                cudaStream_t stream);

/*
 * A whole mixture-of-experts layer for a few tokens (decode), in one launch:
 *   out[t] = residual[t] + sum_j weights[t,j] * W2[e] . Q(act(g) * u),   (g; u) = W13[e] . Q(x[t]),   e = ids[t,j]
 *   x        [T, H] bf16
 *   ids      [T, k] int32 (device)      weights [T, k] fp32      as dg_moe_route gives them; an id outside
 *                                                                 [0, E) is an empty slot
 *   W13      [E, 2I, H] e4m3            s13 [E, 2I/128, H/128]   gate rows [0, I), up rows [I, 2I)
 *   W2       [E, H, I] e4m3             s2  [E, H/128, I/128]
 *   residual [T, H] bf16, or null; may be out or x
 *   out      [T, H] bf16, overwritten; may be x
 * Q is the 1x128 quantisation of dg_epilogue_backward; the products, the activation and the sum over a token's
 * experts are FP32, rounded to BF16 once. The weights are the operands of the grouped GEMMs unchanged, and
 * only those of experts that a token meets are read.
 * 1 <= T <= 64 (0: no-op), T * k <= 1024, E <= 1024, H and I multiples of 128.
 * workspace: device memory of dg_moe_layer_workspace(T, k, E, H, I) bytes (-1 for sizes outside these), 256-byte
 * aligned, its first DG_MOE_LAYER_ZEROED bytes zero before its first use; every call leaves it ready for the
 * next one, of any sizes it is large enough for. After DG_DEVICE_TIMEOUT zero those again. The launch is cooperative: its CTAs, one per SM, run at
 * the same time.
 */
enum { DG_MOE_LAYER_ZEROED = 4096 };
dg_status dg_moe_layer(const void* x, const int32_t* ids, const float* weights, const uint8_t* W13, const float* s13,
                       const uint8_t* W2, const float* s2, const void* residual, void* out, void* workspace,
                       int64_t workspace_bytes, int T, int k, int E, int H, int I, int act, cudaStream_t stream);
int64_t dg_moe_layer_workspace(int T, int k, int E, int H, int I);

/* ------------------------------------------------- between the grouped products (prefill and training) */

/*
 * Tokens by expert: the row that each routed slot has in a grouped layout. ids [T, k] int32 as dg_moe_route gives them; an
 * id outside [0, E) has no row (-1). An expert's rows are in the order of its slots (t, then j), whatever the timing.
 *   rows    [T, k] int32
 *   counts, masked_m  [E] int32: the slots of each expert
 * Contiguous (dg_m_grouped_contiguous): the experts one after the other, each from a multiple of 128 on.
 *   m_indices [Mt] int32, 16-byte aligned: the expert of each row, -1 where there is none. Mt a multiple of 128, at least
 *   dg_moe_sort_rows(T, k, E), which every routing fits (DG_UNSUPPORTED_SHAPE otherwise). The rows in use end with the
 *   last expert's block: a caller that knows the counts may pass later calls that many rows.
 * Masked (dg_m_grouped_masked): expert e from row e * max_m on. Slots past max_m get no row (-1) and masked_m still counts
 *   them; the product and dg_glu take no more than max_m.
 * 1 <= E <= 1024, k <= 32, T * k <= 2^23, E * max_m < 2^31. No output overlaps ids.
 * workspace: device memory of dg_moe_sort_workspace(T, k, E) bytes, 16-byte aligned, with anything in it; 0 bytes (and null)
 * up to 16384 slots. dg_moe_sort_rows and dg_moe_sort_workspace return -1 for sizes outside these.
 */
dg_status dg_moe_sort_contiguous(const int32_t* ids, int32_t* rows, int32_t* counts, int32_t* m_indices, void* workspace,
                                 int64_t workspace_bytes, int T, int k, int E, int Mt, cudaStream_t stream);
dg_status dg_moe_sort_masked(const int32_t* ids, int32_t* rows, int32_t* masked_m, void* workspace, int64_t workspace_bytes,
                             int T, int k, int E, int max_m, cudaStream_t stream);
int64_t dg_moe_sort_rows(int T, int k, int E);
int64_t dg_moe_sort_workspace(int T, int k, int E);

/*
 * The tokens' rows in a grouped layout: out[rows[t,j]] = x[t] for every slot whose row is in [0, Mt); no two slots may have
 * the same one.
 *   x_type DG_TYPE_E4M3   x [T, H], out [Mt, H] codes; sf [T, H/128], out_sf [Mt, H/128]; H a multiple of 128
 *   x_type DG_TYPE_BF16   x [T, H], out [Mt, H] bf16; sf, out_sf null; H a multiple of 8
 *   m_indices [Mt] of the contiguous layout, or null. With it the rows without a token in a block of 128 that has some are
 *   zeros (of scale 1e-4 / 448), so that a weight gradient over the padded segments adds nothing for them. All other rows
 *   stay as they were. Mt is then a multiple of 128.
 * x and out 16-byte aligned and apart, k <= 32, about T * H / 256 + Mt < 2^31 (as in the next two calls). Its gradient is
 * dg_moe_combine without weights.
 */
dg_status dg_moe_gather(const void* x, const float* sf, int x_type, const int32_t* rows, const int32_t* m_indices, void* out, float* out_sf,
                        int T, int k, int H, int Mt, cudaStream_t stream);

/*
 * The way back: out[t] = residual[t] + sum_j weights[t,j] * y[rows[t,j]], over the slots whose row is in [0, Mt).
 *   y [Mt, H] bf16, weights [T, k] fp32 or null (1), residual [T, H] bf16 or null, may be out; out [T, H] bf16
 * FP32 sums in the order of j, the residual last, rounded once. H a multiple of 8, k <= 32; y, residual and out 16-byte aligned;
 * out must not overlap y.
 */
dg_status dg_moe_combine(const void* y, const int32_t* rows, const float* weights, const void* residual, void* out, int T, int k,
                         int H, int Mt, cudaStream_t stream);

/*
 * Its gradient (the residual's is dout itself):
 *   dy       [Mt, H] bf16, or null: dy[rows[t,j]] = weights[t,j] * dout[t]; with m_indices zeros as in dg_moe_gather, other
 *            rows as they were
 *   dweights [T, k] fp32, or null: the product of y[rows[t,j]] and dout[t], 0 for a slot without a row. Needs y.
 * weights null: 1. H a multiple of 8, k <= 32; dout, y and dy 16-byte aligned; dy must not overlap y or dout.
 */
dg_status dg_moe_combine_backward(const void* dout, const void* y, const int32_t* rows, const float* weights, const int32_t* m_indices, void* dy,
                                  float* dweights, int T, int k, int H, int Mt, cudaStream_t stream);

/*
 * Root-mean-square norm with the residual's addition:
 *   s = bf16(x + residual),   y = s * rsqrt(mean(s^2) + eps) * weight
 *   x [T, H] bf16, residual [T, H] bf16 or null, weight [H] of weight_type (BF16 or F32)
 *   sum [T, H] bf16, or null: s, the next residual; may be x or residual
 *   y   [T, H] bf16, or null; may be x
 *   q   [T, H] e4m3, sf [T, H/128] fp32, or both null: y quantised (before its rounding to BF16) as in
 *       dg_epilogue_backward; with pow2 the scale is the power of two above that scale, as the UE8M0 path takes it.
 *       H a multiple of 128 then.
 * Sums are FP32 (a row whose squares pass their range, from about 1e19 on, comes out as zeros; squares below 2^-149, of values under
 * 3.7e-23, are lost, which counts only where eps is as small). H a multiple of 8 up to 16384,
 * eps >= 0; weight and the matrices 16-byte aligned.
 */
dg_status dg_rmsnorm(const void* x, const void* residual, const void* weight, int weight_type, void* sum, void* y, uint8_t* q, float* sf,
                     int pow2, int T, int H, float eps, cudaStream_t stream);

/*
 * Its gradient. x is s, what the norm was of (the kept sum); with r = rsqrt(mean(x^2) + eps):
 *   dx      [T, H] bf16 = r * (weight * dy - x * r^2 * mean(weight * dy * x)) + dsum: of x and of the residual alike; may be
 *           dy, x or dsum
 *   dsum    [T, H] bf16, or null: the gradient that reaches the sum by other ways
 *   dweight [H] fp32, or null: the sum over the rows of dy * x * r, in a fixed order; 0 for T = 0
 * workspace: device memory of dg_rmsnorm_backward_workspace(T, H) bytes (-1 for sizes outside the range), 16-byte aligned, with
 * anything in it, needed for dweight.
 */
dg_status dg_rmsnorm_backward(const void* dy, const void* x, const void* weight, int weight_type, const void* dsum, void* dx, float* dweight,
                              void* workspace, int64_t workspace_bytes, int T, int H, float eps, cudaStream_t stream);
int64_t dg_rmsnorm_backward_workspace(int T, int H);

/*
 * The gated activation between the two products of an expert (or of a dense layer), quantised for the second:
 *   h = act(g) * u,   (g; u) = Z's columns [0, I) and [I, 2I)
 *   Z    [M, 2I] bf16
 *   q    [M, I] e4m3, sf [M, I/128]: h in FP32, quantised as in dg_epilogue_backward; pow2 as in dg_rmsnorm. An
 *        activation of less than 2^-119 in magnitude may count as 0, here and in dg_glu_backward
 *   kept [M, 2I] e4m3, kept_sf [M, 2I/128], or both null: Z quantised as in dg_epilogue_backward, what dg_glu_backward takes
 *        instead of Z
 * At most one of (which rows are computed; all others stay as they were):
 *   m_indices [M] of the contiguous layout: the blocks of 128 rows whose first row has an expert. M a multiple of 128 then.
 *   masked_m  [G] of the masked layout [G, M/G, 2I]: the first masked_m[g] rows of each group, at most M/G
 * I a multiple of 128; Z, q and kept 16-byte aligned; no output overlaps Z.
 */
dg_status dg_glu(const void* Z, uint8_t* q, float* sf, uint8_t* kept, float* kept_sf, const int32_t* m_indices, const int32_t* masked_m, int G,
                 int act, int pow2, int M, int I, cudaStream_t stream);

/*
 * Its backward pass, from Z or from the kept codes (one of them; the other null): dg = dH * u * act'(g), du = dH * act(g).
 *   dH [M, I] bf16 (not read, and may be null, without q and qt)
 *   q  [M, 2I] e4m3,   sf  [M, 2I/128]    (dg; du), 1x128 scales along 2I: A of the product that gives the input's gradient
 *   qt [2I, Mp] e4m3,  sft [2I, Mp/128]   the transpose, 1x128 scales along M, Mp = M rounded up to 128, zeros past M
 *   ht [I, Mp] e4m3,   hsft [I, Mp/128]   h's transpose, so quantised: an operand of the second product's weight gradient
 * q with sf, qt with sft, ht with hsft may each be null. The values are those of Z, or of the codes times their scales in FP32,
 * quantised as in dg_epilogue_backward; every row is computed. I a multiple of 128, M free; matrices 16-byte aligned.
 */
dg_status dg_glu_backward(const void* dH, const void* Z, const uint8_t* kept, const float* kept_sf, int act, uint8_t* q, float* sf, uint8_t* qt,
                          float* sft, uint8_t* ht, float* hsft, int M, int I, cudaStream_t stream);

/*
 * The values of 8-bit codes quantised along the other axis: from q [M, N] e4m3 with sf [M, N/128], what a forward product
 * read, to qt [N, Mp] with sft [N, Mp/128] (Mp = M rounded up to 128, zeros past M), an operand of dg_wgrad_fp8_nt or
 * dg_k_grouped_wgrad: the 8-bit codes are all that has to be kept of an activation for its weight gradient. The value of a
 * code is its product with its scale, rounded to FP32, and quantised as in dg_epilogue_backward. N a multiple of 128, M free;
 * q and qt 16-byte aligned and apart.
 */
dg_status dg_transpose_fp8(const uint8_t* q, const float* sf, uint8_t* qt, float* sft, int M, int N, cudaStream_t stream);

/* Human-readable name of a status code (static storage). */
const char* dg_status_string(dg_status status);

/*
 * Synchronises `stream`, then reports (and clears) the device-side error recorded by any dg kernel on
 * the current device since the last call: DG_DEVICE_TIMEOUT, or DG_SCALE_NOT_UE8M0 from the UE8M0
 * path, else DG_CUDA_ERROR if the synchronisation failed, else DG_OK. Kernels record only the first
 * error (a later one does not overwrite it). Reading and clearing are two steps: an error that a dg
 * kernel on another stream records between them is lost, so call this while no other dg work runs on
 * the device when every error must be seen.
 */
dg_status dg_device_status(cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DG_H */
