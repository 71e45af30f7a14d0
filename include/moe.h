/*
 * libmoe - GB300 (sm_103a) hot path of a LatentMoE sparse expert layer:
 * sigmoid router with top-k selection, token permute, latent projections,
 * grouped SwiGLU experts over ragged expert batches, weighted combine, and
 * the backward of each step.
 *
 * Sources. The pages that describe this layer give its structure, not its
 * formulas:
 *   [MODEL]   "TorchTitan Ascend开源:插件化支持TorchTitan,实现Kimi K3.1 Pro的昇腾适配与训练实践",
 *             section "Kimi K3.1 Pro 模型结构", LatentMoE paragraph: 896 routed and
 *             2 shared experts, 16 routed experts active per token, expert compute
 *             in a low-dimensional latent space.
 *   [OPS]     "昇腾实现Kimi K3.1 Pro模型LoRA训练适配,助力2.8万亿级大模型高效训练",
 *             section "MoE(Mixture of Experts):算子融合与通信协同": dynamic routing,
 *             token dispatch, and Permute / Unpermute / Grouped GEMM as the core
 *             operators, with less data movement during token reordering as a goal.
 *   [LOAD]    "TorchTitan Ascend开源 ...", section "在线负载规划": per-expert load is
 *             counted from the current routing result.
 *   [GGEMM]   same page, section "权重预取与梯度归约": one Grouped GEMM runs all
 *             experts of a device through a unified compute view.
 *   [SWAP]    the [OPS] page, section "Swap Core:算子级精准缓存与异步 Offload 协同,
 *             训练性能提升 15%": outputs of selected MatMul/GMM operators are cached
 *             for the backward, optionally compressed by FP8 activation
 *             quantization and dequantization.
 * Where the pages are silent the library takes these readings: the router is
 * sigmoid(x @ Wr (+ bias)) on the model-width input, the k largest logits are
 * selected (lower expert id wins a tie) and their sigmoids renormalised to sum
 * to 1; an expert is o = (silu(z Wg) * (z Wu)) W2 on the latent z = x W_dn; the
 * routing weight scales the expert output; the shared experts run on z with
 * weight 1; out = (sum_j w_j o_j + sum_s shared_s(z)) W_up; tokens of one expert
 * are kept in ascending token order; no token is dropped.
 *
 * Conventions of every entry point:
 *  - Tensor pointers are DEVICE pointers owned by the caller; the library never
 *    allocates, frees or synchronises. Pointers must be 16-byte aligned.
 *  - bf16 tensors are passed as uint16_t (bfloat16 bit patterns), row-major.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    All work is enqueued on it; the call returns before the work runs.
 *  - Return value: MOE_OK or a negative MOE_ERR_* code. Argument errors are
 *    detected on the host before anything is enqueued. MOE_ERR_CUDA means a
 *    launch failed; moe_last_cuda_error() gives the cudaError_t.
 *  - Data errors found on the device (an expert id outside [0,E), a NaN/Inf
 *    logit, a kernel wait that timed out) OR bits into the caller's device
 *    word `err_flag` (nullable where listed) instead of trapping; the caller
 *    reads it when it chooses. Rows with a bad expert id are skipped.
 *  - Dimension limits: l, f, d multiples of 64; E <= 1024 (and a multiple of
 *    64 where a GEMM has E columns); 1 <= k <= min(E, 32); T*k < 2^31.
 *  - Index arrays that moe_permute writes (offsets, tile_sched, slot_of,
 *    token_of) are trusted by the calls that read them: pass them as written,
 *    or with the same invariants. A negative slot or token entry means "no
 *    row"; other entries are not range-checked on the device. Expert ids
 *    (topk_idx) are checked, as above.
 *  - Weight layouts: W13 [E][l][2f] (gate columns 0..f-1, up columns f..2f-1),
 *    W2 [E][f][l]; shared experts use the same layout with E -> S; Wr [d][E],
 *    W_dn [d][l], W_up [l][d].
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_ERR_ARG (-1)         /* null pointer or dimension out of range        */
#define MOE_ERR_ALIGN (-2)       /* pointer not 16-byte aligned / dim not x64      */
#define MOE_ERR_WORKSPACE (-3)   /* workspace smaller than moe_workspace_size()    */
#define MOE_ERR_UNSUPPORTED (-4) /* shape or option this build does not handle     */
#define MOE_ERR_CUDA (-5)        /* a CUDA call failed, see moe_last_cuda_error()  */

/* bits of the device error word */
#define MOE_FLAG_BAD_EXPERT 1 /* expert id outside [0, E) */
#define MOE_FLAG_NONFINITE 2  /* NaN or Inf router logit   */
#define MOE_FLAG_TIMEOUT 4    /* a kernel wait gave up     */
#define MOE_FLAG_BAD_INDEX 8  /* sequence bounds or cache slot out of range */

/* element types (weight gradients, optimizer tensors) */
#define MOE_DTYPE_F32 0
#define MOE_DTYPE_BF16 1
#define MOE_DTYPE_E4M3 2 /* outputs of moe_rmsnorm_fwd */

/* scores of moe_route_scores */
#define MOE_SCORE_SIGMOID 0
#define MOE_SCORE_SOFTMAX 1

/* operations with a workspace, for moe_workspace_size */
#define MOE_OP_ROUTE_TOPK 1
#define MOE_OP_PERMUTE 2
#define MOE_OP_GROUPED_SWIGLU_BWD 3
#define MOE_OP_SHARED_SWIGLU_BWD 4
#define MOE_OP_ROUTE_TOPK_BWD 5
#define MOE_OP_ROUTER_AUX 6
#define MOE_OP_LINATTN_FWD 7
#define MOE_OP_LINATTN_BWD 8
#define MOE_OP_ADAMW_PLAN 9
#define MOE_OP_ADAMW_STEP 10
#define MOE_OP_RMSNORM_BWD 11
#define MOE_OP_CONV_BWD 12
#define MOE_OP_SCAN_FWD 13
#define MOE_OP_SCAN_BWD 14
#define MOE_OP_SCAN_TILE_STATES 15

int moe_version(void);
const char* moe_status_string(int status);
int moe_last_cuda_error(void);

/* Bytes of workspace `op` needs for these sizes (unused sizes may be 0).
 * The workspace is device memory owned by the caller, 256-byte aligned. */
size_t moe_workspace_size(int op, int T, int d, int l, int E, int k, int f, int S);

/* ---------------------------------------------------------------- routing */

/* Router logits L[T][E] (fp32) = x[T][d] @ Wr[d][E] (bf16 in, fp32 accumulate),
 * the router of [OPS] "dynamic routing" read as a linear scorer on x.
 * E must be a multiple of 64. */
int moe_router_logits(const uint16_t* x, const uint16_t* Wr, int T, int d, int E, float* logits,
                      void* stream);

/* Top-k selection and weights from given fp32 logits ([MODEL]: 16 of 896).
 * For token t: v[e] = logits[t][e] + bias[e] (fp32 add; bias nullable);
 * topk_idx[t][j] (int32) lists the k largest v, ordered by (v desc, id asc);
 * topk_s[t][j] = sigmoid(v) (fp32); topk_w[t][j] = topk_s[t][j] / sum_j topk_s[t][j].
 * A NaN/Inf v sets MOE_FLAG_NONFINITE. Any E <= 1024. err_flag nullable. */
int moe_topk_from_logits(const float* logits, const float* bias, int T, int E, int k,
                         int32_t* topk_idx, float* topk_w, float* topk_s, int32_t* err_flag,
                         void* stream);

/* moe_router_logits followed by moe_topk_from_logits; the logits live in the
 * workspace (moe_workspace_size(MOE_OP_ROUTE_TOPK, T, 0, 0, E, 0, 0, 0) bytes). */
int moe_route_topk(const uint16_t* x, const uint16_t* Wr, const float* bias, int T, int d, int E,
                   int k, int32_t* topk_idx, float* topk_w, float* topk_s, void* ws,
                   size_t ws_bytes, int32_t* err_flag, void* stream);

/* moe_route_topk and the latent down-projection z[T][l] (bf16) = x @ W_dn[d][l]
 * ([MODEL]: experts computed in the latent space; the projection reads the same x)
 * in one call: when T > 128 and E is a multiple of 128 one GEMM over [Wr | W_dn]
 * reads x once (logits and z are bit-identical to the two separate calls), else
 * moe_router_logits + moe_latent_proj. Same workspace as moe_route_topk (the
 * logits stay in it); l a multiple of 64; z 16-byte aligned. */
int moe_route_topk_latent(const uint16_t* x, const uint16_t* Wr, const float* bias,
                          const uint16_t* W_dn, int T, int d, int E, int k, int l,
                          int32_t* topk_idx, float* topk_w, float* topk_s, uint16_t* z, void* ws,
                          size_t ws_bytes, int32_t* err_flag, void* stream);

/* Auxiliary load-balance loss of the routing stage ("大模型落地昇腾" page, section
 * "三、通信侧": an auxiliary loss that constrains the entropy of the routing
 * distribution), read as the negative entropy of the batch's mean routing
 * distribution over all experts:
 *   P(e|t) = s[t][e] / sum_e' s[t][e'],  s = sigmoid(logits + bias)   (bias nullable)
 *   p_mean[e] = (1/T) sum_t P(e|t)  (fp32, E);  loss = sum_e p_mean[e] ln p_mean[e]  (fp32, 1)
 * The loss is -ln E when the routing mass is spread evenly. Deterministic
 * (fixed-order reductions). Workspace: moe_workspace_size(MOE_OP_ROUTER_AUX, T, 0, 0, E, ...).
 * Its gradient is added by moe_route_topk_bwd (aux_* arguments). */
int moe_router_aux_loss(const float* logits, const float* bias, int T, int E, float* p_mean,
                        float* loss, void* ws, size_t ws_bytes, void* stream);

/* The router's logits and the latent z of moe_route_topk_latent without the selection. */
int moe_router_logits_latent(const uint16_t* x, const uint16_t* Wr, const uint16_t* W_dn, int T, int d, int E, int l,
                             float* logits, uint16_t* z, void* stream);

/* Selection from fp32 logits with scores, a bias for balance and groups of experts:
 *   s = sigmoid(logits) or softmax(logits) over the E experts (score)
 *   c = s + bias   (bias fp32 [E] chooses only; without one the logits themselves take c's place)
 * The experts are `groups` runs of E / groups; a group's value is the sum of its group_top (1 or 2) largest c
 * (sums of scores without a bias), and the group_k groups with the largest values stay. Of their experts
 * topk_idx[t][j] (int32) lists the k largest c, ordered by (c desc, id asc); groups of equal value go by their
 * index. topk_s[t][j] = s; topk_w[t][j] = scale * s / (sum of the k scores), or scale * s without renorm.
 * The choice is that of values in 64 bits, so it does not depend on how scores are rounded here.
 * A logit or bias of -infinity takes the expert out: it adds nothing to its group's value, comes after all
 * others, and its score and weight are 0 where there are too few others. A NaN or +infinity does the same and sets
 * MOE_FLAG_NONFINITE. Renormalised weights stay right where the scores themselves leave fp32.
 * groups divides E and is at most 32; group_k * (E / groups) >= k. err_flag nullable. */
int moe_route_scores(const float* logits, const float* bias, int T, int E, int k, int score, int groups, int group_k,
                     int group_top, int renorm, float scale, int32_t* topk_idx, float* topk_w, float* topk_s,
                     int32_t* err_flag, void* stream);

/* Gradient of moe_route_scores' logits, d_logits[T][E] (fp32 or bf16), for the weights' gradient g:
 *   renorm            d_l = w_j (g_j - sum_i w_i g_i / scale), times (1 - s_j) for the sigmoid; 0 for the others
 *   sigmoid           d_l = g_j w_j (1 - s_j); 0 for the others
 *   softmax           d_l[e] = scale p_e (g_e [e chosen] - sum_j s_j g_j), p the softmax of `logits` (needed here)
 *                     (16-byte aligned where E is a multiple of 4)
 * For the sigmoid `logits` may be NULL: 1 - s_j is then that of the fp32 score, off by 2^-23, which is 4 % of it at a logit of 14 and
 * all of it above 17; from the logits it is right to fp32. With renormalised softmax scores they are not read.
 * g_j = d_w[t][j], or, with slot_of (of moe_permute), d_w[slot_of[t][j]] of moe_grouped_swiglu_bwd's d_row_w (0 for a
 * negative slot; one of T k or above sets MOE_FLAG_BAD_INDEX and counts as one). d_topk_w (nullable) receives g. The choice is piecewise constant and the bias a constant: no
 * gradient. An id outside [0, E), or one that its row has named before, has none either and sets
 * MOE_FLAG_BAD_EXPERT. scale must not be 0. */
int moe_route_scores_bwd(const float* d_w, const int32_t* slot_of, const float* logits, const int32_t* topk_idx,
                         const float* topk_w, const float* topk_s, int T, int E, int k, int score, int renorm, float scale,
                         void* d_logits, int dtype, float* d_topk_w, int32_t* err_flag, void* stream);

/* The products of moe_route_topk_bwd for a given dL = d_logits (bf16 [T][E]): dx_accum += dL @ Wr^T, or, with dz,
 * dx_accum = dz @ W_dn^T + dL @ Wr^T; dWr = x^T @ dL (fp32 or bf16). */
int moe_router_grads(const uint16_t* d_logits, const uint16_t* x, const uint16_t* Wr, int T, int d, int E,
                     uint16_t* dx_accum, void* dWr, int wgrad_dtype, const uint16_t* dz, const uint16_t* W_dn, int l,
                     void* stream);

/* ---------------------------------------------------------------- norm */

/* Root-mean-square norm of x + residual:
 *   u = x + residual (residual nullable: u = x);  rstd = 1 / sqrt(mean(u^2) + eps);  y = u rstd weight
 * x bf16 [T][d], ldx elements between rows; residual and sum [T][d] of res_dtype (fp32 or bf16); weight fp32 [d]. sum
 * receives u (given exactly when residual is, and may be residual); y is computed from u before it is rounded. y_dtype MOE_DTYPE_BF16:
 * y bf16 [T][d]. MOE_DTYPE_E4M3: y holds E4M3 bytes of y / y_scale (rounded to nearest even), y_scale fp32 [T][ceil(d / block)] = each
 * block's largest magnitude / 448, for blocks of 64 or 128 columns or of the whole row (block = d); a block
 * whose largest magnitude is below 2^-100 has scale 0. Any
 * finite u is handled, those whose squares pass fp32 too. d is a multiple of 8 up to 16384, ldx of 8; eps > 0. */
int moe_rmsnorm_fwd(const uint16_t* x, const void* residual, const float* weight, int T, int d, int ldx, int res_dtype,
                    float eps, void* sum, void* y, int y_dtype, float* y_scale, int block, void* stream);

/* Backward of moe_rmsnorm_fwd for dy (bf16 [T][d]) and d_sum = d loss / d sum (res_dtype [T][d], nullable), from u (sum, or x where
 * there was no residual; ldu elements between rows, res_dtype): with rstd of u, g = dy weight, n = u rstd,
 *   du = rstd (g - n mean(g n)) + d_sum;  dw[d] = sum_t dy n   (fp32, nullable)
 * du is the gradient of x and of residual alike: dx receives it in bf16, d_residual in res_dtype (either may be NULL).
 * Either may take the place of dy, u or d_sum (of its type and row distance), and shares no other memory with them.
 * Deterministic. Workspace (for dw): moe_workspace_size(MOE_OP_RMSNORM_BWD, T, d, ...). */
int moe_rmsnorm_bwd(const uint16_t* dy, const void* u, const float* weight, const void* d_sum, int T, int d,
                    int ldu, int res_dtype, float eps, uint16_t* dx, void* d_residual, float* dw, void* ws,
                    size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- permute */

/* Token Permute of [OPS] with the per-expert load count of [LOAD].
 *   counts[e]      = #{(t,j) : topk_idx[t][j] == e}                      (int32, E)
 *   offsets[e]     = counts[0] + ... + counts[e-1]; offsets[E] = total  (int32, E+1)
 *   slot_of[t][j]  = offsets[e] + #{t' < t : e in topk_idx[t']}, e = topk_idx[t][j]
 *                    (tokens of one expert in ascending token order; -1 for a bad id)
 *   token_of[r]    = t with slot_of[t][j] == r (int32, T*k; -1 past offsets[E])
 *   tile_sched[e]  = sum_{e'<e} ceil(counts[e'] / 128) (int32, E+1): the 128-row
 *                    tile ranges the grouped GEMMs walk on the device
 *   row_w[r]       = topk_w[t][j] for r = slot_of[t][j] (fp32 [T*k]; skipped when
 *                    topk_w or row_w is NULL): the routing weight of each permuted row
 *   z_perm[r][:]   = z[token_of[r]][:] (bf16 [T*k][l]); skipped when z is NULL.
 * The k ids of a token must be distinct (a repeat sets MOE_FLAG_BAD_EXPERT).
 * Deterministic, no atomics on the output. Workspace:
 * moe_workspace_size(MOE_OP_PERMUTE, T, 0, 0, E, 0, 0, 0). err_flag nullable. */
int moe_permute(const uint16_t* z, const int32_t* topk_idx, const float* topk_w, int T, int l,
                int E, int k, uint16_t* z_perm, int32_t* counts, int32_t* offsets,
                int32_t* slot_of, int32_t* token_of, int32_t* tile_sched, float* row_w,
                void* ws, size_t ws_bytes, int32_t* err_flag, void* stream);

/* Allocation-free variant of moe_permute, for callers that cannot allocate
 * device memory (a caller that is handed only its input and output buffers,
 * or one on a fixed memory budget that must not call cudaMalloc/cudaFree,
 * which may also synchronise the device). The pages describe nothing like it;
 * it computes exactly what moe_permute computes, with the same arguments
 * except ws / ws_bytes. Its scratch is a fixed 1 MiB array inside the library
 * (held on every GPU that loads the library until it is unloaded), so it
 * handles permute_chunks(T) * E <= 262144, i.e. ceil(T / 256) * E <= 262144
 * (T <= 74,752 at E = 896); larger problems return MOE_ERR_WORKSPACE without
 * launching anything. The first call on a device (and the first one after the
 * device's current CUDA context changed, e.g. after cudaDeviceReset) looks up
 * the array's device address; make that first call before any stream capture.
 * All calls share the array, which keeps the last call's contents (no entry of
 * it needs to start at zero): calls that may overlap on the GPU race on it and
 * must be serialised by the caller. MOE_ERR_CUDA, when the address lookup
 * fails, comes with its cause in moe_last_cuda_error(). */
int moe_permute_noalloc(const uint16_t* z, const int32_t* topk_idx, const float* topk_w, int T,
                        int l, int E, int k, uint16_t* z_perm, int32_t* counts, int32_t* offsets,
                        int32_t* slot_of, int32_t* token_of, int32_t* tile_sched, float* row_w,
                        int32_t* err_flag, void* stream);

/* Online load plan with dynamic expert replicas for an expert-parallel layout
 * ("TorchTitan Ascend开源" page, sections "在线负载规划" and
 * "MoonEP动态负载均衡与专家并行优化": per-expert loads of the current batch and
 * each device's remaining capacity decide the replicas of hot experts; a token
 * keeps its expert). Reading: P ranks, rank r owns experts [r*E/P, (r+1)*E/P)
 * (E divisible by P), every rank processes at most C = ceil(sum counts / P)
 * rows. Ranks first take their own experts' rows while they have room; the
 * rest of each expert goes, in rank order, to ranks with spare capacity.
 * Output: pieces[i][4] = {expert, rank, first row within the expert's
 * segment, rows} for i < *n_pieces (capacity 2E + P pieces, int32),
 * rank_load[P] = rows per rank (max = C). Runs on the device from the counts
 * of moe_permute (no host synchronisation). E + P <= 2048. Counts that are
 * negative or sum to 2^31 or more give *n_pieces = -1 and no plan. */
int moe_replica_plan(const int32_t* counts, int E, int P, int32_t* pieces, int32_t* n_pieces,
                     int32_t* rank_load, void* stream);

/* ---------------------------------------------------------------- projections */

/* Latent projection of [MODEL]: out[M][N] (bf16) = in[M][K] @ W[K][N] (bf16,
 * fp32 accumulate) on the tcgen05 tensor cores. K, N multiples of 64. */
int moe_latent_proj(const uint16_t* in, const uint16_t* W, int M, int K, int N, uint16_t* out,
                    void* stream);

/* Backward of moe_latent_proj for dout[M][N]:
 *   din[M][K] (bf16) = dout @ W^T      (skipped when din is NULL)
 *   dW[K][N]          = in^T @ dout    (skipped when dW is NULL; fp32 or bf16 per wgrad_dtype) */
int moe_latent_proj_bwd(const uint16_t* dout, const uint16_t* in, const uint16_t* W, int M, int K,
                        int N, uint16_t* din, void* dW, int wgrad_dtype, void* stream);

/* ---------------------------------------------------------------- experts */

/* Grouped SwiGLU experts over the permuted rows ([OPS] Grouped GEMM, [GGEMM]).
 * For every expert e and row r in [offsets[e], offsets[e+1]):
 *   [g|u][r] = z_perm[r] @ W13[e]              (fp32 accumulate)
 *   h[r]     = silu(g[r]) * u[r]               (bf16 [R][f])
 *   y_perm[r]= row_w[r] * (h[r] @ W2[e])       (bf16 [R][l]; row_w nullable => 1)
 *   gu_save[r] = [g|u][r] in bf16 ([R][2f], nullable) for the backward.
 * R is the row capacity of the buffers (>= offsets[E]); rows past offsets[E]
 * are not touched. offsets/tile_sched come from moe_permute. Empty experts
 * cost nothing (no tile, no weight read). No host synchronisation. */
int moe_grouped_swiglu(const uint16_t* z_perm, const uint16_t* W13, const uint16_t* W2,
                       const int32_t* offsets, const int32_t* tile_sched, const float* row_w,
                       int E, int R, int l, int f, uint16_t* gu_save, uint16_t* h,
                       uint16_t* y_perm, void* stream);

/* moe_grouped_swiglu with the GMM output [g|u] cached for the backward in FP8
 * ([SWAP]) instead of bf16: E4M3 (round to nearest even, saturating at +-448)
 * of g / s and u / s, with one power-of-two scale s per row and 64-feature block,
 * the smallest with max |block| <= 448 s (1 when that maximum is below 2^-100):
 *   gu8[r][32q + i]         E4M3 bytes [R][2f]: g[r][16q + i] (i < 16), u[r][16q + i - 16]
 *                           (16 <= i < 32): 16-feature groups of g and u in turn
 *   gu_scale[r][b]          fp32 [R][2f/64]: blocks of g (b < f/64), then of u
 * h and y_perm are exactly those of moe_grouped_swiglu. f must be a multiple of
 * 128 (MOE_ERR_UNSUPPORTED otherwise); gu8 16-byte aligned. The cache takes 1 + 1/16
 * bytes per value instead of 2. */
int moe_grouped_swiglu_fp8cache(const uint16_t* z_perm, const uint16_t* W13, const uint16_t* W2,
                                const int32_t* offsets, const int32_t* tile_sched,
                                const float* row_w, int E, int R, int l, int f, uint8_t* gu8,
                                float* gu_scale, uint16_t* h, uint16_t* y_perm, void* stream);

/* Multi-bucket batching ("大模型落地昇腾" page, section "二、算力侧": experts with
 * similar token counts grouped into buckets, each with one batch shape), read
 * for this engine as an expert order: bucket class 0 for an empty expert, else
 * 1 + floor(log2(ceil(count / 128))); experts by class, largest first,
 * ascending id within a class, empty experts last (expert_order[E]); and
 * tile_sched_ordered[E+1], the exclusive scan of ceil(count / 128) in that
 * order. One CTA on the device from moe_permute's counts; E <= 1024. */
int moe_expert_buckets(const int32_t* counts, int E, int32_t* expert_order,
                       int32_t* tile_sched_ordered, void* stream);

/* moe_grouped_swiglu walking the experts in a given order (tile_sched_ordered
 * and expert_order from moe_expert_buckets): the persistent tiles then run
 * the big experts first. Results are identical to moe_grouped_swiglu. */
int moe_grouped_swiglu_ordered(const uint16_t* z_perm, const uint16_t* W13, const uint16_t* W2,
                               const int32_t* offsets, const int32_t* tile_sched_ordered,
                               const int32_t* expert_order, const float* row_w, int E, int R,
                               int l, int f, uint16_t* gu_save, uint16_t* h, uint16_t* y_perm,
                               void* stream);

/* moe_grouped_swiglu with the permute fused into GEMM1's operand load: the
 * permuted rows are never written. z is the unpermuted latent [T][l] and
 * permuted row r is z[token_of[r]] (token_of from moe_permute, which can then
 * be called with z = NULL); warps of the GEMM kernel copy the rows (16-byte
 * cp.async, z kept in L2) straight into the swizzled shared-memory tile. Results
 * are identical to moe_permute + moe_grouped_swiglu. This is the "less data
 * movement during token reordering" direction of [OPS]. */
int moe_grouped_swiglu_gather(const uint16_t* z, const int32_t* token_of, int T,
                              const uint16_t* W13, const uint16_t* W2, const int32_t* offsets,
                              const int32_t* tile_sched, const float* row_w, int E, int R, int l,
                              int f, uint16_t* gu_save, uint16_t* h, uint16_t* y_perm,
                              void* stream);

/* Shared experts of [MODEL] on all T latent rows, weight 1:
 *   [g_s|u_s] = z @ W13_sh[s];  h[:, s*f:(s+1)*f] = silu(g_s) * u_s   (h: bf16 [T][S*f])
 *   y_sh = sum_s h_s @ W2_sh[s]  (bf16 [T][l]);  gu_save: bf16 [T][S*2f], block s
 *   at columns s*2f.. (nullable). */
int moe_shared_swiglu(const uint16_t* z, const uint16_t* W13_sh, const uint16_t* W2_sh, int T,
                      int l, int f, int S, uint16_t* gu_save, uint16_t* h, uint16_t* y_sh,
                      void* stream);

/* ---------------------------------------------------------------- combine */

/* Unpermute + weighted combine of [OPS]: for every token t,
 *   y_lat[t] = sum_{j=0..k-1} y_perm[slot_of[t][j]] (+ y_shared[t])
 * summed in fp32 in that order, stored as bf16 [T][l]. y_shared nullable;
 * slot_of entries < 0 are skipped. With k = 1 this is the return of permuted
 * rows to arrival order. */
int moe_unpermute_combine(const uint16_t* y_perm, const int32_t* slot_of,
                          const uint16_t* y_shared, int T, int k, int l, uint16_t* y_lat,
                          void* stream);

/* Backward of the combine: dy_perm[r] = dy_lat[token_of[r]] for r < T*k
 * (zeros where token_of[r] < 0). bf16. */
int moe_unpermute_combine_bwd(const uint16_t* dy_lat, const int32_t* token_of, int T, int k, int l,
                              uint16_t* dy_perm, void* stream);

/* ---------------------------------------------------------------- backward */

/* Backward of moe_grouped_swiglu for dy_perm = d loss / d y_perm, routing fixed:
 *   dh_u[r]   = dy_perm[r] @ W2[e]^T;  d_row_w[r] = <dh_u[r], h[r]>  (fp32 [R])
 *   dh[r]     = row_w[r] * dh_u[r]
 *   dg = dh * u * s(g) * (1 + g (1 - s(g))),  du = dh * silu(g)   (s = sigmoid)
 *   dz_perm[r]= [dg|du][r] @ W13[e]^T                               (bf16 [R][l])
 *   dW2[e]    = sum_r (row_w[r] h[r])^T dy_perm[r]                  ([E][f][l])
 *   dW13[e]   = sum_r z_perm[r]^T [dg|du][r]                         ([E][l][2f])
 * dW13/dW2 are fp32 or bf16 per wgrad_dtype; an expert with no rows gets exact
 * zeros. The weight gradients of expert e read no more than a few of the rows
 * that follow its segment, multiplied by zero: they are exact as long as every
 * row of dy_perm / [dg|du] is finite (a non-finite row of expert e+1 may also
 * turn dW of expert e into NaN). gu_save and h from the forward are required. Workspace:
 * moe_workspace_size(MOE_OP_GROUPED_SWIGLU_BWD, 0, 0, l, E, 0, f, 0) with T*k = R
 * passed as T (k = 1). */
int moe_grouped_swiglu_bwd(const uint16_t* dy_perm, const uint16_t* z_perm, const uint16_t* W13,
                           const uint16_t* W2, const uint16_t* gu_save, const uint16_t* h,
                           const float* row_w, const int32_t* offsets, const int32_t* tile_sched,
                           int E, int R, int l, int f, uint16_t* dz_perm, float* d_row_w,
                           void* dW13, void* dW2, int wgrad_dtype, void* ws, size_t ws_bytes,
                           void* stream);

/* moe_grouped_swiglu_bwd reading g and u from the FP8 cache of
 * moe_grouped_swiglu_fp8cache (gu8 * scale of its block) in the SwiGLU
 * derivative (dg, du); h, and with it dW2 and d_row_w, is the bf16 forward's
 * as in moe_grouped_swiglu_bwd. Same workspace. */
int moe_grouped_swiglu_bwd_fp8cache(const uint16_t* dy_perm, const uint16_t* z_perm,
                                    const uint16_t* W13, const uint16_t* W2, const uint8_t* gu8,
                                    const float* gu_scale, const uint16_t* h, const float* row_w,
                                    const int32_t* offsets, const int32_t* tile_sched, int E,
                                    int R, int l, int f, uint16_t* dz_perm, float* d_row_w,
                                    void* dW13, void* dW2, int wgrad_dtype, void* ws,
                                    size_t ws_bytes, void* stream);

/* moe_grouped_swiglu_bwd with both permutes fused into the operand loads:
 * dy_perm[r] = dy_lat[token_of[r]] and z_perm[r] = z[token_of[r]] are gathered
 * inside the dgrad and wgrad GEMMs (dy_lat, z: [T][l]), so neither the
 * combine backward gather nor the permuted activations are materialised.
 * Results are identical to moe_grouped_swiglu_bwd on the permuted tensors. */
int moe_grouped_swiglu_bwd_gather(const uint16_t* dy_lat, const uint16_t* z,
                                  const int32_t* token_of, int T, const uint16_t* W13,
                                  const uint16_t* W2, const uint16_t* gu_save, const uint16_t* h,
                                  const float* row_w, const int32_t* offsets,
                                  const int32_t* tile_sched, int E, int R, int l, int f,
                                  uint16_t* dz_perm, float* d_row_w, void* dW13, void* dW2,
                                  int wgrad_dtype, void* ws, size_t ws_bytes, void* stream);

/* Backward of moe_shared_swiglu for dy = d loss / d y_sh ([T][l]):
 *   dz_sh = sum_s [dg_s|du_s] @ W13_sh[s]^T (bf16 [T][l]); dW13_sh [S][l][2f];
 *   dW2_sh [S][f][l] (fp32 or bf16). gu_save from the forward is required; `h`
 *   (the forward's [T][S*f] SwiGLU output) is the A operand of the dW2_sh product.
 * Workspace: moe_workspace_size(MOE_OP_SHARED_SWIGLU_BWD, T, 0, l, 0, 0, f, S) (the gate/up
 * gradients plus, at large T, fp32 partials of the K-split weight gradients). */
int moe_shared_swiglu_bwd(const uint16_t* dy, const uint16_t* z, const uint16_t* W13_sh,
                          const uint16_t* W2_sh, const uint16_t* gu_save, const uint16_t* h,
                          int T, int l, int f, int S, uint16_t* dz_sh, void* dW13_sh,
                          void* dW2_sh, int wgrad_dtype, void* ws, size_t ws_bytes,
                          void* stream);

/* Backward of the permute: dz[t] = sum_j dz_perm[slot_of[t][j]] (+ dz_shared[t]),
 * fp32 sum in j order, bf16 [T][l]. dz_shared nullable. */
int moe_permute_bwd(const uint16_t* dz_perm, const int32_t* slot_of, const uint16_t* dz_shared,
                    int T, int k, int l, uint16_t* dz, void* stream);

/* Backward of the router for d_row_w (from moe_grouped_swiglu_bwd):
 *   d_topk_w[t][j] = d_row_w[slot_of[t][j]]                         (fp32, nullable out)
 *   ds_j = (d_topk_w_j - sum_i w_i d_topk_w_i) / sum_i s_i;  dL[t][idx_j] = ds_j s_j (1 - s_j),
 *   zero for unselected experts (the selection is piecewise constant; the bias
 *   is a constant and gets no gradient)
 *   with aux_logits != NULL, dL also gets the gradient of aux_scale * the
 *   auxiliary balance loss (moe_router_aux_loss on aux_logits + aux_bias, whose
 *   p_mean is aux_p_mean): dense over all E experts,
 *   dL[t][e] += aux_scale s(1-s) / (T S_t) (ln p_mean[e] - sum_e' P(e'|t) ln p_mean[e'])
 *   dx_accum[T][d] += dL @ Wr^T  (bf16, read-modify-write), or, when dz is given,
 *   dx_accum = dz @ W_dn^T + dL @ Wr^T (overwrite; one GEMM over K = l + E that
 *   fuses the down-projection's input gradient: dz [T][l], W_dn [d][l])
 *   dWr[d][E] = x^T @ dL         (fp32 or bf16)
 * E must be a multiple of 64. Workspace (dL in bf16):
 * moe_workspace_size(MOE_OP_ROUTE_TOPK_BWD, T, 0, 0, E, 0, 0, 0). */
int moe_route_topk_bwd(const float* d_row_w, const int32_t* slot_of, const int32_t* topk_idx,
                       const float* topk_w, const float* topk_s, const uint16_t* x,
                       const uint16_t* Wr, int T, int d, int E, int k, float* d_topk_w,
                       uint16_t* dx_accum, void* dWr, int wgrad_dtype, const float* aux_logits,
                       const float* aux_bias, const float* aux_p_mean, float aux_scale,
                       const uint16_t* dz, const uint16_t* W_dn, int l, void* ws,
                       size_t ws_bytes, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------- sequence mixer */

/* Linear attention with a decay for each state head. Hs state heads, each shared
 * by r query heads (query head h*r + a reads state head h), so Hq = Hs * r. With
 * lam = exp(log_decay[h]), for the tokens of one sequence in order:
 *   S_t     = lam S_{t-1} + k_t v_t^T              (Dk x Dv, fp32)
 *   o_t^(a) = scale * S_t^T q_t^(a)
 * log_decay is a constant of the head (fp32 [Hs], <= 0; 0 keeps everything, -inf
 * keeps nothing): it gets no gradient. A NaN or positive entry sets
 * MOE_FLAG_NONFINITE and counts as 0.
 * Tensors: q [T][Hq][Dk], k [T][Hs][Dk], v [T][Hs][Dv], o [T][Hq][Dv], bf16; the heads
 * of one token are contiguous and ld* elements lie between tokens (ld* >= heads *
 * width), so q, k and v may be slices of one fused projection's rows. Dk and Dv are
 * multiples of 8 up to 128; ld* are multiples of 8. States are fp32 [N][Hs][Dk][Dv],
 * 32-byte aligned.
 * Sequences: N of them packed on the token axis; sequence n is the tokens
 * cu_seqlens[n] .. cu_seqlens[n+1]-1 (int32 [N+1], device) and may be empty.
 * max_seqlen is an upper bound of their lengths, known on the host (any int32; the time axis is
 * split by it, so a loose one costs time and workspace). A sequence
 * that is out of order, past T or longer than max_seqlen sets MOE_FLAG_BAD_INDEX and is
 * skipped: nothing of it is written. cu_seqlens == NULL means N sequences of T / N
 * tokens (T divisible by N).
 * state_in (nullable: zeros) is each sequence's state before its first token,
 * state_out (nullable) its state after the last; an empty sequence copies one to
 * the other. state_out may be state_in, but not overlap it in part; o shares no memory with
 * the inputs. Rows of o that belong to no sequence keep what they hold; rows that two
 * sequences claim (the second one's start lying before the first one's end) get either's values.
 * Precision: states are held, carried and summed in fp32, but the tensor cores that make the sums take
 * bf16. The decayed keys enter a state as two bf16 terms (16 bits): 3e-6 of the state (rms), where fp32
 * throughout has 5e-7. The scores, and the copy of the state that a chunk's queries read, are one bf16
 * term for Dk > 64: o is then 2.4e-3 off (rms), rounding o alone being 1.7e-3. For Dk <= 64 they are
 * two terms and o has its own rounding's error. moe_linattn_step is fp32 throughout.
 * Workspace: moe_workspace_size(MOE_OP_LINATTN_FWD, max_seqlen, Dk, Dv, Hs, r, T, N), 32-byte
 * aligned. */
int moe_linattn_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                    const float* log_decay, const int32_t* cu_seqlens, const float* state_in,
                    int N, int T, int max_seqlen, int Hs, int r, int Dk, int Dv, int ldq, int ldk,
                    int ldv, int ldo, float scale, uint16_t* o, float* state_out, void* ws,
                    size_t ws_bytes, int32_t* err_flag, void* stream);

/* Backward of moe_linattn_fwd for dout = d loss / d o and d_state_out = d loss / d
 * state_out (nullable: zeros), from the forward's inputs alone. With X the
 * gradient that reaches a state from the later tokens (X = d_state_out after the
 * last token):
 *   R_t = X + scale * sum_a q_t^(a) (dout_t^(a))^T
 *   dq_t^(a) = scale * S_t dout_t^(a);  dk_t = R_t v_t;  dv_t = R_t^T k_t;  then X = lam R_t
 * dk and dv are the sums over the r query heads. d_state_in (nullable) is X before the
 * first token; it must not share memory with d_state_out or state_in. dq, dk, dv are bf16 with lddq,
 * lddk, lddv elements between tokens and share no memory with the inputs.
 * Precision is the forward's: dv is as precise as its o, dq and dk are with Dv in Dk's place (2.4e-3 for
 * Dv > 64), d_state_in is 3e-6 off.
 * Workspace: moe_workspace_size(MOE_OP_LINATTN_BWD, max_seqlen, Dk, Dv, Hs, r, T, N), 32-byte
 * aligned. */
int moe_linattn_bwd(const uint16_t* dout, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                    const float* log_decay, const int32_t* cu_seqlens, const float* state_in,
                    const float* d_state_out, int N, int T, int max_seqlen, int Hs, int r, int Dk,
                    int Dv, int lddo, int ldq, int ldk, int ldv, float scale, uint16_t* dq,
                    uint16_t* dk, uint16_t* dv, int lddq, int lddk, int lddv, float* d_state_in,
                    void* ws, size_t ws_bytes, int32_t* err_flag, void* stream);

/* One token for each of B rows: the recurrent form, for decoding. Row b updates
 * the state cache [n_slots][Hs][Dk][Dv] (fp32) in place at slot state_idx[b]
 * (int32 [B]; NULL: slot b) and writes o[b]. A negative slot is an empty row: its o is
 * zero and no state changes. A slot >= n_slots sets MOE_FLAG_BAD_INDEX and counts
 * as empty. The slots of one call must differ from one another. state is 32-byte
 * aligned; B * Hs < 2^28. */
int moe_linattn_step(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                     const float* log_decay, float* state, const int32_t* state_idx, int n_slots,
                     int B, int Hs, int r, int Dk, int Dv, int ldq, int ldk, int ldv, int ldo,
                     float scale, uint16_t* o, int32_t* err_flag, void* stream);

/* Causal depthwise convolution of W taps (2 to 4) along the tokens of packed sequences (as in moe_linattn_fwd, of any
 * length), with silu or without:
 *   p_t[c] = bias[c] + sum_j weight[c][j] x_{t - (W-1) + j}[c];  y = p or p sigmoid(p)
 * x, y bf16 [T][D], ld* elements between tokens; weight fp32 [D][W], bias fp32 [D] (nullable). state_in (bf16
 * [N][W-1][D], nullable: zeros) holds the W - 1 inputs before each sequence, the oldest first; state_out (nullable) receives the
 * last W - 1 of state_in and sequence. The two share no memory, and neither do x and y (which may be columns of one buffer). A sequence that ends before it starts or past T, or starts
 * before an earlier bound, sets MOE_FLAG_BAD_INDEX and is skipped. Rows that belong to no sequence keep what they hold. D and ld*
 * are multiples of 8. */
int moe_conv_fwd(const uint16_t* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                 const uint16_t* state_in, int N, int T, int D, int W, int ldx, int ldy, int silu, uint16_t* y,
                 uint16_t* state_out, int32_t* err_flag, void* stream);

/* Backward of moe_conv_fwd for dy and d_state_out (bf16 [N][W-1][D], nullable), from the forward's inputs: dx (bf16), dw
 * (fp32 [D][W], nullable), db (fp32 [D], nullable), d_state_in (bf16 [N][W-1][D], nullable; shares no memory with the states given, nor dx with x and dy). dw and db
 * are sums over all sequences that were not skipped. Deterministic. Workspace (for dw, db):
 * moe_workspace_size(MOE_OP_CONV_BWD, T, D, W, 0, 0, 0, N). */
int moe_conv_bwd(const uint16_t* dy, const uint16_t* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                 const uint16_t* state_in, const uint16_t* d_state_out, int N, int T, int D, int W, int lddy, int ldx,
                 int lddx, int silu, uint16_t* dx, float* dw, float* db, uint16_t* d_state_in, void* ws, size_t ws_bytes,
                 int32_t* err_flag, void* stream);

/* One token for each of B rows: y[b] from x[b] and the W - 1 inputs at slot state_idx[b] of the cache state (bf16
 * [n_slots][W-1][D]), which takes x[b] in. Slots as in moe_linattn_step: negative is an empty row (y = 0). y may be x. */
int moe_conv_step(const uint16_t* x, const float* weight, const float* bias, uint16_t* state, const int32_t* state_idx,
                  int n_slots, int B, int D, int W, int ldx, int ldy, int silu, uint16_t* y, int32_t* err_flag,
                  void* stream);

/* Selective state space scan over packed sequences (as in moe_linattn_fwd): channel c has `states` states with
 * decays of their own and a step that depends on the token,
 *   dt_t[c] = softplus(delta_t[c] + dt_bias[c])   (without softplus: the sum itself; dt_bias fp32 [D], nullable)
 *   h_t[c]  = exp(dt_t[c] A[c]) h_{t-1}[c] + dt_t[c] u_t[c] B_t[g]      (fp32, A fp32 [D][states])
 *   y_t[c]  = (C_t[g] . h_t[c] + skip[c] u_t[c]) silu(z_t[c])          (skip fp32 [D], z: nullable)
 * with B and C shared by the D / G channels of a group g. u, delta, z, y bf16 [T][D], B, C bf16 [T][G][states], ld*
 * elements between tokens. state_in, state_out fp32 [N][D][states] (nullable; state_out may be state_in). tile_states (nullable,
 * moe_workspace_size(MOE_OP_SCAN_TILE_STATES, 0, D, states, 0, 0, T, N) bytes) receives what moe_scan_bwd needs of this call. A
 * sequence longer than max_seqlen, or out of place as in moe_conv_fwd, sets MOE_FLAG_BAD_INDEX and is skipped.
 * A time step of -infinity, or of its type's lowest value, is 0 after softplus: that token leaves the state as it is.
 * Everything is fp32: states are within 1e-6 (rms) of their values, y has its own rounding to bf16. Time steps
 * and decays are taken as they come: exp(dt A) that passes fp32 makes infinities. D is a multiple of 8 and D / G of 4; states is 4, 8, 12 or 16; ld* of u, delta, z, y are
 * multiples of 8, of B and C of 4 (8-byte aligned). y shares no memory with what is read. Workspace:
 * moe_workspace_size(MOE_OP_SCAN_FWD, max_seqlen, D, states, G, 0, T, N). */
int moe_scan_fwd(const uint16_t* u, const uint16_t* delta, const float* A, const uint16_t* B, const uint16_t* C,
                 const float* skip, const uint16_t* z, const float* dt_bias, const int32_t* cu_seqlens,
                 const float* state_in, int N, int T, int max_seqlen, int D, int states, int G, int ldu, int lddelta,
                 int ldB, int ldC, int ldz, int ldy, int softplus, uint16_t* y, float* state_out, float* tile_states,
                 void* ws, size_t ws_bytes, int32_t* err_flag, void* stream);

/* Backward of moe_scan_fwd for dy (bf16 [T][D]) and d_state_out (fp32, nullable), from the forward's inputs and tile_states:
 * du, ddelta, dz (bf16 [T][D]; dz nullable, unused without z), dB, dC (bf16 [T][G][states], contiguous), dA (fp32
 * [D][states]), dskip, d_dt_bias (fp32 [D], nullable), d_state_in (fp32 [N][D][states], nullable; not over d_state_out). With X the gradient
 * that reaches a state from the later tokens and g_t = dy_t silu(z_t):
 *   R_t = X + g_t C_t;  q = R_t exp(dt A) h_{t-1};  dC_t = sum_c g_t h_t;  dB_t = sum_c dt u_t R_t
 *   du_t = dt (R_t . B_t) + skip g_t;  d dt_t = A . q + u_t (R_t . B_t);  dA += dt q;  then X = exp(dt A) R_t
 * du, ddelta and dz share no memory with what is read. Deterministic. Workspace: moe_workspace_size(MOE_OP_SCAN_BWD, max_seqlen, D, states, G, 0, T, N). */
int moe_scan_bwd(const uint16_t* dy, const uint16_t* u, const uint16_t* delta, const float* A, const uint16_t* B,
                 const uint16_t* C, const float* skip, const uint16_t* z, const float* dt_bias,
                 const int32_t* cu_seqlens, const float* tile_states, const float* d_state_out, int N, int T,
                 int max_seqlen, int D, int states, int G, int lddy, int ldu, int lddelta, int ldB, int ldC, int ldz,
                 int softplus, uint16_t* du, uint16_t* ddelta, uint16_t* dB, uint16_t* dC, uint16_t* dz, int lddu,
                 int ldddelta, int lddz, float* dA, float* dskip, float* d_dt_bias, float* d_state_in, void* ws,
                 size_t ws_bytes, int32_t* err_flag, void* stream);

/* One token for each of `rows` rows: updates the state cache (fp32 [n_slots][D][states]) in place at slot
 * state_idx[row] and writes y[row]. Slots as in moe_linattn_step. y may be u, delta or z. */
int moe_scan_step(const uint16_t* u, const uint16_t* delta, const float* A, const uint16_t* B, const uint16_t* C,
                  const float* skip, const uint16_t* z, const float* dt_bias, float* state, const int32_t* state_idx,
                  int n_slots, int rows, int D, int states, int G, int ldu, int lddelta, int ldB, int ldC, int ldz, int ldy,
                  int softplus, uint16_t* y, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------- optimizer */

/* One tensor of an AdamW step. p, g, m, v hold n values each (device). p and g are
 * fp32 or bf16 (MOE_DTYPE_*). With master (fp32 [n], nullable, p in bf16) the update
 * runs on master and p is its rounded copy; without it a bf16 p is rounded
 * stochastically. States in 32 bits: m and v fp32. In 8 bits: blocks of 256
 * consecutive values (the last one shorter); m holds E4M3 bytes of m / m_scale[block], v E4M3
 * bytes of sqrt(v) / v_scale[block], scales fp32 [ceil(n / 256)] = the block's largest
 * magnitude / 448, rounded stochastically. Zeroed states are a fresh start. */
typedef struct {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  long long n;
  float weight_decay;
  int p_dtype;
  int g_dtype;
} moe_adamw_tensor;

#define MOE_ADAMW_CTL_BYTES 64

/* Checks n_tensors tensors (host array, device pointers in it) and writes the
 * step's plan to `plan` (host memory, plan_bytes >= moe_workspace_size(MOE_OP_ADAMW_PLAN,
 * n_tensors, 0, ...)), which the caller copies to the device once; *chunks is the
 * amount of work that moe_adamw_step takes. Arrays aligned to 32 bytes (fp32), 16
 * (bf16) and 8 (codes) take whole vector accesses, others are walked by value. n may be 0. */
int moe_adamw_plan(const moe_adamw_tensor* tensors, int n_tensors, int state_bits, void* plan,
                   size_t plan_bytes, long long* chunks);

/* One AdamW step over every tensor of `plan` (device copy), t = steps taken + 1,
 * beta = 1 - rate (the rates are passed because 1 - beta in fp32 would lose digits):
 *   c = min(1, max_norm / (|g| + 1e-6)) over all tensors (1 when max_norm <= 0)
 *   m = beta1 m + (1 - beta1) c g;  v = beta2 v + (1 - beta2) (c g)^2
 *   p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * ctl (device, MOE_ADAMW_CTL_BYTES, zeroed before the first step) holds the number
 * of steps taken (int64 at byte 0), the last gradient norm (fp32 at byte 8) and the
 * clip factor (byte 12), so a captured step counts by itself; lr_dev (device fp32,
 * nullable) takes the place of lr. The norm is right to 2^-21 at any number of values (those
 * under 1e-19, whose squares are below fp32's normal numbers, may count for less). With
 * max_norm > 0 a norm that is not finite in fp32 leaves every tensor and the count as they are and
 * sets MOE_FLAG_NONFINITE; with max_norm <= 0 no norm is computed and such values pass into the tensors. Where v itself passes
 * fp32 (|c g| above 1.8e19 / sqrt(1 - beta2)), 32-bit states hold infinity, after which the weight only decays;
 * with 8-bit states that value's weight and states become NaN. Stochastic
 * rounding depends on (seed, t, tensor, index) alone; results do not depend on
 * timing. Workspace: moe_workspace_size(MOE_OP_ADAMW_STEP, 0, ...). */
int moe_adamw_step(const void* plan, int n_tensors, long long chunks, int state_bits, float lr,
                   const float* lr_dev, float rate1, float rate2, float eps, float max_norm,
                   int seed, void* ctl, void* ws, size_t ws_bytes, int32_t* err_flag,
                   void* stream);

/* ---------------------------------------------------------------- diagnostics */

/* Per-kernel timing. While enabled, every kernel launch of the library is
 * bracketed by two CUDA events recorded on the launch's own stream (event
 * objects are created on first use and reused). moe_timing_report, called
 * after the caller synchronised those streams, writes one line per kernel
 * label, "label launches total_ms", into buf (NUL-terminated, truncated to
 * len), forgets the recorded pairs and returns the length of the full text.
 * With buf == NULL it only returns that length and keeps the pairs. */
int moe_timing_enable(int on);
int moe_timing_report(char* buf, size_t len);

/* Check of the bounded waits. Every wait of a library kernel on an mbarrier
 * (a copy landing, an accumulator filling or draining) gives up after a time
 * limit, ORs MOE_FLAG_TIMEOUT into the caller's error word and lets the kernel
 * return, so a wait that can never end does not hang the GPU. This call runs
 * that same wait, with the limit `limit_ns` (1e3 .. 1e9 ns), in one thread of
 * a one-warp kernel, on an mbarrier that nothing arrives at: it always times
 * out, sets MOE_FLAG_TIMEOUT in *err_flag (device int32) and writes the
 * nanoseconds it waited to *waited_ns (device int64). It uses no TMA copy, no
 * tensor map and no tensor memory. The pages describe nothing like it. */
int moe_diag_wait_timeout(long long limit_ns, int32_t* err_flag, long long* waited_ns,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
