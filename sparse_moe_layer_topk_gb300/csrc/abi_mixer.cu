// C-ABI entry points of the routing with scores and groups, the residual norm, the causal convolution and the selective
// scan: host-side argument checks and the launch sequence of each (moe.h has the contracts).
#include <cmath>

#include "common.cuh"
#include "gemm.h"
#include "mixer.h"
#include "scan.h"

namespace moe {
void record_cuda_error(cudaError_t e);
int router_latent_gemm(const uint16_t* x, const uint16_t* Wr, const uint16_t* W_dn, int T, int d, int E, int l,
                       float* logits, uint16_t* z, cudaStream_t st);
int router_grads(const uint16_t* dL, const uint16_t* x, const uint16_t* Wr, int T, int d, int E, uint16_t* dx_accum,
                 void* dWr, int wgrad_dtype, const uint16_t* dz, const uint16_t* W_dn, int l, cudaStream_t st);
}  // namespace moe

using namespace moe;

namespace {

inline cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool aligned(const void* p, uintptr_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; }

inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  record_cuda_error(e);
  return MOE_ERR_CUDA;
}

#define MOE_CHECK(expr)            \
  do {                             \
    const int _st = (expr);        \
    if (_st != MOE_OK) return _st; \
  } while (0)

#define MOE_REQUIRE(cond, code) \
  do {                          \
    if (!(cond)) return (code); \
  } while (0)

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  if (a == nullptr || b == nullptr) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// Whether two [T][width] arrays with ld elements between rows share memory (rows of equal distance may lie between one another).
struct Rows {
  const void* p;
  long long width, ld;
  int size = 2;  // bytes of a value
};
bool meet(const Rows& a, const Rows& b, int T) {
  if (a.p == nullptr || b.p == nullptr || T <= 0) return false;
  const auto bytes = [&](const Rows& r) { return static_cast<size_t>((T - 1) * r.ld + r.width) * r.size; };
  if (!overlap(a.p, bytes(a), b.p, bytes(b))) return false;
  const long long step = a.ld * a.size;
  if (T == 1 || step != b.ld * b.size) return true;
  const long long apart = static_cast<long long>(reinterpret_cast<uintptr_t>(a.p) - reinterpret_cast<uintptr_t>(b.p));
  const long long at = (apart % step + step) % step;  // where a's rows begin in b's
  return at < b.width * b.size || at + a.width * a.size > step;
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.ld == b.ld && a.width == b.width && a.size == b.size; }

// A [tokens][width] bf16 operand with ld elements between tokens, read `bytes` at a time.
int check_rows(const void* p, long long width, int ld, int bytes = 16) {
  MOE_REQUIRE(p != nullptr && ld >= width, MOE_ERR_ARG);
  MOE_REQUIRE(ld % (bytes / 2) == 0 && aligned(p, bytes), MOE_ERR_ALIGN);
  return MOE_OK;
}

int check_sequences(const int32_t* cu_seqlens, int N, int T, int max_seqlen) {
  MOE_REQUIRE(N >= 0 && T >= 0 && max_seqlen >= 0, MOE_ERR_ARG);
  if (N > 0 && cu_seqlens == nullptr) MOE_REQUIRE(T % N == 0 && max_seqlen >= T / N, MOE_ERR_ARG);
  return MOE_OK;
}

int check_route(int T, int E, int k, int score) {
  MOE_REQUIRE(T >= 0 && E > 0 && E <= 1024 && k >= 1 && k <= 32 && k <= E, MOE_ERR_ARG);
  MOE_REQUIRE(score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SOFTMAX, MOE_ERR_ARG);
  return MOE_OK;
}

int check_conv(int D, int W) {
  MOE_REQUIRE(D > 0 && D <= (1 << 20) && W > 0, MOE_ERR_ARG);
  MOE_REQUIRE(W >= 2 && W <= 4, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(D % 8 == 0, MOE_ERR_ALIGN);
  return MOE_OK;
}

int check_scan(int D, int S_, int G) {
  MOE_REQUIRE(D > 0 && D <= (1 << 20) && S_ > 0 && G > 0 && G <= D && D % G == 0, MOE_ERR_ARG);
  MOE_REQUIRE(S_ <= 16, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(D % 8 == 0 && D / G % 4 == 0 && S_ % 4 == 0, MOE_ERR_ALIGN);
  return MOE_OK;
}

// CTAs of a launch stay far below the grid's limit of 2^31 - 1.
bool grid_fits(long long parts, long long blocks) { return parts * blocks < (1ll << 31) - 1; }

}  // namespace

extern "C" {

// ---------------------------------------------------------------- routing

int moe_router_logits_latent(const uint16_t* x, const uint16_t* Wr, const uint16_t* W_dn, int T, int d, int E, int l,
                             float* logits, uint16_t* z, void* stream) {
  MOE_REQUIRE(x && Wr && W_dn && logits && z, MOE_ERR_ARG);
  MOE_REQUIRE(T >= 0 && d > 0 && l > 0 && E > 0 && E <= 1024, MOE_ERR_ARG);
  MOE_REQUIRE(d % 64 == 0 && E % 64 == 0 && l % 64 == 0, MOE_ERR_ALIGN);
  MOE_REQUIRE(aligned(x, 16) && aligned(Wr, 16) && aligned(W_dn, 16) && aligned(logits, 16) && aligned(z, 16), MOE_ERR_ALIGN);
  if (T == 0) return MOE_OK;
  return router_latent_gemm(x, Wr, W_dn, T, d, E, l, logits, z, S(stream));
}

int moe_route_scores(const float* logits, const float* bias, int T, int E, int k, int score, int groups, int group_k,
                     int group_top, int renorm, float scale, int32_t* topk_idx, float* topk_w, float* topk_s,
                     int32_t* err_flag, void* stream) {
  MOE_REQUIRE(logits && topk_idx && topk_w && topk_s, MOE_ERR_ARG);
  MOE_CHECK(check_route(T, E, k, score));
  MOE_REQUIRE(groups >= 1 && groups <= E && E % groups == 0 && group_k >= 1 && group_k <= groups, MOE_ERR_ARG);
  MOE_REQUIRE(group_top == 1 || group_top == 2, MOE_ERR_ARG);
  MOE_REQUIRE(groups <= 32, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(static_cast<long long>(group_k) * (E / groups) >= k, MOE_ERR_ARG);
  MOE_REQUIRE(std::isfinite(scale), MOE_ERR_ARG);
  MOE_REQUIRE(aligned(logits, 4) && aligned(bias, 4) && aligned(topk_idx, 4) && aligned(topk_w, 4) && aligned(topk_s, 4),
              MOE_ERR_ALIGN);
  if (T == 0) return MOE_OK;
  const RouteArgs a{logits, bias, T, E, k, score == MOE_SCORE_SOFTMAX, groups, group_k, group_top, renorm != 0, scale,
                    topk_idx, topk_w, topk_s, err_flag};
  return cuda_status(launch_route_scores(a, S(stream)));
}

int moe_route_scores_bwd(const float* d_w, const int32_t* slot_of, const float* logits, const int32_t* topk_idx,
                         const float* topk_w, const float* topk_s, int T, int E, int k, int score, int renorm, float scale,
                         void* d_logits, int dtype, float* d_topk_w, int32_t* err_flag, void* stream) {
  MOE_REQUIRE(d_w && topk_idx && topk_w && topk_s && d_logits, MOE_ERR_ARG);
  MOE_CHECK(check_route(T, E, k, score));
  MOE_REQUIRE(dtype == MOE_DTYPE_F32 || dtype == MOE_DTYPE_BF16, MOE_ERR_ARG);
  MOE_REQUIRE(std::isfinite(scale) && scale != 0.0f, MOE_ERR_ARG);
  const bool dense = score == MOE_SCORE_SOFTMAX && !renorm;
  MOE_REQUIRE(!dense || logits != nullptr, MOE_ERR_ARG);
  MOE_REQUIRE(aligned(d_logits, 16) && aligned(logits, dense && E % 4 == 0 ? 16 : 4), MOE_ERR_ALIGN);
  if (T == 0) return MOE_OK;
  const RouteBwdArgs a{d_w, slot_of, logits, topk_idx, topk_w, topk_s, T, E, k, score == MOE_SCORE_SOFTMAX, renorm != 0,
                       scale, d_logits, dtype == MOE_DTYPE_BF16, d_topk_w, err_flag};
  return cuda_status(launch_route_scores_bwd(a, S(stream)));
}

int moe_router_grads(const uint16_t* d_logits, const uint16_t* x, const uint16_t* Wr, int T, int d, int E,
                     uint16_t* dx_accum, void* dWr, int wgrad_dtype, const uint16_t* dz, const uint16_t* W_dn, int l,
                     void* stream) {
  MOE_REQUIRE(d_logits != nullptr, MOE_ERR_ARG);
  MOE_REQUIRE(T >= 0 && d > 0 && E > 0 && E <= 1024, MOE_ERR_ARG);
  MOE_REQUIRE(wgrad_dtype == MOE_DTYPE_F32 || wgrad_dtype == MOE_DTYPE_BF16, MOE_ERR_ARG);
  MOE_REQUIRE(d % 64 == 0 && E % 64 == 0 && aligned(d_logits, 16), MOE_ERR_ALIGN);
  MOE_REQUIRE(!(dx_accum && !Wr) && !(dWr && !x), MOE_ERR_ARG);
  MOE_REQUIRE(!dx_accum || (aligned(dx_accum, 16) && aligned(Wr, 16)), MOE_ERR_ALIGN);
  MOE_REQUIRE(!dWr || (aligned(dWr, 16) && aligned(x, 16)), MOE_ERR_ALIGN);
  if (dx_accum && dz) {
    MOE_REQUIRE(W_dn != nullptr && l > 0, MOE_ERR_ARG);
    MOE_REQUIRE(l % 64 == 0 && aligned(dz, 16) && aligned(W_dn, 16), MOE_ERR_ALIGN);
  }
  if (T == 0) {
    if (!dWr) return MOE_OK;
    return cuda_status(cudaMemsetAsync(dWr, 0, static_cast<size_t>(d) * E * (wgrad_dtype == MOE_DTYPE_F32 ? 4 : 2), S(stream)));
  }
  return router_grads(d_logits, x, Wr, T, d, E, dx_accum, dWr, wgrad_dtype, dz, W_dn, l, S(stream));
}

// ---------------------------------------------------------------- norm

int moe_rmsnorm_fwd(const uint16_t* x, const void* residual, const float* weight, int T, int d, int ldx, int res_dtype,
                    float eps, void* sum, void* y, int y_dtype, float* y_scale, int block, void* stream) {
  MOE_REQUIRE(weight && y, MOE_ERR_ARG);
  MOE_REQUIRE(T >= 0 && d > 0 && eps > 0.0f && std::isfinite(eps), MOE_ERR_ARG);
  MOE_REQUIRE(d <= 16384, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(d % 8 == 0, MOE_ERR_ALIGN);
  MOE_CHECK(check_rows(x, d, ldx));
  MOE_REQUIRE(res_dtype == MOE_DTYPE_F32 || res_dtype == MOE_DTYPE_BF16, MOE_ERR_ARG);
  MOE_REQUIRE((residual == nullptr) == (sum == nullptr), MOE_ERR_ARG);
  MOE_REQUIRE(y_dtype == MOE_DTYPE_BF16 || y_dtype == MOE_DTYPE_E4M3, MOE_ERR_ARG);
  const bool fp8 = y_dtype == MOE_DTYPE_E4M3;
  if (fp8) {
    MOE_REQUIRE(y_scale != nullptr, MOE_ERR_ARG);
    MOE_REQUIRE(block == 64 || block == 128 || block == d, MOE_ERR_UNSUPPORTED);
  }
  MOE_REQUIRE(aligned(residual, 16) && aligned(sum, 16) && aligned(weight, 16) && aligned(y, fp8 ? 8 : 16) &&
                  aligned(y_scale, 4),
              MOE_ERR_ALIGN);
  const size_t n = static_cast<size_t>(T) * d, x_bytes = T ? (static_cast<size_t>(T - 1) * ldx + d) * 2 : 0;
  const size_t r_bytes = n * (res_dtype == MOE_DTYPE_F32 ? 4 : 2), y_bytes = n * (fp8 ? 1 : 2);
  // the sum may take the residual's place; nothing else is read and written by one call
  MOE_REQUIRE(sum == residual || !overlap(sum, r_bytes, residual, r_bytes), MOE_ERR_ARG);
  MOE_REQUIRE(!overlap(sum, r_bytes, x, x_bytes) && !overlap(y, y_bytes, x, x_bytes) &&
                  !overlap(y, y_bytes, residual, r_bytes) && !overlap(y, y_bytes, sum, r_bytes),
              MOE_ERR_ARG);
  if (T == 0) return MOE_OK;
  const NormArgs a{x, residual, weight, T, d, ldx, eps, residual && res_dtype == MOE_DTYPE_F32, fp8, sum, y, y_scale,
                   block};
  return cuda_status(launch_rmsnorm_fwd(a, S(stream)));
}

int moe_rmsnorm_bwd(const uint16_t* dy, const void* u, const float* weight, const void* d_sum, int T, int d,
                    int ldu, int res_dtype, float eps, uint16_t* dx, void* d_residual, float* dw, void* ws, size_t ws_bytes,
                    void* stream) {
  MOE_REQUIRE(dy && u && weight, MOE_ERR_ARG);
  MOE_REQUIRE(T >= 0 && d > 0 && ldu >= d && eps > 0.0f && std::isfinite(eps), MOE_ERR_ARG);
  MOE_REQUIRE(d <= 16384, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(res_dtype == MOE_DTYPE_F32 || res_dtype == MOE_DTYPE_BF16, MOE_ERR_ARG);
  MOE_REQUIRE(d % 8 == 0 && ldu % 8 == 0, MOE_ERR_ALIGN);
  MOE_REQUIRE(aligned(dy, 16) && aligned(u, 16) && aligned(weight, 16) && aligned(d_sum, 16) &&
                  aligned(dx, 16) && aligned(d_residual, 16) && aligned(dw, 4) && aligned(ws, 16),
              MOE_ERR_ALIGN);
  MOE_REQUIRE(!dw || (ws && ws_bytes >= moe_workspace_size(MOE_OP_RMSNORM_BWD, T, d, 0, 0, 0, 0, 0)), MOE_ERR_WORKSPACE);
  if (T == 0) return dw ? cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(d) * 4, S(stream))) : MOE_OK;
  const int res = res_dtype == MOE_DTYPE_F32 ? 4 : 2;
  for (const Rows& out : {Rows{dx, d, d, 2}, Rows{d_residual, d, d, res}})  // (a row's own input may be written over)
    for (const Rows& in : {Rows{dy, d, d, 2}, Rows{u, d, ldu, res}, Rows{d_sum, d, d, res}})
      MOE_REQUIRE(same(out, in) || !meet(out, in, T), MOE_ERR_ARG);
  const NormBwdArgs a{dy, u, weight, d_sum, T, d, ldu, eps, res_dtype == MOE_DTYPE_F32, dx, d_residual, dw,
                      static_cast<float*>(ws)};
  return cuda_status(launch_rmsnorm_bwd(a, S(stream)));
}

// ---------------------------------------------------------------- convolution

int moe_conv_fwd(const uint16_t* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                 const uint16_t* state_in, int N, int T, int D, int W, int ldx, int ldy, int silu, uint16_t* y,
                 uint16_t* state_out, int32_t* err_flag, void* stream) {
  MOE_REQUIRE(weight != nullptr, MOE_ERR_ARG);
  MOE_CHECK(check_conv(D, W));
  MOE_CHECK(check_sequences(cu_seqlens, N, T, T));
  MOE_CHECK(check_rows(x, D, ldx));
  MOE_CHECK(check_rows(y, D, ldy));
  MOE_REQUIRE(aligned(weight, 16) && aligned(bias, 4) && aligned(state_in, 16) && aligned(state_out, 16), MOE_ERR_ALIGN);
  // (a sequence's last state may be written before another CTA has read its first)
  const size_t state = static_cast<size_t>(N) * (W - 1) * D * 2;
  MOE_REQUIRE(!overlap(state_in, state, state_out, state), MOE_ERR_ARG);
  MOE_REQUIRE(grid_fits(T / 32 + static_cast<long long>(N), D / 512 + 1), MOE_ERR_ARG);
  if (N == 0) return MOE_OK;
  MOE_REQUIRE(!meet({y, D, ldy}, {x, D, ldx}, T), MOE_ERR_ARG);  // (tokens are read by their neighbours)
  const ConvArgs a{x, weight, bias, cu_seqlens, state_in, N, T, D, W, ldx, ldy, silu != 0, y, state_out, err_flag};
  return cuda_status(launch_conv_fwd(a, S(stream)));
}

int moe_conv_bwd(const uint16_t* dy, const uint16_t* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                 const uint16_t* state_in, const uint16_t* d_state_out, int N, int T, int D, int W, int lddy, int ldx,
                 int lddx, int silu, uint16_t* dx, float* dw, float* db, uint16_t* d_state_in, void* ws, size_t ws_bytes,
                 int32_t* err_flag, void* stream) {
  MOE_REQUIRE(weight != nullptr, MOE_ERR_ARG);
  MOE_CHECK(check_conv(D, W));
  MOE_CHECK(check_sequences(cu_seqlens, N, T, T));
  MOE_CHECK(check_rows(dy, D, lddy));
  MOE_CHECK(check_rows(x, D, ldx));
  MOE_CHECK(check_rows(dx, D, lddx));
  MOE_REQUIRE(aligned(weight, 16) && aligned(bias, 4) && aligned(state_in, 16) && aligned(d_state_out, 16) &&
                  aligned(d_state_in, 16) && aligned(dw, 4) && aligned(db, 4) && aligned(ws, 16),
              MOE_ERR_ALIGN);
  const size_t state = static_cast<size_t>(N) * (W - 1) * D * 2;
  MOE_REQUIRE(!overlap(d_state_in, state, state_in, state) && !overlap(d_state_in, state, d_state_out, state), MOE_ERR_ARG);
  MOE_REQUIRE(grid_fits(T / 64 + static_cast<long long>(N), D / 512 + 1), MOE_ERR_ARG);
  const bool sums = dw || db;
  MOE_REQUIRE(!sums || N == 0 || (ws && ws_bytes >= moe_workspace_size(MOE_OP_CONV_BWD, T, D, W, 0, 0, 0, N)), MOE_ERR_WORKSPACE);
  if (N == 0) {
    if (dw) MOE_CHECK(cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(D) * W * 4, S(stream))));
    if (db) MOE_CHECK(cuda_status(cudaMemsetAsync(db, 0, static_cast<size_t>(D) * 4, S(stream))));
    return MOE_OK;
  }
  MOE_REQUIRE(!meet({dx, D, lddx}, {x, D, ldx}, T) && !meet({dx, D, lddx}, {dy, D, lddy}, T), MOE_ERR_ARG);
  const ConvBwdArgs a{dy, x, weight, bias, cu_seqlens, state_in, d_state_out, N, T, D, W, lddy, ldx, lddx, silu != 0, dx,
                      sums ? static_cast<float*>(ws) : nullptr, d_state_in, err_flag};
  return cuda_status(launch_conv_bwd(a, dw, db, S(stream)));
}

int moe_conv_step(const uint16_t* x, const float* weight, const float* bias, uint16_t* state, const int32_t* state_idx,
                  int n_slots, int B, int D, int W, int ldx, int ldy, int silu, uint16_t* y, int32_t* err_flag,
                  void* stream) {
  MOE_REQUIRE(weight && state && B >= 0 && n_slots >= 0, MOE_ERR_ARG);
  MOE_REQUIRE(state_idx != nullptr || B <= n_slots, MOE_ERR_ARG);
  MOE_CHECK(check_conv(D, W));
  MOE_CHECK(check_rows(x, D, ldx));
  MOE_CHECK(check_rows(y, D, ldy));
  MOE_REQUIRE(aligned(weight, 16) && aligned(bias, 4) && aligned(state, 16), MOE_ERR_ALIGN);
  MOE_REQUIRE(grid_fits(B, D / 512 + 1), MOE_ERR_ARG);
  if (B == 0) return MOE_OK;
  const Rows from{x, D, ldx}, to{y, D, ldy};
  MOE_REQUIRE(same(from, to) || !meet(from, to, B), MOE_ERR_ARG);
  const ConvStepArgs a{x, weight, bias, state, state_idx, n_slots, B, D, W, ldx, ldy, silu != 0, y, err_flag};
  return cuda_status(launch_conv_step(a, S(stream)));
}

// ---------------------------------------------------------------- selective scan

int moe_scan_fwd(const uint16_t* u, const uint16_t* delta, const float* A, const uint16_t* B, const uint16_t* C,
                 const float* skip, const uint16_t* z, const float* dt_bias, const int32_t* cu_seqlens,
                 const float* state_in, int N, int T, int max_seqlen, int D, int states, int G, int ldu, int lddelta,
                 int ldB, int ldC, int ldz, int ldy, int softplus, uint16_t* y, float* state_out, float* tile_states,
                 void* ws, size_t ws_bytes, int32_t* err_flag, void* stream) {
  MOE_REQUIRE(A != nullptr, MOE_ERR_ARG);
  MOE_CHECK(check_scan(D, states, G));
  MOE_CHECK(check_sequences(cu_seqlens, N, T, max_seqlen));
  MOE_CHECK(check_rows(u, D, ldu));
  MOE_CHECK(check_rows(delta, D, lddelta));
  MOE_CHECK(check_rows(B, static_cast<long long>(G) * states, ldB, 8));
  MOE_CHECK(check_rows(C, static_cast<long long>(G) * states, ldC, 8));
  if (z) MOE_CHECK(check_rows(z, D, ldz));
  MOE_CHECK(check_rows(y, D, ldy));
  MOE_REQUIRE(aligned(A, 16) && aligned(skip, 4) && aligned(dt_bias, 4) && aligned(state_in, 16) && aligned(state_out, 16) &&
                  aligned(tile_states, 16) && aligned(ws, 16),
              MOE_ERR_ALIGN);
  const size_t state = static_cast<size_t>(N) * D * states * 4;
  MOE_REQUIRE(state_in == state_out || !overlap(state_in, state, state_out, state), MOE_ERR_ARG);
  MOE_REQUIRE(grid_fits(T / 32 + static_cast<long long>(N), static_cast<long long>(D) * states / 512 + G), MOE_ERR_ARG);
  if (N == 0) return MOE_OK;
  const size_t need = moe_workspace_size(MOE_OP_SCAN_FWD, max_seqlen, D, states, G, 0, T, N);
  MOE_REQUIRE(need == 0 || (ws && ws_bytes >= need), MOE_ERR_WORKSPACE);
  const long long per_token = static_cast<long long>(G) * states;
  for (const Rows& in : {Rows{u, D, ldu}, Rows{delta, D, lddelta}, Rows{z, D, ldz}, Rows{B, per_token, ldB}, Rows{C, per_token, ldC}})
    MOE_REQUIRE(!meet({y, D, ldy}, in, T), MOE_ERR_ARG);
  const ScanArgs a{u, delta, A, B, C, skip, z, dt_bias, cu_seqlens, state_in, N, T, max_seqlen, D, states, G, ldu, lddelta,
                   ldB, ldC, ldz, ldy, softplus != 0, y, state_out, tile_states, static_cast<float*>(ws), err_flag};
  return cuda_status(launch_scan_fwd(a, S(stream)));
}

int moe_scan_bwd(const uint16_t* dy, const uint16_t* u, const uint16_t* delta, const float* A, const uint16_t* B,
                 const uint16_t* C, const float* skip, const uint16_t* z, const float* dt_bias,
                 const int32_t* cu_seqlens, const float* tile_states, const float* d_state_out, int N, int T,
                 int max_seqlen, int D, int states, int G, int lddy, int ldu, int lddelta, int ldB, int ldC, int ldz,
                 int softplus, uint16_t* du, uint16_t* ddelta, uint16_t* dB, uint16_t* dC, uint16_t* dz, int lddu,
                 int ldddelta, int lddz, float* dA, float* dskip, float* d_dt_bias, float* d_state_in, void* ws,
                 size_t ws_bytes, int32_t* err_flag, void* stream) {
  MOE_REQUIRE(A && tile_states && dB && dC && dA, MOE_ERR_ARG);
  MOE_CHECK(check_scan(D, states, G));
  MOE_CHECK(check_sequences(cu_seqlens, N, T, max_seqlen));
  MOE_CHECK(check_rows(dy, D, lddy));
  MOE_CHECK(check_rows(u, D, ldu));
  MOE_CHECK(check_rows(delta, D, lddelta));
  MOE_CHECK(check_rows(B, static_cast<long long>(G) * states, ldB, 8));
  MOE_CHECK(check_rows(C, static_cast<long long>(G) * states, ldC, 8));
  MOE_CHECK(check_rows(du, D, lddu));
  MOE_CHECK(check_rows(ddelta, D, ldddelta));
  if (z) MOE_CHECK(check_rows(z, D, ldz));
  if (z && dz) MOE_CHECK(check_rows(dz, D, lddz));
  MOE_REQUIRE(aligned(A, 16) && aligned(skip, 4) && aligned(dt_bias, 4) && aligned(tile_states, 16) && aligned(d_state_out, 16) &&
                  aligned(d_state_in, 16) && aligned(dB, 8) && aligned(dC, 8) && aligned(dA, 4) && aligned(dskip, 4) &&
                  aligned(d_dt_bias, 4) && aligned(ws, 16),
              MOE_ERR_ALIGN);
  const size_t state = static_cast<size_t>(N) * D * states * 4;
  MOE_REQUIRE(!overlap(d_state_in, state, d_state_out, state), MOE_ERR_ARG);
  MOE_REQUIRE(grid_fits(T / 32 + static_cast<long long>(N), static_cast<long long>(D) * states / 512 + G), MOE_ERR_ARG);
  if (N == 0) {
    MOE_CHECK(cuda_status(cudaMemsetAsync(dA, 0, static_cast<size_t>(D) * states * 4, S(stream))));
    if (dskip) MOE_CHECK(cuda_status(cudaMemsetAsync(dskip, 0, static_cast<size_t>(D) * 4, S(stream))));
    if (d_dt_bias) MOE_CHECK(cuda_status(cudaMemsetAsync(d_dt_bias, 0, static_cast<size_t>(D) * 4, S(stream))));
    return MOE_OK;
  }
  const size_t need = moe_workspace_size(MOE_OP_SCAN_BWD, max_seqlen, D, states, G, 0, T, N);
  MOE_REQUIRE(ws && ws_bytes >= need, MOE_ERR_WORKSPACE);
  const long long per_token = static_cast<long long>(G) * states;
  for (const Rows& in : {Rows{dy, D, lddy}, Rows{u, D, ldu}, Rows{delta, D, lddelta}, Rows{z, D, ldz}, Rows{B, per_token, ldB}, Rows{C, per_token, ldC}})
    for (const Rows& out : {Rows{du, D, lddu}, Rows{ddelta, D, ldddelta}, Rows{z ? dz : nullptr, D, lddz}})
      MOE_REQUIRE(!meet(out, in, T), MOE_ERR_ARG);
  ScanBwdArgs a{};
  a.f = ScanArgs{u, delta, A, B, C, skip, z, dt_bias, cu_seqlens, nullptr, N, T, max_seqlen, D, states, G, ldu, lddelta, ldB,
                 ldC, ldz, 0, softplus != 0, nullptr, nullptr, const_cast<float*>(tile_states), static_cast<float*>(ws), err_flag};
  a.dy = dy, a.d_state_out = d_state_out, a.lddy = lddy;
  a.du = du, a.dd = ddelta, a.dB = dB, a.dC = dC, a.dz = dz;
  a.lddu = lddu, a.lddd = ldddelta, a.lddz = lddz;
  a.dA = dA, a.dskip = dskip, a.d_dt_bias = d_dt_bias, a.d_state_in = d_state_in;
  return cuda_status(launch_scan_bwd(a, S(stream)));
}

int moe_scan_step(const uint16_t* u, const uint16_t* delta, const float* A, const uint16_t* B, const uint16_t* C,
                  const float* skip, const uint16_t* z, const float* dt_bias, float* state, const int32_t* state_idx,
                  int n_slots, int rows, int D, int states, int G, int ldu, int lddelta, int ldB, int ldC, int ldz, int ldy,
                  int softplus, uint16_t* y, int32_t* err_flag, void* stream) {
  MOE_REQUIRE(A && state && rows >= 0 && n_slots >= 0, MOE_ERR_ARG);
  MOE_REQUIRE(state_idx != nullptr || rows <= n_slots, MOE_ERR_ARG);
  MOE_CHECK(check_scan(D, states, G));
  MOE_CHECK(check_rows(u, D, ldu));
  MOE_CHECK(check_rows(delta, D, lddelta));
  MOE_CHECK(check_rows(B, static_cast<long long>(G) * states, ldB, 8));
  MOE_CHECK(check_rows(C, static_cast<long long>(G) * states, ldC, 8));
  if (z) MOE_CHECK(check_rows(z, D, ldz));
  MOE_CHECK(check_rows(y, D, ldy));
  MOE_REQUIRE(aligned(A, 16) && aligned(skip, 4) && aligned(dt_bias, 4) && aligned(state, 16), MOE_ERR_ALIGN);
  MOE_REQUIRE(grid_fits(rows / 4 + 1ll, G), MOE_ERR_ARG);
  if (rows == 0) return MOE_OK;
  const Rows to{y, D, ldy};
  for (const Rows& in : {Rows{u, D, ldu}, Rows{delta, D, lddelta}, Rows{z, D, ldz}})  // (read by the lane that writes there)
    MOE_REQUIRE(same(to, in) || !meet(to, in, rows), MOE_ERR_ARG);
  const long long per_token = static_cast<long long>(G) * states;
  MOE_REQUIRE(!meet(to, {B, per_token, ldB}, rows) && !meet(to, {C, per_token, ldC}, rows), MOE_ERR_ARG);
  const ScanStepArgs a{u, delta, A, B, C, skip, z, dt_bias, state, state_idx, n_slots, rows, D, states, G, ldu, lddelta, ldB,
                       ldC, ldz, ldy, softplus != 0, y, err_flag};
  return cuda_status(launch_scan_step(a, S(stream)));
}

}  // extern "C"
