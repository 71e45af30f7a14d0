// C-ABI entry points of the sequence mixer and the optimizer step: host-side
// argument checks and the launch sequence of each (moe.h has the contracts).
#include <cmath>
#include <cstring>

#include "linattn.h"
#include "optim.h"

namespace moe {
void record_cuda_error(cudaError_t e);
}

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

// Head counts and widths of the mixer's calls.
int check_heads(int Hs, int r, int Dk, int Dv) {
  MOE_REQUIRE(Hs > 0 && Hs <= 65536 && r > 0 && r <= 1024 && Dk > 0 && Dv > 0, MOE_ERR_ARG);
  MOE_REQUIRE(Dk <= 128 && Dv <= 128, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(Dk % 8 == 0 && Dv % 8 == 0, MOE_ERR_ALIGN);
  return MOE_OK;
}

// A [tokens][heads][width] bf16 tensor with ld elements between tokens.
int check_rows(const void* p, long long heads, int width, int ld) {
  MOE_REQUIRE(p != nullptr && ld >= heads * width, MOE_ERR_ARG);
  MOE_REQUIRE(ld % 8 == 0 && aligned(p, 16), MOE_ERR_ALIGN);
  return MOE_OK;
}

// Whether two fp32 arrays of n values share memory.
bool overlap(const float* a, const float* b, long long n) {
  if (a == nullptr || b == nullptr) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return (x > y ? x - y : y - x) < static_cast<uintptr_t>(n) * 4;
}

int check_sequences(const int32_t* cu_seqlens, int N, int T, int max_seqlen) {
  MOE_REQUIRE(N >= 0 && T >= 0 && max_seqlen >= 0, MOE_ERR_ARG);
  if (N > 0 && cu_seqlens == nullptr)
    MOE_REQUIRE(T % N == 0 && max_seqlen >= T / N, MOE_ERR_ARG);
  return MOE_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- sequence mixer

int moe_linattn_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                    const float* log_decay, const int32_t* cu_seqlens, const float* state_in,
                    int N, int T, int max_seqlen, int Hs, int r, int Dk, int Dv, int ldq, int ldk,
                    int ldv, int ldo, float scale, uint16_t* o, float* state_out, void* ws,
                    size_t ws_bytes, int32_t* err_flag, void* stream) {
  MOE_REQUIRE(log_decay != nullptr, MOE_ERR_ARG);
  MOE_CHECK(check_heads(Hs, r, Dk, Dv));
  MOE_CHECK(check_sequences(cu_seqlens, N, T, max_seqlen));
  const long long Hq = static_cast<long long>(Hs) * r;
  MOE_CHECK(check_rows(q, Hq, Dk, ldq));
  MOE_CHECK(check_rows(k, Hs, Dk, ldk));
  MOE_CHECK(check_rows(v, Hs, Dv, ldv));
  MOE_CHECK(check_rows(o, Hq, Dv, ldo));
  MOE_REQUIRE(aligned(state_in, 32) && aligned(state_out, 32), MOE_ERR_ALIGN);
  // in place, or apart: a sequence's last state may not fall on another's first
  MOE_REQUIRE(state_out == state_in || !overlap(state_out, state_in, static_cast<long long>(N) * Hs * Dk * Dv),
              MOE_ERR_ARG);
  if (N == 0) return MOE_OK;
  const size_t need = moe_workspace_size(MOE_OP_LINATTN_FWD, max_seqlen, Dk, Dv, Hs, r, T, N);
  MOE_REQUIRE(need == 0 || (ws != nullptr && ws_bytes >= need), MOE_ERR_WORKSPACE);
  MOE_REQUIRE(need == 0 || aligned(ws, 32), MOE_ERR_ALIGN);  // (states: 32-byte accesses)
  const LinShape s{cu_seqlens, log_decay, N, T, max_seqlen, Hs, err_flag};
  const LinProblem p{q, k, v, ldq, ldk, ldv, ldo, o, r, 1, Dk, Dv, 0, 1.0f, scale, state_in, state_out, Dv, 1, -1};
  return linattn_run(&p, 1, s, ws, S(stream));
}

int moe_linattn_bwd(const uint16_t* dout, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                    const float* log_decay, const int32_t* cu_seqlens, const float* state_in,
                    const float* d_state_out, int N, int T, int max_seqlen, int Hs, int r, int Dk,
                    int Dv, int lddo, int ldq, int ldk, int ldv, float scale, uint16_t* dq,
                    uint16_t* dk, uint16_t* dv, int lddq, int lddk, int lddv, float* d_state_in,
                    void* ws, size_t ws_bytes, int32_t* err_flag, void* stream) {
  MOE_REQUIRE(log_decay != nullptr, MOE_ERR_ARG);
  MOE_CHECK(check_heads(Hs, r, Dk, Dv));
  MOE_CHECK(check_sequences(cu_seqlens, N, T, max_seqlen));
  const long long Hq = static_cast<long long>(Hs) * r;
  MOE_CHECK(check_rows(dout, Hq, Dv, lddo));
  MOE_CHECK(check_rows(q, Hq, Dk, ldq));
  MOE_CHECK(check_rows(k, Hs, Dk, ldk));
  MOE_CHECK(check_rows(v, Hs, Dv, ldv));
  MOE_CHECK(check_rows(dq, Hq, Dk, lddq));
  MOE_CHECK(check_rows(dk, Hs, Dk, lddk));
  MOE_CHECK(check_rows(dv, Hs, Dv, lddv));
  // dk's recurrence reads d_state_out, and dq's state_in, while dv's writes d_state_in
  const long long states = static_cast<long long>(N) * Hs * Dk * Dv;
  MOE_REQUIRE(d_state_in == nullptr || d_state_in != d_state_out, MOE_ERR_ARG);
  MOE_REQUIRE(!overlap(d_state_in, d_state_out, states) && !overlap(d_state_in, state_in, states), MOE_ERR_ARG);
  MOE_REQUIRE(aligned(state_in, 32) && aligned(d_state_out, 32) && aligned(d_state_in, 32),
              MOE_ERR_ALIGN);
  if (N == 0) return MOE_OK;
  const size_t need = moe_workspace_size(MOE_OP_LINATTN_BWD, max_seqlen, Dk, Dv, Hs, r, T, N);
  MOE_REQUIRE(need == 0 || (ws != nullptr && ws_bytes >= need), MOE_ERR_WORKSPACE);
  MOE_REQUIRE(need == 0 || aligned(ws, 32), MOE_ERR_ALIGN);  // (states: 32-byte accesses)
  const LinShape s{cu_seqlens, log_decay, N, T, max_seqlen, Hs, err_flag};
  // dq_t = scale S_t dout_t: the forward's recurrence with k and v exchanged
  const LinProblem pq{dout, v, k, lddo, ldv, ldk, lddq, dq, r, 1, Dv, Dk, 0, 1.0f, scale, state_in, nullptr, 1, Dv, -1};
  // dv_t = R_t^T k_t and dk_t = R_t v_t: from the last token to the first
  const LinProblem pv{k, q, dout, ldk, ldq, lddo, lddv, dv, 1, r, Dk, Dv, 1, scale, 1.0f, d_state_out, d_state_in, Dv, 1, -1};
  const LinProblem pk{v, dout, q, ldv, lddo, ldq, lddk, dk, 1, r, Dv, Dk, 1, scale, 1.0f, d_state_out, nullptr, 1, Dv, 1};
  const LinProblem p[3] = {pq, pv, pk};  // (dk's states are dv's transposed)
  return linattn_run(p, 3, s, ws, S(stream));
}

int moe_linattn_step(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                     const float* log_decay, float* state, const int32_t* state_idx, int n_slots,
                     int B, int Hs, int r, int Dk, int Dv, int ldq, int ldk, int ldv, int ldo,
                     float scale, uint16_t* o, int32_t* err_flag, void* stream) {
  MOE_REQUIRE(log_decay != nullptr && state != nullptr && B >= 0 && n_slots >= 0, MOE_ERR_ARG);
  MOE_REQUIRE(state_idx != nullptr || B <= n_slots, MOE_ERR_ARG);
  MOE_CHECK(check_heads(Hs, r, Dk, Dv));
  MOE_REQUIRE(static_cast<long long>(B) * Hs < (1ll << 28), MOE_ERR_ARG);
  const long long Hq = static_cast<long long>(Hs) * r;
  MOE_CHECK(check_rows(q, Hq, Dk, ldq));
  MOE_CHECK(check_rows(k, Hs, Dk, ldk));
  MOE_CHECK(check_rows(v, Hs, Dv, ldv));
  MOE_CHECK(check_rows(o, Hq, Dv, ldo));
  MOE_REQUIRE(aligned(state, 32), MOE_ERR_ALIGN);
  if (B == 0) return MOE_OK;
  return cuda_status(launch_linattn_step(q, k, v, log_decay, state, state_idx, n_slots, B, Hs, r,
                                         Dk, Dv, ldq, ldk, ldv, ldo, scale, o, err_flag, S(stream)));
}

// ---------------------------------------------------------------- optimizer

int moe_adamw_plan(const moe_adamw_tensor* tensors, int n_tensors, int state_bits, void* plan,
                   size_t plan_bytes, long long* chunks) {
  MOE_REQUIRE(tensors && plan && chunks && n_tensors > 0, MOE_ERR_ARG);
  MOE_REQUIRE(state_bits == 32 || state_bits == 8, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(plan_bytes >= moe_workspace_size(MOE_OP_ADAMW_PLAN, n_tensors, 0, 0, 0, 0, 0, 0),
              MOE_ERR_WORKSPACE);
  const auto width = [](int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; };
  long long at = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor& x = tensors[i];
    MOE_REQUIRE(x.n >= 0, MOE_ERR_ARG);
    MOE_REQUIRE(x.n == 0 || (x.p && x.g && x.m && x.v), MOE_ERR_ARG);
    MOE_REQUIRE(x.n == 0 || state_bits == 32 || (x.m_scale && x.v_scale), MOE_ERR_ARG);
    MOE_REQUIRE(x.p_dtype == MOE_DTYPE_F32 || x.p_dtype == MOE_DTYPE_BF16, MOE_ERR_ARG);
    MOE_REQUIRE(x.g_dtype == MOE_DTYPE_F32 || x.g_dtype == MOE_DTYPE_BF16, MOE_ERR_ARG);
    MOE_REQUIRE(!x.master || x.p_dtype == MOE_DTYPE_BF16, MOE_ERR_ARG);
    const int state_width = state_bits == 32 ? 4 : 1;
    MOE_REQUIRE(aligned(x.p, width(x.p_dtype)) && aligned(x.g, width(x.g_dtype)) &&
                    aligned(x.master, 4) && aligned(x.m, state_width) &&
                    aligned(x.v, state_width) && aligned(x.m_scale, 4) && aligned(x.v_scale, 4),
                MOE_ERR_ALIGN);
    // eight values of a lane in one access
    const bool vec = aligned(x.p, 8 * width(x.p_dtype)) && aligned(x.g, 8 * width(x.g_dtype)) &&
                     aligned(x.master, 32) && aligned(x.m, 8 * state_width) &&
                     aligned(x.v, 8 * state_width);
    const AdamwEntry e{x.p, x.g, x.m, x.v, x.m_scale, x.v_scale, x.master, x.n, at,
                       x.weight_decay, x.p_dtype, x.g_dtype, vec ? 1 : 0};
    std::memcpy(static_cast<char*>(plan) + static_cast<size_t>(i) * sizeof(AdamwEntry), &e, sizeof e);
    at += (x.n + kAdamwChunk - 1) / kAdamwChunk;
  }
  *chunks = at;
  return MOE_OK;
}

int moe_adamw_step(const void* plan, int n_tensors, long long chunks, int state_bits, float lr,
                   const float* lr_dev, float rate1, float rate2, float eps, float max_norm,
                   int seed, void* ctl, void* ws, size_t ws_bytes, int32_t* err_flag,
                   void* stream) {
  static_assert(sizeof(AdamwControl) <= MOE_ADAMW_CTL_BYTES, "control block");
  MOE_REQUIRE(plan && ctl && n_tensors > 0 && chunks >= 0, MOE_ERR_ARG);
  MOE_REQUIRE(state_bits == 32 || state_bits == 8, MOE_ERR_UNSUPPORTED);
  MOE_REQUIRE(rate1 > 0.0f && rate1 <= 1.0f && rate2 > 0.0f && rate2 <= 1.0f && eps >= 0.0f &&
                  std::isfinite(lr) && !std::isnan(max_norm),
              MOE_ERR_ARG);
  MOE_REQUIRE(aligned(plan, 16) && aligned(ctl, 8) && aligned(ws, 16) && aligned(lr_dev, 4),
              MOE_ERR_ALIGN);
  const bool clipped = max_norm > 0.0f;
  MOE_REQUIRE(!clipped || (ws && ws_bytes >= moe_workspace_size(MOE_OP_ADAMW_STEP, 0, 0, 0, 0, 0, 0, 0)),
              MOE_ERR_WORKSPACE);
  if (chunks == 0) return MOE_OK;
  const AdamwEntry* const e = static_cast<const AdamwEntry*>(plan);
  AdamwControl* const c = static_cast<AdamwControl*>(ctl);
  if (clipped)
    MOE_CHECK(cuda_status(launch_grad_norm(e, n_tensors, chunks, max_norm, static_cast<double*>(ws), c, S(stream))));
  const AdamwHyper h{lr, static_cast<float>(1.0 - static_cast<double>(rate1)),
                     static_cast<float>(1.0 - static_cast<double>(rate2)), rate1, rate2, eps, std::log1p(-static_cast<double>(rate1)),
                     std::log1p(-static_cast<double>(rate2)), static_cast<uint32_t>(seed)};
  return cuda_status(launch_adamw_step(e, n_tensors, chunks, state_bits, h, lr_dev, c, clipped, err_flag, S(stream)));
}

}  // extern "C"
