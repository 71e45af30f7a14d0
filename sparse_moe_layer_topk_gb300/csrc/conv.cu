// Causal depthwise convolution of 2 to 4 taps over packed sequences, its backward, and its step.
//
//   p_t = bias + sum_j w[j] x_{t - (W-1) + j};  y_t = p_t or silu(p_t)
//
// A thread owns four channels (8-byte accesses, a warp's 256 bytes of a row) and walks tokens with the last W inputs
// in registers, so every input is read once but for the W - 1 rows before a part. All three kernels are bound by HBM.
#include "common.cuh"
#include "mixer.h"
#include "seq.cuh"
#include "timing.h"

namespace moe {

int num_sms();

namespace {

constexpr int kThreads = 128;       // 512 channels
constexpr int kFwdTokens = 32;      // tokens of a part
constexpr int kBwdTokens = 64;
constexpr int kStep = 8;            // tokens whose loads are under way together

struct F4 {
  float v[4];
};

__device__ __forceinline__ F4 load4(const bf16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return F4{{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)}};
}
__device__ __forceinline__ void store4(bf16* p, const F4& x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[2], x.v[3]));
}
__device__ __forceinline__ F4 zero4() { return F4{{0.0f, 0.0f, 0.0f, 0.0f}}; }

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// The weights of four channels, tap by tap, from [D][W].
template <int W>
__device__ __forceinline__ void load_taps(const float* w, int c, F4 (&tap)[W]) {
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) tap[j].v[i] = __ldg(w + static_cast<long long>(c + i) * W + j);
}

// Input `at` (from -(W-1)) of a sequence: its tokens, and before them its state.
template <int W>
__device__ __forceinline__ F4 input_at(const bf16* x, long long ldx, const bf16* state, int D, const SeqPart& s, int at, int c) {
  if (at >= 0) return load4(x + (s.start + at) * ldx + c);
  if (state == nullptr) return zero4();
  return load4(state + (static_cast<long long>(s.n) * (W - 1) + (W - 1) + at) * D + c);
}

template <int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a, int blocks) {
  const int block = blockIdx.x % blocks;  // of channels
  SeqPart s;
  if (!find_part(a.cu, a.N, a.T, a.T, kFwdTokens, blockIdx.x / blocks, s, block == 0 && threadIdx.x < 32 ? a.err_flag : nullptr)) return;
  const int c = 4 * (block * kThreads + threadIdx.x);
  if (c >= a.D) return;
  const bf16* const x = static_cast<const bf16*>(a.x);
  const bf16* const state = static_cast<const bf16*>(a.state_in);
  bf16* const y = static_cast<bf16*>(a.y);
  const int t0 = s.part * kFwdTokens, t1 = min(s.len, t0 + kFwdTokens);
  F4 tap[W], win[W];  // win[W - 1]: the newest input
  load_taps<W>(a.weight, c, tap);
  F4 bias = zero4();
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i) bias.v[i] = __ldg(a.bias + c + i);
  }
#pragma unroll
  for (int j = 1; j < W; ++j) win[j] = input_at<W>(x, a.ldx, state, a.D, s, t0 - W + j, c);
  for (int t = t0; t < t1; t += kStep) {
    F4 in[kStep];
#pragma unroll
    for (int q = 0; q < kStep; ++q)
      if (t + q < t1) in[q] = load4(x + static_cast<long long>(s.start + t + q) * a.ldx + c);
#pragma unroll
    for (int q = 0; q < kStep; ++q) {
      if (t + q >= t1) break;
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) win[j] = win[j + 1];
      win[W - 1] = in[q];
      F4 p = bias;
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) p.v[i] = fmaf(tap[j].v[i], win[j].v[i], p.v[i]);
      if (SILU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p.v[i] *= sigmoid(p.v[i]);
      }
      store4(y + static_cast<long long>(s.start + t + q) * a.ldy + c, p);
    }
  }
  if (a.state_out && t1 == s.len) {
    bf16* const out = static_cast<bf16*>(a.state_out) + static_cast<long long>(s.n) * (W - 1) * a.D + c;
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) {
      // (read again: an empty sequence hands its state on)
      const F4 v = input_at<W>(x, a.ldx, state, a.D, s, s.len - (W - 1) + j, c);
      store4(out + static_cast<long long>(j) * a.D, v);
    }
  }
}

// With dp_t = dy_t silu'(p_t), p recomputed: dx_t = sum_i w[W-1-i] dp_{t+i}, dw[j] = sum_t dp_t x_{t-(W-1)+j}. A part reads W - 1
// tokens on either side for p and dp. A CTA takes every walkers-th part, so its sums of dw and dbias stay in
// registers; they are joined in a fixed order afterwards.
template <int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvBwdArgs a, int blocks) {
  const int block = blockIdx.x % blocks, walker = blockIdx.x / blocks, walkers = gridDim.x / blocks;
  const int c = 4 * (block * kThreads + threadIdx.x);
  const bool mine = c < a.D;
  const bf16* const x = static_cast<const bf16*>(a.x);
  const bf16* const dy = static_cast<const bf16*>(a.dy);
  const bf16* const state = static_cast<const bf16*>(a.state_in);
  const bf16* const d_out = static_cast<const bf16*>(a.d_state_out);
  bf16* const dx = static_cast<bf16*>(a.dx);
  bf16* const d_in = static_cast<bf16*>(a.d_state_in);
  F4 tap[W], dw[W], db = zero4(), bias = zero4();
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j] = tap[j] = zero4();
  if (mine) {
    load_taps<W>(a.weight, c, tap);
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < 4; ++i) bias.v[i] = __ldg(a.bias + c + i);
    }
  }
  SeqPart s;
  for (int part = walker;
       find_part(a.cu, a.N, a.T, a.T, kBwdTokens, part, s, block == 0 && threadIdx.x < 32 ? a.err_flag : nullptr);
       part += walkers) {
    if (!mine) continue;
    const int t0 = s.part * kBwdTokens, t1 = min(s.len, t0 + kBwdTokens);
    const bool first = s.part == 0;
    const int end = min(s.len, t1 + W - 1);  // dp is needed up to there
    F4 win[W], dp[W];  // dp[W - 1]: the newest
#pragma unroll
    for (int j = 1; j < W; ++j) win[j] = input_at<W>(x, a.ldx, state, a.D, s, t0 - W + j, c), dp[j] = zero4();
    // token t gives dx of t - (W - 1); a first part's first W - 1 are the state's
    for (int t = t0; t < t1 + W - 1; t += kStep) {
      F4 in[kStep], g[kStep];
#pragma unroll
      for (int q = 0; q < kStep; ++q) {
        in[q] = g[q] = zero4();
        if (t + q < end) {
          in[q] = load4(x + static_cast<long long>(s.start + t + q) * a.ldx + c);
          g[q] = load4(dy + static_cast<long long>(s.start + t + q) * a.lddy + c);
        }
      }
#pragma unroll
      for (int q = 0; q < kStep; ++q) {
        const int at = t + q;
        if (at >= t1 + W - 1) break;
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) win[j] = win[j + 1], dp[j] = dp[j + 1];
        win[W - 1] = in[q];
        F4 d = g[q];  // (zero past the sequence's end)
        if (SILU) {
          F4 p = bias;
#pragma unroll
          for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) p.v[i] = fmaf(tap[j].v[i], win[j].v[i], p.v[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float sg = sigmoid(p.v[i]);
            d.v[i] *= sg * fmaf(p.v[i], 1.0f - sg, 1.0f);
          }
        }
        if (at >= end) d = zero4();
        dp[W - 1] = d;
        if (at < t1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) db.v[i] += d.v[i];
#pragma unroll
          for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) dw[j].v[i] = fmaf(d.v[i], win[j].v[i], dw[j].v[i]);
        }
        const int to = at - (W - 1);  // dx_to = sum_i w[W-1-i] dp_{to+i}; dp[i] is dp_{to+i}
        if (to < t0 && !(first && d_in)) continue;
        F4 r = zero4();
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) r.v[i] = fmaf(tap[W - 1 - j].v[i], dp[j].v[i], r.v[i]);
        const int late = to - (s.len - (W - 1));  // inputs that are part of the last state
        if (d_out && late >= 0) {
          const F4 e = load4(d_out + (static_cast<long long>(s.n) * (W - 1) + late) * a.D + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) r.v[i] += e.v[i];
        }
        if (to >= 0) store4(dx + static_cast<long long>(s.start + to) * a.lddx + c, r);
        else store4(d_in + (static_cast<long long>(s.n) * (W - 1) + (W - 1) + to) * a.D + c, r);
      }
    }
  }
  if (!mine || a.part == nullptr) return;
  float* const out = a.part + static_cast<long long>(walker) * (W + 1) * a.D + c;
#pragma unroll
  for (int j = 0; j < W; ++j)
    *reinterpret_cast<float4*>(out + static_cast<long long>(j) * a.D) = make_float4(dw[j].v[0], dw[j].v[1], dw[j].v[2], dw[j].v[3]);
  *reinterpret_cast<float4*>(out + static_cast<long long>(W) * a.D) = make_float4(db.v[0], db.v[1], db.v[2], db.v[3]);
}

// dw [D][W] and db [D] from the parts' [parts][W + 1][D]: eight warps share 32 channels of one row.
__global__ void __launch_bounds__(256) conv_weight_sums_kernel(const float* __restrict__ part, int parts, int D, int W,
                                                               float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sums[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
  float sum = 0.0f;
  if (c < D) {
#pragma unroll 8
    for (int p = g; p < parts; p += 8) sum += __ldg(part + (static_cast<long long>(p) * (W + 1) + j) * D + c);
  }
  sums[g][lane] = sum;
  __syncthreads();
  if (g != 0 || c >= D) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) sum += sums[i][lane];
  if (j < W) {
    if (dw) dw[static_cast<long long>(c) * W + j] = sum;
  } else if (db) {
    db[c] = sum;
  }
}

template <int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepArgs a, int blocks) {
  const int b = blockIdx.x / blocks, c = 4 * (blockIdx.x % blocks * kThreads + threadIdx.x);
  if (c >= a.D) return;
  int slot = a.state_idx ? __ldg(a.state_idx + b) : b;
  if (slot >= a.n_slots) {
    if (c == 0) set_flag(a.err_flag, MOE_FLAG_BAD_INDEX);
    slot = -1;
  }
  bf16* const y = static_cast<bf16*>(a.y) + b * a.ldy + c;
  if (slot < 0) {
    store4(y, zero4());
    return;
  }
  bf16* const state = static_cast<bf16*>(a.state) + static_cast<long long>(slot) * (W - 1) * a.D + c;
  F4 in[W], tap[W];
#pragma unroll
  for (int j = 0; j + 1 < W; ++j) in[j] = load4(state + static_cast<long long>(j) * a.D);
  in[W - 1] = load4(static_cast<const bf16*>(a.x) + b * a.ldx + c);
  load_taps<W>(a.weight, c, tap);
  // Every operation is rounded by itself (no fused products, an exact quotient): the row's scan reads y as rounded to bf16, and a
  // neighbouring bf16 there would be 2^-8 of what it adds to the state. The cache bounds the time all the same.
  F4 p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p.v[i] = __fmul_rn(tap[0].v[i], in[0].v[i]);
#pragma unroll
    for (int j = 1; j < W; ++j) p.v[i] = __fadd_rn(p.v[i], __fmul_rn(tap[j].v[i], in[j].v[i]));
    if (a.bias) p.v[i] = __fadd_rn(__ldg(a.bias + c + i), p.v[i]);
    if (SILU) p.v[i] = __fmul_rn(p.v[i], __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-p.v[i]))));
  }
  store4(y, p);
#pragma unroll
  for (int j = 0; j + 1 < W; ++j) store4(state + static_cast<long long>(j) * a.D, in[j + 1]);
}

int channel_blocks(int D) { return (D / 4 + kThreads - 1) / kThreads; }

// Parts of `length` tokens that N sequences of T tokens can have at most.
int most_parts(int N, int T, int length) { return T / length + N; }

#define MOE_CONV_DISPATCH(KERNEL, GRID)                                                   \
  do {                                                                                     \
    if (a.W == 2) { if (a.silu) KERNEL<2, true><<<(GRID) * blocks, kThreads, 0, st>>>(a, blocks); else KERNEL<2, false><<<(GRID) * blocks, kThreads, 0, st>>>(a, blocks); } \
    else if (a.W == 3) { if (a.silu) KERNEL<3, true><<<(GRID) * blocks, kThreads, 0, st>>>(a, blocks); else KERNEL<3, false><<<(GRID) * blocks, kThreads, 0, st>>>(a, blocks); } \
    else { if (a.silu) KERNEL<4, true><<<(GRID) * blocks, kThreads, 0, st>>>(a, blocks); else KERNEL<4, false><<<(GRID) * blocks, kThreads, 0, st>>>(a, blocks); } \
  } while (0)

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t st) {
  LaunchTimer lt("conv_fwd", st);
  const int blocks = channel_blocks(a.D);
  MOE_CONV_DISPATCH(conv_fwd_kernel, most_parts(a.N, a.T, kFwdTokens));
  return cudaGetLastError();
}

int conv_bwd_parts(int N, int T, int D) {
  const int parts = most_parts(N, T, kBwdTokens), blocks = channel_blocks(D);
  const int most = (num_sms() * 4 + blocks - 1) / blocks;
  return parts < most ? parts : most;
}

cudaError_t launch_conv_bwd(const ConvBwdArgs& a, float* dw, float* db, cudaStream_t st) {
  const int parts = conv_bwd_parts(a.N, a.T, a.D);
  {
    LaunchTimer lt("conv_bwd", st);
    const int blocks = channel_blocks(a.D);
    MOE_CONV_DISPATCH(conv_bwd_kernel, parts);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.part == nullptr) return e;
  }
  LaunchTimer lt("conv_dw", st);
  conv_weight_sums_kernel<<<dim3((a.D + 31) / 32, a.W + 1), 256, 0, st>>>(a.part, parts, a.D, a.W, dw, db);
  return cudaGetLastError();
}

cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t st) {
  LaunchTimer lt("conv_step", st);
  const int blocks = channel_blocks(a.D);
  MOE_CONV_DISPATCH(conv_step_kernel, a.B);
  return cudaGetLastError();
}

}  // namespace moe
