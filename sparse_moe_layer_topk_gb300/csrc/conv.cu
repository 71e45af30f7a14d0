// Causal depthwise convolution of 2 to 4 taps over packed sequences, its backward, and its step.
//
//   p_t = bias + sum_j w[j] x_{t - (W-1) + j};  y_t = p_t or silu(p_t)
//
// A thread owns four channels (8-byte accesses, a warp's 256 bytes of a row) and walks tokens with the last W inputs
// in registers, so every input is read once but for the W - 1 rows before a part. A group of tokens is on its way while the one
// before it is computed, two values an instruction. HBM bounds the forward: 7,864 packed tokens x 8,192 channels in 46 us, 38 of them the
// bytes (parts of 32 tokens in groups of 4: 60; parts of 128: 55).
#include <type_traits>

#include "common.cuh"
#include "mixer.h"
#include "seq.cuh"
#include "timing.h"

namespace moe {

int num_sms();

namespace {

constexpr int kThreads = 128;       // 512 channels
constexpr int kFwdTokens = 64;      // tokens of a part
constexpr int kBwdRing = 4;         // groups of tokens that the backward holds or has on their way
constexpr int kBwdCtas = 4;         // an SM
constexpr float kLog2e = 1.4426950408889634f;

// Four channels.
struct F4 {
  f32x2 a, b;
};

__device__ __forceinline__ F4 make4(float x, float y, float z, float w) { return F4{pack2(x, y), pack2(z, w)}; }
__device__ __forceinline__ F4 widen(uint2 w) { return make4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)); }
__device__ __forceinline__ F4 zero4() { return make4(0.0f, 0.0f, 0.0f, 0.0f); }
__device__ __forceinline__ F4 splat4(float x) { return make4(x, x, x, x); }
__device__ __forceinline__ F4 fma4(const F4& x, const F4& y, const F4& z) { return F4{fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)}; }
__device__ __forceinline__ F4 mul4(const F4& x, const F4& y) { return F4{mul2(x.a, y.a), mul2(x.b, y.b)}; }
__device__ __forceinline__ F4 add4(const F4& x, const F4& y) { return F4{add2(x.a, y.a), add2(x.b, y.b)}; }
__device__ __forceinline__ uint2 load4(const bf16* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ uint2 narrow(const F4& x) { return make_uint2(pack_bf16(x.a), pack_bf16(x.b)); }
__device__ __forceinline__ void store4(bf16* p, uint2 x) { *reinterpret_cast<uint2*>(p) = x; }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 1 / (1 + exp(-x)).
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
  float a, b;
  unpack2(mul2(x, pack2(-kLog2e, -kLog2e)), a, b);
  unpack2(add2(pack2(ex2(a), ex2(b)), pack2(1.0f, 1.0f)), a, b);
  return pack2(rcp(a), rcp(b));
}
__device__ __forceinline__ F4 sigmoid4(const F4& x) { return F4{sigmoid2(x.a), sigmoid2(x.b)}; }

// An asynchronous copy of 8 bytes; `real` false: nothing is read and zeros are written.
__device__ __forceinline__ void copy8(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(real ? 8 : 0) : "memory");
}

// The weights of four channels from [D][W], 4 W values one behind the other.
template <int W>
__device__ __forceinline__ void load_taps(const float* w, int c, float (&v)[4 * W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(w + static_cast<long long>(c) * W) + i);
    v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
  }
}
template <int W>
__device__ __forceinline__ void load_taps(const float* w, int c, F4 (&tap)[W]) {
  float v[4 * W];
  load_taps<W>(w, c, v);
#pragma unroll
  for (int j = 0; j < W; ++j) tap[j] = make4(v[j], v[W + j], v[2 * W + j], v[3 * W + j]);
}
__device__ __forceinline__ F4 load_bias(const float* bias, int c) {
  return bias ? make4(__ldg(bias + c), __ldg(bias + c + 1), __ldg(bias + c + 2), __ldg(bias + c + 3)) : zero4();
}

// Input `at` (from -(W-1)) of a sequence: its tokens, and before them its state.
template <int W>
__device__ __forceinline__ uint2 input_at(const bf16* x, long long ldx, const bf16* state, int D, const SeqPart& s, int at, int c) {
  if (at >= 0) return load4(x + (s.start + at) * ldx + c);
  if (state == nullptr) return make_uint2(0, 0);
  return load4(state + (static_cast<long long>(s.n) * (W - 1) + (W - 1) + at) * D + c);
}

template <int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 5) conv_fwd_kernel(ConvArgs a, int blocks) {
  constexpr int kStep = 8;
  const int block = blockIdx.x % blocks;  // of channels
  SeqPart s;
  if (!find_part(a.cu, a.N, a.T, a.T, kFwdTokens, blockIdx.x / blocks, s, block == 0 && threadIdx.x < 32 ? a.err_flag : nullptr)) return;
  const int c = 4 * (block * kThreads + threadIdx.x);
  if (c >= a.D) return;
  const bf16* const x = static_cast<const bf16*>(a.x);
  const bf16* const state = static_cast<const bf16*>(a.state_in);
  const int t0 = s.part * kFwdTokens, t1 = min(s.len, t0 + kFwdTokens);
  const bf16* from = x + static_cast<long long>(s.start + t0) * a.ldx + c;
  bf16* to = static_cast<bf16*>(a.y) + static_cast<long long>(s.start + t0) * a.ldy + c;
  uint2 next[kStep];
  const auto fetch = [&](int left) {  // the next group of tokens
#pragma unroll
    for (int q = 0; q < kStep; ++q) {
      next[q] = make_uint2(0, 0);
      if (q < left) next[q] = load4(from + q * a.ldx);
    }
    from += kStep * a.ldx;
  };
  fetch(t1 - t0);
  F4 tap[W], in[W - 1 + kStep];
  load_taps<W>(a.weight, c, tap);
  const F4 bias = load_bias(a.bias, c);
#pragma unroll
  for (int j = 0; j + 1 < W; ++j) in[j] = widen(input_at<W>(x, a.ldx, state, a.D, s, t0 - (W - 1) + j, c));
  for (int t = t0; t < t1; t += kStep) {
#pragma unroll
    for (int q = 0; q < kStep; ++q) in[W - 1 + q] = widen(next[q]);
    fetch(t1 - t - kStep);
#pragma unroll
    for (int q = 0; q < kStep; ++q) {
      F4 p = bias;
#pragma unroll
      for (int j = 0; j < W; ++j) p = fma4(tap[j], in[q + j], p);
      if (SILU) p = mul4(p, sigmoid4(p));
      if (t + q < t1) store4(to + q * a.ldy, narrow(p));
    }
    to += kStep * a.ldy;
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) in[j] = in[kStep + j];
  }
  if (a.state_out && t1 == s.len) {
    bf16* const out = static_cast<bf16*>(a.state_out) + static_cast<long long>(s.n) * (W - 1) * a.D + c;
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)  // (read again: an empty sequence hands its state on)
      store4(out + static_cast<long long>(j) * a.D, input_at<W>(x, a.ldx, state, a.D, s, s.len - (W - 1) + j, c));
  }
}

// With dp_t = dy_t silu'(p_t), p recomputed: dx_t = sum_i w[W-1-i] dp_{t+i}, dw[j] = sum_t dp_t x_{t-(W-1)+j}. A part reads W - 1
// tokens on either side for p and dp. A CTA takes every walkers-th part, so its sums of dw and dbias stay in
// registers; they are joined in a fixed order afterwards. Tokens come by asynchronous copies three groups ahead, which a thread makes and
// waits for by itself: in registers there is room for one group, and it waits for memory. 40 registers of weights and sums and the two
// windows leave 16 warps an SM, whose arithmetic bounds it: 16,384 tokens x 8,192 channels in 149 us, 119 of them the bytes (with one group ahead in
// registers 184; groups of 2 tokens instead of 4: 166, of 6: 153; three CTAs an SM: 165, five spill: 190 and more).
// FEW: less than 128 sequences, as find_part takes it. (Its walk over more of them in the parts' loop costs the tokens' loop registers: 157 us for 153.)
template <int W, bool SILU, bool FEW>
__global__ void __launch_bounds__(kThreads, kBwdCtas) conv_bwd_kernel(ConvBwdArgs a, int blocks, int length) {
  constexpr int kStep = 4;
  __shared__ uint2 ring[kBwdRing][kStep][2][kThreads];  // (x, dy) of a thread's channels, its own to write and to read
  const uint32_t to_ring = smem_u32(&ring[0][0][0][threadIdx.x]);
  const int block = blockIdx.x % blocks, walker = blockIdx.x / blocks, walkers = gridDim.x / blocks;
  const int c = 4 * (block * kThreads + threadIdx.x);
  const bool mine = c < a.D;
  const bf16* const x = static_cast<const bf16*>(a.x);
  const bf16* const state = static_cast<const bf16*>(a.state_in);
  const bf16* const d_out = static_cast<const bf16*>(a.d_state_out);
  bf16* const d_in = static_cast<bf16*>(a.d_state_in);
  F4 tap[W], dw[W], db = zero4(), bias = zero4();
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j] = tap[j] = zero4();
  if (mine) {
    load_taps<W>(a.weight, c, tap);
    bias = load_bias(a.bias, c);
  }
  SeqPart s;
  for (int part = walker;
       find_part<FEW>(a.cu, a.N, a.T, a.T, length, part, s, block == 0 && threadIdx.x < 32 ? a.err_flag : nullptr);
       part += walkers) {
    if (!mine) continue;
    const int t0 = s.part * length, t1 = min(s.len, t0 + length);
    const int end = min(s.len, t1 + W - 1);  // dp is needed up to there
    const int first = s.part == 0 && d_in ? -(W - 1) : t0;  // the first dx of this part
    const bf16* fx = x + static_cast<long long>(s.start + t0) * a.ldx + c;
    const bf16* fg = static_cast<const bf16*>(a.dy) + static_cast<long long>(s.start + t0) * a.lddy + c;
    bf16* to = static_cast<bf16*>(a.dx) + static_cast<long long>(s.start + t0 - (W - 1)) * a.lddx + c;
    int ahead = t0, slot = 0;  // of the next group of tokens to be fetched
    const auto fetch = [&] {
#pragma unroll
      for (int q = 0; q < kStep; ++q) {
        const bool some = ahead + q < end;  // (zeros past the sequence's end)
        const uint32_t to = to_ring + slot * (kStep * 2 * kThreads * 8) + q * (2 * kThreads * 8);
        copy8(to, some ? fx + q * a.ldx : fx, some);
        copy8(to + kThreads * 8, some ? fg + q * a.lddy : fg, some);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (ahead + kStep < end) fx += kStep * a.ldx, fg += kStep * a.lddy;  // (never past what there is)
      ahead += kStep, slot = (slot + 1) % kBwdRing;
    };
#pragma unroll
    for (int g = 0; g + 1 < kBwdRing; ++g) fetch();
    int now = 0;  // the group in hand
    F4 in[W], dp[W];  // the newest last
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) in[j] = widen(input_at<W>(x, a.ldx, state, a.D, s, t0 - (W - 1) + j, c)), dp[j] = zero4();
    // token t gives dx of t - (W - 1); a first part's first W - 1 are the state's
    const auto group = [&](int t, auto inside) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kBwdRing - 2) : "memory");
      const uint2(*const own)[2][kThreads] = ring[now];
      now = (now + 1) % kBwdRing;
      fetch();  // into the place of the group before this one
#pragma unroll
      for (int q = 0; q < kStep; ++q) {
        const int at = t + q;
        in[W - 1] = widen(own[q][0][threadIdx.x]);
        F4& d = dp[W - 1];
        d = widen(own[q][1][threadIdx.x]);
        if (SILU) {
          F4 p = bias;
#pragma unroll
          for (int j = 0; j < W; ++j) p = fma4(tap[j], in[j], p);
          const F4 sg = sigmoid4(p);
          // silu' = sg (1 + p (1 - sg))
          d = mul4(mul4(d, sg), fma4(p, fma4(sg, splat4(-1.0f), splat4(1.0f)), splat4(1.0f)));
        }
        if (inside.value || at < t1) {
          db = add4(db, d);
#pragma unroll
          for (int j = 0; j < W; ++j) dw[j] = fma4(d, in[j], dw[j]);
        }
        const int out = at - (W - 1);  // dx_out = sum_i w[W-1-i] dp_{out+i}; dp[i] is dp_{out+i}
        if (inside.value || (out >= first && out < t1)) {
          F4 r = zero4();
#pragma unroll
          for (int j = 0; j < W; ++j) r = fma4(tap[W - 1 - j], dp[j], r);
          const int late = out - (s.len - (W - 1));  // inputs that are part of the last state
          if (!inside.value && d_out && late >= 0) r = add4(r, widen(load4(d_out + (static_cast<long long>(s.n) * (W - 1) + late) * a.D + c)));
          if (inside.value || out >= 0) store4(to + q * a.lddx, narrow(r));
          else store4(d_in + (static_cast<long long>(s.n) * (W - 1) + (W - 1) + out) * a.D + c, narrow(r));
        }
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) in[j] = in[j + 1], dp[j] = dp[j + 1];
      }
      to += kStep * a.lddx;
    };
    for (int t = t0; t < t1 + W - 1; t += kStep) {
      // inside: all of the group's tokens are the part's, and all of its dx too (none is late either: t + kStep <= s.len)
      if (t - (W - 1) >= t0 && t + kStep <= t1) group(t, std::true_type{});
      else group(t, std::false_type{});
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  allow_next_kernel();
  if (!mine || a.part == nullptr) return;
  float* const out = a.part + static_cast<long long>(walker) * (W + 1) * a.D + c;
  const auto put = [&](int j, const F4& v) {
    float4 f;
    unpack2(v.a, f.x, f.y);
    unpack2(v.b, f.z, f.w);
    *reinterpret_cast<float4*>(out + static_cast<long long>(j) * a.D) = f;
  };
#pragma unroll
  for (int j = 0; j < W; ++j) put(j, dw[j]);
  put(W, db);
}

// dw [D][W] and db [D] from the walkers' [walkers][W + 1][D], in one order: 16 warps share 32 channels of one row.
__global__ void __launch_bounds__(512) conv_weight_sums_kernel(const float* __restrict__ part, int parts, int D, int W,
                                                               float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sums[16][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
  wait_for_last_kernel();
  float sum = 0.0f;
  if (c < D) {
#pragma unroll 4
    for (int p = g; p < parts; p += 16) sum += __ldg(part + (static_cast<long long>(p) * (W + 1) + j) * D + c);
  }
  sums[g][lane] = sum;
  __syncthreads();
  if (g != 0 || c >= D) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) sum += sums[i][lane];
  if (j < W) {
    if (dw) dw[static_cast<long long>(c) * W + j] = sum;
  } else if (db) {
    db[c] = sum;
  }
}

template <int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepArgs a, int blocks) {
  const int b = blockIdx.x / blocks, c = 4 * (blockIdx.x % blocks * kThreads + threadIdx.x);
  allow_next_kernel();  // (a scan's step, which waits for y before it reads anything that is written here)
  if (c >= a.D) return;
  int slot = a.state_idx ? __ldg(a.state_idx + b) : b;
  if (slot >= a.n_slots) {
    if (c == 0) set_flag(a.err_flag, MOE_FLAG_BAD_INDEX);
    slot = -1;
  }
  bf16* const y = static_cast<bf16*>(a.y) + b * a.ldy + c;
  if (slot < 0) {
    store4(y, make_uint2(0, 0));
    return;
  }
  bf16* const state = static_cast<bf16*>(a.state) + static_cast<long long>(slot) * (W - 1) * a.D + c;
  uint2 in[W];
  float tap[4 * W];
#pragma unroll
  for (int j = 0; j + 1 < W; ++j) in[j] = load4(state + static_cast<long long>(j) * a.D);
  in[W - 1] = load4(static_cast<const bf16*>(a.x) + b * a.ldx + c);
  load_taps<W>(a.weight, c, tap);
  // Every operation is rounded by itself (no fused products, an exact quotient), so that y is what the formula gives step by step in fp32: the
  // row's scan reads it as rounded to bf16, and a neighbouring bf16 there is 2^-8 of what it adds to the state. The packed pass fuses its products
  // and takes a quick reciprocal, so a few of its outputs are such neighbours of these. The cache bounds the time all the same.
  float p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto value = [&](int j) { return i == 0 ? bf16_lo(in[j].x) : i == 1 ? bf16_hi(in[j].x) : i == 2 ? bf16_lo(in[j].y) : bf16_hi(in[j].y); };
    p[i] = __fmul_rn(tap[i * W], value(0));
#pragma unroll
    for (int j = 1; j < W; ++j) p[i] = __fadd_rn(p[i], __fmul_rn(tap[i * W + j], value(j)));
    if (a.bias) p[i] = __fadd_rn(__ldg(a.bias + c + i), p[i]);
    if (SILU) p[i] = __fmul_rn(p[i], __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-p[i]))));
  }
  store4(y, make_uint2(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3])));
#pragma unroll
  for (int j = 0; j + 1 < W; ++j) store4(state + static_cast<long long>(j) * a.D, in[j + 1]);
}

int channel_blocks(int D) { return (D / 4 + kThreads - 1) / kThreads; }

// Parts of `length` tokens that N sequences of T tokens can have at most.
int most_parts(int N, int T, int length) { return T / length + N; }

#define MOE_CONV_DISPATCH(KERNEL, GRID, ...)                                                   \
  do {                                                                                          \
    const auto run = [&](auto kernel) { kernel<<<(GRID) * blocks, kThreads, 0, st>>>(__VA_ARGS__); }; \
    if (a.W == 2) a.silu ? run(KERNEL(2, true)) : run(KERNEL(2, false));                        \
    else if (a.W == 3) a.silu ? run(KERNEL(3, true)) : run(KERNEL(3, false));                   \
    else a.silu ? run(KERNEL(4, true)) : run(KERNEL(4, false));                                 \
  } while (0)
#define MOE_CONV_FWD(W, SILU) conv_fwd_kernel<W, SILU>
#define MOE_CONV_BWD_FEW(W, SILU) conv_bwd_kernel<W, SILU, true>
#define MOE_CONV_BWD_MANY(W, SILU) conv_bwd_kernel<W, SILU, false>
#define MOE_CONV_STEP(W, SILU) conv_step_kernel<W, SILU>

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t st) {
  LaunchTimer lt("conv_fwd", st);
  const int blocks = channel_blocks(a.D);
  MOE_CONV_DISPATCH(MOE_CONV_FWD, most_parts(a.N, a.T, kFwdTokens), a, blocks);
  return cudaGetLastError();
}

// The backward's division: CTAs that walk the parts of a channel block, and a part's tokens, of which there are enough that the last round of
// parts is a full one, if the sequences are equally long (a part costs ten tokens more than it has: its start, its neighbours).
struct BwdDivision {
  int walkers, length;
};
static BwdDivision divide_bwd(int N, int T, int D) {
  const int blocks = channel_blocks(D), most = (num_sms() * kBwdCtas + blocks - 1) / blocks;
  const long long each = (static_cast<long long>(T) + N - 1) / N;
  BwdDivision best{1, 16};
  long long least = 1ll << 62;
  for (int length = 16; length <= 256; length += 4) {
    const long long parts = N * ((each + length - 1) / length), cost = (parts + most - 1) / most * (length + 10);
    if (cost < least) least = cost, best.length = length;
  }
  const int parts = most_parts(N, T, best.length);
  best.walkers = parts < most ? parts : most;
  return best;
}

int conv_bwd_parts(int N, int T, int D) { return divide_bwd(N, T, D).walkers; }

cudaError_t launch_conv_bwd(const ConvBwdArgs& a, float* dw, float* db, cudaStream_t st) {
  const BwdDivision d = divide_bwd(a.N, a.T, a.D);
  const int parts = d.walkers;
  {
    LaunchTimer lt("conv_bwd", st);
    const int blocks = channel_blocks(a.D);
    if (a.cu == nullptr || a.N < kWalk) MOE_CONV_DISPATCH(MOE_CONV_BWD_FEW, parts, a, blocks, d.length);
    else MOE_CONV_DISPATCH(MOE_CONV_BWD_MANY, parts, a, blocks, d.length);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.part == nullptr) return e;
  }
  LaunchTimer lt("conv_dw", st);
  return launch_behind(conv_weight_sums_kernel, dim3((a.D + 31) / 32, a.W + 1), 512, 0, st, static_cast<const float*>(a.part), parts, a.D, a.W, dw, db);
}

cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t st) {
  LaunchTimer lt("conv_step", st);
  const int blocks = channel_blocks(a.D);
  MOE_CONV_DISPATCH(MOE_CONV_STEP, a.B, a, blocks);
  return cudaGetLastError();
}

}  // namespace moe
