// Selective state space scan over packed sequences, its backward, and its step.
//
//   dt_t = softplus(delta_t + dt_bias);  h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t;
//   y_t = (C_t . h_t + skip u_t) silu(z_t)
//
// Every channel has S <= 16 states with decays of their own, so nothing of this is a matrix product: it is an
// exponential, two products and two sums for each state and token. Four lanes share two channels, four states of each
// in a lane's fp32 registers, so that a B and a C from shared memory serve both. (One channel a lane: shared memory bounds it. Four:
// too few warps to hide the arithmetic's latency.) A CTA takes 32 tokens of its channels at a time: whole rows of 128 or 256 bytes
// arrive by asynchronous copies a tile ahead (a warp fetching its own 16 channels touches four times the cache lines, which cost as
// much time as the recurrence); (dt, dt u) of four neighbouring channels a thread go to shared memory; then each warp walks
// the tokens with its 16 channels' states; then skip, gate and store, four neighbouring channels a thread again.
// 4 x 1,024 tokens x 8,192 channels take 188 us, 40 of them the bytes and 75 the exponentials: seven instructions a state and token, of which 12 warps
// an SM issue 2.4 of 4 a clock, and the latencies between them.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "mixer.h"
#include "scan.h"
#include "seq.cuh"
#include "timing.h"

namespace moe {

int num_sms();

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 2.2e-8f;
constexpr int kTile = kScanTile;
constexpr int kBRow = 20;  // floats of a token's B or C: sixteen and four of padding (no bank conflicts)
constexpr int kC = 2;           // channels of a lane in the recurrence
constexpr int kCh = 16;         // channels of a warp
constexpr int kFwdWarps = 4;
constexpr int kBwdWarps = 8;

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

// 1 / (1 + exp(-x)) of two values.
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
  float a, b;
  unpack2(mul2(x, pack2(-kLog2e, -kLog2e)), a, b);
  unpack2(add2(pack2(ex2(a), ex2(b)), pack2(1.0f, 1.0f)), a, b);
  return pack2(rcp(a), rcp(b));
}

// The magnitude of x up to 128, where exp(-|x|) is 0 already: the product below may not pass fp32 for a token that is masked by the lowest
// value of its type or by -infinity. NaN stays NaN.
__device__ __forceinline__ float up_to_128(float x) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(x)), "f"(128.0f));
  return r;
}

// max(x, 0) + log(1 + e), e = exp(-|x|), of two values. The exponent's product is taken in two terms (it would lose |x| 2^-24
// of e), and log(1 + e) / e is a polynomial of degree 9, fitted on [0, 1] with equal relative errors (5e-9; 1.5e-7 with its
// roundings), so that small results keep their relative precision: dt multiplies all that reaches a state.
__device__ __forceinline__ f32x2 softplus2(f32x2 x) {
  float a, b;
  unpack2(x, a, b);
  const f32x2 n = pack2(up_to_128(a), up_to_128(b)), above = pack2(fmaxf(a, 0.0f), fmaxf(b, 0.0f)), l2e = pack2(-kLog2e, -kLog2e);
  const f32x2 m = mul2(n, l2e);
  const f32x2 lost = fma2(n, pack2(kLog2e, kLog2e), m);
  unpack2(m, a, b);
  f32x2 e = pack2(ex2(a), ex2(b));
  e = fma2(mul2(e, pack2(-kLn2, -kLn2)), lost, e);
  constexpr float c[9] = {0.019851261749863625f, -0.056959159672260284f, 0.10603617131710052f, -0.15305569767951965f, 0.19675931334495544f,
                          -0.24954132735729218f, 0.3332996368408203f,    -0.4999990165233612f, 1.0f};
  f32x2 p = pack2(-0.003243980696424842f, -0.003243980696424842f);
#pragma unroll
  for (int i = 0; i < 9; ++i) p = fma2(p, e, pack2(c[i], c[i]));
  return fma2(p, e, above);
}
__device__ __forceinline__ float softplus(float x) {
  float a, b;
  unpack2(softplus2(pack2(x, 0.0f)), a, b);
  return a;
}

// Shared-memory loads that the compiler may move over stores (it cannot tell that those go to other places, and would
// otherwise begin no token before the one ahead of it has stored its results). They stay below the `after_sync` that
// their address comes from, and above whatever uses their values.
__device__ __forceinline__ uint32_t after_sync(const void* p) {
  uint32_t a = smem_u32(p);
  asm volatile("" : "+r"(a)::"memory");
  return a;
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
  float4 v;
  asm("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float2 lds2(uint32_t a) {
  float2 v;
  asm("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}

// The channels of a CTA: `c0` the first, `have` how many of them there are, all in `group`.
struct Channels {
  int c0, have, group;
};

// Blocks of `width` channels, none across a group's end.
__device__ __forceinline__ Channels block_channels(int block, int D, int G, int width) {
  const int per = D / G, blocks = (per + width - 1) / width;
  const int g = block / blocks, at = (block - g * blocks) * width;
  return Channels{g * per + at, min(width, per - at), g};
}

// Asynchronous copies of 16 or 8 bytes; `real` false: nothing is read and zeros are written.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(real ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// A CTA's channels of one tile after another into shared memory, [token][channel] (bf16). `wide`: rows start on 16 bytes
// (pieces of eight channels), else on 8 (of four).
template <int WARPS>
struct RowStream {
  static constexpr int kPieces = 2 * WARPS;  // of eight channels in a row
  const bf16* at;                            // this thread's first piece of the next tile
  long long ld;
  bool mine;                                 // whether its channels exist
  __device__ __forceinline__ RowStream(const void* rows, long long first_row, long long ld_, const Channels& ch, bool wide) {
    ld = ld_;
    const int i = threadIdx.x, c = wide ? 8 * (i % kPieces) : 4 * (i % (2 * kPieces)), t = wide ? i / kPieces : i / (2 * kPieces);
    mine = c < ch.have;
    at = static_cast<const bf16*>(rows) + (mine ? (first_row + t) * ld + ch.c0 + c : 0);
  }
  __device__ __forceinline__ void fetch(uint32_t to, int n, bool wide) const {  // the next tile's first n tokens
    const int i = threadIdx.x;
    if (wide) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool real = mine && i / kPieces + 16 * k < n;
        copy16(to + 16 * (i + 32 * WARPS * k), real ? at + 16 * k * ld : at, real);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool real = mine && i / (2 * kPieces) + 8 * k < n;
        copy8(to + 8 * (i + 32 * WARPS * k), real ? at + 8 * k * ld : at, real);
      }
    }
  }
  __device__ __forceinline__ void move(int tiles) { at += mine ? tiles * kTile * ld : 0; }
};

// B (and C) of one tile after another, S values a token (a multiple of 4 up to 16), through registers to shared memory, where they are
// fp32: [token][16] with padding, C after B. A thread has four values of a token, of every WARPS * 4-th one.
template <int WARPS>
struct BcStream {
  static constexpr int kEach = 8 / WARPS;
  const bf16* at;
  long long ld;
  bool mine;
  uint2 v[kEach];
  __device__ __forceinline__ BcStream(const void* B, const void* C, long long first_row, long long ldb, long long ldc, const Channels& ch, int S) {
    const int i = threadIdx.x, piece = i & 3;
    const bool is_c = i & 4;
    ld = is_c ? ldc : ldb;
    mine = 4 * piece < S && (is_c ? C : B) != nullptr;
    at = static_cast<const bf16*>(is_c ? C : B) + (mine ? (first_row + (i >> 3)) * ld + ch.group * S + 4 * piece : 0);
  }
  __device__ __forceinline__ void fetch(int n) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      v[k] = make_uint2(0, 0);
      if (mine && static_cast<int>(threadIdx.x >> 3) + 4 * WARPS * k < n) v[k] = *reinterpret_cast<const uint2*>(at + 4 * WARPS * k * ld);
    }
  }
  __device__ __forceinline__ void put(float* to) const {
    const int i = threadIdx.x;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      *reinterpret_cast<float4*>(to + (i & 4 ? kTile * kBRow : 0) + ((i >> 3) + 4 * WARPS * k) * kBRow + 4 * (i & 3)) =
          make_float4(bf16_lo(v[k].x), bf16_hi(v[k].x), bf16_lo(v[k].y), bf16_hi(v[k].y));
  }
  __device__ __forceinline__ void move(int tiles) { at += mine ? tiles * kTile * ld : 0; }
};

// Four neighbouring channels.
struct Quad {
  f32x2 a, b;
};
__device__ __forceinline__ Quad quad(float x, float y, float z, float w) { return Quad{pack2(x, y), pack2(z, w)}; }
__device__ __forceinline__ Quad quad(float4 v) { return quad(v.x, v.y, v.z, v.w); }
__device__ __forceinline__ Quad zero_quad() { return quad(0.0f, 0.0f, 0.0f, 0.0f); }
__device__ __forceinline__ float4 floats(const Quad& v) {
  float4 f;
  unpack2(v.a, f.x, f.y);
  unpack2(v.b, f.z, f.w);
  return f;
}
__device__ __forceinline__ Quad quad_at(const bf16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return quad(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ Quad quad_at(const float* p) { return quad(*reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ Quad weights_at(const float* p, int c, bool real) {  // of four channels
  return p && real ? quad(__ldg(p + c), __ldg(p + c + 1), __ldg(p + c + 2), __ldg(p + c + 3)) : zero_quad();
}
__device__ __forceinline__ void put_quad(bf16* p, const Quad& v) { *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.a), pack_bf16(v.b)); }
__device__ __forceinline__ Quad add(const Quad& x, const Quad& y) { return Quad{add2(x.a, y.a), add2(x.b, y.b)}; }
__device__ __forceinline__ Quad mul(const Quad& x, const Quad& y) { return Quad{mul2(x.a, y.a), mul2(x.b, y.b)}; }
__device__ __forceinline__ Quad fma(const Quad& x, const Quad& y, const Quad& z) { return Quad{fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)}; }
__device__ __forceinline__ Quad sigmoid(const Quad& x) { return Quad{sigmoid2(x.a), sigmoid2(x.b)}; }
__device__ __forceinline__ Quad softplus(const Quad& x) { return Quad{softplus2(x.a), softplus2(x.b)}; }
// (x, y) of four channels, one channel's pair behind the other.
__device__ __forceinline__ void put_pairs(float* p, const Quad& x, const Quad& y) {
  const float4 u = floats(x), v = floats(y);
  *reinterpret_cast<float4*>(p) = make_float4(u.x, v.x, u.y, v.y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(u.z, v.z, u.w, v.w);
}
__device__ __forceinline__ void get_pairs(const float* p, Quad& x, Quad& y) {
  const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
  x = quad(u.x, u.z, v.x, v.z), y = quad(u.y, u.w, v.y, v.w);
}

struct State4 {
  f32x2 a, b;
};
__device__ __forceinline__ State4 pack4(float4 v) { return State4{pack2(v.x, v.y), pack2(v.z, v.w)}; }
__device__ __forceinline__ float4 unpack4(const State4& s) {
  float4 v;
  unpack2(s.a, v.x, v.y);
  unpack2(s.b, v.z, v.w);
  return v;
}
__device__ __forceinline__ State4 ex2(const State4& s) {
  const float4 v = unpack4(s);
  return pack4(make_float4(ex2(v.x), ex2(v.y), ex2(v.z), ex2(v.w)));
}
__device__ __forceinline__ State4 mul4(f32x2 x, const State4& s) { return State4{mul2(x, s.a), mul2(x, s.b)}; }
__device__ __forceinline__ State4 mul4(const State4& x, const State4& s) { return State4{mul2(x.a, s.a), mul2(x.b, s.b)}; }
__device__ __forceinline__ State4 fma4(const State4& x, const State4& s, const State4& c) {
  return State4{fma2(x.a, s.a, c.a), fma2(x.b, s.b, c.b)};
}
__device__ __forceinline__ State4 fma4(f32x2 x, const State4& s, const State4& c) {
  return State4{fma2(x, s.a, c.a), fma2(x, s.b, c.b)};
}
// exp(dt A) of four states, `decay` being A / ln 2. The exponential unit's results just below one are 1e-8 too small on average (measured:
// 0.6e-8 for arguments of 1e-4 to 1e-3, 1.2e-8 to 1e-2, 2.2e-8 to 0.1), which a state with a memory of a thousand tokens adds up to
// 1e-5 of itself. The argument is raised by as much (log2 of it), in the product's own instruction; it still gives 1 for dt = 0. Gradients
// of A over 3,000 tokens: 1.7e-6 off without, 0.7e-6 with it.
__device__ __forceinline__ State4 decays(f32x2 dt, const State4& decay) {
  const f32x2 raise = pack2(kRaise, kRaise);
  return ex2(State4{fma2(dt, decay.a, raise), fma2(dt, decay.b, raise)});
}
__device__ __forceinline__ float sum4(const State4& x, const State4& y) {  // x . y
  float a, b;
  unpack2(fma2(x.b, y.b, mul2(x.a, y.a)), a, b);
  return a + b;
}
__device__ __forceinline__ State4 zero4() { return pack4(make_float4(0, 0, 0, 0)); }

// v[0..3] of four lanes (lane bits 0 and 1) joined: lane q gets the sum over the four lanes of their v[q].
__device__ __forceinline__ float join4(float v0, float v1, float v2, float v3, int q) {
  const bool odd = q & 1, high = q & 2;
  const float a = (odd ? v1 : v0) + __shfl_xor_sync(kAll, odd ? v0 : v1, 1);
  const float b = (odd ? v3 : v2) + __shfl_xor_sync(kAll, odd ? v2 : v3, 1);
  return (high ? b : a) + __shfl_xor_sync(kAll, high ? a : b, 2);
}

// Where a sequence's tile states begin: tiles of kTile tokens, so that all sequences' are at most T / kTile + N.
__device__ __forceinline__ long long tile_base(const SeqPart& s) { return static_cast<long long>(s.start) / kTile + s.n; }

constexpr int kFwdRow = kCh * kFwdWarps;      // channels of a CTA
constexpr int kFwdTile = kTile * kFwdRow;     // values of a tile
constexpr int kFwdQuads = kFwdRow / 4;        // a thread's place where it takes four neighbouring channels of every eighth token
// Shared memory: two stages of u, delta and z; the pairs; two stages of B and C.
constexpr int kFwdSmem = (2 * 3 * kFwdTile / 2 + 2 * kFwdTile + 2 * 2 * kTile * kBRow) * 4;

// SUMS: only the state that a part leaves from a zero state and the sum of its dt, for parts of long sequences. FEW: less than 128 sequences, as
// find_part takes it (its call for more of them costs 1 % in the registers that are left).
template <bool SUMS, bool FEW>
__global__ void __launch_bounds__(kFwdWarps * 32, 4) scan_fwd_kernel(ScanArgs a, int blocks, int length, const float* starts,
                                                                     float* sums, float* dt_sums) {
  extern __shared__ float pool[];
  const int warp = threadIdx.x >> 5, lane = static_cast<int>(lane_id());
  const int part = blockIdx.x / blocks;
  SeqPart s;
  if (!find_part<FEW>(a.cu, a.N, a.T, a.max_seqlen, length, part, s, !SUMS && blockIdx.x % blocks == 0 && warp == 0 ? a.err_flag : nullptr)) return;
  const Channels ch = block_channels(blockIdx.x % blocks, a.D, a.G, kFwdRow);
  const int t0 = s.part * length, count = min(length, s.len - t0);  // (0 in an empty sequence)
  if (SUMS && length >= s.len - t0) return;  // nothing reads the last part's
  bf16* const raw = reinterpret_cast<bf16*>(pool);  // [stage][u, delta, z]
  float* const s_dt = pool + 2 * 3 * kFwdTile / 2;  // [token][channel] (dt, dt u); then y in the first half of a warp's part
  float* const s_bc = s_dt + 2 * kFwdTile;          // [stage][B, C]

  if (SUMS) allow_next_kernel();
  else wait_for_last_kernel();  // (behind the join where the sequences are cut)
  const int q = lane & 3, first = warp * kCh + (lane >> 2) * kC;  // four states of two channels
  const long long all = static_cast<long long>(a.D) * a.S;
  const long long state_at = (static_cast<long long>(ch.c0) + first) * a.S + 4 * q;
  State4 decay[kC], h[kC];
  bool real[kC];
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    real[j] = first + j < ch.have && 4 * q < a.S;
    decay[j] = h[j] = zero4();
    if (real[j]) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.A + state_at + j * a.S));
      decay[j] = pack4(make_float4(v.x * kLog2e, v.y * kLog2e, v.z * kLog2e, v.w * kLog2e));
      const float* const from = SUMS ? nullptr : starts ? starts + part * all : a.state_in ? a.state_in + s.n * all : nullptr;
      if (from) h[j] = pack4(*reinterpret_cast<const float4*>(from + state_at + j * a.S));
    }
  }
  const bool wide = (a.D / a.G) % 8 == 0, gated = !SUMS && a.z != nullptr;
  const long long row0 = s.start + t0;
  RowStream<kFwdWarps> u(a.u, row0, a.ldu, ch, wide), delta(a.delta, row0, a.ldd, ch, wide),
      z(gated ? a.z : a.u, row0, gated ? a.ldz : a.ldu, ch, wide);
  BcStream<kFwdWarps> bc(a.B, SUMS ? nullptr : a.C, row0, a.ldb, a.ldc, ch, a.S);
  const auto fetch = [&](int n, int stage) {
    if (n > 0) {
      const uint32_t to = smem_u32(raw + stage * 3 * kFwdTile);
      u.fetch(to, n, wide), u.move(1);
      delta.fetch(to + 2 * kFwdTile, n, wide), delta.move(1);
      if (gated) z.fetch(to + 4 * kFwdTile, n, wide), z.move(1);
      bc.fetch(n), bc.move(1);
    }
    copies_commit();
  };
  const int four = 4 * (threadIdx.x % kFwdQuads), token = threadIdx.x / kFwdQuads;
  const bool four_real = four < ch.have;
  const Quad bias = weights_at(a.dt_bias, ch.c0 + four, four_real), skip = weights_at(a.skip, ch.c0 + four, four_real);
  float dt_sum[kC] = {0.0f, 0.0f};
  float* tiles = !SUMS && a.tile_states ? a.tile_states + (tile_base(s) + t0 / kTile) * all + state_at : nullptr;
  bf16* out = SUMS ? nullptr : static_cast<bf16*>(a.y) + (row0 + token) * a.ldy + ch.c0 + four;
  fetch(count, 0);
  int stage = 0;
  for (int tile = 0; tile < count; tile += kTile, stage ^= 1) {
    const int n = min(kTile, count - tile);
    float* const s_b = s_bc + stage * 2 * kTile * kBRow;
    bc.put(s_b);
    copies_done();
    __syncthreads();  // the tile is here, and nothing reads the one before it any more
    fetch(count - tile - kTile, stage ^ 1);
    const bf16* const now = raw + stage * 3 * kFwdTile + token * kFwdRow + four;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = 8 * k * kFwdRow;
      const Quad v = quad_at(now + at);
      Quad x = add(quad_at(now + kFwdTile + at), bias);
      if (a.softplus) x = softplus(x);
      if (token + 8 * k >= n) x = zero_quad();  // (a token that is none keeps the state)
      put_pairs(s_dt + 2 * (at + token * kFwdRow + four), x, mul(x, v));
    }
    if (tiles) {
#pragma unroll
      for (int j = 0; j < kC; ++j)
        if (real[j]) *reinterpret_cast<float4*>(tiles + j * a.S) = unpack4(h[j]);
      tiles += all;
    }
    __syncthreads();
    const uint32_t at_dt = after_sync(s_dt + 2 * first), at_b = after_sync(s_b + 4 * q), at_c = at_b + 4 * kTile * kBRow;
    if constexpr (SUMS) {
#pragma unroll 8
      for (int t = 0; t < kTile; ++t) {
        const float4 d = lds4(at_dt + t * 8 * kFwdRow);
        const State4 b = pack4(lds4(at_b + t * 4 * kBRow));
        h[0] = fma4(decays(pack2(d.x, d.x), decay[0]), h[0], mul4(pack2(d.y, d.y), b));
        h[1] = fma4(decays(pack2(d.z, d.z), decay[1]), h[1], mul4(pack2(d.w, d.w), b));
        dt_sum[0] += d.x, dt_sum[1] += d.z;
      }
    } else {
      // Two tokens at a time, in three stages one pair apart, so that a warp's own latencies overlap: shared memory to registers;
      // decays and inputs; the recurrence and y.
      float4 d[2];
      State4 b[2], c[2], e[2][kC], in[2][kC], cc[2];
      float y[2][kC] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
      const auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          d[i] = lds4(at_dt + (t + i) * 8 * kFwdRow);
          b[i] = pack4(lds4(at_b + (t + i) * 4 * kBRow));
          c[i] = pack4(lds4(at_c + (t + i) * 4 * kBRow));
        }
      };
      const auto prepare = [&]() {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          e[i][0] = decays(pack2(d[i].x, d[i].x), decay[0]), in[i][0] = mul4(pack2(d[i].y, d[i].y), b[i]);
          e[i][1] = decays(pack2(d[i].z, d[i].z), decay[1]), in[i][1] = mul4(pack2(d[i].w, d[i].w), b[i]);
          cc[i] = c[i];
        }
      };
      // (over the pairs, of tokens that every lane of the warp has read by now)
      const auto join = [&](int t) {
        s_dt[(t + (q >> 1)) * 2 * kFwdRow + warp * kCh + first + (q & 1)] = join4(y[0][0], y[0][1], y[1][0], y[1][1], q);
      };
      load(0);
      prepare();
      load(2);
#pragma unroll
      for (int t = 0; t < kTile; t += 2) {
        State4 e0[2][kC], in0[2][kC], c0[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          c0[i] = cc[i];
#pragma unroll
          for (int j = 0; j < kC; ++j) e0[i][j] = e[i][j], in0[i][j] = in[i][j];
        }
        if (t + 2 < kTile) prepare();
        if (t + 4 < kTile) load(t + 4);
        if (t > 0) join(t - 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < kC; ++j) {
            h[j] = fma4(e0[i][j], h[j], in0[i][j]);
            y[i][j] = sum4(c0[i], h[j]);
          }
      }
      join(kTile - 2);
    }
    if (!SUMS) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (token + 8 * k < n && four_real) {
          const int at = 8 * k * kFwdRow;
          Quad y = fma(skip, quad_at(now + at), quad_at(s_dt + 2 * (at + token * kFwdRow) + four / kCh * kCh + four));
          if (gated) {
            const Quad g = quad_at(now + 2 * kFwdTile + at);
            y = mul(y, mul(g, sigmoid(g)));
          }
          put_quad(out + 8 * k * a.ldy, y);
        }
      }
      out += kTile * a.ldy;
    }
  }
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    if (SUMS) {
      if (real[j]) *reinterpret_cast<float4*>(sums + part * all + state_at + j * a.S) = unpack4(h[j]);
      if (first + j < ch.have && q == 0) dt_sums[static_cast<long long>(part) * a.D + ch.c0 + first + j] = dt_sum[j];
    } else if (a.state_out && real[j] && t0 + count == s.len) {
      *reinterpret_cast<float4*>(a.state_out + s.n * all + state_at + j * a.S) = unpack4(h[j]);
    }
  }
}

// The states at the parts' starts (REVERSE: the gradients at their ends) from what each part leaves from zero, in place:
// a thread walks the parts of one sequence with four states.
template <bool REVERSE>
__global__ void __launch_bounds__(128) scan_join_kernel(ScanArgs a, int length, const float* first, float* sums,
                                                        const float* dt_sums) {
  const int blocks = (a.D * (a.S / 4) + 127) / 128;
  const int part = blockIdx.x / blocks, i = blockIdx.x % blocks * 128 + threadIdx.x;
  SeqPart s;
  if (!find_part(a.cu, a.N, a.T, a.max_seqlen, length, part, s, nullptr) || s.part != 0) return;
  if (i >= a.D * (a.S / 4)) return;
  allow_next_kernel();
  wait_for_last_kernel();
  const int c = i / (a.S / 4);
  const long long at = 4ll * i, all = static_cast<long long>(a.D) * a.S;
  const int parts = parts_of(s.len, length);
  const float4 A = __ldg(reinterpret_cast<const float4*>(a.A + at));
  float4 h = make_float4(0, 0, 0, 0);
  if (first) h = *reinterpret_cast<const float4*>(first + s.n * all + at);
  constexpr int kBatch = 4;  // parts whose sums are on their way together
  for (int k0 = 0; k0 < parts; k0 += kBatch) {
    float4 e[kBatch];
    float d[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const long long p = part + (REVERSE ? parts - 1 - (k0 + i) : k0 + i);
      e[i] = make_float4(0, 0, 0, 0), d[i] = 0.0f;
      // (the last part in the walk's direction has no sums: nothing follows it)
      if (k0 + i + 1 < parts) e[i] = *reinterpret_cast<const float4*>(sums + p * all + at), d[i] = __ldg(dt_sums + p * a.D + c);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (k0 + i >= parts) break;
      const long long p = part + (REVERSE ? parts - 1 - (k0 + i) : k0 + i);
      *reinterpret_cast<float4*>(sums + p * all + at) = h;
      h.x = fmaf(ex2(A.x * d[i] * kLog2e), h.x, e[i].x);
      h.y = fmaf(ex2(A.y * d[i] * kLog2e), h.y, e[i].y);
      h.z = fmaf(ex2(A.z * d[i] * kLog2e), h.z, e[i].z);
      h.w = fmaf(ex2(A.w * d[i] * kLog2e), h.w, e[i].w);
    }
  }
}

// ------------------------------------------------------------------ backward
//
// With X the gradient that reaches a state from the later tokens:
//   g_t = dy_t silu(z_t);  R_t = X + g_t C_t;  dC_t = g_t h_t;  dB_t = dt_t u_t R_t;  (both summed over the channels)
//   to_b = R_t . B_t;  q = R_t exp(dt_t A) h_{t-1};  ddt = A . q + to_b u_t;  dA += dt_t q;
//   du_t = to_b dt_t + skip g_t;  X = exp(dt_t A) R_t
// Tiles of 32 tokens from the last to the first. The forward kept the state before each; from it the tile's states
// are made again, first all of them (the gate's gradient needs y; every fourth state is noted), then four at a
// time in registers, which the four tokens' backward reads. dB and dC are summed over a warp's channels by exchanging
// halves between lanes, over a CTA's warps in shared memory, and over the CTAs by a second kernel, always in one order.
// 4 x 1,024 tokens x 8,192 channels take 825 us and the sums behind them 17. 241 registers a thread and 213 KB of shared memory leave eight warps
// an SM, and a token takes them 400 ns, nearly as long as it takes five: the latency of its chain bounds it. (Tiles of 16 tokens and
// twelve warps: 979 us.)
constexpr int kBwdRow = kCh * kBwdWarps;      // channels of a CTA
constexpr int kBwdTile = kTile * kBwdRow;
constexpr int kBwdQuads = kBwdRow / 4;
// Shared memory: two stages of u, delta, dy and z; the pairs; y, then g; the warps' noted states; their dB and dC; B and C.
constexpr int kNotes = (kTile / 4) * kC * 128;
constexpr int kBwdSmem = (2 * 4 * kBwdTile / 2 + 2 * kBwdTile + kBwdTile + kBwdWarps * (kNotes + kTile * 32) + 2 * kTile * kBRow) * 4;

struct BwdWs {
  float* tails;     // [parts][D][S] gradients at the parts' ends, where sequences are cut
  float* bc_part;   // [channel blocks][T][32]
  float* dA_part;   // [parts][D][S]
  float* d_part;    // [2][parts][D]: skip, dt_bias
};

template <bool FEW>
__global__ void __launch_bounds__(kBwdWarps * 32, 1) scan_bwd_kernel(ScanBwdArgs a, int blocks, int parts, int length, bool cut, BwdWs ws) {
  extern __shared__ float pool[];
  const ScanArgs& f = a.f;
  const int warp = threadIdx.x >> 5, lane = static_cast<int>(lane_id());
  const int part = blockIdx.x / blocks, block = blockIdx.x % blocks;
  const long long all = static_cast<long long>(f.D) * f.S;
  const Channels ch = block_channels(block, f.D, f.G, kBwdRow);
  SeqPart s;
  if (!find_part<FEW>(f.cu, f.N, f.T, f.max_seqlen, length, part, s, block == 0 && warp == 0 ? f.err_flag : nullptr)) {
    // a part that does not exist adds nothing to the sums over the parts
    for (int i = threadIdx.x; i < ch.have * f.S; i += kBwdWarps * 32) ws.dA_part[part * all + static_cast<long long>(ch.c0) * f.S + i] = 0.0f;
    for (int i = threadIdx.x; i < ch.have; i += kBwdWarps * 32)
      for (int j = 0; j < 2; ++j) ws.d_part[(static_cast<long long>(j) * parts + part) * f.D + ch.c0 + i] = 0.0f;
    return;
  }
  const int t0 = s.part * length, count = min(length, s.len - t0);
  bf16* const raw = reinterpret_cast<bf16*>(pool);  // [stage][u, delta, dy, z]
  float* const s_dt = pool + 2 * 4 * kBwdTile / 2;  // [token][channel] (dt, dt u)
  float* const s_g = s_dt + 2 * kBwdTile;           // [token][channel] y, then g
  float* const s_notes = s_g + kBwdTile;            // [warp][token / 4][channel of a lane][lane] states; then (to_b, r)
  float* const s_sums = s_notes + kBwdWarps * kNotes;  // [warp][token][dB, dC]
  float* const s_b = s_sums + kBwdWarps * kTile * 32;  // B, then C
  float* const s_note = s_notes + warp * kNotes;
  float* const s_sum = s_sums + warp * kTile * 32;

  wait_for_last_kernel();  // (behind the join where the sequences are cut)
  const int q = lane & 3, mine = lane >> 2, first = warp * kCh + mine * kC;
  const long long state_at = (static_cast<long long>(ch.c0) + first) * f.S + 4 * q;
  State4 decay[kC], X[kC], dA[kC], dA_rest[kC];
  bool real[kC];
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    real[j] = first + j < ch.have && 4 * q < f.S;
    decay[j] = X[j] = dA[j] = dA_rest[j] = zero4();
    if (real[j]) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(f.A + state_at + j * f.S));
      decay[j] = pack4(make_float4(v.x * kLog2e, v.y * kLog2e, v.z * kLog2e, v.w * kLog2e));
      const float* const from = cut ? ws.tails + part * all : a.d_state_out ? a.d_state_out + s.n * all : nullptr;
      if (from) X[j] = pack4(*reinterpret_cast<const float4*>(from + state_at + j * f.S));
    }
  }
  const bool wide = (f.D / f.G) % 8 == 0, gated = f.z != nullptr;
  const int last = count > 0 ? (count - 1) / kTile * kTile : -kTile;
  const long long row0 = s.start + t0 + max(last, 0);  // of the tile in hand, walking back
  RowStream<kBwdWarps> u(f.u, row0, f.ldu, ch, wide), delta(f.delta, row0, f.ldd, ch, wide), dy(a.dy, row0, a.lddy, ch, wide),
      z(gated ? f.z : f.u, row0, gated ? f.ldz : f.ldu, ch, wide);
  BcStream<kBwdWarps> bc(f.B, f.C, row0, f.ldb, f.ldc, ch, f.S);
  const float* tiles = f.tile_states + (tile_base(s) + (t0 + max(last, 0)) / kTile) * all + state_at;
  State4 next[kC];
  const auto fetch = [&](int tile, int stage) {
    if (tile >= 0) {
      const int n = count - tile;
      const uint32_t to = smem_u32(raw + stage * 4 * kBwdTile);
      u.fetch(to, n, wide), u.move(-1);
      delta.fetch(to + 2 * kBwdTile, n, wide), delta.move(-1);
      dy.fetch(to + 4 * kBwdTile, n, wide), dy.move(-1);
      if (gated) z.fetch(to + 6 * kBwdTile, n, wide), z.move(-1);
      bc.fetch(n), bc.move(-1);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        next[j] = zero4();
        if (real[j]) next[j] = pack4(*reinterpret_cast<const float4*>(tiles + j * f.S));
      }
      tiles -= all;
    }
    copies_commit();
  };
  const int four = 4 * (threadIdx.x % kBwdQuads), token = threadIdx.x / kBwdQuads;
  const bool four_real = four < ch.have;
  const Quad bias = weights_at(f.dt_bias, ch.c0 + four, four_real), skip = weights_at(f.skip, ch.c0 + four, four_real);
  Quad d_skip = zero_quad(), d_bias = zero_quad();
  const int four_at = token * kBwdRow + four;  // this thread's place in a tile
  bf16* dz = a.dz ? static_cast<bf16*>(a.dz) + (row0 + token) * a.lddz + ch.c0 + four : nullptr;
  bf16* du = static_cast<bf16*>(a.du) + (row0 + token) * a.lddu + ch.c0 + four;
  bf16* dd = static_cast<bf16*>(a.dd) + (row0 + token) * a.lddd + ch.c0 + four;
  fetch(last, 0);
  float* bc_sum = ws.bc_part + (static_cast<long long>(block) * f.T + row0) * 32;
  int stage = 0;
  for (int tile = last; tile >= 0; tile -= kTile, stage ^= 1) {
    const int n = min(kTile, count - tile);
    State4 h[kC] = {next[0], next[1]};
    bc.put(s_b);
    copies_done();
    __syncthreads();  // the tile is here, and nothing reads the one before it any more
    fetch(tile - kTile, stage ^ 1);
    const bf16* const now = raw + stage * 4 * kBwdTile + four_at;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = 8 * k * kBwdRow;
      const Quad v = quad_at(now + at);
      Quad x = add(quad_at(now + kBwdTile + at), bias);
      if (f.softplus) x = softplus(x);
      if (token + 8 * k >= n) x = zero_quad();
      put_pairs(s_dt + 2 * (four_at + at), x, mul(x, v));
    }
    __syncthreads();
    const uint32_t at_dt = after_sync(s_dt + 2 * first), at_b = after_sync(s_b + 4 * q), at_c = at_b + 4 * kTile * kBRow;
    // forward through the tile
#pragma unroll 2
    for (int t4 = 0; t4 < kTile; t4 += 4) {
#pragma unroll
      for (int j = 0; j < kC; ++j) *reinterpret_cast<float4*>(s_note + (t4 / 4 * kC + j) * 128 + 4 * lane) = unpack4(h[j]);
      float y[4][kC];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 d = lds4(at_dt + (t4 + i) * 8 * kBwdRow);
        const State4 b = pack4(lds4(at_b + (t4 + i) * 4 * kBRow));
        h[0] = fma4(decays(pack2(d.x, d.x), decay[0]), h[0], mul4(pack2(d.y, d.y), b));
        h[1] = fma4(decays(pack2(d.z, d.z), decay[1]), h[1], mul4(pack2(d.w, d.w), b));
        if (gated) {
          const State4 c = pack4(lds4(at_c + (t4 + i) * 4 * kBRow));
          y[i][0] = sum4(c, h[0]), y[i][1] = sum4(c, h[1]);
        }
      }
      if (gated) {
#pragma unroll
        for (int i = 0; i < 4; i += 2)
          s_g[(t4 + i + (q >> 1)) * kBwdRow + first + (q & 1)] = join4(y[i][0], y[i][1], y[i + 1][0], y[i + 1][1], q);
      }
    }
    if (gated) __syncthreads();
    // the gate's gradient; g
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = 8 * k * kBwdRow;
      const Quad v = quad_at(now + at);
      Quad g = quad_at(now + 2 * kBwdTile + at);
      if (gated) {
        const Quad zz = quad_at(now + 3 * kBwdTile + at), sg = sigmoid(zz), silu = mul(zz, sg);
        if (dz && token + 8 * k < n && four_real) {  // silu' = sg + silu (1 - sg)
          const Quad y = fma(skip, v, quad_at(s_g + four_at + at)), rest = fma(sg, quad(-1.0f, -1.0f, -1.0f, -1.0f), quad(1.0f, 1.0f, 1.0f, 1.0f));
          put_quad(dz + 8 * k * a.lddz, mul(mul(g, y), fma(silu, rest, sg)));
        }
        g = mul(g, silu);
      }
      *reinterpret_cast<float4*>(s_g + four_at + at) = floats(g);
      d_skip = fma(g, v, d_skip);
    }
    if (dz) dz -= kTile * a.lddz;
    __syncthreads();
    const uint32_t at_note = after_sync(s_note + 4 * lane), at_g = after_sync(s_g + first);
    State4 dA_tile[kC] = {zero4(), zero4()};
#pragma unroll 1
    for (int t4 = kTile - 4; t4 >= 0; t4 -= 4) {
      State4 hs[5][kC], es[4][kC], b[4];
      float4 d[4];
#pragma unroll
      for (int j = 0; j < kC; ++j) hs[0][j] = pack4(lds4(at_note + (t4 / 4 * kC + j) * 512));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i] = lds4(at_dt + (t4 + i) * 8 * kBwdRow);
        b[i] = pack4(lds4(at_b + (t4 + i) * 4 * kBRow));
        es[i][0] = decays(pack2(d[i].x, d[i].x), decay[0]);
        es[i][1] = decays(pack2(d[i].z, d[i].z), decay[1]);
        hs[i + 1][0] = fma4(es[i][0], hs[i][0], mul4(pack2(d[i].y, d[i].y), b[i]));
        hs[i + 1][1] = fma4(es[i][1], hs[i][1], mul4(pack2(d[i].w, d[i].w), b[i]));
      }
      float to_b[4][kC], r[4][kC];
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const float2 g = lds2(at_g + (t4 + i) * 4 * kBwdRow);
        const State4 c = pack4(lds4(at_c + (t4 + i) * 4 * kBRow));
        State4 sum_b = zero4(), sum_c = zero4();
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          const float gj = j ? g.y : g.x, dt = j ? d[i].z : d[i].x, dtu = j ? d[i].w : d[i].y;
          const f32x2 gg = pack2(gj, gj), uu = pack2(dtu, dtu);
          X[j] = fma4(gg, c, X[j]);
          sum_c = j ? fma4(gg, hs[i + 1][j], sum_c) : mul4(gg, hs[i + 1][j]);
          sum_b = j ? fma4(uu, X[j], sum_b) : mul4(uu, X[j]);
          to_b[i][j] = sum4(X[j], b[i]);
          X[j] = mul4(X[j], es[i][j]);
          const State4 qq = mul4(X[j], hs[i][j]);
          r[i][j] = sum4(decay[j], qq);
          dA_tile[j] = fma4(pack2(dt, dt), qq, dA_tile[j]);
        }
        const float4 dc = unpack4(sum_c), db = unpack4(sum_b);
        // eight values over the eight lanes of one q: lane (mine, q) ends with the sum of the mine-th
        const bool k4 = mine & 4, k2 = mine & 2, k1 = mine & 1;
        float v0 = (k4 ? dc.x : db.x) + __shfl_xor_sync(kAll, k4 ? db.x : dc.x, 16);
        float v1 = (k4 ? dc.y : db.y) + __shfl_xor_sync(kAll, k4 ? db.y : dc.y, 16);
        const float v2 = (k4 ? dc.z : db.z) + __shfl_xor_sync(kAll, k4 ? db.z : dc.z, 16);
        const float v3 = (k4 ? dc.w : db.w) + __shfl_xor_sync(kAll, k4 ? db.w : dc.w, 16);
        v0 = (k2 ? v2 : v0) + __shfl_xor_sync(kAll, k2 ? v0 : v2, 8);
        v1 = (k2 ? v3 : v1) + __shfl_xor_sync(kAll, k2 ? v1 : v3, 8);
        s_sum[(t4 + i) * 32 + (mine >> 2) * 16 + 4 * q + (mine & 3)] = (k1 ? v1 : v0) + __shfl_xor_sync(kAll, k1 ? v0 : v1, 4);
        // (to_b, r) [token][channel] over the noted states of these four tokens, which every lane has read by now
        s_note[t4 / 4 * kC * 128 + i * 2 * kCh + 2 * (mine * kC + (q & 1)) + (q >> 1)] =
            join4(to_b[i][0], to_b[i][1], r[i][0], r[i][1], q);
      }
    }
#pragma unroll
    for (int j = 0; j < kC; ++j) {  // dA: the tile's sum joins the others with what the addition before lost
      const f32x2 neg = pack2(-1.0f, -1.0f);
      const State4 add{fma2(dA_rest[j].a, neg, dA_tile[j].a), fma2(dA_rest[j].b, neg, dA_tile[j].b)};
      const State4 sum{add2(add.a, dA[j].a), add2(add.b, dA[j].b)};
      dA_rest[j] = State4{fma2(add.a, neg, fma2(dA[j].a, neg, sum.a)), fma2(add.b, neg, fma2(dA[j].b, neg, sum.b))};
      dA[j] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (token + 8 * k < n && four_real) {
        const int at = 8 * k * kBwdRow, t = token + 8 * k;
        Quad to_b, r, dt, dtu;
        get_pairs(s_notes + four / kCh * kNotes + t / 4 * kC * 128 + t % 4 * 2 * kCh + four % kCh * 2, to_b, r);
        get_pairs(s_dt + 2 * (four_at + at), dt, dtu);
        const Quad v = quad_at(now + at), g = quad_at(s_g + four_at + at);
        put_quad(du + 8 * k * a.lddu, fma(to_b, dt, mul(skip, g)));
        Quad e = fma(to_b, v, mul(r, quad(kLn2, kLn2, kLn2, kLn2)));
        if (f.softplus) e = mul(e, sigmoid(add(quad_at(now + kBwdTile + at), bias)));
        put_quad(dd + 8 * k * a.lddd, e);
        d_bias = add(d_bias, e);
      }
    }
    du -= kTile * a.lddu, dd -= kTile * a.lddd;
    // dB and dC over the warps
    for (int i = threadIdx.x; i < n * 32; i += kBwdWarps * 32) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kBwdWarps; ++w) sum += s_sums[w * kTile * 32 + i];
      bc_sum[i] = sum;
    }
    bc_sum -= kTile * 32;
  }
#pragma unroll
  for (int j = 0; j < kC; ++j)
    if (real[j]) {
      *reinterpret_cast<float4*>(ws.dA_part + part * all + state_at + j * f.S) = unpack4(dA[j]);
      if (a.d_state_in && s.part == 0) *reinterpret_cast<float4*>(a.d_state_in + s.n * all + state_at + j * f.S) = unpack4(X[j]);
    }
  // the eight threads that share four channels
  allow_next_kernel();
  __syncthreads();
  float4* const join = reinterpret_cast<float4*>(pool);
  join[2 * threadIdx.x] = floats(d_skip), join[2 * threadIdx.x + 1] = floats(d_bias);
  __syncthreads();
  if (threadIdx.x < kBwdQuads && four_real) {
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      d_skip = add(d_skip, quad(join[2 * (threadIdx.x + i * kBwdQuads)]));
      d_bias = add(d_bias, quad(join[2 * (threadIdx.x + i * kBwdQuads) + 1]));
    }
    float* const to = ws.d_part + static_cast<long long>(part) * f.D + ch.c0 + four;
    *reinterpret_cast<float4*>(to) = floats(d_skip);
    *reinterpret_cast<float4*>(to + static_cast<long long>(parts) * f.D) = floats(d_bias);
  }
}

// The gradient that a part hands to the one before it, from zero at its end, and the sum of its dt.
__global__ void __launch_bounds__(kFwdWarps * 32, 4) scan_bwd_sums_kernel(ScanBwdArgs a, int blocks, int length, float* sums, float* dt_sums) {
  extern __shared__ float pool[];
  const ScanArgs& f = a.f;
  const int warp = threadIdx.x >> 5, lane = static_cast<int>(lane_id());
  const int part = blockIdx.x / blocks;
  SeqPart s;
  if (!find_part(f.cu, f.N, f.T, f.max_seqlen, length, part, s, nullptr) || s.part == 0) return;  // (nothing comes before a first part)
  const Channels ch = block_channels(blockIdx.x % blocks, f.D, f.G, kFwdRow);
  const int t0 = s.part * length, count = min(length, s.len - t0);
  bf16* const raw = reinterpret_cast<bf16*>(pool);  // [stage][delta, dy, z]
  allow_next_kernel();
  float* const s_dt = pool + 2 * 3 * kFwdTile / 2;  // [token][channel] (dt, g)
  float* const s_bc = s_dt + 2 * kFwdTile;          // [stage][nothing, C]
  const int q = lane & 3, first = warp * kCh + (lane >> 2) * kC;
  const long long all = static_cast<long long>(f.D) * f.S;
  const long long state_at = (static_cast<long long>(ch.c0) + first) * f.S + 4 * q;
  State4 decay[kC], X[kC];
  float dt_sum[kC] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    decay[j] = X[j] = zero4();
    if (first + j < ch.have && 4 * q < f.S) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(f.A + state_at + j * f.S));
      decay[j] = pack4(make_float4(v.x * kLog2e, v.y * kLog2e, v.z * kLog2e, v.w * kLog2e));
    }
  }
  const bool wide = (f.D / f.G) % 8 == 0, gated = f.z != nullptr;
  const int last = (count - 1) / kTile * kTile;
  const long long row0 = s.start + t0 + last;
  RowStream<kFwdWarps> delta(f.delta, row0, f.ldd, ch, wide), dy(a.dy, row0, a.lddy, ch, wide),
      z(gated ? f.z : f.delta, row0, gated ? f.ldz : f.ldd, ch, wide);
  BcStream<kFwdWarps> bc(nullptr, f.C, row0, f.ldb, f.ldc, ch, f.S);
  const auto fetch = [&](int tile, int stage) {
    if (tile >= 0) {
      const int n = count - tile;
      const uint32_t to = smem_u32(raw + stage * 3 * kFwdTile);
      delta.fetch(to, n, wide), delta.move(-1);
      dy.fetch(to + 2 * kFwdTile, n, wide), dy.move(-1);
      if (gated) z.fetch(to + 4 * kFwdTile, n, wide), z.move(-1);
      bc.fetch(n), bc.move(-1);
    }
    copies_commit();
  };
  const int four = 4 * (threadIdx.x % kFwdQuads), token = threadIdx.x / kFwdQuads;
  const Quad bias = weights_at(f.dt_bias, ch.c0 + four, four < ch.have);
  fetch(last, 0);
  int stage = 0;
  for (int tile = last; tile >= 0; tile -= kTile, stage ^= 1) {
    const int n = min(kTile, count - tile);
    float* const s_b = s_bc + stage * 2 * kTile * kBRow;
    bc.put(s_b);
    copies_done();
    __syncthreads();  // the tile is here, and nothing reads the one before it any more
    fetch(tile - kTile, stage ^ 1);
    const bf16* const now = raw + stage * 3 * kFwdTile + token * kFwdRow + four;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = 8 * k * kFwdRow;
      Quad g = quad_at(now + kFwdTile + at), x = add(quad_at(now + at), bias);
      if (f.softplus) x = softplus(x);
      if (token + 8 * k >= n) x = zero_quad();
      if (gated) {
        const Quad zz = quad_at(now + 2 * kFwdTile + at);
        g = mul(g, mul(zz, sigmoid(zz)));
      }
      put_pairs(s_dt + 2 * (at + token * kFwdRow + four), x, g);
    }
    __syncthreads();
    const uint32_t at_dt = after_sync(s_dt + 2 * first), at_c = after_sync(s_b + kTile * kBRow + 4 * q);
#pragma unroll 8
    for (int t = kTile - 1; t >= 0; --t) {
      const float4 d = lds4(at_dt + t * 8 * kFwdRow);
      const State4 c = pack4(lds4(at_c + t * 4 * kBRow));
      X[0] = mul4(fma4(pack2(d.y, d.y), c, X[0]), decays(pack2(d.x, d.x), decay[0]));
      X[1] = mul4(fma4(pack2(d.w, d.w), c, X[1]), decays(pack2(d.z, d.z), decay[1]));
      dt_sum[0] += d.x, dt_sum[1] += d.z;
    }
  }
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    if (first + j >= ch.have) continue;
    if (4 * q < f.S) *reinterpret_cast<float4*>(sums + part * all + state_at + j * f.S) = unpack4(X[j]);
    if (q == 0) dt_sums[static_cast<long long>(part) * f.D + ch.c0 + first + j] = dt_sum[j];
  }
}

// What is left to add up, in one launch, always in one order. dB and dC [T][G][S] (bf16) from the channel blocks' sums
// [blocks][T][32]: a CTA has eight tokens of a sequence and 64 pieces of four values, each the sum of four threads' shares of the
// blocks. dA, dskip and d_dt_bias from the parts' sums: a CTA has 32 columns, eight warps share the parts.
__global__ void __launch_bounds__(256) scan_tail_kernel(ScanBwdArgs a, BwdWs ws, int blocks, int parts, int bc_ctas) {
  __shared__ float4 share[4][64];
  wait_for_last_kernel();
  const ScanArgs& f = a.f;
  if (static_cast<int>(blockIdx.x) < bc_ctas) {
    SeqPart s;
    if (!find_part(f.cu, f.N, f.T, f.max_seqlen, 8, blockIdx.x, s, nullptr)) return;
    const int piece = threadIdx.x & 63, quarter = threadIdx.x >> 6, value = piece & 7, state = 4 * (value & 3);
    const int at = s.part * 8 + (piece >> 3);
    const bool real = at < s.len && state < f.S;
    const long long t = s.start + at;
    const int per = blocks / f.G;
    for (int g = 0; g < f.G; ++g) {
      float4 sum = make_float4(0, 0, 0, 0);
      if (real) {
#pragma unroll 4
        for (int b = g * per + quarter; b < (g + 1) * per; b += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(ws.bc_part + (static_cast<long long>(b) * f.T + t) * 32 + 4 * value));
          sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
      }
      share[quarter][piece] = sum;
      __syncthreads();
      if (quarter == 0 && real) {
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          const float4 v = share[i][piece];
          sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        bf16* const to = static_cast<bf16*>(value < 4 ? a.dB : a.dC) + (t * f.G + g) * f.S + state;
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
      }
      __syncthreads();
    }
    return;
  }
  // columns: dA's, then dskip's, then d_dt_bias'
  const long long all = static_cast<long long>(f.D) * f.S;
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const long long c = (static_cast<long long>(blockIdx.x) - bc_ctas) * 32 + lane;
  const float* from = ws.dA_part + c;
  float* to = a.dA + c;
  long long ld = all;
  if (c >= all) {
    const long long i = c - all;
    const bool second = i >= f.D;
    from = ws.d_part + (second ? static_cast<long long>(parts) * f.D : 0) + (second ? i - f.D : i), ld = f.D;
    float* const base = second ? a.d_dt_bias : a.dskip;
    to = base && i < 2ll * f.D ? base + (second ? i - f.D : i) : nullptr;
  }
  float sum = 0.0f;
  if (to) {
#pragma unroll 4
    for (int p = g; p < parts; p += 8) sum += __ldg(from + p * ld);
  }
  float* const sums = reinterpret_cast<float*>(share);
  sums[g * 32 + lane] = sum;
  __syncthreads();
  if (g == 0 && to) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += sums[i * 32 + lane];
    *to = sum;
  }
}

// ------------------------------------------------------------------ step

constexpr int kStepWarps = 4;

// One token for each of four rows: a lane has four states of a channel in each, whose loads are under way together, and reads
// A once for all of them. Time step, gate and output of a row are the work of one of the four lanes that share a channel.
// 61 rows x 8,192 channels x 16 states in 14.5 us, 9.4 of them the states' bytes; the rest is arithmetic (some 520 instructions a warp).
// A row a CTA: 24 us; eight warps a CTA 15.4.
__global__ void __launch_bounds__(kStepWarps * 32) scan_step_kernel(ScanStepArgs a, int per) {
  constexpr int kRows = 4;
  const int lane = static_cast<int>(lane_id()), q = lane & 3;
  // grid: rows x groups, a group's channels (`per` of them); a division only where there are groups
  const int part = a.G > 1 ? blockIdx.x / a.G : blockIdx.x, group = blockIdx.x - part * a.G;
  const int at = blockIdx.y * 8 * kStepWarps + static_cast<int>(threadIdx.x >> 2), c = group * per + at, b0 = part * kRows;
  const bool in = at < per, real = in && 4 * q < a.S;
  wait_for_last_kernel();
  float4 A = make_float4(0, 0, 0, 0);
  if (real) A = __ldg(reinterpret_cast<const float4*>(a.A + static_cast<long long>(c) * a.S + 4 * q));
  const float bias = a.dt_bias && in ? __ldg(a.dt_bias + c) : 0.0f, skip = a.skip && in ? __ldg(a.skip + c) : 0.0f;
  const int rows = min(kRows, a.B_rows - b0);
  int slot[kRows];  // -1: an empty row
#pragma unroll
  for (int r = 0; r < kRows; ++r) slot[r] = r >= rows ? -1 : a.state_idx ? __ldg(a.state_idx + b0 + r) : b0 + r;
  const long long row_states = static_cast<long long>(a.D) * a.S;
  float* const states = a.state + static_cast<long long>(c) * a.S + 4 * q;
  const bf16* const Bs = static_cast<const bf16*>(a.B) + b0 * a.ldb + group * a.S + 4 * q;
  const bf16* const Cs = static_cast<const bf16*>(a.C) + b0 * a.ldc + group * a.S + 4 * q;
  float4 h[kRows];
  uint2 Bv[kRows], Cv[kRows];
  bool own = false;  // whether this lane's row, b0 + q, is no empty one
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (slot[r] >= a.n_slots) {
      if (threadIdx.x == 0) set_flag(a.err_flag, MOE_FLAG_BAD_INDEX);
      slot[r] = -1;
    }
    if (r == q) own = slot[r] >= 0;
    h[r] = make_float4(0, 0, 0, 0);
    Bv[r] = Cv[r] = make_uint2(0, 0);
    if (!real) slot[r] = -1;
    if (slot[r] < 0) continue;
    h[r] = *reinterpret_cast<const float4*>(states + slot[r] * row_states);
    Bv[r] = *reinterpret_cast<const uint2*>(Bs + r * a.ldb);
    Cv[r] = *reinterpret_cast<const uint2*>(Cs + r * a.ldc);
  }
  const long long row = b0 + q;
  float u = 0.0f, dt = 0.0f, z = 0.0f;
  if (own && in) {
    u = __bfloat162float(static_cast<const bf16*>(a.u)[row * a.ldu + c]);
    dt = __bfloat162float(static_cast<const bf16*>(a.delta)[row * a.ldd + c]) + bias;
    if (a.z) z = __bfloat162float(static_cast<const bf16*>(a.z)[row * a.ldz + c]);
  }
  if (a.softplus) dt = softplus(dt);
  const float step = dt * kLog2e, du = dt * u;
  float o[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float k = __shfl_sync(kAll, step, (lane & ~3) | r), d = __shfl_sync(kAll, du, (lane & ~3) | r);
    h[r].x = fmaf(ex2(fmaf(k, A.x, kRaise)), h[r].x, d * bf16_lo(Bv[r].x));
    h[r].y = fmaf(ex2(fmaf(k, A.y, kRaise)), h[r].y, d * bf16_hi(Bv[r].x));
    h[r].z = fmaf(ex2(fmaf(k, A.z, kRaise)), h[r].z, d * bf16_lo(Bv[r].y));
    h[r].w = fmaf(ex2(fmaf(k, A.w, kRaise)), h[r].w, d * bf16_hi(Bv[r].y));
    if (slot[r] >= 0) *reinterpret_cast<float4*>(states + slot[r] * row_states) = h[r];
    o[r] = fmaf(bf16_lo(Cv[r].x), h[r].x, bf16_hi(Cv[r].x) * h[r].y) + fmaf(bf16_lo(Cv[r].y), h[r].z, bf16_hi(Cv[r].y) * h[r].w);
  }
  float y = join4(o[0], o[1], o[2], o[3], q);
  if (!in || row >= a.B_rows) return;
  y = fmaf(skip, u, y);
  if (a.z) y *= z * rcp(1.0f + ex2(-z * kLog2e));
  static_cast<bf16*>(a.y)[row * a.ldy + c] = __float2bfloat16_rn(own ? y : 0.0f);
}

// Channel blocks of `channels` channels.
int blocks_of(int D, int G, int channels) { return G * ((D / G + channels - 1) / channels); }
size_t up256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

// How a launch is divided: channel blocks, tokens of a part.
struct Division {
  int blocks, length;
  long long parts;
  bool cut;
};

// Cutting the sequences gives more CTAs but costs a second run over all parts but the last ones (the sums), so the
// cheapest of some lengths is taken by an estimate from measured costs (nanoseconds; blocks of 64 channels in the forward and the
// sums, of 128 in the backward). A CTA's chain of one token takes 150 in the forward and 140 in the sums, and a token of a block
// 0.30 and 0.21 of the whole GPU's time; the larger of the two rules, and where they are near one another both count (fourth
// powers). A backward CTA has an SM alone: 410 a token, in whole rounds. The launches and the join take 8 us and 0.5 us a part in a
// row. The lengths are known by their bound and sum alone: the last parts are taken for half full. (7,864 tokens of prompts of 1 to 4,096 tokens
// x 8,192 channels: 625 us in one piece, 541 in parts of 1,024, 485 of 512, 517 of 256.)
Division divide(int max_seqlen, int T, int N, int D, int G, bool backward) {
  Division d;
  d.blocks = blocks_of(D, G, kCh * (backward ? kBwdWarps : kFwdWarps));
  const double sms = num_sms(), fwd_blocks = blocks_of(D, G, kCh * kFwdWarps);
  long long whole = max_seqlen > 0 ? (static_cast<long long>(max_seqlen) + kTile - 1) / kTile * kTile : kTile;
  if (whole > 0x7FFFFFE0) whole = 0x7FFFFFE0;
  // (a bound above T says no more than T does)
  const long long longest = whole < T ? whole : (static_cast<long long>(T) + kTile - 1) / kTile * kTile + kTile;
  const auto both = [](double x, double y) { return std::sqrt(std::sqrt(x * x * x * x + y * y * y * y)); };
  const auto cost = [&](long long length, int pieces) {
    const double tokens = static_cast<double>(length), rest = std::max(0.0, T - 0.5 * N * tokens), share = fwd_blocks * 152.0 / sms;
    double ns = backward ? std::ceil(std::max(1.0, T / tokens) * d.blocks / sms) * tokens * 410.0
                         : both(tokens * 150.0, T * share * 0.30);
    if (pieces > 1) ns += both(tokens * 140.0, rest * share * 0.21) + 8000.0 + 500.0 * pieces;
    return ns;
  };
  long long best = whole;
  double least = cost(longest, 1);
  for (int pieces : {2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 20, 24, 32, 48, 64, 96, 128}) {
    const long long length = (longest / kTile + pieces - 1) / pieces * kTile;
    if (length < 64) break;
    const double ns = cost(length, pieces);
    if (ns < 0.95 * least) least = ns, best = length;
  }
  d.length = static_cast<int>(best);
  d.parts = T / d.length + static_cast<long long>(N);
  d.cut = max_seqlen > d.length;
  return d;
}

// A kernel's dynamic shared memory, allowed once a device.
template <auto KERNEL>
cudaError_t prepare_kernel(int smem) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && ready[dev].load())) return e;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) ready[dev].store(true);
  return e;
}

}  // namespace

size_t scan_tile_states_bytes(int T, int N, int D, int S) {
  return up256((static_cast<size_t>(T) / kTile + N) * D * S * 4);
}

size_t scan_workspace(int max_seqlen, int T, int N, int D, int S, int G, bool backward) {
  const Division d = divide(max_seqlen, T, N, D, G, backward);
  const size_t parts = static_cast<size_t>(d.parts), all = static_cast<size_t>(D) * S;
  size_t bytes = d.cut ? up256(parts * all * 4) + up256(parts * D * 4) : 0;
  if (backward) bytes += up256(static_cast<size_t>(d.blocks) * T * 32 * 4) + up256(parts * all * 4) + up256(2 * parts * D * 4);
  return bytes;
}

template <bool FEW>
static cudaError_t scan_fwd(const ScanArgs& a, cudaStream_t st) {
  const Division d = divide(a.max_seqlen, a.T, a.N, a.D, a.G, false);
  const unsigned grid = static_cast<unsigned>(d.parts * d.blocks);
  const int smem = kFwdSmem;
  cudaError_t e = prepare_kernel<scan_fwd_kernel<false, FEW>>(smem);
  if (e != cudaSuccess) return e;
  float* starts = nullptr;
  if (d.cut) {
    starts = a.ws;
    float* const dt_sums = reinterpret_cast<float*>(reinterpret_cast<char*>(a.ws) + up256(static_cast<size_t>(d.parts) * a.D * a.S * 4));
    e = prepare_kernel<scan_fwd_kernel<true, FEW>>(smem);
    if (e != cudaSuccess) return e;
    {
      LaunchTimer lt("scan_fwd_sums", st);
      scan_fwd_kernel<true, FEW><<<grid, kFwdWarps * 32, smem, st>>>(a, d.blocks, d.length, nullptr, starts, dt_sums);
    }
    LaunchTimer lt("scan_join", st);
    const unsigned join = static_cast<unsigned>(d.parts * ((a.D * (a.S / 4) + 127) / 128));
    e = launch_behind(scan_join_kernel<false>, dim3(join), 128, 0, st, a, d.length, a.state_in, starts, static_cast<const float*>(dt_sums));
    if (e != cudaSuccess) return e;
  }
  LaunchTimer lt("scan_fwd", st);
  if (d.cut)
    return launch_behind(scan_fwd_kernel<false, FEW>, dim3(grid), kFwdWarps * 32, smem, st, a, d.blocks, d.length,
                         static_cast<const float*>(starts), static_cast<float*>(nullptr), static_cast<float*>(nullptr));
  scan_fwd_kernel<false, FEW><<<grid, kFwdWarps * 32, smem, st>>>(a, d.blocks, d.length, nullptr, nullptr, nullptr);
  return cudaGetLastError();
}

static bool few(const ScanArgs& a) { return a.cu == nullptr || a.N < kWalk; }

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t st) { return few(a) ? scan_fwd<true>(a, st) : scan_fwd<false>(a, st); }

cudaError_t launch_scan_bwd(const ScanBwdArgs& a, cudaStream_t st) {
  const ScanArgs& f = a.f;
  const Division d = divide(f.max_seqlen, f.T, f.N, f.D, f.G, true);
  const size_t all = static_cast<size_t>(f.D) * f.S;
  char* at = reinterpret_cast<char*>(f.ws);
  const auto take = [&](size_t bytes) {
    float* const p = reinterpret_cast<float*>(at);
    at += up256(bytes);
    return p;
  };
  BwdWs ws{};
  float* dt_sums = nullptr;
  if (d.cut) ws.tails = take(d.parts * all * 4), dt_sums = take(d.parts * static_cast<size_t>(f.D) * 4);
  ws.bc_part = take(static_cast<size_t>(d.blocks) * f.T * 32 * 4);
  ws.dA_part = take(d.parts * all * 4);
  ws.d_part = take(2 * d.parts * static_cast<size_t>(f.D) * 4);
  const bool is_few = few(f);
  cudaError_t e = is_few ? prepare_kernel<scan_bwd_kernel<true>>(kBwdSmem) : prepare_kernel<scan_bwd_kernel<false>>(kBwdSmem);
  if (e != cudaSuccess) return e;
  if (d.cut) {
    const int b = blocks_of(f.D, f.G, kCh * kFwdWarps), smem = kFwdSmem;
    e = prepare_kernel<scan_bwd_sums_kernel>(smem);
    if (e != cudaSuccess) return e;
    {
      LaunchTimer lt("scan_bwd_sums", st);
      scan_bwd_sums_kernel<<<static_cast<unsigned>(d.parts * b), kFwdWarps * 32, smem, st>>>(a, b, d.length, ws.tails, dt_sums);
    }
    LaunchTimer lt("scan_join", st);
    const unsigned join = static_cast<unsigned>(d.parts * ((f.D * (f.S / 4) + 127) / 128));
    e = launch_behind(scan_join_kernel<true>, dim3(join), 128, 0, st, f, d.length, a.d_state_out, ws.tails, static_cast<const float*>(dt_sums));
    if (e != cudaSuccess) return e;
  }
  {
    LaunchTimer lt("scan_bwd", st);
    const unsigned grid = static_cast<unsigned>(d.parts * d.blocks);
    const int parts = static_cast<int>(d.parts);
    const auto kernel = is_few ? scan_bwd_kernel<true> : scan_bwd_kernel<false>;
    if (d.cut) e = launch_behind(kernel, dim3(grid), kBwdWarps * 32, kBwdSmem, st, a, d.blocks, parts, d.length, true, ws);
    else kernel<<<grid, kBwdWarps * 32, kBwdSmem, st>>>(a, d.blocks, parts, d.length, false, ws);
    if (e != cudaSuccess) return e;
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  LaunchTimer lt("scan_tail", st);
  const long long bc_ctas = f.T / 8 + static_cast<long long>(f.N), columns = static_cast<long long>(all) + 2ll * f.D;
  return launch_behind(scan_tail_kernel, dim3(static_cast<unsigned>(bc_ctas + (columns + 31) / 32)), 256, 0, st, a, ws, d.blocks,
                       static_cast<int>(d.parts), static_cast<int>(bc_ctas));
}

cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t st) {
  LaunchTimer lt("scan_step", st);
  const int per = a.D / a.G;
  const dim3 grid((static_cast<unsigned>(a.B_rows) + 3) / 4 * a.G, (per + 8 * kStepWarps - 1) / (8 * kStepWarps));
  return launch_behind(scan_step_kernel, grid, kStepWarps * 32, 0, st, a, per);
}

}  // namespace moe
