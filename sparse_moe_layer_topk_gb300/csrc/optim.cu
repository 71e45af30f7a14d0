// AdamW over many tensors in one launch, states in 32 or 8 bits, with the global
// gradient norm in a launch before it when the step is clipped.
//
//   g' = c g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Nothing is reused, so the 32-bit step is bound by HBM: p, m, v in and out and g in. Each warp takes
// runs of blocks of 256 values (a prefix of the tensors' chunk counts, searched where a run enters a
// tensor, says whose), eight consecutive values a lane: 32-byte loads and stores of fp32, 16-byte of
// bf16, 8-byte of codes. A block is also what shares a scale in the 8-bit states: its largest magnitude
// is one warp reduction. The 8-bit step moves 10 bytes a value (bf16 weights and gradients) with 73
// instructions, which weigh more than its bytes: arithmetic runs two values to an instruction, and
// types are told apart once a run. The 8-bit forms spill 24 - 76 bytes a thread at the 64 registers that four
// CTAs an SM allow.
// Measured (67 M values, no clip, in a graph): 32-bit states, bf16 weights with a master copy, fp32 gradients
// 321 us, 6.3 TB/s (0.92 of a plain copy's rate); 8-bit states, bf16 weights and gradients 177 us, 3.8 TB/s,
// issue slots 73% taken; 8-bit states, bf16 weights with a master copy, fp32 gradients 218 us, 5.5 TB/s.

#include "common.cuh"
#include "optim.h"
#include "timing.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPerLane = 8;
constexpr int kBlock = 32 * kPerLane;  // values of one warp, and of one 8-bit block
constexpr int kChunkBlocks = kAdamwChunk / kBlock;
static_assert(kAdamwChunk % kBlock == 0, "chunk");
static_assert(kBlock == kAdamwBlock, "block");

// ------------------------------------------------------------------ random numbers

// Counter hash: two rounds of xor-shift and odd multiplication. Every output bit
// flips with a probability between 0.47 and 0.54 when one input bit does.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x45D9F3B5u;
  x ^= x >> 15;
  x *= 0x2F7D9D4Bu;
  return x ^ (x >> 16);
}

// ------------------------------------------------------------------ loads and stores

// Eight values as they lie in memory: 8 words of fp32, 4 of bf16 pairs or 2 of E4M3 codes; `n` of
// them exist, the others are zeros. `whole`: all eight, aligned for one access.
__device__ __forceinline__ void load_raw(const char* at, int n, bool whole, uint32_t (&r)[8]) {
  if (whole) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7])
                 : "l"(at));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = i < n ? reinterpret_cast<const uint32_t*>(at)[i] : 0u;
  }
}

__device__ __forceinline__ void load_raw(const char* at, int n, bool whole, uint32_t (&r)[4]) {
  if (whole) {
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "l"(at));
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = (2 * i < n ? p[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(p[2 * i + 1]) << 16 : 0u);
  }
}

__device__ __forceinline__ void load_raw(const char* at, int n, bool whole, uint32_t (&r)[2]) {
  if (whole) {
    asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(at));
  } else {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(at);
    r[0] = r[1] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) r[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  }
}

__device__ __forceinline__ void to_f32(const uint32_t (&r)[8], f32x2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

__device__ __forceinline__ void to_f32(const uint32_t (&r)[4], f32x2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(bf16_lo(r[i]), bf16_hi(r[i]));
}

__device__ __forceinline__ void store8_f32(char* at, int n, bool whole, const f32x2 (&x)[4]) {
  float* p = reinterpret_cast<float*>(at);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(x[i], v[2 * i], v[2 * i + 1]);
  if (whole) {
    store_f32x8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

// Four words of bf16 pairs.
__device__ __forceinline__ void store8_b16(char* at, int n, bool whole, const uint32_t (&w)[4]) {
  uint16_t* p = reinterpret_cast<uint16_t*>(at);
  if (whole) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}

__device__ __forceinline__ void store8_codes(char* at, int n, bool whole, uint2 c) {
  uint8_t* p = reinterpret_cast<uint8_t*>(at);
  if (whole) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// ------------------------------------------------------------------ 8-bit states

__device__ __forceinline__ void decode8(uint2 c, float scale, f32x2 (&v)[4]) {
  float x[8];
  e4m3x4_to_f32(c.x, x);
  e4m3x4_to_f32(c.y, x + 4);
  const f32x2 s = pack2(scale, scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul2(pack2(x[2 * i], x[2 * i + 1]), s);
}

// Eight values of a warp's 256-value block as E4M3 codes and the block's scale,
// the largest finite magnitude / 448. Times 2^-120 an E4M3 value's bits are those
// of the fp32 with the code in bits 20..26, subnormals included, so adding a
// random number below 2^20 and cutting rounds up with a probability equal to
// the part cut off (nearest rounding would freeze v: at b2 = 0.999 it moves by
// less than half a step). The random number has 16 bits, and the largest value falls within a few
// units of 448, so the sum stays below the next code. A non-finite value gets the NaN code; that
// there is one in the block is seen from `check`, the sum of 0 times every value.
// HIGH: the random numbers are the upper halves of rand (else the lower ones), and the values have no sign.
template <bool HIGH>
__device__ __forceinline__ uint2 encode8(const f32x2 (&x)[4], const uint32_t (&rand)[8], float& scale) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(x[i], v[2 * i], v[2 * i + 1]);
  const f32x2 zero = pack2(0.0f, 0.0f);
  f32x2 check = zero;
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) check = fma2(x[i], zero, check);
#pragma unroll
  for (int i = 0; i < 8; i += 2) top = fmaxf(fmaxf(top, fabsf(v[i])), fabsf(v[i + 1]));
  float c0, c1;
  unpack2(check, c0, c1);
  const bool bad = __any_sync(0xFFFFFFFFu, !(c0 + c1 == 0.0f));
  if (bad) {
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]) < INFINITY ? fabsf(v[i]) : 0.0f);
  }
  // (magnitudes order as their bits)
  top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));
  // below 2^-100 a block counts as zero (448 / top would overflow)
  const float inv = top > 7.8886e-31f ? __fmul_rn(__frcp_rn(top), 448.0f) : 0.0f;
  scale = top * (1.0f / 448.0f);
  const f32x2 inv2 = pack2(inv, inv), down = pack2(0x1p-120f, 0x1p-120f);
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float y[2];
    unpack2(mul2(mul2(x[i / 2], inv2), down), y[0], y[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // the code moves to the top byte (the sign stays above it); 16 x the random half is added in one
      // instruction
      const uint32_t t = __dp2a_lo(rand[i + k], HIGH ? 0x1000u : 0x10u, __float_as_uint(y[k]));
      u[i + k] = HIGH ? t * 16u : ((t * 16u) & 0x7FFFFFFFu) | (t & 0x80000000u);
    }
  }
  if (bad) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(fabsf(v[i]) < INFINITY)) u[i] = 0x7F000000u;
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __byte_perm(__byte_perm(u[4 * i], u[4 * i + 1], 0x0073), __byte_perm(u[4 * i + 2], u[4 * i + 3], 0x0073), 0x5410);
  return make_uint2(w[0], w[1]);
}

// Square roots by one Newton step (in Markstein's form: the residual of the product from a fused
// multiply-add) on the hardware's reciprocal root; 0 for 0. Equal to the IEEE root for all but a
// few in a million values above 1e-36.
__device__ __forceinline__ f32x2 sqrt2(f32x2 v) {
  float a, b;
  unpack2(fma2(v, pack2(1.0f, 1.0f), pack2(1e-38f, 1e-38f)), a, b);  // (keeps the root of 0 finite)
  float ra, rb;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(ra) : "f"(a));
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(rb) : "f"(b));
  const f32x2 y = pack2(ra, rb);
  const f32x2 g = mul2(v, y);
  const f32x2 d = fma2(mul2(g, pack2(-1.0f, -1.0f)), g, v);
  return fma2(d, mul2(y, pack2(0.5f, 0.5f)), g);
}

// The root where v is finite: sqrt2 makes NaN of an infinite v, which a finite gradient above 1.8e19 /
// sqrt(1 - b2) leaves, and the weight would be lost. (8-bit states hold no infinity and lose the value anyway.)
__device__ __forceinline__ f32x2 root_or_inf(f32x2 v, f32x2 root) {
  float a, b, ra, rb;
  unpack2(v, a, b);
  unpack2(root, ra, rb);
  return pack2(a == INFINITY ? a : ra, b == INFINITY ? b : rb);
}

// ------------------------------------------------------------------ the chunk's tensor

__device__ __forceinline__ int find_tensor(const AdamwEntry* e, int n, long long chunk) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(&e[mid].chunk0) <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ gradient norm

constexpr int kNormRun = 4;  // blocks that a warp loads at a time
static_assert(kChunkBlocks % kNormRun == 0, "a run lies in one tensor");

// Sum of the squares of kNormRun blocks of a gradient from byte `at` (the lane's first) on; `left` values of
// the tensor are there from the lane's first on. A lane's 32 squares are summed in fp32, in fp64 where
// one of them is past fp32 (the sum is then infinite, or NaN).
template <int BYTES>
__device__ __forceinline__ double sum_squares(const char* at, long long left, bool vec) {
  uint32_t raw[kNormRun][2 * BYTES];
#pragma unroll
  for (int u = 0; u < kNormRun; ++u) {
    const long long here = left - u * kBlock;
    const int n = here > 0 ? static_cast<int>(here < 8 ? here : 8) : 0;
    load_raw(at + u * kBlock * BYTES, n, vec && n == 8, raw[u]);
  }
  f32x2 acc[4] = {{0}, {0}, {0}, {0}};
#pragma unroll
  for (int u = 0; u < kNormRun; ++u) {
    f32x2 g[4];
    to_f32(raw[u], g);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fma2(g[i], g[i], acc[i]);
  }
  float x, y, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unpack2(acc[i], x, y);
    sum += x + y;
  }
  if (sum < INFINITY) return sum;
  double exact = 0.0;
#pragma unroll
  for (int u = 0; u < kNormRun; ++u) {
    f32x2 g[4];
    to_f32(raw[u], g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unpack2(g[i], x, y);
      exact += static_cast<double>(x) * x + static_cast<double>(y) * y;
    }
  }
  return exact;
}

// Sum of squares of all gradients, from the first to the last, each warp a run of blocks in turn. Each CTA
// writes one partial; the last one to finish adds them in a fixed order, so the norm does not depend
// on timing. Four blocks a warp are loaded at once, and a small step has few CTAs, whose tickets and partials
// are its time: a clipped step of 1 M values in a graph 11.9 us, with two blocks and a CTA a chunk 17.0.
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const AdamwEntry* entries, int n_tensors, long long chunks, float max_norm, double* partial,
                     AdamwControl* ctl) {
  allow_next_kernel();
  double s = 0.0;
  const long long blocks = chunks * kChunkBlocks, step = static_cast<long long>(gridDim.x) * (kThreads / 32) * kNormRun;
  for (long long from = (static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kNormRun;
       from < blocks; from += step) {
    // (a tensor's blocks are a multiple of a run's: a run lies in one)
    const AdamwEntry& e = entries[find_tensor(entries, n_tensors, from / kChunkBlocks)];
    const long long at = (from - e.chunk0 * kChunkBlocks) * kBlock + (threadIdx.x & 31) * kPerLane;
    if (e.g_dtype == MOE_DTYPE_F32) s += sum_squares<4>(static_cast<const char*>(e.g) + at * 4, e.n - at, e.vec);
    else s += sum_squares<2>(static_cast<const char*>(e.g) + at * 2, e.n - at, e.vec);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  __shared__ double warp_sum[kThreads / 32];
  __shared__ bool last;
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) s += warp_sum[i];
    partial[blockIdx.x] = s;
    __threadfence();
    last = atomicAdd(&ctl->norm_ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  s = 0.0;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kThreads)
    s += *static_cast<volatile double*>(partial + i);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) s += warp_sum[i];
    const float norm = static_cast<float>(__dsqrt_rn(s));
    ctl->grad_norm = norm;
    ctl->clip = fminf(1.0f, max_norm / (norm + 1e-6f));
    ctl->skip = norm < INFINITY ? 0 : 1;
    ctl->norm_ticket = 0;
  }
}

// ------------------------------------------------------------------ step

struct StepConsts {
  float clip, lr, step_size, inv_sqrt_bc2, b1, b2, rate1, rate2, eps;
  uint32_t key;
  int skip;
};

// The sum of two products, each rounded by itself: which E4M3 neighbour a value gets then follows from
// the formula alone, not from how a compiler pairs products with sums (ptxas fuses a packed product
// with a packed sum, rounding modes or not).
__device__ __forceinline__ f32x2 sum2(f32x2 x, f32x2 y) {
  float a, b, c, d;
  unpack2(x, a, b);
  unpack2(y, c, d);
  return pack2(__fadd_rn(a, c), __fadd_rn(b, d));
}

// Weight types: fp32, bf16, bf16 with an fp32 master copy (which is then what is read).
enum WeightKind { W_F32 = 0, W_BF16 = 1, W_MASTER = 2 };

// Where a lane's eight values of a block lie in a tensor's arrays.
template <bool Q8, int W, bool GB>
struct Place {
  static constexpr int GS = GB ? 2 : 4, PS = W == W_BF16 ? 2 : 4, SS = Q8 ? 1 : 4;  // bytes a value
  const char* g;
  char *p, *m, *v, *copy;  // copy: the bf16 weights beside a master copy
  float *m_scale, *v_scale;
  int left;  // values of the tensor from here on (or 2^30)

  __device__ __forceinline__ Place(const AdamwEntry& e, long long at) {
    g = static_cast<const char*>(e.g) + at * GS;
    p = (W == W_MASTER ? reinterpret_cast<char*>(e.master) : static_cast<char*>(e.p)) + at * PS;
    m = static_cast<char*>(e.m) + at * SS;
    v = static_cast<char*>(e.v) + at * SS;
    copy = W == W_MASTER ? static_cast<char*>(e.p) + at * 2 : nullptr;
    m_scale = Q8 ? e.m_scale + static_cast<unsigned long long>(at) / kBlock : nullptr;
    v_scale = Q8 ? e.v_scale + static_cast<unsigned long long>(at) / kBlock : nullptr;
    const long long n = e.n - at;
    left = n < (1 << 30) ? static_cast<int>(n) : 1 << 30;
  }

  __device__ __forceinline__ void next_block() {
    g += kBlock * GS;
    p += kBlock * PS;
    m += kBlock * SS;
    v += kBlock * SS;
    if (W == W_MASTER) copy += kBlock * 2;
    if (Q8) {
      ++m_scale;
      ++v_scale;
    }
    left -= kBlock;
  }
};

// The eight values, as loaded.
template <bool Q8, int W, bool GB>
struct Lane {
  using At = Place<Q8, W, GB>;
  uint32_t g[GB ? 4 : 8], p[W == W_BF16 ? 4 : 8];
  uint32_t m[Q8 ? 2 : 8], v[Q8 ? 2 : 8];
  float m_scale, v_scale;

  __device__ __forceinline__ void load(const At& a, bool vec) {
    const bool whole = vec && a.left >= 8;
    load_raw(a.g, a.left, whole, g);
    load_raw(a.p, a.left, whole, p);
    load_raw(a.m, a.left, whole, m);
    load_raw(a.v, a.left, whole, v);
    if (Q8) {
      m_scale = *a.m_scale;
      v_scale = *a.v_scale;
    }
  }

  __device__ __forceinline__ void update(const At& a, bool vec, float decay, uint32_t first, const StepConsts& s) const {
    const auto both = [](float x) { return pack2(x, x); };
    f32x2 gf[4], pf[4], mf[4], vf[4], root[4];
    to_f32(g, gf);
    to_f32(p, pf);
    if constexpr (Q8) {
      decode8(make_uint2(m[0], m[1]), m_scale, mf);
      decode8(make_uint2(v[0], v[1]), v_scale, vf);
#pragma unroll
      for (int i = 0; i < 4; ++i) vf[i] = mul2(vf[i], vf[i]);
    } else {
      to_f32(m, mf);
      to_f32(v, vf);
    }
    const f32x2 clip = both(s.clip), b1 = both(s.b1), b2 = both(s.b2), rate1 = both(s.rate1), rate2 = both(s.rate2);
    const f32x2 keep = both(1.0f - s.lr * decay), size = both(-s.step_size), isq = both(s.inv_sqrt_bc2), eps = both(s.eps);
    const f32x2 zero = both(0.0f);
    f32x2 check = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 gi = mul2(gf[i], clip);
      mf[i] = sum2(mul2(b1, mf[i]), mul2(rate1, gi));
      vf[i] = sum2(mul2(b2, vf[i]), mul2(mul2(rate2, gi), gi));
      root[i] = sqrt2(vf[i]);
      if constexpr (!Q8) root[i] = root_or_inf(vf[i], root[i]);
      float da, db, qa, qb;
      unpack2(fma2(root[i], isq, eps), da, db);
      asm("rcp.approx.f32 %0, %1;" : "=f"(qa) : "f"(da));
      asm("rcp.approx.f32 %0, %1;" : "=f"(qb) : "f"(db));
      pf[i] = fma2(mul2(mf[i], pack2(qa, qb)), size, mul2(pf[i], keep));
      if (W == W_BF16) check = fma2(pf[i], zero, check);
    }
    const int n = a.left;
    const bool whole = vec && n >= 8;
    uint32_t x[8];
    if (Q8 || W == W_BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mix32(first ^ i);
    }
    if (W == W_BF16) {
      // without a master copy nearest rounding would lose updates below half a step of the weight
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y0, y1;
        unpack2(pf[i], y0, y1);
        b[2 * i] = __float_as_uint(y0);
        b[2 * i + 1] = __float_as_uint(y1);
      }
      float c0, c1;
      unpack2(check, c0, c1);
      if (c0 + c1 == 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] += ((x[i] ^ (x[i] >> 15)) * 0x1B56C4E9u) >> 16;
      } else {  // (a NaN's bits would run over)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (fabsf(__uint_as_float(b[i])) < INFINITY) b[i] += ((x[i] ^ (x[i] >> 15)) * 0x1B56C4E9u) >> 16;
      }
      const uint32_t w[4] = {__byte_perm(b[0], b[1], 0x7632), __byte_perm(b[2], b[3], 0x7632),
                             __byte_perm(b[4], b[5], 0x7632), __byte_perm(b[6], b[7], 0x7632)};
      store8_b16(a.p, n, whole, w);
    } else {
      store8_f32(a.p, n, whole, pf);
      if (W == W_MASTER) {
        const uint32_t w[4] = {pack_bf16(pf[0]), pack_bf16(pf[1]), pack_bf16(pf[2]), pack_bf16(pf[3])};
        store8_b16(a.copy, n, whole, w);
      }
    }
    if constexpr (Q8) {
      float sm, sr;
      store8_codes(a.m, n, whole, encode8<false>(mf, x, sm));
      store8_codes(a.v, n, whole, encode8<true>(root, x, sr));
      if ((threadIdx.x & 31) == 0) {
        *a.m_scale = sm;
        *a.v_scale = sr;
      }
    } else {
      store8_f32(a.m, n, whole, mf);
      store8_f32(a.v, n, whole, vf);
    }
  }
};

// `count` blocks of a tensor from value `at` (the lane's first) on, by one warp. The warps of three or
// four CTAs an SM cover one another's loads (a block's loads issued ahead of the one before it took the
// registers of a CTA and 2% more time). Out of line: each pair of types has its own registers
// (inlined into one kernel, six of them spilled 950 bytes a thread).
template <bool Q8, int W, bool GB>
__device__ __noinline__ void run_blocks(const AdamwEntry* entry, long long at, int count, uint32_t key,
                                        const StepConsts* consts) {
  Place<Q8, W, GB> a(*entry, at);
  const bool vec = entry->vec;
  const float decay = entry->weight_decay;
  const StepConsts& s = *consts;
  // (a lane's eight values share all but the last three bits of their index)
  uint32_t high = mix32(static_cast<uint32_t>(at >> 32) + key);
  uint32_t low = static_cast<uint32_t>(at);
#pragma unroll 1
  for (int k = 0; k < count; ++k) {
    Lane<Q8, W, GB> x;
    x.load(a, vec);
    x.update(a, vec, decay, low ^ high, s);
    a.next_block();
    low += kBlock;
    at += kBlock;
    if (low < kBlock) high = mix32(static_cast<uint32_t>(at >> 32) + key);
  }
}

template <bool Q8>
__global__ void __launch_bounds__(kThreads, Q8 ? 4 : 3)
    adamw_step_kernel(const AdamwEntry* entries, int n_tensors, long long chunks, AdamwHyper h,
                      const float* lr_dev, AdamwControl* ctl, int clipped, long long run, int* err_flag) {
  __shared__ StepConsts sc;
  if (threadIdx.x == 0) {
    const long long t = ctl->step + 1;
    sc.lr = lr_dev ? *lr_dev : h.lr;
    // 1 - b^t without cancellation for b near 1
    const float bc1 = -expm1f(static_cast<float>(h.log_b1 * static_cast<double>(t)));
    const float bc2 = -expm1f(static_cast<float>(h.log_b2 * static_cast<double>(t)));
    sc.step_size = sc.lr / bc1;
    sc.inv_sqrt_bc2 = 1.0f / sqrtf(bc2);
    sc.b1 = h.b1;
    sc.b2 = h.b2;
    sc.rate1 = h.rate1;
    sc.rate2 = h.rate2;
    sc.eps = h.eps;
    sc.key = mix32(h.seed ^ mix32(static_cast<uint32_t>(t)));
    if (clipped) wait_for_last_kernel();  // (the norm's; what stands above is the step's before it)
    sc.clip = clipped ? ctl->clip : 1.0f;
    sc.skip = clipped ? ctl->skip : 0;
  }
  __syncthreads();
  if (!sc.skip) {
    // runs of blocks (a tensor's last chunk counts whole), one warp each in turn
    const long long blocks = chunks * kChunkBlocks;
    const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
    const long long runs = (blocks + run - 1) / run;
    for (long long i = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < runs; i += warps) {
      // (last to first after a norm, whose last gradients are still in L2)
      const long long r = (clipped ? runs - 1 - i : i) * run;
      const long long b1 = r + run < blocks ? r + run : blocks;
      for (long long b0 = r; b0 < b1;) {
        const int t = find_tensor(entries, n_tensors, b0 / kChunkBlocks);
        const AdamwEntry& e = entries[t];
        const long long end = (e.chunk0 + (e.n + kAdamwChunk - 1) / kAdamwChunk) * kChunkBlocks;  // the next one's first
        const long long first = b0 - e.chunk0 * kChunkBlocks;
        const long long to = end < b1 ? end : b1;
        const long long exist = (e.n + kBlock - 1) / kBlock - first;
        const int count = static_cast<int>(exist < to - b0 ? exist : to - b0);
        const long long here = first * kBlock;
        b0 = to;
        if (count <= 0) continue;
        const long long at = here + (threadIdx.x & 31) * kPerLane;
        const uint32_t key = mix32(sc.key + 0x9E3779B9u * static_cast<uint32_t>(t + 1));
        const bool gb = e.g_dtype == MOE_DTYPE_BF16;
        if (e.master) {
          if (gb) run_blocks<Q8, W_MASTER, true>(&e, at, count, key, &sc);
          else run_blocks<Q8, W_MASTER, false>(&e, at, count, key, &sc);
        } else if (e.p_dtype == MOE_DTYPE_BF16) {
          if (gb) run_blocks<Q8, W_BF16, true>(&e, at, count, key, &sc);
          else run_blocks<Q8, W_BF16, false>(&e, at, count, key, &sc);
        } else {
          if (gb) run_blocks<Q8, W_F32, true>(&e, at, count, key, &sc);
          else run_blocks<Q8, W_F32, false>(&e, at, count, key, &sc);
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&ctl->step_ticket, 1u) == gridDim.x - 1) {  // every CTA has read the control block
      ctl->step_ticket = 0;
      if (sc.skip) set_flag(err_flag, MOE_FLAG_NONFINITE);
      else ctl->step += 1;
    }
  }
}

}  // namespace

int adamw_norm_ctas() { return 4 * num_sms(); }

cudaError_t launch_grad_norm(const AdamwEntry* entries, int n, long long chunks, float max_norm,
                             double* partial, AdamwControl* ctl, cudaStream_t st) {
  const long long most = adamw_norm_ctas(), of_cta = kThreads / 32 * kNormRun;
  const long long want = (chunks * kChunkBlocks + of_cta - 1) / of_cta;
  const int grid = static_cast<int>(want < most ? want : most);
  LaunchTimer lt("grad_norm", st);
  grad_norm_kernel<<<grid, kThreads, 0, st>>>(entries, n, chunks, max_norm, partial, ctl);
  return cudaGetLastError();
}

cudaError_t launch_adamw_step(const AdamwEntry* entries, int n, long long chunks, int state_bits,
                              const AdamwHyper& h, const float* lr_dev, AdamwControl* ctl,
                              bool clipped, int* err_flag, cudaStream_t st) {
  // Four or three CTAs an SM (8- and 32-bit states), fewer where there is not a block for every warp.
  const long long ctas = (state_bits == 8 ? 4ll : 3ll) * num_sms();
  const int grid = static_cast<int>(chunks < ctas ? chunks : ctas);
  // A warp's run: an equal share of all blocks with 8-bit states, whose instructions have to be spread
  // evenly (67 M bf16 values: 177 us, in runs of 8 blocks 10% more); at most 8 blocks with 32-bit ones, which
  // HBM bounds and which want neighbouring addresses (fp32: 295 us, equal shares 7% more).
  const long long warps = static_cast<long long>(grid) * (kThreads / 32);
  long long run = (chunks * kChunkBlocks + warps - 1) / warps;
  if (state_bits == 32 && run > kChunkBlocks) run = kChunkBlocks;
  LaunchTimer lt(state_bits == 8 ? "adamw_step8" : "adamw_step32", st);
  // (behind the norm, if there is one: its CTAs are then in place when it ends)
  const auto kernel = state_bits == 8 ? adamw_step_kernel<true> : adamw_step_kernel<false>;
  if (clipped)
    return launch_behind(kernel, grid, kThreads, 0, st, entries, n, chunks, h, lr_dev, ctl, 1, run, err_flag);
  kernel<<<grid, kThreads, 0, st>>>(entries, n, chunks, h, lr_dev, ctl, 0, run, err_flag);
  return cudaGetLastError();
}

}  // namespace moe
