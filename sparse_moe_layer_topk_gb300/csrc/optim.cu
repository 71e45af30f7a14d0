// AdamW over many tensors in one launch, states in 32 or 8 bits, with the global
// gradient norm in a launch before it when the step is clipped.
//
//   g' = c g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Nothing is reused, so the step is bound by HBM: p, m, v in and out and g in.
// One CTA takes chunks of 2048 values of one tensor (a prefix of the tensors'
// chunk counts, searched once a chunk, says which), eight consecutive values a
// lane: 32-byte loads and stores of fp32, 16-byte of bf16, 8-byte of codes, all
// of a chunk's loads before its first use. A warp holds 256 values, the 8-bit
// states' block, whose largest magnitude is then one warp reduction.
#include "common.cuh"
#include "optim.h"
#include "timing.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPerLane = 8;
constexpr int kBlock = 32 * kPerLane;  // values of one warp, and of one 8-bit block
static_assert(kThreads * kPerLane == kAdamwChunk, "chunk");
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

__device__ __forceinline__ void ld_f32x8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}

__device__ __forceinline__ void st_f32x8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Eight values from element `at` of an fp32 or bf16 array; `n` of them exist.
__device__ __forceinline__ void load8(const void* base, int dtype, long long at, int n, bool vec,
                                      float (&v)[8]) {
  if (dtype == MOE_DTYPE_F32) {
    const float* p = static_cast<const float*>(base) + at;
    if (vec && n == 8) {
      ld_f32x8(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
  } else {
    const bf16* p = static_cast<const bf16*>(base) + at;
    if (vec && n == 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(u[i]);
        v[2 * i + 1] = bf16_hi(u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
    }
  }
}

__device__ __forceinline__ void store8_f32(float* p, int n, bool vec, const float (&v)[8]) {
  if (vec && n == 8) {
    st_f32x8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

__device__ __forceinline__ void store8_b16(bf16* p, int n, bool vec, const uint32_t (&h)[8]) {
  if (vec && n == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16),
                                              h[4] | (h[5] << 16), h[6] | (h[7] << 16));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(h[i]);
  }
}

__device__ __forceinline__ uint2 load8_codes(const uint8_t* p, int n, bool vec) {
  if (vec && n == 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store8_codes(uint8_t* p, int n, bool vec, uint2 c) {
  if (vec && n == 8) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// ------------------------------------------------------------------ 8-bit states

__device__ __forceinline__ void decode8(uint2 c, float scale, float (&v)[8]) {
  e4m3x4_to_f32(c.x, v);
  e4m3x4_to_f32(c.y, v + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= scale;
}

// Eight values of a warp's 256-value block as E4M3 codes and the block's scale,
// the largest finite magnitude / 448. Times 2^-120 an E4M3 value's bits are those
// of the fp32 with the code in bits 20..26, subnormals included, so adding a
// random number below 2^20 and cutting rounds up with a probability equal to
// the part cut off (nearest rounding would freeze v: at b2 = 0.999 it moves by
// less than half a step). The random number has 16 bits. A non-finite value
// gets the NaN code.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], const uint32_t (&rand16)[8],
                                         float& scale) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    top = fmaxf(top, a < INFINITY ? a : 0.0f);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  // below 2^-100 a block counts as zero (448 / top would overflow)
  const float inv = top > 7.8886e-31f ? __fmul_rn(__frcp_rn(top), 448.0f) : 0.0f;
  scale = top * (1.0f / 448.0f);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    const uint32_t bits = __float_as_uint(a * inv * 0x1p-120f);
    uint32_t code = min((bits + (rand16[i] << 4)) >> 20, 0x7Eu);
    if (!(a < INFINITY)) code = 0x7Fu;
    code |= (__float_as_uint(x[i]) >> 24) & 0x80u;
    w[i >> 2] |= code << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
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

// Sum of squares of all gradients. Each CTA writes one partial; the last one to
// finish adds them in a fixed order, so the norm does not depend on timing.
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const AdamwEntry* entries, int n_tensors, long long chunks, float max_norm,
                     double* partial, AdamwControl* ctl) {
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (long long c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = find_tensor(entries, n_tensors, c);
    const AdamwEntry& e = entries[t];
    const long long at = (c - e.chunk0) * kAdamwChunk + threadIdx.x * kPerLane;
    const long long left = e.n - at;
    if (left <= 0) continue;
    float g[8];
    load8(e.g, e.g_dtype, at, static_cast<int>(left < 8 ? left : 8), e.vec, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(g[i], g[i], acc[i]);
  }
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += static_cast<double>(acc[i]);
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
    const float norm = static_cast<float>(sqrt(s));
    ctl->grad_norm = norm;
    ctl->clip = fminf(1.0f, max_norm / (norm + 1e-6f));
    ctl->skip = norm < INFINITY ? 0 : 1;
    ctl->norm_ticket = 0;
  }
}

// ------------------------------------------------------------------ step

struct StepConsts {
  float clip, lr, step_size, inv_sqrt_bc2;
  uint32_t key;
  int skip;
};

template <bool Q8>
__global__ void __launch_bounds__(kThreads)
    adamw_step_kernel(const AdamwEntry* entries, int n_tensors, long long chunks, AdamwHyper h,
                      const float* lr_dev, AdamwControl* ctl, int clipped, int* err_flag) {
  __shared__ StepConsts sc;
  if (threadIdx.x == 0) {
    const long long t = ctl->step + 1;
    sc.lr = lr_dev ? *lr_dev : h.lr;
    // 1 - b^t without cancellation for b near 1
    const float bc1 = -expm1f(static_cast<float>(h.log_b1 * static_cast<double>(t)));
    const float bc2 = -expm1f(static_cast<float>(h.log_b2 * static_cast<double>(t)));
    sc.step_size = sc.lr / bc1;
    sc.inv_sqrt_bc2 = 1.0f / sqrtf(bc2);
    sc.clip = clipped ? ctl->clip : 1.0f;
    sc.skip = clipped ? ctl->skip : 0;
    sc.key = mix32(h.seed ^ mix32(static_cast<uint32_t>(t)));
  }
  __syncthreads();
  const StepConsts s = sc;
  if (!s.skip) {
    for (long long c = blockIdx.x; c < chunks; c += gridDim.x) {
      const int t = find_tensor(entries, n_tensors, c);
      const AdamwEntry& e = entries[t];
      const long long at = (c - e.chunk0) * kAdamwChunk + threadIdx.x * kPerLane;
      const long long left = e.n - at;
      const int n = left <= 0 ? 0 : static_cast<int>(left < 8 ? left : 8);
      const bool vec = e.vec;
      if (__all_sync(0xFFFFFFFFu, n == 0)) continue;
      float g[8], p[8], m[8], v[8];
      const bool wide = e.master != nullptr;
      const long long blk = at / kBlock;
      load8(e.g, e.g_dtype, at, n, vec, g);
      load8(wide ? static_cast<const void*>(e.master) : e.p, wide ? MOE_DTYPE_F32 : e.p_dtype, at,
            n, vec, p);
      if constexpr (Q8) {
        const uint2 cm = load8_codes(static_cast<const uint8_t*>(e.m) + at, n, vec);
        const uint2 cv = load8_codes(static_cast<const uint8_t*>(e.v) + at, n, vec);
        decode8(cm, __ldg(e.m_scale + blk), m);
        decode8(cv, __ldg(e.v_scale + blk), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= v[i];
      } else {
        load8(e.m, MOE_DTYPE_F32, at, n, vec, m);
        load8(e.v, MOE_DTYPE_F32, at, n, vec, v);
      }
      const float keep = 1.0f - s.lr * e.weight_decay;
      float r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gi = g[i] * s.clip;
        // each operation rounded by itself: which E4M3 neighbour a value gets then follows
        // from the formula alone, not from how a compiler pairs products with sums
        m[i] = __fadd_rn(__fmul_rn(h.b1, m[i]), __fmul_rn(h.rate1, gi));
        v[i] = __fadd_rn(__fmul_rn(h.b2, v[i]), __fmul_rn(__fmul_rn(h.rate2, gi), gi));
        r[i] = __fsqrt_rn(v[i]);
        p[i] = fmaf(p[i], keep, -s.step_size * __fdividef(m[i], fmaf(r[i], s.inv_sqrt_bc2, h.eps)));
      }
      const bool bf = e.p_dtype == MOE_DTYPE_BF16;
      uint32_t um[8], ur[8], up[8];
      if (Q8 || (bf && !wide)) {
        // (a lane's eight values share the upper half of their index)
        const uint32_t key = mix32(s.key + 0x9E3779B9u * static_cast<uint32_t>(t + 1));
        const uint32_t kb = mix32(static_cast<uint32_t>(at >> 32) + key);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = mix32((static_cast<uint32_t>(at) + i) ^ kb);
          um[i] = x & 0xFFFFu;
          ur[i] = x >> 16;
          up[i] = ((x ^ (x >> 15)) * 0x1B56C4E9u) >> 16;
        }
      }
      if constexpr (Q8) {
        float sm, sr;
        const uint2 cm = encode8(m, um, sm);
        const uint2 cv = encode8(r, ur, sr);
        store8_codes(static_cast<uint8_t*>(e.m) + at, n, vec, cm);
        store8_codes(static_cast<uint8_t*>(e.v) + at, n, vec, cv);
        if ((threadIdx.x & 31) == 0) {
          e.m_scale[blk] = sm;
          e.v_scale[blk] = sr;
        }
      } else {
        store8_f32(static_cast<float*>(e.m) + at, n, vec, m);
        store8_f32(static_cast<float*>(e.v) + at, n, vec, v);
      }
      if (wide) store8_f32(e.master + at, n, vec, p);
      if (!bf) {
        store8_f32(static_cast<float*>(e.p) + at, n, vec, p);
      } else {
        uint32_t hb[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (wide) {
            hb[i] = __bfloat16_as_ushort(__float2bfloat16_rn(p[i]));
          } else {
            // without a master copy nearest rounding would lose updates below half
            // a step of the weight; non-finite values are passed on as they are
            const uint32_t b = __float_as_uint(p[i]);
            hb[i] = fabsf(p[i]) < INFINITY ? (b + up[i]) >> 16
                                           : __bfloat16_as_ushort(__float2bfloat16_rn(p[i]));
          }
        }
        store8_b16(static_cast<bf16*>(e.p) + at, n, vec, hb);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&ctl->step_ticket, 1u) == gridDim.x - 1) {  // every CTA has read the control block
      ctl->step_ticket = 0;
      if (s.skip) set_flag(err_flag, MOE_FLAG_NONFINITE);
      else ctl->step += 1;
    }
  }
}

}  // namespace

int adamw_norm_ctas() { return 4 * num_sms(); }

cudaError_t launch_grad_norm(const AdamwEntry* entries, int n, long long chunks, float max_norm,
                             double* partial, AdamwControl* ctl, cudaStream_t st) {
  const long long most = adamw_norm_ctas();
  const int grid = static_cast<int>(chunks < most ? chunks : most);
  LaunchTimer lt("grad_norm", st);
  grad_norm_kernel<<<grid, kThreads, 0, st>>>(entries, n, chunks, max_norm, partial, ctl);
  return cudaGetLastError();
}

cudaError_t launch_adamw_step(const AdamwEntry* entries, int n, long long chunks, int state_bits,
                              const AdamwHyper& h, const float* lr_dev, AdamwControl* ctl,
                              bool clipped, int* err_flag, cudaStream_t st) {
  const long long most = 4ll * num_sms();
  const int grid = static_cast<int>(chunks < most ? chunks : most);
  LaunchTimer lt(state_bits == 8 ? "adamw_step8" : "adamw_step32", st);
  if (state_bits == 8)
    adamw_step_kernel<true><<<grid, kThreads, 0, st>>>(entries, n, chunks, h, lr_dev, ctl,
                                                       clipped ? 1 : 0, err_flag);
  else
    adamw_step_kernel<false><<<grid, kThreads, 0, st>>>(entries, n, chunks, h, lr_dev, ctl,
                                                        clipped ? 1 : 0, err_flag);
  return cudaGetLastError();
}

}  // namespace moe
