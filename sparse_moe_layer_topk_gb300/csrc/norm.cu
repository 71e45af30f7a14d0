// Root-mean-square norm of x + residual, output in bf16 or E4M3, and its backward.
#include "common.cuh"
#include "mixer.h"
#include "timing.h"

namespace moe {

int num_sms();

namespace {

constexpr int kBwdVec = 2;  // 16-byte vectors (of bf16) of a row that a thread of the backward holds, of each tensor, and of the next row

// Eight consecutive values as fp32.
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(u[j]);
    v[2 * j + 1] = bf16_hi(u[j]);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                            pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Eight values on their way.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16> {
  uint4 v;
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = bf16_lo(u[j]), f[2 * j + 1] = bf16_hi(u[j]);
  }
};
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v[j];
  }
};

// Sum (or maximum) over the THREADS threads of a row, the same for all of them. `slot`: THREADS / 32 floats of
// shared memory that nothing else uses until every thread has passed the next barrier.
template <int THREADS, bool MAX>
__device__ __forceinline__ float row_reduce(float x, float* slot) {
  const auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = join(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  if (THREADS == 32) return x;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = x;
  __syncthreads();
  float y = slot[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) y = join(y, slot[w]);
  return y;
}

// Two sums over a row's threads at once.
template <int THREADS>
__device__ __forceinline__ void row_sums(float& a, float& b, float (*slot)[THREADS / 32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  if (THREADS == 32) return;
  if ((threadIdx.x & 31) == 0) slot[0][threadIdx.x >> 5] = a, slot[1][threadIdx.x >> 5] = b;
  __syncthreads();
  a = slot[0][0], b = slot[1][0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) a += slot[0][w], b += slot[1][w];
}

// 1 / sqrt(mean(u^2) + eps) of a row from its squares' sum. Squares past fp32 (values above 1e19 / sqrt(d)) are summed once
// more, 2^-160 as large; eps is nothing beside them.
template <int THREADS, int VEC>
__device__ __forceinline__ float row_rstd(const float (&u)[VEC][8], float ss, int d, float eps, float* slot) {
  if (ss < 3e38f) return rsqrtf(ss / d + eps);
  float s2 = 0.0f;
#pragma unroll
  for (int i = 0; i < VEC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = u[i][j] * 0x1p-80f;
      s2 = fmaf(v, v, s2);
    }
  s2 = row_reduce<THREADS, false>(s2, slot);
  return rsqrtf(s2 / d) * 0x1p-80f;
}

// y = u w / sqrt(mean(u^2) + eps), u = x + residual in fp32: u goes to the norm unrounded and to the residual
// stream rounded once. A row is held in the registers of THREADS threads (one warp up to 1024 columns, then a
// CTA), VEC vectors each, so that HBM is read and written once and bounds it: 16,384 rows of 4,096 in 86 us, 79 of them the
// bytes. Few vectors a thread, so that 1,536 threads fit an SM: 4,000 rows of 5,120 with a fp32 stream and E4M3 outputs in 48 us with three
// vectors and 256 threads (43 in a graph, 33 of them the bytes: a CTA's one row is read, joined and written in turn), 54 with four, 54 with two and 512 threads, 51 with five and 128.
template <int THREADS, int VEC, typename R, bool FP8>
__global__ void __launch_bounds__(THREADS == 32 ? 128 : THREADS, THREADS * VEC <= 512 ? 1 : THREADS == 256 ? 6 : VEC <= 3 ? 3 : 2)
    rmsnorm_fwd_kernel(const bf16* __restrict__ x, const R* residual, const float* __restrict__ weight, int T, int d,
                       long long ldx, float eps, R* sum, void* y, float* y_scale, int block) {
  __shared__ float slots[3][THREADS / 32];
  constexpr int kRows = THREADS == 32 ? 4 : 1;
  const int t = blockIdx.x * kRows + (THREADS == 32 ? threadIdx.x >> 5 : 0);
  if (t >= T) return;  // (whole warps or CTAs)
  const int tid = threadIdx.x % THREADS, vectors = d / 8;
  const long long at = static_cast<long long>(t) * d;
  float u[VEC][8];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = tid + i * THREADS;
    if (c < vectors) {
      load8(x + t * ldx + 8 * c, u[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] = 0.0f;
    }
  }
  if (residual != nullptr) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = tid + i * THREADS;
      if (c < vectors) {
        float r[8];
        load8(residual + at + 8 * c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] += r[j];
        store8(sum + at + 8 * c, u[i]);
      }
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VEC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(u[i][j], u[i][j], ss);
  ss = row_reduce<THREADS, false>(ss, slots[0]);
  const float scale = row_rstd<THREADS, VEC>(u, ss, d, eps, slots[1]);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = tid + i * THREADS;
    if (c < vectors) {
      float w[8];
      load8(weight + 8 * c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[i][j] = u[i][j] * scale * w[j];
        if (FP8) top = fmaxf(top, fabsf(u[i][j]));
      }
      if (!FP8) store8(static_cast<bf16*>(y) + at + 8 * c, u[i]);
    }
  }
  if (!FP8) return;
  const bool whole = block >= d;
  if (whole) top = row_reduce<THREADS, true>(top, slots[2]);
  const int blocks = (d + block - 1) / block;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = tid + i * THREADS;
    float m = top;
    if (!whole) {  // blocks of 64 or 128 columns: 8 or 16 lanes side by side
      m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, c < vectors ? fabsf(u[i][j]) : 0.0f);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (block == 128) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
    }
    if (c >= vectors) continue;
    // (a block whose largest magnitude is below 2^-100 holds zeros: its reciprocal scale would leave fp32)
    const bool some = m >= 0x1p-100f;
    const float inv = some ? 448.0f / m : 0.0f;
    const uint32_t lo = f32x2_to_e4m3x2(u[i][0] * inv, u[i][1] * inv) | (f32x2_to_e4m3x2(u[i][2] * inv, u[i][3] * inv) << 16);
    const uint32_t hi = f32x2_to_e4m3x2(u[i][4] * inv, u[i][5] * inv) | (f32x2_to_e4m3x2(u[i][6] * inv, u[i][7] * inv) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(y) + at + 8 * c) = make_uint2(lo, hi);
    if (8 * c % block == 0) y_scale[static_cast<long long>(t) * blocks + 8 * c / block] = some ? m / 448.0f : 0.0f;
  }
}

// du = rstd (g - n mean(g n)) + d_sum with g = dy w, n = u rstd; dw = sum_t dy n. The row's sums of u^2 and of g u, which
// give rstd and the mean, are joined together, so nothing is kept from the forward but u. A CTA (THREADS threads; with
// 32 four warps, each its own rows) walks rows with a stride of the grid and keeps its columns' part of dw in
// registers; the parts are summed in a fixed order afterwards. HBM bounds it: 16,384 rows of 4,096 in 85 us, 79 of them the bytes; with a fp32 stream
// 165 and 158. 8,192 rows of 8,192 with a fp32 stream, where no row is ahead, 185 and 158.
template <int THREADS, typename U, typename R>
__global__ void __launch_bounds__(THREADS == 32 ? 128 : THREADS, THREADS <= 128 ? 4 : THREADS <= 512 ? 512 / THREADS : 1)
    rmsnorm_bwd_kernel(const bf16* __restrict__ dy, const U* __restrict__ from, const float* __restrict__ weight,
                       const R* d_sum, int T, int d, long long ldu, float eps, bf16* dx,
                       R* d_residual, float* part) {
  __shared__ float slots[3][2][THREADS / 32];
  constexpr int kRows = THREADS == 32 ? 4 : 1;
  // (a row ahead where the registers allow it: 64 a thread at 1,024 threads do not)
  constexpr bool kAhead = THREADS * (sizeof(R) == 4 ? 2 : 1) <= 512;
  const int tid = threadIdx.x % THREADS, vectors = d / 8;
  const unsigned first = blockIdx.x * kRows + (THREADS == 32 ? threadIdx.x >> 5 : 0), stride = gridDim.x * kRows, rows = T;
  float w[kBwdVec][8], dw[kBwdVec][8];
#pragma unroll
  for (int i = 0; i < kBwdVec; ++i) {
    const int c = tid + i * THREADS;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = dw[i][j] = 0.0f;
    if (c < vectors) load8(weight + 8 * c, w[i]);
  }
  Raw8<U> nu[kBwdVec];
  Raw8<bf16> ng[kBwdVec];
  Raw8<R> ns[kBwdVec];
  const auto fetch = [&](unsigned t) {
#pragma unroll
    for (int i = 0; i < kBwdVec; ++i) {
      const int c = tid + i * THREADS;
      nu[i].clear(), ng[i].clear(), ns[i].clear();
      if (t < rows && c < vectors) {
        nu[i].load(from + t * ldu + 8 * c);
        ng[i].load(dy + static_cast<long long>(t) * d + 8 * c);
        if (d_sum != nullptr) ns[i].load(d_sum + static_cast<long long>(t) * d + 8 * c);
      }
    }
  };
  if (kAhead) fetch(first);
  int turn = 0;
  for (unsigned t = first; t < rows; t += stride) {
    const long long at = static_cast<long long>(t) * d;
    float u[kBwdVec][8], g[kBwdVec][8];
    Raw8<R> s[kBwdVec];
    float ss = 0.0f, dot = 0.0f;
    if (!kAhead) fetch(t);
#pragma unroll
    for (int i = 0; i < kBwdVec; ++i) nu[i].floats(u[i]), ng[i].floats(g[i]), s[i] = ns[i];
    if (kAhead) fetch(t + stride);
#pragma unroll
    for (int i = 0; i < kBwdVec; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(u[i][j], u[i][j], ss);
        dot = fmaf(g[i][j] * w[i][j], u[i][j], dot);
      }
    row_sums<THREADS>(ss, dot, slots[turn]);  // (two slots in turn: one barrier a row)
    turn ^= 1;
    const float r = row_rstd<THREADS, kBwdVec>(u, ss, d, eps, slots[2][0]);
    dot = r * dot / d;  // mean(g n)
    if (!(ss < 3e38f)) {  // (u is too large for the sum above as well)
      dot = 0.0f;
#pragma unroll
      for (int i = 0; i < kBwdVec; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dot = fmaf(g[i][j] * w[i][j], u[i][j] * r, dot);
      dot = row_reduce<THREADS, false>(dot, slots[2][1]) / d;
    }
#pragma unroll
    for (int i = 0; i < kBwdVec; ++i) {
      const int c = tid + i * THREADS;
      if (c < vectors) {
        float add[8];
        s[i].floats(add);  // (zeros without d_sum)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = u[i][j] * r;
          dw[i][j] = fmaf(g[i][j], n, dw[i][j]);
          g[i][j] = fmaf(r, g[i][j] * w[i][j] - n * dot, add[j]);
        }
        if (dx != nullptr) store8(dx + at + 8 * c, g[i]);
        if (d_residual != nullptr) store8(d_residual + at + 8 * c, g[i]);
      }
    }
  }
  allow_next_kernel();
  if (part == nullptr) return;
  float* const mine = part + static_cast<long long>(first) * d;
#pragma unroll
  for (int i = 0; i < kBwdVec; ++i) {
    const int c = tid + i * THREADS;
    if (c < vectors) store8(mine + 8 * c, dw[i]);
  }
}

int bwd_threads(int d) { return d <= 512 ? 32 : d <= 2048 ? 128 : d <= 4096 ? 256 : d <= 8192 ? 512 : 1024; }

}  // namespace

// out[c] = sum over `parts` rows of part[.][c], in an order that depends on the sizes alone: 32 warps share 32 columns' rows.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* __restrict__ part, int parts, int cols, float* __restrict__ out) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  wait_for_last_kernel();
  float sum = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int p = g; p < parts; p += 32) sum += __ldg(part + static_cast<long long>(p) * cols + c);
  }
  s[g][lane] = sum;
  __syncthreads();
  sum = s[lane][g];  // (a warp has one column now)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const int mine = blockIdx.x * 32 + g;
  if (lane == 0 && mine < cols) out[mine] = sum;
}

// Rows of partial weight gradients that a backward writes.
int rmsnorm_bwd_parts(int T, int d) {
  const int th = bwd_threads(d), rows = th == 32 ? 4 : 1;
  const int ctas = T / rows + (T % rows != 0), most = num_sms() * (th <= 128 ? 4 : th == 256 ? 2 : 1);
  return (ctas < most ? ctas : most) * rows;
}

template <int THREADS, int VEC, typename R>
static void norm_fwd(const NormArgs& a, cudaStream_t st) {
  const int rows = THREADS == 32 ? 4 : 1, threads = THREADS == 32 ? 128 : THREADS;
  const unsigned grid = (static_cast<unsigned>(a.T) + rows - 1) / rows;
  const auto run = [&](auto kernel) {
    kernel<<<grid, threads, 0, st>>>(static_cast<const bf16*>(a.x), static_cast<const R*>(a.residual), a.weight, a.T, a.d,
                                     a.ldx, a.eps, static_cast<R*>(a.sum), a.y, a.y_scale, a.block);
  };
  if (a.fp8) run(rmsnorm_fwd_kernel<THREADS, VEC, R, true>);
  else run(rmsnorm_fwd_kernel<THREADS, VEC, R, false>);
}

template <int THREADS, typename U, typename R>
static void norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
  const int rows = THREADS == 32 ? 4 : 1, threads = THREADS == 32 ? 128 : THREADS;
  const unsigned grid = static_cast<unsigned>(rmsnorm_bwd_parts(a.T, a.d) / rows);
  rmsnorm_bwd_kernel<THREADS, U, R><<<grid, threads, 0, st>>>(
      static_cast<const bf16*>(a.dy), static_cast<const U*>(a.u), a.weight, static_cast<const R*>(a.d_sum), a.T, a.d,
      a.ldu, a.eps, static_cast<bf16*>(a.dx), static_cast<R*>(a.d_residual), a.dw ? a.part : nullptr);
}

template <typename R>
static void norm_fwd(const NormArgs& a, cudaStream_t st) {
  if (a.d <= 512) norm_fwd<32, 2, R>(a, st);
  else if (a.d <= 1024) norm_fwd<32, 4, R>(a, st);
  else if (a.d <= 2048) norm_fwd<128, 2, R>(a, st);
  else if (a.d <= 4096) norm_fwd<256, 2, R>(a, st);
  else if (a.d <= 6144) norm_fwd<256, 3, R>(a, st);
  else if (a.d <= 12288) norm_fwd<512, 3, R>(a, st);
  else norm_fwd<512, 4, R>(a, st);
}

cudaError_t launch_rmsnorm_fwd(const NormArgs& a, cudaStream_t st) {
  LaunchTimer lt("rmsnorm_fwd", st);
  if (a.res_f32) norm_fwd<float>(a, st);
  else norm_fwd<bf16>(a, st);
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, cudaStream_t st) {
  {
    LaunchTimer lt("rmsnorm_bwd", st);
    const auto run = [&](auto threads) {
      constexpr int TH = decltype(threads)::value;
      if (a.res_f32) norm_bwd<TH, float, float>(a, st);
      else norm_bwd<TH, bf16, bf16>(a, st);
    };
    switch (bwd_threads(a.d)) {
      case 32: run(std::integral_constant<int, 32>{}); break;
      case 128: run(std::integral_constant<int, 128>{}); break;
      case 256: run(std::integral_constant<int, 256>{}); break;
      case 512: run(std::integral_constant<int, 512>{}); break;
      default: run(std::integral_constant<int, 1024>{}); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.dw) return e;
  }
  LaunchTimer lt("rmsnorm_dw", st);
  return launch_behind(column_sums_kernel, dim3((a.d + 31) / 32), 1024, 0, st, static_cast<const float*>(a.part), rmsnorm_bwd_parts(a.T, a.d), a.d, a.dw);
}

}  // namespace moe
