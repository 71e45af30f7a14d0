// Linear attention with a decay for each state head: the step of a decoding batch
// (linattn_chunk.cu has the chunked form).
#include "common.cuh"
#include "linattn.h"
#include "timing.h"

namespace moe {

int num_sms();

namespace {

// log of the head's decay; NaN and positive entries count as 0 and are flagged.
__device__ __forceinline__ float head_log_decay(const float* log_decay, int h, int* err_flag) {
  const float g = __ldg(log_decay + h);
  if (g <= 0.0f) return g;
  set_flag(err_flag, MOE_FLAG_NONFINITE);
  return 0.0f;
}

// ------------------------------------------------------------------ decoding step
//
// S = lam S + k v^T and o = scale S^T q for one token of a row: every state value
// is read and written once, 8 bytes for 2 + r multiply-adds, so HBM bounds it. A CTA
// takes `cols` columns of one row's state head (128 threads: cols / 4 float4
// columns x the state's rows in turn), which cuts a state into up to four pieces
// when the batch is too small to fill the GPU; the partial sums of o are joined
// in shared memory in a fixed order.
constexpr int kStepThreads = 256;

__global__ void __launch_bounds__(kStepThreads)
    linattn_step_kernel(const bf16* q, const bf16* k, const bf16* v, const float* log_decay,
                        float* state, const int* state_idx, int n_slots, int Hs, int r, int Dk,
                        int Dv, long long ldq, long long ldk, long long ldv, long long ldo,
                        float scale, bf16* o, int* err_flag, int cols) {
  const int h = blockIdx.x % Hs, b = blockIdx.x / Hs;
  const int col0 = blockIdx.y * cols;
  const int nc = min(cols, Dv - col0);  // columns of this CTA, a multiple of 8
  const int tid = threadIdx.x;
  int slot = state_idx ? __ldg(state_idx + b) : b;
  if (slot >= n_slots) {
    if (tid == 0) set_flag(err_flag, MOE_FLAG_BAD_INDEX);
    slot = -1;
  }
  bf16* const orow = o + b * ldo + static_cast<long long>(h) * r * Dv + col0;
  if (slot < 0) {
    for (int i = tid; i < r * nc; i += kStepThreads)
      orow[static_cast<long long>(i / nc) * Dv + i % nc] = __float2bfloat16_rn(0.0f);
    return;
  }
  const float lam = expf(head_log_decay(log_decay, h, tid == 0 ? err_flag : nullptr));
  __shared__ float sk[128], sq[128];
  __shared__ float4 part[kStepThreads];
  const int groups = cols / 4;            // float4 columns side by side
  const int rows = kStepThreads / groups;  // rows at a time
  const int c = tid % groups, row0 = tid / groups;
  const bool mine = c * 4 < nc;
  float* const S = state + (static_cast<long long>(slot) * Hs + h) * Dk * Dv + col0 + 4 * c;
  if (tid < Dk) sk[tid] = __bfloat162float(k[b * ldk + static_cast<long long>(h) * Dk + tid]);
  float4 vv = make_float4(0, 0, 0, 0);
  if (mine) {
    const uint2 w = *reinterpret_cast<const uint2*>(v + b * ldv + static_cast<long long>(h) * Dv + col0 + 4 * c);
    vv = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  }
  // at most 16 rows a thread (128 rows, 8 at a time for 128 columns)
  float4 x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int row = row0 + i * rows;
    if (mine && row < Dk) x[i] = *reinterpret_cast<const float4*>(S + static_cast<long long>(row) * Dv);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int row = row0 + i * rows;
    if (mine && row < Dk) {
      const float kr = sk[row];
      x[i].x = fmaf(lam, x[i].x, kr * vv.x);
      x[i].y = fmaf(lam, x[i].y, kr * vv.y);
      x[i].z = fmaf(lam, x[i].z, kr * vv.z);
      x[i].w = fmaf(lam, x[i].w, kr * vv.w);
      *reinterpret_cast<float4*>(S + static_cast<long long>(row) * Dv) = x[i];
    }
  }
  for (int a = 0; a < r; ++a) {
    if (tid < Dk)
      sq[tid] = __bfloat162float(q[b * ldq + (static_cast<long long>(h) * r + a) * Dk + tid]);
    __syncthreads();
    float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = row0 + i * rows;
      if (mine && row < Dk) {
        const float qr = sq[row];
        acc.x = fmaf(qr, x[i].x, acc.x);
        acc.y = fmaf(qr, x[i].y, acc.y);
        acc.z = fmaf(qr, x[i].z, acc.z);
        acc.w = fmaf(qr, x[i].w, acc.w);
      }
    }
    part[tid] = acc;
    __syncthreads();
    if (tid < nc) {
      float sum = 0.0f;
      for (int i = 0; i < rows; ++i)
        sum += reinterpret_cast<const float*>(part)[(i * groups + (tid >> 2)) * 4 + (tid & 3)];
      orow[static_cast<long long>(a) * Dv + tid] = __float2bfloat16_rn(scale * sum);
    }
  }
}

}  // namespace

cudaError_t launch_linattn_step(const void* q, const void* k, const void* v,
                                const float* log_decay, float* state, const int* state_idx,
                                int n_slots, int B, int Hs, int r, int Dk, int Dv, long long ldq,
                                long long ldk, long long ldv, long long ldo, float scale, void* o,
                                int* err_flag, cudaStream_t st) {
  int cols = 128;
  while (cols > 32 && static_cast<long long>(B) * Hs * ((Dv + cols - 1) / cols) < 2ll * num_sms())
    cols /= 2;
  LaunchTimer lt("linattn_step", st);
  const dim3 grid(static_cast<unsigned>(B) * Hs, (Dv + cols - 1) / cols);
  linattn_step_kernel<<<grid, kStepThreads, 0, st>>>(
      static_cast<const bf16*>(q), static_cast<const bf16*>(k), static_cast<const bf16*>(v),
      log_decay, state, state_idx, n_slots, Hs, r, Dk, Dv, ldq, ldk, ldv, ldo, scale,
      static_cast<bf16*>(o), err_flag, cols);
  return cudaGetLastError();
}

}  // namespace moe
