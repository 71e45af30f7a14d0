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
// is read and written once, 8 bytes for 2 + r multiply-adds, so HBM bounds it. A CTA takes COLS
// columns of one row's state head, a lane 8 columns (32-byte accesses) of Dk / (256 * 8 / COLS) rows, all
// of whose loads are under way before the first is used; four CTAs an SM hold 128 KB in flight. The
// partial sums of o over the rows are joined by shuffles and in shared memory, in a fixed order.
// Measured: 256 rows x 32 heads, 128 x 128 (1.08 GB): 185 us, 5.8 TB/s, 0.86 of a plain copy's rate;
// with 16-byte accesses and three CTAs an SM 246. (Tiles of 64 columns spill 48 bytes a thread at the
// 64 registers that four CTAs an SM allow.) One row: 10 us a call from Python, 2.5 in a graph.
constexpr int kStepThreads = 256;
constexpr int kStepHeads = 4;  // query heads whose partial sums share one exchange

template <int COLS>
__global__ void __launch_bounds__(kStepThreads, 4)
    linattn_step_kernel(const bf16* q, const bf16* k, const bf16* v, const float* log_decay,
                        float* state, const int* state_idx, int n_slots, int Hs, int r, int Dk,
                        int Dv, long long ldq, long long ldk, long long ldv, long long ldo,
                        float scale, bf16* o, int* err_flag) {
  constexpr int GROUPS = COLS / 8;               // lanes side by side
  constexpr int ROWS = kStepThreads / GROUPS;    // rows at a time
  constexpr int N = 128 / ROWS;                  // rows of a lane
  constexpr int WARPS = kStepThreads / 32;
  const int tiles = (Dv + COLS - 1) / COLS;
  const int tile = blockIdx.x % tiles;
  const int h = blockIdx.x / tiles % Hs, b = blockIdx.x / tiles / Hs;
  const int col0 = tile * COLS;
  const int nc = min(COLS, Dv - col0);  // columns of this CTA, a multiple of 8
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
  const int c = tid % GROUPS, row0 = tid / GROUPS;
  const bool mine = c * 8 < nc;
  float* const S = state + (static_cast<long long>(slot) * Hs + h) * Dk * Dv + col0 + 8 * c;
  float x[N][8];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = row0 + i * ROWS;
    if (mine && row < Dk) {
      load_f32x8(S + row * Dv, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
    }
  }
  __shared__ float sk[128], sq[kStepHeads][128];
  __shared__ float part[kStepHeads][WARPS][COLS];
  if (tid < Dk) sk[tid] = __bfloat162float(k[b * ldk + static_cast<long long>(h) * Dk + tid]);
  float vv[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (mine) {
    const uint4 w = *reinterpret_cast<const uint4*>(v + b * ldv + static_cast<long long>(h) * Dv + col0 + 8 * c);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      vv[2 * j] = bf16_lo(u[j]);
      vv[2 * j + 1] = bf16_hi(u[j]);
    }
  }
  const float lam = expf(head_log_decay(log_decay, h, tid == 0 ? err_flag : nullptr));
  const bf16* const qrow = q + b * ldq + static_cast<long long>(h) * r * Dk;
  for (int i = tid; i < min(kStepHeads, r) * Dk; i += kStepThreads) sq[i / Dk][i % Dk] = __bfloat162float(qrow[i]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = row0 + i * ROWS;
    if (mine && row < Dk) {
      const float kr = sk[row];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = fmaf(lam, x[i][j], kr * vv[j]);
      store_f32x8(S + row * Dv, x[i]);
    }
  }
  for (int a0 = 0; a0 < r; a0 += kStepHeads) {
    const int heads = min(kStepHeads, r - a0);
    if (a0 > 0) {
      __syncthreads();
      for (int i = tid; i < heads * Dk; i += kStepThreads)
        sq[i / Dk][i % Dk] = __bfloat162float(qrow[static_cast<long long>(a0) * Dk + i]);
      __syncthreads();
    }
    for (int a = 0; a < heads; ++a) {
      float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = row0 + i * ROWS;
        const float qr = row < Dk ? sq[a][row] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(qr, x[i][j], acc[j]);
      }
#pragma unroll
      for (int d = GROUPS; d < 32; d <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], d);
      if ((tid & 31) < GROUPS) {
#pragma unroll
        for (int j = 0; j < 8; ++j) part[a][tid >> 5][8 * c + j] = acc[j];
      }
    }
    __syncthreads();
    for (int i = tid; i < heads * nc; i += kStepThreads) {
      const int a = i / nc, j = i - a * nc;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) sum += part[a][w][j];
      orow[static_cast<long long>(a0 + a) * Dv + j] = __float2bfloat16_rn(scale * sum);
    }
  }
}

}  // namespace

cudaError_t launch_linattn_step(const void* q, const void* k, const void* v,
                                const float* log_decay, float* state, const int* state_idx,
                                int n_slots, int B, int Hs, int r, int Dk, int Dv, long long ldq,
                                long long ldk, long long ldv, long long ldo, float scale, void* o,
                                int* err_flag, cudaStream_t st) {
  const auto tiles = [&](int cols) { return static_cast<unsigned>((Dv + cols - 1) / cols) * B * Hs; };
  LaunchTimer lt("linattn_step", st);
  const auto run = [&](auto kernel, unsigned grid) {
    kernel<<<grid, kStepThreads, 0, st>>>(static_cast<const bf16*>(q), static_cast<const bf16*>(k),
                                          static_cast<const bf16*>(v), log_decay, state, state_idx, n_slots, Hs, r, Dk,
                                          Dv, ldq, ldk, ldv, ldo, scale, static_cast<bf16*>(o), err_flag);
  };
  // Tiles of 64 columns where they fill the SMs twice over (32 heads of 128 x 128, in a graph: 64 rows
  // 49.2 us, in tiles of 32 columns 51.9), of 32 where there are fewer (5 rows 4.95 us, in tiles of 64 5.39).
  if (tiles(64) >= 8u * num_sms()) run(linattn_step_kernel<64>, tiles(64));
  else run(linattn_step_kernel<32>, tiles(32));
  return cudaGetLastError();
}

}  // namespace moe
