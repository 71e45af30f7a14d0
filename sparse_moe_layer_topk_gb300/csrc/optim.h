// Launchers of the optimizer step (optim.cu) and the layout of its plan.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kAdamwChunk = 2048;  // values one CTA takes at a time, of one tensor
constexpr int kAdamwBlock = 256;   // values that share a scale in the 8-bit states

// One tensor of a plan, as moe_adamw_plan writes it.
struct AdamwEntry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  long long n;
  long long chunk0;  // chunks of the tensors before it
  float weight_decay;
  int p_dtype, g_dtype;
  int vec;  // every array is aligned for whole vector accesses
};

// The caller's control block (MOE_ADAMW_CTL_BYTES, zeroed once).
struct AdamwControl {
  long long step;   // steps taken
  float grad_norm;  // of the last clipped step
  float clip;
  int skip;
  unsigned norm_ticket, step_ticket;
};

struct AdamwHyper {
  float lr, b1, b2, rate1, rate2, eps;  // rate = 1 - b
  double log_b1, log_b2;
  uint32_t seed;
};

int num_sms();
int adamw_norm_ctas();  // partial sums of the norm at most

cudaError_t launch_grad_norm(const AdamwEntry* entries, int n, long long chunks, float max_norm,
                             double* partial, AdamwControl* ctl, cudaStream_t st);
cudaError_t launch_adamw_step(const AdamwEntry* entries, int n, long long chunks, int state_bits,
                              const AdamwHyper& h, const float* lr_dev, AdamwControl* ctl,
                              bool clipped, int* err_flag, cudaStream_t st);

}  // namespace moe
