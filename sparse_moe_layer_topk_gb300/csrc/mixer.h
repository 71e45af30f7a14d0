// Launchers of the routing with scores and groups, the residual norm, the causal convolution and the
// selective scan.
#pragma once

#include <cuda_runtime.h>

namespace moe {

struct RouteArgs {
  const float* logits;
  const float* bias;
  int T, E, k, softmax, groups, group_k, group_top, renorm;
  float scale;
  int* idx;
  float* w;
  float* s;
  int* err_flag;
};
cudaError_t launch_route_scores(const RouteArgs& a, cudaStream_t st);

struct RouteBwdArgs {
  const float* d_w;
  const int* slot_of;
  const float* logits;
  const int* idx;
  const float* w;
  const float* s;
  int T, E, k, softmax, renorm;
  float scale;
  void* dL;
  int bf16_out;
  float* d_topk_w;
  int* err_flag;
};
cudaError_t launch_route_scores_bwd(const RouteBwdArgs& a, cudaStream_t st);

struct NormArgs {
  const void* x;
  const void* residual;
  const float* weight;
  int T, d;
  long long ldx;
  float eps;
  int res_f32, fp8;
  void* sum;
  void* y;
  float* y_scale;
  int block;
};
cudaError_t launch_rmsnorm_fwd(const NormArgs& a, cudaStream_t st);

struct NormBwdArgs {
  const void* dy;
  const void* u;
  const float* weight;
  const void* d_sum;
  int T, d;
  long long ldu;
  float eps;
  int res_f32;
  void* dx;
  void* d_residual;
  float* dw;
  float* part;
};
int rmsnorm_bwd_parts(int T, int d);
cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, cudaStream_t st);

struct ConvArgs {
  const void* x;
  const float* weight;
  const float* bias;
  const int* cu;
  const void* state_in;
  int N, T, D, W;
  long long ldx, ldy;
  int silu;
  void* y;
  void* state_out;
  int* err_flag;
};
cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t st);

struct ConvBwdArgs {
  const void* dy;
  const void* x;
  const float* weight;
  const float* bias;
  const int* cu;
  const void* state_in;
  const void* d_state_out;
  int N, T, D, W;
  long long lddy, ldx, lddx;
  int silu;
  void* dx;
  float* part;  // [parts][W + 1][D]: the taps' gradients, then the bias'; null: not wanted
  void* d_state_in;
  int* err_flag;
};
int conv_bwd_parts(int N, int T, int D);
cudaError_t launch_conv_bwd(const ConvBwdArgs& a, float* dw, float* db, cudaStream_t st);

struct ConvStepArgs {
  const void* x;
  const float* weight;
  const float* bias;
  void* state;
  const int* state_idx;
  int n_slots, B, D, W;
  long long ldx, ldy;
  int silu;
  void* y;
  int* err_flag;
};
cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t st);

}  // namespace moe
