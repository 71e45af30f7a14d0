// Launchers of the selective scan.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace moe {

constexpr int kScanTile = 32;  // tokens between two states that a forward keeps for its backward

struct ScanArgs {
  const void* u;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* skip;
  const void* z;
  const float* dt_bias;
  const int* cu;
  const float* state_in;
  int N, T, max_seqlen, D, S, G;
  long long ldu, ldd, ldb, ldc, ldz, ldy;
  int softplus;
  void* y;
  float* state_out;
  float* tile_states;  // nullable: the state before each tile, for the backward
  float* ws;
  int* err_flag;
};

struct ScanBwdArgs {
  ScanArgs f;  // the forward's inputs; y, state_in and state_out unused, ldy unused
  const void* dy;
  const float* d_state_out;
  long long lddy;
  void* du;
  void* dd;
  void* dB;
  void* dC;
  void* dz;
  long long lddu, lddd, lddz;  // dB and dC are [T][G][S]
  float* dA;
  float* dskip;
  float* d_dt_bias;
  float* d_state_in;
};

struct ScanStepArgs {
  const void* u;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* skip;
  const void* z;
  const float* dt_bias;
  float* state;
  const int* state_idx;
  int n_slots, B_rows, D, S, G;
  long long ldu, ldd, ldb, ldc, ldz, ldy;
  int softplus;
  void* y;
  int* err_flag;
};

size_t scan_tile_states_bytes(int T, int N, int D, int S);
size_t scan_workspace(int max_seqlen, int T, int N, int D, int S, int G, bool backward);
cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t st);
cudaError_t launch_scan_bwd(const ScanBwdArgs& a, cudaStream_t st);
cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t st);

}  // namespace moe
