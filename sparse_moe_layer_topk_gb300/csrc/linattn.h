// One recurrence of the linear attention, as the forward and the three products
// of the backward run it (linattn.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// Forward (rev = 0), tokens in order:  S = lam S + upd sum_b k_b v_b^T;  o_a = inter S^T q_a
// Reverse (rev = 1), last token first: S = S + upd sum_b k_b v_b^T;  o_a = inter S^T q_a;  S = lam S
// for each sequence and state head; query heads a < nq, key/value heads b < nkv of
// the state head's group (one of nq, nkv is 1).
struct LinProblem {
  const void *q, *k, *v;  // [T][Hs * nq][dk], [T][Hs * nkv][dk], [T][Hs * nkv][dv]
  long long ldq, ldk, ldv, ldo;
  void* o;  // [T][Hs * nq][dv]
  int nq, nkv, dk, dv, rev;
  float upd, inter;
  // fp32 states [N][Hs][dk][dv], element (i, j) at i * s_row + j * s_col of each
  const float* s_in;
  float* s_out;
  int s_row, s_col;
  int shares;  // index of the problem whose states are this one's transposed; -1: none
};

struct LinShape {
  const int* cu_seqlens;
  const float* log_decay;
  int N, T, max_seqlen, Hs;
  int* err_flag;
};

// The first token and length of sequence n; a length of -1 for one to skip.
__device__ __forceinline__ void lin_sequence(const LinShape& s, int n, int& start, int& len) {
  if (s.cu_seqlens == nullptr) {
    len = s.T / s.N;
    start = n * len;
    return;
  }
  start = __ldg(s.cu_seqlens + n);
  const long long end = __ldg(s.cu_seqlens + n + 1);
  const long long d = end - start;
  len = (start < 0 || end > s.T || d < 0 || d > s.max_seqlen) ? -1 : static_cast<int>(d);
}

// Runs np (1 to 3) recurrences over the same sequences. ws: linattn_workspace bytes (device); an MOE_*
// status.
size_t linattn_workspace(int max_seqlen, int Dk, int Dv, int Hs, int r, int T, int N, bool backward);
int linattn_run(const LinProblem* p, int np, const LinShape& s, void* ws, cudaStream_t st);

cudaError_t launch_linattn_step(const void* q, const void* k, const void* v,
                                const float* log_decay, float* state, const int* state_idx,
                                int n_slots, int B, int Hs, int r, int Dk, int Dv, long long ldq,
                                long long ldk, long long ldv, long long ldo, float scale, void* o,
                                int* err_flag, cudaStream_t st);

}  // namespace moe
