// Packed sequences: which part of which sequence a CTA works on.
#pragma once

#include "common.cuh"

namespace moe {

struct SeqPart {
  int n;      // sequence
  int start;  // its first token
  int len;    // its tokens
  int part;   // this part of it, `length` tokens each
};

__device__ __forceinline__ int parts_of(int len, int length) { return len > 0 ? (len - 1) / length + 1 : 1; }

// Part c of all sequences' parts of `length` tokens, a sequence having at least one (an empty sequence's
// part has no tokens). False where there are no more. Called by whole warps; every lane gets the answer.
// A sequence that ends before it starts or past T, starts before an earlier bound, or has more than `longest`
// tokens has no part; the warp that asks for part 0 flags it. So the parts of all sequences are at most T / length + N.
__device__ __forceinline__ bool find_part(const int* cu, int N, int T, int longest, int length, int c, SeqPart& out,
                                          int* err_flag) {
  if (cu == nullptr) {
    out.len = T / N;
    const int per = parts_of(out.len, length);
    out.n = c / per;
    out.part = c - out.n * per;
    out.start = out.n * out.len;
    return out.n < N;
  }
  const int lane = static_cast<int>(lane_id());
  int before = 0, highest = 0;
  bool found = false;
  for (int base = 0; base < N; base += 32) {
    const int i = base + lane;
    const int a = i < N ? __ldg(cu + i) : 0, b = i < N ? __ldg(cu + i + 1) : 0;
    int top = i < N ? a : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, top, o);
      if (lane >= o) top = max(top, x);
    }
    top = max(top, highest);
    const bool good = i < N && a == top && b >= a && b <= T && b - a <= longest;
    if (c == 0 && i < N && !good) set_flag(err_flag, MOE_FLAG_BAD_INDEX);
    const int mine = good ? parts_of(b - a, length) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += x;
    }
    const int at = c - before - (incl - mine);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, at >= 0 && at < mine);
    if (!found && hit) {
      const int src = __ffs(hit) - 1;
      found = true;
      out.n = base + src;
      out.start = __shfl_sync(0xFFFFFFFFu, a, src);
      out.len = __shfl_sync(0xFFFFFFFFu, b, src) - out.start;
      out.part = __shfl_sync(0xFFFFFFFFu, at, src);
      if (c != 0) return true;  // (part 0's warp looks at all sequences)
    }
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
    highest = __shfl_sync(0xFFFFFFFFu, top, 31);
  }
  return found;
}

}  // namespace moe
