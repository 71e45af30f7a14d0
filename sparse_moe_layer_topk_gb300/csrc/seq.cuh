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

// Sequences that need no look of their own: 128 that are all in order, which one vote tells, and that hold `left` parts at most, the
// next 128 on their way meanwhile. From `base`, with `highest` the last bound before it. A call of its own, so that nothing of it stays in the
// registers of the kernels. (65,536 tokens x 2,048 channels in 2,048 sequences, without it and with it: convolution 331 -> 142 us and its
// backward 394 -> 229, scan 5.6 -> 1.5 ms and its backward 13.1 -> 4.7; in 8,192: 2.45 -> 0.57, 3.6 -> 0.82, 47 -> 8.1, 98 -> 22 ms, where sequences
// of equal length without bounds take 0.12, 0.28, 2.9, 11.4.)
constexpr int kWalk = 128;
struct Walk {
  int base, parts, highest;
};
static __device__ __noinline__ Walk walk_ordered(const int* cu, int N, int T, int longest, int length, int left, int base, int highest) {
  constexpr int kSets = kWalk / 32;
  const int lane = static_cast<int>(lane_id());
  int a[kSets], b[kSets], walked = 0;
  const auto fetch = [&](int from) {
#pragma unroll
    for (int w = 0; w < kSets; ++w) {
      const int i = from + 32 * w + lane;
      a[w] = i < N ? __ldg(cu + i) : 0, b[w] = i < N ? __ldg(cu + i + 1) : 0;
    }
  };
  fetch(base);
  while (N - base >= kWalk) {
    int sum = 0;
    bool ordered = lane > 0 || a[0] >= highest;
    const int last = b[kSets - 1];
#pragma unroll
    for (int w = 0; w < kSets; ++w) {
      ordered &= b[w] >= a[w] && b[w] <= T && b[w] - a[w] <= longest;
      sum += b[w] - a[w] <= length ? 1 : parts_of(b[w] - a[w], length);
    }
    fetch(base + kWalk);
    const int all = static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(sum)));
    if (!__all_sync(0xFFFFFFFFu, ordered) || walked + all > left) break;
    walked += all, base += kWalk;
    highest = __shfl_sync(0xFFFFFFFFu, last, 31);  // (the next one's start, if there is one)
  }
  return Walk{base, walked, highest};
}

// Part c of all sequences' parts of `length` tokens, a sequence having at least one (an empty sequence's
// part has no tokens). False where there are no more. Called by whole warps; every lane gets the answer.
// A sequence that ends before it starts or past T, starts before an earlier bound, or has more than `longest`
// tokens has no part; the warp that asks for part 0 flags it. So the parts of all sequences are at most T / length + N.
// FEW: known to be less than kWalk sequences.
template <bool FEW = false>
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
    if (!FEW && base % kWalk == 0 && N - base >= kWalk) {
      const Walk w = walk_ordered(cu, N, T, longest, length, found ? 0x7FFFFFFF : c - before, base, highest);
      base = w.base, before += w.parts, highest = w.highest;
    }
    if (base >= N) break;
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
