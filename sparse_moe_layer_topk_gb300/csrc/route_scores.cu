// Routing with sigmoid or softmax scores, a bias for balance and groups of experts, and its backward
// (route_permute.cu has the plain sigmoid form).
#include "common.cuh"
#include "mixer.h"
#include "timing.h"

namespace moe {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 4;      // tokens of a CTA, one for each warp
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_quick(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_quick(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xFF800000); }

// Order-preserving bits of a float (+0 and -0 are one value); 0 is below every number's.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float bits_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

struct Params {
  const float* logits;
  const float* bias;
  int T, E, k, groups, group_k, group_top, renorm;
  float scale;
  int* idx;
  float* w;
  float* s;
  int* err_flag;
};

// Bitonic sort of one value a lane, descending.
template <typename V, typename Less>
__device__ __forceinline__ V sort_lanes(V x, int lane, Less less) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const V o = __shfl_xor_sync(kAll, x, stride);
      const bool keep_larger = ((lane & size) == 0) == ((lane & stride) == 0);
      x = keep_larger == less(x, o) ? o : x;
    }
  }
  return x;
}

// A value and what tells it apart, for the sorts in 64 bits: larger values first, then lower ids.
struct Exact {
  double c;
  int id;
};
__device__ __forceinline__ bool behind(const Exact& a, const Exact& b) { return a.c < b.c || (a.c == b.c && a.id > b.id); }
__device__ __forceinline__ Exact sort_exact(Exact x, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const Exact o{__shfl_xor_sync(kAll, x.c, stride), __shfl_xor_sync(kAll, x.id, stride)};
      const bool keep_larger = ((lane & size) == 0) == ((lane & stride) == 0);
      if (keep_larger == behind(x, o)) x = o;
    }
  }
  return x;
}

// Lanes that share a group where the groups lie side by side on a warp (a power of two).
__device__ __forceinline__ int lanes_of_group(int groups) { return 1 << (31 - __clz(32 / groups)); }

// The whole selection in 64 bits, for the very rare tokens that the steps before leave open: lane j gets the j-th
// expert. A lane holds every lanes-th expert of one group. Values that are not numbers below infinity count as masked.
template <bool SOFTMAX>
__device__ __noinline__ int select_exactly(const Params& p, const float* row) {
  const int lane = static_cast<int>(lane_id());
  const int size = p.E / p.groups, lanes = lanes_of_group(p.groups), group = lane / lanes, sub = lane % lanes;
  const int n = group < p.groups ? (size - sub + lanes - 1) / lanes : 0;  // (at most 61)
  const auto id_of = [&](int i) { return group * size + sub + lanes * i; };
  // A padded row (equal logits, equal biases): the first experts, without any arithmetic.
  bool equal = row[0] < -neg_inf() && row[0] > neg_inf();
  for (int i = lane; i < p.E; i += 32) equal &= row[i] == row[0] && (!p.bias || p.bias[i] == p.bias[0]);
  if (__all_sync(kAll, equal && (!p.bias || fabsf(p.bias[0]) < -neg_inf()))) return lane;
  double c[64];
  float top = neg_inf();
  for (int i = 0; i < n; ++i) {
    const float l = row[id_of(i)];
    c[i] = l < -neg_inf() ? l : neg_inf();
    top = fmaxf(top, static_cast<float>(c[i]));
  }
  double total = 1.0;
  if (SOFTMAX) {
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    total = 0.0;
    for (int i = 0; i < n; ++i) total += c[i] > -1e300 ? exp(c[i] - top) : 0.0;
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  }
  const auto score = [&](double l) { return SOFTMAX ? exp(l - top) / total : 1.0 / (1.0 + exp(-l)); };
  unsigned long long taken = 0;
  for (int i = 0; i < n; ++i) {
    const float b = p.bias ? p.bias[id_of(i)] : 0.0f;
    if (!(c[i] > -1e300 && b < -neg_inf() && b > neg_inf())) c[i] = -INFINITY;
    else if (p.bias) c[i] = score(c[i]) + b;  // (without a bias the logits order the experts, which scores near one no longer can)
  }
  if (p.groups > 1) {
    double t1 = -INFINITY, t2 = -INFINITY;
    for (int i = 0; i < n; ++i) {
      if (c[i] > t1) t2 = t1, t1 = c[i];
      else if (c[i] > t2) t2 = c[i];
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const double x = __shfl_xor_sync(kAll, t1, o), y = __shfl_xor_sync(kAll, t2, o);
      t2 = fmax(fmin(t1, x), fmax(t2, y));
      t1 = fmax(t1, x);
    }
    if (!p.bias && p.group_top > 1) {
      t1 = t1 < -1e300 ? t1 : score(t1);
      t2 = t2 < -1e300 ? t2 : score(t2);
    }
    const double value = p.group_top > 1 && t2 > -1e300 ? t1 + t2 : t1;
    int rank = 0;
    for (int q = 0; q < p.groups; ++q) {
      const double v = __shfl_sync(kAll, value, q * lanes);
      rank += v > value || (v == value && q < group);
    }
    if (rank >= p.group_k) taken = ~0ull;
  }
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    Exact best{-INFINITY, 0x7FFFFFFF};
    int at = -1;
    for (int i = 0; i < n; ++i) {
      const Exact x{c[i], id_of(i)};
      if (!(taken >> i & 1) && (at < 0 || behind(best, x))) best = x, at = i;
    }
    const int own = best.id;
    for (int o = 16; o > 0; o >>= 1) {
      const Exact x{__shfl_xor_sync(kAll, best.c, o), __shfl_xor_sync(kAll, best.id, o)};
      if (behind(best, x)) best = x;
    }
    if (at >= 0 && own == best.id) taken |= 1ull << at;
    if (lane == j) mine = best.id;
  }
  return mine;
}

// What the groups' choice needs of one group's lanes, in 64 bits: the value of the group from its largest member, or its two largest,
// found again in `row_c` (the 32-bit values by expert; `tol`: how far apart those of members in the wrong order can be). False, on one of the
// group's lanes at least, where that leaves open which members they are.
template <bool SOFTMAX>
__device__ __noinline__ bool group_value_exactly(const Params& p, const float* row, const float* row_c, int size, int lanes, int group, int sub,
                                                 float t1, float t2, float tol, float top, float inv, double& value, double& scores) {
  const bool mine = group < p.groups && t1 > neg_inf();
  const auto exactly = [&](int at, double& s) {
    const int e = group * size + at;
    const double l = row[e];
    s = SOFTMAX ? exp(l - static_cast<double>(top)) * static_cast<double>(inv) : 1.0 / (1.0 + exp(-l));
    return p.bias ? s + static_cast<double>(p.bias[e]) : s;
  };
  value = -INFINITY, scores = 0.0;
  if (p.group_top == 1) {  // (only with a bias: logits need no rounding) the largest of all that could be
    double v = 0.0, s = 0.0;
    float seen_l = 0.0f, seen_b = 0.0f;  // (members of one logit and bias are computed once: padded rows)
    bool some = false, again = false;
    const auto meet = [&](auto use) {
      some = false;
      for (int i = sub; mine && i < size; i += lanes) {
        const int e = group * size + i;
        if (!(row_c[e] >= t1 - tol)) continue;
        const float l = row[e], b = p.bias[e];
        if (!some || l != seen_l || b != seen_b) v = exactly(i, s), seen_l = l, seen_b = b, some = true, use();
      }
    };
    meet([&] {
      if (v > value) value = v, scores = s;
    });
    for (int o = 1; o < lanes; o <<= 1) {
      const double x = __shfl_xor_sync(kAll, value, o), xs = __shfl_xor_sync(kAll, scores, o);
      if (x > value) value = x, scores = xs;
    }
    if (SOFTMAX)  // (the sum's rounding moves values by 2^-20 of their scores)
      meet([&] { again |= (s != scores || v != value) && value - v <= 0x1p-20 * fabs(s - scores) + 0x1p-45 * fabs(scores); });
    return !again;
  }
  int at1 = 0x7FFFFFFF, at2 = 0x7FFFFFFF, close = 0;
  for (int i = sub; mine && i < size; i += lanes)
    if (row_c[group * size + i] == t1) at1 = min(at1, i);
  for (int o = 1; o < lanes; o <<= 1) at1 = min(at1, __shfl_xor_sync(kAll, at1, o));
  for (int i = sub; mine && i < size; i += lanes) {
    const float c = row_c[group * size + i];
    if (c == t2 && i != at1) at2 = min(at2, i);
    close += c > neg_inf() && c >= t2 - tol;
  }
  for (int o = 1; o < lanes; o <<= 1) {
    at2 = min(at2, __shfl_xor_sync(kAll, at2, o));
    close += __shfl_xor_sync(kAll, close, o);
  }
  if (!mine) return true;
  double s1 = 0.0, s2 = 0.0;
  value = exactly(at1, s1);
  if (t2 > neg_inf()) value += exactly(at2, s2);
  scores = s1 + s2;
  return close <= 2;
}

// One warp routes one token; the logits are read once. Latency bounds it, at the 16 to 20 warps an SM that the row's registers allow, as much
// as instructions (2.15 of 4 a clock in groups, warps waiting for one another's shuffles and for memory): 16,384 tokens x 896 experts, 16 chosen,
// take 24 us from the logits alone, 32 with a bias, 44 in 8 groups, where the bytes would take 9; softmax 26 and 29; 24 of 896 for 4,096 tokens 18.
//
// The values that choose (score + bias, or the logits themselves without a bias) are held as order-preserving bits,
// NPL a lane, runs of four (VEC) or single ones spread over all lanes. Groups: the values pass through shared memory to lanes that lie
// by groups, which find each group's two largest and rank the groups by counting those ahead; the other groups' values
// are cleared. Of the lanes' maxima the (k+1)-th is a bound tau that at least k + 1 values reach; those that do (some twenty
// of 896 for k = 16) are sorted across the warp. Where more than 32 reach it (k above 18 or so), a bound that fewer reach is found by
// halving the distance to the largest value; where equal values leave none, k rounds of a warp-wide maximum (always in rounds: 34, 42 and 54 us,
// and 66 for 24 of 896).
//
// Which experts are chosen does not depend on the rounding here (65,000 random calls, half of them made to meet at fp32's rounding, against the
// definition in 64 bits: no other choice). A 32-bit score is within
// tol = 2^-21 s (2 + |l - m|) + 2^-22 |c| + 2^-126 of its value (the exponent's argument is rounded once, 2^-24 of it, the exponential and
// the reciprocal are right to 2 ulp, the sum over the experts to 4; m is the row's maximum, 0 for the sigmoid, where of a positive l only
// (1 - s) l counts, which is below 1). Where two
// neighbours in the order, or two groups, are nearer than that, all that could be meant are compared by values in 64
// bits. (A softmax keeps its 32-bit sum there, a common factor: only the scores' difference is uncertain by 2^-20 of itself,
// and where that is not enough either the token starts over in 64 bits: its warp takes some 110 us. Of
// random logits and biases one token in 100,000 does.) Two experts with the same logit and bias are
// equal in any precision and go by their index.
template <int NPL, bool VEC, bool SOFTMAX, bool GROUPED>
__global__ void __launch_bounds__(kWarps * 32, NPL < 28 ? 1 : GROUPED ? 4 : 5) route_scores_kernel(Params p) {
  extern __shared__ float pool[];
  __shared__ unsigned long long cand_s[kWarps][32];
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = static_cast<int>(lane_id()), wib = threadIdx.x >> 5;
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  const float* const row = p.logits + static_cast<size_t>(t) * E;
  const bool by_logit = p.bias == nullptr;
  const auto expert_of = [&](int i) { return VEC ? 128 * (i >> 2) + 4 * lane + (i & 3) : lane + 32 * i; };
  const auto here = [&](int i) { return VEC ? 128 * (i >> 2) + 4 * lane < E : lane + 32 * i < E; };

  const auto spread = [&](const float* from, float (&to)[NPL]) {  // a row over the lanes, 0 where there is nothing
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NPL / 4; ++i) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (here(4 * i)) x = __ldg(reinterpret_cast<const float4*>(from) + 32 * i + lane);
        to[4 * i] = x.x, to[4 * i + 1] = x.y, to[4 * i + 2] = x.z, to[4 * i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i) to[i] = here(i) ? __ldg(from + expert_of(i)) : 0.0f;
    }
  };
  const auto any_odd = [&](const float (&x)[NPL]) {  // an infinity or NaN in the row: only then is it looked at value by value
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < NPL; ++i) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return __any_sync(kAll, most >= 0x7F800000u) != 0;
  };

  float v[NPL];  // logits, then the values that choose
  spread(row, v);
  bool bad = false, odd = any_odd(v);
  if (odd) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      if (!(v[i] < -neg_inf())) {  // NaN and infinity: flagged, and as if masked
        bad = true;
        v[i] = neg_inf();
      }
    }
  }
  float top = neg_inf();
  if (SOFTMAX) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      if (!here(i)) v[i] = neg_inf();
      top = fmaxf(top, v[i]);
    }
  }
  float inv = 1.0f;
  if (SOFTMAX) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    top = top > neg_inf() ? top : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) sum += exp2_quick((v[i] - top) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  }
  const auto quick_score = [&](float l) {
    return SOFTMAX ? exp2_quick((l - top) * kLog2e) * inv : rcp_quick(1.0f + exp2_quick(-l * kLog2e));
  };
  uint32_t kv[NPL];  // 0: no expert of this lane
  if (!by_logit) {
    float b[NPL];
    spread(p.bias, b);
    if (any_odd(b)) odd = true;
    if (odd) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        bad |= !(b[i] < -neg_inf());
        v[i] = v[i] > neg_inf() && b[i] < -neg_inf() ? quick_score(v[i]) + b[i] : neg_inf();
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i) v[i] = quick_score(v[i]) + b[i];
    }
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) kv[i] = here(i) ? order_bits(v[i]) : 0u;
  if (odd && __any_sync(kAll, bad) && lane == 0) set_flag(p.err_flag, MOE_FLAG_NONFINITE);

  bool exact = false;  // whether the token starts over in 64 bits
  if (GROUPED) {
    const int size = E / p.groups, lanes = lanes_of_group(p.groups), group = lane / lanes, sub = lane % lanes;
    float* const row_c = pool + static_cast<size_t>(wib) * E;
#pragma unroll
    for (int i = 0; i < NPL; i += VEC ? 4 : 1) {
      if (!here(i)) continue;
      if (VEC) *reinterpret_cast<float4*>(row_c + expert_of(i)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      else row_c[expert_of(i)] = v[i];
    }
    __syncwarp();
    float t1 = neg_inf(), t2 = neg_inf();
    const auto meet = [&](float x) {
      t2 = fmaxf(t2, fminf(t1, x));
      t1 = fmaxf(t1, x);
    };
    if (group < p.groups) {
      const float* const from = row_c + group * size;
      if (VEC) {
#pragma unroll 4
        for (int i = 4 * sub; i < size; i += 4 * lanes) {
          const float4 x = *reinterpret_cast<const float4*>(from + i);
          meet(x.x), meet(x.y), meet(x.z), meet(x.w);
        }
      } else {
#pragma unroll 4
        for (int i = sub; i < size; i += lanes) meet(from[i]);
      }
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const float a = __shfl_xor_sync(kAll, t1, o), b = __shfl_xor_sync(kAll, t2, o);
      t2 = fmaxf(fminf(t1, a), fmaxf(t2, b));
      t1 = fmaxf(t1, a);
    }
    const bool sums = p.group_top > 1;
    float value = t1;
    if (by_logit && sums && t1 > neg_inf()) {
      value = quick_score(t1);
      if (t2 > neg_inf()) value += quick_score(t2);
    } else if (sums && t2 > neg_inf()) {
      value = t1 + t2;
    }
    int rank = 0;
    for (int q = 0; q < p.groups; ++q) {
      const float x = __shfl_sync(kAll, value, q * lanes);
      rank += x > value || (x == value && q < group);
    }
    const bool some = group < p.groups;
    bool keep = some && rank < p.group_k;
    unsigned kept = __ballot_sync(kAll, keep);  // a group's bit is that of its first lane
    // (scores are at most 1, with softmax at most the row's largest, and off by 2^-22 of that for every 2 of |l|: 2^-19 for two of them)
    const float slack = sums || !by_logit ? 0x1p-19f * (SOFTMAX ? fminf(1.0f, inv) : 1.0f) : 0.0f;
    // The last group that stays and the first that goes: too close to tell apart? (Where one is all masked they are not, and where none
    // goes `next` is NaN.) Each by as much as its roundings could have moved it: those of its terms, which may cancel; sums of two
    // biases may pass fp32.
    const float moved = 0x1p-21f * (by_logit ? value : sums && t2 > neg_inf() ? fmaxf(fabsf(t1), fabsf(t2)) : fabsf(t1));
    const float low = value > neg_inf() ? fmaxf(value - moved, -3.4028235e38f) : value, high = value > neg_inf() ? value + moved : value;
    const float least = bits_value(__reduce_min_sync(kAll, keep ? order_bits(low) : 0xFFFFFFFFu));
    const float next = bits_value(__reduce_max_sync(kAll, some && !keep ? order_bits(high) : 0u));
    const bool close = least - next <= slack || least == -neg_inf();
    if (slack > 0.0f && close && least > neg_inf() && next > neg_inf()) {
      double value64, scores;
      const float* const row_v = by_logit ? row : row_c;  // (where t1 and t2 were found)
      // (of two members each is off by its score's error, at most 5 x 2^-23 of the largest score, and the rounding of the sum with its bias)
      const float last = fabsf(sums ? t2 : t1), tol = by_logit ? last * 0x1p-20f + 0x1p-20f : slack + last * 0x1p-21f;
      const bool sure = group_value_exactly<SOFTMAX>(p, row, row_v, size, lanes, group, sub, t1, t2, tol, top, inv, value64, scores);
      int rank64 = 0;
      bool open = !sure;
      for (int q = 0; q < p.groups; ++q) {
        const double x = __shfl_sync(kAll, value64, q * lanes), xs = __shfl_sync(kAll, scores, q * lanes);
        rank64 += x > value64 || (x == value64 && q < group);
        if (SOFTMAX && q != group && x > -1e300 && fabs(x - value64) <= 0x1p-20 * fabs(xs - scores) + 0x1p-45 * fabs(xs)) open = true;
      }
      exact = __any_sync(kAll, open && some);
      keep = some && rank64 < p.group_k;
      kept = __ballot_sync(kAll, keep);
    }
    const float per = 1.0f / static_cast<float>(size);
#pragma unroll
    for (int i = 0; i < NPL; i += VEC ? 4 : 1) {  // (x + 1/2) / size is at least 2^-11 from a whole number, and x < 2^10: the cut is right
      const bool stays = here(i) && (kept >> (static_cast<int>((static_cast<float>(expert_of(i)) + 0.5f) * per) * lanes) & 1u);
#pragma unroll
      for (int j = 0; j < (VEC ? 4 : 1); ++j) kv[i + j] = stays ? kv[i + j] : 0u;
    }
  }
  const auto key_of = [&](int i) {
    return kv[i] ? (static_cast<unsigned long long>(kv[i]) << 32) | ~static_cast<uint32_t>(expert_of(i)) : 0ull;
  };
  // The experts whose bits reach `bound`, one a lane (0 past them); more than 32: none, and the count.
  const auto collect = [&](uint32_t bound, unsigned long long& key) {
    unsigned cand = 0u;
#pragma unroll
    for (int i = 0; i < NPL; ++i) cand |= kv[i] >= bound ? 1u << i : 0u;
    const int count = __popc(cand);
    int pos = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kAll, pos, o);
      if (lane >= o) pos += x;
    }
    const int total = __shfl_sync(kAll, pos, 31);
    if (total <= 32) {
      pos -= count;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (cand >> i & 1u) cand_s[wib][pos++] = (static_cast<unsigned long long>(kv[i]) << 32) | ~static_cast<uint32_t>(expert_of(i));
      __syncwarp();
      key = lane < total ? cand_s[wib][lane] : 0ull;
      __syncwarp();
    }
    return total;
  };

  unsigned long long mine = 0ull;  // lane j: the j-th expert's key
  if (!exact) {
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < NPL; ++i) most = max(most, kv[i]);
    const uint32_t sorted = sort_lanes(most, lane, [](uint32_t a, uint32_t b) { return a < b; });
    uint32_t tau = max(__shfl_sync(kAll, sorted, min(k, 31)), 1u);
    int total = collect(tau, mine);
    if (total > 32) {  // a bound that k to 32 values reach lies between tau and the largest value, unless equal ones straddle it
      uint32_t high = __shfl_sync(kAll, sorted, 0) + 1u;
      while (high - tau > 1u) {
        const uint32_t mid = tau + (high - tau) / 2u;
        int n = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) n += kv[i] >= mid;
        n = __reduce_add_sync(kAll, n);
        if (n < k) {
          high = mid;
        } else {
          tau = mid;
          if (n <= 32) break;
        }
      }
      total = collect(tau, mine);
    }
    const bool listed = total <= 32;
    if (listed) {
      mine = sort_lanes(mine, lane, [](unsigned long long a, unsigned long long b) { return a < b; });
    } else {
      unsigned taken = 0u;
      for (int j = 0; j < min(k + 1, 32); ++j) {
        unsigned long long best = 0ull;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const unsigned long long x = taken >> i & 1u ? 0ull : key_of(i);
          if (x > best) best = x, at = i;
        }
        const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(best >> 32));
        const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
        const unsigned long long m = static_cast<unsigned long long>(hi) << 32 | lo;
        if (m != 0ull && best == m) taken |= 1u << at;
        if (lane == j) mine = m;
      }
    }
    if (!by_logit) {
      // neighbours in the order, the first that is left out among them
      const auto tolerance = [&](float c, float l, float b) {  // (2^-126: scores below that are flushed to zero)
        return 0x1p-21f * fabsf(c - b) * (2.0f + fminf(SOFTMAX ? top - l : fmaxf(-l, fminf(l, 1.0f)), 1e38f)) + (0x1p-22f * fabsf(c) + 0x1p-126f);
      };
      const int listed_n = listed ? total : min(k + 1, 32);
      const float c = bits_value(static_cast<uint32_t>(mine >> 32));
      const bool real = mine != 0ull && c > neg_inf() && lane < listed_n;
      const int e = real ? static_cast<int>(~static_cast<uint32_t>(mine)) : 0;
      const float l = real ? __ldg(row + e) : 0.0f, b = real ? __ldg(p.bias + e) : 0.0f;
      const float tol = real ? tolerance(c, l, b) : 0.0f;
      const float nc = __shfl_down_sync(kAll, c, 1), nl = __shfl_down_sync(kAll, l, 1), nb = __shfl_down_sync(kAll, b, 1),
                  nt = __shfl_down_sync(kAll, tol, 1);
      const unsigned reals = __ballot_sync(kAll, real);
      const bool pair = real && (reals >> lane >> 1 & 1u);
      // what the last chosen one could be taken for: down to `reach`
      float wide = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(tol)));
      const float last = __shfl_sync(kAll, c, k - 1), reach = last - 2.0f * wide;
      bool near = pair && (lane + 1 < k || nc >= reach) && (nl != l || nb != b) && c - nc <= tol + nt;
      if (listed) {
        near |= last > neg_inf() && reach <= bits_value(tau);  // something below tau may be as near
      } else if (last > neg_inf()) {  // anything behind the list that differs from the last?
        const float ll = __shfl_sync(kAll, l, k - 1), lb = __shfl_sync(kAll, b, k - 1);
        for (int i = 0; i < NPL; ++i)
          if (kv[i] != 0u && bits_value(kv[i]) >= reach && bits_value(kv[i]) <= last) near |= row[expert_of(i)] != ll || p.bias[expert_of(i)] != lb;
      }
      // Below `reach` there may be one that is off by more than all that are listed: a large score and a bias that all but cancels it, beside
      // small scores. s (2 + |l - m|) is below 3, and below twice the largest score of a softmax.
      const float any = 3.0f * 0x1p-21f * (SOFTMAX ? fminf(1.0f, inv) : 1.0f) + 0x1p-22f * fabsf(last), deep = last - wide - any;
      if (last > neg_inf() && any > wide && (!listed || deep <= bits_value(tau))) {
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float x = bits_value(kv[i]);
          if (kv[i] == 0u || !(x >= deep) || x >= reach) continue;
          const float t = tolerance(x, __ldg(row + expert_of(i)), __ldg(p.bias + expert_of(i)));
          if (x + t >= last - wide) near = true, most = fmaxf(most, t);
        }
        wide = fmaxf(wide, __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(most))));
      }
      if (__any_sync(kAll, near)) {
        exact = true;
        unsigned long long key = 0ull;
        const int n = last > neg_inf() ? collect(order_bits(last - 4.0f * wide), key) : 33;
        if (n >= k && n <= 32) {  // all that could be among the first k, by their 64-bit values
          const bool some = lane < n;
          const int id = some ? static_cast<int>(~static_cast<uint32_t>(key)) : 0x7FFFFFFF;
          const double l64 = some ? row[id] : 0.0, b64 = some ? p.bias[id] : 0.0;
          const double s64 = SOFTMAX ? exp(l64 - static_cast<double>(top)) * static_cast<double>(inv) : 1.0 / (1.0 + exp(-l64));
          const Exact x = sort_exact(Exact{some ? s64 + b64 : -INFINITY, id}, lane);
          exact = false;
          if (SOFTMAX) {  // the sum's rounding moves neighbours by 2^-20 of their scores' difference
            const bool in = x.id != 0x7FFFFFFF;
            const float xl = in ? row[x.id] : 0.0f, xb = in ? p.bias[x.id] : 0.0f;
            const double y = __shfl_down_sync(kAll, x.c, 1);
            const float yl = __shfl_down_sync(kAll, xl, 1), yb = __shfl_down_sync(kAll, xb, 1);
            const bool open = lane + 1 < n && (xl != yl || xb != yb) && x.c - y <= 0x1p-20 * fabs(static_cast<double>(xb) - yb) + 0x1p-45 * fabs(x.c);
            exact = __any_sync(kAll, open);
          }
          mine = (1ull << 32) | ~static_cast<uint32_t>(x.id);
        }
      }
    }
  }
  int e = static_cast<int>(~static_cast<uint32_t>(mine));
  if (exact) e = select_exactly<SOFTMAX>(p, row);
  const bool out = lane < k;
  const float l = out ? row[e] : neg_inf();
  const float b = out && p.bias ? p.bias[e] : 0.0f;
  const bool masked = !(l < -neg_inf()) || l == neg_inf() || !(b < -neg_inf()) || b == neg_inf();
  // weights relative to the largest chosen score, which may be too small for fp32 itself
  float s = 0.0f, part = 0.0f;
  if (SOFTMAX) {
    float m = masked ? neg_inf() : l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    if (!masked) s = expf(l - top) * inv, part = expf(l - m);
  } else {
    float m = masked ? neg_inf() : fminf(l, 0.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    if (!masked) {
      const float d = 1.0f / (1.0f + expf(-fabsf(l)));
      s = expf(fminf(l, 0.0f)) * d, part = expf(fminf(l, 0.0f) - m) * d;
    }
  }
  float sum = part;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (out) {
    const size_t at = static_cast<size_t>(t) * k + lane;
    p.idx[at] = e;
    p.s[at] = s;
    p.w[at] = p.scale * (p.renorm ? (sum > 0.0f ? part / sum : 0.0f) : s);
  }
}

// Gradient of the logits from that of the weights, one warp a token:
//   renormalised  dl_j = w_j (g_j - sum_i w_i g_i / scale) (1 - s_j for the sigmoid), 0 for the others
//   sigmoid       dl_j = g_j w_j (1 - s_j), 0 for the others
//   softmax       dl_e = scale p_e (g_e [chosen] - sum_j s_j g_j), for which the logits are read again
// The row is written whole by all lanes, then the chosen entries over it by theirs. 1 - s of a sigmoid comes from the logit where the logits are
// given: from s itself it has lost 4 % at a logit of 14, and all above 17.
template <bool DENSE, bool SOFTMAX, bool FROM_LOGITS, typename OUT>
__global__ void __launch_bounds__(256) route_scores_bwd_kernel(RouteBwdArgs a) {
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= a.T) return;
  // the row's logits, on their way while the chosen ones are looked at
  const float* const l = a.logits + static_cast<size_t>(t) * a.E;
  // (1,024 experts at most: 8 runs of four a lane)
  float4 x[8];
  if (DENSE && a.E % 4 == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = make_float4(neg_inf(), neg_inf(), neg_inf(), neg_inf());
      if (4 * (lane + 32 * i) < a.E) x[i] = __ldg(reinterpret_cast<const float4*>(l) + lane + 32 * i);
    }
  } else if (DENSE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = 4 * (lane + 32 * i) + j;
        y[j] = at < a.E ? __ldg(l + at) : neg_inf();
      }
      x[i] = make_float4(y[0], y[1], y[2], y[3]);
    }
  }
  const size_t o = static_cast<size_t>(t) * a.k + lane;
  float gw = 0.0f, w = 0.0f, s = 0.0f, x_j = 0.0f;
  int e = -1 - lane;  // (different from one another)
  if (lane < a.k) {
    if (a.slot_of) {
      const int slot = __ldg(a.slot_of + o);
      if (slot >= 0 && slot < static_cast<long long>(a.T) * a.k) gw = __ldg(a.d_w + slot);
      else if (slot >= 0) set_flag(a.err_flag, MOE_FLAG_BAD_INDEX);
    } else {
      gw = __ldg(a.d_w + o);
    }
    w = __ldg(a.w + o);
    s = __ldg(a.s + o);
    const int id = __ldg(a.idx + o);
    if (a.d_topk_w) a.d_topk_w[o] = gw;
    if (id >= 0 && id < a.E) {
      e = id;
      if (FROM_LOGITS) x_j = __ldg(l + id);
    } else {
      set_flag(a.err_flag, MOE_FLAG_BAD_EXPERT);
      gw = 0.0f;
    }
  }
  const unsigned same = __match_any_sync(kAll, e);
  if (e >= 0 && (same & ((1u << lane) - 1u))) {  // named before in this row: flagged, and without a gradient
    set_flag(a.err_flag, MOE_FLAG_BAD_EXPERT);
    gw = 0.0f;
    e = -1 - lane;
  }
  float dot = (DENSE ? s : w) * gw;
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) dot += __shfl_xor_sync(kAll, dot, i);
  OUT* const row = static_cast<OUT*>(a.dL) + static_cast<size_t>(t) * a.E;
  const bool f32 = sizeof(OUT) == 4;
  const bool vec = a.E % (f32 ? 4 : 8) == 0;
  if (!DENSE) {
    if (vec) {
      uint4* const r4 = reinterpret_cast<uint4*>(row);
      for (int i = lane; i < a.E / (f32 ? 4 : 8); i += 32) r4[i] = make_uint4(0, 0, 0, 0);
    } else {
      for (int i = lane; i < a.E; i += 32) row[i] = OUT(0.0f);
    }
    __syncwarp();
    float d = gw * w;
    if (a.renorm) d = w * (gw - dot / a.scale);
    if (!SOFTMAX) d *= FROM_LOGITS && x_j < -neg_inf() ? 1.0f / (1.0f + expf(x_j)) : 1.0f - s;
    if (e >= 0) row[e] = OUT(d);
    return;
  }
  float top = neg_inf();
  const auto usable = [](float v) { return v < -neg_inf() ? v : neg_inf(); };  // as the forward reads them
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = make_float4(usable(x[i].x), usable(x[i].y), usable(x[i].z), usable(x[i].w));
    top = fmaxf(fmaxf(top, fmaxf(x[i].x, x[i].y)), fmaxf(x[i].z, x[i].w));
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, i));
  top = top > neg_inf() ? top : 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = make_float4(exp2_quick((x[i].x - top) * kLog2e), exp2_quick((x[i].y - top) * kLog2e), exp2_quick((x[i].z - top) * kLog2e),
                       exp2_quick((x[i].w - top) * kLog2e));
    sum += (x[i].x + x[i].y) + (x[i].z + x[i].w);
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(kAll, sum, i);
  const float f = sum > 0.0f ? -a.scale * dot / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = 4 * (lane + 32 * i);
    const float y[4] = {f * x[i].x, f * x[i].y, f * x[i].z, f * x[i].w};
    if (a.E % 4 == 0) {
      if (at < a.E) {
        if (f32) *reinterpret_cast<float4*>(row + at) = make_float4(y[0], y[1], y[2], y[3]);
        else *reinterpret_cast<uint2*>(row + at) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at + j < a.E) row[at + j] = OUT(y[j]);
    }
  }
  __syncwarp();
  if (e >= 0) row[e] = OUT(a.scale * s * (gw - dot));
}

template <int NPL, bool VEC, bool SOFTMAX>
cudaError_t route_launch(const Params& p, cudaStream_t st) {
  const unsigned grid = (static_cast<unsigned>(p.T) + kWarps - 1) / kWarps;
  if (p.groups > 1 && p.group_k < p.groups)
    route_scores_kernel<NPL, VEC, SOFTMAX, true><<<grid, kWarps * 32, static_cast<size_t>(kWarps) * p.E * 4, st>>>(p);
  else
    route_scores_kernel<NPL, VEC, SOFTMAX, false><<<grid, kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool VEC, bool SOFTMAX>
cudaError_t route_pick(const Params& p, cudaStream_t st) {
  const int npl = VEC ? (p.E + 127) / 128 * 4 : (p.E + 31) / 32;
  if (npl <= 4) return route_launch<4, VEC, SOFTMAX>(p, st);
  if (npl <= 8) return route_launch<8, VEC, SOFTMAX>(p, st);
  if (npl <= 16) return route_launch<16, VEC, SOFTMAX>(p, st);
  if (npl <= 28) return route_launch<28, VEC, SOFTMAX>(p, st);
  return route_launch<32, VEC, SOFTMAX>(p, st);
}

}  // namespace

cudaError_t launch_route_scores(const RouteArgs& a, cudaStream_t st) {
  LaunchTimer lt("route_scores", st);
  const Params p{a.logits, a.bias, a.T, a.E, a.k, a.groups, a.group_k, a.group_top, a.renorm, a.scale, a.idx, a.w, a.s, a.err_flag};
  const bool vec = a.E / a.groups % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.bias)) & 15u) == 0;
  if (a.softmax) return vec ? route_pick<true, true>(p, st) : route_pick<false, true>(p, st);
  return vec ? route_pick<true, false>(p, st) : route_pick<false, false>(p, st);
}

cudaError_t launch_route_scores_bwd(const RouteBwdArgs& a, cudaStream_t st) {
  LaunchTimer lt("route_scores_bwd", st);
  const unsigned grid = (static_cast<unsigned>(a.T) + 7) / 8;
  const bool dense = a.softmax && !a.renorm;
  const auto run = [&](auto f32, auto b16) {
    if (a.bf16_out) b16<<<grid, 256, 0, st>>>(a);
    else f32<<<grid, 256, 0, st>>>(a);
  };
  if (dense) run(route_scores_bwd_kernel<true, true, false, float>, route_scores_bwd_kernel<true, true, false, bf16>);
  else if (a.softmax) run(route_scores_bwd_kernel<false, true, false, float>, route_scores_bwd_kernel<false, true, false, bf16>);
  else if (a.logits) run(route_scores_bwd_kernel<false, false, true, float>, route_scores_bwd_kernel<false, false, true, bf16>);
  else run(route_scores_bwd_kernel<false, false, false, float>, route_scores_bwd_kernel<false, false, false, bf16>);
  return cudaGetLastError();
}

}  // namespace moe
