// Routing with sigmoid or softmax scores, a bias for balance and groups of experts, and its backward
// (route_permute.cu has the plain sigmoid form).
#include "common.cuh"
#include "mixer.h"
#include "timing.h"

namespace moe {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 8;      // tokens of a CTA, one for each warp
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xFF800000); }

// Order-preserving bits of a float (+0 and -0 are one value); 0 is below every number's.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float bits_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// How the experts of a token lie on the lanes: the groups side by side, `lanes` lanes each (a power of two), a
// lane holding every lanes-th expert (or every lanes-th run of four) of its group.
struct Layout {
  int size, lanes, group, sub;
  bool mine;  // whether this lane has a group
};

template <bool VEC>
__device__ __forceinline__ int place_in_group(const Layout& g, int i) {
  return VEC ? 4 * (g.sub + g.lanes * (i >> 2)) + (i & 3) : g.sub + g.lanes * i;
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

// The same selection in 64 bits, for the rare tokens whose 32-bit values are too close to tell apart: lane j gets the
// j-th expert. Values that are not numbers below infinity count as masked, as in the kernel.
template <bool SOFTMAX, bool VEC>
__device__ __noinline__ int select_exactly(const Params& p, const float* row, Layout g, int npl) {
  const int lane = static_cast<int>(lane_id());
  double c[64];
  float top = neg_inf();
  // A padded row (equal logits, equal biases): the first experts, without any arithmetic.
  bool equal = row[0] < -neg_inf() && row[0] > neg_inf();
  for (int i = lane; i < p.E; i += 32) equal &= row[i] == row[0] && (!p.bias || p.bias[i] == p.bias[0]);
  if (__all_sync(kAll, equal && (!p.bias || fabsf(p.bias[0]) < -neg_inf()))) return lane;
  for (int i = 0; i < npl; ++i) {
    const int at = place_in_group<VEC>(g, i);
    const float l = g.mine && at < g.size ? row[g.group * g.size + at] : neg_inf();
    c[i] = l < -neg_inf() ? l : neg_inf();
    top = fmaxf(top, static_cast<float>(c[i]));
  }
  double total = 1.0;
  if (SOFTMAX) {
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    total = 0.0;
    for (int i = 0; i < npl; ++i) total += c[i] > -1e300 ? exp(c[i] - top) : 0.0;
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  }
  unsigned long long taken = 0;
  for (int i = 0; i < npl; ++i) {
    const int at = place_in_group<VEC>(g, i);
    if (!g.mine || at >= g.size) {
      taken |= 1ull << i;
      continue;
    }
    const float b = p.bias ? p.bias[g.group * g.size + at] : 0.0f;
    if (c[i] > -1e300 && b < -neg_inf() && b > neg_inf()) {
      const double s = SOFTMAX ? exp(c[i] - top) / total : 1.0 / (1.0 + exp(-c[i]));
      // (without a bias the logits order the experts, which scores near one no longer can)
      c[i] = p.bias ? s + b : c[i];
    } else {
      c[i] = -INFINITY;
    }
  }
  if (p.groups > 1) {
    double t1 = -INFINITY, t2 = -INFINITY;
    for (int i = 0; i < npl; ++i) {
      if (taken >> i & 1) continue;
      if (c[i] > t1) t2 = t1, t1 = c[i];
      else if (c[i] > t2) t2 = c[i];
    }
    for (int o = 1; o < g.lanes; o <<= 1) {
      const double a = __shfl_xor_sync(kAll, t1, o), b = __shfl_xor_sync(kAll, t2, o);
      t2 = fmax(fmin(t1, a), fmax(t2, b));
      t1 = fmax(t1, a);
    }
    if (!p.bias) {
      const auto score = [&](double l) { return l < -1e300 ? l : SOFTMAX ? exp(l - top) / total : 1.0 / (1.0 + exp(-l)); };
      t1 = p.group_top == 1 ? t1 : score(t1);
      t2 = score(t2);
    }
    const double value = p.group_top > 1 && t2 > -1e300 ? t1 + t2 : t1;
    int rank = 0;
    for (int q = 0; q < p.groups; ++q) {
      const double v = __shfl_sync(kAll, value, q * g.lanes);
      rank += v > value || (v == value && q < g.group);
    }
    if (rank >= p.group_k) taken = ~0ull;
  }
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    double best = -INFINITY;
    int e = 0x7FFFFFFF, at = -1;
    for (int i = 0; i < npl; ++i) {
      const int id = g.group * g.size + place_in_group<VEC>(g, i);
      if (!(taken >> i & 1) && (c[i] > best || (c[i] == best && id < e))) best = c[i], e = id, at = i;
    }
    double top_c = best;
    int top_e = e;
    for (int o = 16; o > 0; o >>= 1) {
      const double oc = __shfl_xor_sync(kAll, top_c, o);
      const int oe = __shfl_xor_sync(kAll, top_e, o);
      if (oe != 0x7FFFFFFF && (top_e == 0x7FFFFFFF || oc > top_c || (oc == top_c && oe < top_e))) top_c = oc, top_e = oe;
    }
    if (e == top_e && at >= 0) taken |= 1ull << at;
    if (lane == j) mine = top_e;
  }
  return mine;
}

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

// One warp routes one token; the logits are read once and HBM bounds it.
//
// The values that choose (score + bias, or the logits themselves without a bias) are held as order-preserving bits,
// NPL a lane. Groups: a lane's two largest, joined over the group's lanes; each group is ranked by counting those
// ahead of it; the experts of the groups that stay are spread over all lanes by way of shared memory. Of the lanes'
// maxima the (k+1)-th is a bound tau that at least k + 1 values reach; those that do (some twenty of 896) are sorted
// across the warp. More than 32 of them, or too few lanes for the bound: k rounds of a warp-wide maximum.
//
// Which experts are chosen does not depend on the rounding here: a 32-bit score is within
// tol = 2^-21 s (2 + |l - m|) + 2^-22 |c| of its value (the exponent's argument is rounded once, 2^-24 of it, the exponential and
// the reciprocal are right to 2 ulp, the sum over the experts to 4; m is the row's maximum, 0 for the sigmoid), and where two
// neighbours in the order are nearer than that, the candidates are sorted again by their values in 64 bits. Two
// experts with the same logit and bias are equal in any precision and go by their index.
template <int NPL, bool VEC, bool SOFTMAX>
__global__ void __launch_bounds__(kWarps * 32) route_scores_kernel(Params p) {
  extern __shared__ uint32_t pool[];
  __shared__ unsigned long long cand_s[kWarps][32];
  __shared__ int kept_s[kWarps][32];
  const int t = (blockIdx.x * kWarps * 32 + threadIdx.x) >> 5;
  const int lane = static_cast<int>(lane_id()), wib = threadIdx.x >> 5;
  if (t >= p.T) return;
  const float* const row = p.logits + static_cast<size_t>(t) * p.E;
  Layout g;
  g.size = p.E / p.groups;
  g.lanes = 1 << (31 - __clz(32 / p.groups));
  g.group = lane / g.lanes;
  g.sub = lane % g.lanes;
  g.mine = g.group < p.groups;
  const int k = p.k;
  const bool by_logit = p.bias == nullptr;

  float v[NPL];  // logits, then the values that choose
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NPL; i += VEC ? 4 : 1) {
    const int at = place_in_group<VEC>(g, i);
    const bool in = g.mine && at < g.size;
    if (VEC) {
      float4 x = make_float4(neg_inf(), neg_inf(), neg_inf(), neg_inf());
      if (in) x = __ldg(reinterpret_cast<const float4*>(row + g.group * g.size + at));
      v[i] = x.x;
      if (i + 1 < NPL) v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
    } else {
      v[i] = in ? __ldg(row + g.group * g.size + at) : neg_inf();
    }
  }
  float top = neg_inf();
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if (!(v[i] < -neg_inf())) {  // NaN and infinity: flagged, and as if masked
      bad = true;
      v[i] = neg_inf();
    }
    if (SOFTMAX) top = fmaxf(top, v[i]);
  }
  float inv = 1.0f;
  if (SOFTMAX) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    top = top > neg_inf() ? top : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) sum += exp2f((v[i] - top) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  }
  const auto quick_score = [&](float l) {
    return SOFTMAX ? exp2f((l - top) * kLog2e) * inv : __fdividef(1.0f, 1.0f + __expf(-l));
  };
  uint32_t kv[NPL];  // 0: no expert of this lane
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int at = place_in_group<VEC>(g, i);
    const bool in = g.mine && at < g.size;
    if (!by_logit && in) {
      const float b = __ldg(p.bias + g.group * g.size + at);
      bad |= !(b < -neg_inf());
      const float s = quick_score(v[i]);
      v[i] = v[i] > neg_inf() && b < -neg_inf() ? s + b : neg_inf();
    }
    kv[i] = in ? order_bits(v[i]) : 0u;
  }
  if (__any_sync(kAll, bad) && lane == 0) set_flag(p.err_flag, MOE_FLAG_NONFINITE);

  bool exact = false;  // whether the order has to be found in 64 bits
  const bool grouped = p.groups > 1 && p.group_k < p.groups;
  if (grouped) {
    float t1 = neg_inf(), t2 = neg_inf();
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const float x = kv[i] ? v[i] : neg_inf();
      t2 = fmaxf(t2, fminf(t1, x));
      t1 = fmaxf(t1, x);
    }
    for (int o = 1; o < g.lanes; o <<= 1) {
      const float a = __shfl_xor_sync(kAll, t1, o), b = __shfl_xor_sync(kAll, t2, o);
      t2 = fmaxf(fminf(t1, a), fmaxf(t2, b));
      t1 = fmaxf(t1, a);
    }
    const bool sums = p.group_top > 1;
    float value = t1, slack = 0.0f;
    if (by_logit) {
      const float s1 = t1 > neg_inf() ? quick_score(t1) : t1, s2 = t2 > neg_inf() ? quick_score(t2) : t2;
      if (sums) value = s2 > neg_inf() ? s1 + s2 : s1;
    } else if (sums && t2 > neg_inf()) {
      value = t1 + t2;
    }
    // (a score is at most 1, with softmax at most the row's largest; two of them and the sum's rounding)
    if (sums || !by_logit) slack = 0x1p-18f * (SOFTMAX ? fminf(1.0f, inv) : 1.0f);
    int rank = 0;
    unsigned near = 0;  // groups whose value is too close to this one's to tell apart
    for (int q = 0; q < p.groups; ++q) {
      const float x = __shfl_sync(kAll, value, q * g.lanes), x1 = __shfl_sync(kAll, t1, q * g.lanes),
                  x2 = __shfl_sync(kAll, t2, q * g.lanes);
      rank += x > value || (x == value && q < g.group);
      const bool same = by_logit && x1 == t1 && x2 == t2;
      const float d = fabsf(x - value);  // (NaN where both are empty)
      if (slack > 0.0f && !same && d <= 2.0f * slack + 0x1p-21f * (fabsf(x) + fabsf(value)) && d < -neg_inf()) near |= 1u << q;
    }
    const bool keep = g.mine && rank < p.group_k;
    const unsigned kept_lanes = __ballot_sync(kAll, keep);
    unsigned kept = 0;  // by group
    for (int q = 0; q < p.groups; ++q) kept |= (kept_lanes >> (q * g.lanes) & 1u) << q;
    const unsigned groups_mask = p.groups < 32 ? (1u << p.groups) - 1u : kAll;
    exact = __any_sync(kAll, g.mine && (near & (keep ? groups_mask & ~kept : kept)));
    if (!exact) {
      // the experts of the groups that stay, over all lanes
      uint32_t* const mine = pool + static_cast<size_t>(wib) * p.group_k * g.size;
      const int order = __popc(kept & ((1u << g.group) - 1u));
      if (keep) {
        if (g.sub == 0) kept_s[wib][order] = g.group;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const int at = place_in_group<VEC>(g, i);
          if (at < g.size) mine[order * g.size + at] = kv[i];
        }
      }
      __syncwarp();
      const int n = p.group_k * g.size;
#pragma unroll
      for (int i = 0; i < NPL; ++i) kv[i] = 0u;
#pragma unroll
      for (int i = 0; i < (NPL < 32 ? NPL : 32); ++i)
        if (lane + 32 * i < n) kv[i] = mine[lane + 32 * i];
    }
  }
  const auto expert_of = [&](int i) {
    if (!grouped) return g.group * g.size + place_in_group<VEC>(g, i);
    const int at = lane + 32 * i, o = at / g.size;
    return kept_s[wib][o] * g.size + (at - o * g.size);
  };
  const auto key_of = [&](int i) {
    return kv[i] ? (static_cast<unsigned long long>(kv[i]) << 32) | ~static_cast<uint32_t>(expert_of(i)) : 0ull;
  };

  unsigned long long mine = 0ull;  // lane j: the j-th expert's key
  if (!exact) {
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < NPL; ++i) most = max(most, kv[i]);
    const uint32_t sorted = sort_lanes(most, lane, [](uint32_t a, uint32_t b) { return a < b; });
    const uint32_t tau = k < 32 ? __shfl_sync(kAll, sorted, k) : 0u;
    unsigned cand = 0u;
    unsigned cand_hi = 0u;
    int count = 0, total = 33;
    if (tau != 0u) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (kv[i] >= tau) (i < 32 ? cand : cand_hi) |= 1u << (i & 31);
      count = __popc(cand) + __popc(cand_hi);
      total = __reduce_add_sync(kAll, count);
    }
    bool listed = total <= 32;
    if (listed) {
      int pos = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kAll, pos, o);
        if (lane >= o) pos += x;
      }
      pos -= count;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if ((i < 32 ? cand : cand_hi) >> (i & 31) & 1u) cand_s[wib][pos++] = key_of(i);
      __syncwarp();
      mine = sort_lanes(lane < total ? cand_s[wib][lane] : 0ull, lane,
                        [](unsigned long long a, unsigned long long b) { return a < b; });
    } else {
      unsigned long long taken = 0ull;
      for (int j = 0; j < min(k + 1, 32); ++j) {
        unsigned long long best = 0ull;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const unsigned long long x = taken >> i & 1ull ? 0ull : key_of(i);
          if (x > best) best = x, at = i;
        }
        const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(best >> 32));
        const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
        const unsigned long long m = static_cast<unsigned long long>(hi) << 32 | lo;
        if (m != 0ull && best == m) taken |= 1ull << at;
        if (lane == j) mine = m;
      }
      if (!by_logit) {  // anything left near the last one that differs from it?
        const unsigned long long last = __shfl_sync(kAll, mine, k - 1);
        const float c = bits_value(static_cast<uint32_t>(last >> 32));
        const int e = static_cast<int>(~static_cast<uint32_t>(last));
        if (c > neg_inf()) {
          const float l = row[e], b = p.bias[e];
          const float tol = 0x1p-18f * (SOFTMAX ? fminf(1.0f, inv) : 1.0f) + 0x1p-20f * fabsf(c);
          bool near = false;
          for (int i = 0; i < NPL; ++i) {
            if (kv[i] == 0u || taken >> i & 1ull) continue;
            if (bits_value(kv[i]) >= c - tol) {
              const int o = expert_of(i);
              near |= row[o] != l || p.bias[o] != b;
            }
          }
          exact = __any_sync(kAll, near);
        }
      }
    }
    if (!by_logit && !exact) {
      // neighbours in the order, the first that is left out among them
      const int checked = min(k + 1, 32);
      const float c = bits_value(static_cast<uint32_t>(mine >> 32));
      const bool real = mine != 0ull && c > neg_inf() && lane < (listed ? total : checked);
      const int e = real ? static_cast<int>(~static_cast<uint32_t>(mine)) : 0;
      const float l = real ? __ldg(row + e) : 0.0f, b = real ? __ldg(p.bias + e) : 0.0f;
      const float tol = real ? 0x1p-21f * fabsf(c - b) * (2.0f + fabsf(l - (SOFTMAX ? top : 0.0f))) + 0x1p-22f * fabsf(c) : 0.0f;
      const float nc = __shfl_down_sync(kAll, c, 1), nl = __shfl_down_sync(kAll, l, 1), nb = __shfl_down_sync(kAll, b, 1),
                  nt = __shfl_down_sync(kAll, tol, 1);
      const bool next_real = __shfl_down_sync(kAll, static_cast<int>(real), 1) != 0 && lane < 31;
      const float wide = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(tol)));
      const float last = __shfl_sync(kAll, c, k - 1);
      const bool counts = lane + 1 < checked || last - c <= 2.0f * wide;
      const bool near = real && next_real && counts && (nl != l || nb != b) && c - nc <= tol + nt;
      const bool beyond = listed && last - bits_value(tau) <= 2.0f * wide;  // something below tau may be as near
      if (__any_sync(kAll, near) || beyond) {
        exact = true;
        if (listed && !SOFTMAX && !beyond) {
          // every expert that could be among the first k is a candidate: sort these by their 64-bit values
          const double c64 = real ? 1.0 / (1.0 + exp(-static_cast<double>(l))) + static_cast<double>(b) : -INFINITY;
          unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(c64 + 0.0));
          u = u ^ (static_cast<unsigned long long>(static_cast<long long>(u) >> 63) | 0x8000000000000000ull);
          int id = real ? e : 0x7FFFFFFF - lane;
          if (!real && mine != 0ull) id = static_cast<int>(~static_cast<uint32_t>(mine));
          if (mine == 0ull) u = 0ull;
#pragma unroll
          for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
            for (int stride = size >> 1; stride > 0; stride >>= 1) {
              const unsigned long long ou = __shfl_xor_sync(kAll, u, stride);
              const int oi = __shfl_xor_sync(kAll, id, stride);
              const bool keep_larger = ((lane & size) == 0) == ((lane & stride) == 0);
              const bool smaller = u < ou || (u == ou && id > oi);
              if (keep_larger == smaller) u = ou, id = oi;
            }
          }
          mine = (1ull << 32) | ~static_cast<uint32_t>(id);
          exact = false;
        }
      }
    }
  }
  int e = static_cast<int>(~static_cast<uint32_t>(mine));
  if (exact) e = select_exactly<SOFTMAX, VEC>(p, row, g, NPL);
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
// The row is written whole by all lanes, then the chosen entries over it by theirs.
template <bool DENSE, bool SOFTMAX, typename OUT>
__global__ void __launch_bounds__(256) route_scores_bwd_kernel(RouteBwdArgs a) {
  const int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= a.T) return;
  const size_t o = static_cast<size_t>(t) * a.k + lane;
  float gw = 0.0f, w = 0.0f, s = 0.0f;
  int e = -1 - lane;  // (different from one another)
  if (lane < a.k) {
    if (a.slot_of) {
      const int slot = __ldg(a.slot_of + o);
      gw = slot >= 0 ? __ldg(a.d_w + slot) : 0.0f;
    } else {
      gw = __ldg(a.d_w + o);
    }
    w = __ldg(a.w + o);
    s = __ldg(a.s + o);
    const int id = __ldg(a.idx + o);
    if (a.d_topk_w) a.d_topk_w[o] = gw;
    if (id >= 0 && id < a.E) {
      e = id;
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
    if (!SOFTMAX) d *= 1.0f - s;
    if (e >= 0) row[e] = OUT(d);
    return;
  }
  const float* const l = a.logits + static_cast<size_t>(t) * a.E;
  // (1,024 experts at most: 8 runs of four a lane)
  float4 x[8];
  float top = neg_inf();
  if (a.E % 4 == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = make_float4(neg_inf(), neg_inf(), neg_inf(), neg_inf());
      if (4 * (lane + 32 * i) < a.E) x[i] = __ldg(reinterpret_cast<const float4*>(l) + lane + 32 * i);
    }
  } else {
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
    x[i] = make_float4(exp2f((x[i].x - top) * kLog2e), exp2f((x[i].y - top) * kLog2e), exp2f((x[i].z - top) * kLog2e),
                       exp2f((x[i].w - top) * kLog2e));
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
  const bool grouped = p.groups > 1 && p.group_k < p.groups;
  const size_t smem = grouped ? static_cast<size_t>(kWarps) * p.group_k * (p.E / p.groups) * 4 : 0;
  route_scores_kernel<NPL, VEC, SOFTMAX><<<(p.T + kWarps - 1) / kWarps, kWarps * 32, smem, st>>>(p);
  return cudaGetLastError();
}

template <bool VEC, bool SOFTMAX>
cudaError_t route_pick(const Params& p, int npl, cudaStream_t st) {
  if (npl <= 4) return route_launch<4, VEC, SOFTMAX>(p, st);
  if (npl <= 8) return route_launch<8, VEC, SOFTMAX>(p, st);
  if (npl <= 16) return route_launch<16, VEC, SOFTMAX>(p, st);
  if (npl <= 28) return route_launch<28, VEC, SOFTMAX>(p, st);
  if (npl <= 32) return route_launch<32, VEC, SOFTMAX>(p, st);
  return route_launch<64, VEC, SOFTMAX>(p, st);
}

}  // namespace

cudaError_t launch_route_scores(const RouteArgs& a, cudaStream_t st) {
  LaunchTimer lt("route_scores", st);
  const Params p{a.logits, a.bias, a.T, a.E, a.k, a.groups, a.group_k, a.group_top, a.renorm, a.scale, a.idx, a.w, a.s, a.err_flag};
  const int size = a.E / a.groups;
  int lanes = 32;
  while (lanes * a.groups > 32) lanes >>= 1;
  const bool vec = size % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0;
  const int npl = vec ? 4 * ((size / 4 + lanes - 1) / lanes) : (size + lanes - 1) / lanes;
  if (a.softmax) return vec ? route_pick<true, true>(p, npl, st) : route_pick<false, true>(p, npl, st);
  return vec ? route_pick<true, false>(p, npl, st) : route_pick<false, false>(p, npl, st);
}

cudaError_t launch_route_scores_bwd(const RouteBwdArgs& a, cudaStream_t st) {
  LaunchTimer lt("route_scores_bwd", st);
  const unsigned grid = static_cast<unsigned>((a.T + 7) / 8);
  const bool dense = a.softmax && !a.renorm;
  const auto run = [&](auto f32, auto b16) {
    if (a.bf16_out) b16<<<grid, 256, 0, st>>>(a);
    else f32<<<grid, 256, 0, st>>>(a);
  };
  if (dense) run(route_scores_bwd_kernel<true, true, float>, route_scores_bwd_kernel<true, true, bf16>);
  else if (a.softmax) run(route_scores_bwd_kernel<false, true, float>, route_scores_bwd_kernel<false, true, bf16>);
  else run(route_scores_bwd_kernel<false, false, float>, route_scores_bwd_kernel<false, false, bf16>);
  return cudaGetLastError();
}

}  // namespace moe
