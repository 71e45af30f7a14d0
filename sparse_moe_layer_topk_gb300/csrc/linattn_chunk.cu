// Linear attention with a decay for each state head in chunks of 128 tokens, on
// the tcgen05 tensor cores: the forward and the three products of the backward
// are runs of one recurrence (linattn.h). With lam the head's decay, for a
// chunk of n tokens and the state S before it (forward order):
//   P   = (Q K^T) . L,  L_ij = lam^(i-j) for j <= i, else 0
//   O   = inter lam^(i+1) (Q S) + inter upd (P V)
//   S'  = lam^n S + upd sum_j (lam^(n-1-j) k_j) v_j^T
// and in reverse L_ij = lam^(j-i) for j >= i, lam^(n-1-i) for the rows, lam^(j+1)
// for the state's weights.
//
// One CTA walks the chunks of one sequence and state head (or of a segment of
// them), so the state never leaves the SM: per chunk it reads q, k, v and writes o once.
// Tokens arrive by TMA in tiles of 128 x width (128-byte swizzle). Warp roles:
//   warp 0       TMA producer over a ring of tile slots
//   warp 1       MMA issue: QK^T, QS, PV, K~^T V into four accumulators that fill
//                tensor memory (512 columns at width 128)
//   warp 2       stores of the output tiles that the score warps leave in shared memory
//   warps 4-11   scores: P out of tensor memory, times the decay factors, back as the
//                bf16 A operand of PV (in place); then the output rows
//   warps 12-19  state: the decayed keys K~ into shared memory; S in registers (fp32), its
//                bf16 copy as the B operand of QS
// Rounding: P and the copy of S that QS reads are bf16 (their error is that of the output's own
// rounding; with keys of up to 64 values, two bf16 terms). The state itself is summed in fp32 and K~
// enters the product as two bf16 terms (16 bits and a sign: 2.5e-6 of the state, rms; one term 1.7e-3),
// because the state is an output of the call and is carried over thousands of chunks. A chunk's sum
// starts from zero and is added in fp32 registers, not in tensor memory, whose accumulation truncates.
//
// Measured: 152 heads x 4,096 tokens, 128 wide (637 MB): 111 us, 5.7 TB/s, 0.85 of a plain copy's rate.
// 3.3 us a chunk: of its 6,200 clocks the shared-memory pipe is taken for 4,800 (operands 2,304, TMA in
// 768, K~ 768, the state's copy, the scores' tables and the output), the tensor cores work for 2,700, and
// the chain from a state to the next one (QS 830, keys 1,600, K~^T V 1,340, sum 600, copy 700, the waits
// between them) takes nearly all of them.

#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <utility>

#include "common.cuh"
#include "gemm.h"
#include "linattn.h"
#include "timing.h"

namespace moe {
namespace {

constexpr int C = 128;  // tokens of a chunk

// (unsigned: a length, or a bound given as "any", may lie within a chunk of 2^31)
__host__ __device__ constexpr int chunks_of(int tokens) { return static_cast<int>((static_cast<unsigned>(tokens) + C - 1) / C); }
constexpr int kScoreWarps = 8, kStateWarps = 8;
constexpr int kThreads = 128 + 32 * (kScoreWarps + kStateWarps);
// Registers a thread of each warpgroup; together no more than what the block is launched with
// (640 threads of 96).
constexpr int kIssueRegs = 80, kScoreRegs = 80, kStateRegs = 120;
static_assert(kIssueRegs + 2 * kScoreRegs + 2 * kStateRegs <= 5 * 96, "register split");

template <int DK, int DV>
struct Cfg {
  static constexpr int TK = C * DK * 2, TV = C * DV * 2;  // bytes of a q / k and of a v tile
  static constexpr int SLOT = TK > TV ? TK : TV;
  // P and the state's copy in two bf16 terms for keys of up to 64 values: the fewer values a product
  // sums, the less their rounding errors average out, and QS is short then.
  static constexpr int TERMS = DK <= 64 ? 2 : 1;
  // The state's sum has the wider of keys and values as its rows (the tensor memory's lanes, a thread
  // each): with 64 rows half of the lanes would be idle and the others have twice the columns.
  static constexpr bool BY_VALUE = DK < DV;
  static constexpr int ROWS = BY_VALUE ? DV : DK, COLS = BY_VALUE ? DK : DV;
  static constexpr int COPY = DK * DV * 2;  // a term of the state's copy
  static constexpr int MISC = 256 + 1024 + 768;  // barriers; decay factors and powers
  static constexpr int LIMIT = 232448 - 1024;
  // slots of the ring: what fits beside the state's copy
  static constexpr int FIT = (LIMIT - MISC - TERMS * COPY) / SLOT;
  static constexpr int SLOTS = FIT > 9 ? 9 : FIT;
  // the states alone: two places for second terms of the keys, the rest a ring of k and v
  static constexpr int SUM_FIT = (LIMIT - MISC) / SLOT;
  static constexpr int SUM_SLOTS = (SUM_FIT > 11 ? 11 : SUM_FIT) - 2;
  template <bool SO>
  static constexpr int SMEM = (SO ? (SUM_SLOTS + 2) * SLOT : SLOTS * SLOT + TERMS * COPY) + MISC + 1024;
  static_assert(SLOTS >= 6, "a chunk's three tiles and the next one's");
  // tensor memory columns
  static constexpr int P = 0, Z = 128, O1 = 256, O2 = 384;
};

struct Problem {
  CUtensorMap q, k, v, o;
  LinProblem p;
  // states at the segments' starts, [sequence][head][segment][dk * dv], element (i, j) at
  // i * seg_row + j * seg_col (null: one segment)
  float* seg;
  int seg_row, seg_col;
};

constexpr int kEven = 320;  // CTAs of an even split

struct Args {
  Problem prob[3];
  LinShape s;
  int nprob;
  int nseg;         // segments a sequence may have
  int seg_chunks;   // chunks of one
  int states_only;  // the segments' own sums alone, for the scan
  // even split: CTA i's state head << 8 | segment (n_even of them; 0: equal segments of every head)
  int n_even, even_chunks;
  uint16_t even[kEven];
};

// ------------------------------------------------------------------ powers of the decay

// exp(e * g) with the product's rounding error added back.
__device__ __forceinline__ float power(float g, int e) {
  if (e == 0) return 1.0f;
  const float fe = static_cast<float>(e);
  const float y = fe * g;
  const float x = expf(y);
  return x > 0.0f ? fmaf(x, fmaf(fe, g, -y), x) : 0.0f;
}

// The same as hi + lo: a state is multiplied by it once a chunk, and a rounding error
// of a factor near 1 would grow with the number of chunks.
__device__ __forceinline__ void power2(float g, int e, float& hi, float& lo) {
  const float fe = static_cast<float>(e);
  const float y = fe * g;
  if (!(y > -0.3f) || e == 0) {
    hi = power(g, e);
    lo = 0.0f;
    return;
  }
  float m = expm1f(y);
  m = fmaf(1.0f + m, fmaf(fe, g, -y), m);
  hi = 1.0f + m;
  lo = m - (hi - 1.0f);
}

__device__ __forceinline__ void store32(void* p, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Chunks that the first segment of state head h is short of: an even split (of one sequence) cuts the heads'
// chunks, laid one behind the other, into parts of seg_chunks.
__device__ __forceinline__ int first_short(int n_even, int even_chunks, int seg_chunks, int h) {
  return n_even ? static_cast<int>(static_cast<long long>(h) * even_chunks % seg_chunks) : 0;
}

// What a CTA works on.
struct Work {
  int prob, n, h, seg;
  int start, len;   // the sequence's tokens
  int chunks;       // of the whole sequence
  int c0, c1;       // this CTA's, in processing order
  bool last;        // it holds the sequence's last state
};

__device__ __forceinline__ bool find_work(const Args& a, Work& w) {
  int b = blockIdx.x;
  if (a.n_even) {
    w.prob = w.n = 0;
    w.h = a.even[b] >> 8;
    w.seg = a.even[b] & 255;
  } else {
    w.prob = b % a.nprob;
    b /= a.nprob;
    const int segs = a.states_only ? a.nseg - 1 : a.nseg;
    w.seg = b % segs;
    b /= segs;
    w.h = b % a.s.Hs;
    w.n = b / a.s.Hs;
  }
  lin_sequence(a.s, w.n, w.start, w.len);
  // (what follows from them is then uniform to the compiler, the MMA descriptors above all)
  w.start = __shfl_sync(0xFFFFFFFFu, w.start, 0);
  w.len = __shfl_sync(0xFFFFFFFFu, w.len, 0);
  if (w.len < 0) {
    if (threadIdx.x == 0 && w.seg == 0 && w.h == 0) set_flag(a.s.err_flag, MOE_FLAG_BAD_INDEX);
    return false;
  }
  w.chunks = chunks_of(w.len);
  const int c0 = w.seg * a.seg_chunks - first_short(a.n_even, a.even_chunks, a.seg_chunks, w.h);
  w.c0 = max(c0, 0);
  w.c1 = min(w.chunks, c0 + a.seg_chunks);
  w.last = w.c1 == w.chunks;
  if (a.states_only) return c0 + a.seg_chunks < w.chunks;  // a later segment starts from it
  return w.c0 < w.chunks || w.seg == 0;
}

// First token and token count of the c-th chunk in processing order.
__device__ __forceinline__ void chunk_at(const Work& w, int rev, int c, int& tok, int& n) {
  const int i = rev ? w.chunks - 1 - c : c;
  tok = w.start + i * C;
  n = min(C, w.len - i * C);
}

// The group's heads of each chunk in turn.
struct Item {
  int i = 0, sub = 0, c, group;
  __device__ __forceinline__ Item(const Work& w, int g) : c(w.c0), group(g) {}
  __device__ __forceinline__ void next() {
    ++i;
    if (++sub == group) {
      sub = 0;
      ++c;
    }
  }
};

struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// K~: rows 32 b0 .. 32 b1 - 1 of a k tile times the powers of the decay, as two bf16 terms in the
// places of k and of q (256 threads).
template <int DK>
__device__ __forceinline__ void decay_keys(uint8_t* tk, uint8_t* tq, const float* power_of, int rev, int n,
                                           int tid, int b0, int b1) {
  const int row0 = tid >> 3;  // a thread takes 16 bytes of rows row0 + 32 b
  const uint32_t at0 = row0 * 128 + (((tid & 7) ^ (row0 & 7)) << 4);
  const f32x2 minus = pack2(-1.0f, -1.0f);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int j = row0 + 32 * b;
    const float wt = j < n ? power_of[rev ? j + 1 : n - 1 - j] : 0.0f;
    const f32x2 wt2 = pack2(wt, wt);
    const uint32_t at = at0 + b * 4096;
    uint4 x[DK / 64];
#pragma unroll
    for (int c = 0; c < DK / 64; ++c) x[c] = *reinterpret_cast<const uint4*>(tk + at + c * C * 128);
#pragma unroll
    for (int c = 0; c < DK / 64; ++c) {
      if (j >= n) x[c] = make_uint4(0, 0, 0, 0);  // (possibly NaN)
      const uint32_t in[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
      uint32_t t0[4], t1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x2 v = mul2(pack2(bf16_lo(in[e]), bf16_hi(in[e])), wt2);
        t0[e] = pack_bf16(v);
        t1[e] = pack_bf16(fma2(pack2(bf16_lo(t0[e]), bf16_hi(t0[e])), minus, v));
      }
      *reinterpret_cast<uint4*>(tk + at + c * C * 128) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
      *reinterpret_cast<uint4*>(tq + at + c * C * 128) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
    }
  }
}

// Rows of a v tile past the chunk's n tokens are another sequence's, possibly NaN: zeros (256 threads).
template <int DV>
__device__ __forceinline__ void clear_values(uint8_t* tv, int n, int tid) {
#pragma unroll 1
  for (int x = n * 8 + tid; x < C * 8; x += 256) {
#pragma unroll
    for (int c = 0; c < DV / 64; ++c) *reinterpret_cast<uint4*>(tv + c * C * 128 + x * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// A CTA's chunks. SO: the states alone (the segments' own sums): the score warps decay the keys, with two
// places for their second terms, and k and v have the rest of shared memory (five tiles and not the four of a
// ring with q's place: 64 chunks of 96 CTAs 99 us instead of 111).
template <int DK, int DV, bool SO>
__device__ __forceinline__ void run_chunks(const Args& a, const Work& w, uint8_t* smem_raw) {
  using F = Cfg<DK, DV>;
  const LinProblem& p = a.prob[w.prob].p;

  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int SLOTS = SO ? F::SUM_SLOTS : F::SLOTS;
  uint8_t* const copy = smem + SLOTS * F::SLOT;  // the state in bf16 (the states alone: second terms of the keys)
  // A wait tells a phase from the next one alone, so no barrier may complete twice before each of its
  // waiters has returned: every phase is waited for, and the next one needs an arrival made after that.
  uint64_t* const full = reinterpret_cast<uint64_t*>(copy + (SO ? 2 * F::SLOT : F::TERMS * F::COPY));
  uint64_t* const empty = full + SLOTS;
  uint64_t* const p_full = empty + SLOTS;   // QK^T done
  // QS done: the q tile may be overwritten (with each set of keys; states alone: a set has entered)
  uint64_t* const qs_done = p_full + 1;
  uint64_t* const p_ready = p_full + 2;        // P back in tensor memory
  uint64_t* const o_full = p_full + 3;
  uint64_t* const o_empty = p_full + 4;
  uint64_t* const k_ready = p_full + 5;        // decayed keys written
  uint64_t* const z_full = p_full + 6;         // the chunk's sum of keys and values
  uint64_t* const s_ready = p_full + 7;        // the state's copy written, Z read
  uint64_t* const o_gone = p_full + 8;         // the output has left its staging place
  uint64_t* const drain = p_full + 9;
  uint64_t* const o_staged = p_full + 10;      // three, used in turn
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(p_full + 13);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // factor[128 + j - i] is L_ij, zero outside the mask; power_of[m] = lam^m, 0 <= m <= 128;
  // falling[m] = lam^(15-m), 0 <= m < 16
  float* const factor = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + 256);
  float* const power_of = factor + 2 * C;
  float* const falling = power_of + C + 4;

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);  // (uniform to the compiler)
  const int lane = static_cast<int>(lane_id());
  if (threadIdx.x == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(p_full, 1);
    mbar_init(qs_done, 1);
    mbar_init(p_ready, kScoreWarps);
    mbar_init(o_full, 1);
    mbar_init(o_empty, kScoreWarps);
    mbar_init(k_ready, SO ? kScoreWarps : kStateWarps + kScoreWarps);
    mbar_init(z_full, 1);
    mbar_init(s_ready, kStateWarps);
    mbar_init(o_gone, 1);
    for (int i = 0; i < 3; ++i) mbar_init(&o_staged[i], kScoreWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&a.prob[w.prob].q);
    tma_prefetch_desc(&a.prob[w.prob].k);
    tma_prefetch_desc(&a.prob[w.prob].v);
    tma_prefetch_desc(&a.prob[w.prob].o);
  }
  const float log_decay = __ldg(a.s.log_decay + w.h);
  if (threadIdx.x >= kThreads - C) {
    const int m = threadIdx.x - (kThreads - C);
    const float g = fminf(log_decay, 0.0f);
    const float x = power(g, m);
    power_of[m] = x;
    factor[p.rev ? C + m : C - m] = x;
    if (m > 0) factor[p.rev ? C - m : C + m] = 0.0f;
    if (m < 16) falling[15 - m] = x;
    if (m == 0) {
      factor[0] = 0.0f;
      power_of[C] = power(g, C);
      if (!(log_decay <= 0.0f)) set_flag(a.s.err_flag, MOE_FLAG_NONFINITE);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);

  // Items: the group's query heads (or key / value heads) of each chunk in turn.
  constexpr bool so = SO;
  const int group = so ? p.nkv : max(p.nq, p.nkv);
  const bool many_q = group > 1 && p.nq > 1;
  const int items = (w.c1 - w.c0) * group;
  // per item: QS and a new PV sum start with the first of a shared output, the
  // output ends with the last; the keys of a shared state enter with the last query head
  const auto first_q = [&](int sub) { return many_q || sub == 0; };
  const auto last_q = [&](int sub) { return many_q || sub == group - 1; };
  const auto adds_k = [&](int sub) { return !many_q || sub == group - 1; };
  // At widths of 128 a whole chunk's output rows leave through shared memory and a TMA store (stores of one
  // row a lane take 1,024 clocks of the shared-memory pipe a chunk): through the place of the state's
  // copy, which is idle from the chunk's last QS to the next state, or, while another query head's QS is
  // to read that, through the item's q tile. (At narrower widths the copy is sooner done and would wait
  // for the store: 152 heads x 4,096 tokens, 64 wide, 84 us, staged 87.)
  constexpr bool STAGED = DK == C && DV == C;
  static_assert(!STAGED || F::COPY >= C * DV * 2, "room for an output tile");
  const auto staged = [&](int n) { return STAGED && n == C; };
  const auto in_q = [&](int sub, int n) { return staged(n) && many_q && sub < group - 1; };
  const auto fail = [&]() {
    *abort_flag = 1;
    set_flag(a.s.err_flag, MOE_FLAG_TIMEOUT);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
      if (elect_one()) {
        Ring r;
        long long issued = 0;
        bool ok = true;
        for (Item it(w, group); it.i < items && ok; it.next()) {
          const int sub = it.sub;
          int tok, n;
          chunk_at(w, p.rev, it.c, tok, n);
          const int hq = p.nq > 1 ? w.h * p.nq + sub : w.h;
          const int hk = p.nkv > 1 ? w.h * p.nkv + sub : w.h;
          for (int t = so ? 1 : 0; t < 3; ++t) {
            if (!mbar_wait_short(&empty[r.slot], r.phase ^ 1u)) {
              fail();
              ok = false;
              break;
            }
            const CUtensorMap* m = t == 0 ? &a.prob[w.prob].q : t == 1 ? &a.prob[w.prob].k : &a.prob[w.prob].v;
            const int width = t == 2 ? DV : DK;
            const uint32_t dst = smem_u32(smem + r.slot * F::SLOT);
            mbar_arrive_expect_tx(&full[r.slot], C * width * 2);
            for (int c = 0; c < width / 64; ++c)
              tma_load_3d(dst + c * C * 128, m, &full[r.slot], 64 * c, tok, t == 0 ? hq : hk);
            ++issued;
            r.next(SLOTS);
          }
        }
        if (ok) {
          // the last commits must not reach this CTA's barriers after it left
          for (int i = 0; i < SLOTS; ++i) {
            if (!mbar_wait_short(&empty[r.slot], r.phase ^ 1u)) {
              fail();
              break;
            }
            r.next(SLOTS);
          }
        } else {
          // nothing may land in shared memory after the CTA left
          int s = r.slot;
          uint32_t ph = r.phase;
          for (long long i = 0; i < issued && i < SLOTS; ++i) {
            if (--s < 0) {
              s = SLOTS - 1;
              ph ^= 1u;
            }
            mbar_wait_short(&full[s], ph);
          }
        }
      }
    } else if (warp == 2) {
      // Stores the staged outputs. (Before the fourth is staged the first one's place was given back.)
      if (!so && STAGED && elect_one()) {
        Ring r;
        int n_st = 0;
        for (Item it(w, group); it.i < items; it.next()) {
          const int rq = r.slot;
          r.next(SLOTS);
          r.next(SLOTS);
          r.next(SLOTS);
          int tok, n;
          chunk_at(w, p.rev, it.c, tok, n);
          if (!last_q(it.sub) || !staged(n)) continue;
          if (!mbar_wait_short(&o_staged[n_st % 3], n_st / 3 & 1)) {
            fail();
            break;
          }
          ++n_st;
          const bool q_place = in_q(it.sub, n);
          const uint32_t from = smem_u32(q_place ? smem + rq * F::SLOT : copy);
          const int hq = p.nq > 1 ? w.h * p.nq + it.sub : w.h;
          for (int c = 0; c < DV / 64; ++c) tma_store_3d(&a.prob[w.prob].o, from + c * C * 128, 64 * c, tok, hq);
          bulk_commit();
          bulk_wait_read_all();
          mbar_arrive(q_place ? &empty[rq] : o_gone);
        }
        bulk_wait_all();
      }
    } else if (warp == 1) {
      // The whole warp walks the items and one lane issues, batch by batch: the descriptors then
      // stay in uniform registers and an MMA of 128 x 128 x 16 issues in 67 clocks (a single
      // thread's loop took over 100).
      {
        const uint32_t i_qk = make_idesc_bf16(C, C, 0, 0), i_qs = make_idesc_bf16(C, DV, 0, F::BY_VALUE ? 0 : 1);
        const uint32_t i_pv = make_idesc_bf16(C, DV, 0, 1), i_kv = make_idesc_bf16(F::ROWS, F::COLS, 1, 1);
        Ring r, rn;  // the item's first slot, and that of the next one's q
        uint32_t n_o = 0, n_s = 0, n_k = 0;  // outputs, states, key sets so far
        bool ok = true;
        const auto wait = [&](uint64_t* b, uint32_t parity) {
          if (ok && !__all_sync(0xFFFFFFFFu, mbar_wait_short(b, parity & 1u))) {
            fail();
            ok = false;
          }
        };
        const auto scores = [&]() {  // QK^T of the item whose q is in slot rn
          const uint32_t sq = smem_u32(smem + rn.slot * F::SLOT);
          wait(&full[rn.slot], rn.phase);
          rn.next(SLOTS);
          const uint32_t sk = smem_u32(smem + rn.slot * F::SLOT);
          wait(&full[rn.slot], rn.phase);
          rn.next(SLOTS);
          rn.next(SLOTS);
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C * 128 + (kk & 3) * 32;
              mma_bf16_ss(tmem + F::P, make_sdesc(sq + off, 16, 1024), make_sdesc(sk + off, 16, 1024),
                          i_qk, kk != 0);
            }
            mma_commit(p_full);
          }
          __syncwarp();
        };
        if (!so && items > 0) scores();
        for (Item it(w, group); it.i < items && ok; it.next()) {
          const int i = it.i, sub = it.sub;
          bool early = false;
          int tok, n;
          chunk_at(w, p.rev, it.c, tok, n);
          const Ring rq = r;
          if (!so) r.next(SLOTS);
          const Ring rk = r;
          r.next(SLOTS);
          const Ring rv = r;
          r.next(SLOTS);
          // (the second terms of the keys take the place of q)
          const uint32_t sq = smem_u32(so ? copy + (i & 1) * F::SLOT : smem + rq.slot * F::SLOT), sk = smem_u32(smem + rk.slot * F::SLOT),
                         sv = smem_u32(smem + rv.slot * F::SLOT);
          if (!so) {
            if (first_q(sub)) {
              wait(s_ready, n_s);       // the state before this chunk
              wait(o_empty, n_o ^ 1u);  // the previous output read
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int t = 0; t < F::TERMS; ++t)
#pragma unroll
                  for (int kk = 0; kk < DK / 16; ++kk)
                    mma_bf16_ss(tmem + F::O1, make_sdesc(sq + (kk >> 2) * C * 128 + (kk & 3) * 32, 16, 1024),
                                F::BY_VALUE ? make_sdesc(smem_u32(copy) + t * F::COPY + kk * 32, 16, 1024)
                                            : make_sdesc(smem_u32(copy) + t * F::COPY + kk * 2048, DK * 128, 1024), i_qs,
                                t != 0 || kk != 0);
              }
              __syncwarp();
            }
            if (adds_k(sub) && elect_one()) mma_commit(qs_done);
            __syncwarp();
            wait(&full[rv.slot], rv.phase);
            wait(p_ready, i);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int t = 0; t < F::TERMS; ++t)
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                  mma_bf16_ts(tmem + F::O2, tmem + F::P + kk * 16 + t * 8, make_sdesc(sv + kk * 2048, C * 128, 1024),
                              i_pv, t != 0 || kk != 0 || !first_q(sub));
              if (last_q(sub)) mma_commit(o_full);
            }
            __syncwarp();
            if (last_q(sub)) ++n_o;
            // the next item's scores before this one's keys enter, if its tiles are there
            if (i + 1 < items) {
              Ring x = rn;
              x.next(SLOTS);
              early = __all_sync(0xFFFFFFFFu, mbar_test(&full[rn.slot], rn.phase) && mbar_test(&full[x.slot], x.phase));
              if (early) scores();
            }
          }
          if (adds_k(sub)) {
            if (so) wait(&full[rv.slot], rv.phase);
            wait(s_ready, n_s);  // (the sum of the chunk before was read)
            wait(k_ready, n_k);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 2 * C / 16; ++kk) {
                const uint64_t keys = make_sdesc((kk < C / 16 ? sk : sq) + (kk & 7) * 2048, C * 128, 1024);
                const uint64_t values = make_sdesc(sv + (kk & 7) * 2048, C * 128, 1024);
                mma_bf16_ss(tmem + F::Z, F::BY_VALUE ? values : keys, F::BY_VALUE ? keys : values, i_kv,
                            kk != 0 || !(many_q || sub == 0));
              }
              if (so) mma_commit(qs_done);
              if (sub == group - 1) mma_commit(z_full);
            }
            __syncwarp();
            ++n_k;
          }
          if (sub == group - 1) ++n_s;
          if (elect_one()) {
            if (!so && !in_q(sub, n)) mma_commit(&empty[rq.slot]);
            mma_commit(&empty[rk.slot]);
            mma_commit(&empty[rv.slot]);
          }
          __syncwarp();
          if (!so && !early && i + 1 < items) scores();
        }
        if (*abort_flag) {
          // every issued MMA ends before tensor memory is released
          if (elect_one()) mma_commit(drain);
          __syncwarp();
          mbar_wait_short(drain, 0);
        }
      }
    }
    __syncwarp();
  } else if (warp < 4 + kScoreWarps) {
    // ---------------------------------------------------------------- score warps
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kScoreRegs));
    const int qd = warp & 3;  // tensor memory lanes 32 qd .. 32 qd + 31: rows of the chunk
    const int half = (warp - 4) >> 2;  // half of the scores' and of the output's columns
    const int row = 32 * qd + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * qd) << 16);
    const f32x2 intra = pack2(p.inter * p.upd, p.inter * p.upd);
    const bool wide = (p.ldo % 16 == 0) && (p.dv % 16 == 0) && (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0;
    const int tid = threadIdx.x - 128;
    uint32_t n_o = 0, n_k = 0;
    int n_st = 0;
    Ring r;
    if (so) {
      // the segments' own sums: these warps prepare the keys, the state warps sum
      for (Item it(w, group); it.i < items; it.next()) {
        int tok, n;
        chunk_at(w, p.rev, it.c, tok, n);
        const Ring rk = r;
        r.next(SLOTS);
        const Ring rv = r;
        r.next(SLOTS);
        bool ok = mbar_wait_short(&full[rk.slot], rk.phase);
        if (ok && n < C) {
          ok = mbar_wait_short(&full[rv.slot], rv.phase);
          if (ok) clear_values<DV>(smem + rv.slot * F::SLOT, n, tid);
        }
        if (ok) decay_keys<DK>(smem + rk.slot * F::SLOT, copy + (it.i & 1) * F::SLOT, power_of, p.rev, n, tid, 0, 4);
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && n_k > 0) ok = mbar_wait_short(qs_done, (n_k - 1) & 1);  // (no more than one set ahead)
        if (!ok) {
          fail();
          break;
        }
        if (lane == 0) mbar_arrive(k_ready);
        ++n_k;
      }
    }
    for (Item it(w, group); it.i < items && !so; it.next()) {
      const int i = it.i, sub = it.sub;
      int tok, n;
      chunk_at(w, p.rev, it.c, tok, n);
      const int rq = r.slot;
      r.next(SLOTS);
      const int rk = r.slot;
      r.next(SLOTS);
      const Ring rv = r;
      r.next(SLOTS);
      if (n < C) {
        if (!mbar_wait_short(&full[rv.slot], rv.phase)) {
          fail();
          break;
        }
        clear_values<DV>(smem + rv.slot * F::SLOT, n, tid);
      }
      if (!mbar_wait_short(p_full, i & 1)) {
        fail();
        break;
      }
      tc_fence_after();
      // P: 16 fp32 columns become 8 of bf16 pairs, and 8 of their second term, in place
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        const int c0 = 64 * half + 16 * b;
        uint32_t out[F::TERMS][8];
        if (p.rev ? c0 + 16 > 32 * qd : c0 < 32 * qd + 32) {
          uint32_t x[16];
          tmem_ld_32x32b_x16(trow + F::P + c0, x);
          float y[16];  // (the factors are read while the scores are on their way)
          if (c0 >> 5 == qd) {
            // selected, not multiplied by zero: what lies outside the mask may be NaN
            const float* const f = factor + C - row + c0;
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = f[j];
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = y[j] > 0.0f ? __uint_as_float(x[j]) * y[j] : 0.0f;
          } else {
            // beside the diagonal blocks lam^|i-j| is the power of the row's distance from the 16
            // columns' near edge times that of the column's
            const float d = power_of[p.rev ? c0 - row : row - c0 - 15];
            const f32x2 d2 = pack2(d, d);
            const float4* const e = reinterpret_cast<const float4*>(p.rev ? power_of : falling);
            f32x2 f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 e4 = e[j];
              f[2 * j] = mul2(pack2(e4.x, e4.y), d2);
              f[2 * j + 1] = mul2(pack2(e4.z, e4.w), d2);
            }
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              unpack2(mul2(pack2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), f[j]), y[2 * j], y[2 * j + 1]);
          }
          if (p.rev && c0 + 16 > n) {  // keys past the chunk's tokens
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = c0 + j < n ? y[j] : 0.0f;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            out[0][j] = pack_bf16(y[2 * j], y[2 * j + 1]);
            if (F::TERMS == 2)
              out[F::TERMS - 1][j] = pack_bf16(fma2(pack2(bf16_lo(out[0][j]), bf16_hi(out[0][j])), pack2(-1.0f, -1.0f),
                                                    pack2(y[2 * j], y[2 * j + 1])));
          }
        } else {
#pragma unroll
          for (int t = 0; t < F::TERMS; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) out[t][j] = 0u;
        }
#pragma unroll
        for (int t = 0; t < F::TERMS; ++t) tmem_st_32x32b_x8(trow + F::P + c0 + 8 * t, out[t]);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);
      // half of the keys, once QS has read the q tile
      if (adds_k(sub)) {
        if (!mbar_wait_short(qs_done, n_k++ & 1)) {
          fail();
          break;
        }
        decay_keys<DK>(smem + rk * F::SLOT, smem + rq * F::SLOT, power_of, p.rev, n, tid, 2, 4);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_ready);
      }
      if (!last_q(sub)) continue;
      if (!mbar_wait_short(o_full, n_o & 1)) {
        fail();
        break;
      }
      ++n_o;
      tc_fence_after();
      const float rsf = p.inter * power_of[p.rev ? max(n - 1 - row, 0) : row + 1];
      const f32x2 rs = pack2(rsf, rsf);
      const int hq = p.nq > 1 ? w.h * p.nq + sub : w.h;
      bf16* const orow = static_cast<bf16*>(p.o) + (static_cast<long long>(tok) + row) * p.ldo +
                         static_cast<long long>(hq) * p.dv;
#pragma unroll 1
      for (int b = 0; b < DV / 32; ++b) {
        const int c0 = half * (DV / 2) + 16 * b;
        uint32_t x1[16], x2[16];
        tmem_ld_32x32b_x16(trow + F::O1 + c0, x1);
        tmem_ld_32x32b_x16(trow + F::O2 + c0, x2);
        tmem_ld_wait();
        if (b == DV / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty);
        }
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          u[j] = pack_bf16(fma2(rs, pack2(__uint_as_float(x1[2 * j]), __uint_as_float(x1[2 * j + 1])),
                                mul2(intra, pack2(__uint_as_float(x2[2 * j]), __uint_as_float(x2[2 * j + 1])))));
        const uint4 lo4 = make_uint4(u[0], u[1], u[2], u[3]), hi4 = make_uint4(u[4], u[5], u[6], u[7]);
        if (staged(n)) {
          uint8_t* const line = (in_q(sub, n) ? smem + rq * F::SLOT : copy) + (c0 >> 6) * C * 128 + row * 128;
          const int at = (c0 & 63) >> 3, sw = row & 7;
          *reinterpret_cast<uint4*>(line + ((at ^ sw) << 4)) = lo4;
          *reinterpret_cast<uint4*>(line + (((at + 1) ^ sw) << 4)) = hi4;
        } else if (row < n) {
          if (wide && c0 + 16 <= p.dv) {
            store32(orow + c0, lo4, hi4);
          } else {
            if (c0 + 8 <= p.dv) *reinterpret_cast<uint4*>(orow + c0) = lo4;
            if (c0 + 16 <= p.dv) *reinterpret_cast<uint4*>(orow + c0 + 8) = hi4;
          }
        }
      }
      if (staged(n)) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_staged[n_st % 3]);
        ++n_st;
      }
    }
  } else {
    // ---------------------------------------------------------------- state warps
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
    const int tid = threadIdx.x - 128 - 32 * kScoreWarps;
    const float g = fminf(log_decay, 0.0f);
    constexpr int NC = F::COLS / 2;  // columns of a thread
    const int qd = warp & 3, half = (warp - 4 - kScoreWarps) >> 2;
    const bool mine = F::ROWS == 128 || lane < 16;
    const int row = F::ROWS == 128 ? 32 * qd + lane : 16 * qd + (lane & 15);
    const int rows = F::BY_VALUE ? p.dv : p.dk, cols = F::BY_VALUE ? p.dk : p.dv;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * qd) << 16) + F::Z + half * NC;
    f32x2 S[NC / 2];
    const long long state = (static_cast<long long>(w.n) * a.s.Hs + w.h) * p.dk * p.dv;
    const Problem& pr = a.prob[w.prob];
    float* const seg = pr.seg == nullptr ? nullptr
        : pr.seg + ((static_cast<long long>(w.n) * a.s.Hs + w.h) * a.nseg + w.seg) * p.dk * p.dv;
    {
      if (!so && seg) wait_for_last_kernel();  // (until here the CTA needs no state)
      const float* in = so ? nullptr : seg ? seg : p.s_in ? p.s_in + state : nullptr;
      const int sk = seg ? pr.seg_row : p.s_row, sv = seg ? pr.seg_col : p.s_col;
      const int sr = F::BY_VALUE ? sv : sk, sc = F::BY_VALUE ? sk : sv;
      const float* const at = in + static_cast<long long>(row) * sr;
      const bool have = in && mine && row < rows;
      if (sc == 1) {
#pragma unroll
        for (int j = 0; j < NC / 8; ++j) {
          float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          const int c = half * NC + 8 * j;
          if (have && c < cols) load_f32x8(at + c, x);
#pragma unroll
          for (int e = 0; e < 4; ++e) S[4 * j + e] = pack2(x[2 * e], x[2 * e + 1]);
        }
      } else {  // (the lanes' values are neighbours)
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
          const int c = half * NC + 2 * j;
          const bool real = have && c < cols;
          S[j] = pack2(real ? at[static_cast<long long>(c) * sc] : 0.0f, real ? at[static_cast<long long>(c + 1) * sc] : 0.0f);
        }
      }
    }
    // row `row` of QS' operand, 64 columns to a 128-byte line: columns c .. c + 7
    const auto copy8 = [&](int j) {
      const int c = half * NC + 8 * j;
      uint8_t* const at = copy + (c >> 6) * F::ROWS * 128 + row * 128 + ((((c & 63) >> 3) ^ (row & 7)) << 4);
      const uint4 t0 = make_uint4(pack_bf16(S[4 * j]), pack_bf16(S[4 * j + 1]), pack_bf16(S[4 * j + 2]), pack_bf16(S[4 * j + 3]));
      if (mine) *reinterpret_cast<uint4*>(at) = t0;
      if (F::TERMS == 2) {
        const f32x2 minus = pack2(-1.0f, -1.0f);
        const auto rest = [&](uint32_t u, f32x2 x) { return pack_bf16(fma2(pack2(bf16_lo(u), bf16_hi(u)), minus, x)); };
        if (mine)
          *reinterpret_cast<uint4*>(at + F::COPY) =
              make_uint4(rest(t0.x, S[4 * j]), rest(t0.y, S[4 * j + 1]), rest(t0.z, S[4 * j + 2]), rest(t0.w, S[4 * j + 3]));
      }
    };
    const auto copied = [&]() {
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_ready);
    };
    if (!so) {
#pragma unroll
      for (int j = 0; j < NC / 8; ++j) copy8(j);
    }
    copied();
    float hi = 0.0f, lo = 0.0f;
    int n_was = -1;
    uint32_t n_k = 0, n_z = 0, n_out = 0;
    const f32x2 upd = pack2(p.upd, p.upd);
    Ring r;
    for (Item it(w, group); it.i < items; it.next()) {
      int tok, n;
      chunk_at(w, p.rev, it.c, tok, n);
      const Ring rq = r;
      r.next(SLOTS);
      const Ring rk = r;
      r.next(SLOTS);
      r.next(SLOTS);
      if (!adds_k(it.sub)) continue;
      if (n != n_was) {
        n_was = n;
        power2(g, n, hi, lo);
      }
      if (!so) {
        // QS has read the q tile, and QK^T the keys: both may be overwritten
        if (!mbar_wait_short(&full[rk.slot], rk.phase) || !mbar_wait_short(qs_done, n_k++ & 1)) {
          fail();
          break;
        }
        decay_keys<DK>(smem + rk.slot * F::SLOT, smem + rq.slot * F::SLOT, power_of, p.rev, n, tid, 0, 2);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_ready);
      }
      if (it.sub != group - 1) continue;
      if (!mbar_wait_short(z_full, n_z++ & 1)) {
        fail();
        break;
      }
      tc_fence_after();
      const f32x2 hi2 = pack2(hi, hi), lo2 = pack2(lo, lo);
#pragma unroll
      for (int cb = 0; cb < NC / 32; ++cb) {
        uint32_t x[2][16];
        tmem_ld_32x32b_x16(trow + cb * 32, x[0]);
        tmem_ld_32x32b_x16(trow + cb * 32 + 16, x[1]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          f32x2& s = S[16 * cb + j];
          const uint32_t* const z = &x[j >> 3][2 * (j & 7)];
          s = fma2(hi2, s, fma2(lo2, s, mul2(upd, pack2(__uint_as_float(z[0]), __uint_as_float(z[1])))));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (!so && !STAGED) copy8(4 * cb + j);
      }
      if (!so && STAGED) {  // (an output may stand in the copy's place; the sum need not wait for it)
        if (staged(n) && !mbar_wait_short(o_gone, n_out++ & 1)) {
          fail();
          break;
        }
#pragma unroll
        for (int j = 0; j < NC / 8; ++j) copy8(j);
      }
      copied();
    }
    if (so || (w.last && p.s_out)) {
      // the segment's own sum goes where the scan turns it into the next one's start
      // (a call's state_out is never transposed)
      float* const out = so ? seg + static_cast<long long>(p.dk) * p.dv : p.s_out + state;
#pragma unroll
      for (int j = 0; j < NC / 8; ++j) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack2(S[4 * j + e], x[2 * e], x[2 * e + 1]);
        const int c = half * NC + 8 * j;
        if (!(mine && row < rows && c < cols)) continue;
        if (F::BY_VALUE) {
#pragma unroll
          for (int e = 0; e < 8; ++e) out[static_cast<long long>(c + e) * p.dv + row] = x[e];
        } else {
          store_f32x8(out + static_cast<long long>(row) * p.dv + c, x);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Width classes of keys and values, the smaller first: one kernel runs the forward's and the
// backward's problems, half of which have keys and values exchanged.
template <int D0, int D1, bool SO>
__global__ void __launch_bounds__(kThreads, 1) linattn_chunk_kernel(const __grid_constant__ Args a) {
  extern __shared__ uint8_t smem_raw[];
  if (SO) allow_next_kernel();
  Work w;
  if (!find_work(a, w)) {
    if (!SO && a.nseg > 1) wait_for_last_kernel();  // (no call ends before its kernels)
    return;
  }
  if (D0 == D1 || a.prob[w.prob].p.dk <= 64) run_chunks<D0, D1, SO>(a, w, smem_raw);
  else run_chunks<D1, D0, SO>(a, w, smem_raw);
}

// ------------------------------------------------------------------ segments

// The states at the segments' starts from their own sums (written by a states_only launch one slot
// further): slot 0 is the sequence's first state, slot s + 1 = lam^(tokens of s) slot s + the sum of s.
__global__ void __launch_bounds__(128) segment_scan_kernel(LinProblem p, LinShape s, float* seg, int nseg, int seg_chunks,
                                                           int n_even, int even_chunks) {
  const int h = blockIdx.x % s.Hs, n = blockIdx.x / s.Hs;
  allow_next_kernel();
  wait_for_last_kernel();
  int start, len;
  lin_sequence(s, n, start, len);
  if (len < 0) return;
  const int chunks = chunks_of(len);
  const int lack = first_short(n_even, even_chunks, seg_chunks, h), first_chunks = seg_chunks - lack;
  const int used = (chunks + lack + seg_chunks - 1) / seg_chunks;
  const float g = fminf(__ldg(s.log_decay + h), 0.0f);
  const int size = p.dk * p.dv;
  const long long base = static_cast<long long>(n) * s.Hs + h;
  // (a reverse recurrence starts with the sequence's last, short chunk)
  float hi0, lo0, hi, lo;
  power2(g, p.rev ? len - (chunks - first_chunks) * C : first_chunks * C, hi0, lo0);
  power2(g, seg_chunks * C, hi, lo);
  const int e = (blockIdx.y * blockDim.x + threadIdx.x) * 8;  // eight values of one row
  if (e >= size) return;
  float* const out = seg + base * nseg * size + e;
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (p.s_in) {
    const float* const in = p.s_in + base * size;
    const int i = e / p.dv, j = e - i * p.dv;
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = in[static_cast<long long>(i) * p.s_row + static_cast<long long>(j + u) * p.s_col];
  }
  store_f32x8(out, x);
  constexpr int AHEAD = 4;  // slots read at a time
  for (int k0 = 1; k0 < used; k0 += AHEAD) {
    float y[AHEAD][8];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (k0 + u < used) load_f32x8(out + static_cast<long long>(k0 + u) * size, y[u]);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (k0 + u >= used) continue;
      const bool first = k0 + u == 1;
#pragma unroll
      for (int v = 0; v < 8; ++v)
        x[v] = first ? fmaf(hi0, x[v], fmaf(lo0, x[v], y[u][v])) : fmaf(hi, x[v], fmaf(lo, x[v], y[u][v]));
      store_f32x8(out + static_cast<long long>(k0 + u) * size, x);
    }
  }
}

// ------------------------------------------------------------------ host side

int status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  record_cuda_error(e);
  return MOE_ERR_CUDA;
}

template <int D0, int D1, bool SO>
int launch(const char* name, const Args& a, bool behind, cudaStream_t st) {
  constexpr int SMEM = std::max(Cfg<D0, D1>::template SMEM<SO>, Cfg<D1, D0>::template SMEM<SO>);
  const auto kernel = linattn_chunk_kernel<D0, D1, SO>;
  static std::atomic<bool> ready[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status(e);
  if (dev < 0 || dev >= 64 || !ready[dev].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return status(e);
    if (dev >= 0 && dev < 64) ready[dev].store(true);
  }
  const long long grid = a.n_even ? a.n_even : static_cast<long long>(a.nprob) * a.s.N * a.s.Hs * (SO ? a.nseg - 1 : a.nseg);
  if (grid >= (1ll << 31)) return MOE_ERR_ARG;
  {
    LaunchTimer lt(name, st);
    if (behind) e = launch_behind(kernel, static_cast<unsigned>(grid), kThreads, SMEM, st, a);
    else kernel<<<static_cast<unsigned>(grid), kThreads, SMEM, st>>>(a);
  }
  return status(e == cudaSuccess ? cudaGetLastError() : e);
}

template <bool SO>
int launch_widths(const char* name, const Args& a, bool behind, cudaStream_t st) {
  const bool k64 = a.prob[0].p.dk <= 64, v64 = a.prob[0].p.dv <= 64;
  if (k64 && v64) return launch<64, 64, SO>(name, a, behind, st);
  if (k64 != v64) return launch<64, 128, SO>(name, a, behind, st);
  return launch<128, 128, SO>(name, a, behind, st);
}

struct Split {
  int nseg, seg_chunks;
  int n_even;  // CTAs of an even split, or 0
};

// Segments of state head h in an even split.
int segments_of(int h, int chunks, int per) {
  const int lack = static_cast<int>(static_cast<long long>(h) * chunks % per);
  return (chunks + lack + per - 1) / per;
}

// The CTAs of an even split: whole segments, then the others, the longer first: an SM that ends one of
// those early takes the longest of the rest.
void even_order(const Split& sp, int Hs, int chunks, uint16_t* order) {
  int n = 0, parts = 0;
  std::pair<int, uint16_t> part[2 * kEven];
  for (int h = 0; h < Hs; ++h) {
    const int lack = static_cast<int>(static_cast<long long>(h) * chunks % sp.seg_chunks);
    const int segs = segments_of(h, chunks, sp.seg_chunks);
    for (int k = 0; k < segs; ++k) {
      const int c0 = std::max(k * sp.seg_chunks - lack, 0), c1 = std::min(chunks, (k + 1) * sp.seg_chunks - lack);
      const uint16_t id = static_cast<uint16_t>(h << 8 | k);
      if (c1 - c0 == sp.seg_chunks) order[n++] = id;
      else part[parts++] = {c0 - c1, id};
    }
  }
  std::sort(part, part + parts);
  for (int i = 0; i < parts; ++i) order[n++] = part[i].second;
}

// Segments of the time axis. Estimated from what was measured (us, widths of 128): a CTA takes 6 and
// 3.2 a chunk and head of its group (64 wide 2.5), one that sums the state alone 5 and 1.4 (1.0) a chunk and
// head of the keys, one that finds nothing to do 1; the scan moves every segment's state twice at 5 GB a ms; two more
// launches 4. The lengths of ragged sequences are on the device: the CTAs with a whole segment are
// counted as if every sequence but for its last chunk were full of them, and run in rounds over the SMs
// unless the chunks spread over all SMs take longer. The split with the shortest estimate is taken.
Split split(int N, int T, int max_seqlen, int Hs, int np, int group, int keys, int Dk, int Dv) {
  const int chunks = chunks_of(max_seqlen);
  // (a workspace may be asked for before the tokens are counted)
  if (T <= 0) T = static_cast<int>(std::min(static_cast<long long>(N) * max_seqlen, 0x7FFFFFFFll));
  Split best{1, chunks > 0 ? chunks : 1, 0};
  const double sms = num_sms(), heads = static_cast<double>(Hs) * np;
  const bool narrow = Dk <= 64 && Dv <= 64;
  const double chunk = (narrow ? 2.5 : 3.2) * group, sum = (narrow ? 1.0 : 1.4) * keys;
  const double all_chunks = std::min(static_cast<double>(N) * chunks, static_cast<double>(T / C) + N);
  double least = 0.0;
  for (int n = 1; n <= 64 && n <= chunks && (n == 1 || heads * N * n <= 16 * sms); ++n) {
    const int per = (chunks + n - 1) / n;
    if ((chunks + per - 1) / per != n) continue;
    const double all = heads * N * n;
    const double busy = std::min(all, heads * (std::floor(all_chunks / per) + N));
    const double whole = heads * (N == 1 ? n : std::max(1.0, std::floor(all_chunks / per)));
    const double idle = (all - busy) / sms;
    const auto pass = [&](double part, double cta, double per_chunk) {
      return std::max(std::ceil(whole * part / sms) * (cta + per_chunk * per),
                      (busy * part * cta + heads * all_chunks * part * per_chunk) / sms) + idle;
    };
    double t = pass(1.0, 6.0, chunk);
    if (n > 1) t += pass((n - 1.0) / n, 5.0, sum) + busy * Dk * Dv * 8.0 / 5.0e6 + 4.0;
    if (n == 1 || t < least) {
      least = t;
      best = Split{n, per, 0};
    }
  }
  // One sequence: the heads' chunks laid one behind the other and cut evenly over the SMs. A part that holds
  // the end of one head and the start of the next is two CTAs, which fill an SM one after the other. (32 heads
  // of 32,768 tokens: 280 us, in four equal segments on 128 of 152 SMs 304.)
  if (N == 1 && np == 1 && Hs < sms && chunks > 1) {
    const int per = static_cast<int>(std::ceil(static_cast<double>(Hs) * chunks / sms));
    const int slots = (chunks + per - 2) / per + 1;  // of a head, at most
    int ctas = 0;
    for (int h = 0; h < Hs; ++h) ctas += segments_of(h, chunks, per);
    const double t = 12.0 + chunk * per + 10.0 + sum * per + static_cast<double>(Hs) * slots * Dk * Dv * 8.0 / 5.0e6 + 4.0;
    if (per < chunks && slots < 256 && Hs < 256 && ctas <= kEven && t < least) best = Split{slots, per, ctas};
  }
  return best;
}

size_t slots_bytes(const LinShape& s, const Split& sp, int dk, int dv) {
  return static_cast<size_t>(s.N) * s.Hs * sp.nseg * dk * dv * 4;
}

}  // namespace

size_t linattn_workspace(int max_seqlen, int Dk, int Dv, int Hs, int r, int T, int N, bool backward) {
  if (max_seqlen <= 0 || N <= 0 || Hs <= 0 || Dk <= 0 || Dv <= 0) return 0;
  const Split sp = split(N, T, max_seqlen, Hs, backward ? 3 : 1, r, backward ? r : 1, Dk, Dv);
  if (sp.nseg == 1) return 0;
  LinShape s{};
  s.N = N;
  s.Hs = Hs;
  return (slots_bytes(s, sp, Dk, Dv) * (backward ? 2 : 1) + 255) & ~static_cast<size_t>(255);
}

int linattn_run(const LinProblem* p, int np, const LinShape& s, void* ws, cudaStream_t st) {
  const int r = std::max(p[0].nq, p[0].nkv);
  const Split sp = split(s.N, s.T, s.max_seqlen, s.Hs, np, r, np > 1 ? r : 1, p[0].dk, p[0].dv);
  Args a;
  std::memset(static_cast<void*>(&a), 0, sizeof a);
  a.s = s;
  a.nprob = np;
  a.nseg = sp.nseg;
  a.seg_chunks = sp.seg_chunks;
  a.n_even = sp.n_even;
  if (sp.n_even) {
    a.even_chunks = chunks_of(s.max_seqlen);
    even_order(sp, s.Hs, a.even_chunks, a.even);
  }
  const long long T = s.T > 0 ? s.T : 1;
  float* slots = static_cast<float*>(ws);
  for (int i = 0; i < np; ++i) {
    Problem& x = a.prob[i];
    x.p = p[i];
    const long long hq = static_cast<long long>(s.Hs) * p[i].nq, hk = static_cast<long long>(s.Hs) * p[i].nkv;
    if (!make_rows_map(&x.q, p[i].q, p[i].dk, T, hq, p[i].ldq, p[i].dk, C) ||
        !make_rows_map(&x.k, p[i].k, p[i].dk, T, hk, p[i].ldk, p[i].dk, C) ||
        !make_rows_map(&x.v, p[i].v, p[i].dv, T, hk, p[i].ldv, p[i].dv, C) ||
        !make_rows_map(&x.o, p[i].o, p[i].dv, T, hq, p[i].ldo, p[i].dv, C))
      return MOE_ERR_CUDA;
    if (sp.nseg > 1) {
      if (p[i].shares < 0) {
        x.seg = slots;
        x.seg_row = p[i].dv;
        x.seg_col = 1;
        slots += slots_bytes(s, sp, p[i].dk, p[i].dv) / 4;
      } else {  // the transposed states of another problem
        x.seg = a.prob[p[i].shares].seg;
        x.seg_row = 1;
        x.seg_col = p[i].dk;
      }
    }
  }
  if (sp.nseg > 1) {
    Args own = a;  // (the problems with states of their own come first)
    own.states_only = 1;
    while (p[own.nprob - 1].shares >= 0) --own.nprob;
    const int e = launch_widths<true>("linattn_segments", own, false, st);
    if (e != MOE_OK) return e;
    for (int i = 0; i < own.nprob; ++i) {
      LaunchTimer lt("linattn_scan", st);
      const dim3 grid(static_cast<unsigned>(s.N) * s.Hs, (p[i].dk * p[i].dv + 1023) / 1024);
      const int se = status(launch_behind(segment_scan_kernel, grid, 128, 0, st, p[i], s, a.prob[i].seg, sp.nseg, sp.seg_chunks, a.n_even, a.even_chunks));
      if (se != MOE_OK) return se;
    }
  }
  return launch_widths<false>(np == 1 ? "linattn_fwd" : "linattn_bwd", a, sp.nseg > 1, st);
}

}  // namespace moe
