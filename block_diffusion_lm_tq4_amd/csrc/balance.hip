// The training step of the router in front of the MoE layer (Nemotron-TheHobbit-30B-A3B
// model card, The model underneath: 128 experts, top-6): per-expert counts, mean
// probabilities and the balance loss, and the gradient of the gates and of that loss with
// respect to the router logits.
//
// Per token t with scores p_e of its logits (softmax over the experts, or sigmoid) and
// q_e = p_e / sum_i p_i; an expert with a logit of -inf or NaN has p = q = 0:
//   counts_e = number of (token, slot) pairs of expert e, N their sum;
//   live tokens have an id in [0, E); T is their number, P_e = (1/T) sum_live q_te;
//   loss = E sum_e (counts_e / N) P_e, a function of the logits through P alone.
// Gates as the scored router forms them: w_j = s p_j, or s p_j / sum of the token's chosen
// p.  With c_e = dloss E counts_e / (N T) and u = p_j / sum of the chosen:
//   softmax: dl_e = q_e (c_e - sum_i q_i c_i) + gates' part;  sigmoid: (1 - p_e) times that;
//   gates:   softmax     dl_e += p_e (a_e - sum_j p_j a_j),  a_e = s dw of e's slots
//            sigmoid     dl_j += p_j (1 - p_j) s dw_j
//            normalized  dl_j += u_j s (dw_j - sum_i u_i dw_i)  [(1 - p_j) if sigmoid].
// Scores are fp32, taken relative to the largest logit they are divided by the sum of, so
// no row under- or overflows; sums over tokens are fp32 for up to kRun tokens of a lane and fp64
// beyond, through the scratch memory too.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mxfp4.h"

namespace tq4 {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kLanes = 16;  // lanes of a token
constexpr int kMaxE = 512;
constexpr float kOff = -__builtin_inff();

template <int CTRL>
__device__ inline float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// Reductions over the 16 lanes of a token: partners l ^ 1, l ^ 2, 7 - l and 15 - l; each
// step is commutative, so all lanes end with the same bits.
template <class F>
__device__ inline float row_reduce(float v, F f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  return f(v, dpp<0x140>(v));
}
__device__ inline float row_max(float v) {
  return row_reduce(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ inline float row_sum(float v) {
  return row_reduce(v, [](float a, float b) { return a + b; });
}

// e^x for x <= 0 with a relative error of about 2 ulp: 2^t of the rounded product t = x
// log2(e), times the first two terms of e^r for what its rounding left.  0 from -104 on,
// past fp32's smallest number, and for NaN (of two infinities).
__device__ inline float exp_neg(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kLow = 0x1.4ae0cp-26f;  // log2(e) in two parts
  constexpr float kLn2 = 0x1.62e43p-1f;
  x = __builtin_fmaxf(x, -104.f);
  const float t = x * kLog2e;
  const float r = __builtin_fmaf(x, kLow, __builtin_fmaf(x, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * kLn2, e);
}

// A logit as the scores take it: off at -inf and NaN, finite above.
__device__ inline float usable(float l) {
  return l > kOff ? __builtin_fminf(l, 3.402823466e38f) : kOff;
}

// The token's logits: lane l of 16 holds experts 4 l + 64 i + v.
template <int NV, bool VEC>
struct Row {
  float l[NV][4];
  float top;

  __device__ void load(const float *row, int n_experts, int lane) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 64 * i + 4 * lane;
      if constexpr (VEC) {
        floatx4 d = {kOff, kOff, kOff, kOff};
        if (e < n_experts) d = *reinterpret_cast<const floatx4 *>(row + e);
#pragma unroll
        for (int v = 0; v < 4; ++v) l[i][v] = d[v];
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) l[i][v] = e + v < n_experts ? row[e + v] : kOff;
      }
    }
  }

  __device__ void clean() {
    top = kOff;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        l[i][v] = usable(l[i][v]);
        top = __builtin_fmaxf(top, l[i][v]);
      }
    top = row_max(top);
  }
};

// A score relative to e^top (softmax) or to e^min(top, 0) (sigmoid), and 1 - p of the
// sigmoid.  With z = e^-|l| the sigmoid is 1 / (1 + z) or z / (1 + z) and 1 - p the other
// one; only where every logit is negative does the base need an exponential of its own.
template <bool SIGMOID>
__device__ inline float score(float l, float top, float &rest) {
  if constexpr (SIGMOID) {
    const float z = exp_neg(-__builtin_fabsf(l));
    const float inv = __builtin_amdgcn_rcpf(1.f + z);
    const bool pos = l >= 0.f;
    rest = (pos ? z : 1.f) * inv;
    const float base = top >= 0.f ? (pos ? 1.f : z) : exp_neg(l - top);
    return base * inv;
  } else {
    rest = 1.f;
    return exp_neg(l - top);
  }
}

// Scores of a whole row and 1 / their sum (0 for a row without experts).  (An expert that
// is off has l = -inf, hence e^-inf = 0 throughout; a row of only such ones has the base
// -inf too and is left out.)
template <bool SIGMOID, int NV, bool VEC>
__device__ inline float row_scores(const Row<NV, VEC> &row, float (&p)[NV][4],
                                   float (&rest)[NV][4]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      p[i][v] = score<SIGMOID>(row.l[i][v], row.top, rest[i][v]);
      sum += p[i][v];
    }
  sum = row_sum(sum);
  return sum > 0.f ? 1.f / sum : 0.f;
}

__device__ inline bool routed(int id, int n_experts) { return id >= 0 && id < n_experts; }

// ---- counts, mean probabilities, loss ----------------------------------------

constexpr int kSumThreads = 1024;
constexpr int kSumTokens = kSumThreads / kLanes;  // of a workgroup at a time
constexpr int kMaxGroups = 256;                   // one per compute unit
constexpr int kRun = 8;                           // tokens that a lane adds in fp32

struct BalanceOut {
  float *loss, *mean_p;
  int32_t *counts, *tokens;
};

// The experts of one workgroup of the second launch.  Its sums of a group are one cache
// line (a compute unit has few misses under way: slices of 64 experts, whose sums and
// counts were two lines each, took 15 us for 256 groups of 256 experts).
constexpr int kSlice = 8;

struct __attribute__((aligned(128))) SliceSums {
  double q[kSlice];
  int32_t n[kSlice];
};

// A group's sums in scratch, and what the slices of experts add up.
struct BalanceParts {
  SliceSums *sums;  // [slices][groups]
  int32_t *t;       // [groups]
  double *dot;      // [slices]: sum of mean * count
  int64_t *pairs;   // [slices]
  uint32_t *done;   // slices that are through (cleared by the sums' launch)
};

// Sums over a wave; every lane has the results, and the same bits.
__device__ inline void wave_sums(double &d, int64_t &n) {
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    d += __shfl_xor(d, x);
    n += __shfl_xor(n, x);
  }
}

// Sums over a workgroup, in wave order; every thread calls, thread 0 has the results.
__device__ inline void group_sums(double &d, int64_t &n, double *lds_d, int64_t *lds_n) {
  const int tid = threadIdx.x;
  wave_sums(d, n);
  if (tid % 64 == 0) {
    lds_d[tid / 64] = d;
    lds_n[tid / 64] = n;
  }
  __syncthreads();
  if (tid == 0)
    for (int w = 1; w < kSumThreads / 64; ++w) {
      d += lds_d[w];
      n += lds_n[w];
    }
}

__device__ inline float balance_loss(int n_experts, double dot, int64_t pairs) {
  return pairs > 0 ? static_cast<float>(n_experts * dot / static_cast<double>(pairs)) : 0.f;
}

// One expert's totals to the outputs; adds its share of the loss.
__device__ inline void balance_expert(const BalanceOut &o, int e, double p, int32_t c,
                                      int32_t live, double &dot, int64_t &pairs) {
  const double mean = live > 0 ? p / static_cast<double>(live) : 0.0;
  o.counts[e] = c;
  o.mean_p[e] = static_cast<float>(mean);
  dot += mean * static_cast<double>(c);
  pairs += c;
}

// A workgroup's share of the tokens.  With ONE workgroup its sums are the result, else its
// sums of q and its counts go to scratch.  A token's row, and the ids, are fetched a round
// ahead where the registers hold two rows.  Every kRun rounds, and at the end, the lanes' sums
// go to LDS, 64 of an expert, where kParts threads add a part of them each in fp64.  (fp32
// sums of a whole batch's tokens are off by 160 2^-24 at 2^24 equal rows, where every addition
// rounds the same way.)  16411 x 256, sigmoid: 8.4 us, vector instructions
// busy in 64 % of the cycles (17 MB at the copy's rate: 3.4 us).
template <bool SIGMOID, int NV, bool VEC, bool ONE>
__global__ __launch_bounds__(kSumThreads) void balance_sums_kernel(BalanceArgs a, BalanceOut o,
                                                                   BalanceParts parts) {
  constexpr int kWaves = kSumThreads / 64;
  constexpr int kCols = 64 * NV;
  constexpr int kParts = kSumThreads / kCols;
  __shared__ __attribute__((aligned(16))) float sums[kSumTokens][kCols];
  __shared__ double part_sums[kParts][kCols];
  __shared__ int32_t hist[kCols];
  __shared__ int32_t tokens;
  __shared__ double dot[kWaves];
  __shared__ int64_t all[kWaves];
  const int tid = threadIdx.x;
  const int lane = tid % kLanes, group = tid / kLanes;
  const int col = tid % kCols, part = tid / kCols;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSumTokens;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kSumTokens;
  constexpr bool kAhead = NV <= 4;
  Row<NV, VEC> next;
  int next_id = -1;
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    next.load(a.logits + t * a.n_experts, a.n_experts, lane);
    if (lane < a.topk) next_id = a.ids[t * a.topk + lane];
  };
  if (kAhead && base + group < a.t) fetch(base + group);
  for (int e = tid; e < kCols; e += kSumThreads) hist[e] = 0;
  if (tid == 0) tokens = 0;
  __syncthreads();
  float acc[NV][4] = {};
  double p = 0.0;
  // (all threads of the workgroup call)
  auto join = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      *reinterpret_cast<floatx4 *>(&sums[group][64 * i + 4 * lane]) =
          floatx4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][v] = 0.f;
    }
    __syncthreads();
    constexpr int kRows = kSumTokens / kParts;
#pragma unroll
    for (int r = 0; r < kRows; ++r) p += static_cast<double>(sums[kRows * part + r][col]);
  };
  int run = 0;
  for (int64_t t0 = base; t0 < a.t; t0 += stride) {
    const int64_t t = t0 + group;
    if (t < a.t) {
      if (!kAhead) fetch(t);
      Row<NV, VEC> row = next;
      const int own_id = next_id;
      if (kAhead && t + stride < a.t) fetch(t + stride);
      bool any = routed(own_id, a.n_experts);
      if (any) atomicAdd(&hist[own_id], 1);
      for (int j = lane + kLanes; j < a.topk; j += kLanes) {
        const int id = a.ids[t * a.topk + j];
        if (!routed(id, a.n_experts)) continue;
        atomicAdd(&hist[id], 1);
        any = true;
      }
      if (row_max(any ? 1.f : 0.f) != 0.f) {  // else routed nowhere
        if (lane == 0) atomicAdd(&tokens, 1);
        row.clean();
        float q[NV][4], rest[NV][4];
        const float inv = row_scores<SIGMOID, NV, VEC>(row, q, rest);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][v] = __builtin_fmaf(q[i][v], inv, acc[i][v]);
      }
    }
    if (++run == kRun && t0 + stride < a.t) {
      join();
      __syncthreads();  // these reads before the next sums
      run = 0;
    }
  }
  join();
  part_sums[part][col] = p;
  __syncthreads();
  p = 0.0;
  int32_t c = 0;
  if (tid < a.n_experts) {
#pragma unroll
    for (int r = 0; r < kParts; ++r) p += part_sums[r][tid];
    c = hist[tid];
  }
  if constexpr (ONE) {
    double d = 0.0;
    int64_t n = 0;
    if (tid < a.n_experts) balance_expert(o, tid, p, c, tokens, d, n);
    group_sums(d, n, dot, all);
    if (tid == 0) {
      *o.loss = balance_loss(a.n_experts, d, n);
      *o.tokens = tokens;
    }
  } else {
    if (tid < a.n_experts) {
      SliceSums &to = parts.sums[(tid / kSlice) * gridDim.x + blockIdx.x];
      to.q[tid % kSlice] = p;
      to.n[tid % kSlice] = c;
    }
    if (tid == 0) {
      parts.t[blockIdx.x] = tokens;
      if (blockIdx.x == 0) *parts.done = 0;
    }
  }
}

// A workgroup adds the groups' sums of its slice in a fixed order, fp64: thread e + 8 i
// takes groups i and i + 128 of expert e, both on their way at once.  The last workgroup
// through adds the slices' shares of the loss, a lane each, in a fixed order.  256 groups of
// 256 experts 6.8 us: latencies, of the lines (from other XCDs' L2), the fence and the counter.
__global__ __launch_bounds__(kSumThreads) void balance_loss_kernel(BalanceParts parts, int groups,
                                                                   int n_experts, BalanceOut o) {
  constexpr int kParts = kSumThreads / kSlice;
  constexpr int kAhead = kMaxGroups / kParts;
  constexpr int kWaves = kSumThreads / 64;
  __shared__ double sp[kWaves][kSlice];
  __shared__ int32_t sc[kWaves][kSlice];
  __shared__ int32_t st;
  const int tid = threadIdx.x;
  const int col = tid % kSlice, part = tid / kSlice;
  const int e = static_cast<int>(blockIdx.x) * kSlice + col;
  double dp[kAhead];
  int32_t dc[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int g = part + kParts * i;
    const bool in = g < groups && e < n_experts;
    const SliceSums *from = parts.sums + static_cast<int>(blockIdx.x) * groups + g;
    dp[i] = in ? from->q[col] : 0.0;
    dc[i] = in ? from->n[col] : 0;
  }
  const int32_t t = tid < groups ? parts.t[tid] : 0;
  if (tid == 0) st = 0;
  double p = 0.0;
  int32_t c = 0;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    p += dp[i];
    c += dc[i];
  }
  // the wave's eight parts, then the waves in order
#pragma unroll
  for (int x = kSlice; x < 64; x <<= 1) {
    p += __shfl_xor(p, x);
    c += __shfl_xor(c, x);
  }
  if (tid % 64 < kSlice) {
    sp[tid / 64][col] = p;
    sc[tid / 64][col] = c;
  }
  __syncthreads();
  if (t != 0) atomicAdd(&st, t);
  __syncthreads();
  if (tid >= 64) return;  // lanes 0 .. 7 of wave 0 have the slice's experts
  double d = 0.0;
  int64_t n = 0;
  if (part == 0 && e < n_experts) {
#pragma unroll
    for (int q = 1; q < kWaves; ++q) {
      p += sp[q][col];
      c += sc[q][col];
    }
    balance_expert(o, e, p, c, st, d, n);
  }
  wave_sums(d, n);
  if (tid == 0 && blockIdx.x == 0) *o.tokens = st;
  if (gridDim.x > 1) {
    uint32_t before = 0;
    if (tid == 0) {
      parts.dot[blockIdx.x] = d;
      parts.pairs[blockIdx.x] = n;
      __threadfence();
      before = atomicAdd(parts.done, 1u);
    }
    if (__builtin_amdgcn_readfirstlane(before) + 1 < gridDim.x) return;
    __threadfence();
    const bool in = tid < static_cast<int>(gridDim.x);  // at most 64 slices
    d = in ? __hip_atomic_load(parts.dot + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    n = in ? __hip_atomic_load(parts.pairs + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
    wave_sums(d, n);
  }
  if (tid == 0) *o.loss = balance_loss(n_experts, d, n);
}

// ---- gradient ------------------------------------------------------------------

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / kLanes;  // of a workgroup at a time

// Slot j of a token as lane j % 16 sees it: its expert (-1: none), that expert's logit and
// the gate's gradient (0 for an expert that is off, whatever stands there: its gate is a constant
// 0, and 0 times an infinity would spoil the row).
struct Slot {
  int id;
  float l, d;
  __device__ void load(const RouterGradArgs &g, int64_t t, int j) {
    id = -1;
    l = kOff;
    d = 0.f;
    if (j >= g.b.topk) return;
    const int at = g.b.ids[t * g.b.topk + j];
    if (!routed(at, g.b.n_experts)) return;
    id = at;
    if (g.dgates == nullptr) return;
    d = g.dgates[t * g.b.topk + j];
    l = usable(g.b.logits[t * g.b.n_experts + at]);
    d = l > kOff ? d : 0.f;
  }
};

// The gates' contributions of one token to `delta` (its row of LDS): their gradient with respect
// to the logits, but with SUMS_ONLY (softmax without renormalization) the sums of dw alone.
// Lane j of the token takes slots j, j + 16, ...; `own` is its first.
template <bool SIGMOID, bool SUMS_ONLY>
__device__ inline void gate_part(const RouterGradArgs &g, int64_t t, const Slot &own, float *delta,
                                 int lane) {
  const int blocks = (g.b.topk + kLanes - 1) / kLanes;
  auto slot = [&](int b) __attribute__((always_inline)) {
    Slot s = own;
    if (b > 0) s.load(g, t, b * kLanes + lane);
    return s;
  };
  // without renormalization: the scores (sigmoid) themselves
  float base = 0.f, norm = 1.f, mean = 0.f, ref = 0.f;
  if (!SUMS_ONLY && g.renormalize) {  // relative to the largest chosen one
    base = kOff;
    for (int b = 0; b < blocks; ++b) base = __builtin_fmaxf(base, slot(b).l);
    base = row_max(base);
    // dw_j - sum_i u_i dw_i is taken relative to the dw of the largest one: with one slot, or
    // one that has nearly all the weight, the two sides of the difference are all but equal
    ref = kOff;
    for (int b = 0; b < blocks; ++b) {
      const Slot s = slot(b);
      if (s.l > kOff && s.l == base) ref = __builtin_fmaxf(ref, s.d);
    }
    ref = row_max(ref);
    ref = ref > kOff ? ref : 0.f;
    float sum = 0.f, dot = 0.f;
    for (int b = 0; b < blocks; ++b) {
      const Slot s = slot(b);
      float rest;
      const float p = s.l > kOff ? score<SIGMOID>(s.l, base, rest) : 0.f;
      sum += p;
      dot += p * (s.d - ref);
    }
    sum = row_sum(sum);
    norm = sum > 0.f ? 1.f / sum : 0.f;
    mean = row_sum(dot) * norm;
  }
  for (int b = 0; b < blocks; ++b) {
    const Slot s = slot(b);
    const int id = s.id;
    float add = s.d;
    if constexpr (!SUMS_ONLY) {
      float rest = 1.f;
      const float p = s.l > kOff ? score<SIGMOID>(s.l, base, rest) * norm : 0.f;
      add = p * (g.scale * ((s.d - ref) - mean));
      if (SIGMOID) add *= rest;
    }
    // Slots that all have experts of their own, as a router's have, add without a look at
    // each other: a lane leaves its number at its expert and finds it there again.
    if (b == 0) {
      int *mark = reinterpret_cast<int *>(delta);
      if (id >= 0) mark[id] = lane;
      wave_lds_fence();
      const bool alone = id < 0 || mark[id] == lane;
      wave_lds_fence();
      if (id >= 0) delta[id] = 0.f;
      wave_lds_fence();
      if (__builtin_amdgcn_ballot_w64(!alone) == 0) {
        if (id >= 0) delta[id] = add;
        wave_lds_fence();
        continue;
      }
    }
    // else the lowest lane of an expert adds the others', always in the same order
    float all = add;
    bool first = id >= 0;
    auto turn = [&](int oid, float o, int from) __attribute__((always_inline)) {
      const bool same = oid == id;
      all += same ? o : 0.f;
      first = first && !(same && from < lane);
    };
#define TQ4_TURN(R)                                                                      \
  turn(__builtin_amdgcn_mov_dpp(id, 0x120 + R, 0xF, 0xF, false), dpp<0x120 + R>(add), \
       __builtin_amdgcn_mov_dpp(lane, 0x120 + R, 0xF, 0xF, false));
    TQ4_TURN(1) TQ4_TURN(2) TQ4_TURN(3) TQ4_TURN(4) TQ4_TURN(5) TQ4_TURN(6) TQ4_TURN(7)
    TQ4_TURN(8) TQ4_TURN(9) TQ4_TURN(10) TQ4_TURN(11) TQ4_TURN(12) TQ4_TURN(13) TQ4_TURN(14)
    TQ4_TURN(15)
#undef TQ4_TURN
    if (first) delta[id] += all;
    wave_lds_fence();
  }
}

// 16 lanes per token, 16 tokens per workgroup at a time.  A token's row and slots are
// fetched before anything waits.  16411 x 256, sigmoid, 8 slots: 15.3 us, vector
// instructions busy in 68 % of the cycles (reading and writing alone 8.7).
template <bool SIGMOID, int NV, bool VEC>
__global__ __launch_bounds__(kThreads) void router_backward_kernel(RouterGradArgs g) {
  __shared__ __attribute__((aligned(16))) float delta_all[kTokens][64 * NV];
  __shared__ __attribute__((aligned(16))) float share[64 * NV];  // counts, less their mean
  __shared__ int32_t total[kThreads / 64];
  const int tid = threadIdx.x;
  const int lane = tid % kLanes, group = tid / kLanes;
  const int n_experts = g.b.n_experts;
  const bool has_loss = g.counts != nullptr;
  const bool has_gates = g.dgates != nullptr;
  // softmax weights as they are: every expert's gradient sees every slot's
  const bool whole = !SIGMOID && has_gates && !g.renormalize;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kTokens + group;
  Row<NV, VEC> row;
  Slot own;
  if (first < g.b.t) {
    row.load(g.b.logits + first * n_experts, n_experts, lane);
    own.load(g, first, lane);
  }
  float unit = 0.f;  // c_e of the loss per pair
  if (has_loss) {
    constexpr int kPer = (64 * NV + kThreads - 1) / kThreads;
    int32_t count[kPer], n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + kThreads * i;
      count[i] = e < n_experts ? g.counts[e] : 0;
      n += count[i];
    }
    const double tokens = *g.tokens, dloss = *g.dloss;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
    if (tid % 64 == 0) total[tid / 64] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kThreads / 64; ++w) n += total[w];
    const double pairs = n;
    unit = pairs > 0.0 && tokens > 0.0
               ? static_cast<float>(dloss * n_experts / (pairs * tokens))
               : 0.f;
    const int mean = n / n_experts;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + kThreads * i;
      if (e < 64 * NV) share[e] = static_cast<float>(count[i] - mean);
    }
  }
  __syncthreads();
  float *delta = delta_all[group];
  for (int64_t t = first; t < g.b.t; t += static_cast<int64_t>(gridDim.x) * kTokens) {
    if (t > first) {
      row.load(g.b.logits + t * n_experts, n_experts, lane);
      own.load(g, t, lane);
    }
    row.clean();
    float p[NV][4], rest[NV][4];
    const float inv = row_scores<SIGMOID, NV, VEC>(row, p, rest);
    if (has_gates) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        *reinterpret_cast<floatx4 *>(delta + 64 * i + 4 * lane) = floatx4{0.f, 0.f, 0.f, 0.f};
      wave_lds_fence();
      if (whole)
        gate_part<SIGMOID, true>(g, t, own, delta, lane);
      else
        gate_part<SIGMOID, false>(g, t, own, delta, lane);
    }
    // live: an id in range in any slot
    bool any = own.id >= 0;
    if (has_loss)
      for (int j = lane + kLanes; j < g.b.topk; j += kLanes)
        any = any || routed(g.b.ids[t * g.b.topk + j], n_experts);
    const bool live = has_loss && row_max(any ? 1.f : 0.f) > 0.f;
    // The loss's part: c_e - sum_i q_i c_i = unit * ((n_e - m) - sum_i q_i (n_i - m)) for any
    // m.  With the row's mean count as m, rounded, so that n_e - m is exact, no term is more than
    // three times sum_i q_i |c_e - c_i|, and the difference is right relative to that: where one
    // expert has nearly all the weight the two sides are all but equal.  The same with the sums a_e
    // of the gates' gradients, whose mean need not be rounded.
    floatx4 c[NV];
    float m = 0.f, m_a = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = live ? *reinterpret_cast<const floatx4 *>(share + 64 * i + 4 * lane)
                  : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        p[i][v] *= inv;
        m = __builtin_fmaf(p[i][v], c[i][v], m);
      }
    }
    m = __builtin_rintf(row_sum(m));
    // (`delta` is read where it is used: registers for it would cost a wave per SIMD)
    auto delta_at = [&](int i) __attribute__((always_inline)) {
      return *reinterpret_cast<const floatx4 *>(delta + 64 * i + 4 * lane);
    };
    if (whole) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const floatx4 a = delta_at(i);
#pragma unroll
        for (int v = 0; v < 4; ++v) m_a = __builtin_fmaf(p[i][v], a[v], m_a);
      }
      m_a = row_sum(m_a);
    }
    const float of_pair = live ? unit : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int v = 0; v < 4; ++v) c[i][v] = of_pair * (c[i][v] - m);
      if (whole) {
        const floatx4 a = delta_at(i);
#pragma unroll
        for (int v = 0; v < 4; ++v) c[i][v] = __builtin_fmaf(g.scale, a[v] - m_a, c[i][v]);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) dot = __builtin_fmaf(p[i][v], c[i][v], dot);
    }
    dot = row_sum(dot);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 64 * i + 4 * lane;
      floatx4 d = {0.f, 0.f, 0.f, 0.f};
      if (has_gates && !whole) d = delta_at(i);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float w = p[i][v] * rest[i][v];
        d[v] += __builtin_fmaf(w, c[i][v], -(w * dot));
      }
      float *out = g.dlogits + t * n_experts + e;
      if constexpr (VEC) {
        if (e < n_experts) *reinterpret_cast<floatx4 *>(out) = d;
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (e + v < n_experts) out[v] = d[v];
      }
    }
    wave_lds_fence();  // this token's reads before the next one's zeros
  }
}

template <class F>
void by_experts(int n_experts, bool vec, F f) {
  auto with = [&](auto nv) {
    if (vec)
      f(nv, std::true_type{});
    else
      f(nv, std::false_type{});
  };
  if (n_experts <= 64)
    with(std::integral_constant<int, 1>{});
  else if (n_experts <= 128)
    with(std::integral_constant<int, 2>{});
  else if (n_experts <= 256)
    with(std::integral_constant<int, 4>{});
  else
    with(std::integral_constant<int, 8>{});
}

}  // namespace

static int balance_groups(int64_t t) {
  if (t <= 4 * kSumTokens) return 1;
  const int64_t groups = (t + kSumTokens - 1) / kSumTokens;
  return static_cast<int>(groups < kMaxGroups ? groups : kMaxGroups);
}

namespace {

// Scratch: the slices' shares first (16 bytes each), then the groups' sums.
constexpr size_t kShares = (16 * (kMaxE / kSlice) + 16 + 127) / 128 * 128;
static_assert(sizeof(SliceSums) == 128 && kMaxE / kSlice <= 64, "a line a group, a lane a slice");

}  // namespace

size_t balance_scratch(int64_t t, int32_t n_experts) {
  const size_t groups = static_cast<size_t>(balance_groups(t));
  const size_t slices = (static_cast<size_t>(n_experts) + kSlice - 1) / kSlice;
  return groups > 1 ? kShares + groups * (sizeof(SliceSums) * slices + 4) : 0;
}

hipError_t launch_moe_balance(const BalanceArgs &a, float *loss, int32_t *counts, int32_t *tokens,
                              float *mean_p, void *scratch, hipStream_t s) {
  if (a.n_experts < 1 || a.n_experts > kMaxE) return hipErrorInvalidValue;
  const int groups = balance_groups(a.t);
  const BalanceOut out{loss, mean_p, counts, tokens};
  BalanceParts parts{};
  if (groups > 1) {
    char *at = static_cast<char *>(scratch);
    parts.dot = reinterpret_cast<double *>(at);
    parts.pairs = reinterpret_cast<int64_t *>(at + 8 * (kMaxE / kSlice));
    parts.done = reinterpret_cast<uint32_t *>(at + 16 * (kMaxE / kSlice));
    parts.sums = reinterpret_cast<SliceSums *>(at + kShares);
    parts.t = reinterpret_cast<int32_t *>(
        parts.sums + static_cast<int64_t>(groups) * ((a.n_experts + kSlice - 1) / kSlice));
  }
  const bool vec = a.n_experts % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  by_experts(a.n_experts, vec, [&](auto nv, auto v) {
    auto launch = [&](auto sigmoid, auto one) {
      hipLaunchKernelGGL((balance_sums_kernel<sigmoid.value, nv.value, v.value, one.value>),
                         dim3(groups), dim3(kSumThreads), 0, s, a, out, parts);
    };
    auto with = [&](auto sigmoid) {
      if (groups == 1)
        launch(sigmoid, std::true_type{});
      else
        launch(sigmoid, std::false_type{});
    };
    if (a.sigmoid)
      with(std::true_type{});
    else
      with(std::false_type{});
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || groups == 1) return e;
  hipLaunchKernelGGL(balance_loss_kernel, dim3((a.n_experts + kSlice - 1) / kSlice),
                     dim3(kSumThreads), 0, s, parts, groups, a.n_experts, out);
  return hipGetLastError();
}

hipError_t launch_router_backward(const RouterGradArgs &a, hipStream_t s) {
  if (a.b.n_experts < 1 || a.b.n_experts > kMaxE) return hipErrorInvalidValue;
  if (a.b.t == 0) return hipSuccess;
  const int64_t groups = (a.b.t + kTokens - 1) / kTokens;
  const dim3 grid(static_cast<unsigned>(groups < 4096 ? groups : 4096));
  const bool vec = a.b.n_experts % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(a.b.logits) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.dlogits) % 16 == 0;
  by_experts(a.b.n_experts, vec, [&](auto nv, auto v) {
    if (a.b.sigmoid)
      hipLaunchKernelGGL((router_backward_kernel<true, nv.value, v.value>), grid, dim3(kThreads),
                         0, s, a);
    else
      hipLaunchKernelGGL((router_backward_kernel<false, nv.value, v.value>), grid, dim3(kThreads),
                         0, s, a);
  });
  return hipGetLastError();
}

}  // namespace tq4
