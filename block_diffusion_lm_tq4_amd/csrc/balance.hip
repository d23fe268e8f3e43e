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
// no row under- or overflows; sums over tokens are fp32 within a lane, fp64 beyond.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mxfp4.h"

namespace tq4 {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kLanes = 16;                 // lanes of a token
constexpr int kTokens = kThreads / kLanes; // tokens of a workgroup at a time
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
// log2(e), times the first two terms of e^r for what its rounding left.
__device__ inline float exp_neg(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kLow = 0x1.4ae0cp-26f;  // log2(e) in two parts
  constexpr float kLn2 = 0x1.62e43p-1f;
  const float t = x * kLog2e;
  const float r = __builtin_fmaf(x, kLow, __builtin_fmaf(x, kLog2e, -t)) * kLn2;
  const float e = __builtin_amdgcn_exp2f(t);
  return t > -150.f ? __builtin_fmaf(e, r, e) : 0.f;  // also for x = -inf
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
    top = kOff;
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
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        l[i][v] = usable(l[i][v]);
        top = __builtin_fmaxf(top, l[i][v]);
      }
    }
    top = row_max(top);
  }
};

// A score relative to e^top (softmax) or to e^min(top, 0) (sigmoid), and 1 - p of the
// sigmoid.
template <bool SIGMOID>
__device__ inline float score(float l, float top, float &rest) {
  if constexpr (SIGMOID) {
    const float inv = __builtin_amdgcn_rcpf(1.f + exp_neg(-__builtin_fabsf(l)));
    rest = exp_neg(-__builtin_fmaxf(l, 0.f)) * inv;
    return exp_neg(__builtin_fminf(l, 0.f) - __builtin_fminf(top, 0.f)) * inv;
  } else {
    rest = 1.f;
    return exp_neg(l - top);
  }
}

// Scores of a whole row and 1 / their sum (0 for a row without experts).
template <bool SIGMOID, int NV, bool VEC>
__device__ inline float row_scores(const Row<NV, VEC> &row, float (&p)[NV][4],
                                   float (&rest)[NV][4]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float s = score<SIGMOID>(row.l[i][v], row.top, rest[i][v]);
      p[i][v] = row.l[i][v] > kOff ? s : 0.f;
      sum += p[i][v];
    }
  sum = row_sum(sum);
  return sum > 0.f ? 1.f / sum : 0.f;
}

__device__ inline bool routed(int id, int n_experts) { return id >= 0 && id < n_experts; }

// Whether the token has an id in range (all lanes of the token agree).
__device__ inline bool row_live(const int32_t *ids, int topk, int n_experts, int lane) {
  float any = 0.f;
  for (int j = lane; j < topk; j += kLanes) any = routed(ids[j], n_experts) ? 1.f : any;
  return row_max(any) > 0.f;
}

// ---- counts, mean probabilities, loss ----------------------------------------

// A workgroup's share of the tokens: its sums of q and its counts go to scratch
// ([groups][E] fp32, [groups][E] int32, [groups] int32).
template <bool SIGMOID, int NV, bool VEC>
__global__ __launch_bounds__(kThreads) void balance_sums_kernel(BalanceArgs a, float *part_p,
                                                                int32_t *part_c, int32_t *part_t) {
  __shared__ float sums[kTokens][64 * NV];
  __shared__ int32_t hist[64 * NV];
  __shared__ int32_t tokens;
  const int tid = threadIdx.x;
  const int lane = tid % kLanes, group = tid / kLanes;
  for (int e = tid; e < 64 * NV; e += kThreads) hist[e] = 0;
  if (tid == 0) tokens = 0;
  __syncthreads();
  float acc[NV][4] = {};
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + group; t < a.t;
       t += static_cast<int64_t>(gridDim.x) * kTokens) {
    const int32_t *ids = a.ids + t * a.topk;
    bool any = false;
    for (int j = lane; j < a.topk; j += kLanes) {
      const int id = ids[j];
      if (!routed(id, a.n_experts)) continue;
      atomicAdd(&hist[id], 1);
      any = true;
    }
    if (row_max(any ? 1.f : 0.f) == 0.f) continue;  // routed nowhere
    if (lane == 0) atomicAdd(&tokens, 1);
    Row<NV, VEC> row;
    row.load(a.logits + t * a.n_experts, a.n_experts, lane);
    float p[NV][4], rest[NV][4];
    const float inv = row_scores<SIGMOID, NV, VEC>(row, p, rest);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][v] += p[i][v] * inv;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) sums[group][64 * i + 4 * lane + v] = acc[i][v];
  __syncthreads();
  for (int e = tid; e < a.n_experts; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kTokens; ++g) s += sums[g][e];
    part_p[static_cast<int64_t>(blockIdx.x) * a.n_experts + e] = s;
    part_c[static_cast<int64_t>(blockIdx.x) * a.n_experts + e] = hist[e];
  }
  if (tid == 0) part_t[blockIdx.x] = tokens;
}

constexpr int kFinalThreads = 1024;

// One workgroup adds the groups' sums in a fixed order, fp64.
__global__ __launch_bounds__(kFinalThreads) void balance_loss_kernel(
    const float *__restrict__ part_p, const int32_t *__restrict__ part_c,
    const int32_t *__restrict__ part_t, int groups, int n_experts, float *loss, int32_t *counts,
    int32_t *tokens, float *mean_p) {
  __shared__ double sp[kFinalThreads];
  __shared__ int32_t sc[kFinalThreads];
  __shared__ int32_t st;
  __shared__ double dot[kFinalThreads / 64];
  __shared__ int64_t all[kFinalThreads / 64];
  const int tid = threadIdx.x;
  int cols = 1;
  while (cols < n_experts) cols *= 2;
  const int parts = kFinalThreads / cols;
  const int e = tid % cols, part = tid / cols;
  double p = 0.0;
  int32_t c = 0;
  if (e < n_experts)
    for (int g = part; g < groups; g += parts) {
      p += static_cast<double>(part_p[g * n_experts + e]);
      c += part_c[g * n_experts + e];
    }
  sp[tid] = p;
  sc[tid] = c;
  if (tid == 0) st = 0;
  __syncthreads();
  int32_t t = 0;
  for (int g = tid; g < groups; g += kFinalThreads) t += part_t[g];
  if (t != 0) atomicAdd(&st, t);
  __syncthreads();
  const int32_t live = st;
  double part_dot = 0.0;
  int64_t part_all = 0;
  if (tid < n_experts) {
    for (int q = 1; q < parts; ++q) {
      p += sp[q * cols + e];
      c += sc[q * cols + e];
    }
    const double mean = live > 0 ? p / static_cast<double>(live) : 0.0;
    counts[e] = c;
    mean_p[e] = static_cast<float>(mean);
    part_dot = mean * static_cast<double>(c);
    part_all = c;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    part_dot += __shfl_xor(part_dot, d);
    part_all += __shfl_xor(part_all, d);
  }
  if (tid % 64 == 0) {
    dot[tid / 64] = part_dot;
    all[tid / 64] = part_all;
  }
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    int64_t n = 0;
    for (int w = 0; w < kFinalThreads / 64; ++w) {
      s += dot[w];
      n += all[w];
    }
    *loss = n > 0 ? static_cast<float>(n_experts * s / static_cast<double>(n)) : 0.f;
    *tokens = live;
  }
}

// ---- gradient ------------------------------------------------------------------

// The gates' contributions of one token to `delta` (its row of LDS), and what a softmax
// without renormalization takes from every expert (sum_j p_j a_j).  Lane j of the
// token takes slots j, j + 16, ....
template <bool SIGMOID>
__device__ inline float gate_part(const RouterGradArgs &g, int64_t t, float top, float inv,
                                  float *delta, int lane) {
  const float *row = g.b.logits + t * g.b.n_experts;
  const int32_t *ids = g.b.ids + t * g.b.topk;
  const float *dw = g.dgates + t * g.b.topk;
  const int blocks = (g.b.topk + kLanes - 1) / kLanes;
  auto slot = [&](int b, int &id, float &l, float &d) __attribute__((always_inline)) {
    const int j = b * kLanes + lane;
    id = j < g.b.topk ? ids[j] : -1;
    l = kOff;
    d = 0.f;
    if (routed(id, g.b.n_experts)) {
      l = usable(row[id]);
      d = dw[j];
    } else {
      id = -1;
    }
  };
  float base = top, norm = inv, mean = 0.f;
  if (g.renormalize) {  // scores relative to the largest chosen one
    base = kOff;
    for (int b = 0; b < blocks; ++b) {
      int id;
      float l, d;
      slot(b, id, l, d);
      base = __builtin_fmaxf(base, l);
    }
    base = row_max(base);
    float sum = 0.f, dot = 0.f;
    for (int b = 0; b < blocks; ++b) {
      int id;
      float l, d, rest;
      slot(b, id, l, d);
      const float p = l > kOff ? score<SIGMOID>(l, base, rest) : 0.f;
      sum += p;
      dot += p * d;
    }
    sum = row_sum(sum);
    norm = sum > 0.f ? 1.f / sum : 0.f;
    mean = row_sum(dot) * norm;
  } else if (SIGMOID) {  // the scores themselves
    base = 0.f;
    norm = 1.f;
  }
  float taken = 0.f;
  for (int b = 0; b < blocks; ++b) {
    int id;
    float l, d, rest = 1.f;
    slot(b, id, l, d);
    const float p = l > kOff ? score<SIGMOID>(l, base, rest) * norm : 0.f;
    float add = p * (g.scale * (d - mean));
    taken += add;
    if (SIGMOID) add *= rest;
    // slots of one expert: the lowest lane adds the others', always in the same order
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
  return SIGMOID || g.renormalize ? 0.f : row_sum(taken);
}

// 16 lanes per token, 16 tokens per workgroup at a time.
template <bool SIGMOID, int NV, bool VEC>
__global__ __launch_bounds__(kThreads) void router_backward_kernel(RouterGradArgs g) {
  __shared__ __attribute__((aligned(16))) float delta_all[kTokens][64 * NV];
  __shared__ __attribute__((aligned(16))) float share[64 * NV];  // c_e of the loss
  __shared__ int32_t total[kThreads / 64];
  const int tid = threadIdx.x;
  const int lane = tid % kLanes, group = tid / kLanes;
  const int n_experts = g.b.n_experts;
  const bool has_loss = g.counts != nullptr;
  if (has_loss) {
    int32_t n = 0;
    for (int e = tid; e < n_experts; e += kThreads) n += g.counts[e];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
    if (tid % 64 == 0) total[tid / 64] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kThreads / 64; ++w) n += total[w];
    const double pairs = n, tokens = *g.tokens;
    const double c0 = pairs > 0.0 && tokens > 0.0
                          ? static_cast<double>(*g.dloss) * n_experts / (pairs * tokens)
                          : 0.0;
    for (int e = tid; e < 64 * NV; e += kThreads)
      share[e] = e < n_experts ? static_cast<float>(c0 * g.counts[e]) : 0.f;
  }
  __syncthreads();
  float *delta = delta_all[group];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + group; t < g.b.t;
       t += static_cast<int64_t>(gridDim.x) * kTokens) {
    Row<NV, VEC> row;
    row.load(g.b.logits + t * n_experts, n_experts, lane);
    float p[NV][4], rest[NV][4];
    const float inv = row_scores<SIGMOID, NV, VEC>(row, p, rest);
    float taken = 0.f;
    if (g.dgates != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        *reinterpret_cast<floatx4 *>(delta + 64 * i + 4 * lane) = floatx4{0.f, 0.f, 0.f, 0.f};
      wave_lds_fence();
      taken = gate_part<SIGMOID>(g, t, row.top, inv, delta, lane);
    }
    floatx4 c[NV];
    float dot = 0.f;
    const bool live =
        has_loss && row_live(g.b.ids + t * g.b.topk, g.b.topk, n_experts, lane);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = live ? *reinterpret_cast<const floatx4 *>(share + 64 * i + 4 * lane)
                  : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        p[i][v] *= inv;
        dot += p[i][v] * c[i][v];
      }
    }
    dot = row_sum(dot) + taken;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 64 * i + 4 * lane;
      floatx4 d = {0.f, 0.f, 0.f, 0.f};
      if (g.dgates != nullptr) d = *reinterpret_cast<const floatx4 *>(delta + e);
#pragma unroll
      for (int v = 0; v < 4; ++v) d[v] += p[i][v] * rest[i][v] * (c[i][v] - dot);
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

int balance_groups(int64_t t) {
  const int64_t groups = (t + 4 * kTokens - 1) / (4 * kTokens);
  return static_cast<int>(groups < 1 ? 1 : (groups < 256 ? groups : 256));
}

hipError_t launch_moe_balance(const BalanceArgs &a, float *loss, int32_t *counts, int32_t *tokens,
                              float *mean_p, void *scratch, hipStream_t s) {
  if (a.n_experts < 1 || a.n_experts > kMaxE) return hipErrorInvalidValue;
  const int groups = balance_groups(a.t);
  float *part_p = static_cast<float *>(scratch);
  int32_t *part_c = reinterpret_cast<int32_t *>(part_p + groups * a.n_experts);
  int32_t *part_t = part_c + groups * a.n_experts;
  const bool vec = a.n_experts % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  by_experts(a.n_experts, vec, [&](auto nv, auto v) {
    if (a.sigmoid)
      hipLaunchKernelGGL((balance_sums_kernel<true, nv.value, v.value>), dim3(groups),
                         dim3(kThreads), 0, s, a, part_p, part_c, part_t);
    else
      hipLaunchKernelGGL((balance_sums_kernel<false, nv.value, v.value>), dim3(groups),
                         dim3(kThreads), 0, s, a, part_p, part_c, part_t);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(kFinalThreads), 0, s, part_p, part_c,
                     part_t, groups, a.n_experts, loss, counts, tokens, mean_p);
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
