// The general router in front of the MoE layer (Nemotron-TheHobbit-30B-A3B
// model card, The model underneath: 128 experts, top-6): softmax or sigmoid
// scores, a balance bias that only the choice sees, groups of experts of
// which the best are kept, and weights that may be renormalized and scaled.
//
// Per token, with scores p_e and choice values c_e = p_e + bias_e:
//   - an expert whose logit is -inf or NaN, or whose c is, is never chosen;
//   - with groups, a group's value is the sum of its two largest c (of the
//     one, if only one may be chosen); the keep groups with the largest values
//     stay (ties to the lower group);
//   - the topk largest c of what stays are the token's experts, in decreasing
//     order, ties to the lower id; slots left over get id -1 and weight 0;
//   - weights are the scores p (divided by the sum of the token's, if asked
//     for and not zero) times a factor.
// Scores and comparisons are fp64: two experts a few fp32 ulps apart are
// common among thousands of tokens, and the choice must not depend on how a
// score was rounded.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq4_internal.h"

namespace tq4 {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kPer = kMaxExperts / 64;
constexpr double kNone = -__builtin_inf();

__device__ inline double shfl_xor_f64(double v, int d) {
  return __shfl_xor(v, d);
}

__device__ inline double wave_max(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = __builtin_fmax(v, shfl_xor_f64(v, d));
  return v;
}

__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += shfl_xor_f64(v, d);
  return v;
}

// The largest (value, index) over the wave, ties to the lower index.
__device__ inline void wave_best(double &v, int &i) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double ov = shfl_xor_f64(v, d);
    const int oi = __shfl_xor(i, d);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

// One wave per token; lane l holds experts l, l + 64, ...
__global__ __launch_bounds__(256) void router_scored_kernel(
    const float *__restrict__ logits, int64_t t, RouterConfig cfg,
    const float *__restrict__ bias, int32_t *__restrict__ ids, float *__restrict__ w) {
  __shared__ double group[4][kMaxExperts];
  const int wave = threadIdx.x / 64;
  const int lane = threadIdx.x % 64;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (tok >= t) return;
  const float *row = logits + tok * cfg.n_experts;

  double p[kPer], c[kPer];
  double top = kNone;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    const float l = e < cfg.n_experts ? row[e] : -__builtin_inff();
    // the sign test also rejects NaN
    c[i] = l > -__builtin_inff() ? static_cast<double>(__builtin_fminf(l, 3.402823466e38f)) : kNone;
    top = __builtin_fmax(top, c[i]);
  }
  if (cfg.sigmoid) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] = c[i] > kNone ? 1.0 / (1.0 + exp(-c[i])) : 0.0;
  } else {
    top = wave_max(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      p[i] = c[i] > kNone ? exp(c[i] - top) : 0.0;
      sum += p[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] = sum > 0.0 ? p[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    if (c[i] > kNone) {
      c[i] = p[i] + (bias != nullptr ? static_cast<double>(bias[e]) : 0.0);
      if (!(c[i] > kNone)) c[i] = kNone;
    }
  }

  if (cfg.n_groups > 1) {
    // values to LDS; lane g then sums its groups' two largest
    double *gv = group[wave];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 64 * i < cfg.n_experts) gv[lane + 64 * i] = c[i];
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int per = cfg.n_experts / cfg.n_groups;
    double gs[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int grp = lane + 64 * j;
      gs[j] = kNone;
      if (grp < cfg.n_groups) {
        double a = kNone, b = kNone;
        for (int e = grp * per; e < (grp + 1) * per; ++e) {
          const double x = gv[e];
          b = __builtin_fmax(b, __builtin_fmin(a, x));
          a = __builtin_fmax(a, x);
        }
        gs[j] = b > kNone ? a + b : a;
      }
    }
    // mark the kept groups one after another
    uint32_t kept = 0;
    for (int n = 0; n < cfg.topk_groups; ++n) {
      double bv = kNone;
      int bi = 0x7FFFFFFF;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int grp = lane + 64 * j;
        if (!((kept >> j) & 1u) && (gs[j] > bv || (gs[j] == bv && gs[j] > kNone && grp < bi))) {
          bv = gs[j];
          bi = grp;
        }
      }
      wave_best(bv, bi);
      if (bv > kNone && lane == bi % 64) kept |= 1u << (bi / 64);
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (lane + 64 * j < cfg.n_groups) gv[lane + 64 * j] = (kept >> j) & 1u ? 1.0 : 0.0;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 64 * i;
      if (e < cfg.n_experts && gv[e / per] == 0.0) c[i] = kNone;
    }
  }

  // slot j is kept by lane j % 64, in its register j / 64
  uint32_t taken = 0;
  double total = 0.0;
  double slot_w[kPer];
  int slot_id[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    slot_w[q] = 0.0;
    slot_id[q] = -1;
  }
  for (int j = 0; j < cfg.topk; ++j) {
    double bv = kNone, bp = 0.0;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (!((taken >> i) & 1u) && c[i] > bv) {
        bv = c[i];
        bi = lane + 64 * i;
        bp = p[i];
      }
    const int own = bi;
    wave_best(bv, bi);
    if (!(bv > kNone)) break;  // nothing left to choose
    if (own == bi) taken |= 1u << (bi / 64);
    bp = __shfl(bp, bi % 64);
    total += bp;
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (j == lane + 64 * q) {
        slot_w[q] = bp;
        slot_id[q] = bi;
      }
  }
  double f = static_cast<double>(cfg.scale);
  if (cfg.renormalize) f = total > 0.0 ? f / total : 0.0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int j = lane + 64 * q;
    if (j < cfg.topk) {
      ids[tok * cfg.topk + j] = slot_id[q];
      w[tok * cfg.topk + j] = static_cast<float>(slot_w[q] * f);
    }
  }
}

}  // namespace

hipError_t launch_router_scored(const float *logits, int64_t t, const RouterConfig &cfg,
                                const float *bias, int32_t *ids, float *w, hipStream_t s) {
  if (t == 0) return hipSuccess;
  hipLaunchKernelGGL(router_scored_kernel, dim3(static_cast<unsigned>((t + 3) / 4)), dim3(256), 0,
                     s, logits, t, cfg, bias, ids, w);
  return hipGetLastError();
}

}  // namespace tq4
