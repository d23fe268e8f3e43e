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
constexpr float kNoneF = -__builtin_inff();

// ---- one token by one wave, all in fp64 -------------------------------------
// Any number of groups and slots.  Lane l holds experts l, l + 64, ...

__device__ inline double wave_max(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = __builtin_fmax(v, __shfl_xor(v, d));
  return v;
}

__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// The largest (value, index) over the wave, ties to the lower index.
__device__ inline void wave_best(double &v, int &i) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double ov = __shfl_xor(v, d);
    const int oi = __shfl_xor(i, d);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

// A wave's LDS writes before its later reads.
__device__ inline void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Writes the token's ids[0 .. topk) and w[0 .. topk); gv: kMaxExperts doubles of
// the wave's own LDS.  n_experts <= 64 PER, topk <= 64 SLOTS.
template <int PER, int SLOTS>
__device__ inline void route_token_f64(const float *__restrict__ row, const RouterConfig &cfg,
                                       const float *__restrict__ bias, double *gv, int lane,
                                       int32_t *ids, float *w) {
  double p[PER], c[PER];
  double top = kNone;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    const float l = e < cfg.n_experts ? row[e] : kNoneF;
    // the comparison also rejects NaN
    c[i] = l > kNoneF ? static_cast<double>(__builtin_fminf(l, 3.402823466e38f)) : kNone;
    top = __builtin_fmax(top, c[i]);
  }
  if (cfg.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] = c[i] > kNone ? 1.0 / (1.0 + exp(-c[i])) : 0.0;
  } else {
    top = wave_max(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      p[i] = c[i] > kNone ? exp(c[i] - top) : 0.0;
      sum += p[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] = sum > 0.0 ? p[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    if (c[i] > kNone) {
      c[i] = p[i] + (bias != nullptr ? static_cast<double>(bias[e]) : 0.0);
      if (!(c[i] > kNone)) c[i] = kNone;
    }
  }

  if (cfg.n_groups > 1) {
    // values to LDS; lane g then sums its groups' two largest
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i < cfg.n_experts) gv[lane + 64 * i] = c[i];
    wave_lds_fence();
    const int per = cfg.n_experts / cfg.n_groups;
    double gs[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
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
      for (int j = 0; j < PER; ++j)
        if (!((kept >> j) & 1u) && gs[j] > bv) {
          bv = gs[j];
          bi = lane + 64 * j;
        }
      wave_best(bv, bi);
      if (bv > kNone && lane == bi % 64) kept |= 1u << (bi / 64);
    }
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (lane + 64 * j < cfg.n_groups) gv[lane + 64 * j] = (kept >> j) & 1u ? 1.0 : 0.0;
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 64 * i;
      if (e < cfg.n_experts && gv[e / per] == 0.0) c[i] = kNone;
    }
    wave_lds_fence();
  }

  // slot j is kept by lane j % 64, in its register j / 64
  uint32_t taken = 0;
  double total = 0.0;
  double slot_w[SLOTS];
  int slot_id[SLOTS];
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    slot_w[q] = 0.0;
    slot_id[q] = -1;
  }
  for (int j = 0; j < cfg.topk; ++j) {
    double bv = kNone, bp = 0.0;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < PER; ++i)
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
    for (int q = 0; q < SLOTS; ++q)
      if (j == lane + 64 * q) {
        slot_w[q] = bp;
        slot_id[q] = bi;
      }
  }
  double f = static_cast<double>(cfg.scale);
  if (cfg.renormalize) f = total > 0.0 ? f / total : 0.0;
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    const int j = lane + 64 * q;
    if (j < cfg.topk) {
      ids[j] = slot_id[q];
      w[j] = static_cast<float>(slot_w[q] * f);
    }
  }
}

__global__ __launch_bounds__(256) void router_f64_kernel(
    const float *__restrict__ logits, int64_t t, RouterConfig cfg,
    const float *__restrict__ bias, int32_t *__restrict__ ids, float *__restrict__ w) {
  __shared__ double group[4][kMaxExperts];
  const int wave = threadIdx.x / 64;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (tok >= t) return;
  route_token_f64<kPer, kPer>(logits + tok * cfg.n_experts, cfg, bias, group[wave], threadIdx.x % 64,
                  ids + tok * cfg.topk, w + tok * cfg.topk);
}

// ---- four tokens by one wave, decided in fp32 where that decides --------------
// Sixteen lanes (a DPP row) per token, lane l with the P experts l P ... .
// Choice values are formed in fp32.  Their errors: a score comes from exp2 of a
// rounded product, so it is off by 2^-24 |x| p for the exponent x (l, or l - top
// for a softmax) and a few steps more; added to a bias, by 2^-24 |c| more.
// Relative to the token's largest score pmax that is at most 2^-20 + 2^-23
// |top| (p |l| is largest at the top for negative logits, and at most 0.28
// otherwise; p (top - l) is at most pmax / e).
// The topk + 1 largest are found with ties to the lower id.  If each is further
// from the next than both errors, or, among the chosen, has the very same logit
// and bias (then so are the exact values, and the lower id is right), their
// order is the exact one.  Groups likewise: only the border between the kept
// and the others has to be clear, of sums of two.  A token that fails a test
// (about 1 in 300 of random ones) is done again by route_token_f64.  Weights
// are formed from the chosen logits in fp64; only a softmax without
// renormalization needs all of them for that.
// Bound by its instructions, not by the logits' bytes.

template <int CTRL>
__device__ inline float dpp_f(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ inline int dpp_i(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ inline double dpp_d(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = dpp_i<CTRL>(static_cast<int>(b));
  const uint32_t hi = dpp_i<CTRL>(static_cast<int>(b >> 32));
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Over the 16 lanes of a row: partners l ^ 1, l ^ 2, 7 - l and 15 - l, each
// combine commutative, so every lane ends with the same result.
template <class F>
__device__ inline float row_reduce(float v, F f) {
  v = f(v, dpp_f<0xB1>(v));
  v = f(v, dpp_f<0x4E>(v));
  v = f(v, dpp_f<0x141>(v));
  return f(v, dpp_f<0x140>(v));
}
__device__ inline float row_max(float v) {
  return row_reduce(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ inline float row_sum(float v) {
  return row_reduce(v, [](float a, float b) { return a + b; });
}
__device__ inline double row_sum_f64(double v) {
  v += dpp_d<0xB1>(v);
  v += dpp_d<0x4E>(v);
  v += dpp_d<0x141>(v);
  return v + dpp_d<0x140>(v);
}
__device__ inline int row_min(int v) {
  int o = dpp_i<0xB1>(v);
  v = o < v ? o : v;
  o = dpp_i<0x4E>(v);
  v = o < v ? o : v;
  o = dpp_i<0x141>(v);
  v = o < v ? o : v;
  o = dpp_i<0x140>(v);
  return o < v ? o : v;
}

constexpr int kFastGroups = 16;  // groups the row's lanes hold
constexpr int kFastSlots = 15;   // slots, with the runner-up in one more lane

// exp(x), off by at most (2^-24 |x| + 2^-22) of itself.
__device__ inline float exp_fast(float x) {
  return __builtin_amdgcn_exp2f(x * 0x1.715476p+0f);
}

template <int P>
__global__ __launch_bounds__(64) void router_fast_kernel(
    const float *__restrict__ logits, int64_t t, RouterConfig cfg,
    const float *__restrict__ bias, int32_t *__restrict__ ids, float *__restrict__ w) {
  // four tokens' choice values where groups do not fall on lanes; the fp64
  // pass uses the space afterwards
  constexpr int kRow = 16 * P + 1;
  constexpr int kBytes = 4 * kRow * 4 > kMaxExperts * 8 ? 4 * kRow * 4 : kMaxExperts * 8;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kBytes];
  const int lane = threadIdx.x;
  const int l16 = lane % 16;
  const int64_t tok_raw = static_cast<int64_t>(blockIdx.x) * 4 + lane / 16;
  const bool real = tok_raw < t;
  const int64_t tok = real ? tok_raw : t - 1;  // spare rows repeat the last token
  const int n = cfg.n_experts;
  const float *row = logits + tok * n;
  const int e0 = l16 * P;

  float l[P], c[P];
  const bool full = n == 16 * P && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(bias) % 16 == 0;
  if (full) {
#pragma unroll
    for (int q = 0; q < P; q += 4) {
      const float4 d = *reinterpret_cast<const float4 *>(row + e0 + q);
      l[q] = d.x;
      l[q + 1] = d.y;
      l[q + 2] = d.z;
      l[q + 3] = d.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float d = row[e0 + i < n ? e0 + i : n - 1];
      l[i] = e0 + i < n ? d : kNoneF;
    }
  }
  if (bias == nullptr) {
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] = 0.f;
  } else if (full) {
#pragma unroll
    for (int q = 0; q < P; q += 4) {
      const float4 d = *reinterpret_cast<const float4 *>(bias + e0 + q);
      c[q] = d.x;
      c[q + 1] = d.y;
      c[q + 2] = d.z;
      c[q + 3] = d.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] = bias[e0 + i < n ? e0 + i : n - 1];
  }
  float top = kNoneF;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    // (fmax takes the other operand for a NaN: masked as well)
    l[i] = __builtin_fminf(__builtin_fmaxf(l[i], kNoneF), 3.402823466e38f);
    top = __builtin_fmaxf(top, l[i]);
  }
  top = row_max(top);
  const bool any = top > kNoneF;
  const float m = any ? top : 0.f;

  // scores and choice values
  float pmax;
  if (cfg.sigmoid) {
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] += __builtin_amdgcn_rcpf(1.f + exp_fast(-l[i]));
    pmax = __builtin_amdgcn_rcpf(1.f + exp_fast(-m));
  } else {
    float z[P];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      z[i] = exp_fast(l[i] - m);
      sum += z[i];
    }
    sum = row_sum(sum);
    const float inv = any ? __builtin_amdgcn_rcpf(sum) : 0.f;
    pmax = inv;  // the top expert's score
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] += z[i] * inv;
  }
  // an expert is off if its logit is, or its bias is -inf or NaN
  float cmax = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    c[i] = l[i] > kNoneF ? __builtin_fmaxf(c[i], kNoneF) : kNoneF;
    cmax = __builtin_fmaxf(cmax, c[i] > kNoneF ? __builtin_fabsf(c[i]) : 0.f);
  }
  cmax = row_max(cmax);
  // the error of one choice value, at most (infinite if a bias is: then the
  // token is left to fp64)
  const float err = pmax * (0x1p-20f + 0x1p-23f * __builtin_fabsf(m)) + 0x1p-23f * cmax + 0x1p-110f;
  bool clear = err < __builtin_inff();

  if (cfg.n_groups > 1) {
    // the two largest of each group
    float a = kNoneF, b = kNoneF;
    auto take = [&](float x) __attribute__((always_inline)) {
      b = __builtin_fmaxf(b, __builtin_fminf(a, x));
      a = __builtin_fmaxf(a, x);
    };
    const int span = 16 / cfg.n_groups;  // lanes per group
    const bool on_lanes = n == 16 * P && 16 % cfg.n_groups == 0;
    if (on_lanes) {
#pragma unroll
      for (int i = 0; i < P; ++i) take(c[i]);
      auto merge = [&](float oa, float ob) __attribute__((always_inline)) {
        b = __builtin_fmaxf(__builtin_fminf(a, oa), __builtin_fmaxf(b, ob));
        a = __builtin_fmaxf(a, oa);
      };
      if (span >= 2) merge(dpp_f<0xB1>(a), dpp_f<0xB1>(b));
      if (span >= 4) merge(dpp_f<0x4E>(a), dpp_f<0x4E>(b));
      if (span >= 8) merge(dpp_f<0x141>(a), dpp_f<0x141>(b));
    } else {
      float *gv = reinterpret_cast<float *>(smem) + (lane / 16) * kRow;
#pragma unroll
      for (int i = 0; i < P; ++i) gv[e0 + i] = c[i];
      wave_lds_fence();
      const int per = n / cfg.n_groups;
      if (l16 < cfg.n_groups)
        for (int e = l16 * per; e < (l16 + 1) * per; ++e) take(gv[e]);
    }
    const float gs = b > kNoneF ? a + b : a;
    // a group's rank: how many come before it (row_ror:s brings lane l - s)
    const int step = on_lanes ? span : 1;
    const int mine = l16 / step;
    int rank = 0;
    auto before = [&](float o, int s) __attribute__((always_inline)) {
      const int j = ((l16 - s) & 15) / step;
      rank += (o > gs || (o == gs && j < mine)) ? 1 : 0;
    };
    if (step < 2) {
      before(dpp_f<0x121>(gs), 1);
      before(dpp_f<0x123>(gs), 3);
      before(dpp_f<0x125>(gs), 5);
      before(dpp_f<0x127>(gs), 7);
      before(dpp_f<0x129>(gs), 9);
      before(dpp_f<0x12B>(gs), 11);
      before(dpp_f<0x12D>(gs), 13);
      before(dpp_f<0x12F>(gs), 15);
    }
    if (step < 4) {
      before(dpp_f<0x122>(gs), 2);
      before(dpp_f<0x126>(gs), 6);
      before(dpp_f<0x12A>(gs), 10);
      before(dpp_f<0x12E>(gs), 14);
    }
    if (step < 8) {
      before(dpp_f<0x124>(gs), 4);
      before(dpp_f<0x12C>(gs), 12);
    }
    before(dpp_f<0x128>(gs), 8);
    const bool keep = rank < cfg.topk_groups && gs > kNoneF;
    const float last = -row_max(keep ? -gs : kNoneF);
    const float next = row_max(keep ? kNoneF : gs);
    // (no group kept, or no other left: last or next is infinite)
    clear = clear && last - next > 2.f * (2.f * err + 0x1p-23f * cmax);
    if (on_lanes) {
#pragma unroll
      for (int i = 0; i < P; ++i) c[i] = keep ? c[i] : kNoneF;
    } else {
      const uint32_t mask = static_cast<uint32_t>(__ballot(keep) >> (lane & 48)) & 0xFFFFu;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        // e / per, exact: e < 512, the reciprocal rounded up to 2^-20
        const uint32_t grp = static_cast<uint32_t>(e0 + i) * cfg.per_inv >> 20;
        if (!((mask >> (grp & 31u)) & 1u)) c[i] = kNoneF;
      }
    }
  }

  // the topk + 1 largest, result j in lane j of the row
  float my_c = kNoneF;
  int my_id = -1;
  for (int j = 0; j <= cfg.topk; ++j) {
    float best = c[0];
#pragma unroll
    for (int i = 1; i < P; ++i) best = __builtin_fmaxf(best, c[i]);
    best = row_max(best);
    int pos = P;  // the lane's lowest position of it
#pragma unroll
    for (int i = P - 1; i >= 0; --i) pos = c[i] == best ? i : pos;
    const int at = row_min(pos < P ? e0 + pos : 0x7FFFFFFF);
    if (l16 == j && best > kNoneF) {
      my_c = best;
      my_id = at;
    }
    const int gone = at - e0;
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] = i == gone ? kNoneF : c[i];
  }

  // each result against the next one (row_shl:1 brings lane l + 1)
  const bool found = my_id >= 0;
  const float my_l = found ? row[my_id] : 0.f;
  const float my_b = found && bias != nullptr ? bias[my_id] : 0.f;
  const float next_c = dpp_f<0x101>(my_c);
  const float next_l = dpp_f<0x101>(my_l);
  const float next_b = dpp_f<0x101>(my_b);
  const int next_id = dpp_i<0x101>(my_id);
  // without a bias the errors are relative to the values themselves (for a
  // softmax, that of l - top as well)
  const float tol = bias != nullptr
                        ? 2.f * err
                        : my_c * (0x1p-18f + 0x1p-21f * (cfg.sigmoid ? __builtin_fabsf(my_l) : top - my_l));
  const bool apart = my_c - next_c > tol && (bias != nullptr || my_c > 0x1p-100f);
  // at the last slot equal inputs do not settle it: a third expert may be near
  const bool equal = my_l == next_l && my_b == next_b && l16 + 1 < cfg.topk;
  if (l16 < cfg.topk && found && next_id >= 0 && !apart && !equal) clear = false;

  // weights of the chosen, in fp64
  const bool chosen = found && l16 < cfg.topk;
  const double dl = static_cast<double>(__builtin_fminf(my_l, 3.402823466e38f));
  double p = 0.0;
  if (cfg.sigmoid) {
    if (chosen) p = 1.0 / (1.0 + exp(-dl));
  } else {
    if (chosen) p = exp(dl - static_cast<double>(top));
    if (!cfg.renormalize) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < P; ++i)
        sum += l[i] > kNoneF ? exp(static_cast<double>(l[i]) - static_cast<double>(top)) : 0.0;
      sum = row_sum_f64(sum);
      if (chosen) p /= sum;
    }
  }
  double f = static_cast<double>(cfg.scale);
  if (cfg.renormalize) {
    const double total = row_sum_f64(p);
    f = total > 0.0 ? f / total : 0.0;
  }
  if (real && l16 < cfg.topk) {
    ids[tok * cfg.topk + l16] = my_id;
    w[tok * cfg.topk + l16] = static_cast<float>(p * f);
  }

  // unclear tokens again, one after another, by the whole wave
  uint64_t again = __ballot(real && !clear);
  while (again != 0) {
    const int first = __builtin_ctzll(again) & 48;
    again &= ~(0xFFFFull << first);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + first / 16;
    wave_lds_fence();
    route_token_f64<P / 4, 1>(logits + at * n, cfg, bias, reinterpret_cast<double *>(smem), lane,
                    ids + at * cfg.topk, w + at * cfg.topk);
  }
}

}  // namespace

hipError_t launch_router_scored(const float *logits, int64_t t, const RouterConfig &config,
                                const float *bias, int32_t *ids, float *w, hipStream_t s) {
  if (t == 0) return hipSuccess;
  RouterConfig cfg = config;
  const int32_t per = cfg.n_experts / cfg.n_groups;
  cfg.per_inv = static_cast<uint32_t>(((1 << 20) + per - 1) / per);
  if (cfg.topk > kFastSlots || cfg.n_groups > kFastGroups) {
    hipLaunchKernelGGL(router_f64_kernel, dim3(static_cast<unsigned>((t + 3) / 4)), dim3(256), 0,
                       s, logits, t, cfg, bias, ids, w);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>((t + 3) / 4));
  if (cfg.n_experts <= 64)
    hipLaunchKernelGGL(router_fast_kernel<4>, grid, dim3(64), 0, s, logits, t, cfg, bias, ids, w);
  else if (cfg.n_experts <= 128)
    hipLaunchKernelGGL(router_fast_kernel<8>, grid, dim3(64), 0, s, logits, t, cfg, bias, ids, w);
  else if (cfg.n_experts <= 256)
    hipLaunchKernelGGL(router_fast_kernel<16>, grid, dim3(64), 0, s, logits, t, cfg, bias, ids,
                       w);
  else
    hipLaunchKernelGGL(router_fast_kernel<32>, grid, dim3(64), 0, s, logits, t, cfg, bias, ids,
                       w);
  return hipGetLastError();
}

}  // namespace tq4
