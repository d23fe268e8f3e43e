// The general router in front of the MoE layer (Nemotron-TheHobbit-30B-A3B
// model card, The model underneath: 128 experts, top-6): softmax or sigmoid
// scores, a balance bias that only the choice sees, groups of experts of
// which the best are kept, and weights that may be renormalized and scaled.
//
// Per token, with scores p_e and choice values c_e = p_e + bias_e:
//   - an expert whose logit is -inf or NaN takes no part; one whose bias is only
//     cannot be chosen (its score still counts in the others' softmax);
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

#include "int8_router.h"

namespace tq4 {
namespace {

#include "moe_route.h"

constexpr int kPer = kMaxExperts / 64;
constexpr double kNone = -__builtin_inf();
constexpr float kNoneF = -__builtin_inff();

// ---- one token by one wave, all in fp64 -------------------------------------
// Any number of groups and slots.  Lane l holds experts l, l + 64, ....  Bound by the
// chain of fp64 reductions, one for each slot: 16411 tokens of 256 experts, 15 slots,
// 82 us captured, 8 slots of 8 among 32 groups 83; 1024 of 128 experts, 16 slots, 14.

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

// The values of lanes l and l ^ 16 (or l ^ 32), lower lane first.
template <int D>
__device__ inline void lane_pair_f64(double v, double &lower, double &upper) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  uint32_t l0, u0, l1, u1;
  if constexpr (D == 16) {
    lane_pair16(static_cast<uint32_t>(b), l0, u0);
    lane_pair16(static_cast<uint32_t>(b >> 32), l1, u1);
  } else {
    lane_pair32(static_cast<uint32_t>(b), l0, u0);
    lane_pair32(static_cast<uint32_t>(b >> 32), l1, u1);
  }
  lower = __builtin_bit_cast(double, static_cast<uint64_t>(l1) << 32 | l0);
  upper = __builtin_bit_cast(double, static_cast<uint64_t>(u1) << 32 | u0);
}

// Wave-wide reductions in registers: partners l ^ 1, l ^ 2, 7 - l and 15 - l
// within a row of 16 lanes, then l ^ 16 and l ^ 32; each combine commutative, so
// every lane ends with the same result.
template <class F>
__device__ inline double row_reduce_f64(double v, F f) {
  v = f(v, dpp_d<0xB1>(v));
  v = f(v, dpp_d<0x4E>(v));
  v = f(v, dpp_d<0x141>(v));
  return f(v, dpp_d<0x140>(v));
}
template <class F>
__device__ inline double wave_reduce_f64(double v, F f) {
  v = row_reduce_f64(v, f);
  double lo, hi;
  lane_pair_f64<16>(v, lo, hi);
  v = f(lo, hi);
  lane_pair_f64<32>(v, lo, hi);
  return f(lo, hi);
}
__device__ inline double wave_max(double v) {
  return wave_reduce_f64(v, [](double a, double b) { return __builtin_fmax(a, b); });
}
__device__ inline double wave_sum(double v) {
  return wave_reduce_f64(v, [](double a, double b) { return a + b; });
}
__device__ inline double row_sum_f64(double v) {
  return row_reduce_f64(v, [](double a, double b) { return a + b; });
}

// The largest (value, index) over the wave, ties to the lower index.
__device__ inline void better_f64(double &v, int &i, double ov, int oi) {
  if (ov > v || (ov == v && oi < i)) {
    v = ov;
    i = oi;
  }
}
__device__ inline void wave_best(double &v, int &i) {
  better_f64(v, i, dpp_d<0xB1>(v), dpp_i<0xB1>(i));
  better_f64(v, i, dpp_d<0x4E>(v), dpp_i<0x4E>(i));
  better_f64(v, i, dpp_d<0x141>(v), dpp_i<0x141>(i));
  better_f64(v, i, dpp_d<0x140>(v), dpp_i<0x140>(i));
  double vl, vh;
  uint32_t il, ih;
  lane_pair_f64<16>(v, vl, vh);
  lane_pair16(static_cast<uint32_t>(i), il, ih);
  v = vl;
  i = static_cast<int>(il);
  better_f64(v, i, vh, static_cast<int>(ih));
  lane_pair_f64<32>(v, vl, vh);
  lane_pair32(static_cast<uint32_t>(i), il, ih);
  v = vl;
  i = static_cast<int>(il);
  better_f64(v, i, vh, static_cast<int>(ih));
}

// A slot's weight from its expert's score p and the sum of the token's; 0 without
// an expert, and where the sum is, whatever the factor.  The quotient comes
// first: a sum below 2^-1022, as of experts that only their bias brought in, has
// no finite reciprocal.
__device__ inline float weight(bool found, double p, double total, const RouterConfig &cfg) {
  if (cfg.renormalize) {
    found = found && total > 0.0;
    p /= total;
  }
  const float w = static_cast<float>(p * static_cast<double>(cfg.scale));
  return found ? w : 0.f;
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
#pragma unroll
  for (int q = 0; q < SLOTS; ++q) {
    const int j = lane + 64 * q;
    if (j < cfg.topk) {
      ids[j] = slot_id[q];
      w[j] = weight(slot_id[q] >= 0, slot_w[q], total, cfg);
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
  route_token_f64<kPer, kPer>(logits + tok * cfg.n_experts, cfg, bias, group[wave],
                              threadIdx.x % 64, ids + tok * cfg.topk, w + tok * cfg.topk);
}

// ---- four tokens by one wave, decided in fp32 where that decides --------------
// Sixteen lanes (a DPP row) per token, lane l with the P experts l P ... .
// Choice values c are formed in fp32, and each becomes one integer that orders
// like it, its last 6 to 9 bits given to the expert (ties to the lower id), so
// that the largest of a token is found by integer maxima alone.  The topk + 2
// largest are candidates; their exact values (which the weights need anyway)
// are formed in fp64, one in each lane, and where two neighbours among them are
// near, the candidates are ranked by those.  The choice is then the exact one if
// the last candidate, above which no other expert is, lies clear of the last
// chosen by the fp32 values.  Groups likewise: the border between the kept and
// the others has to be clear.  A token that fails either test is done again by
// route_token_f64, a wave's four one after another: about 1 in 15000 of random
// logits, and all of them where fp32 cannot tell topk + 2 experts apart.  For
// 16411 tokens of 256 experts, 8 groups, sigmoid, 8 slots (us): N(0, 1.5) 15.5;
// rounded to bf16 15.8, without a bias 21.7; without a bias all equal, or N(12, 1.5)
// where sigmoid is flat, 87; under a bias of 1000 on each expert 71.
//
// "Clear" is more than both errors.  exp_fast is off by 2^-23 + 1.5 * 2^-24 |x|
// of itself.  A sigmoid score adds 1 + e and the reciprocal, 1.5 * 2^-23 more;
// with p (1 - p) |l| at most 0.23, or |l| p where the token's top logit is
// negative, that is at most pmax 2^-23 (3 + max(0, -top)), pmax the largest
// score.  A softmax score has the rounding of l - top as well, p (top - l) is
// at most pmax / e, and the sum's error is common to the token: at most 18 *
// 2^-23 pmax.  Adding the bias costs 2^-24 |c|.  Without a bias the errors are
// taken relative to the value itself.  Dropping B bits costs 2^(B - 23) |c|.
//
// Bound by its instructions, not by the logits' bytes: 16411 tokens of 256 experts
// (8 groups, sigmoid) 15.5 us captured, of which the bytes need 3.5, and 13.4 to 21.6
// (median 18.5) one call after another; a wave issues 1270 vector instructions for
// its four tokens, which keep the vector units busy in 75 % of the compute units'
// cycles.  1024 tokens of 128 experts: 3.9 us captured, 4.8 to 10.3 (5.1) one after
// another, the latency of one wave's chain (25 %).

// Over the 16 lanes of a row, as above.
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
__device__ inline int row_max_i(int v) {
  int o = dpp_i<0xB1>(v);
  v = o > v ? o : v;
  o = dpp_i<0x4E>(v);
  v = o > v ? o : v;
  o = dpp_i<0x141>(v);
  v = o > v ? o : v;
  o = dpp_i<0x140>(v);
  return o > v ? o : v;
}

constexpr int kFastGroups = 16;  // groups the row's lanes hold
constexpr int kFastSlots = 14;   // slots, with two more candidates in the lanes left

// exp(x), off by at most (1.5 * 2^-24 |x| + 2^-23) of itself.
__device__ inline float exp_fast(float x) {
  return __builtin_amdgcn_exp2f(x * 0x1.715476p+0f);
}

// (Workgroups of one wave took 26 us for 16411 tokens of 256 experts: 4103 of
// them are dispatched no faster.)
constexpr int kFastWaves = 4;

template <int P>
__global__ __launch_bounds__(64 * kFastWaves) void router_fast_kernel(
    const float *__restrict__ logits, int64_t t, RouterConfig cfg,
    const float *__restrict__ bias, int32_t *__restrict__ ids, float *__restrict__ w) {
  // four tokens' choice values where groups do not fall on lanes; the fp64
  // pass uses the space afterwards
  constexpr int kRow = 16 * P + 1;
  constexpr int kBytes = 4 * kRow * 4 > kMaxExperts * 8 ? 4 * kRow * 4 : kMaxExperts * 8;
  __shared__ __attribute__((aligned(16))) uint8_t all[kFastWaves][(kBytes + 15) / 16 * 16];
  uint8_t *smem = all[threadIdx.x / 64];
  const int lane = threadIdx.x % 64;
  const int l16 = lane % 16;
  // the wave's first token
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * (4 * kFastWaves) + threadIdx.x / 64 * 4;
  if (tok0 >= t) return;
  const int64_t tok_raw = tok0 + lane / 16;
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
  const float err =
      pmax * 0x1p-23f * (cfg.sigmoid ? 3.f + __builtin_fmaxf(0.f, -m) : 18.f) +
      0x1p-24f * cmax + 0x1p-110f;
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
    const int own = l16 / step;
    int rank = 0;
    auto before = [&](float o, int s) __attribute__((always_inline)) {
      const int j = ((l16 - s) & 15) / step;
      rank += (o > gs || (o == gs && j < own)) ? 1 : 0;
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
    clear = clear && last - next > 2.f * (2.f * err + 0x1p-23f * cmax);  // sums of two
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

  // keys: integers in the order of the values, the last kBits the expert
  constexpr int kBits = P == 4 ? 6 : (P == 8 ? 7 : (P == 16 ? 8 : 9));
  constexpr int kMask = (1 << kBits) - 1;
  constexpr int kNoKey = -0x7FFFFFFF - 1;
  int key[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int bits = __builtin_bit_cast(int, c[i]);
    const int ordered = bits ^ ((bits >> 31) & 0x7FFFFFFF);
    key[i] = c[i] > kNoneF ? (ordered & ~kMask) | (kMask - (e0 + i)) : kNoKey;
  }
  // the topk + 2 largest, candidate j in lane j of the row
  int mine = kNoKey;
  for (int j = 0; j < cfg.topk + 2; ++j) {
    int best = key[0];
#pragma unroll
    for (int i = 1; i < P; ++i) best = key[i] > best ? key[i] : best;
    best = row_max_i(best);
    mine = l16 == j ? best : mine;
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = key[i] == best ? kNoKey : key[i];
  }
  const bool found = mine != kNoKey;
  const int my_id = found ? kMask - (mine & kMask) : -1;
  const int cut = mine & ~kMask;
  const float my_c =
      found ? __builtin_bit_cast(float, cut ^ ((cut >> 31) & 0x7FFFFFFF)) : kNoneF;
  const float my_l = found ? __builtin_fminf(row[my_id], 3.402823466e38f) : 0.f;
  const float my_b = found && bias != nullptr ? bias[my_id] : 0.f;

  // the distance below which two values are near
  constexpr float kDrop = 1.f / static_cast<float>(1 << (23 - kBits));
  const float tol =
      bias != nullptr
          ? 2.f * err + kDrop * cmax
          : my_c * (kDrop + 0x1p-18f + 0x1p-21f * (cfg.sigmoid ? __builtin_fabsf(my_l) : m - my_l));
  const bool tiny = bias == nullptr && !(my_c > 0x1p-100f);
  const float next_c = dpp_f<0x101>(my_c);   // lane l + 1
  const float after_c = dpp_f<0x102>(my_c);  // lane l + 2
  // among the chosen and the first after them
  const bool near = found && l16 < cfg.topk && (tiny || !(my_c - next_c > tol));
  // the last chosen against the last candidate
  if (found && l16 == cfg.topk - 1 && after_c > kNoneF && (tiny || !(my_c - after_c > tol)))
    clear = false;

  // the candidates' scores in fp64
  const double dl = static_cast<double>(my_l);
  double p = 0.0;
  if (cfg.sigmoid) {
    if (found) p = 1.0 / (1.0 + exp(-dl));
  } else {
    if (found) p = exp(dl - static_cast<double>(m));
    if (!cfg.renormalize || bias != nullptr) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < P; ++i)
        sum += l[i] > kNoneF ? exp(static_cast<double>(l[i]) - static_cast<double>(m)) : 0.0;
      sum = row_sum_f64(sum);
      if (found) p /= sum;
    }
  }
  int slot = l16;
  if (__any(near)) {
    // ranks by the exact values, ties to the lower id
    const double d = found ? p + static_cast<double>(my_b) : kNone;
    slot = 0;
    auto count = [&](double od, int oid) __attribute__((always_inline)) {
      slot += (od > d || (od == d && oid < my_id)) ? 1 : 0;
    };
    count(dpp_d<0x121>(d), dpp_i<0x121>(my_id));
    count(dpp_d<0x122>(d), dpp_i<0x122>(my_id));
    count(dpp_d<0x123>(d), dpp_i<0x123>(my_id));
    count(dpp_d<0x124>(d), dpp_i<0x124>(my_id));
    count(dpp_d<0x125>(d), dpp_i<0x125>(my_id));
    count(dpp_d<0x126>(d), dpp_i<0x126>(my_id));
    count(dpp_d<0x127>(d), dpp_i<0x127>(my_id));
    count(dpp_d<0x128>(d), dpp_i<0x128>(my_id));
    count(dpp_d<0x129>(d), dpp_i<0x129>(my_id));
    count(dpp_d<0x12A>(d), dpp_i<0x12A>(my_id));
    count(dpp_d<0x12B>(d), dpp_i<0x12B>(my_id));
    count(dpp_d<0x12C>(d), dpp_i<0x12C>(my_id));
    count(dpp_d<0x12D>(d), dpp_i<0x12D>(my_id));
    count(dpp_d<0x12E>(d), dpp_i<0x12E>(my_id));
    count(dpp_d<0x12F>(d), dpp_i<0x12F>(my_id));
    if (!found) slot = l16;  // the lanes behind the candidates keep their places
  }
  const bool chosen = slot < cfg.topk;
  if (!found) p = 0.0;
  const double total = cfg.renormalize ? row_sum_f64(chosen ? p : 0.0) : 0.0;
  if (real && chosen) {
    ids[tok * cfg.topk + slot] = my_id;
    w[tok * cfg.topk + slot] = weight(found, p, total, cfg);
  }

  // unclear tokens again, one after another, by the whole wave
  uint64_t again = __ballot(real && !clear);
  while (again != 0) {
    const int first = __builtin_ctzll(again) & 48;
    again &= ~(0xFFFFull << first);
    const int64_t at = tok0 + first / 16;
    wave_lds_fence();
    route_token_f64<P / 4, 1>(logits + at * n, cfg, bias, reinterpret_cast<double *>(smem), lane,
                    ids + at * cfg.topk, w + at * cfg.topk);
  }
}

hipError_t launch_some(const float *logits, int64_t t, const RouterConfig &cfg, const float *bias,
                       int32_t *ids, float *w, hipStream_t s) {
  if (cfg.topk > kFastSlots || cfg.n_groups > kFastGroups) {
    hipLaunchKernelGGL(router_f64_kernel, dim3(static_cast<unsigned>((t + 3) / 4)), dim3(256), 0,
                       s, logits, t, cfg, bias, ids, w);
    return hipGetLastError();
  }
  constexpr int64_t kTokens = 4 * kFastWaves;
  const dim3 grid(static_cast<unsigned>((t + kTokens - 1) / kTokens));
  const dim3 block(64 * kFastWaves);
  if (cfg.n_experts <= 64)
    hipLaunchKernelGGL(router_fast_kernel<4>, grid, block, 0, s, logits, t, cfg, bias, ids, w);
  else if (cfg.n_experts <= 128)
    hipLaunchKernelGGL(router_fast_kernel<8>, grid, block, 0, s, logits, t, cfg, bias, ids, w);
  else if (cfg.n_experts <= 256)
    hipLaunchKernelGGL(router_fast_kernel<16>, grid, block, 0, s, logits, t, cfg, bias, ids,
                       w);
  else
    hipLaunchKernelGGL(router_fast_kernel<32>, grid, block, 0, s, logits, t, cfg, bias, ids,
                       w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_scored(const float *logits, int64_t t, const RouterConfig &config,
                                const float *bias, int32_t *ids, float *w, hipStream_t s) {
  RouterConfig cfg = config;
  const int32_t per = cfg.n_experts / cfg.n_groups;
  cfg.per_inv = static_cast<uint32_t>(((1 << 20) + per - 1) / per);
  for (int64_t at = 0; at < t; at += kRouterLaunchTokens) {
    const int64_t n = t - at < kRouterLaunchTokens ? t - at : kRouterLaunchTokens;
    const hipError_t e = launch_some(logits + at * cfg.n_experts, n, cfg, bias,
                                     ids + at * cfg.topk, w + at * cfg.topk, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tq4
