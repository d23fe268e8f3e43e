// What int8.hip (the int8 products) and router.hip (the scored router) share and
// their launchers, apart from tq4_internal.h: the committed traffic counters of the
// TQ4_1S kernels belong to that header's text, which these are no part of.
#pragma once

#include "tq4_internal.h"

namespace tq4 {

// A wave's LDS writes before its later reads, its own lanes' and the others'
// (nothing but the compiler could change their order).
__device__ inline void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// int8 products (codes [rows][int8_padded_k(k)] with zero codes behind k, one
// fp32 scale per row).
int64_t int8_padded_k(int64_t k);
hipError_t launch_act_int8(const uint16_t *x, int64_t m, int64_t k, int8_t *codes, float *scales,
                           hipStream_t s);
hipError_t launch_int8_cache(const uint8_t *packed, int64_t n, int64_t k, uint32_t sign_bits,
                             int8_t *codes, float *scales, hipStream_t s);
// y[m, n] = (sum of code products) * xs[m] * ws[n] + tail (fp32 or bf16).
hipError_t launch_linear_int8(const int8_t *xq, const float *xs, int64_t m, int64_t k,
                              const int8_t *wq, const float *ws, int64_t n, const Tail &tail,
                              void *y, hipStream_t s);
// The same from bf16 rows in one launch, for the few rows and the k that
// int8_direct_fits takes; bit-equal.
bool int8_direct_fits(int64_t m, int64_t k);
hipError_t launch_linear_int8_direct(const uint16_t *x, int64_t m, int64_t k, const int8_t *wq,
                                     const float *ws, int64_t n, const Tail &tail, void *y,
                                     hipStream_t s);
// The MoE layer of a few tokens in two launches, without bucketing (h: bf16
// [t * topk][n1], in pair order); bit-equal to the batched steps.
bool int8_moe_direct_fits(int64_t t, int32_t topk, int64_t n1, int64_t k);
hipError_t launch_moe_int8_direct(const uint16_t *x, int64_t t, int64_t k, const int32_t *ids,
                                  const float *gates, int32_t topk, int32_t n_experts,
                                  const int8_t *w1, const float *s1, int64_t n1, const int8_t *w2,
                                  const float *s2, uint16_t *h, float *out, hipStream_t s);
// The MoE layer's first step: launch_route's outputs for the pairs, and x's
// codes and scales.
hipError_t launch_moe_int8_prepare(const uint16_t *x, int64_t t, int64_t k, const int32_t *ids,
                                   int32_t topk, int32_t n_experts, int32_t *counts,
                                   int32_t *offsets, int32_t *perm, int32_t *inv, MoETile *tiles,
                                   int32_t *n_tiles, int32_t tile_rows, int8_t *xq, float *xs,
                                   hipStream_t s);
// Grouped products over stacked int8 experts (expert e's rows at e * n of the
// [E * n, k] cache).  mode 0 (up): rows gathered as perm[row] / topk; out is
// bf16 [pairs][n], relu(u)^2.  a_rows: rows of aq.  mode 1 (down): bucket rows; out is fp32
// [pairs][n].  tile_rows as int8_moe_tile_rows gives (and launch_route got).
int int8_moe_tile_rows(int64_t pairs, int32_t n_experts);
hipError_t launch_moe_int8(int mode, int tile_rows, const int8_t *aq, const float *as,
                           int64_t a_rows, int64_t k, const int32_t *perm, int32_t topk,
                           const int8_t *wq, const float *ws, int64_t n, const MoETile *tiles,
                           const int32_t *n_tiles, int64_t max_tiles, void *out, hipStream_t s);

// A launch counts its threads in 32 bits.  Up to 64 of them route a token, so
// the routers take more tokens than this in several launches.
constexpr int64_t kRouterLaunchTokens = int64_t{1} << 25;

// The scored router (router.hip).
struct RouterConfig {
  int32_t n_experts, topk;
  int32_t sigmoid;     // 0: softmax over the token's experts, 1: sigmoid
  int32_t n_groups, topk_groups;
  int32_t renormalize;
  float scale;
  uint32_t per_inv;    // set by the launcher: 2^20 / (experts per group), rounded up
};
hipError_t launch_router_scored(const float *logits, int64_t t, const RouterConfig &cfg,
                                const float *bias, int32_t *ids, float *w, hipStream_t s);

}  // namespace tq4
