// Launchers of the MXFP4 products (mxfp4.hip) and of the router's training step
// (balance.hip).
#pragma once

#include "int8_router.h"

namespace tq4 {

// MXFP4 rows: codes [rows][mxfp4_padded_k(k) / 2], two e2m1 codes a byte, and scale
// bytes [rows][mxfp4_padded_k(k) / 32]; zeros behind k.
int64_t mxfp4_padded_k(int64_t k);
hipError_t launch_act_mxfp4(const uint16_t *x, int64_t m, int64_t k, uint8_t *codes,
                            uint8_t *scales, hipStream_t s);
hipError_t launch_mxfp4_values(const uint8_t *codes, const uint8_t *scales, int64_t m, int64_t k,
                               uint16_t *out, hipStream_t s);
hipError_t launch_mxfp4_cache(const uint8_t *packed, int64_t n, int64_t k, uint32_t sign_bits,
                              uint8_t *codes, uint8_t *scales, hipStream_t s);
// y[m, n] = dq(xq, xs) . dq(wq, ws)^T + tail (fp32 or bf16).
hipError_t launch_linear_mxfp4(const uint8_t *xq, const uint8_t *xs, int64_t m, int64_t k,
                               const uint8_t *wq, const uint8_t *ws, int64_t n, const Tail &tail,
                               void *y, hipStream_t s);
// The same from bf16 rows in one launch, for the few rows that mxfp4_direct_fits
// takes; bit-equal where sums are exact (its waves split k).
bool mxfp4_direct_fits(int64_t m);
hipError_t launch_linear_mxfp4_direct(const uint16_t *x, int64_t m, int64_t k, const uint8_t *wq,
                                      const uint8_t *ws, int64_t n, const Tail &tail, void *y,
                                      hipStream_t s);
// The MoE layer's first step: launch_route's outputs for the pairs, and x's codes and
// scale bytes.
hipError_t launch_moe_mxfp4_prepare(const uint16_t *x, int64_t t, int64_t k, const int32_t *ids,
                                    int32_t topk, int32_t n_experts, int32_t *counts,
                                    int32_t *offsets, int32_t *perm, int32_t *inv, MoETile *tiles,
                                    int32_t *n_tiles, int32_t tile_rows, uint8_t *xq, uint8_t *xs,
                                    hipStream_t s);
// Grouped products over stacked MXFP4 experts (expert e's rows at e * n of the
// [E * n, k] cache).  mode 0 (up): rows gathered as perm[row] / topk; writes the codes
// and scale bytes of fp32(relu(u)^2) to hq and hs, in bucket order.  mode 1 (down):
// bucket rows; out is fp32 [pairs][n].  tile_rows as mxfp4_moe_tile_rows gives (and
// launch_route got).
int mxfp4_moe_tile_rows(int64_t pairs, int32_t n_experts, int64_t n1, int64_t k);
hipError_t launch_moe_mxfp4(int mode, int tile_rows, const uint8_t *aq, const uint8_t *as,
                            int64_t a_rows, int64_t k, const int32_t *perm, int32_t topk,
                            int32_t n_experts, const uint8_t *wq, const uint8_t *ws, int64_t n,
                            const MoETile *tiles, const int32_t *n_tiles, int64_t max_tiles,
                            float *out, uint8_t *hq, uint8_t *hs, hipStream_t s);
// The MoE layer of a few tokens in two launches, without bucketing (hq, hs: t * topk
// hidden rows, in pair order).
bool mxfp4_moe_direct_fits(int64_t t, int32_t topk);
hipError_t launch_moe_mxfp4_direct(const uint16_t *x, int64_t t, int64_t k, const int32_t *ids,
                                   const float *gates, int32_t topk, int32_t n_experts,
                                   const uint8_t *w1, const uint8_t *s1, int64_t n1,
                                   const uint8_t *w2, const uint8_t *s2, uint8_t *hq, uint8_t *hs,
                                   float *out, hipStream_t s);

// The router's training step.
struct BalanceArgs {
  const float *logits;  // [t][n_experts]
  const int32_t *ids;   // [t][topk]
  int64_t t;
  int32_t n_experts, topk;
  int32_t sigmoid;
};
// Bytes of scratch that launch_moe_balance needs (0: none), 8-byte aligned.
size_t balance_scratch(int64_t t, int32_t n_experts);
hipError_t launch_moe_balance(const BalanceArgs &a, float *loss, int32_t *counts, int32_t *tokens,
                              float *mean_p, void *scratch, hipStream_t s);
struct RouterGradArgs {
  BalanceArgs b;
  const float *dgates;    // [t][topk], or null
  int32_t renormalize;
  float scale;
  const int32_t *counts;  // [n_experts], tokens [1], dloss [1]: all or none
  const int32_t *tokens;
  const float *dloss;
  float *dlogits;         // [t][n_experts]
};
hipError_t launch_router_backward(const RouterGradArgs &a, hipStream_t s);

}  // namespace tq4
