// MXFP4 products: the linear layer and the MoE layer of the model
// (Nemotron-TheHobbit-30B-A3B model card, Running it and The model underneath; Help
// wanted: a resident copy that no forward decodes) on 4-bit floating-point operands.
//
// Rows.  32 consecutive values of a row share a scale 2^e, held as the byte e + 127;
// with a = max|v|, e is the smallest integer from -127 to 127 with a < 7 * 2^e (127 where there
// is none: byte 255 is no scale, and weights that packed rows decode to reach 2^132).  A value is
// held as the e2m1 code (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6) nearest to v / 2^e, ties to the even code; what lies between 6 and 7 becomes
// 6.  (Letting a up to 7 * 2^e in costs the largest values at most as much as
// rounding them among 4 and 6 does, and the others half a step less: the relative error of
// Gaussian rows is 0.112 with the limit at 7, 0.1155 at 6 and 0.115 at 8; of Student-t
// rows with 5 degrees of freedom 0.124, 0.133 and 0.126.)  A block with a NaN or
// an infinity has scale byte 255, the format's NaN, and zero codes.
//
// Layout.  Two codes a byte, the first in the low half; rows padded with zero codes and
// zero scale bytes to kp, k rounded up to a multiple of 128 (the k of one MFMA step).
//
// Products run on v_mfma_scale_f32_16x16x128_f8f6f4 and v_mfma_scale_f32_32x32x64_f8f6f4:
// lane i + 16 g (i + 32 g) holds the 32 values k = 32 g .. 32 g + 31 of row i of each operand as
// they lie in memory (16 bytes), and their scale byte.  In a pure loop on random codes they reach
// 4.3 to 4.7 and 5.7 to 6.0 PF.  A product of two codes is a multiple of 0.25 up to 36, so a
// block's sum is exact, and a row's is while 2^24 times the smallest unit 0.25 * 2^(e + f) it
// meets holds it; below that every split of k gives the same bits, past it sums round to
// fp32.  The weights are the first operand: a lane of the result holds outputs of one token, four
// consecutive columns at a time.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mxfp4.h"

namespace tq4 {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t ushortx2 __attribute__((ext_vector_type(2)));

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
#include "moe_route.h"

constexpr int kStep = 128;              // values of k in one product step
constexpr int kStepBytes = kStep / 2;   // of a row's codes

// ---------------------------------------------------------------------------
// Rows to codes

constexpr int kQThreads = 256;
constexpr uint32_t kNanScale = 255;

// The scale byte of a block from its largest magnitude's bits.  A quarter of an
// exponent's step carries magnitudes of 1.75 * 2^j and more into the next exponent, so
// 7 * 2^e = 1.75 * 2^(e + 2) is where e goes up.
__device__ inline uint32_t scale_of_bf16(uint32_t top) {
  const int b = static_cast<int>((top + 0x20u) >> 7) - 2;
  return top >= 0x7F80u ? kNanScale : static_cast<uint32_t>(b > 0 ? b : 0);
}
__device__ inline uint32_t scale_of_f32(uint32_t top) {
  const int b = static_cast<int>((top + 0x200000u) >> 23) - 2;
  return top >= 0x7F800000u ? kNanScale : static_cast<uint32_t>(b > 0 ? b : 0);
}

// The conversions divide by the scale operand's exponent (its byte 0 is 2^-127), round
// to nearest even and saturate at 6: the rule above.
__device__ inline float scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes of one 16-byte piece of a bf16 row.
__device__ inline uint32_t codes_of(uint4 d, uint32_t byte) {
  const float s = scale_operand(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, d.x), s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, d.y), s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, d.z), s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, d.w), s, 3);
  return byte == kNanScale ? 0u : r;
}

// The largest magnitude bits of a piece, the even and the odd values apart.
// Magnitude bits of bf16 order like the magnitudes, infinities and NaN last.
__device__ inline ushortx2 top_of(uint4 d) {
  auto mag = [](uint32_t w) { return __builtin_bit_cast(ushortx2, w & 0x7FFF7FFFu); };
  return __builtin_elementwise_max(__builtin_elementwise_max(mag(d.x), mag(d.y)),
                                   __builtin_elementwise_max(mag(d.z), mag(d.w)));
}
__device__ inline uint32_t top_of(ushortx2 t) { return t[0] > t[1] ? t[0] : t[1]; }

// The largest value over lanes l, l ^ 1, l ^ 2, l ^ 3.
__device__ inline uint32_t quad_max(uint32_t v) {
  uint32_t o = __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, false);
  v = o > v ? o : v;
  o = __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, false);
  return o > v ? o : v;
}

// V pieces of 8 values of a row per thread, `stride` pieces apart from at0; four lanes share
// a block (a row's pieces are a multiple of 16, so the lanes of a block stay together).
template <int V>
__device__ inline void act_pieces(const uint4 *xr, int64_t k, int64_t kp, int64_t at0, int stride,
                                  uint32_t *qr, uint8_t *sr) {
  const int64_t n_vec = k / 8, n_out = kp / 8;  // k is a multiple of 32
  uint4 d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t at = at0 + static_cast<int64_t>(stride) * i;
    d[i] = at < n_vec ? xr[at] : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t at = at0 + static_cast<int64_t>(stride) * i;
    const uint32_t byte = scale_of_bf16(quad_max(top_of(top_of(d[i]))));
    if (at >= n_out) continue;
    qr[at] = codes_of(d[i], byte);
    if (threadIdx.x % 4 == 0) sr[at / 4] = static_cast<uint8_t>(byte);
  }
}

// Grid: pieces of a row x rows.  Bound by memory, 2.53 bytes per value (4096 x 8192 15.4 us,
// 5.5 TB/s; what a copy reaches).  Two pieces per thread keep enough loads on their way.
template <int V>
__global__ __launch_bounds__(kQThreads) void act_mxfp4_kernel(const uint16_t *__restrict__ x,
                                                              int64_t rows, int64_t k, int64_t kp,
                                                              uint8_t *__restrict__ codes,
                                                              uint8_t *__restrict__ scales) {
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y)
    for (int64_t at0 = static_cast<int64_t>(blockIdx.x) * (kQThreads * V) + threadIdx.x;
         at0 < kp / 8; at0 += static_cast<int64_t>(gridDim.x) * (kQThreads * V))
      act_pieces<V>(reinterpret_cast<const uint4 *>(x + row * k), k, kp, at0, kQThreads,
                    reinterpret_cast<uint32_t *>(codes + row * (kp / 2)),
                    scales + row * (kp / 32));
}

// The MoE layer's first launch: workgroup 0 buckets the pairs, the waves of the others
// quantize the tokens, 128 pieces of a row each.  Neither needs the other's result, and
// the bucketing is one workgroup's chain of latencies in which the rest of the device is
// free (16 tokens 6.4 us, 1024 11.2: the bucketing's own time), and a launch costs the host
// 3.1 to 3.6 us.
__global__ __launch_bounds__(kRouteThreads) void fp4_route_act_kernel(
    const int32_t *ids, int64_t pairs, int32_t n_experts, int32_t *counts, int32_t *offsets,
    int32_t *perm, int32_t *inv, MoETile *tiles, int32_t *n_tiles, int32_t tile_rows,
    const uint16_t *__restrict__ x, int64_t t, int32_t k, int32_t kp, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales) {
  __shared__ int32_t hist[kRouteWaves][kMaxExperts];
  __shared__ int32_t base[kMaxExperts + 1];
  __shared__ int32_t tile_base[kMaxExperts + 1];
  if (blockIdx.x > 0) {
    const uint32_t chunks = (static_cast<uint32_t>(kp) / 8 + 127) / 128;
    const uint32_t at = (blockIdx.x - 1) * kRouteWaves + threadIdx.x / 64;
    const int64_t row = at / chunks;
    if (row >= t) return;
    act_pieces<2>(reinterpret_cast<const uint4 *>(x + row * k), k, kp,
                  128 * (at % chunks) + threadIdx.x % 64, 64,
                  reinterpret_cast<uint32_t *>(codes + row * (kp / 2)), scales + row * (kp / 32));
    return;
  }
  bucket_group<kRouteWaves>(hist, base, tile_base, ids, pairs, n_experts, counts, offsets, perm,
                            inv, tiles, n_tiles, tile_rows, nullptr);
}

// The values that codes stand for, as bf16 (exact: a code has one mantissa bit; what
// the largest scales put past bf16's range is infinite).  A thread takes 8.  Bound by
// memory (4096 x 8192 14.4 us, 5.9 TB/s).
__global__ __launch_bounds__(kQThreads) void mxfp4_values_kernel(
    const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows,
    int64_t k, int64_t kp, uint16_t *__restrict__ out) {
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y)
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; at < k / 8;
         at += static_cast<int64_t>(gridDim.x) * kQThreads) {
      const uint32_t c = reinterpret_cast<const uint32_t *>(codes + row * (kp / 2))[at];
      const uint32_t byte = scales[row * (kp / 32) + at / 4];
      const float s = scale_operand(byte);
      bf16x2 v[4];
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2);
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = byte == kNanScale ? 0x7FC07FC0u : __builtin_bit_cast(uint32_t, v[i]);
      reinterpret_cast<uint4 *>(out + row * k)[at] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Packed TQ4_1S rows: one thread per block, decoded (rotation undone) and encoded in
// fp64, so that the codes are those of the rule.  Offline: 237568 x 2688 (128 experts) 633 us,
// bound by the fp64 arithmetic (its 738 MB take 143 at the copy's rate; the bf16 form 275).
__device__ inline uint32_t e2m1_from_f64(double u) {
  const double a = __builtin_fabs(u);
  const uint32_t c = (a > 0.25) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
                     (a >= 3.5) + (a > 5.0);
  return c | (u < 0.0 ? 8u : 0u);
}

__global__ __launch_bounds__(kQThreads) void mxfp4_cache_kernel(
    const uint8_t *__restrict__ packed, int64_t n, int32_t kb, int32_t kpb, uint32_t sign_bits,
    Codebook cb, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; t < n * kpb;
       t += static_cast<int64_t>(gridDim.x) * kQThreads) {
    const int64_t row = t / kpb;
    const int32_t col = static_cast<int32_t>(t % kpb);
    uint32_t out[4] = {0, 0, 0, 0};
    uint32_t byte = 0;
    if (col < kb) {
      const uint32_t *p = reinterpret_cast<const uint32_t *>(packed + (row * kb + col) * 20);
      uint32_t wd[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) wd[i] = p[i];
      const float f0 = __uint_as_float((wd[4] & 0xFFFFu) << 16);
      const float f1 = __uint_as_float(wd[4] & 0xFFFF0000u);
      double v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint32_t q = (wd[i / 8] >> (4 * (i % 8))) & 15u;
        v[i] = static_cast<double>(i < 16 ? f0 : f1) * static_cast<double>(cb.c[q]);
      }
#pragma unroll
      for (int h = 1; h < 32; h <<= 1) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if ((i & h) == 0) {
            const double a = v[i], c = v[i + h];
            v[i] = a + c;
            v[i + h] = a - c;
          }
        }
      }
      const double rs32 = 0x1.6a09e667f3bcdp-3;  // 1/sqrt(32)
      double top = 0.0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        v[i] *= (sign_bits >> i) & 1u ? -rs32 : rs32;
        const double a = __builtin_fabs(v[i]);
        top = a > top ? a : top;
      }
      if (!__builtin_isfinite(f0) || !__builtin_isfinite(f1)) {
        byte = kNanScale;
      } else {
        // top = f * 2^p, f in [0.5, 1): 7 * 2^e = 0.875 * 2^(e + 3)
        int e = -127;
        if (top > 0.0) {
          int p2;
          const double f = __builtin_frexp(top, &p2);
          e = p2 - 3 + (f >= 0.875 ? 1 : 0);
          e = e < -127 ? -127 : (e > 127 ? 127 : e);  // (codes of 6 where it stops)
        }
        byte = static_cast<uint32_t>(e + 127);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          out[i / 8] |= e2m1_from_f64(__builtin_ldexp(v[i], -e)) << (4 * (i % 8));
      }
    }
    *reinterpret_cast<uint4 *>(codes + t * 16) = make_uint4(out[0], out[1], out[2], out[3]);
    scales[t] = static_cast<uint8_t>(byte);
  }
}

// ---------------------------------------------------------------------------
// Products

struct Fp4Args {
  const uint16_t *x;   // bf16 rows of k (quantized by the product's own waves), or
  const uint8_t *xq;   // codes [rows][kp / 2] and
  const uint8_t *xs;   // scale bytes [rows][kp / 32]
  const uint8_t *wq;   // weights (experts stacked)
  const uint8_t *ws;
  void *y;             // dense: [m][n] fp32 or bf16; down: fp32 [pairs][n]
  uint8_t *hq, *hs;    // up: hidden codes [pairs][n_store / 2], scale bytes
  Tail tail;           // dense only
  int64_t m, n;
  int32_t k, kp;
  int32_t n_store;     // up: n rounded up to a multiple of 128
  int32_t tiles_m, tiles_n;
  int32_t vec;         // n % 4 == 0 and y, residual aligned for 4 outputs
  const int32_t *perm; // MoE: bucket order (up gathers through it)
  const MoETile *tiles;
  const int32_t *n_tiles;
  int32_t tile_run;    // consecutive tiles that an XCD takes (tiles of more than 64 rows)
  int64_t a_rows;      // MoE: rows of xq
  int32_t topk;
  const int32_t *ids;  // MoE of few pairs: [t][topk], and
  const float *gates;
  int32_t n_experts;
};

enum { kDense = 0, kUp = 1, kDown = 2 };

// Two values rounded to bf16 (ties to even), a in the low half.
__device__ inline uint32_t bf16_pair(float a, float b) {
  typedef float pair __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((pair{a, b}), bf16x2));
}

// A wave's 16 x 16 block of a dense output: row lane % 16 of `rows` valid ones, columns n0 +
// 4 (lane / 16) .. + 3.
template <bool BF16, bool VEC>
__device__ inline void store_block(const Fp4Args &g, floatx4 acc, int rows, int64_t n0, int lane) {
#pragma clang fp contract(off)
  const int r = lane % 16;
  const int64_t n = n0 + 4 * (lane / 16);
  const int left = g.n - n < 4 ? static_cast<int>(g.n - n) : 4;
  if (r >= rows || left <= 0) return;
  const int64_t at = r * g.n + n;
  float *y = static_cast<float *>(g.y);
  if (g.tail.bias != nullptr) {
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] += v < left ? g.tail.bias[n + v] : 0.f;
  }
  if (g.tail.residual != nullptr) {
    if constexpr (VEC && BF16) {
      const uint2 d =
          *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(g.tail.residual) + at);
      acc[0] += __uint_as_float(d.x << 16);
      acc[1] += __uint_as_float(d.x & 0xFFFF0000u);
      acc[2] += __uint_as_float(d.y << 16);
      acc[3] += __uint_as_float(d.y & 0xFFFF0000u);
    } else if constexpr (VEC) {
      acc += *reinterpret_cast<const floatx4 *>(static_cast<const float *>(g.tail.residual) + at);
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (v < left) acc[v] += tail_residual_as<BF16>(g.tail.residual, at + v);
    }
  }
  if constexpr (VEC && BF16) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.y) + at) =
        make_uint2(bf16_pair(acc[0], acc[1]), bf16_pair(acc[2], acc[3]));
  } else if constexpr (VEC) {
    *reinterpret_cast<floatx4 *>(y + at) = acc;
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v < left) tail_store_as<BF16>(y, at + v, acc[v]);
  }
}

__device__ inline void store_any(const Fp4Args &g, floatx4 acc, int rows, int64_t n0, int lane) {
  if (g.vec) {
    if (g.tail.bf16)
      store_block<true, true>(g, acc, rows, n0, lane);
    else
      store_block<false, true>(g, acc, rows, n0, lane);
  } else {
    if (g.tail.bf16)
      store_block<true, false>(g, acc, rows, n0, lane);
    else
      store_block<false, false>(g, acc, rows, n0, lane);
  }
}

// The hidden value (a NaN stays one), and the codes of eight of them.
__device__ inline float hidden(float u) {
  const float p = u < 0.f ? 0.f : u;
  return p * p;
}
__device__ inline uint32_t codes_of_hidden(const float *h, uint32_t byte) {
  const float s = scale_operand(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[0], h[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[2], h[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[4], h[5], s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[6], h[7], s, 3);
  return byte == kNanScale ? 0u : r;
}

// The hidden block of a lane's row from two 16 x 16 products: columns 16 j + 4 g .. + 3 of
// sub-tiles j = 0 and 1 are 8 of its 32 values, the others are in lanes l ^ 16, l ^ 32, l
// ^ 48.  Sub-tile 0's codes in the low half.
__device__ inline uint32_t hidden_block(floatx4 a, floatx4 b, uint32_t &byte) {
  float h[8];
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    h[v] = hidden(v < 4 ? a[v % 4] : b[v % 4]);
    const uint32_t m = __float_as_uint(h[v]) & 0x7FFFFFFFu;
    top = m > top ? m : top;
  }
  uint32_t lo, hi;
  lane_pair16(top, lo, hi);
  top = lo > hi ? lo : hi;
  lane_pair32(top, lo, hi);
  byte = scale_of_f32(lo > hi ? lo : hi);
  return codes_of_hidden(h, byte);
}

// ---- few rows ---------------------------------------------------------------
// Up to 16 rows: the weights are read once, straight into registers.  A wave takes its steps
// in pairs: of the eight blocks of 256 k, lane i + 16 g takes 2 g and 2 g + 1, one
// for each of two products (both operands alike, so no sum changes).  Its 32 bytes and its
// row's other lanes' make whole cache lines, and one 16-bit load brings both scale bytes,
// which the products pick by the operand's byte select.  The last step of an odd number
// goes alone, block g to group g.

// The first byte of a lane's codes in pair p, and of its scales; `full`: two steps.
struct Pair {
  int p;
  bool full;
  __device__ int64_t codes(int grp) const {
    return static_cast<int64_t>(p) * (2 * kStepBytes) + (full ? 32 : 16) * grp;
  }
  __device__ int64_t scales(int grp) const {
    return static_cast<int64_t>(p) * 8 + (full ? 2 : 1) * grp;
  }
  __device__ int block(int grp) const { return 8 * p + (full ? 2 : 1) * grp; }
};

// One operand's 16 rows of a pair: codes and scale bytes.
struct Frag {
  intx4 c[2];
  int s;
  // row_codes, row_scales: the lane's row
  __device__ void load(const uint8_t *row_codes, const uint8_t *row_scales, Pair p, int grp) {
    const uint8_t *at = row_codes + p.codes(grp);
    c[0] = *reinterpret_cast<const intx4 *>(at);
    if (p.full) {
      c[1] = *reinterpret_cast<const intx4 *>(at + 16);
      s = *reinterpret_cast<const uint16_t *>(row_scales + p.scales(grp));
    } else {
      s = row_scales[p.scales(grp)];
    }
  }
};

// The same from a bf16 row of k values: a block's 32 are one lane's, so quantizing them
// takes no exchange between lanes.
struct RawFrag {
  uint4 d[2][4];
  __device__ void load(const uint16_t *row, int k, Pair p, int grp) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int blk = p.block(grp) + u;
      const bool in = 32 * blk < k && (u == 0 || p.full);  // whole blocks: k % 32 == 0
      const uint4 *at = reinterpret_cast<const uint4 *>(row) + 4 * static_cast<int64_t>(blk);
#pragma unroll
      for (int q = 0; q < 4; ++q) d[u][q] = in ? at[q] : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ Frag quantized() const {
    Frag f;
    f.s = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ushortx2 t = top_of(d[u][0]);
#pragma unroll
      for (int q = 1; q < 4; ++q) t = __builtin_elementwise_max(t, top_of(d[u][q]));
      const uint32_t byte = scale_of_bf16(top_of(t));
#pragma unroll
      for (int q = 0; q < 4; ++q) f.c[u][q] = static_cast<int>(codes_of(d[u][q], byte));
      f.s |= static_cast<int>(byte << (8 * u));
    }
    return f;
  }
};

template <int SEL>
__device__ inline floatx4 mfma_sel(intx4 a, intx4 b, floatx4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      intx8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, intx8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4,
      4, SEL, sa, SEL, sb);
}
__device__ inline floatx4 mfma_pair(const Frag &w, const Frag &x, floatx4 c, Pair p) {
  c = mfma_sel<0>(w.c[0], x.c[0], c, w.s, x.s);
  return p.full ? mfma_sel<1>(w.c[1], x.c[1], c, w.s, x.s) : c;
}

// The products of NT column sub-tiles over pairs [p0, p1), B pairs at a time, all loads of a
// batch issued before its first product.
template <bool QX, int NT, int B>
__device__ inline void stream(const uint8_t *const (&wq)[NT], const uint8_t *const (&ws)[NT],
                              const uint8_t *xq, const uint8_t *xs, const uint16_t *x, int k,
                              int steps, int p0, int p1, int grp, floatx4 (&acc)[NT]) {
  for (int p = p0; p < p1; p += B) {
    Frag w[B][NT], f[B];
    RawFrag raw[QX ? B : 1];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (p + u >= p1) break;
      const Pair at{p + u, 2 * (p + u) + 1 < steps};
      if constexpr (QX)
        raw[u].load(x, k, at, grp);
#pragma unroll
      for (int j = 0; j < NT; ++j) w[u][j].load(wq[j], ws[j], at, grp);
      if constexpr (!QX) f[u].load(xq, xs, at, grp);
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (p + u >= p1) break;
      const Pair at{p + u, 2 * (p + u) + 1 < steps};
      if constexpr (QX) f[u] = raw[u].quantized();
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = mfma_pair(w[u][j], f[u], acc[j], at);
    }
  }
}

// bf16 rows against 16 NT columns per workgroup of KW waves, which share k.  Their sums meet
// in LDS and are added in wave order.  Every workgroup quantizes the rows for itself: a
// launch of its own would cost the host more (one row of 2688 x 8192 5.4 us, 2.2 TB/s of
// weights: the ramp of a short stream; 16 rows 7.7, the row pieces 2.3 of them).  Dense: up to
// 16 rows.  Up: a workgroup row per pair, the expert from the ids, hidden rows in pair order.
template <int MODE, int NT, int KW, int B>
__global__ __launch_bounds__(64 * KW) void fp4_skinny_kernel(Fp4Args g) {
  static_assert(MODE == kDense || (MODE == kUp && NT == 2), "a hidden block is two sub-tiles");
  __shared__ floatx4 red[KW - 1][NT][64];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % 16;
  const int grp = lane / 16;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT);

  int64_t pair = 0, w0 = 0;
  int rows = static_cast<int>(g.m);
  if constexpr (MODE == kUp) {
    pair = blockIdx.y;
    rows = 1;
    const int e = g.ids[pair];
    if (e < 0 || e >= g.n_experts) return;
    w0 = static_cast<int64_t>(e) * g.n;
  }

  const int32_t row_bytes = g.kp / 2, row_scales = g.kp / 32;
  const uint8_t *wq[NT], *ws[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = n0 + 16 * j + r;
    const int64_t nr = w0 + (n < g.n ? n : g.n - 1);  // past n: read n - 1
    wq[j] = g.wq + nr * row_bytes;
    ws[j] = g.ws + nr * row_scales;
  }
  const int64_t src = MODE == kUp ? pair / g.topk : (r < rows ? r : 0);  // past the rows: the first
  floatx4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};

  const int steps = g.kp / kStep;
  const int pairs = (steps + 1) / 2;
  const int per = (pairs + KW - 1) / KW;
  const int p0 = wave * per;
  const int p1 = p0 + per < pairs ? p0 + per : pairs;
  stream<true, NT, B>(wq, ws, nullptr, nullptr, g.x + src * g.k, g.k, steps, p0, p1, grp, acc);
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < NT; ++j) red[wave - 1][j][lane] = acc[j];
  }
  __syncthreads();
  if (wave > 0) return;  // wave 0 adds the others' sums and stores
#pragma unroll
  for (int w = 0; w < KW - 1; ++w)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] += red[w][j][lane];
  if constexpr (MODE == kDense) {
#pragma unroll
    for (int j = 0; j < NT; ++j) store_any(g, acc[j], rows, n0 + 16 * j, lane);
  } else {
    uint32_t byte;
    if (n0 >= g.n) acc[0] = acc[1] = floatx4{0.f, 0.f, 0.f, 0.f};  // n % 32 == 0
    const uint32_t c = hidden_block(acc[0], acc[1], byte);
    if (r > 0) return;
    uint16_t *q = reinterpret_cast<uint16_t *>(g.hq + pair * (g.n_store / 2) + n0 / 2);
    q[grp] = static_cast<uint16_t>(c);
    q[4 + grp] = static_cast<uint16_t>(c >> 16);
    if (grp == 0) g.hs[pair * (g.n_store / 32) + n0 / 32] = static_cast<uint8_t>(byte);
  }
}

// The down product of few tokens with the weighted sum over their slots: grid (blocks of 16
// columns, tokens); waves KW j .. KW j + KW - 1 share the k of slot j.  Hidden rows are in pair
// order.  The sum runs in slot order with the combine kernel's fused multiply-adds.  One
// token of six slots, 1856 x 2688: 6.2 us (2.7 TB/s), the ramp of a 16 MB stream.
constexpr int kDirectSlots = 8;

template <int KW, int B>
__global__ __launch_bounds__(64 * KW * kDirectSlots) void fp4_direct_down_kernel(Fp4Args g) {
  __shared__ floatx4 sums[KW * kDirectSlots][4];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % 16;
  const int grp = lane / 16;
  const int64_t tok = blockIdx.y;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int32_t row_bytes = g.kp / 2, row_scales = g.kp / 32;
  const int64_t src = tok * g.topk + wave / KW;
  const int e = g.ids[src];
  if (e >= 0 && e < g.n_experts) {
    const int64_t nr = e * g.n + (n0 + r < g.n ? n0 + r : g.n - 1);
    const uint8_t *wq[1] = {g.wq + nr * row_bytes}, *ws[1] = {g.ws + nr * row_scales};
    floatx4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    const int steps = g.kp / kStep;
    const int pairs = (steps + 1) / 2;
    const int per = (pairs + KW - 1) / KW;
    const int p0 = wave % KW * per;
    const int p1 = p0 + per < pairs ? p0 + per : pairs;
    stream<false, 1, B>(wq, ws, g.xq + src * row_bytes, g.xs + src * row_scales, nullptr, g.k,
                        steps, p0, p1, grp, acc);
    if (r == 0) sums[wave][grp] = acc[0];
  }
  __syncthreads();
  const int64_t n = n0 + tid;
  if (tid >= 16 || n >= g.n) return;
  float out = 0.f;
  for (int j = 0; j < g.topk; ++j) {
    const int ej = g.ids[tok * g.topk + j];
    if (ej < 0 || ej >= g.n_experts) continue;
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) o += sums[KW * j + w][tid / 4][tid % 4];
    out = __builtin_fmaf(g.gates[tok * g.topk + j], o, out);
  }
  static_cast<float *>(g.y)[tok * g.n + n] = out;
}

// ---- many rows --------------------------------------------------------------

// The accumulator of a T x T product: lane i + T g holds columns 4 g .. 4 g + 3 (T =
// 16), or 8 q + 4 g .. + 3 for q = 0 .. 3 (T = 32), of token i.
template <int T>
using Acc = std::conditional_t<T == 16, floatx4, floatx16>;
template <int T>
constexpr int kQuads = T == 16 ? 1 : 4;

template <int T>
__device__ inline floatx4 quad_of(const Acc<T> &acc, int q) {
  if constexpr (T == 16)
    return acc;
  else
    return floatx4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
}

// A wave's MS x NS sub-tiles to memory through LDS.  Straight from the product's
// layout a store instruction would write rows of 64 bytes (32 for bf16), half a cache
// line each; instead T rows at a time go to a wave's own LDS buffer (rows 16 bytes
// longer than their data, so that neither the writes nor the reads share banks) and
// come back as whole row segments of T * NS outputs.  Stores are non-temporal: nothing
// reads the output before the operands that it would push out of the caches are
// needed.  Residual values are loaded several groups of T rows ahead of their use, as
// many as 40 registers hold, and before the stores of earlier rows, since a wait for a
// load is also one for every store before it.
template <int T, int NS>
constexpr int tile_store_bytes() {
  return T * (T * NS + 4) * 4;
}

typedef uint32_t uintx2 __attribute__((ext_vector_type(2)));

template <int MODE, int T, int MS, int NS, int WM, bool BF16, bool VEC>
__device__ inline void store_rows(const Fp4Args &g, const Acc<T> (&acc)[MS][NS], uint8_t *lds,
                                  int64_t m0, int rows, int64_t n0, int lane) {
#pragma clang fp contract(off)
  constexpr int kCols = T * NS;
  constexpr int kStride = kCols + 4;
  constexpr int E = VEC ? 4 : 1;             // outputs per lane and access
  constexpr int kGroups = 16 * kCols / (64 * E);
  constexpr int kUnits = MS * T / 16;        // of 16 rows
  const int r = lane % T;
  const int grp = lane / T;
  const bool has_bias = MODE == kDense && g.tail.bias != nullptr;
  const bool has_res = MODE == kDense && g.tail.residual != nullptr;
  using Raw = std::conditional_t<VEC, std::conditional_t<BF16, uintx2, floatx4>, float>;
  constexpr int kWords = kGroups * static_cast<int>(sizeof(Raw)) / 4;
  constexpr int kAhead = 40 / kWords < kUnits ? 40 / kWords : kUnits;
  static_assert(kAhead >= 1, "a group of rows fits");
  Raw res[MODE == kDense ? kAhead : 1][kGroups];
  // row of unit u's element f, in the wave's rows
  auto row_of = [&](int u, int f) __attribute__((always_inline)) {
    return T * WM * (u / (T / 16)) + 16 * (u % (T / 16)) + f / kCols;
  };
  auto load_res = [&](int u) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int f = 64 * E * q + E * lane;
      const int row = row_of(u, f);
      const int64_t n = n0 + f % kCols;
      Raw &d = res[u % kAhead][q];
      d = Raw{};
      if (row < rows && n < g.n) {
        const int64_t at = (m0 + row) * g.n + n;
        if constexpr (VEC && BF16)
          d = *reinterpret_cast<const Raw *>(static_cast<const uint16_t *>(g.tail.residual) + at);
        else if constexpr (VEC)
          d = *reinterpret_cast<const Raw *>(static_cast<const float *>(g.tail.residual) + at);
        else
          d = tail_residual_as<BF16>(g.tail.residual, at);
      }
    }
  };
  auto res_at = [&](int u, int q, int v) __attribute__((always_inline)) {
    const Raw &d = res[u % kAhead][q];
    if constexpr (VEC && BF16) {
      const uint32_t w = d[v / 2];
      return __uint_as_float(v % 2 == 0 ? w << 16 : w & 0xFFFF0000u);
    } else if constexpr (VEC) {
      return static_cast<float>(d[v]);
    } else {
      return d;
    }
  };
  float bias[kGroups][E];
  if constexpr (MODE == kDense) {
    if (has_res) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load_res(u);
    }
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int64_t n = n0 + (64 * E * q + E * lane) % kCols;
#pragma unroll
      for (int v = 0; v < E; ++v) bias[q][v] = has_bias && n < g.n ? g.tail.bias[n + v] : 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    constexpr int kParts = T / 16;
    const int i = u / kParts;
    if (MODE != kDense && row_of(u, 0) >= rows) break;
    float *buf = reinterpret_cast<float *>(lds);
    if (u % kParts == 0) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int q = 0; q < kQuads<T>; ++q)
          *reinterpret_cast<floatx4 *>(buf + r * kStride + T * j + 8 * q + 4 * grp) =
              quad_of<T>(acc[i][j], q);
      wave_lds_fence();
    }
    float val[kGroups][E];
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int f = 64 * E * q + E * lane;
      const float *src = buf + (16 * (u % kParts) + f / kCols) * kStride + f % kCols;
      if constexpr (VEC) {
        const floatx4 d = *reinterpret_cast<const floatx4 *>(src);
#pragma unroll
        for (int v = 0; v < 4; ++v) val[q][v] = d[v];
      } else {
        val[q][0] = *src;
      }
      if constexpr (MODE == kDense) {
#pragma unroll
        for (int v = 0; v < E; ++v) {
          if (has_bias) val[q][v] += bias[q][v];
          if (has_res) val[q][v] += res_at(u, q, v);
        }
      }
    }
    wave_lds_fence();  // these reads before the next rows' writes
    if constexpr (MODE == kDense) {
      if (has_res && u + kAhead < kUnits) load_res(u + kAhead);
    }
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int f = 64 * E * q + E * lane;
      const int row = row_of(u, f);
      const int64_t n = n0 + f % kCols;
      if (row >= rows || n >= g.n) continue;
      const int64_t at = (m0 + row) * g.n + n;
      if constexpr (VEC && BF16) {
        const uintx2 d = {bf16_pair(val[q][0], val[q][1]), bf16_pair(val[q][2], val[q][3])};
        uintx2 *dst = reinterpret_cast<uintx2 *>(static_cast<uint16_t *>(g.y) + at);
        __builtin_nontemporal_store(d, dst);
      } else if constexpr (VEC) {
        const floatx4 d = {val[q][0], val[q][1], val[q][2], val[q][3]};
        floatx4 *dst = reinterpret_cast<floatx4 *>(static_cast<float *>(g.y) + at);
        __builtin_nontemporal_store(d, dst);
      } else {
        tail_store_as<BF16>(static_cast<float *>(g.y), at, val[q][0]);
      }
    }
  }
}

// Hidden codes and scales of a wave's 32 x 32 sub-tiles, each a block of every row: lanes
// i and i + 32 hold half of row i's block each.  Their codes are 16-bit words in turn
// (columns 8 q + 4 g); one exchange leaves lane i + 32 g with bytes 8 g .. 8 g + 7.
template <int MS, int NS, int WM>
__device__ inline void store_hidden(const Fp4Args &g, const floatx16 (&acc)[MS][NS], int64_t m0,
                                    int rows, int64_t n0, int lane) {
  const int grp = lane / 32;
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    if (32 * WM * i >= rows) break;
    const int row = 32 * WM * i + lane % 32;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      float h[16];
      uint32_t top = 0;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        h[v] = hidden(acc[i][j][v]);
        const uint32_t m = __float_as_uint(h[v]) & 0x7FFFFFFFu;
        top = m > top ? m : top;
      }
      uint32_t lo, hi;
      lane_pair32(top, lo, hi);
      const uint32_t byte = scale_of_f32(lo > hi ? lo : hi);
      const auto c = __builtin_amdgcn_permlane32_swap(
          codes_of_hidden(h, byte), codes_of_hidden(h + 8, byte), false, false);
      const int64_t n = n0 + 32 * j;
      if (row >= rows || n >= g.n_store) continue;
      *reinterpret_cast<uint2 *>(g.hq + (m0 + row) * (g.n_store / 2) + n / 2 + 8 * grp) =
          make_uint2(__builtin_amdgcn_perm(c[1], c[0], 0x05040100u),
                     __builtin_amdgcn_perm(c[1], c[0], 0x07060302u));
      if (grp == 0) g.hs[(m0 + row) * (g.n_store / 32) + n / 32] = static_cast<uint8_t>(byte);
    }
  }
}

typedef __attribute__((address_space(3))) void lds_void;
constexpr int kBufferFlags = 0x00020000;

// TM x TN output tile per workgroup of WM x WN waves, each wave MS x NS
// T x T products.  KB bytes (64 or 128, one or two steps) of codes of the tile's TM
// activation rows and TN weight rows, and their scale bytes, go to LDS by LDS-direct
// buffer loads into S stages, S - 1 ahead, with exact load-count waits and one barrier
// per stage.
//
// Loads issue between the products (SPREAD, and always with PP): eight waves that first put a
// stage's 60 loads into the memory pipe stand in front of it instead (4096 x 8192 x 2688:
// 192 x 256 tiles 54.4 -> 51.7 us, 256 x 256 56.6 -> 52.0).  Only the MoE's 256-row tiles where
// every expert's weights are read once, with one stage on its way, want it as early as can
// be.  PP: two waves per SIMD half a step apart, one reading while the other multiplies.
//
// Scale bytes are fetched CH steps at a time, 16 bytes a lane: 4 bytes of every row for
// every step are as many cache lines to look up as the codes themselves (1024 tokens of
// 128 experts: 245 us with them, 211 without any).
//
// 4096 x 8192 x 2688 in 192 x 256 tiles: 54 us a call on quantized rows, calls one after
// another, 3.3 PF (58 of the layer's 74 with bf16 residual and output); matrix units busy in
// 48 % of the cycles, the rest loads into LDS; weights straight to registers took 79 to 101.  MoE
// layer of 128 experts of 1856 x 2688: 16 tokens 46 us up and 39 down (4.4 and 5.3 TB/s of
// weights), 1024 tokens 96 and 101 (4.8 and 5.2 TB/s with rows that two XCDs read), 4096 tokens
// 118 and 146 (3.8 and 4.7 TB/s with what they write): bound by memory, the up product of 4096
// tokens by the one stage on its way, and deeper forms of fewer columns read more and took
// longer.
//
// LDS image of a stage: 1 KB pieces of 1024 / KB rows; a row's 16-byte slots
// are stored at slot ^ key(row).  A 16-byte read takes the wave in phases of 16
// lanes, which are not consecutive (0-3, 12-15, 20-23, 24-27 make the first):
// of lane r + 16 g reading row r, a phase holds rows 0-3 and 12-15 at one slot
// and 4-11 at another.  key = (row / 2) % 8 for 128-byte rows and 0, 2, 3, 1 for
// row / 4 = 0 .. 3 of 64-byte rows put the 16 lanes of every phase on all 64
// banks (T = 32: (row / 2) % 8 and (row / 4) % 4).  Rows past the tile's end read zeros
// (dense; the buffer range ends there) or the tile's first row (MoE) and are not stored.
template <int MODE, int T, int WM, int WN, int MS, int NS, int KB, int S, int CH, bool PP,
          bool SPREAD>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp4_tile_kernel(Fp4Args g) {
  constexpr int W = WM * WN;
  constexpr int TM = T * MS * WM;
  constexpr int TN = T * NS * WN;
  constexpr int kPieceRows = 1024 / KB;
  constexpr int kSlots = KB / 16;
  constexpr int kAPieces = TM / kPieceRows;
  constexpr int kWPieces = TN / kPieceRows;
  static_assert(TM % kPieceRows == 0 && TN % kPieceRows == 0, "whole pieces");
  // every wave loads the same number of pieces; where that is more than there are, the last
  // one again (the same bytes to the same place)
  constexpr int kALoads = (kAPieces + W - 1) / W;
  constexpr int kWLoads = (kWPieces + W - 1) / W;
  constexpr int kLoads = kALoads + kWLoads;
  constexpr int kWBase = TM * KB;
  constexpr int kStage = (TM + TN) * KB;
  // scales: chunks of CH steps, two in turn
  constexpr int kRowScales = 4 * CH;                // scale bytes of a row and chunk
  constexpr int kSSlots = kRowScales / 16;
  constexpr int kSRows = 1024 / kRowScales;         // rows of a piece of scales
  static_assert(TM % kSRows == 0 && TN % kSRows == 0, "whole pieces of scales");
  constexpr int kSPieces = (TM + TN) / kSRows;
  constexpr int kSLoads = (kSPieces + W - 1) / W;
  constexpr int kChunk = (TM + TN) * kRowScales;
  constexpr int kStageSteps = KB / kStepBytes;
  constexpr int kChunkStages = CH / kStageSteps;
  static_assert(kChunkStages >= S - 1, "a chunk is older than the loads that may be in flight");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * kStage + 2 * kChunk];
  uint8_t *const chunks = smem + S * kStage;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % T;
  const int grp = lane / T;
  const int wm = wave / WN;
  const int wn = wave % WN;
  const int row_bytes = g.kp / 2, row_scales = g.kp / 32;

  int64_t m_base, n_base, w0 = 0;
  int rows;  // valid rows of the tile
  if constexpr (MODE == kDense) {
    // Workgroup ids go round robin over the 8 XCDs.  Each XCD takes one
    // contiguous run of an order that walks blocks of 8 tile columns down
    // all tile rows, so the tiles it holds at a time share their operands in
    // its L2.
    const int total = g.tiles_m * g.tiles_n;
    const int id = static_cast<int>(blockIdx.x);
    const int x = id % 8;
    const int q = total / 8, rem = total % 8;
    const int at = x * q + (x < rem ? x : rem) + id / 8;
    const int blk = at / (8 * g.tiles_m);
    const int in = at % (8 * g.tiles_m);
    const int width = g.tiles_n - 8 * blk < 8 ? g.tiles_n - 8 * blk : 8;
    m_base = static_cast<int64_t>(in / width) * TM;
    n_base = static_cast<int64_t>(8 * blk + in % width) * TN;
    rows = g.m - m_base < TM ? static_cast<int>(g.m - m_base) : TM;
  } else {
    int i, j;
    if constexpr (TM <= 64) {
      // Tiles of few rows: their column blocks in a row, over all XCDs.  The rows that every XCD
      // then reads are small beside the weights, and no XCD gets a tile more than another (16
      // tokens 97 us with whole tiles to an XCD, 87 so, on other boxes 86 to 96; 128-row tiles
      // 201 and 202, 256-row 339 and 347).
      i = static_cast<int>(blockIdx.x) / g.tiles_n;
      j = static_cast<int>(blockIdx.x) % g.tiles_n;
    } else {
      // XCD x (workgroup id % 8) takes runs of g.tile_run tiles, x, x + 8, ..., a tile's
      // column blocks in a row: the tile's rows then stay in one L2
      const int q = static_cast<int>(blockIdx.x) / 8;
      const int s = q / g.tiles_n;
      i = (s / g.tile_run * 8 + static_cast<int>(blockIdx.x) % 8) * g.tile_run + s % g.tile_run;
      j = q % g.tiles_n;
    }
    if (i >= *g.n_tiles) return;
    const MoETile t = g.tiles[i];
    m_base = t.row0;
    rows = t.rows;
    n_base = static_cast<int64_t>(j) * TN;
    w0 = static_cast<int64_t>(t.expert) * g.n;
  }
  // up: the columns of the padding read no weights (zeros)
  const int64_t left = g.n - n_base;
  const int cols = left < TN ? (left > 0 ? static_cast<int>(left) : 0) : TN;

  // A piece's lane l fills row l / kSlots at stored slot l % kSlots; the key of
  // a row depends on row % 16, so the pieces of 8 rows alternate between two.
  const int prow = lane / kSlots;
  auto key_of = [](int row) __attribute__((always_inline)) {
    if constexpr (KB == 64 && T == 16) return ((row >> 1) & 2) ^ ((row >> 3) & 1) * 3;
    if constexpr (KB == 64) return (row >> 2) & 3;
    return (row >> 1) & 7;
  };
  auto slot_of = [&](int row)
      __attribute__((always_inline)) { return (lane % kSlots) ^ key_of(row); };
  // the row of the activation arrays that tile row `row` is
  auto a_row = [&](int row) __attribute__((always_inline)) {
    if constexpr (MODE == kDense) return static_cast<int64_t>(row);
    const int64_t b = m_base + (row < rows ? row : 0);
    return MODE == kUp ? static_cast<int64_t>(g.perm[b] / g.topk) : b;
  };
  const int64_t a_base = MODE == kDense ? m_base : 0;
  const int64_t a_rows = MODE == kDense ? rows : g.a_rows;
  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(g.xq + a_base * row_bytes), static_cast<short>(0),
      static_cast<int>(a_rows * row_bytes), kBufferFlags);
  const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(g.wq + (w0 + n_base) * row_bytes), static_cast<short>(0),
      cols * row_bytes, kBufferFlags);
  static_assert(kALoads <= 8 && kWLoads <= 8 && kSLoads <= 4, "offsets held per load");
  auto a_piece = [&](int i) __attribute__((always_inline)) {
    const int p = kALoads * wave + i;
    return p < kAPieces ? p : kAPieces - 1;
  };
  auto w_piece = [&](int i) __attribute__((always_inline)) {
    const int p = kWLoads * wave + i;
    return p < kWPieces ? p : kWPieces - 1;
  };
  // (a bound that depends on the template made the host pass drop launch stubs)
  uint32_t a_voff[8];
#pragma unroll
  for (int i = 0; i < kALoads; ++i) {
    const int row = kPieceRows * a_piece(i) + prow;
    a_voff[i] = static_cast<uint32_t>(a_row(row) * row_bytes + 16 * slot_of(row));
  }
  uint32_t w_voff[8];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) {
    const int row = kPieceRows * w_piece(i) + prow;
    w_voff[i] = static_cast<uint32_t>(row * row_bytes + 16 * slot_of(row));
  }
  // Rows r and r + 8 hold their two 16-byte slots in opposite order, so that 32 rows read
  // at one step meet two at a bank.
  auto scale_key = [](int row) __attribute__((always_inline)) {
    return kSSlots == 2 ? (row >> 3) & 1 : 0;
  };
  __amdgpu_buffer_rsrc_t s_rsrc[4];
  uint32_t s_voff[4];
  int s_piece[4];
#pragma unroll
  for (int i = 0; i < kSLoads; ++i) {
    const int p = wave + W * i < kSPieces ? wave + W * i : kSPieces - 1;
    const int row = kSRows * p + lane / kSSlots;
    const bool act = kSRows * p < TM;
    s_piece[i] = p;
    s_rsrc[i] = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(act ? g.xs + a_base * row_scales
                                  : g.ws + (w0 + n_base) * row_scales),
        static_cast<short>(0),
        act ? static_cast<int>(a_rows * row_scales) : cols * row_scales, kBufferFlags);
    s_voff[i] = static_cast<uint32_t>((act ? a_row(row) : row - TM) * row_scales +
                                      16 * ((lane % kSSlots) ^ scale_key(row)));
  }

  // with 128-byte rows the second half of a last odd step is read (the next row's start,
  // or zeros) but not multiplied
  const int halves = g.kp / kStep;
  const int steps = KB == 64 ? halves : (halves + 1) / 2;
  // load i of a stage
  auto issue_one = [&](int c, uint8_t *st, int i) __attribute__((always_inline)) {
    const int k0 = (c < steps ? c : steps - 1) * KB;  // padding steps reload the last one
    if (i < kALoads)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rsrc, (lds_void *)(st + a_piece(i) * 1024), 16,
                                               a_voff[i], k0, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          w_rsrc, (lds_void *)(st + kWBase + w_piece(i - kALoads) * 1024), 16,
          w_voff[i - kALoads], k0, 0, 0);
  };
  auto issue = [&](int c, uint8_t *st) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) issue_one(c, st, i);
  };
  auto issue_chunk = [&](int q) __attribute__((always_inline)) {
    if (q * CH >= halves) return;
    uint8_t *to = chunks + (q % 2) * kChunk;
#pragma unroll
    for (int i = 0; i < kSLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s_rsrc[i], (lds_void *)(to + s_piece[i] * 1024), 16,
                                               s_voff[i], q * kRowScales, 0, 0);
  };

  const int64_t m0 = m_base + T * wm;
  const int64_t n0 = n_base + wn * (T * NS);
  Acc<T> acc[MS][NS] = {};

  // fragment addresses: row T * x + r, whose key depends on r alone
  const int key = key_of(r);
  const int a_frag = (T * wm + r) * KB;
  const int w_frag = kWBase + (wn * (T * NS) + r) * KB;
  const int a_scale = (T * wm + r) * kRowScales;
  const int w_scale = (TM + wn * (T * NS) + r) * kRowScales;
  const int s_key = 16 * scale_key(r);
  // A wave's sub-tile i holds rows T (WM i + wm) ..., so that the rows of a
  // part-filled tile are spread over the waves; sub-tiles past the rows are skipped.
  const int live = MODE == kDense ? MS : (rows - T * wm + T * WM - 1) / (T * WM);
  // Lane i + T g of product p of a step (one of 128 k, T = 16; two of 64, T = 32) reads
  // slot kParts p + g and scale byte kParts p + g.
  constexpr int kProducts = T / 16, kParts = 64 / T;
  // a row's four scale bytes of a step, moved so that byte kParts p is product p's
  auto scale_at = [&](int base, int step) __attribute__((always_inline)) {
    const uint8_t *at = chunks + (step / CH % 2) * kChunk + base + ((4 * (step % CH)) ^ s_key);
    return static_cast<int>(*reinterpret_cast<const uint32_t *>(at) >> (8 * grp));
  };
  auto slot_at = [&](int h, int p) __attribute__((always_inline)) {
    return 16 * ((4 * h + kParts * p + grp) ^ key);
  };
  auto product = [&](intx4 w, intx4 a, Acc<T> c, int ws, int as, int p)
      __attribute__((always_inline)) {
    const intx8 w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    const intx8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
    if constexpr (T == 16)
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, a8, c, 4, 4, 0, ws, 0, as);
    else
      return p == 0
                 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, a8, c, 4, 4, 0, ws, 0, as)
                 : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, a8, c, 4, 4, 2, ws, 2, as);
  };
  // the products of step h of a stage; `between` after every row sub-tile
  auto half = [&](const uint8_t *st, int h, int step, auto between)
      __attribute__((always_inline)) {
    intx4 wf[NS][kProducts];
    int ws[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
#pragma unroll
      for (int p = 0; p < kProducts; ++p)
        wf[j][p] = *reinterpret_cast<const intx4 *>(st + w_frag + T * j * KB + slot_at(h, p));
      ws[j] = scale_at(w_scale + T * j * kRowScales, step);
    }
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      if (MODE == kDense || i < live) {
        const int as = scale_at(a_scale + T * WM * i * kRowScales, step);
#pragma unroll
        for (int p = 0; p < kProducts; ++p) {
          const intx4 af =
              *reinterpret_cast<const intx4 *>(st + a_frag + T * WM * i * KB + slot_at(h, p));
#pragma unroll
          for (int j = 0; j < NS; ++j) acc[i][j] = product(wf[j][p], af, acc[i][j], ws[j], as, p);
        }
      }
      between(i);
    }
  };

  constexpr int kAhead = (S - 2) * kLoads;
  constexpr int kWait = 0x0F70 | (kAhead & 15) | ((kAhead >> 4) << 14);
  static_assert(kAhead < 64, "the wait counts up to 63 loads");
  issue_chunk(0);
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(s, smem + s * kStage);
  if constexpr (PP) {
    static_assert(W == 8 && KB == 64, "two waves per SIMD, one product step per stage");
    const bool late = wave >= 4;
    intx4 wf[NS][kProducts], af[MS][kProducts];
    int ws[NS], as[MS];
    auto phase_end = [&]() __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    // in a step's read phase the loads of S - 2 steps behind it have been issued, and those of
    // the next one have to be through
    constexpr int kAheadPP = (S - 3) * kLoads;
    constexpr int kWaitPP = 0x0F70 | (kAheadPP & 15) | ((kAheadPP >> 4) << 14);
    static_assert(S >= 3, "a step is in flight behind the next one");
    __builtin_amdgcn_s_waitcnt(kWait);  // step 0
    phase_end();
    if (late) phase_end();
    for (int c = 0; c < steps; c += S) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (c + s < steps) {
          const uint8_t *st = smem + s * kStage;
#pragma unroll
          for (int j = 0; j < NS; ++j) {
#pragma unroll
            for (int p = 0; p < kProducts; ++p)
              wf[j][p] =
                  *reinterpret_cast<const intx4 *>(st + w_frag + T * j * KB + slot_at(0, p));
            ws[j] = scale_at(w_scale + T * j * kRowScales, c + s);
          }
#pragma unroll
          for (int i = 0; i < MS; ++i) {
#pragma unroll
            for (int p = 0; p < kProducts; ++p)
              af[i][p] =
                  *reinterpret_cast<const intx4 *>(st + a_frag + T * WM * i * KB + slot_at(0, p));
            as[i] = scale_at(a_scale + T * WM * i * kRowScales, c + s);
          }
          __builtin_amdgcn_s_waitcnt(kWaitPP);  // step c + s + 1
          __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
          phase_end();
          // the stage read in the phase before last is refilled, a load at a time between the
          // products
          if ((c + s) % kChunkStages == 0) issue_chunk((c + s) / kChunkStages + 1);
#pragma unroll
          for (int i = 0; i < MS; ++i) {
            if (MODE == kDense || i < live) {
#pragma unroll
              for (int p = 0; p < kProducts; ++p)
#pragma unroll
                for (int j = 0; j < NS; ++j)
                  acc[i][j] = product(wf[j][p], af[i][p], acc[i][j], ws[j], as[i], p);
            }
#pragma unroll
            for (int l = i * kLoads / MS; l < (i + 1) * kLoads / MS; ++l)
              issue_one(c + s + S - 1, smem + ((s + S - 1) % S) * kStage, l);
            __builtin_amdgcn_sched_barrier(0);
          }
          phase_end();
        }
      }
    }
    if (!late) phase_end();
  } else {
    for (int c = 0; c < steps; c += S) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        // step c + s has landed when only the S - 2 steps after it are in
        // flight; behind the barrier it has for every wave, and every wave has
        // read step c + s - 1, whose stage is then refilled
        __builtin_amdgcn_s_waitcnt(kWait);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        if (c + s >= steps) break;
        if ((c + s) % kChunkStages == 0) issue_chunk((c + s) / kChunkStages + 1);
        uint8_t *to = smem + ((s + S - 1) % S) * kStage;
        if constexpr (SPREAD) {
          auto between = [&](int i) __attribute__((always_inline)) {
#pragma unroll
            for (int l = i * kLoads / MS; l < (i + 1) * kLoads / MS; ++l)
              issue_one(c + s + S - 1, to, l);
            if (MS > 1) __builtin_amdgcn_sched_barrier(0);
          };
          half(smem + s * kStage, 0, kStageSteps * (c + s), between);
        } else {
          issue(c + s + S - 1, to);
          half(smem + s * kStage, 0, kStageSteps * (c + s), [](int) {});
        }
        if (KB == 128 && 2 * (c + s) + 1 < halves)
          half(smem + s * kStage, 1, kStageSteps * (c + s) + 1, [](int) {});
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // the padding steps' loads
  __builtin_amdgcn_s_waitcnt(0xC07F);  // the last reads of the stages
  rows -= T * wm;
  if constexpr (MODE == kUp) {
    store_hidden<MS, NS, WM>(g, acc, m0, rows, n0, lane);
    return;
  }
  static_assert(W * tile_store_bytes<T, NS>() <= S * kStage + 2 * kChunk,
                "the stages hold the store buffers");
  __syncthreads();  // for every wave: the stages become store buffers
  uint8_t *lds = smem + wave * tile_store_bytes<T, NS>();
  if constexpr (MODE == kDown) {
    store_rows<MODE, T, MS, NS, WM, false, true>(g, acc, lds, m0, rows, n0, lane);
  } else if (g.vec) {
    if (g.tail.bf16)
      store_rows<MODE, T, MS, NS, WM, true, true>(g, acc, lds, m0, rows, n0, lane);
    else
      store_rows<MODE, T, MS, NS, WM, false, true>(g, acc, lds, m0, rows, n0, lane);
  } else {
    if (g.tail.bf16)
      store_rows<MODE, T, MS, NS, WM, true, false>(g, acc, lds, m0, rows, n0, lane);
    else
      store_rows<MODE, T, MS, NS, WM, false, false>(g, acc, lds, m0, rows, n0, lane);
  }
}

template <int MODE, int T, int WM, int WN, int MS, int NS, int KB, int S, int CH = 8,
          bool PP = false, bool SPREAD = true>
hipError_t launch_tile(Fp4Args g, int64_t max_tiles, hipStream_t s) {
  constexpr int TM = T * MS * WM, TN = T * NS * WN;
  const int64_t n = MODE == kUp ? g.n_store : g.n;
  g.tiles_n = static_cast<int32_t>((n + TN - 1) / TN);
  int64_t grid;
  if (MODE == kDense) {
    g.tiles_m = static_cast<int32_t>((g.m + TM - 1) / TM);
    grid = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  } else {
    const int64_t round = 8 * g.tile_run;
    grid = (max_tiles + round - 1) / round * round * g.tiles_n;
  }
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((fp4_tile_kernel<MODE, T, WM, WN, MS, NS, KB, S, CH, PP, SPREAD>),
                     dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), 0, s, g);
  return hipGetLastError();
}

// The dense tile: the one with the least time, from the number of tiles and what each
// kernel was measured to need (us): `alone` a step of 128 k with one workgroup on a compute
// unit, `each` what every one adds where there are several, `slots` how many fit, `end`
// a tile's start and stores; 256 compute units.  Fitted to sweeps of 11 shapes, m = 64 .. 4096 at
// (k, n) = (2688, 8192), (8192, 2688) and (1856, 2688), together with 2.5 us of a launch that are
// left out here, the same for all.  With them the model is off by 3 to 5 % rms for the tiles up to
// 128 x 128 and by 13 and 18 % for the largest two, whose times it gives up to 27 % too low.  The
// tile that it gives was the fastest, or as fast, at all 11; other (k, n) were not swept.
// (Times of the neighbours: 333 x 1856 x 2688 in 32 x 64
// tiles 6.8 us, 64 x 64 6.1, 64 x 128 8.8; 512 x 2688 x 8192 in 64 x 64 16.9, 128 x 128 13.2,
// 192 x 256 18.6; 4096 x 2688 x 8192 in 128 x 128 70.4, 192 x 256 67.3, 256 x 256 63.6;
// 4096 x 8192 x 2688 61.9, 51.7, 52.7.)
int pick_tile(int64_t m, int64_t k, int64_t n) {
  struct Cost {
    int tm, tn, slots;
    double alone, each, end;
  };
  static constexpr Cost kCosts[] = {
      {32, 32, 3, 0.109, 0.0475, 0.56},  {32, 64, 3, 0.106, 0.0724, 0.98},
      {64, 64, 3, 0.144, 0.0995, 1.35},  {64, 128, 2, 0.269, 0.148, 2.22},
      {128, 128, 2, 0.295, 0.252, 3.00}, {192, 256, 1, 0.484, 0.484, 8.04},
      {256, 256, 1, 0.481, 0.481, 11.7},
  };
  const double steps = static_cast<double>(mxfp4_padded_k(k) / kStep);
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < static_cast<int>(sizeof(kCosts) / sizeof(kCosts[0])); ++i) {
    const Cost &c = kCosts[i];
    const int64_t tiles = ((m + c.tm - 1) / c.tm) * ((n + c.tn - 1) / c.tn);
    const int64_t per_cu = (tiles + 255) / 256;
    auto step = [&](int64_t w) {
      const double t = c.each * static_cast<double>(w);
      return w == 0 ? 0.0 : (t > c.alone ? t : c.alone);
    };
    const double cost =
        steps * (static_cast<double>(per_cu / c.slots) * step(c.slots) + step(per_cu % c.slots)) +
        static_cast<double>(per_cu) * c.end;
    if (i == 0 || cost < least) {
      best = i;
      least = cost;
    }
  }
  return best;
}

Fp4Args dense_args(int64_t m, int64_t k, const uint8_t *wq, const uint8_t *ws, int64_t n,
                   const Tail &tail, void *y) {
  Fp4Args g{};
  g.wq = wq;
  g.ws = ws;
  g.y = y;
  g.tail = tail;
  g.m = m;
  g.n = n;
  g.k = static_cast<int32_t>(k);
  g.kp = static_cast<int32_t>(mxfp4_padded_k(k));
  const size_t quad = tail.bf16 ? 8 : 16;
  g.vec = n % 4 == 0 && reinterpret_cast<uintptr_t>(y) % quad == 0 &&
          reinterpret_cast<uintptr_t>(tail.residual) % quad == 0;
  return g;
}

}  // namespace

int64_t mxfp4_padded_k(int64_t k) { return (k + kStep - 1) / kStep * kStep; }

hipError_t launch_act_mxfp4(const uint16_t *x, int64_t m, int64_t k, uint8_t *codes,
                            uint8_t *scales, hipStream_t s) {
  if (m == 0 || k == 0) return hipSuccess;
  int64_t kp = mxfp4_padded_k(k);
  if (k == kp) {  // no padding: one long row
    k *= m;
    kp = k;
    m = 1;
  }
  constexpr int V = 2;
  const int64_t groups = (kp / 8 + kQThreads * V - 1) / (kQThreads * V);
  const dim3 grid(static_cast<unsigned>(groups < 1 << 20 ? groups : 1 << 20),
                  static_cast<unsigned>(m < 65535 ? m : 65535));
  hipLaunchKernelGGL((act_mxfp4_kernel<V>), grid, dim3(kQThreads), 0, s, x, m, k, kp, codes,
                     scales);
  return hipGetLastError();
}

// In one launch where one workgroup buckets (and the waves that quantize count in 32
// bits), in two or four otherwise.
hipError_t launch_moe_mxfp4_prepare(const uint16_t *x, int64_t t, int64_t k, const int32_t *ids,
                                    int32_t topk, int32_t n_experts, int32_t *counts,
                                    int32_t *offsets, int32_t *perm, int32_t *inv, MoETile *tiles,
                                    int32_t *n_tiles, int32_t tile_rows, uint8_t *xq, uint8_t *xs,
                                    hipStream_t s) {
  const int64_t pairs = t * topk;
  const int64_t kp = mxfp4_padded_k(k);
  if (pairs > kRouteOneGroupPairs) {
    const hipError_t e = launch_act_mxfp4(x, t, k, xq, xs, s);
    if (e != hipSuccess) return e;
    return launch_route(ids, pairs, topk, n_experts, counts, offsets, perm, inv, tiles, n_tiles,
                        tile_rows, nullptr, s);
  }
  if (n_experts < 1 || n_experts > kMaxExperts || pairs < 0) return hipErrorInvalidValue;
  const int64_t chunks = (kp / 8 + 127) / 128;
  const int64_t groups = 1 + (t * chunks + kRouteWaves - 1) / kRouteWaves;
  hipLaunchKernelGGL(fp4_route_act_kernel, dim3(static_cast<unsigned>(groups)),
                     dim3(kRouteThreads), 0, s, ids, pairs, n_experts, counts, offsets, perm, inv,
                     tiles, n_tiles, tile_rows, x, t, static_cast<int32_t>(k),
                     static_cast<int32_t>(kp), xq, xs);
  return hipGetLastError();
}

hipError_t launch_mxfp4_values(const uint8_t *codes, const uint8_t *scales, int64_t m, int64_t k,
                               uint16_t *out, hipStream_t s) {
  if (m == 0 || k == 0) return hipSuccess;
  int64_t kp = mxfp4_padded_k(k);
  if (k == kp) {
    k *= m;
    kp = k;
    m = 1;
  }
  const int64_t groups = (k / 8 + kQThreads - 1) / kQThreads;
  const dim3 grid(static_cast<unsigned>(groups < 1 << 20 ? groups : 1 << 20),
                  static_cast<unsigned>(m < 65535 ? m : 65535));
  hipLaunchKernelGGL(mxfp4_values_kernel, grid, dim3(kQThreads), 0, s, codes, scales, m, k, kp,
                     out);
  return hipGetLastError();
}

hipError_t launch_mxfp4_cache(const uint8_t *packed, int64_t n, int64_t k, uint32_t sign_bits,
                              uint8_t *codes, uint8_t *scales, hipStream_t s) {
  if (n == 0 || k == 0) return hipSuccess;
  const int64_t kpb = mxfp4_padded_k(k) / 32;
  const int64_t groups = (n * kpb + kQThreads - 1) / kQThreads;
  const int64_t grid = groups < 1 << 20 ? groups : 1 << 20;
  hipLaunchKernelGGL(mxfp4_cache_kernel, dim3(static_cast<unsigned>(grid)), dim3(kQThreads), 0, s,
                     packed, n, static_cast<int32_t>(k / 32), static_cast<int32_t>(kpb), sign_bits,
                     codebook(), codes, scales);
  return hipGetLastError();
}

bool mxfp4_direct_fits(int64_t m) { return m <= 16; }

hipError_t launch_linear_mxfp4_direct(const uint16_t *x, int64_t m, int64_t k, const uint8_t *wq,
                                      const uint8_t *ws, int64_t n, const Tail &tail, void *y,
                                      hipStream_t s) {
  if (!mxfp4_direct_fits(m)) return hipErrorInvalidValue;
  Fp4Args g = dense_args(m, k, wq, ws, n, tail, y);
  g.x = x;
  // 32 columns a workgroup where that still gives every compute unit one: the rows are read
  // and quantized half as often (2688 x 8192: one row 5.1 us, 16 rows 7.4, with 16 columns
  // 5.4 and 9.8; 16 x 4096 x 4096 9.9 and, 16 columns, 8.5; 16 x 8192 x 2688 16.4 and 13.4;
  // nothing was timed for n between 4096 and 8192).
  const int64_t wide = (n + 31) / 32;
  if (wide >= 256)
    hipLaunchKernelGGL((fp4_skinny_kernel<kDense, 2, 16, 1>),
                       dim3(static_cast<unsigned>(wide)), dim3(1024), 0, s, g);
  else
    hipLaunchKernelGGL((fp4_skinny_kernel<kDense, 1, 8, 1>),
                       dim3(static_cast<unsigned>((n + 15) / 16)), dim3(512), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_linear_mxfp4(const uint8_t *xq, const uint8_t *xs, int64_t m, int64_t k,
                               const uint8_t *wq, const uint8_t *ws, int64_t n, const Tail &tail,
                               void *y, hipStream_t s) {
  Fp4Args g = dense_args(m, k, wq, ws, n, tail, y);
  g.xq = xq;
  g.xs = xs;
  switch (pick_tile(m, k, n)) {
    case 0: return launch_tile<kDense, 16, 2, 2, 1, 1, 128, 5>(g, 0, s);
    case 1: return launch_tile<kDense, 16, 2, 2, 1, 2, 128, 4>(g, 0, s);
    case 2: return launch_tile<kDense, 16, 2, 2, 2, 2, 128, 3>(g, 0, s);
    case 3: return launch_tile<kDense, 32, 2, 2, 1, 2, 128, 2>(g, 0, s);
    case 4: return launch_tile<kDense, 32, 2, 4, 2, 1, 128, 2>(g, 0, s);
    case 5: return launch_tile<kDense, 32, 2, 4, 3, 2, 128, 2>(g, 0, s);
    default: return launch_tile<kDense, 32, 2, 4, 4, 2, 64, 4, 8, true>(g, 0, s);
  }
}

// Rows per tile by the average number of rows per expert, from sweeps of the layer over 128
// experts of 1856 x 2688 (us, uniform routing / Zipf): 0.75 rows 64-row tiles 96, 32-row
// 95 to 105; 1.5 rows 130 and 123; 12 rows 161 / 159, 32-row 158 / 170, 128-row 164 / 161; 48
// rows 197 / 232, 128-row 202 / 219, 256-row 210 / 228; 96 rows 128-row 258 / 286, 256-row
// 253 / 286; 192 rows 410 / 425 and 330 / 387.
// A height is halved where its workgroups (256 or, up to 128 rows, 128 columns each) would leave
// half of the compute units idle: 300 tokens of 8 experts, topk 6, 256-row tiles 57, 128-row 41
// (500 tokens 55 and 61); 500 tokens of 2 experts, one slot, 128-row 34, 64-row 28 (2000 tokens
// 45 and 52).
int mxfp4_moe_tile_rows(int64_t pairs, int32_t n_experts, int64_t n1, int64_t k) {
  const int64_t e = n_experts;
  const int64_t busy = pairs < e ? pairs : e;
  int rows = pairs <= 36 * e ? 64 : pairs <= 80 * e ? 128 : 256;
  while (rows > 64) {
    const int64_t tiles = busy * ((pairs + busy * rows - 1) / (busy * rows));
    const int64_t cols = rows == 256 ? 256 : 128;
    const int64_t blocks = (mxfp4_padded_k(n1) + cols - 1) / cols + (k + cols - 1) / cols;
    if (tiles * blocks >= 256) break;  // of both products: 128 each
    rows /= 2;
  }
  return rows;
}

// Up to 24 pairs (four tokens of six slots): one to four tokens 14.7, 22.0, 29.9 and 38.9 us,
// 24 to 25, 28, 33 and 37 to 40 for the batched steps, which are two launches more for the
// host.  That is six slots of 128 experts; an expert that several pairs share is read once for
// each of them here, and where there are few experts the batched steps read less (5 tokens of
// 8 experts 24.0).
bool mxfp4_moe_direct_fits(int64_t t, int32_t topk) {
  return t * topk <= 24 && topk <= kDirectSlots;
}

hipError_t launch_moe_mxfp4_direct(const uint16_t *x, int64_t t, int64_t k, const int32_t *ids,
                                   const float *gates, int32_t topk, int32_t n_experts,
                                   const uint8_t *w1, const uint8_t *s1, int64_t n1,
                                   const uint8_t *w2, const uint8_t *s2, uint8_t *hq, uint8_t *hs,
                                   float *out, hipStream_t s) {
  if (!mxfp4_moe_direct_fits(t, topk)) return hipErrorInvalidValue;
  Fp4Args g{};
  g.x = x;
  g.wq = w1;
  g.ws = s1;
  g.hq = hq;
  g.hs = hs;
  g.n = n1;
  g.n_store = static_cast<int32_t>(mxfp4_padded_k(n1));
  g.k = static_cast<int32_t>(k);
  g.kp = static_cast<int32_t>(mxfp4_padded_k(k));
  g.topk = topk;
  g.ids = ids;
  g.gates = gates;
  g.n_experts = n_experts;
  hipLaunchKernelGGL((fp4_skinny_kernel<kUp, 2, 4, 1>),
                     dim3(static_cast<unsigned>(g.n_store / 32), static_cast<unsigned>(t * topk)),
                     dim3(256), 0, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  g.xq = hq;
  g.xs = hs;
  g.wq = w2;
  g.ws = s2;
  g.y = out;
  g.n = k;
  g.k = static_cast<int32_t>(n1);
  g.kp = static_cast<int32_t>(mxfp4_padded_k(n1));
  hipLaunchKernelGGL((fp4_direct_down_kernel<2, 4>),
                     dim3(static_cast<unsigned>((k + 15) / 16), static_cast<unsigned>(t)),
                     dim3(static_cast<unsigned>(64 * 2 * topk)), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_moe_mxfp4(int mode, int tile_rows, const uint8_t *aq, const uint8_t *as,
                            int64_t a_rows, int64_t k, const int32_t *perm, int32_t topk,
                            int32_t n_experts, const uint8_t *wq, const uint8_t *ws, int64_t n,
                            const MoETile *tiles, const int32_t *n_tiles, int64_t max_tiles,
                            float *out, uint8_t *hq, uint8_t *hs, hipStream_t s) {
  if (max_tiles > 65535 || n % 32 != 0) return hipErrorInvalidValue;
  if (max_tiles == 0) return hipSuccess;
  Fp4Args g{};
  g.xq = aq;
  g.xs = as;
  g.wq = wq;
  g.ws = ws;
  g.y = out;
  g.hq = hq;
  g.hs = hs;
  g.n = n;
  g.n_store = static_cast<int32_t>(mxfp4_padded_k(n));
  g.k = static_cast<int32_t>(k);
  g.kp = static_cast<int32_t>(mxfp4_padded_k(k));
  g.perm = perm;
  g.tiles = tiles;
  g.n_tiles = n_tiles;
  g.a_rows = a_rows;
  g.topk = topk;
  g.tile_run = 1;
  switch (tile_rows) {
    case 64: {
      // 64 columns and three stages where workgroups of 128 columns leave compute units idle: 5
      // tokens of 8 experts 28.6 -> 24.0 us, 40 30.7 -> 25.6; but 40 of 24 43.8 -> 50.1, 16 of
      // 128 87 -> 92 (and four waves there, a tile each way, with two stages 42.5 and 88).
      const bool narrow = max_tiles * ((g.n_store + 127) / 128) <= 256;
      if (mode == 0)
        return narrow ? launch_tile<kUp, 32, 2, 2, 1, 1, 128, 3>(g, max_tiles, s)
                      : launch_tile<kUp, 32, 1, 4, 2, 1, 128, 2>(g, max_tiles, s);
      return narrow ? launch_tile<kDown, 32, 2, 2, 1, 1, 128, 3>(g, max_tiles, s)
                    : launch_tile<kDown, 32, 1, 4, 2, 1, 128, 2>(g, max_tiles, s);
    }
    case 128:
      if (mode == 0) return launch_tile<kUp, 32, 2, 4, 2, 1, 128, 2>(g, max_tiles, s);
      return launch_tile<kDown, 32, 2, 4, 2, 1, 128, 2>(g, max_tiles, s);
    case 256: {
      // With several tiles to an expert the loads go between the products (see the kernel):
      // 8192 tokens of 128 experts 622 -> 606 us, 3000 of 8 230 -> 220, but 4096 of 128
      // (192 rows an expert) 329 -> 334 and 2048 252 -> 265.
      const int64_t pairs = mode == 0 ? a_rows * topk : a_rows;
      const bool spread = pairs > 240 * static_cast<int64_t>(n_experts);
      // Two tiles, mostly of one expert, then follow each other on an XCD, whose L2 has the
      // weights for the second (8192 tokens 627 -> 596 us, 3000 of 64 experts 285 -> 272; 4096
      // of 128, one tile to an expert, 340 -> 342, 16 tokens 96 -> 104).
      if (spread) g.tile_run = 2;
      if (mode == 0)
        return spread ? launch_tile<kUp, 32, 2, 4, 4, 2, 128, 2>(g, max_tiles, s)
                      : launch_tile<kUp, 32, 2, 4, 4, 2, 128, 2, 8, false, false>(g, max_tiles, s);
      return spread ? launch_tile<kDown, 32, 2, 4, 4, 2, 128, 2>(g, max_tiles, s)
                    : launch_tile<kDown, 32, 2, 4, 4, 2, 128, 2, 8, false, false>(g, max_tiles, s);
    }
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tq4
