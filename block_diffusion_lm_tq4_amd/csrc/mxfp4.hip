// MXFP4 products: the linear layer and the MoE layer of the model
// (Nemotron-TheHobbit-30B-A3B model card, Running it and The model underneath; Help
// wanted: a resident copy that no forward decodes) on 4-bit floating-point operands.
//
// Rows.  32 consecutive values of a row share a scale 2^e, held as the byte e + 127;
// with a = max|v|, e is the smallest integer from -127 with a < 7 * 2^e.  A value is
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
// Products run on v_mfma_scale_f32_16x16x128_f8f6f4: lane i + 16 g holds the 32 values
// k = 32 g .. 32 g + 31 of row i of each operand as they lie in memory (16 bytes), and
// their scale byte.  A product of two codes is a multiple of 0.25 up to 36, so a block's
// sum is exact, and a row's is while 2^24 times the smallest unit 0.25 * 2^(e + f) it
// meets holds it; below that every split of k gives the same bits, past it sums round to
// fp32.  The weights are the first operand: lane i + 16 g of the result
// holds columns n = 4 g .. 4 g + 3 of token i, four consecutive outputs.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxfp4.h"

namespace tq4 {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t ushortx2 __attribute__((ext_vector_type(2)));

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

// Pieces of 8 values, V per thread; four lanes share a block.  Grid: pieces of a row x
// rows.  HBM-bound: 2.53 bytes per value.
template <int V>
__global__ __launch_bounds__(kQThreads) void act_mxfp4_kernel(const uint16_t *__restrict__ x,
                                                              int64_t rows, int64_t k, int64_t kp,
                                                              uint8_t *__restrict__ codes,
                                                              uint8_t *__restrict__ scales) {
  const int64_t n_vec = k / 8, n_out = kp / 8;  // k is a multiple of 32
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const uint4 *xr = reinterpret_cast<const uint4 *>(x + row * k);
    uint32_t *qr = reinterpret_cast<uint32_t *>(codes + row * (kp / 2));
    uint8_t *sr = scales + row * (kp / 32);
    // a row's pieces are a multiple of 16, so the lanes of a block stay together
    for (int64_t at0 = static_cast<int64_t>(blockIdx.x) * (kQThreads * V) + threadIdx.x;
         at0 < n_out; at0 += static_cast<int64_t>(gridDim.x) * (kQThreads * V)) {
      uint4 d[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int64_t at = at0 + kQThreads * i;
        d[i] = at < n_vec ? xr[at] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int64_t at = at0 + kQThreads * i;
        const uint32_t byte = scale_of_bf16(quad_max(top_of(top_of(d[i]))));
        if (at >= n_out) continue;
        qr[at] = codes_of(d[i], byte);
        if (threadIdx.x % 4 == 0) sr[at / 4] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// The values that codes stand for, as bf16 (exact: a code has one mantissa bit; what
// the largest scales put past bf16's range is infinite).  A thread takes 8.
__global__ __launch_bounds__(kQThreads) void mxfp4_values_kernel(
    const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows,
    int64_t k, int64_t kp, uint16_t *__restrict__ out) {
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y)
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; at < k / 8;
       at += static_cast<int64_t>(gridDim.x) * kQThreads) {
    const uint32_t c = reinterpret_cast<const uint32_t *>(codes + row * (kp / 2))[at];
    const uint32_t byte = scales[row * (kp / 32) + at / 4];
    // 2^(byte - 127), its last three binades and NaN made by two factors
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t half[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t q = (c >> (8 * i + 4 * h)) & 15u;
        const uint32_t e = (q >> 1) & 3u, man = q & 1u;
        // 2^(e - 1) * (1 + man / 2) for e > 0, man / 2 for e = 0
        const float mag = e == 0 ? 0.5f * static_cast<float>(man)
                                 : __uint_as_float((126u + e) << 23 | man << 22);
        const float lo = byte < 64 ? mag * 0x1p-96f * __uint_as_float((byte + 96u) << 23)
                                   : mag * 0x1p+32f * __uint_as_float((byte - 32u) << 23);
        uint32_t b = __float_as_uint(lo) >> 16;
        if (byte == kNanScale) b = 0x7FC0u;
        half[h] = b | (q & 8u) << 12;
      }
      w[i] = half[0] | half[1] << 16;
    }
    reinterpret_cast<uint4 *>(out + row * k)[at] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Packed TQ4_1S rows: one thread per block, decoded (rotation undone) and encoded in
// fp64, so that the codes are those of the rule.  Offline.
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
          e = e < -127 ? -127 : e;
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
  int64_t a_rows;      // MoE: rows of xq
  int32_t topk;
};

enum { kDense = 0, kUp = 1, kDown = 2 };

__device__ inline floatx4 mfma_fp4(intx4 a, intx4 b, floatx4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      intx8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, intx8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4,
      4, 0, sa, 0, sb);
}

// Two values rounded to bf16 (ties to even), a in the low half.
__device__ inline uint32_t bf16_pair(float a, float b) {
  typedef float pair __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((pair{a, b}), bf16x2));
}

// A wave's 16 x 16 block of a dense output: row lane % 16 of `rows` valid ones from m0,
// columns n0 + 4 (lane / 16) ....
template <bool BF16, bool VEC>
__device__ inline void store_block(const Fp4Args &g, floatx4 acc, int64_t m0, int rows, int64_t n0,
                                   int lane) {
#pragma clang fp contract(off)
  const int r = lane % 16;
  const int64_t n = n0 + 4 * (lane / 16);
  const int left = g.n - n < 4 ? static_cast<int>(g.n - n) : 4;
  if (r >= rows || left <= 0) return;
  const int64_t at = (m0 + r) * g.n + n;
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

__device__ inline void store_any(const Fp4Args &g, floatx4 acc, int64_t m0, int rows, int64_t n0,
                                 int lane) {
  if (g.vec) {
    if (g.tail.bf16)
      store_block<true, true>(g, acc, m0, rows, n0, lane);
    else
      store_block<false, true>(g, acc, m0, rows, n0, lane);
  } else {
    if (g.tail.bf16)
      store_block<true, false>(g, acc, m0, rows, n0, lane);
    else
      store_block<false, false>(g, acc, m0, rows, n0, lane);
  }
}

// The hidden block of a lane's row: columns 16 j + 4 g .. + 3 of sub-tiles j = 0 and 1 are
// 8 of its 32 values, the others are in lanes l ^ 16, l ^ 32, l ^ 48.  Squares of the
// positive parts (fp32) to scale byte and codes, sub-tile 0's in the low half.
__device__ inline uint32_t hidden_block(floatx4 a, floatx4 b, uint32_t &byte) {
  float h[8];
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    const float u = v < 4 ? a[v % 4] : b[v % 4];
    const float p = u < 0.f ? 0.f : u;  // a NaN stays one
    h[v] = p * p;
    const uint32_t m = __float_as_uint(h[v]) & 0x7FFFFFFFu;
    top = m > top ? m : top;
  }
  uint32_t lo, hi;
  lane_pair16(top, lo, hi);
  top = lo > hi ? lo : hi;
  lane_pair32(top, lo, hi);
  top = lo > hi ? lo : hi;
  byte = scale_of_f32(top);
  const float s = scale_operand(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[0], h[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[2], h[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[4], h[5], s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[6], h[7], s, 3);
  return byte == kNanScale ? 0u : r;
}

// ---- few rows ---------------------------------------------------------------
// 16 rows and 16 NT columns per workgroup of KW waves; wave w takes the steps [w * per,
// (w + 1) * per), B at a time, all loads of a batch issued before its first product.  The
// weights are read once, straight into registers.  With QX the rows come as bf16 and
// each lane quantizes the blocks that it holds: a block's 32 values are one lane's, so
// that takes no exchange.  The waves' sums meet in LDS, added in wave order.
template <int MODE, bool QX, int NT, int KW, int B>
__global__ __launch_bounds__(64 * KW) void fp4_skinny_kernel(Fp4Args g) {
  __shared__ floatx4 red[KW > 1 ? KW - 1 : 1][NT][64];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % 16;
  const int grp = lane / 16;

  int64_t n0, m0, w0 = 0;
  int rows;
  if constexpr (MODE == kDense) {
    n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT);
    m0 = static_cast<int64_t>(blockIdx.y) * 16;
    rows = g.m - m0 < 16 ? static_cast<int>(g.m - m0) : 16;
  } else {
    // column blocks are dealt to the XCDs (workgroup id % 8), rotated by the
    // expert, so that an expert's tiles of one column block share an L2 and
    // every XCD gets its share of blocks
    const int per = (g.tiles_n + 7) / 8;
    const int q = static_cast<int>(blockIdx.x) / 8;
    const int i = q / per;
    if (i >= *g.n_tiles) return;
    const MoETile t = g.tiles[i];
    const int j = (static_cast<int>(blockIdx.x) + t.expert) % 8 + 8 * (q % per);
    if (j >= g.tiles_n) return;
    n0 = static_cast<int64_t>(j) * (16 * NT);
    m0 = t.row0;
    rows = t.rows;
    w0 = static_cast<int64_t>(t.expert) * g.n;
  }

  const int32_t row_bytes = g.kp / 2, row_scales = g.kp / 32;
  const uint8_t *wp[NT], *wsp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = n0 + 16 * j + r;
    const int64_t nr = w0 + (n < g.n ? n : g.n - 1);  // past n: read n - 1
    wp[j] = g.wq + nr * row_bytes + 16 * grp;
    wsp[j] = g.ws + nr * row_scales + grp;
  }
  const int64_t mr = m0 + (r < rows ? r : 0);  // past the rows: the first
  const int64_t src = MODE == kUp ? g.perm[mr] / g.topk : mr;
  const uint8_t *xp = QX ? nullptr : g.xq + src * row_bytes + 16 * grp;
  const uint8_t *xsp = QX ? nullptr : g.xs + src * row_scales + grp;
  const uint4 *xb = QX ? reinterpret_cast<const uint4 *>(g.x + src * g.k) + 4 * grp : nullptr;
  floatx4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};

  const int steps = g.kp / kStep;
  const int per = (steps + KW - 1) / KW;
  const int s0 = wave * per;
  const int s1 = s0 + per < steps ? s0 + per : steps;
  for (int s = s0; s < s1; s += B) {
    intx4 a[B][NT], b[B];
    uint4 raw[QX ? B : 1][4];
    int sa[B][NT], sb[B];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      // steps past the wave's end reload its last one and are not multiplied
      const int at = s + u < s1 ? s + u : s1 - 1;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        a[u][j] = *reinterpret_cast<const intx4 *>(wp[j] + static_cast<int64_t>(at) * kStepBytes);
        sa[u][j] = wsp[j][4 * at];
      }
      if constexpr (QX) {
        const bool in = kStep * at + 32 * grp < g.k;  // whole blocks: k % 32 == 0
#pragma unroll
        for (int q = 0; q < 4; ++q)
          raw[u][q] = in ? xb[16 * at + q] : make_uint4(0u, 0u, 0u, 0u);
      } else {
        b[u] = *reinterpret_cast<const intx4 *>(xp + static_cast<int64_t>(at) * kStepBytes);
        sb[u] = xsp[4 * at];
      }
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if constexpr (QX) {
        ushortx2 t = top_of(raw[u][0]);
#pragma unroll
        for (int q = 1; q < 4; ++q) t = __builtin_elementwise_max(t, top_of(raw[u][q]));
        const uint32_t byte = scale_of_bf16(top_of(t));
#pragma unroll
        for (int q = 0; q < 4; ++q) b[u][q] = static_cast<int>(codes_of(raw[u][q], byte));
        sb[u] = static_cast<int>(byte);
      }
      if (s + u < s1) {
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = mfma_fp4(a[u][j], b[u], acc[j], sa[u][j], sb[u]);
      }
    }
  }
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
    for (int j = 0; j < NT; ++j) store_any(g, acc[j], m0, rows, n0 + 16 * j, lane);
  } else if constexpr (MODE == kUp) {
    static_assert(MODE != kUp || NT == 2, "a hidden block is two sub-tiles");
    uint32_t byte;
    if (n0 >= g.n) acc[0] = acc[1] = floatx4{0.f, 0.f, 0.f, 0.f};  // n % 32 == 0
    const uint32_t c = hidden_block(acc[0], acc[NT - 1], byte);
    if (r >= rows || n0 >= g.n_store) return;
    uint16_t *q = reinterpret_cast<uint16_t *>(g.hq + (m0 + r) * (g.n_store / 2) + n0 / 2);
    q[grp] = static_cast<uint16_t>(c);
    q[4 + grp] = static_cast<uint16_t>(c >> 16);
    if (grp == 0) g.hs[(m0 + r) * (g.n_store / 32) + n0 / 32] = static_cast<uint8_t>(byte);
  } else {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t n = n0 + 16 * j + 4 * grp;
      if (r < rows && n < g.n)
        *reinterpret_cast<floatx4 *>(static_cast<float *>(g.y) + (m0 + r) * g.n + n) = acc[j];
    }
  }
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
  hipLaunchKernelGGL((fp4_skinny_kernel<kDense, true, 1, 8, 2>),
                     dim3(static_cast<unsigned>((n + 15) / 16)), dim3(512), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_linear_mxfp4(const uint8_t *xq, const uint8_t *xs, int64_t m, int64_t k,
                               const uint8_t *wq, const uint8_t *ws, int64_t n, const Tail &tail,
                               void *y, hipStream_t s) {
  Fp4Args g = dense_args(m, k, wq, ws, n, tail, y);
  // 2^16 - 16 tile rows of 16 at a time
  constexpr int64_t kRows = 16 * 65520;
  for (int64_t m0 = 0; m0 < m; m0 += kRows) {
    const int64_t rows = m - m0 < kRows ? m - m0 : kRows;
    g.xq = xq + m0 * (g.kp / 2);
    g.xs = xs + m0 * (g.kp / 32);
    g.m = rows;
    const size_t each = tail.bf16 ? 2 : 4;
    g.y = static_cast<char *>(y) + static_cast<size_t>(m0 * n) * each;
    if (tail.residual != nullptr)
      g.tail.residual =
          static_cast<const char *>(tail.residual) + static_cast<size_t>(m0 * n) * each;
    hipLaunchKernelGGL((fp4_skinny_kernel<kDense, false, 1, 4, 4>),
                       dim3(static_cast<unsigned>((n + 15) / 16),
                            static_cast<unsigned>((rows + 15) / 16)),
                       dim3(256), 0, s, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int mxfp4_moe_tile_rows(int64_t, int32_t) { return 16; }

hipError_t launch_moe_mxfp4(int mode, int tile_rows, const uint8_t *aq, const uint8_t *as,
                            int64_t a_rows, int64_t k, const int32_t *perm, int32_t topk,
                            const uint8_t *wq, const uint8_t *ws, int64_t n, const MoETile *tiles,
                            const int32_t *n_tiles, int64_t max_tiles, float *out, uint8_t *hq,
                            uint8_t *hs, hipStream_t s) {
  if (max_tiles > 65535 || n % 32 != 0 || tile_rows != 16) return hipErrorInvalidValue;
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
  g.tiles_n = static_cast<int32_t>(((mode == 0 ? g.n_store : n) + 31) / 32);
  const int64_t grid = max_tiles * ((g.tiles_n + 7) / 8 * 8);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  if (mode == 0)
    hipLaunchKernelGGL((fp4_skinny_kernel<kUp, false, 2, 4, 3>),
                       dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((fp4_skinny_kernel<kDown, false, 2, 4, 4>),
                       dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace tq4
