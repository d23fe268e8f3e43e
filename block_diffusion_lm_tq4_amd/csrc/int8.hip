// 8-bit integer products: the linear layer and the MoE layer of the model
// (Nemotron-TheHobbit-30B-A3B model card, Running it and The model
// underneath) on int8 weights with one scale per output channel and int8
// activations with one scale per token.
//
// Rows.  A row v[0..k) with a = max|v| is held as codes q_i = rint(127 v_i /
// a) (ties to even) and the scale s = fp32(a / 127); an all-zero row has s =
// 0, a row with a NaN or an infinity has s = NaN and zero codes.  For bf16 v
// the exact codes come out of fp32: with v_i = p 2^x, a = r 2^y (p, r in
// 128..255, d = y - x >= 0) the quotient is 127 p / (r 2^d); 127 p is exact,
// and the quotient is either a half-integer or at least 1 / (255 2^(d+1))
// away from one, while one correctly rounded fp32 division moves it by at
// most 2^(-17-d).  So the rounded quotient rounds to the same integer, and a
// tie is seen as a tie.
//
// Layout.  Codes are [rows][kp], kp = k rounded up to a multiple of 64 (the
// k of one MFMA step) with zero codes behind k, which add nothing.
//
// Products run on v_mfma_i32_16x16x64_i8: lane i + 16 g holds 16 bytes of
// row i of each operand, and both operands are read the same way, so the
// order of k inside a step does not matter.  Sums are exact in int32 (k <=
// 131072: 127^2 k < 2^31), so every split of k gives the same result.  The
// weights are the first operand: lane i + 16 g of the result holds columns n
// = 4 g .. 4 g + 3 of token i, four consecutive outputs.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq4_internal.h"

namespace tq4 {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

constexpr int kI8Step = 64;

// ---------------------------------------------------------------------------
// Rows to codes

constexpr int kQThreads = 256;

// Largest value over the workgroup; `red` holds one value per wave.
template <typename T>
__device__ inline T group_max(T v, T *red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
  __syncthreads();
  T m = red[0];
  for (int w = 1; w < kQThreads / 64; ++w) m = red[w] > m ? red[w] : m;
  return m;
}

__device__ inline int8_t code_of(float v, float a) {
  return static_cast<int8_t>(static_cast<int>(__builtin_rintf((v * 127.f) / a)));
}

// bf16 rows, one workgroup per row.  The magnitude bits of bf16 order like
// the magnitudes, infinities and NaN last (0x7F80 and above), so the largest
// magnitude is a maximum of integers.
__global__ __launch_bounds__(kQThreads) void act_int8_kernel(const uint16_t *__restrict__ x,
                                                             int64_t m, int64_t k, int64_t kp,
                                                             int8_t *__restrict__ codes,
                                                             float *__restrict__ scales) {
  __shared__ int red[kQThreads / 64];
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    const uint16_t *xr = x + row * k;
    int top = 0;
    for (int64_t i = threadIdx.x; i < k; i += kQThreads) {
      const int mag = xr[i] & 0x7FFF;
      top = mag > top ? mag : top;
    }
    top = group_max(top, red);
    __syncthreads();
    const bool finite = top < 0x7F80;
    // 2^-8 keeps 127 v finite for the largest rows; it changes no quotient of
    // a row that large, since codes below 1/2 are zero either way
    const float sc = top >= 0x7000 ? 0x1p-8f : 1.f;
    const float amax = __uint_as_float(static_cast<uint32_t>(top) << 16);
    const float a = amax * sc;
    int8_t *qr = codes + row * kp;
    for (int64_t i = threadIdx.x; i < kp; i += kQThreads) {
      int8_t q = 0;
      if (i < k && finite && top != 0)
        q = code_of(__uint_as_float(static_cast<uint32_t>(xr[i]) << 16) * sc, a);
      qr[i] = q;
    }
    if (threadIdx.x == 0) scales[row] = finite ? amax / 127.f : __builtin_nanf("");
  }
}

// Packed TQ4_1S rows, one workgroup per row, in fp64: the butterfly's sums v
// (sign undone) carry the row without its common factor 1/sqrt(32), which
// leaves the codes' quotient; the scale takes it back in.  The row is decoded
// twice, once for the maximum and once for the codes (offline work).
__device__ inline bool decode_block(const uint32_t *p, uint32_t sign_bits, const Codebook &cb,
                                    double (&v)[32]) {
  uint32_t wd[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) wd[i] = p[i];
  const float f0 = __uint_as_float((wd[4] & 0xFFFFu) << 16);
  const float f1 = __uint_as_float(wd[4] & 0xFFFF0000u);
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
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if ((sign_bits >> i) & 1u) v[i] = -v[i];
  return __builtin_isfinite(f0) && __builtin_isfinite(f1);
}

__global__ __launch_bounds__(kQThreads) void int8_cache_kernel(
    const uint8_t *__restrict__ packed, int64_t n, int64_t kb, int64_t kp, uint32_t sign_bits,
    Codebook cb, int8_t *__restrict__ codes, float *__restrict__ scales) {
  __shared__ double red[kQThreads / 64];
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const uint32_t *pr = reinterpret_cast<const uint32_t *>(packed + row * kb * 20);
    double top = 0.0;
    for (int64_t b = threadIdx.x; b < kb; b += kQThreads) {
      double v[32];
      if (!decode_block(pr + b * 5, sign_bits, cb, v)) top = __builtin_inf();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const double a = __builtin_fabs(v[i]);
        top = a > top ? a : top;
      }
    }
    top = group_max(top, red);
    __syncthreads();
    const bool finite = top < __builtin_inf();
    const double rs32 = 0x1.6a09e667f3bcdp-3;  // 1/sqrt(32)
    for (int64_t b = threadIdx.x; b < kp / 32; b += kQThreads) {
      uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (b < kb && finite && top > 0.0) {
        double v[32];
        decode_block(pr + b * 5, sign_bits, cb, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int q = static_cast<int>(__builtin_rint((v[i] * 127.0) / top));
          out[i / 4] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * (i % 4));
        }
      }
      uint4 *dst = reinterpret_cast<uint4 *>(codes + row * kp + b * 32);
      dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
      dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
    if (threadIdx.x == 0)
      scales[row] = finite ? static_cast<float>((top * rs32) / 127.0) : __builtin_nanf("");
  }
}

// ---------------------------------------------------------------------------
// Products

struct I8Args {
  const int8_t *xq;   // activation codes [rows][kp]
  const float *xs;    // their scales
  const int8_t *wq;   // weight codes [n][kp] (experts stacked)
  const float *ws;    // their scales
  void *y;            // dense: [m][n] fp32 or bf16; up: h bf16; down: fp32
  Tail tail;          // dense only
  int64_t m, n, kp;
  const int32_t *perm;    // MoE: bucket order (up gathers through it)
  const MoETile *tiles;
  const int32_t *n_tiles;
  int32_t topk;
};

enum { kI8Dense = 0, kI8Up = 1, kI8Down = 2 };

// The hidden value: u decided in fp64 (a product of an exact sum and two
// scales), relu(u)^2 rounded to fp32 and then to bf16.  A NaN stays one.
__device__ inline uint16_t hidden_of(int acc, float sx, float sw) {
  const double u = (static_cast<double>(acc) * static_cast<double>(sx)) * static_cast<double>(sw);
  const double h = u < 0.0 ? 0.0 : u * u;
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(static_cast<float>(h)));
}

// One wave per 16 tokens x 16 columns, operands straight from memory.
template <int MODE>
__global__ __launch_bounds__(64) void i8_plain_kernel(I8Args g) {
  const int lane = threadIdx.x;
  const int r = lane % 16;
  const int grp = lane / 16;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  int64_t m0, rows, w0 = 0;
  if constexpr (MODE == kI8Dense) {
    m0 = static_cast<int64_t>(blockIdx.y) * 16;
    rows = g.m - m0 < 16 ? g.m - m0 : 16;
  } else {
    if (static_cast<int32_t>(blockIdx.y) >= *g.n_tiles) return;
    const MoETile t = g.tiles[blockIdx.y];
    m0 = t.row0;
    rows = t.rows;
    w0 = static_cast<int64_t>(t.expert) * g.n;
  }
  const int64_t nr = n0 + r < g.n ? n0 + r : g.n - 1;
  const int64_t mr = m0 + (r < rows ? r : 0);
  const int64_t src = MODE == kI8Up ? g.perm[mr] / g.topk : mr;
  const int8_t *wp = g.wq + (w0 + nr) * g.kp + 16 * grp;
  const int8_t *xp = g.xq + src * g.kp + 16 * grp;
  intx4 acc = {0, 0, 0, 0};
  for (int64_t k0 = 0; k0 < g.kp; k0 += kI8Step) {
    const intx4 a = *reinterpret_cast<const intx4 *>(wp + k0);
    const intx4 b = *reinterpret_cast<const intx4 *>(xp + k0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc, 0, 0, 0);
  }
  if (r >= rows) return;
  const float sx = g.xs[src];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t n = n0 + 4 * grp + v;
    if (n >= g.n) continue;
    const float sw = g.ws[w0 + n];
    if constexpr (MODE == kI8Up) {
      static_cast<uint16_t *>(g.y)[(m0 + r) * g.n + n] = hidden_of(acc[v], sx, sw);
    } else {
      const float p = (static_cast<float>(acc[v]) * sx) * sw;
      if constexpr (MODE == kI8Down)
        static_cast<float *>(g.y)[(m0 + r) * g.n + n] = p;
      else
        tail_apply(g.tail, static_cast<float *>(g.y), m0 + r, n, g.n, p);
    }
  }
}

}  // namespace

int64_t int8_padded_k(int64_t k) { return (k + kI8Step - 1) / kI8Step * kI8Step; }

hipError_t launch_act_int8(const uint16_t *x, int64_t m, int64_t k, int8_t *codes, float *scales,
                           hipStream_t s) {
  if (m == 0 || k == 0) return hipSuccess;
  const int64_t grid = m < 65536 ? m : 65536;
  hipLaunchKernelGGL(act_int8_kernel, dim3(static_cast<unsigned>(grid)), dim3(kQThreads), 0, s, x,
                     m, k, int8_padded_k(k), codes, scales);
  return hipGetLastError();
}

hipError_t launch_int8_cache(const uint8_t *packed, int64_t n, int64_t k, uint32_t sign_bits,
                             int8_t *codes, float *scales, hipStream_t s) {
  if (n == 0 || k == 0) return hipSuccess;
  const int64_t grid = n < 65536 ? n : 65536;
  hipLaunchKernelGGL(int8_cache_kernel, dim3(static_cast<unsigned>(grid)), dim3(kQThreads), 0, s,
                     packed, n, k / 32, int8_padded_k(k), sign_bits, codebook(), codes, scales);
  return hipGetLastError();
}

hipError_t launch_linear_int8(const int8_t *xq, const float *xs, int64_t m, int64_t k,
                              const int8_t *wq, const float *ws, int64_t n, const Tail &tail,
                              void *y, hipStream_t s) {
  I8Args g{};
  g.xq = xq;
  g.xs = xs;
  g.wq = wq;
  g.ws = ws;
  g.y = y;
  g.tail = tail;
  g.m = m;
  g.n = n;
  g.kp = int8_padded_k(k);
  const dim3 grid(static_cast<unsigned>((n + 15) / 16), static_cast<unsigned>((m + 15) / 16));
  hipLaunchKernelGGL(i8_plain_kernel<kI8Dense>, grid, dim3(64), 0, s, g);
  return hipGetLastError();
}

int int8_moe_tile_rows(int64_t pairs, int32_t n_experts) {
  (void)pairs;
  (void)n_experts;
  return 16;
}

hipError_t launch_moe_int8(int mode, int tile_rows, const int8_t *aq, const float *as, int64_t k,
                           const int32_t *perm, int32_t topk, const int8_t *wq, const float *ws,
                           int64_t n, const MoETile *tiles, const int32_t *n_tiles,
                           int64_t max_tiles, void *out, hipStream_t s) {
  if (max_tiles > 65535 || tile_rows != 16) return hipErrorInvalidValue;
  if (max_tiles == 0) return hipSuccess;
  I8Args g{};
  g.xq = aq;
  g.xs = as;
  g.wq = wq;
  g.ws = ws;
  g.y = out;
  g.n = n;
  g.kp = int8_padded_k(k);
  g.perm = perm;
  g.tiles = tiles;
  g.n_tiles = n_tiles;
  g.topk = topk;
  const dim3 grid(static_cast<unsigned>((n + 15) / 16), static_cast<unsigned>(max_tiles));
  if (mode == 0)
    hipLaunchKernelGGL(i8_plain_kernel<kI8Up>, grid, dim3(64), 0, s, g);
  else
    hipLaunchKernelGGL(i8_plain_kernel<kI8Down>, grid, dim3(64), 0, s, g);
  return hipGetLastError();
}

}  // namespace tq4
