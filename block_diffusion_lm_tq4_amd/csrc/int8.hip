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

#include <type_traits>

#include "int8_router.h"

namespace tq4 {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

constexpr int kI8Step = 64;

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
#include "moe_route.h"

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

// What a row's largest magnitude bits say about it.
struct RowScale {
  float c127, inv, a, half, scale;
  bool live;
  __device__ explicit RowScale(uint32_t top) {
    // a power of two that keeps 127 v and 1 / a in range; it changes no
    // quotient: what the smaller one could drop has the code 0
    const float sc = top >= 0x7000u ? 0x1p-8f : (top < 0x1000u ? 0x1p+96f : 1.f);
    const float amax = __uint_as_float(top << 16);
    c127 = sc * 127.f;
    a = amax * sc;
    half = 0.5f * a;
    inv = __builtin_amdgcn_rcpf(a);
    const bool finite = top < 0x7F80u;
    live = finite && top != 0;
    scale = finite ? amax / 127.f : __builtin_nanf("");
  }
};

// Eight codes of one 16-byte piece of a bf16 row.  fma(127 v, 1 / a, 1.5 * 2^23)
// rounds the quotient to an integer, whose code is the low byte of the result:
// one rounding of a value that is off by at most 2^-23 of itself, so it is the
// exact quotient's unless that is a half-integer (see above).  Then, and only
// then, the remainder 127 v - q a (exact in one fma: both terms are multiples of
// v's last bit, and it is at most a / 2) is plus or minus a / 2, and the even
// neighbour is taken.  Seven instructions for a code, the piece's ties apart;
// with a division it was about 20.
__device__ inline uint2 codes_of(uint4 d, const RowScale &rs) {
  constexpr float kMagic = 12582912.f;
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
  float t[8], rho[8];
  bool tie = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    const float p = v * rs.c127;
    t[j] = __builtin_fmaf(p, rs.inv, kMagic);
    rho[j] = __builtin_fmaf(kMagic - t[j], rs.a, p);
    tie |= __builtin_fabsf(rho[j]) == rs.half;
  }
  if (__builtin_expect(tie, 0)) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (__builtin_fabsf(rho[j]) == rs.half && (__float_as_uint(t[j]) & 1u))
        t[j] += rho[j] > 0.f ? 1.f : -1.f;
  }
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 1]),
                                              __float_as_uint(t[4 * h]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 3]),
                                              __float_as_uint(t[4 * h + 2]), 0x04000C0Cu);
    out[h] = lo | hi;
  }
  return make_uint2(out[0], out[1]);
}

// The largest magnitude bits of a piece, the even and the odd values apart.
// Magnitude bits of bf16 order like the magnitudes, infinities and NaN last
// (0x7F80 and above).
typedef uint16_t ushortx2 __attribute__((ext_vector_type(2)));

__device__ inline ushortx2 top_of(uint4 d) {
  auto mag = [](uint32_t w) { return __builtin_bit_cast(ushortx2, w & 0x7FFF7FFFu); };
  return __builtin_elementwise_max(__builtin_elementwise_max(mag(d.x), mag(d.y)),
                                   __builtin_elementwise_max(mag(d.z), mag(d.w)));
}
__device__ inline uint32_t top_of(ushortx2 t) { return t[0] > t[1] ? t[0] : t[1]; }

// One bf16 row by T threads (thread tid of them); `red` is for T > 64, which all
// threads of the workgroup enter together.  A row of up to T * 8 * V values
// stays in registers between the maximum and the codes; longer ones are read
// twice.
template <int T, int V>
__device__ inline void act_row(const uint4 *xr, int32_t k, int32_t kp, int tid, uint32_t *red,
                               uint2 *qr, float *scale) {
  const int n_vec = k / 8;    // k is a multiple of 32
  const int n_out = kp / 8;
  uint4 d[V];
  ushortx2 tops = {0, 0};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = tid + T * i;
    d[i] = at < n_vec ? xr[at] : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) tops = __builtin_elementwise_max(tops, top_of(d[i]));
  for (int at = tid + T * V; at < n_vec; at += T)
    tops = __builtin_elementwise_max(tops, top_of(xr[at]));
  uint32_t top = top_of(tops);
  if constexpr (T == 64) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const uint32_t o = __shfl_xor(top, s);
      top = top > o ? top : o;
    }
  } else {
    top = group_max(top, red);
    __syncthreads();
  }
  const RowScale rs(top);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = tid + T * i;
    if (at < n_out)
      qr[at] = rs.live ? codes_of(d[i], rs) : make_uint2(0u, 0u);
  }
  for (int at = tid + T * V; at < n_out; at += T)
    qr[at] = rs.live && at < n_vec ? codes_of(xr[at], rs) : make_uint2(0u, 0u);
  if (tid == 0) *scale = rs.scale;
}

// Rows of a matrix, T threads each (64: a wave per row, four rows per workgroup,
// no barrier; 256: the workgroup).  HBM-bound: 3 bytes per value.
template <int T, int V>
__global__ __launch_bounds__(kQThreads) void act_int8_kernel(const uint16_t *__restrict__ x,
                                                             int64_t m, int32_t k, int32_t kp,
                                                             int8_t *__restrict__ codes,
                                                             float *__restrict__ scales) {
  __shared__ uint32_t red[kQThreads / 64];
  constexpr int kRows = kQThreads / T;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T; row < m;
       row += static_cast<int64_t>(gridDim.x) * kRows)
    act_row<T, V>(reinterpret_cast<const uint4 *>(x + row * k), k, kp, threadIdx.x % T, red,
                  reinterpret_cast<uint2 *>(codes + row * kp), scales + row);
}

// The MoE layer's first launch: workgroup 0 buckets the pairs, the others
// quantize the tokens, a wave per row.  Neither needs the other's result, and
// the bucketing is one workgroup's chain of latencies (7 us for 16 tokens, 12
// for 1024) in which the rest of the device is free.
__global__ __launch_bounds__(kRouteThreads) void i8_route_act_kernel(
    const int32_t *ids, int64_t pairs, int32_t n_experts, int32_t *counts, int32_t *offsets,
    int32_t *perm, int32_t *inv, MoETile *tiles, int32_t *n_tiles, int32_t tile_rows,
    const uint16_t *__restrict__ x, int64_t t, int32_t k, int32_t kp, int8_t *__restrict__ codes,
    float *__restrict__ scales) {
  __shared__ int32_t hist[kRouteWaves][kMaxExperts];
  __shared__ int32_t base[kMaxExperts + 1];
  __shared__ int32_t tile_base[kMaxExperts + 1];
  if (blockIdx.x > 0) {
    const int64_t row =
        static_cast<int64_t>(blockIdx.x - 1) * kRouteWaves + threadIdx.x / 64;
    if (row < t)
      act_row<64, 8>(reinterpret_cast<const uint4 *>(x + row * k), k, kp, threadIdx.x % 64,
                     nullptr, reinterpret_cast<uint2 *>(codes + row * kp), scales + row);
    return;
  }
  bucket_group<kRouteWaves>(hist, base, tile_base, ids, pairs, n_experts, counts, offsets, perm,
                            inv, tiles, n_tiles, tile_rows, nullptr);
}

// Packed TQ4_1S rows, one workgroup per row, in fp64: the butterfly's sums v
// (sign undone) carry the row without its common factor 1/sqrt(32), which
// leaves the codes' quotient; the scale takes it back in.  The row is decoded
// twice, once for the maximum and once for the codes (offline work): 237568 rows of
// 2688 take 1.8 ms, 0.6 TB/s of what they read and write, bound by the fp64.
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
  int64_t m, n;
  int32_t kp;
  int32_t tiles_m, tiles_n;
  int32_t vec;            // n % 4 == 0 and y, bias, residual aligned for 4 outputs
  const int32_t *perm;    // MoE: bucket order (up gathers through it)
  const MoETile *tiles;
  const int32_t *n_tiles;
  int64_t a_rows;         // MoE: rows of xq
  int32_t topk;
};

enum { kI8Dense = 0, kI8Up = 1, kI8Down = 2 };

typedef __attribute__((address_space(3))) void lds_void;
constexpr int kI8BufferFlags = 0x00020000;

// Two values rounded to bf16 (ties to even), a in the low half.
__device__ inline uint32_t bf16_pair(float a, float b) {
  typedef float pair __attribute__((ext_vector_type(2)));
  typedef __bf16 out __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((pair{a, b}), out));
}

// The hidden value by its definition: u in fp64, relu(u)^2 rounded to fp32
// and then to bf16.  A NaN stays one.
__device__ inline float hidden_f64(int acc, float sx, float sw) {
  const double u = (static_cast<double>(acc) * static_cast<double>(sx)) * static_cast<double>(sw);
  const double h = u < 0.0 ? 0.0 : u * u;
  return static_cast<float>(h);
}

// The same for four sums of one row, in fp32 where that decides it.  With both
// scales zero or in [2^-30, 2^16] (`tame`, of all the wave's) nothing leaves
// fp32's normal range: u = acc * (sx * sw) carries at most three roundings and
// its square seven, 7 * 2^-24 relative, i.e. at most 7 fp32 steps, so the bf16
// rounding is settled unless the low 16 bits are within 8 of the tie.  About one
// value in 4000 is not, and its wave's quads take fp64.  The test takes 1.5
// instructions a value, on halves packed in pairs, and one branch a quad: at 4096
// tokens the up product is bound by what its epilogue issues as much as by what
// it stores (a compare and a flag for each value: 6 us of 197 more, a
// branch for each: 100 more).
__device__ inline bool tame_scale(float s) {
  return s == 0.f || (s >= 0x1p-30f && s <= 0x1p+16f);
}

__device__ inline uint2 hidden_quad(intx4 acc, float sx, const float (&sw)[4], bool tame) {
  float h[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float u = static_cast<float>(acc[v] > 0 ? acc[v] : 0) * (sx * sw[v]);
    h[v] = u * u;
  }
  // the low halves, moved so that 8 below the tie is 0
  auto low = [](float a, float b) {
    const uint32_t d = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x05040100u);
    return __builtin_bit_cast(ushortx2, d) + ushortx2{0x8008, 0x8008};
  };
  const ushortx2 near = __builtin_elementwise_min(low(h[0], h[1]), low(h[2], h[3]));
  const uint16_t nearest = near[0] < near[1] ? near[0] : near[1];
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(nearest <= (tame ? 16 : 0xFFFF)) != 0, 0)) {
#pragma unroll
    for (int v = 0; v < 4; ++v) h[v] = hidden_f64(acc[v], sx, sw[v]);
  }
  return make_uint2(bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3]));
}

// One row's four consecutive outputs n .. n + 3 of the MoE products (n % 32
// == 0 columns in all, so a quad is whole or past the end).
template <int MODE>
__device__ inline void store_moe(const I8Args &g, intx4 acc, int64_t row, int64_t n, float sx,
                                 const float (&sw)[4]) {
  if (n >= g.n) return;
  if constexpr (MODE == kI8Up) {
    const bool own = tame_scale(sx) && tame_scale(sw[0]) && tame_scale(sw[1]) &&
                     tame_scale(sw[2]) && tame_scale(sw[3]);
    const bool tame = __builtin_amdgcn_ballot_w64(!own) == 0;
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.y) + row * g.n + n) =
        hidden_quad(acc, sx, sw, tame);
  } else {
    float p[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) p[v] = (static_cast<float>(acc[v]) * sx) * sw[v];
    *reinterpret_cast<float4 *>(static_cast<float *>(g.y) + row * g.n + n) =
        make_float4(p[0], p[1], p[2], p[3]);
  }
}

// Quads of a dense output, VEC at a time as one access (else element by
// element with the matrix's edge).  Loads of the residual are kept apart from
// the stores: it may be y itself, so a store between them would put every
// load behind it.
template <bool BF16, bool VEC>
__device__ inline void load_residual(const I8Args &g, int64_t at, int left, float (&res)[4]) {
  if constexpr (VEC && BF16) {
    const uint2 d =
        *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(g.tail.residual) + at);
    res[0] = __uint_as_float(d.x << 16);
    res[1] = __uint_as_float(d.x & 0xFFFF0000u);
    res[2] = __uint_as_float(d.y << 16);
    res[3] = __uint_as_float(d.y & 0xFFFF0000u);
  } else if constexpr (VEC) {
    const float4 d =
        *reinterpret_cast<const float4 *>(static_cast<const float *>(g.tail.residual) + at);
    res[0] = d.x;
    res[1] = d.y;
    res[2] = d.z;
    res[3] = d.w;
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      res[v] = v < left ? tail_residual_as<BF16>(g.tail.residual, at + v) : 0.f;
  }
}

template <bool BF16, bool VEC>
__device__ inline void store_dense(const I8Args &g, int64_t at, int left, const float (&p)[4]) {
  float *y = static_cast<float *>(g.y);
  if constexpr (VEC && BF16) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.y) + at) =
        make_uint2(bf16_pair(p[0], p[1]), bf16_pair(p[2], p[3]));
  } else if constexpr (VEC) {
    *reinterpret_cast<float4 *>(y + at) = make_float4(p[0], p[1], p[2], p[3]);
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v < left) tail_store_as<BF16>(y, at + v, p[v]);
  }
}

// A wave's 16 x 16 block of a dense output: row lane % 16 of `rows` valid ones,
// columns n0 + 4 (lane / 16) ....
template <bool BF16, bool VEC>
__device__ inline void store_block(const I8Args &g, intx4 acc, int rows, int64_t n0, float sx,
                                   int lane) {
#pragma clang fp contract(off)
  const int r = lane % 16;
  const int64_t n = n0 + 4 * (lane / 16);
  const int left = g.n - n < 4 ? static_cast<int>(g.n - n) : 4;
  if (r >= rows || left <= 0) return;
  const bool has_bias = g.tail.bias != nullptr;
  const bool has_res = g.tail.residual != nullptr;
  float sw[4], bias[4], res[4], p[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    sw[v] = v < left ? g.ws[n + v] : 0.f;
    bias[v] = has_bias && v < left ? g.tail.bias[n + v] : 0.f;
  }
  if (has_res) load_residual<BF16, VEC>(g, r * g.n + n, left, res);
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    p[v] = (static_cast<float>(acc[v]) * sx) * sw[v];
    if (has_bias) p[v] += bias[v];
    if (has_res) p[v] += res[v];
  }
  store_dense<BF16, VEC>(g, r * g.n + n, left, p);
}

__device__ inline void store_any(const I8Args &g, intx4 acc, int rows, int64_t n0, float sx,
                                 int lane) {
  if (g.vec) {
    if (g.tail.bf16)
      store_block<true, true>(g, acc, rows, n0, sx, lane);
    else
      store_block<false, true>(g, acc, rows, n0, sx, lane);
  } else {
    if (g.tail.bf16)
      store_block<true, false>(g, acc, rows, n0, sx, lane);
    else
      store_block<false, false>(g, acc, rows, n0, sx, lane);
  }
}

// Scales of columns n .. n + 3 (row w0 + n of the stacked weights).
__device__ inline void load_sw(const I8Args &g, int64_t w0, int64_t n, float (&sw)[4]) {
  if (n + 4 <= g.n && (w0 + n) % 4 == 0) {
    const float4 d = *reinterpret_cast<const float4 *>(g.ws + w0 + n);
    sw[0] = d.x;
    sw[1] = d.y;
    sw[2] = d.z;
    sw[3] = d.w;
    return;
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) sw[v] = n + v < g.n ? g.ws[w0 + n + v] : 0.f;
}

// ---- few rows ---------------------------------------------------------------
// Up to 16 rows: the weights are read once, straight into registers, and the
// product is bound by that stream.  A workgroup of KW waves takes 16 columns; wave
// w takes the 64-k steps [w * per, (w + 1) * per) of them, B at a time, all loads
// of a batch issued before its first product.  The waves' int32 sums meet in LDS
// (exact in any order).  16 tokens on 128 experts of 1856 x 2688 (median and range of
// 60 calls): up 72 us (65 to 80), down 63 (61 to 67), for 357 MB each: 5.0 and 5.7
// TB/s.
template <int MODE, int KW, int B>
__global__ __launch_bounds__(64 * KW) void i8_skinny_kernel(I8Args g) {
  static_assert(KW > 1, "the waves share k");
  __shared__ intx4 red[KW - 1][64];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % 16;
  const int grp = lane / 16;

  int64_t n0, m0 = 0, w0 = 0;
  int rows;
  if constexpr (MODE == kI8Dense) {
    n0 = static_cast<int64_t>(blockIdx.x) * 16;
    rows = static_cast<int>(g.m);
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
    n0 = static_cast<int64_t>(j) * 16;
    m0 = t.row0;
    rows = t.rows;
    w0 = static_cast<int64_t>(t.expert) * g.n;
  }

  const int64_t nr = n0 + r < g.n ? n0 + r : g.n - 1;  // past n: read n - 1
  const int8_t *wp = g.wq + (w0 + nr) * g.kp + 16 * grp;
  const int64_t mr = m0 + (r < rows ? r : 0);          // past the rows: the first
  const int64_t src = MODE == kI8Up ? g.perm[mr] / g.topk : mr;
  const int8_t *xp = g.xq + src * g.kp + 16 * grp;
  intx4 acc = {0, 0, 0, 0};

  const int steps = g.kp / kI8Step;
  const int per = (steps + KW - 1) / KW;
  const int s0 = wave * per;
  const int s1 = s0 + per < steps ? s0 + per : steps;
  for (int s = s0; s < s1; s += B) {
    intx4 a[B], b[B];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      // steps past the wave's end reload its last one and are not multiplied
      const int64_t k0 = static_cast<int64_t>(s + u < s1 ? s + u : s1 - 1) * kI8Step;
      a[u] = *reinterpret_cast<const intx4 *>(wp + k0);
      b[u] = *reinterpret_cast<const intx4 *>(xp + k0);
    }
#pragma unroll
    for (int u = 0; u < B; ++u)
      if (s + u < s1) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u], b[u], acc, 0, 0, 0);
  }
  if (wave > 0) red[wave - 1][lane] = acc;
  __syncthreads();
  if (wave > 0) return;  // wave 0 adds the others' sums and stores
#pragma unroll
  for (int w = 0; w < KW - 1; ++w) acc += red[w][lane];
  const float sx = g.xs[src];
  if constexpr (MODE == kI8Dense) {
    store_any(g, acc, rows, n0, sx, lane);
  } else if (r < rows) {
    float sw[4];
    load_sw(g, w0, n0 + 4 * grp, sw);
    store_moe<MODE>(g, acc, m0 + r, n0 + 4 * grp, sx, sw);
  }
}

// ---- single tokens ------------------------------------------------------------
// One row: the product needs less time than the launch that would quantize its
// input, so each wave does that for itself.  It requests the whole row (a few
// KB, from the caches after the first wave), its own share of it and then its
// weights, finds the row's largest magnitude and turns its share of k into
// codes, in its own LDS and without a barrier, while the weights are on their
// way (loads return in order, so the row's have to come first).  The product
// is that of the register stream above, the row's codes broadcast to all
// sixteen rows of the operand.
//
// m = 1, 2688 x 8192: 7.4 us against 8.6 for quantizer and product one after the
// other, and one launch for the host instead of two (8.0 against 12.7 us a call);
// 8192 x 2688 7.7 against 10.8.  From two rows on the wave's own quantization costs
// more than it saves (10.2 against 9.1 us).

constexpr int kDirectSteps = 16;  // steps of 64 k per wave

// A wave's row, V pieces of 8 values per lane: request(), then other loads, then
// finish(), which leaves the codes of steps [s0, s1) in `codes` and returns what the
// row's maximum says.
template <int V>
struct DirectRow {
  uint4 all[V], own[2];
  int n_vec, v0, v1;

  __device__ void request(const uint16_t *row, int k, int s0, int s1, int lane) {
    const uint4 *xr = reinterpret_cast<const uint4 *>(row);
    n_vec = k / 8;
    v0 = 8 * s0;
    v1 = 8 * s1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = lane + 64 * i;
      all[i] = xr[at < n_vec ? at : n_vec - 1];  // a repeat changes no maximum
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = v0 + lane + 64 * i;
      own[i] = xr[at < n_vec ? at : n_vec - 1];
    }
  }

  __device__ RowScale finish(uint8_t *codes, int lane) const {
    ushortx2 tops = top_of(all[0]);
#pragma unroll
    for (int i = 1; i < V; ++i) tops = __builtin_elementwise_max(tops, top_of(all[i]));
    uint32_t top = top_of(tops);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const uint32_t o = __shfl_xor(top, s);
      top = top > o ? top : o;
    }
    const RowScale rs(top);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = v0 + lane + 64 * i;
      if (at < v1)
        *reinterpret_cast<uint2 *>(codes + 8 * (at - v0)) =
            rs.live && at < n_vec ? codes_of(own[i], rs) : make_uint2(0u, 0u);
    }
    wave_lds_fence();
    return rs;
  }
};

struct I8Direct {
  const uint16_t *x;   // bf16 rows of k: the input (dense, up) or the hidden rows (down)
  int32_t k;
  const int32_t *ids;  // MoE: [t][topk]
  const float *gates;
  int32_t n_experts;
};

// The sum over steps [s0, s1) of one wave: weights already in a[] for the first
// B steps.
template <int B>
__device__ inline void direct_load(intx4 (&a)[B], const int8_t *wp, int s, int s1) {
#pragma unroll
  for (int u = 0; u < B; ++u) {
    const int at = s + u < s1 ? s + u : (s1 > 0 ? s1 - 1 : 0);
    a[u] = *reinterpret_cast<const intx4 *>(wp + static_cast<int64_t>(at) * kI8Step);
  }
}

template <int B>
__device__ inline intx4 direct_sum(intx4 (&a)[B], const int8_t *wp, const uint8_t *codes, int s0,
                                   int s1) {
  intx4 acc = {0, 0, 0, 0};
  for (int s = s0; s < s1; s += B) {
    if (s > s0) direct_load<B>(a, wp, s, s1);
#pragma unroll
    for (int u = 0; u < B; ++u)
      if (s + u < s1)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            a[u], *reinterpret_cast<const intx4 *>(codes + (s + u - s0) * kI8Step), acc, 0, 0, 0);
  }
  return acc;
}

// Dense: grid (column blocks of 16); up: grid (column blocks, pairs), the row
// of a pair is its token's.
template <int MODE, int KW, int B, int V>
__global__ __launch_bounds__(64 * KW) void i8_direct_kernel(I8Args g, I8Direct d) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[KW][kDirectSteps * kI8Step];
  __shared__ intx4 red[KW - 1][64];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % 16;
  const int grp = lane / 16;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int steps = g.kp / kI8Step;
  const int per = (steps + KW - 1) / KW;
  const int s0 = wave * per < steps ? wave * per : steps;
  const int s1 = s0 + per < steps ? s0 + per : steps;
  DirectRow<V> row;
  row.request(d.x + (MODE == kI8Up ? static_cast<int64_t>(blockIdx.y / g.topk) * d.k : 0), d.k,
              s0, s1, lane);
  int64_t w0 = 0;
  if constexpr (MODE == kI8Up) {
    const int e = d.ids[blockIdx.y];
    if (e < 0 || e >= d.n_experts) return;
    w0 = static_cast<int64_t>(e) * g.n;
  }
  const int64_t nr = n0 + r < g.n ? n0 + r : g.n - 1;
  const int8_t *wp = g.wq + (w0 + nr) * g.kp + 16 * grp;
  intx4 a[B];
  direct_load<B>(a, wp, s0, s1);
  const RowScale rs = row.finish(codes[wave], lane);
  intx4 acc = direct_sum<B>(a, wp, codes[wave] + 16 * grp, s0, s1);
  if (wave > 0) red[wave - 1][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 0; w < KW - 1; ++w) acc += red[w][lane];
  if constexpr (MODE == kI8Dense) {
    store_any(g, acc, 1, n0, rs.scale, lane);
  } else if (r == 0) {
    float sw[4];
    load_sw(g, w0, n0 + 4 * grp, sw);
    store_moe<MODE>(g, acc, blockIdx.y, n0 + 4 * grp, rs.scale, sw);
  }
}

// The down product of single tokens with the weighted sum over their slots:
// grid (column blocks of 16, tokens); waves 2 j and 2 j + 1 take the halves of
// k of slot j.  Hidden rows are in pair order.  The sum runs in slot order with
// the combine kernel's fused multiply-adds, so the bits are those of the
// batched layer.
constexpr int kDirectSlots = 8;

template <int B, int V>
__global__ __launch_bounds__(128 * kDirectSlots) void i8_direct_down_kernel(I8Args g, I8Direct d) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[2 * kDirectSlots][kDirectSteps * kI8Step];
  __shared__ intx4 sums[2 * kDirectSlots][4];
  __shared__ float scales[kDirectSlots];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % 16;
  const int grp = lane / 16;
  const int slot = wave / 2;
  const int64_t tok = blockIdx.y;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int steps = g.kp / kI8Step;
  const int per = (steps + 1) / 2;
  const int s0 = wave % 2 * per;
  const int s1 = s0 + per < steps ? s0 + per : steps;
  DirectRow<V> row;
  row.request(d.x + (tok * g.topk + slot) * d.k, d.k, s0, s1, lane);
  const int e = d.ids[tok * g.topk + slot];
  if (e >= 0 && e < d.n_experts) {
    const int64_t nr = n0 + r < g.n ? n0 + r : g.n - 1;
    const int8_t *wp = g.wq + (e * g.n + nr) * g.kp + 16 * grp;
    intx4 a[B];
    direct_load<B>(a, wp, s0, s1);
    const RowScale rs = row.finish(codes[wave], lane);
    const intx4 acc = direct_sum<B>(a, wp, codes[wave] + 16 * grp, s0, s1);
    if (r == 0) sums[wave][grp] = acc;
    if (lane == 0) scales[slot] = rs.scale;  // the same from both halves
  }
  __syncthreads();
  const int64_t n = n0 + tid;
  if (tid >= 16 || n >= g.n) return;
  float out = 0.f;
  for (int j = 0; j < g.topk; ++j) {
    const int ej = d.ids[tok * g.topk + j];
    if (ej < 0 || ej >= d.n_experts) continue;
    const int acc = sums[2 * j][tid / 4][tid % 4] + sums[2 * j + 1][tid / 4][tid % 4];
    const float o = (static_cast<float>(acc) * scales[j]) * g.ws[ej * g.n + n];
    out = __builtin_fmaf(d.gates[tok * g.topk + j], o, out);
  }
  static_cast<float *>(g.y)[tok * g.n + n] = out;
}

// A wave's MS x NS sub-tiles to memory through LDS.  Straight from the product's
// layout a store instruction would write 16 rows x 64 bytes (32 for bf16),
// half a cache line each; instead 16 rows at a time go to a wave's own LDS
// buffer (two in turn, so that a group's reads are behind the next one's fence
// before they are overwritten; rows 16 bytes longer than their data, so that
// neither the writes nor the reads share banks) and come back as whole row segments
// of 16 * NS outputs.  Stores are non-temporal: nothing reads the output before
// the operands that it would push out of the caches are needed (4096 x 2688 x
// 8192: 107 -> 96 us, the up product of 1024 tokens on 128 experts 134.5 -> 124).
// Residual values of later rows are loaded before the stores of these, since a
// wait for a load is also one for every store before it.
template <int NS>
constexpr int tile_store_bytes() {
  return 2 * 16 * (16 * NS + 4) * 4;
}

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t uintx2 __attribute__((ext_vector_type(2)));

template <int MODE, int MS, int NS, int WM, bool BF16, bool VEC>
__device__ inline void store_rows(const I8Args &g, const intx4 (&acc)[MS][NS], uint8_t *lds,
                                  int64_t m0, int rows, int64_t n0, const float (&sx)[MS],
                                  const float (&sw)[NS][4], int lane) {
#pragma clang fp contract(off)
  constexpr int kCols = 16 * NS;
  constexpr int kStride = kCols + 4;
  constexpr int E = VEC ? 4 : 1;             // outputs per lane and access
  constexpr int kGroups = 16 * kCols / (64 * E);
  const int r = lane % 16;
  const int grp = lane / 16;
  const bool has_bias = MODE == kI8Dense && g.tail.bias != nullptr;
  const bool has_res = MODE == kI8Dense && g.tail.residual != nullptr;
  // Residual values as they lie in memory, loaded several groups of 16 rows
  // ahead of their use, since each is a trip to HBM: as many as 40 registers
  // hold (the operands' are free by now; with more the largest tile spills).
  // One group ahead, the bf16 residual of 1024 x 2688 x 4096 made the product 24.0
  // us, so 18.9; that of 4096 x 8192 x 2688 89.5 and 82.
  using Raw = std::conditional_t<VEC, std::conditional_t<BF16, uintx2, floatx4>, float>;
  constexpr int kWords = kGroups * static_cast<int>(sizeof(Raw)) / 4;
  constexpr int kAhead = 40 / kWords < MS ? 40 / kWords : MS;
  static_assert(kAhead >= 1, "a group of rows fits");
  Raw res[MODE == kI8Dense ? kAhead : 1][kGroups];
  auto load_res = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int f = 64 * E * q + E * lane;
      const int row = 16 * WM * i + f / kCols;
      const int64_t n = n0 + f % kCols;
      Raw &d = res[i % kAhead][q];
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
  auto res_at = [&](int i, int q, int v) __attribute__((always_inline)) {
    const Raw &d = res[i % kAhead][q];
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
  if constexpr (MODE == kI8Dense) {
    if (has_res) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load_res(i);
    }
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int64_t n = n0 + (64 * E * q + E * lane) % kCols;
#pragma unroll
      for (int v = 0; v < E; ++v) bias[q][v] = has_bias && n < g.n ? g.tail.bias[n + v] : 0.f;
    }
  }
  if constexpr (MODE == kI8Up) {
    // the row image is bf16: 2 * kStride bytes per row, eight outputs per lane
    bool tame = true;
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) tame = tame && tame_scale(sw[j][v]);
#pragma unroll
    for (int i = 0; i < MS; ++i) tame = tame && tame_scale(sx[i]);
    tame = __builtin_amdgcn_ballot_w64(!tame) == 0;
    constexpr int kRowBytes = 2 * kCols + 16;
    constexpr int kReads = 16 * kCols / 512;  // of 64 lanes x 8 outputs
    static_assert(kReads >= 1, "two or more column sub-tiles");
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      if (16 * WM * i >= rows) break;
      uint8_t *buf = lds + (i % 2) * (16 * kRowBytes);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        *reinterpret_cast<uint2 *>(buf + r * kRowBytes + 32 * j + 8 * grp) =
            hidden_quad(acc[i][j], sx[i], sw[j], tame);
      wave_lds_fence();
#pragma unroll
      for (int q = 0; q < kReads; ++q) {
        const int f = 512 * q + 8 * lane;
        const intx4 d = *reinterpret_cast<const intx4 *>(buf + (f / kCols) * kRowBytes +
                                                         2 * (f % kCols));
        const int row = 16 * WM * i + f / kCols;
        const int64_t n = n0 + f % kCols;
        if (row < rows && n < g.n)  // n % 32 == 0 columns in all
          __builtin_nontemporal_store(
              d, reinterpret_cast<intx4 *>(static_cast<uint16_t *>(g.y) + (m0 + row) * g.n + n));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    if (MODE != kI8Dense && 16 * WM * i >= rows) break;
    float *buf = reinterpret_cast<float *>(lds) + (i % 2) * (16 * kStride);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      floatx4 p;
#pragma unroll
      for (int v = 0; v < 4; ++v) p[v] = (static_cast<float>(acc[i][j][v]) * sx[i]) * sw[j][v];
      *reinterpret_cast<floatx4 *>(buf + r * kStride + 16 * j + 4 * grp) = p;
    }
    wave_lds_fence();
    float val[kGroups][E];
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int f = 64 * E * q + E * lane;
      const float *src = buf + (f / kCols) * kStride + f % kCols;
      if constexpr (VEC) {
        const floatx4 d = *reinterpret_cast<const floatx4 *>(src);
#pragma unroll
        for (int v = 0; v < 4; ++v) val[q][v] = d[v];
      } else {
        val[q][0] = *src;
      }
      if constexpr (MODE == kI8Dense) {
#pragma unroll
        for (int v = 0; v < E; ++v) {
          if (has_bias) val[q][v] += bias[q][v];
          if (has_res) val[q][v] += res_at(i, q, v);
        }
      }
    }
    if constexpr (MODE == kI8Dense) {
      if (has_res && i + kAhead < MS) load_res(i + kAhead);
    }
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int f = 64 * E * q + E * lane;
      const int row = 16 * WM * i + f / kCols;
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

// ---- many rows --------------------------------------------------------------
// TM x TN output tile per workgroup of WM x WN waves, each wave MS x NS
// 16 x 16 products.  KB bytes (64 or 128) of k of the tile's TM activation
// rows and TN weight rows go to LDS by LDS-direct buffer loads into S stages,
// S - 1 steps ahead, with exact load-count waits and one barrier per step.
//
// LDS image of a stage: 1 KB pieces of 1024 / KB rows; a row's 16-byte slots
// are stored at slot ^ key(row).  A 16-byte read takes the wave in phases of 16
// lanes, which are not consecutive (0-3, 12-15, 20-23, 24-27 make the first):
// of lane r + 16 g reading row r, a phase holds rows 0-3 and 12-15 at one slot
// and 4-11 at another.  key = (row / 2) % 8 for 128-byte rows and 0, 2, 3, 1 for
// row / 4 = 0 .. 3 of 64-byte rows put the 16 lanes of every phase on all 64
// banks.  Rows past the tile's end read zeros (dense; the buffer range ends
// there) or the tile's first row (MoE) and are not stored.
//
// Bound at many rows by MFMA at the clock that the power leaves.  4096 x 2688 x 8192
// (256 x 256 tiles): 95 to 97 us captured (runs from 92 to 124), 1.9 POP/s; in a run
// with counters (96.7 us) MFMA is busy in 53 % of the compute units' cycles, at 1.7
// GHz.  4096 x 8192 x 2688: 90 us (85 to 117), MFMA busy 55 %.  One call after
// another under a profiler: 112 (92 to 117) and 105 (90 to 119).  MoE, 128 experts
// of 1856 x 2688, up / down, medians and ranges of 60 calls: 1024 tokens, popular
// experts, 146 (142 to 156) / 165 (161 to 174) us, 5.4 and 5.3 TB/s; 4096 tokens 197
// (188 to 240) / 230 (221 to 259), of which the loop is 150 / 180 and the rest the
// hidden values and stores of one workgroup per compute unit; MFMA busy 38 / 30 %.
template <int MODE, int WM, int WN, int MS, int NS, int KB, int S, int OCC, bool PP>
__global__ __launch_bounds__(64 * WM * WN, OCC) void i8_tile_kernel(I8Args g) {
  constexpr int W = WM * WN;
  constexpr int TM = 16 * MS * WM;
  constexpr int TN = 16 * NS * WN;
  constexpr int kPieceRows = 1024 / KB;
  constexpr int kSlots = KB / 16;
  constexpr int kAPieces = TM / kPieceRows;
  constexpr int kWPieces = TN / kPieceRows;
  static_assert(kAPieces % W == 0 && kWPieces % W == 0, "every wave loads the same share");
  constexpr int kALoads = kAPieces / W;
  constexpr int kWLoads = kWPieces / W;
  constexpr int kLoads = kALoads + kWLoads;
  constexpr int kStage = (TM + TN) * KB;
  constexpr int kWBase = TM * KB;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * kStage];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % 16;
  const int grp = lane / 16;
  const int wm = wave / WN;
  const int wn = wave % WN;
  const int kp = g.kp;

  int64_t m_base, n_base, w0 = 0;
  int rows;  // valid rows of the tile
  if constexpr (MODE == kI8Dense) {
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
    // XCD x (workgroup id % 8) takes tiles x, x + 8, ... with all their column
    // blocks in a row: the tile's rows then stay in one L2
    const int q = static_cast<int>(blockIdx.x) / 8;
    const int i = q / g.tiles_n * 8 + static_cast<int>(blockIdx.x) % 8;
    if (i >= *g.n_tiles) return;
    const MoETile t = g.tiles[i];
    const int j = q % g.tiles_n;
    m_base = t.row0;
    rows = t.rows;
    n_base = static_cast<int64_t>(j) * TN;
    w0 = static_cast<int64_t>(t.expert) * g.n;
  }
  const int cols = g.n - n_base < TN ? static_cast<int>(g.n - n_base) : TN;

  // A piece's lane l fills row l / kSlots at stored slot l % kSlots; the key of
  // a row depends on row % 16, so the pieces of 8 rows alternate between two.
  const int prow = lane / kSlots;
  auto key_of = [](int row) __attribute__((always_inline)) {
    if constexpr (KB == 64) return ((row >> 1) & 2) ^ ((row >> 3) & 1) * 3;
    return (row >> 1) & 7;
  };
  auto slot_of = [&](int row)
      __attribute__((always_inline)) { return (lane % kSlots) ^ key_of(row); };
  const int64_t a_base = MODE == kI8Dense ? m_base : 0;
  const int64_t a_rows = MODE == kI8Dense ? rows : g.a_rows;
  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t *>(g.xq + a_base * kp), static_cast<short>(0),
      static_cast<int>(a_rows * kp), kI8BufferFlags);
  const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t *>(g.wq + (w0 + n_base) * kp), static_cast<short>(0), cols * kp,
      kI8BufferFlags);
  static_assert(kALoads <= 8 && kWLoads <= 8, "offsets held per load");
  uint32_t a_voff[8];  // (a bound that depends on the template made the host pass drop launch stubs)
#pragma unroll
  for (int i = 0; i < kALoads; ++i) {
    const int row = kPieceRows * (kALoads * wave + i) + prow;
    int64_t from = row;
    if constexpr (MODE != kI8Dense) {
      const int64_t b = m_base + (row < rows ? row : 0);
      from = MODE == kI8Up ? g.perm[b] / g.topk : b;
    }
    a_voff[i] = static_cast<uint32_t>(from * kp + 16 * slot_of(row));
  }
  uint32_t w_voff[8];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) {
    const int row = kPieceRows * (kWLoads * wave + i) + prow;
    w_voff[i] = static_cast<uint32_t>(row * kp + 16 * slot_of(row));
  }

  // kp is a multiple of 64; with 128-byte rows the second half of a last odd
  // step is read (the next row's start, or zeros) but not multiplied
  const int halves = kp / 64;
  const int steps = KB == 64 ? halves : (halves + 1) / 2;
  auto issue = [&](int c, uint8_t *st) __attribute__((always_inline)) {
    const int k0 = (c < steps ? c : steps - 1) * KB;  // padding steps reload the last one
#pragma unroll
    for (int i = 0; i < kALoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          a_rsrc, (lds_void *)(st + (kALoads * wave + i) * 1024), 16, a_voff[i], k0, 0, 0);
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          w_rsrc, (lds_void *)(st + kWBase + (kWLoads * wave + i) * 1024), 16, w_voff[i], k0, 0,
          0);
  };

  // The scales that the epilogue applies, fetched before the k loop: behind it
  // every wave of the tile would stand for them (5 us of the up product's 197 at
  // 4096 tokens).
  const int64_t m0 = m_base + 16 * wm;
  const int64_t n0 = n_base + wn * (16 * NS);
  float sx[MS], sw[NS][4];
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    const int row = 16 * (WM * i + wm) + r;
    const int64_t b = m_base + (row < rows ? row : 0);
    sx[i] = g.xs[MODE == kI8Up ? g.perm[b] / g.topk : b];
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) load_sw(g, w0, n0 + 16 * j + 4 * grp, sw[j]);

  intx4 acc[MS][NS];
#pragma unroll
  for (int i = 0; i < MS; ++i)
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[i][j] = intx4{0, 0, 0, 0};

  // fragment addresses: row 16 * x + r, whose key depends on r alone
  const int key = key_of(r);
  const int a_frag = (16 * wm + r) * KB;
  const int w_frag = kWBase + (wn * (16 * NS) + r) * KB;
  // A wave's sub-tile i holds rows 16 (WM i + wm) ..., so that the rows of a
  // part-filled tile are spread over the waves; sub-tiles past the rows are
  // skipped, two at a time.
  const int live = MODE == kI8Dense ? MS : (rows - 16 * wm + 16 * WM - 1) / (16 * WM);
  auto half = [&](const uint8_t *st, int h) __attribute__((always_inline)) {
    const int slot = 16 * ((4 * h + grp) ^ key);
    intx4 wf[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j)
      wf[j] = *reinterpret_cast<const intx4 *>(st + w_frag + 16 * j * KB + slot);
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      if (MODE != kI8Dense && i % 2 == 0 && i >= live) break;
      const intx4 af = *reinterpret_cast<const intx4 *>(st + a_frag + 16 * WM * i * KB + slot);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[j], af, acc[i][j], 0, 0, 0);
    }
  };

  constexpr int kAhead = (S - 2) * kLoads;
  constexpr int kWait = 0x0F70 | (kAhead & 15) | ((kAhead >> 4) << 14);
  static_assert(kAhead < 64, "the wait counts up to 63 loads");
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(s, smem + s * kStage);
  if constexpr (PP) {
    static_assert(W == 8 && KB == 64, "two waves per SIMD, one product step per stage");
    const bool late = wave >= 4;
    intx4 wf[NS], af[MS];
    const int slot = 16 * (grp ^ key);
    auto phase_end = [&]() __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    __builtin_amdgcn_s_waitcnt(kWait);  // step 0
    phase_end();
    if (late) phase_end();
    for (int c = 0; c < steps; c += S) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (c + s < steps) {
          const uint8_t *st = smem + s * kStage;
#pragma unroll
          for (int j = 0; j < NS; ++j)
            wf[j] = *reinterpret_cast<const intx4 *>(st + w_frag + 16 * j * KB + slot);
#pragma unroll
          for (int i = 0; i < MS; ++i)
            af[i] = *reinterpret_cast<const intx4 *>(st + a_frag + 16 * WM * i * KB + slot);
          issue(c + s + S - 1, smem + ((s + S - 1) % S) * kStage);
          __builtin_amdgcn_s_waitcnt(kWait);   // step c + s + 1
          __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
          phase_end();
#pragma unroll
          for (int i = 0; i < MS; ++i) {
            if (MODE != kI8Dense && i % 2 == 0 && i >= live) break;
#pragma unroll
            for (int j = 0; j < NS; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[j], af[i], acc[i][j], 0, 0, 0);
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
        issue(c + s + S - 1, smem + ((s + S - 1) % S) * kStage);
        if (c + s < steps) {
          half(smem + s * kStage, 0);
          if (KB == 128 && 2 * (c + s) + 1 < halves) half(smem + s * kStage, 1);
        }
      }
    }
  }
  static_assert(W * tile_store_bytes<NS>() <= S * kStage, "the stages hold the store buffers");
  __builtin_amdgcn_s_waitcnt(0x0F70);  // the padding steps' loads
  __builtin_amdgcn_s_waitcnt(0xC07F);  // the last reads of the stages
  __syncthreads();                     // for every wave: the stages become store buffers

  uint8_t *lds = smem + wave * tile_store_bytes<NS>();
  rows -= 16 * wm;
  if constexpr (MODE != kI8Dense) {
    store_rows<MODE, MS, NS, WM, MODE == kI8Up, true>(g, acc, lds, m0, rows, n0, sx, sw, lane);
  } else if (g.vec) {
    if (g.tail.bf16)
      store_rows<MODE, MS, NS, WM, true, true>(g, acc, lds, m0, rows, n0, sx, sw, lane);
    else
      store_rows<MODE, MS, NS, WM, false, true>(g, acc, lds, m0, rows, n0, sx, sw, lane);
  } else {
    if (g.tail.bf16)
      store_rows<MODE, MS, NS, WM, true, false>(g, acc, lds, m0, rows, n0, sx, sw, lane);
    else
      store_rows<MODE, MS, NS, WM, false, false>(g, acc, lds, m0, rows, n0, sx, sw, lane);
  }
}

template <int MODE, int WM, int WN, int MS, int NS, int KB, int S, int OCC, bool PP = false>
hipError_t launch_tile(I8Args g, int64_t max_tiles, hipStream_t s) {
  constexpr int TM = 16 * MS * WM, TN = 16 * NS * WN;
  g.tiles_n = static_cast<int32_t>((g.n + TN - 1) / TN);
  int64_t grid;
  if (MODE == kI8Dense) {
    g.tiles_m = static_cast<int32_t>((g.m + TM - 1) / TM);
    grid = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  } else {
    grid = (max_tiles + 7) / 8 * 8 * g.tiles_n;
  }
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((i8_tile_kernel<MODE, WM, WN, MS, NS, KB, S, OCC, PP>),
                     dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), 0, s, g);
  return hipGetLastError();
}

template <int MODE, int KW, int B>
hipError_t launch_skinny_cfg(I8Args g, int64_t max_tiles, hipStream_t s) {
  g.tiles_n = static_cast<int32_t>((g.n + 15) / 16);
  const int64_t grid =
      MODE == kI8Dense ? g.tiles_n : max_tiles * ((g.tiles_n + 7) / 8 * 8);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((i8_skinny_kernel<MODE, KW, B>), dim3(static_cast<unsigned>(grid)),
                     dim3(64 * KW), 0, s, g);
  return hipGetLastError();
}

// The dense tile: the one with the least time per 128 bytes of k, from the
// number of tiles and what each kernel was measured to need.  `alone` is a
// step's time with one workgroup on a compute unit, `each` what every further
// one adds, `slots` how many fit; 256 compute units.  (us per step, from
// sweeps over m = 32 .. 4096 at (k, n) = (2688, 8192), (8192, 2688) and (1856,
// 2688); the order it gives was that of the measured times at all of them, to
// within 8 %.)
// Where each compute unit gets one of the two largest tiles they are within 5 %
// of each other, either way (192 rows / 256: 4099 x 2688 x 2690 38.9 / 40.8 us,
// 1025 x 2688 x 8192 30.4 / 32.2, 6100 x 1856 x 2000 30.8 / 29.6, 4096 x 8192 x
// 2688 83.4 / 81.3, with a bf16 residual 83.1 / 82.9).
int pick_tile(int64_t m, int64_t n) {
  struct Cost {
    int tm, tn, slots;
    double alone, each;
  };
  static constexpr Cost kCosts[] = {
      {32, 32, 4, 0.15, 0.115},  {32, 64, 3, 0.17, 0.17},  {64, 64, 3, 0.235, 0.19},
      {64, 128, 3, 0.51, 0.28},  {128, 128, 2, 0.59, 0.41}, {192, 256, 1, 1.30, 1.30},
      {256, 256, 1, 1.35, 1.35},
  };
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
        static_cast<double>(per_cu / c.slots) * step(c.slots) + step(per_cu % c.slots);
    if (i == 0 || cost < least) {
      best = i;
      least = cost;
    }
  }
  return best;
}

}  // namespace

int64_t int8_padded_k(int64_t k) { return (k + kI8Step - 1) / kI8Step * kI8Step; }

hipError_t launch_act_int8(const uint16_t *x, int64_t m, int64_t k, int8_t *codes, float *scales,
                           hipStream_t s) {
  if (m == 0 || k == 0) return hipSuccess;
  const int32_t k32 = static_cast<int32_t>(k);
  const int32_t kp = static_cast<int32_t>(int8_padded_k(k));
  // A wave per row needs no barrier, a workgroup per row has the shorter chain
  // (us, wave / workgroup: k = 1856: 1024 rows 4.3 / 3.4, 2048 5.0 / 5.1, 4096 7.1 /
  // 7.8, 24576 24 / 36; k = 2688: 4096 rows 10.0 / 8.9, 24576 37 / 42; k = 8192: 4096
  // rows 23 / 18).  Four pieces of a row per lane where they hold it, else eight
  // (24 / 28 and 40 / 37).
  if ((m >= 4096 && k <= 64 * 8 * 4) || (m >= 12288 && k <= 64 * 8 * 8)) {
    const int64_t groups = (m + 3) / 4;
    const dim3 grid(static_cast<unsigned>(groups < 65536 ? groups : 65536));
    if (k <= 64 * 8 * 4)
      hipLaunchKernelGGL((act_int8_kernel<64, 4>), grid, dim3(kQThreads), 0, s, x, m, k32, kp,
                         codes, scales);
    else
      hipLaunchKernelGGL((act_int8_kernel<64, 8>), grid, dim3(kQThreads), 0, s, x, m, k32, kp,
                         codes, scales);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(m < 65536 ? m : 65536));
  if (k <= 256 * 8 * 2)
    hipLaunchKernelGGL((act_int8_kernel<256, 2>), grid, dim3(kQThreads), 0, s, x, m, k32, kp,
                       codes, scales);
  else
    hipLaunchKernelGGL((act_int8_kernel<256, 4>), grid, dim3(kQThreads), 0, s, x, m, k32, kp,
                       codes, scales);
  return hipGetLastError();
}

// In one launch where one workgroup buckets and a row stays in a wave's
// registers (6.2 to 8.0 us for 16 tokens x 2688, 10.2 to 13.8 for 1024; in two
// launches 4.4 + 6.9 and 6.5 + 10.5), in two or four otherwise.
hipError_t launch_moe_int8_prepare(const uint16_t *x, int64_t t, int64_t k, const int32_t *ids,
                                   int32_t topk, int32_t n_experts, int32_t *counts,
                                   int32_t *offsets, int32_t *perm, int32_t *inv, MoETile *tiles,
                                   int32_t *n_tiles, int32_t tile_rows, int8_t *xq, float *xs,
                                   hipStream_t s) {
  const int64_t pairs = t * topk;
  if (pairs > kRouteOneGroupPairs || k > 64 * 8 * 8) {
    const hipError_t e = launch_act_int8(x, t, k, xq, xs, s);
    if (e != hipSuccess) return e;
    return launch_route(ids, pairs, topk, n_experts, counts, offsets, perm, inv, tiles, n_tiles,
                        tile_rows, nullptr, s);
  }
  if (n_experts < 1 || n_experts > kMaxExperts || pairs < 0) return hipErrorInvalidValue;
  const int64_t groups = 1 + (t + kRouteWaves - 1) / kRouteWaves;
  hipLaunchKernelGGL(i8_route_act_kernel, dim3(static_cast<unsigned>(groups)),
                     dim3(kRouteThreads), 0, s, ids, pairs, n_experts, counts, offsets, perm, inv,
                     tiles, n_tiles, tile_rows, x, t, static_cast<int32_t>(k),
                     static_cast<int32_t>(int8_padded_k(k)), xq, xs);
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

namespace {

int direct_steps(int64_t k, int waves) {
  const int64_t steps = int8_padded_k(k) / kI8Step;
  return static_cast<int>((steps + waves - 1) / waves);
}

// Pieces of 8 values that a lane holds of the longest row whose steps `waves` share.
constexpr int direct_vecs(int waves) { return waves * kDirectSteps * kI8Step / (64 * 8); }

template <int MODE, int KW, int B>
hipError_t launch_direct(const I8Args &g, const I8Direct &d, dim3 grid, hipStream_t s) {
  if (d.k <= 64 * 8 * 6)
    hipLaunchKernelGGL((i8_direct_kernel<MODE, KW, B, 6>), grid, dim3(64 * KW), 0, s, g, d);
  else
    hipLaunchKernelGGL((i8_direct_kernel<MODE, KW, B, direct_vecs(KW)>), grid, dim3(64 * KW), 0, s,
                       g, d);
  return hipGetLastError();
}

}  // namespace

bool int8_direct_fits(int64_t m, int64_t k) {
  return m == 1 && direct_steps(k, 8) <= kDirectSteps;
}

hipError_t launch_linear_int8_direct(const uint16_t *x, int64_t m, int64_t k, const int8_t *wq,
                                     const float *ws, int64_t n, const Tail &tail, void *y,
                                     hipStream_t s) {
  if (!int8_direct_fits(m, k)) return hipErrorInvalidValue;
  I8Args g{};
  g.wq = wq;
  g.ws = ws;
  g.y = y;
  g.tail = tail;
  g.m = m;
  g.n = n;
  g.kp = static_cast<int32_t>(int8_padded_k(k));
  const size_t quad = tail.bf16 ? 8 : 16;
  g.vec = n % 4 == 0 && reinterpret_cast<uintptr_t>(y) % quad == 0 &&
          reinterpret_cast<uintptr_t>(tail.residual) % quad == 0;
  I8Direct d{};
  d.x = x;
  d.k = static_cast<int32_t>(k);
  const dim3 grid(static_cast<unsigned>((n + 15) / 16));
  if (direct_steps(k, 8) <= 6) return launch_direct<kI8Dense, 8, 6>(g, d, grid, s);
  return launch_direct<kI8Dense, 8, 8>(g, d, grid, s);
}

// Up to 12 pairs (two tokens of six slots), and the row and step limits of the
// kernels.  128 experts of 1856 x 2688, top-6: one token 24 us against 31 for
// the batched steps, two 37 against 42, four 65 against 62 (the batched steps
// read an expert that two tokens share once).
bool int8_moe_direct_fits(int64_t t, int32_t topk, int64_t n1, int64_t k) {
  return t * topk <= 12 && topk <= kDirectSlots && direct_steps(k, 4) <= kDirectSteps &&
         direct_steps(n1, 2) <= kDirectSteps;
}

hipError_t launch_moe_int8_direct(const uint16_t *x, int64_t t, int64_t k, const int32_t *ids,
                                  const float *gates, int32_t topk, int32_t n_experts,
                                  const int8_t *w1, const float *s1, int64_t n1, const int8_t *w2,
                                  const float *s2, uint16_t *h, float *out, hipStream_t s) {
  if (!int8_moe_direct_fits(t, topk, n1, k)) return hipErrorInvalidValue;
  I8Args g{};
  g.wq = w1;
  g.ws = s1;
  g.y = h;
  g.n = n1;
  g.kp = static_cast<int32_t>(int8_padded_k(k));
  g.topk = topk;
  I8Direct d{};
  d.x = x;
  d.k = static_cast<int32_t>(k);
  d.ids = ids;
  d.gates = gates;
  d.n_experts = n_experts;
  const dim3 grid1(static_cast<unsigned>((n1 + 15) / 16), static_cast<unsigned>(t * topk));
  const hipError_t e = direct_steps(k, 4) <= 8 ? launch_direct<kI8Up, 4, 8>(g, d, grid1, s)
                                               : launch_direct<kI8Up, 4, 11>(g, d, grid1, s);
  if (e != hipSuccess) return e;
  g.wq = w2;
  g.ws = s2;
  g.y = out;
  g.n = k;
  g.kp = static_cast<int32_t>(int8_padded_k(n1));
  d.x = h;
  d.k = static_cast<int32_t>(n1);
  const dim3 grid2(static_cast<unsigned>((k + 15) / 16), static_cast<unsigned>(t));
  hipLaunchKernelGGL((i8_direct_down_kernel<kDirectSteps, direct_vecs(2)>), grid2,
                     dim3(static_cast<unsigned>(128 * topk)), 0, s, g, d);
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
  g.kp = static_cast<int32_t>(int8_padded_k(k));
  const size_t quad = tail.bf16 ? 8 : 16;
  g.vec = n % 4 == 0 && reinterpret_cast<uintptr_t>(y) % quad == 0 &&
          reinterpret_cast<uintptr_t>(tail.residual) % quad == 0;
  const int32_t halves = g.kp / kI8Step;
  // Up to 16 rows and 4096 columns the workgroups of the tile kernel are too
  // few to pull the weights in, and the register stream, which splits k over
  // 8 waves, is ahead: 16 x 1856 x 2688 3.7 us against 4.2, 16 x 2688 x 1856
  // 4.5 against 5.2, 16 x 8192 x 2688 9.7 against 10.2; at 4096 columns they
  // meet (6.8 against 6.6), and at 8192 the tiles win (7.5 against 6.4 us,
  // k = 2688).  A wave takes its steps in batches of 6 or, from 7 on, of 8
  // (k = 8192, n = 2688: 10.4 us in sixes, 9.7 in eights; k = 2688, n = 8192
  // the other way round, 7.4 and 8.9).
  if (m <= 16 && n <= 4096) {
    if (halves <= 8 * 6) return launch_skinny_cfg<kI8Dense, 8, 6>(g, 0, s);
    return launch_skinny_cfg<kI8Dense, 8, 8>(g, 0, s);
  }
  switch (pick_tile(m, n)) {
    case 0: return launch_tile<kI8Dense, 2, 2, 1, 1, 128, 5, 2>(g, 0, s);
    case 1: return launch_tile<kI8Dense, 2, 2, 1, 2, 128, 4, 2>(g, 0, s);
    case 2: return launch_tile<kI8Dense, 2, 2, 2, 2, 128, 3, 2>(g, 0, s);
    case 3: return launch_tile<kI8Dense, 2, 2, 2, 4, 128, 2, 2>(g, 0, s);
    case 4: return launch_tile<kI8Dense, 2, 2, 4, 4, 128, 2, 2>(g, 0, s);
    case 5: return launch_tile<kI8Dense, 2, 4, 6, 4, 128, 2, 2>(g, 0, s);
    default: return launch_tile<kI8Dense, 2, 4, 8, 4, 64, 4, 2, true>(g, 0, s);
  }
}

// Rows per tile by the average number of rows per expert, from sweeps of the
// two products over 128 experts of 1856 x 2688 (up + down, us; uniform
// routing / Zipf): 1.5 rows 16-row tiles 176 / 119, 64-row tiles 183 / 125; 2.25
// rows 207 / 161 and 206 / 153; 3 rows 226 / 171 and 219 / 155; 24 rows 64-row
// 252 / 275, 128-row 256 / 265; 33 rows 260 / 296 and 261 / 279; 96 rows
// 128-row 296 / 375, 256-row 330 / 386; 136 rows 436 / 435 and 357 / 442.
int int8_moe_tile_rows(int64_t pairs, int32_t n_experts) {
  const int64_t e = n_experts;
  if (pairs <= 2 * e) return 16;
  if (pairs <= 20 * e) return 64;
  return pairs <= 128 * e ? 128 : 256;
}

hipError_t launch_moe_int8(int mode, int tile_rows, const int8_t *aq, const float *as,
                           int64_t a_rows, int64_t k, const int32_t *perm, int32_t topk,
                           const int8_t *wq, const float *ws, int64_t n, const MoETile *tiles,
                           const int32_t *n_tiles, int64_t max_tiles, void *out, hipStream_t s) {
  if (max_tiles > 65535 || n % 32 != 0) return hipErrorInvalidValue;
  if (max_tiles == 0) return hipSuccess;
  I8Args g{};
  g.xq = aq;
  g.xs = as;
  g.wq = wq;
  g.ws = ws;
  g.y = out;
  g.n = n;
  g.kp = static_cast<int32_t>(int8_padded_k(k));
  g.perm = perm;
  g.tiles = tiles;
  g.n_tiles = n_tiles;
  g.a_rows = a_rows;
  g.topk = topk;
  // 16-row tiles: a wave's share of the steps (a quarter) in one batch where
  // it fits (16 tokens: up, 11 steps, 63 us in one batch of 11 and 81-91 in
  // eights; down, 8 steps, 59 us in eights and 63 in elevens)
  const bool eights = g.kp <= 4 * 8 * kI8Step;
  switch (tile_rows) {
    case 16:
      if (mode == 0)
        return eights ? launch_skinny_cfg<kI8Up, 4, 8>(g, max_tiles, s)
                      : launch_skinny_cfg<kI8Up, 4, 11>(g, max_tiles, s);
      return eights ? launch_skinny_cfg<kI8Down, 4, 8>(g, max_tiles, s)
                    : launch_skinny_cfg<kI8Down, 4, 11>(g, max_tiles, s);
    case 64:
      if (mode == 0) return launch_tile<kI8Up, 1, 4, 4, 2, 128, 3, 2>(g, max_tiles, s);
      return launch_tile<kI8Down, 1, 4, 4, 2, 128, 3, 2>(g, max_tiles, s);
    case 128:
      if (mode == 0) return launch_tile<kI8Up, 2, 4, 4, 4, 128, 3, 2>(g, max_tiles, s);
      return launch_tile<kI8Down, 2, 4, 4, 4, 128, 3, 2>(g, max_tiles, s);
    case 256:
      if (mode == 0) return launch_tile<kI8Up, 2, 4, 8, 4, 128, 2, 2>(g, max_tiles, s);
      return launch_tile<kI8Down, 2, 4, 8, 4, 128, 2, 2>(g, max_tiles, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tq4
