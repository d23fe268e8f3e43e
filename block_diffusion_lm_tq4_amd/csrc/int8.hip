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

// Eight codes of one 16-byte piece of a bf16 row.  The quotient 127 v / a is
// taken as (127 v) * rcp(a), off by at most 2^(-15-d) (d as above): it rounds
// like the exact one unless that is a half-integer.  Then, and only then, the
// remainder 127 v - q a (exact in one fma: both terms are multiples of v's
// last bit, and it is at most a / 2) is plus or minus a / 2, and the even
// neighbour is taken.  11 instead of about 20 instructions for each code.
__device__ inline uint2 codes_of(uint4 d, float sc, float a, float inv) {
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t pair = w[2 * h + j / 2];
      const float v = __uint_as_float(j % 2 ? pair & 0xFFFF0000u : pair << 16);
      const float p = (v * sc) * 127.f;
      const float q = __builtin_rintf(p * inv);
      const float rho = __builtin_fmaf(-q, a, p);
      int qi = static_cast<int>(q);
      if ((qi & 1) && __builtin_fabsf(rho) + __builtin_fabsf(rho) == a) qi += rho > 0.f ? 1 : -1;
      word |= (static_cast<uint32_t>(qi) & 0xFFu) << (8 * j);
    }
    out[h] = word;
  }
  return make_uint2(out[0], out[1]);
}

// The largest magnitude bits of a piece.  Magnitude bits of bf16 order like
// the magnitudes, infinities and NaN last (0x7F80 and above).
__device__ inline uint32_t top_of(uint4 d) {
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
    t = t > lo ? t : lo;
    t = t > hi ? t : hi;
  }
  return t;
}

// What a row's largest magnitude bits say about it.
struct RowScale {
  float sc, a, inv, scale;
  bool live;
  __device__ explicit RowScale(uint32_t top) {
    // a power of two that keeps 127 v and 1 / a in range; it changes no
    // quotient: what the smaller one could drop has the code 0
    sc = top >= 0x7000u ? 0x1p-8f : (top < 0x1000u ? 0x1p+96f : 1.f);
    const float amax = __uint_as_float(top << 16);
    a = amax * sc;
    inv = __builtin_amdgcn_rcpf(a);
    const bool finite = top < 0x7F80u;
    live = finite && top != 0;
    scale = finite ? amax / 127.f : __builtin_nanf("");
  }
};

// bf16 rows, T threads each (64: a wave per row, four rows per workgroup, no
// barrier; 256: the workgroup).  A row of up to T * 8 * V values stays in
// registers between the maximum and the codes; longer ones are read twice.
// HBM-bound: 3 bytes per value.
template <int T, int V>
__global__ __launch_bounds__(kQThreads) void act_int8_kernel(const uint16_t *__restrict__ x,
                                                             int64_t m, int32_t k, int32_t kp,
                                                             int8_t *__restrict__ codes,
                                                             float *__restrict__ scales) {
  __shared__ uint32_t red[kQThreads / 64];
  constexpr int kRows = kQThreads / T;
  const int tid = threadIdx.x % T;
  const int n_vec = k / 8;    // k is a multiple of 32
  const int n_out = kp / 8;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T; row < m;
       row += static_cast<int64_t>(gridDim.x) * kRows) {
    const uint4 *xr = reinterpret_cast<const uint4 *>(x + row * k);
    uint2 *qr = reinterpret_cast<uint2 *>(codes + row * kp);
    uint4 d[V];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = tid + T * i;
      d[i] = at < n_vec ? xr[at] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t t = top_of(d[i]);
      top = top > t ? top : t;
    }
    for (int at = tid + T * V; at < n_vec; at += T) {
      const uint32_t t = top_of(xr[at]);
      top = top > t ? top : t;
    }
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
        qr[at] = rs.live ? codes_of(d[i], rs.sc, rs.a, rs.inv) : make_uint2(0u, 0u);
    }
    for (int at = tid + T * V; at < n_out; at += T)
      qr[at] = rs.live && at < n_vec ? codes_of(xr[at], rs.sc, rs.a, rs.inv) : make_uint2(0u, 0u);
    if (tid == 0) scales[row] = rs.scale;
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

__device__ inline uint16_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// The hidden value by its definition: u in fp64, relu(u)^2 rounded to fp32
// and then to bf16.  A NaN stays one.
__device__ inline float hidden_f64(int acc, float sx, float sw) {
  const double u = (static_cast<double>(acc) * static_cast<double>(sx)) * static_cast<double>(sw);
  const double h = u < 0.0 ? 0.0 : u * u;
  return static_cast<float>(h);
}

// The same in fp32 where that decides it: u carries at most three roundings
// and its square seven, 7 * 2^-24 relative, i.e. at most 7 fp32 steps, so the
// bf16 rounding is settled unless the low 16 bits are within 8 of the tie;
// about one value in 4000 takes fp64.
__device__ inline uint16_t hidden_of(int acc, float sx, float sw) {
  const float u = (static_cast<float>(acc) * sx) * sw;
  float h = acc > 0 ? u * u : 0.f;
  const uint32_t low = (__float_as_uint(h) & 0xFFFFu) - (0x8000u - 8u);
  const bool plain = h >= 0x1p-100f && h <= 0x1p+100f && low > 16u;
  // 0 * inf can only come from scales whose product overflows: fp64 tells
  if (!plain && (acc > 0 || __builtin_isnan(u))) h = hidden_f64(acc, sx, sw);
  return bf16_bits(h);
}

// One row's four consecutive outputs n .. n + 3 of the MoE products (n % 32
// == 0 columns in all, so a quad is whole or past the end).
template <int MODE>
__device__ inline void store_moe(const I8Args &g, intx4 acc, int64_t row, int64_t n, float sx,
                                 const float (&sw)[4]) {
  if (n >= g.n) return;
  if constexpr (MODE == kI8Up) {
    uint32_t w[2];
#pragma unroll
    for (int v = 0; v < 2; ++v)
      w[v] = static_cast<uint32_t>(hidden_of(acc[2 * v], sx, sw[2 * v])) |
             static_cast<uint32_t>(hidden_of(acc[2 * v + 1], sx, sw[2 * v + 1])) << 16;
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.y) + row * g.n + n) =
        make_uint2(w[0], w[1]);
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
        make_uint2(bf16_bits(p[0]) | static_cast<uint32_t>(bf16_bits(p[1])) << 16,
                   bf16_bits(p[2]) | static_cast<uint32_t>(bf16_bits(p[3])) << 16);
  } else if constexpr (VEC) {
    *reinterpret_cast<float4 *>(y + at) = make_float4(p[0], p[1], p[2], p[3]);
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v < left) tail_store_as<BF16>(y, at + v, p[v]);
  }
}

// A wave's MS x NS sub-tiles of a dense output: row m0 + 16 i + lane % 16,
// columns n0 + 16 j + 4 (lane / 16) ...; `rows` valid rows from m0.
template <int MS, int NS, bool BF16, bool VEC>
__device__ inline void store_block(const I8Args &g, const intx4 (&acc)[MS][NS], int64_t m0,
                                   int rows, int64_t n0, const float (&sx)[MS], int lane) {
#pragma clang fp contract(off)
  const int r = lane % 16;
  const bool has_bias = g.tail.bias != nullptr;
  const bool has_res = g.tail.residual != nullptr;
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int64_t n = n0 + 16 * j + 4 * (lane / 16);
    const int left = g.n - n < 4 ? static_cast<int>(g.n - n) : 4;
    if (left <= 0) continue;
    float sw[4], bias[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      sw[v] = v < left ? g.ws[n + v] : 0.f;
      bias[v] = has_bias && v < left ? g.tail.bias[n + v] : 0.f;
    }
    float res[MS][4];
    if (has_res) {
#pragma unroll
      for (int i = 0; i < MS; ++i)
        if (16 * i + r < rows)
          load_residual<BF16, VEC>(g, (m0 + 16 * i + r) * g.n + n, left, res[i]);
    }
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      float p[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        p[v] = (static_cast<float>(acc[i][j][v]) * sx[i]) * sw[v];
        if (has_bias) p[v] += bias[v];
        if (has_res) p[v] += res[i][v];
      }
      if (16 * i + r < rows) store_dense<BF16, VEC>(g, (m0 + 16 * i + r) * g.n + n, left, p);
    }
  }
}

template <int MS, int NS>
__device__ inline void store_any(const I8Args &g, const intx4 (&acc)[MS][NS], int64_t m0,
                                 int rows, int64_t n0, const float (&sx)[MS], int lane) {
  if (g.vec) {
    if (g.tail.bf16)
      store_block<MS, NS, true, true>(g, acc, m0, rows, n0, sx, lane);
    else
      store_block<MS, NS, false, true>(g, acc, m0, rows, n0, sx, lane);
  } else {
    if (g.tail.bf16)
      store_block<MS, NS, true, false>(g, acc, m0, rows, n0, sx, lane);
    else
      store_block<MS, NS, false, false>(g, acc, m0, rows, n0, sx, lane);
  }
}

// Scales of columns n .. n + 3 (row w0 + n of the stacked weights).
__device__ inline void load_sw(const I8Args &g, int64_t w0, int64_t n, float (&sw)[4]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) sw[v] = n + v < g.n ? g.ws[w0 + n + v] : 0.f;
}

// ---- few rows ---------------------------------------------------------------
// Up to 16 * MT rows: the weights are read once, straight into registers, and
// the product is bound by that stream.  A workgroup of KW waves takes 16 * NT
// columns; wave w takes the 64-k steps [w * per, (w + 1) * per) of them, B at
// a time, all loads of a batch issued before its first product.  The waves'
// int32 sums meet in LDS (exact in any order).
template <int MODE, int MT, int NT, int KW, int B>
__global__ __launch_bounds__(64 * KW) void i8_skinny_kernel(I8Args g) {
  __shared__ intx4 red[KW > 1 ? KW - 1 : 1][MT][NT][64];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int lane = tid % 64;
  const int r = lane % 16;
  const int grp = lane / 16;

  int64_t n0, m0 = 0, w0 = 0;
  int rows;
  if constexpr (MODE == kI8Dense) {
    n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT);
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
    n0 = static_cast<int64_t>(j) * (16 * NT);
    m0 = t.row0;
    rows = t.rows;
    w0 = static_cast<int64_t>(t.expert) * g.n;
  }

  const int8_t *wp[NT];
  const int8_t *xp[MT];
  int64_t src[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = n0 + 16 * j + r;
    wp[j] = g.wq + (w0 + (n < g.n ? n : g.n - 1)) * g.kp + 16 * grp;  // past n: read n - 1
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = m0 + (16 * i + r < rows ? 16 * i + r : 0);  // past the rows: the first
    src[i] = MODE == kI8Up ? g.perm[m] / g.topk : m;
    xp[i] = g.xq + src[i] * g.kp + 16 * grp;
  }
  intx4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = intx4{0, 0, 0, 0};

  const int steps = g.kp / kI8Step;
  const int per = (steps + KW - 1) / KW;
  const int s0 = wave * per;
  const int s1 = s0 + per < steps ? s0 + per : steps;
  for (int s = s0; s < s1; s += B) {
    intx4 a[B][NT], b[B][MT];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      // steps past the wave's end reload its last one and are not multiplied
      const int64_t k0 = static_cast<int64_t>(s + u < s1 ? s + u : s1 - 1) * kI8Step;
#pragma unroll
      for (int j = 0; j < NT; ++j) a[u][j] = *reinterpret_cast<const intx4 *>(wp[j] + k0);
#pragma unroll
      for (int i = 0; i < MT; ++i) b[u][i] = *reinterpret_cast<const intx4 *>(xp[i] + k0);
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (s + u < s1) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][j], b[u][i], acc[i][j], 0, 0, 0);
      }
    }
  }
  if constexpr (KW > 1) {
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) red[wave - 1][i][j][lane] = acc[i][j];
    }
    __syncthreads();
  }
  // wave w finishes sub-tiles w, w + KW, ... of the MT * NT; wave 0's sums are
  // in its registers, so with one wave there is no exchange
  if constexpr (KW > 1) {
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < KW - 1; ++w)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] += red[w][i][j][lane];
  }
  if constexpr (MODE == kI8Dense) {
    float sx[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) sx[i] = g.xs[src[i]];
    store_any<MT, NT>(g, acc, m0, rows, n0, sx, lane);
  } else {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float sw[4];
      load_sw(g, w0, n0 + 16 * j + 4 * grp, sw);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if (16 * i + r < rows)
          store_moe<MODE>(g, acc[i][j], m0 + 16 * i + r, n0 + 16 * j + 4 * grp, g.xs[src[i]], sw);
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
// are stored at slot ^ key(row), key = (row / 4) % 4 for 64-byte rows and
// (row / 2) % 8 for 128-byte rows, so the 16 rows that a fragment read visits
// at one slot fall on all 64 banks.  Rows past the tile's end read zeros
// (dense; the buffer range ends there) or the tile's first row (MoE) and are
// not stored.
template <int MODE, int WM, int WN, int MS, int NS, int KB, int S, int OCC>
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
    // contiguous run of an order that walks blocks of 4 tile columns down
    // all tile rows, so the tiles it holds at a time share their operands in
    // its L2.
    const int total = g.tiles_m * g.tiles_n;
    const int id = static_cast<int>(blockIdx.x);
    const int x = id % 8;
    const int q = total / 8, rem = total % 8;
    const int at = x * q + (x < rem ? x : rem) + id / 8;
    const int blk = at / (4 * g.tiles_m);
    const int in = at % (4 * g.tiles_m);
    const int width = g.tiles_n - 4 * blk < 4 ? g.tiles_n - 4 * blk : 4;
    m_base = static_cast<int64_t>(in / width) * TM;
    n_base = static_cast<int64_t>(4 * blk + in % width) * TN;
    rows = g.m - m_base < TM ? static_cast<int>(g.m - m_base) : TM;
  } else {
    const int per = (g.tiles_n + 7) / 8;
    const int q = static_cast<int>(blockIdx.x) / 8;
    const int i = q / per;
    if (i >= *g.n_tiles) return;
    const MoETile t = g.tiles[i];
    const int j = (static_cast<int>(blockIdx.x) + t.expert) % 8 + 8 * (q % per);
    if (j >= g.tiles_n) return;
    m_base = t.row0;
    rows = t.rows;
    n_base = static_cast<int64_t>(j) * TN;
    w0 = static_cast<int64_t>(t.expert) * g.n;
  }
  const int cols = g.n - n_base < TN ? static_cast<int>(g.n - n_base) : TN;

  // A piece's lane l fills row l / kSlots at stored slot l % kSlots; the key of
  // a row depends on row % 16, so the pieces of 8 rows alternate between two.
  const int prow = lane / kSlots;
  auto slot_of = [&](int row) __attribute__((always_inline)) {
    return (lane % kSlots) ^ (KB == 64 ? (row >> 2) & 3 : (row >> 1) & 7);
  };
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

  intx4 acc[MS][NS];
#pragma unroll
  for (int i = 0; i < MS; ++i)
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[i][j] = intx4{0, 0, 0, 0};

  // fragment addresses: row 16 * x + r, whose key depends on r alone
  const int key = KB == 64 ? (r >> 2) & 3 : (r >> 1) & 7;
  const int a_frag = (wm * (16 * MS) + r) * KB;
  const int w_frag = kWBase + (wn * (16 * NS) + r) * KB;
  const bool idle = MODE != kI8Dense && wm * (16 * MS) >= rows;
  auto half = [&](const uint8_t *st, int h) __attribute__((always_inline)) {
    const int slot = 16 * ((4 * h + grp) ^ key);
    intx4 wf[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j)
      wf[j] = *reinterpret_cast<const intx4 *>(st + w_frag + 16 * j * KB + slot);
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      const intx4 af = *reinterpret_cast<const intx4 *>(st + a_frag + 16 * i * KB + slot);
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
      if (c + s < steps && !idle) {
        half(smem + s * kStage, 0);
        if (KB == 128 && 2 * (c + s) + 1 < halves) half(smem + s * kStage, 1);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // the padding steps' loads

  if (idle) return;
  float sx[MS];
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    const int row = wm * (16 * MS) + 16 * i + r;
    const int64_t b = m_base + (row < rows ? row : 0);
    sx[i] = g.xs[MODE == kI8Up ? g.perm[b] / g.topk : b];
  }
  if constexpr (MODE == kI8Dense) {
    store_any<MS, NS>(g, acc, m_base + wm * (16 * MS), rows - wm * (16 * MS),
                      n_base + wn * (16 * NS), sx, lane);
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const int64_t n = n_base + wn * (16 * NS) + 16 * j + 4 * grp;
      float sw[4];
      load_sw(g, w0, n, sw);
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        const int row = wm * (16 * MS) + 16 * i + r;
        if (row < rows) store_moe<MODE>(g, acc[i][j], m_base + row, n, sx[i], sw);
      }
    }
  }
}

template <int MODE, int WM, int WN, int MS, int NS, int KB, int S, int OCC>
hipError_t launch_tile(I8Args g, int64_t max_tiles, hipStream_t s) {
  constexpr int TM = 16 * MS * WM, TN = 16 * NS * WN;
  g.tiles_n = static_cast<int32_t>((g.n + TN - 1) / TN);
  int64_t grid;
  if (MODE == kI8Dense) {
    g.tiles_m = static_cast<int32_t>((g.m + TM - 1) / TM);
    grid = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  } else {
    grid = max_tiles * ((g.tiles_n + 7) / 8 * 8);
  }
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((i8_tile_kernel<MODE, WM, WN, MS, NS, KB, S, OCC>),
                     dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), 0, s, g);
  return hipGetLastError();
}

template <int MODE, int MT, int NT, int KW, int B>
hipError_t launch_skinny_cfg(I8Args g, int64_t max_tiles, hipStream_t s) {
  g.tiles_n = static_cast<int32_t>((g.n + 16 * NT - 1) / (16 * NT));
  const int64_t grid =
      MODE == kI8Dense ? g.tiles_n : max_tiles * ((g.tiles_n + 7) / 8 * 8);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((i8_skinny_kernel<MODE, MT, NT, KW, B>), dim3(static_cast<unsigned>(grid)),
                     dim3(64 * KW), 0, s, g);
  return hipGetLastError();
}

}  // namespace

int64_t int8_padded_k(int64_t k) { return (k + kI8Step - 1) / kI8Step * kI8Step; }

hipError_t launch_act_int8(const uint16_t *x, int64_t m, int64_t k, int8_t *codes, float *scales,
                           hipStream_t s) {
  if (m == 0 || k == 0) return hipSuccess;
  const int32_t k32 = static_cast<int32_t>(k);
  const int32_t kp = static_cast<int32_t>(int8_padded_k(k));
  if (m >= 1024 && k <= 64 * 8 * 8) {
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
  g.kp = static_cast<int32_t>(int8_padded_k(k));
  const size_t quad = tail.bf16 ? 8 : 16;
  g.vec = n % 4 == 0 && reinterpret_cast<uintptr_t>(y) % quad == 0 &&
          reinterpret_cast<uintptr_t>(tail.residual) % quad == 0;
  if (m <= 16) return launch_skinny_cfg<kI8Dense, 1, 2, 8, 6>(g, 0, s);
  if (m <= 32) return launch_skinny_cfg<kI8Dense, 2, 2, 8, 6>(g, 0, s);
  if (m <= 64) return launch_skinny_cfg<kI8Dense, 4, 1, 8, 4>(g, 0, s);
  if (m * n < 256 * 128 * 128) return launch_tile<kI8Dense, 2, 2, 2, 2, 128, 3, 2>(g, 0, s);
  if (m * n < 256 * 256 * 256) return launch_tile<kI8Dense, 2, 2, 4, 4, 128, 2, 2>(g, 0, s);
  return launch_tile<kI8Dense, 2, 4, 8, 4, 64, 4, 2>(g, 0, s);
}

int int8_moe_tile_rows(int64_t pairs, int32_t n_experts) {
  if (pairs <= 16 * static_cast<int64_t>(n_experts)) return 16;
  return pairs <= 128 * static_cast<int64_t>(n_experts) ? 64 : 128;
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
  switch (tile_rows) {
    case 16:
      if (mode == 0) return launch_skinny_cfg<kI8Up, 1, 2, 4, 8>(g, max_tiles, s);
      return launch_skinny_cfg<kI8Down, 1, 2, 4, 8>(g, max_tiles, s);
    case 64:
      if (mode == 0) return launch_tile<kI8Up, 1, 4, 4, 2, 128, 3, 2>(g, max_tiles, s);
      return launch_tile<kI8Down, 1, 4, 4, 2, 128, 3, 2>(g, max_tiles, s);
    case 128:
      if (mode == 0) return launch_tile<kI8Up, 2, 4, 4, 4, 128, 3, 2>(g, max_tiles, s);
      return launch_tile<kI8Down, 2, 4, 4, 4, 128, 3, 2>(g, max_tiles, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tq4
