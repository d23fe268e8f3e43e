// Test-only kernels for the instructions that the MXFP4 operators rest on, on
// operands given by the host:
//   - one v_mfma_scale_f32_16x16x128_f8f6f4 on e2m1 operands (one E8M0 scale per
//     32 k on each side);
//   - v_cvt_scalef32_pk_fp4_bf16 and v_cvt_scalef32_pk_fp4_f32.
#include <hip/hip_runtime.h>
#include <stdint.h>

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

//   a, b : [16][64] bytes of two e2m1 codes (row m of A, column n of B)
//   sa, sb : [16][4] E8M0 scale bytes (row m / column n, block k / 32)
//   c : [16][16] fp32 accumulator input, d : [16][16] fp32 output
// The scale byte is taken from byte `sel` (0 .. 3) of the scale operand.
template <int SEL>
__global__ __launch_bounds__(64) void mfma_kernel(const uint8_t *a, const uint8_t *b,
                                                  const uint8_t *sa, const uint8_t *sb,
                                                  const float *c, float *d) {
  const int lane = threadIdx.x;
  const int i = lane % 16;
  const int g = lane / 16;
  // lane i + 16 g holds k = 32 g .. 32 g + 31 of row (column) i, and their scale
  const intx4 av = *reinterpret_cast<const intx4 *>(a + i * 64 + 16 * g);
  const intx4 bv = *reinterpret_cast<const intx4 *>(b + i * 64 + 16 * g);
  const intx8 aq = {av[0], av[1], av[2], av[3], 0, 0, 0, 0};
  const intx8 bq = {bv[0], bv[1], bv[2], bv[3], 0, 0, 0, 0};
  // the other bytes of the scale operands hold something else
  const int sav = (0x11223344 & ~(0xFF << (8 * SEL))) | (sa[i * 4 + g] << (8 * SEL));
  const int sbv = (0x55667788 & ~(0xFF << (8 * SEL))) | (sb[i * 4 + g] << (8 * SEL));
  floatx4 acc;
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] = c[(4 * g + v) * 16 + i];
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aq, bq, acc, 4, 4, SEL, sav, SEL, sbv);
#pragma unroll
  for (int v = 0; v < 4; ++v) d[(4 * g + v) * 16 + i] = acc[v];
}

extern "C" int tq4test_mfma_fp4_probe(const uint8_t *a, const uint8_t *b, const uint8_t *sa,
                                      const uint8_t *sb, const float *c, float *d, int sel,
                                      void *stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (sel < 0 || sel > 3) return 2;
  if (sel == 0) hipLaunchKernelGGL(mfma_kernel<0>, dim3(1), dim3(64), 0, s, a, b, sa, sb, c, d);
  if (sel == 1) hipLaunchKernelGGL(mfma_kernel<1>, dim3(1), dim3(64), 0, s, a, b, sa, sb, c, d);
  if (sel == 2) hipLaunchKernelGGL(mfma_kernel<2>, dim3(1), dim3(64), 0, s, a, b, sa, sb, c, d);
  if (sel == 3) hipLaunchKernelGGL(mfma_kernel<3>, dim3(1), dim3(64), 0, s, a, b, sa, sb, c, d);
  return hipGetLastError() == hipSuccess ? 0 : 5;
}

// Pairs (values 2 i and 2 i + 1) to one byte each, once from bf16 and once from
// fp32, with the scale given by its fp32 bits.
__global__ __launch_bounds__(256) void cvt_kernel(const uint16_t *v, const uint32_t *scale, int n,
                                                  uint8_t *from_bf16, uint8_t *from_f32) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const uint32_t lo = v[2 * i], hi = v[2 * i + 1];
  const float s = __builtin_bit_cast(float, scale[i]);
  const bf16x2 p = __builtin_bit_cast(bf16x2, lo | hi << 16);
  from_bf16[i] = static_cast<uint8_t>(__builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, p, s, 0));
  from_f32[i] = static_cast<uint8_t>(__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(
      0u, __builtin_bit_cast(float, lo << 16), __builtin_bit_cast(float, hi << 16), s, 0));
}

extern "C" int tq4test_cvt_fp4_probe(const uint16_t *v, const uint32_t *scale, int n,
                                     uint8_t *from_bf16, uint8_t *from_f32, void *stream) {
  if (n < 1) return 2;
  hipLaunchKernelGGL(cvt_kernel, dim3((n + 255) / 256), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(stream), v, scale, n, from_bf16, from_f32);
  return hipGetLastError() == hipSuccess ? 0 : 5;
}
