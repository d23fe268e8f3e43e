// Test-only kernel for the wider instruction of the MXFP4 tiles, on operands given by the host:
// one v_mfma_scale_f32_32x32x64_f8f6f4 on e2m1 operands (one E8M0 scale per 32 k on each side).
#include <hip/hip_runtime.h>
#include <stdint.h>

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

//   a, b : [32][32] bytes of two e2m1 codes (row m of A, column n of B)
//   sa, sb : [32][2] E8M0 scale bytes (row m / column n, block k / 32)
//   c : [32][32] fp32 accumulator input, d : [32][32] fp32 output
// The scale byte is taken from byte `sel` (0 .. 3) of the scale operand.
template <int SEL>
__global__ __launch_bounds__(64) void mfma_wide_kernel(const uint8_t *a, const uint8_t *b,
                                                       const uint8_t *sa, const uint8_t *sb,
                                                       const float *c, float *d) {
  const int lane = threadIdx.x;
  const int i = lane % 32;
  const int g = lane / 32;
  // lane i + 32 g holds k = 32 g .. 32 g + 31 of row (column) i, and their scale
  const intx4 av = *reinterpret_cast<const intx4 *>(a + i * 32 + 16 * g);
  const intx4 bv = *reinterpret_cast<const intx4 *>(b + i * 32 + 16 * g);
  const intx8 aq = {av[0], av[1], av[2], av[3], 0, 0, 0, 0};
  const intx8 bq = {bv[0], bv[1], bv[2], bv[3], 0, 0, 0, 0};
  // the other bytes of the scale operands hold something else
  const int sav = (0x11223344 & ~(0xFF << (8 * SEL))) | (sa[i * 2 + g] << (8 * SEL));
  const int sbv = (0x55667788 & ~(0xFF << (8 * SEL))) | (sb[i * 2 + g] << (8 * SEL));
  // lane i + 32 g holds rows 8 q + 4 g .. + 3, q = 0 .. 3, of column i
  floatx16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = c[(8 * (v / 4) + 4 * g + v % 4) * 32 + i];
  acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aq, bq, acc, 4, 4, SEL, sav, SEL, sbv);
#pragma unroll
  for (int v = 0; v < 16; ++v) d[(8 * (v / 4) + 4 * g + v % 4) * 32 + i] = acc[v];
}

extern "C" int tq4test_mfma_fp4_wide_probe(const uint8_t *a, const uint8_t *b, const uint8_t *sa,
                                           const uint8_t *sb, const float *c, float *d, int sel,
                                           void *stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 one(1), wave(64);
  if (sel < 0 || sel > 3) return 2;
  if (sel == 0) hipLaunchKernelGGL(mfma_wide_kernel<0>, one, wave, 0, s, a, b, sa, sb, c, d);
  if (sel == 1) hipLaunchKernelGGL(mfma_wide_kernel<1>, one, wave, 0, s, a, b, sa, sb, c, d);
  if (sel == 2) hipLaunchKernelGGL(mfma_wide_kernel<2>, one, wave, 0, s, a, b, sa, sb, c, d);
  if (sel == 3) hipLaunchKernelGGL(mfma_wide_kernel<3>, one, wave, 0, s, a, b, sa, sb, c, d);
  return hipGetLastError() == hipSuccess ? 0 : 5;
}
