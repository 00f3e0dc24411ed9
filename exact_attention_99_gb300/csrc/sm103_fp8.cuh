// e4m3 values of a cache and their scales, for sm_103a.
#pragma once
#include <cstdint>

#include "sm103_math.cuh"
#include "sm103_ptx.cuh"

namespace fa {

constexpr int kFp8Block = 16;  // tokens of a block that has a scale (for each head)

// Instruction descriptors: kind::f16 with f16 A and B (bf16's without the format
// bits), kind::f8f6f4 with e4m3 A and B, both K-major (format 0 too).
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t a_mn_major, uint32_t b_mn_major) {
  return (1u << 4) | (a_mn_major << 15) | (b_mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_codes_f32(uint32_t M, uint32_t N) { return idesc_f16_f32(M, N, 0, 0); }

// The high descriptor word of rows of 64 bytes with the 64-byte swizzle (layout type
// 4): 512 bytes from one 8-row group to the next.
constexpr uint32_t kSdescHi64 = (512u >> 4) | (1u << 14) | (4u << 29);

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3, 32 per K step, descriptors by their low words
template <uint32_t HI>
__device__ __forceinline__ void mma_codes_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(HI)
      : "memory");
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// the larger of each pair of halves, unsigned (of bf16 without its sign: the larger magnitude)
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// two e4m3 codes to f16 (which holds every e4m3 value)
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
// two values to e4m3, nearest even, past the largest the largest, NaN to NaN
__device__ __forceinline__ uint16_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two values to f16, nearest even
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t x) {
  float r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float f16_hi(uint32_t x) {
  float r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(r) : "r"(x));
  return r;
}

// 0xff where a byte of x is a NaN code, of either sign
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) {
  return (((x & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u) * 0xffu;
}

// four bf16 values (two words) times f, a power of two, to four codes
__device__ __forceinline__ uint32_t e4m3x4_of_bf16(uint32_t x, uint32_t y, float f) {
  const uint64_t f2 = pack2(f, f);
  float a, b, c, d;
  unpack2(fmul2(pack2(u2f(x << 16), u2f(x & 0xffff0000u)), f2), a, b);
  unpack2(fmul2(pack2(u2f(y << 16), u2f(y & 0xffff0000u)), f2), c, d);
  return uint32_t(e4m3x2_of(a, b)) | (uint32_t(e4m3x2_of(c, d)) << 16);
}
// four codes times f, a power of two, rounded to codes again
__device__ __forceinline__ uint32_t e4m3x4_times(uint32_t x, float f) {
  const uint32_t a = f16x2_of_e4m3x2(uint16_t(x)), b = f16x2_of_e4m3x2(uint16_t(x >> 16));
  return uint32_t(e4m3x2_of(f16_lo(a) * f, f16_hi(a) * f)) | (uint32_t(e4m3x2_of(f16_lo(b) * f, f16_hi(b) * f)) << 16);
}


// The same where the product or quotient is not exact: cut to 32 bits with its last bit set, so
// that rounding it to fewer bits is rounding the value itself. (A quotient, or a product with
// more bits, may lie nearer to halfway between two codes than 32 bits can tell.)
__device__ __forceinline__ float odd_of(float cut, float rest) {
  return rest == 0.0f ? cut : u2f(f2u(cut) | 1u);
}
__device__ __forceinline__ float odd_product(float a, float f) {
  const float y = __fmul_rz(a, f);
  return odd_of(y, fmaf(a, f, -y));
}
__device__ __forceinline__ float odd_quotient(float a, float f) {
  const float y = __fdiv_rz(a, f);
  return odd_of(y, fmaf(-y, f, a));
}
// four bf16 values over f, to four codes
__device__ __forceinline__ uint32_t e4m3x4_of_bf16_over(uint32_t x, uint32_t y, float f) {
  return uint32_t(e4m3x2_of(odd_quotient(u2f(x << 16), f), odd_quotient(u2f(x & 0xffff0000u), f))) |
         (uint32_t(e4m3x2_of(odd_quotient(u2f(y << 16), f), odd_quotient(u2f(y & 0xffff0000u), f))) << 16);
}
// four codes times f, rounded to codes again
__device__ __forceinline__ uint32_t e4m3x4_odd_times(uint32_t x, float f) {
  const uint32_t a = f16x2_of_e4m3x2(uint16_t(x)), b = f16x2_of_e4m3x2(uint16_t(x >> 16));
  return uint32_t(e4m3x2_of(odd_product(f16_lo(a), f), odd_product(f16_hi(a), f))) |
         (uint32_t(e4m3x2_of(odd_product(f16_lo(b), f), odd_product(f16_hi(b), f))) << 16);
}

}  // namespace fa
