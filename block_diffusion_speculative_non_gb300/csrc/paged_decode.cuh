// paged_decode.cuh — 4-bit codes of a page into pairs of fp16 or bf16 numbers (internal to libfpd).
//
// Code n + 8 in bits 6..9 (2..5) of an fp16 number of exponent 4 (8) reads 16 + n + 8 (256 + n + 8), and one fused multiply-add with
// s' = s 2^-7 takes it to n s' exactly: 7 bits, multiples of 2^-24, and 264 s' stays in range.  In bf16 the code goes to bits 3..6 of
// exponent 4 and the scale needs no shift.
#pragma once

#include "fpd_paged.cuh"

namespace fpd {

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <uint32_t MASK, uint32_t OR>
__device__ __forceinline__ uint32_t and_or(uint32_t v) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "n"(MASK), "n"(OR));   // (a & b) | c
  return r;
}
constexpr uint32_t h2(uint32_t bits) { return bits * 0x10001u; }

// Two scales (fp16 bits, a pair) as what the codes' multiply-adds need.
struct Scale2 {
  uint32_t s, o24, o264;
  __device__ __forceinline__ explicit Scale2(uint32_t raw) {
    s = hmul2(raw, h2(0x2000));       // 2^-7
    o24 = hmul2(s, h2(0xCE00));       // -24
    o264 = hmul2(s, h2(0xDC20));      // -264
  }
};
// Nibble k of the lower and of the upper half of w as a pair n s', k = 0..3.
__device__ __forceinline__ void decode4(uint32_t w, const Scale2& s, uint32_t (&r)[4]) {
  const uint32_t a = w << 2, b = w >> 6;
  r[0] = hfma2(and_or<0x003C003Cu, 0x5C005C00u>(a), s.s, s.o264);
  r[1] = hfma2(and_or<0x03C003C0u, 0x4C004C00u>(a), s.s, s.o24);
  r[2] = hfma2(and_or<0x003C003Cu, 0x5C005C00u>(b), s.s, s.o264);
  r[3] = hfma2(and_or<0x03C003C0u, 0x4C004C00u>(b), s.s, s.o24);
}

// The same in bf16: a scale s, the pair (nibble k of the lower half, of the upper half) as n s.
struct Scale2Bf {
  uint32_t s, o24;
  __device__ __forceinline__ explicit Scale2Bf(uint32_t byte) {
    const uint32_t raw = byte * 0x00100010u;   // s 2^-112: the exponent's bias is 127, not 15
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(s) : "r"(raw), "r"(h2(0x7780)));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o24) : "r"(s), "r"(h2(0xC1C0)));
  }
};
__device__ __forceinline__ void decode4_bf16(uint32_t w, const Scale2Bf& s, uint32_t (&r)[4]) {
  const uint32_t v[4] = {w << 3, w >> 1, w >> 5, w >> 9};
#pragma unroll
  for (int i = 0; i < 4; i++)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(and_or<0x00780078u, 0x41804180u>(v[i])), "r"(s.s), "r"(s.o24));
}

}  // namespace fpd
