// Activations in 8 bits: 32 consecutive values of a row share a bf16 scale.
//
//   scale = the smallest bf16 number >= max|v| / 127, at least 2^-126 (so that its
//           reciprocal is finite); 0 for a block of zeros; NaN, with codes 0, for a
//           block that holds a NaN or an infinity (the block comes back as NaN)
//   code  = the integer nearest to v / scale, ties to even, in [-127, 127]
//
// The scale has 8 significant bits.  So has a bf16 value, and the quotient of two
// such numbers in [0.5, 127] either is exactly k + 1/2 or is at least 1/510 away
// from it: rounding the quotient in fp32 gives the code of exact arithmetic.
#pragma once
#include "ptx.cuh"

namespace dm {

DM_DEV float act8_scale(float top, bool finite) {
  if (!finite) return __int_as_float(0x7fc00000);
  if (top == 0.f) return 0.f;
  const float s = fmaxf(__fdiv_rn(top, 127.f), 1.17549435e-38f);
  return __int_as_float((__float_as_int(s) + 0xFFFF) & int(0xFFFF0000));
}

// Code of a bf16 value from the rounded reciprocal r of its scale.  v * r is
// within 2e-5 of the quotient; adding and subtracting 3072 rounds it to a
// multiple of 2^-12, which restores exact ties and moves nothing across one.
// 1.5 * 2^23 then leaves the integer in the low bits.
DM_DEV uint32_t act8_code_bf16(float v, float r) {
  const float q = __fadd_rn(__fadd_rn(__fmul_rn(v, r), 3072.f), -3072.f);
  return __float_as_uint(__fadd_rn(q, 12582912.f)) & 0xFFu;
}
// The nearest integer to v * r in the low byte (the others are not cleared).
DM_DEV uint32_t act8_code_fast(float v, float r) {
  return __float_as_uint(__fadd_rn(__fmul_rn(v, r), 12582912.f));
}
// Byte i of w as a signed integer, in fp32: 2^23 + (code ^ 0x80) is one byte permutation
// and an exact subtraction away (the conversion units run at an eighth of their rate).
DM_DEV float act8_int(uint32_t w, int i) {
  return __fsub_rn(__uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4B000000u, 0x7440u + uint32_t(i))),
                   8388736.f);
}
DM_DEV uint32_t act8_code_f32(float v, float s) {
  return uint32_t(__float2int_rn(__fdiv_rn(v, s))) & 0xFFu;
}

}  // namespace dm
