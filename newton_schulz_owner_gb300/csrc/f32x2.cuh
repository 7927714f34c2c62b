// Two fp32 numbers in a register pair, and bf16 pairs to and from them.
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace dm {

using F2 = unsigned long long;
DM_DEV F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
DM_DEV void f2_split(F2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
DM_DEV F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
DM_DEV F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
DM_DEV F2 negate2(F2 v) { return v ^ 0x8000000080000000ull; }

DM_DEV float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
DM_DEV float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
DM_DEV F2 bf16_pair(uint32_t w) { return f2(bf16_lo(w), bf16_hi(w)); }
// Both rounded to nearest, `lo` in the lower half.
DM_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
DM_DEV uint32_t pack_bf16(F2 v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return pack_bf16(lo, hi);
}

// Two bf16 numbers at a time: a b + c, rounded once.
DM_DEV uint32_t bf16_fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
DM_DEV uint32_t bf16_mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace dm
