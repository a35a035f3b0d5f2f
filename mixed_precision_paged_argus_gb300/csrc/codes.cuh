// 8-bit codes to 16-bit operands in registers, exactly.
#pragma once

#include "common.cuh"

namespace argus {

__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// Four codes to four 16-bit values, exactly.
template <bool BF>
__device__ __forceinline__ void fp8_to_16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (!BF) {
    // the word's halves as they are: masks and shifts would be half of the instructions
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // sign to the top, exponent and fraction to the low exponent bits and the
    // top fraction bits: the value times 2^-120 (e4m3's bias is 7, bf16's 127;
    // subnormals land on subnormals), undone by an exact product with 2^120
    const uint32_t a = prmt(w, 0, 0x1404), b = prmt(w, 0, 0x3424);
    lo = bf2_mul(((a >> 4) & 0x07F007F0u) | (a & 0x80008000u), 0x7B807B80u);
    hi = bf2_mul(((b >> 4) & 0x07F007F0u) | (b & 0x80008000u), 0x7B807B80u);
  }
}

template <bool BF>
__device__ __forceinline__ void int8_to_16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (!BF) {
    const uint32_t u = w ^ 0x80808080u;                      // 1024 + (code + 128), minus 1152
    lo = hsub2_u32(prmt(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2_u32(prmt(u, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    // 128 + the low seven bits, minus 128, or 256 for a negative code: the
    // code's sign bit is the lowest exponent bit of 0x43xx
    const uint32_t a = prmt(w, 0x43434343u, 0x4140), b = prmt(w, 0x43434343u, 0x4342);
    lo = bf2_sub(a & 0xFF7FFF7Fu, a & 0xFF80FF80u);
    hi = bf2_sub(b & 0xFF7FFF7Fu, b & 0xFF80FF80u);
  }
}

// Four values to e4m3 codes, to nearest even, saturating; a's in the low byte.
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float a, float b, float c, float d) {
  uint32_t o;
  asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
      : "=r"(o)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return o;
}

}  // namespace argus
