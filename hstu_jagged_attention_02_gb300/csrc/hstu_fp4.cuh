// The 4-bit cache's numbers and its layout in memory (see the cache section
// of hstu_attn.h): e2m1 codes with one e4m3 scale for 16 features.
#pragma once

#include <cuda_fp16.h>

#include "hstu_common.cuh"

namespace hstu {

// One (page, head) block: K codes, K scales, V codes, V scales of page_size tokens.
struct PageLayout {
  int page_size, code_row, scale_row;   // tokens, bytes of a token's codes and scales
  __host__ __device__ PageLayout(int ps, int d) : page_size(ps), code_row(d / 2), scale_row(d / 16) {}
  __host__ __device__ int half() const { return page_size * (code_row + scale_row); }   // the K or the V part
  __host__ __device__ int bytes() const { return 2 * half(); }
  __host__ __device__ int scales() const { return page_size * code_row; }               // within a half
};

// e4m3 byte of x >= 0, to nearest even, at most 448; NaN stays NaN (0x7f).
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
// Two e4m3 bytes as a half2 (exact).
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return *reinterpret_cast<__half2*>(&r);
}
__device__ __forceinline__ float e4m3_float(uint32_t b) { return __low2float(e4m3x2_half2(b & 0xffu)); }

// e2m1 codes of (a, b), to nearest even, at most 6 in magnitude: a in bits 0-3, b in bits 4-7.
__device__ __forceinline__ uint32_t e2m1x2_of(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
// The two codes of byte `which` of w as a half2 (bits 0-3 in the low half; exact).
template <int which>
__device__ __forceinline__ __half2 e2m1x2_half2(uint32_t w) {
  uint32_t r;
  if constexpr (which == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (which == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (which == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return *reinterpret_cast<__half2*>(&r);
}

}  // namespace hstu
