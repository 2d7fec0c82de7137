// E4M3 conversions and the offsets of a batch over the 8-bit cache.
#pragma once

#include <stdint.h>

#include "serving.h"

namespace sda {

// Two E4M3 codes (low byte first) as fp16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}

// Nearest even, saturating at +-448; the first argument lands in the low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}

// What a block's scale may be: finite and not negative (by its bits, so that of several the largest bits tell).
__device__ __forceinline__ bool is_scale(float x) { return __float_as_uint(x) < 0x7f800000u; }

// Four codes under a scale, written anew under another: ratio = old / new <= 1.
// By a power of two fp16 takes the products exactly where they decide: a code
// has 4 significant bits, so what is not below 2^-10 (which rounds to zero) has
// its last bit at 2^-13 or above. Other ratios go through fp32.
struct Rescale {
  float ratio;
  uint32_t half2;  // the ratio as fp16, twice, where it is a power of two
  bool pow2;
  __device__ __forceinline__ explicit Rescale(float r) {
    ratio = r;
    pow2 = (__float_as_uint(r) & 0x7fffffu) == 0u;
    asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(half2) : "f"(r));
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t codes) const {
    const uint32_t lo = e4m3x2_to_f16x2(static_cast<uint16_t>(codes)), hi = e4m3x2_to_f16x2(static_cast<uint16_t>(codes >> 16));
    if (pow2) {
      uint32_t a, b;
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(a) : "r"(lo), "r"(half2));
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(b) : "r"(hi), "r"(half2));
      return f16x2_to_e4m3x2(a) | f16x2_to_e4m3x2(b) << 16;
    }
    const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
    return f32x2_to_e4m3x2(a.x * ratio, a.y * ratio) | f32x2_to_e4m3x2(b.x * ratio, b.y * ratio) << 16;
  }
};

// Sequence b's new rows and tokens, clamped to what the tensors hold.
struct NewRows {
  int row0, n;  // rows of the packed tensor (at most max_new of them are used)
  int first;    // position of row 0 in the sequence (negative: before its start)
  int len;      // tokens that the table can hold
};
__device__ __forceinline__ NewRows new_rows(const Cache& c, const int32_t* seq, const int32_t* lens, int b, bool& bad) {
  const int a = __ldg(seq + b), e = __ldg(seq + b + 1), given = __ldg(lens + b);
  NewRows r;
  r.row0 = min(max(a, 0), c.rows);
  const int n = min(max(e, r.row0), c.rows) - r.row0;
  r.len = min(max(given, 0), c.max_blocks * c.block);
  bad = bad || r.row0 != a || r.row0 + n != e || n > c.max_new || r.len != given;
  r.first = min(max(given, 0), 1 << 30) - n;
  r.n = min(n, c.max_new);
  return r;
}

}  // namespace sda
