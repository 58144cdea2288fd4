// What the kernels over the 4-bit cache share: its layout and codes.
//
// 16 tokens of a (page, kv head) are a block of 9 D bytes: 16 rows of D / 2
// bytes of E2M1 codes, then 16 rows of D / 16 E4M3 scales, one for 16 channels.
// A code has 2 significant bits and a scale 4, and products lie between 2^-10
// and 6 * 448: exact in f16.
#pragma once
#include "common.cuh"

namespace qpkv {

template <int D>
struct Group4 {
  static constexpr int kRow = D / 2;              // bytes of codes of a token
  static constexpr int kScales = D / 16;          // scales of a token
  static constexpr int kScaleAt = 16 * kRow;      // where a block's scales begin
  static constexpr int kBlock = 9 * D;            // bytes of 16 tokens
};

// Eight E2M1 codes as four pairs of f16 (exact), in the order of the channels.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Eight float32 -> eight E2M1 codes (round to nearest even, saturate to +-6).
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The scale as a pair of f16.
__device__ __forceinline__ uint32_t e4m3_to_f16x2_both(uint32_t code) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(code * 0x101u));
}

__device__ __forceinline__ bool e4m3_is_nan(uint32_t code) { return (code & 0x7Fu) == 0x7Fu; }

// The last b in [0, B) with key(b) <= x, for keys that grow with b and key(0) <=
// x, by a whole warp: 32 of them are looked at in a step, as each step waits for
// its loads.
template <typename Key>
__device__ __forceinline__ int warp_last_at_most(int B, long long x, Key key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, m = lo + 1 + lane * step;
    const int below = __popc(__ballot_sync(0xffffffffu, m <= hi && key(m) <= x));
    if (below == 0) {
      hi = lo;
    } else {
      lo += 1 + (below - 1) * step;
      hi = min(hi, lo + step - 1);
    }
  }
  return lo;
}

}  // namespace qpkv
