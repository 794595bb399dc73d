// kv4.cuh — the 4-bit KV page and its arithmetic.
//
// A page holds the 16 positions of one (layer, K or V, KV head) in 1,152 bytes:
//   256*c + 16*t + j   the codes of elements 32c + 2j (low nibble) and
//                      32c + 2j + 1 (high nibble) of position t
//   1024 + 8*t + g     the scale byte of elements 16g .. 16g + 15
// (chunk-major, so that 16 threads that take a 16-byte chunk of neighbouring
// positions read 256 contiguous bytes).  A code is e2m1 (0, .5, 1, 1.5, 2, 3,
// 4, 6 and a sign); a scale byte b is the binary16 number of bits b << 7 (5
// exponent and 3 fraction bits), at most 10240.  A value is code times scale:
// at most 6 significant bits and at most 61440 in magnitude, so it is exact in
// binary16, in bf16 and in fp32.
#pragma once
#include "common.cuh"

namespace spec {

constexpr int kKv4PageBytes = SPEC_KV4_PAGE_BYTES;
constexpr int kKv4Scales = 1024;           // offset of the scale bytes in a page
constexpr int kKv4TopScale = 0xE2;         // the byte of 10240; larger bytes read as it
static_assert(kKv4PageBytes == kKv4Scales + 16 * 8, "page layout");

// offset of the 16-byte chunk c (elements 32c..) of position t
SPEC_DEV int kv4_chunk(int t, int c) { return 256 * c + 16 * t; }

SPEC_DEV float kv4_scale(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(min(byte, (uint32_t)kKv4TopScale) << 7)));
}

// the smallest scale byte whose scale s has 6 s >= amax (the top one if none
// has): amax / 6 truncated to 5 + 3 bits, or the byte after it.  6 s is exact in
// fp32, so the comparison settles which.
SPEC_DEV uint32_t kv4_scale_byte(float amax) {
  if (!(amax <= 6.f * 10240.f)) return kKv4TopScale;
  const uint32_t b = __half_as_ushort(__float2half_rz(amax * (1.0f / 6.0f))) >> 7;
  return 6.f * kv4_scale(b) < amax ? b + 1 : b;
}

// the codes nearest to 8 values, element i in nibble i
SPEC_DEV uint32_t e2m1_word(const float (&y)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}
// the 8 codes of a word as f16 pairs, element 2i in the low half of out[i]
SPEC_DEV void e2m1_word(uint32_t w, uint32_t (&out)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
}
// the 4 codes of 16 bits as f16 pairs
SPEC_DEV void e2m1_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %2;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
SPEC_DEV uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// code of x under scale s > 0: the number of midpoints below |x| (at or below
// it for those whose tie goes up to the even code).  t * s is exact in fp32.
SPEC_DEV uint32_t kv4_code(float x, float s) {
  const float a = fabsf(x);
  const uint32_t m = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) +
                     (a >= 3.5f * s) + (a > 5.0f * s);
  return m | ((__float_as_uint(x) >> 28) & 8u);
}

}  // namespace spec
