// The 4-bit cache format (include/ds.h, "The 4-bit paged cache"): e2m1 codes
// with an e4m3 scale per 16 channels, and its conversions.
//
// code * scale has at most 2 + 4 significant bits and lies between 2^-10 and
// 2688, so f16, bf16 and f32 all hold it exactly: none of the conversions
// below rounds, except quantising itself.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "dev_common.cuh"
#include "tc_ptx.cuh"

namespace ds {

constexpr int kKv4Group = 16;              // channels per scale

__host__ __device__ constexpr int kv4_code_bytes(int d) { return d / 2; }
__host__ __device__ constexpr int kv4_scale_bytes(int d) { return d / kKv4Group; }

// Eight codes (one 32-bit word, channel 0 in the low nibble) as four f16
// pairs, the lower channel in the low half.
DS_DEV void kv4_codes_f16(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}

// Two scale bytes as an f16 pair.  The patterns that are no number read as
// 448: min returns the operand that is one.
DS_DEV uint32_t kv4_scales_f16(uint32_t two_bytes) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h;\n\t"
      "min.f16x2 %0, %0, %2;\n\t}"
      : "=r"(r)
      : "r"(two_bytes), "r"(0x5f005f00u));     // 448 in both halves
  return r;
}

DS_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A bf16 pair as an f16 pair: exact from 2^-14 up, rounded to 2^-24 below,
// clamped to the largest f16 (a NaN stays one).
DS_DEV uint32_t bf16x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;"
      : "=r"(r)
      : "f"(__uint_as_float(w & 0xffff0000u)), "f"(__uint_as_float(w << 16)));
  return r;
}

// Sixteen bf16 values (eight words, in order) times `mult` = 2^-exp as one
// scale byte and eight bytes of codes.  `bad` is set when a value is a NaN
// (stored as 0) or an infinity.
//
// Both roundings only decide between neighbouring values of a small format,
// and an inexact quotient must not move one that lies on a midpoint.  x has 8
// significant bits; a midpoint of the codes times a scale has at most 7, and
// one of the scales times 6 at most 7 as well, so a quotient that is not a
// midpoint is off it by at least one part in 255.  The quotients are formed
// as products with a rounded reciprocal (off by 2^-23 of themselves) and then
// rounded to a grid that holds every midpoint: the maximum's sixth to f16's
// 11 bits, the others to multiples of 2^-11 by adding and subtracting 6144.
// On the grid a midpoint is met exactly, and nothing else reaches one.
DS_DEV void kv4_quantise16(uint32_t (&w)[8], float mult, uint32_t& scale_byte, uint2& codes,
                           bool& bad) {
  auto top = [&]() {               // the largest magnitude, NaN if there is one
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i)
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(m >> 16 | m << 16));
    return __uint_as_float(r << 16);
  };
  float mx = top();
  bad = !(mx < INFINITY);
  if (bad) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((w[i] & 0x7fffu) > 0x7f80u) w[i] &= 0xffff0000u;
      if ((w[i] & 0x7fff0000u) > 0x7f800000u) w[i] &= 0xffffu;
    }
    mx = top();
  }
  const float sf = fminf(mx * mult * 0.16666667f, 448.f);
  uint32_t s2;
  uint16_t sb;
  asm("{\n\t.reg .b32 h;\n\tcvt.rn.f16x2.f32 h, %2, %3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, h;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, %0;\n\t}"
      : "=h"(sb), "=r"(s2)
      : "f"(0.f), "f"(sf));
  scale_byte = sb & 0xffu;
  const float s = __half2float(__ushort_as_half((unsigned short)(s2 & 0xffffu)));
  const float inv = s > 0.f ? __frcp_rn(s) * mult : 0.f;
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lo = fmaf(__uint_as_float(w[i] << 16), inv, 6144.f) - 6144.f;
    const float hi = fmaf(__uint_as_float(w[i] & 0xffff0000u), inv, 6144.f) - 6144.f;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(b[i])
        : "f"(hi), "f"(lo));
  }
  auto pack = [](uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
    return __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
  };
  codes = make_uint2(pack(b[0], b[1], b[2], b[3]), pack(b[4], b[5], b[6], b[7]));
}

}  // namespace ds
