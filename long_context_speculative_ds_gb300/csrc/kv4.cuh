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
  auto clamp = [](float x) { return x > 65504.f ? 65504.f : (x < -65504.f ? -65504.f : x); };
  return ptx::pack_f16x2(clamp(__uint_as_float(w << 16)), clamp(__uint_as_float(w & 0xffff0000u)));
}

// Sixteen values, already multiplied by 2^-exp, as one scale byte and eight
// bytes of codes.  `bad` is set when a value is a NaN (stored as 0) or an
// infinity.
//
// The quotients y / scale only decide between neighbouring e2m1 values, and
// so does the scale's own rounding.  y has 8 significant bits and scale x
// midpoint at most 7, so a quotient that is not exactly a midpoint is off it
// by at least one part in 255: y times the rounded reciprocal, rounded once
// more to f16 (11 bits), is the midpoint when the true quotient is, and on
// its side of it otherwise.
DS_DEV void kv4_quantise16(float (&y)[16], uint32_t& scale_byte, uint2& codes, bool& bad) {
  float mx = 0.f;
  bad = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (!(fabsf(y[i]) < INFINITY)) bad = true;
    if (y[i] != y[i]) y[i] = 0.f;
    mx = fmaxf(mx, fabsf(y[i]));
  }
  const float sf = fminf(__fdiv_rn(mx, 6.f), 448.f);
  uint16_t sb;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.f), "f"(sf));
  scale_byte = sb & 0xffu;
  uint32_t s2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(sb));
  const float s = __half2float(__ushort_as_half((unsigned short)(s2 & 0xffffu)));
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    // at most 6.4 unless the scale was cut at 448: clamped before f16
    const float a = fminf(fmaxf(y[i] * inv, -8.f), 8.f);
    const float b = fminf(fmaxf(y[i + 1] * inv, -8.f), 8.f);
    const float2 q = __half22float2(__floats2half2_rn(a, b));
    uint32_t byte;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(byte)
        : "f"(q.y), "f"(q.x));
    w[i >> 3] |= byte << (4 * (i & 7));
  }
  codes = make_uint2(w[0], w[1]);
}

}  // namespace ds
