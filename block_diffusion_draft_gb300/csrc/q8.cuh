// q8.cuh -- the 8-bit cache formats: one code byte per channel and one
// power-of-two scale per group of 32 channels of a (row, kv head).
//
// A group's scale is 2^e with e the smallest integer for which
// amax <= qmax * 2^e (amax the group's largest magnitude, qmax 448 for e4m3
// and 127 for int8), at least -117; it is stored as the byte e + 127, and as
// 0 for a group of zeros.  A code is x * 2^-e rounded to nearest even: an
// e4m3 number, or an integer plus 128.  Because the scale is a power of two,
// x * 2^-e is exact in fp32 and code * 2^e is exact in bf16 (at most 7
// significant bits, and the bound on e keeps every value a normal number):
// the rounding to the code is the only one between the written row and what
// the tensor cores read.  Magnitudes above 2^126 are stored as 2^126.  A
// group that holds an infinity or NaN gets the scale byte 255 and reads back
// as NaN in every channel.
//
// Decoding is what bounds the attention over such a cache, and fp16 decodes in
// half the instructions of bf16 (two per pair of channels: a byte permute
// that puts the code into the mantissa of 1024, and a fused multiply-add that
// takes 1152 off and applies the scale; or e4m3's own conversion and a
// multiply).  Its range is 20 binades of scale, so every (sequence, kv head)
// keeps the smallest and largest scale byte of its groups, zero groups apart:
// while they lie within kHalfSpan of one another, and no group reads NaN, the
// codes are decoded to fp16 relative to 2^(largest - kHalfTop), exactly;
// otherwise to bf16.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace df {

constexpr uint32_t kQ8NanByte = 255;
constexpr uint32_t kQ8MinByte = 10;          // e = -117
constexpr uint32_t kBf16MaxStored = 0x7e80;  // 2^126
// fp16 factors 2^k with k in [-14, 5] are normal, 1152 * 2^5 and 448 * 2^5
// do not overflow, and 2^-9 * 2^-14 (e4m3's smallest step) is representable
constexpr int kHalfTop = 5, kHalfSpan = 19;
constexpr int kHalfMinUnit = 15;  // smallest k0: bytes from kQ8MinByte are in its range

// scale byte of a group whose largest magnitude has the bf16 bits `amax`
template <int FMT>
DF_DEV uint32_t q8_scale_byte(uint32_t amax) {
  // amax = (1 + mant / 128) * 2^(field - 127): 448 = 1.75 * 2^8 and
  // 127 = (1 + 126 / 128) * 2^6, so that the byte is field - 8 + (mant > 96) and
  // field - 6 + (mant > 126); the comparison is a carry into the field
  const int t = (int)min(amax, kBf16MaxStored);
  const int byte = FMT == Q8_E4M3 ? ((t + 31) >> 7) - 8 : ((t + 1) >> 7) - 6;
  const uint32_t b = (uint32_t)max(byte, (int)kQ8MinByte);
  return amax >= 0x7f80u ? kQ8NanByte : amax == 0u ? 0u : b;
}

// two bf16 values, their magnitudes at most 2^126 (NaN and infinity, too)
DF_DEV uint32_t q8_clamp2(uint32_t w) {
  return (w & 0x80008000u) | __vminu2(w & 0x7fff7fffu, 0x7e807e80u);
}

// codes of four bf16 values (two in each word) scaled by `inv` = 2^-e, exactly
// but for what is far below half a code
template <int FMT>
DF_DEV uint32_t q8_encode4(uint32_t w0, uint32_t w1, float inv) {
  const float a = __uint_as_float(w0 << 16), b = __uint_as_float(w0 & 0xffff0000u);
  const float c = __uint_as_float(w1 << 16), d = __uint_as_float(w1 & 0xffff0000u);
  if (FMT == Q8_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
    return lo | (uint32_t)hi << 16;
  }
  // |y| <= 127: adding 2^23 + 128 rounds to the nearest even integer (the
  // product is exact), and the low byte of the sum is that integer plus 128
  constexpr float add = 8388736.f;
  const uint32_t ab = __byte_perm(__float_as_uint(__fmaf_rn(a, inv, add)),
                                  __float_as_uint(__fmaf_rn(b, inv, add)), 0x0040u);
  const uint32_t cd = __byte_perm(__float_as_uint(__fmaf_rn(c, inv, add)),
                                  __float_as_uint(__fmaf_rn(d, inv, add)), 0x0040u);
  return __byte_perm(ab, cd, 0x5410u);
}

DF_DEV uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

DF_DEV uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// two e4m3 codes -> two fp16 values
DF_DEV uint32_t e4m3x2_f16x2(uint32_t codes16) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)codes16));
  return d;
}

// The scales of a row's four groups as fp16 factors relative to 2^-k0, one
// group per byte: 2^k with k = byte - k0 in [-14, 5] is (k + 15) << 10, all of
// it in the upper byte, and so is -1152 * 2^k but for a lower byte of 0x80.
// (The bytes' differences are the digits of one 32-bit product and sum.)  A
// zero group's byte is replaced by k = -14: its codes decode to zero.
struct HalfScales {
  uint32_t f, z;
};

DF_DEV HalfScales half_scales(uint32_t bytes, int k0) {
  const uint32_t low = (uint32_t)(k0 - 14) * 0x01010101u;
  if (((bytes - 0x01010101u) & ~bytes & 0x80808080u) != 0u)
    bytes |= __vcmpeq4(bytes, 0u) & low;
  HalfScales s;
  s.f = bytes * 4u - (uint32_t)(k0 - 15) * 0x04040404u;
  s.z = s.f + 0xa8a8a8a8u;
  return s;
}

// byte selector of group g's factor, for both halves of a register
DF_DEV uint32_t half_select(int g) { return 0x0404u | (uint32_t)g << 4 | (uint32_t)g << 12; }

// sixteen codes of the group `select`ed -> sixteen fp16 values
template <int FMT>
DF_DEV void half_decode16(uint4 c, HalfScales s, uint32_t select, uint4& a, uint4& b) {
  const uint32_t f = __byte_perm(s.f, 0u, select);
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t v[8];
  if (FMT == Q8_E4M3) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = mul_f16x2(e4m3x2_f16x2(w[i]), f);
      v[2 * i + 1] = mul_f16x2(e4m3x2_f16x2(w[i] >> 16), f);
    }
  } else {
    const uint32_t z = __byte_perm(s.z, 0x80808080u, select);
    constexpr uint32_t m = 0x64646464u;  // upper bytes: 1024 + code
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = fma_f16x2(__byte_perm(w[i], m, 0x4140u), f, z);
      v[2 * i + 1] = fma_f16x2(__byte_perm(w[i], m, 0x4342u), f, z);
    }
  }
  a = make_uint4(v[0], v[1], v[2], v[3]);
  b = make_uint4(v[4], v[5], v[6], v[7]);
}

// two codes (low 16 bits) -> two bf16 values; `scale` = 2^e (0 for a zero
// group, NaN for a group that reads NaN)
template <int FMT>
DF_DEV uint32_t bf16_decode2(uint32_t codes16, float scale) {
  const uint32_t h = FMT == Q8_E4M3
                         ? e4m3x2_f16x2(codes16)
                         : fma_f16x2(__byte_perm(codes16, 0x64646464u, 0x4140u), 0x3c003c00u,
                                     0xe480e480u);
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(v.x * scale, v.y * scale);
}

DF_DEV float bf16_scale(uint32_t byte) {
  return byte == kQ8NanByte ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte << 23);
}

// eight codes of one group -> eight bf16 values
template <int FMT>
DF_DEV uint4 bf16_decode8(uint32_t c0, uint32_t c1, float scale) {
  uint4 r;
  r.x = bf16_decode2<FMT>(c0, scale);
  r.y = bf16_decode2<FMT>(c0 >> 16, scale);
  r.z = bf16_decode2<FMT>(c1, scale);
  r.w = bf16_decode2<FMT>(c1 >> 16, scale);
  return r;
}

}  // namespace df
