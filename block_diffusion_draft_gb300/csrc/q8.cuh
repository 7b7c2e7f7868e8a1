// q8.cuh -- the 8-bit cache formats: one code byte per channel and one
// power-of-two scale per group of 32 channels of a (row, kv head).
//
// A group's scale is 2^e with e the smallest integer for which
// amax <= qmax * 2^e (amax the group's largest magnitude, qmax 448 for e4m3
// and 127 for int8), at least -117; it is stored as the byte e + 127.  A code
// is x * 2^-e rounded to nearest even: an e4m3 number, or a sign bit and a
// 7-bit magnitude.  Because the scale is a power of two, x * 2^-e is exact in
// fp32 and code * 2^e is exact in bf16 (at most 7 significant bits, and the
// bound on e keeps every value a normal number): the rounding to the code is
// the only one between the written row and what the tensor cores read.
// Magnitudes above 2^126 are stored as 2^126.  A group that holds an infinity
// or NaN gets the scale byte 255 and reads back as NaN in every channel.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace df {

constexpr uint32_t kQ8NanByte = 255;
constexpr uint32_t kQ8MinByte = 10;        // e = -117
constexpr uint32_t kBf16MaxStored = 0x7e80;  // 2^126

// scale byte of a group whose largest magnitude has the bf16 bits `amax`
template <int FMT>
DF_DEV uint32_t q8_scale_byte(uint32_t amax) {
  if (amax >= 0x7f80u) return kQ8NanByte;
  amax = min(amax, kBf16MaxStored);
  // amax = (1 + mant / 128) * 2^(field - 127): 448 = 1.75 * 2^8 and
  // 127 = (1 + 126 / 128) * 2^6
  const int field = (int)(amax >> 7), mant = (int)(amax & 0x7fu);
  const int byte = FMT == Q8_E4M3 ? field - 8 + (mant > 96) : field - 6 + (mant > 126);
  return (uint32_t)max(byte, (int)kQ8MinByte);
}

// codes of two bf16 values (packed in `w`) scaled by `inv` = 2^-e, in the low
// 16 bits of the result
template <int FMT>
DF_DEV uint32_t q8_encode2(uint32_t w, float inv) {
  constexpr float top = 8.507059173023462e37f;  // 2^126
  float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
  lo = fminf(fmaxf(lo, -top), top) * inv;
  hi = fminf(fmaxf(hi, -top), top) * inv;
  if (FMT == Q8_E4M3) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
  }
  // |y| <= 127: adding 2^23 rounds it to the nearest even integer, which is
  // then the low byte of the sum
  const uint32_t a = __float_as_uint(fabsf(lo) + 8388608.f) & 0xffu;
  const uint32_t b = __float_as_uint(fabsf(hi) + 8388608.f) & 0xffu;
  return a | ((__float_as_uint(lo) >> 31) << 7) | (b << 8) | ((__float_as_uint(hi) >> 31) << 15);
}

DF_DEV uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

DF_DEV uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// A group's scale as the bf16 factors its codes are multiplied by.
//   int8:  f = 2^e, z = 128 * 2^e
//   e4m3:  f = 2^(120 + e), z = 0 where that is a bf16 number; otherwise
//          f = 2^120 and z = 2^e
// Scale byte 255 gives f = NaN.  q8_zero() is the scale that decodes every
// code to zero.
struct Q8Scale {
  uint32_t f, z;
};

template <int FMT>
DF_DEV Q8Scale q8_scale(uint32_t byte) {
  Q8Scale s;
  if (FMT == Q8_E4M3) {
    const bool wide = byte > 134u;
    s.f = byte == kQ8NanByte ? 0x7fff7fffu : (wide ? 247u : byte + 120u) * 0x00800080u;
    s.z = wide && byte != kQ8NanByte ? byte * 0x00800080u : 0u;
  } else {
    s.f = byte == kQ8NanByte ? 0x7fff7fffu : byte * 0x00800080u;
    s.z = (byte + 7u) * 0x00800080u & 0x7fff7fffu;
  }
  return s;
}

DF_DEV Q8Scale q8_zero() { return Q8Scale{0u, 0u}; }

// two codes (one per half of `h`) -> two bf16 values
//   int8: `h` holds each code in both bytes of its half.  With the magnitude
//   m in the mantissa of 128 the half reads +-(128 + m); times 2^e minus
//   +-128 * 2^e in one fma is +-m * 2^e, exactly.
//   e4m3: `h` holds each code in the upper byte of its half.  Its exponent
//   and mantissa moved four places down are a bf16 number of 2^-120 times
//   the code's value, subnormal codes included.
template <int FMT>
DF_DEV uint32_t q8_decode2(uint32_t h, Q8Scale s) {
  if (FMT == Q8_E4M3) {
    const uint32_t t = ((h >> 4) & 0x07f007f0u) | (h & 0x80008000u);
    const uint32_t v = mul_bf16x2(t, s.f);
    return s.z == 0u ? v : mul_bf16x2(v, s.z);
  }
  const uint32_t y = (h & 0x807f807fu) | 0x43004300u;
  const uint32_t z = (~h & 0x80008000u) | s.z;
  return fma_bf16x2(y, s.f, z);
}

// eight codes of one group -> eight bf16 values
template <int FMT>
DF_DEV uint4 q8_decode8(uint32_t c0, uint32_t c1, Q8Scale s) {
  constexpr uint32_t lo = FMT == Q8_E4M3 ? 0x1404u : 0x1100u;
  constexpr uint32_t hi = FMT == Q8_E4M3 ? 0x3424u : 0x3322u;
  uint4 r;
  r.x = q8_decode2<FMT>(__byte_perm(c0, 0u, lo), s);
  r.y = q8_decode2<FMT>(__byte_perm(c0, 0u, hi), s);
  r.z = q8_decode2<FMT>(__byte_perm(c1, 0u, lo), s);
  r.w = q8_decode2<FMT>(__byte_perm(c1, 0u, hi), s);
  return r;
}

}  // namespace df
