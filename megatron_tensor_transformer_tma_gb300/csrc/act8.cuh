// 8-bit activation checkpoints: 32 consecutive features of a row (a block) become signed
// 8-bit codes with one power-of-two scale.
//
// With amax the block's largest |z| and k the largest integer such that amax 2^k <= 127
// (k <= 126; k = 0 for a block of zeros), code = z 2^k rounded to the nearest integer, ties
// to even, and the scale byte e = 127 - k is the biased exponent of a code's step 2^-k.
// z 2^k, the rounding and code 2^-k are exact in fp32, and code 2^-k is exact in bf16 too
// (7 bits of magnitude), so the codes are a pure function of the bf16 values.  bf16's largest
// value, 127.5 2^121, would so become 64 2^122, an infinity: its block has k = -121 all the same,
// and codes rounded with ties towards zero (127 for it, half a step off like any other).  Signed
// integers rather than E4M3: a block of 32 normal values reaches about 2 sigma, so the step
// is 2^-6 to 2^-5 sigma everywhere, where E4M3's step is 2^-4 to 2^-3 of the value itself
// (a million normal values, each format with its block's power-of-two scale: rms error 0.8 %
// of sigma against 2.7 %).
// A block that holds an infinity or a NaN gets e = 255 and decodes to NaN in all 32 places,
// so that an overflow in the forward is seen in the gradients.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace mlpb {

constexpr int kActBlock = 32;           // features that share a scale
constexpr uint32_t kActNanScale = 255u;  // scale byte of a block with a non-finite value

// max over two packed |bf16| pairs, as 16-bit lanes (|x| is the bits without the sign, and
// the bit patterns of non-negative floats order like the values; NaN is above infinity).
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7fff7fffu);
}

// Scale byte of a block from the bits of its largest |bf16| (exponent E, mantissa M):
// 127 = (2 - 2^-6) 2^6, so k = 133 - E, one less when 1.M > 2 - 2^-6, that is M = 0x7f, but not
// below -121.
__device__ __forceinline__ uint32_t act8_scale_byte(uint32_t amax16) {
  if (amax16 >= 0x7f80u) return kActNanScale;
  const int E = static_cast<int>(amax16 >> 7);
  const int k =
      amax16 == 0u ? 0 : max(-121, min(126, 133 - E - ((amax16 & 0x7fu) == 0x7fu ? 1 : 0)));
  return static_cast<uint32_t>(127 - k);
}

// 2^k, the factor that takes values to codes, of a scale byte and its block's largest |bf16| (any
// finite value for 255; the next one below 2^k where that is bf16's largest).
__device__ __forceinline__ float act8_to_codes(uint32_t e, uint32_t amax16) {
  return __uint_as_float((min(254u - e, 253u) << 23) - (amax16 == 0x7f7fu ? 1u : 0u));
}

// 2^-k, a code's step; NaN for 255 (0 is the subnormal 2^-127).
__device__ __forceinline__ float act8_step(uint32_t e) {
  const uint32_t b = e == kActNanScale ? 0x7fffffffu : e == 0u ? 0x00400000u : e << 23;
  return __uint_as_float(b);
}

// Four values times 2^k (f), rounded to the nearest integer, as the bytes of a word.  Adding
// 1.5 2^23 leaves the integer, rounded to nearest even, in the low bits of the sum.  Values
// of a non-finite block give bytes that mean nothing.
__device__ __forceinline__ uint32_t act8_pack4(float a, float b, float c, float d, float f) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t x = __float_as_uint(fmaf(a, f, kMagic)), y = __float_as_uint(fmaf(b, f, kMagic));
  const uint32_t z = __float_as_uint(fmaf(c, f, kMagic)), w = __float_as_uint(fmaf(d, f, kMagic));
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

// The four values of a word of codes with step s.  A code's byte with its sign bit flipped
// (code + 128) in the low byte of 2^23 reads as 2^23 + 128 + code.
__device__ __forceinline__ void act8_unpack4(uint32_t w, float s, float (&v)[4]) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.0f) * s;
}

}  // namespace mlpb
