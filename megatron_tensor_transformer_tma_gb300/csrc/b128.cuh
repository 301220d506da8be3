// Block-scaled E4M3: one power-of-two scale for each 128 consecutive columns of a row (or of
// 128 rows, for a weight), stored as a byte of exponent.
//
// With amax the block's largest magnitude, k is the largest integer, at most 126, with
// amax 2^k <= 448 (0 for zeros); a code is e4m3(x 2^k), nearest, ties to even, and the scale byte
// is 127 - k, so that a code c stands for c 2^(byte - 127), exactly.  Blocks that hold an infinity
// or a NaN have the byte 255 and NaN codes, and stand for NaN throughout.
//
// Scale bytes lie in the order in which the tensor cores take them: for four consecutive blocks
// of a row a 32-bit word, for 128 rows 32 lanes of four words (rows l, l + 32, l + 64, l + 96),
// 512 bytes that one bulk copy and one copy into tensor memory move:
//   byte(row, kb) at ((kb / 4) * ceil(rows / 128) + row / 128) * 512
//                    + (row % 32) * 16 + (row % 128) / 32 * 4 + kb % 4
// Bytes of rows and blocks past the end are 127 (a scale of one).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "fp8.cuh"

namespace mlpb {

constexpr int kB128 = 128;           // columns that share a scale
constexpr int kB128Chunk = 512;      // scale bytes of 128 rows and four blocks
constexpr uint32_t kB128One = 127u;  // scale byte of 1
constexpr uint32_t kB128Nan = 255u;

__host__ __device__ constexpr int64_t b128_ld(int64_t cols) { return (cols + 15) / 16 * 16; }

__host__ __device__ constexpr int64_t b128_blocks(int64_t n) { return (n + kB128 - 1) / kB128; }

__host__ __device__ constexpr int64_t b128_scale_bytes(int64_t rows, int64_t cols) {
  return (b128_blocks(cols) + 3) / 4 * b128_blocks(rows) * kB128Chunk;
}

// Scale byte of a block whose largest magnitude has these fp32 bits.
__device__ __forceinline__ uint32_t b128_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return kB128Nan;
  if (amax_bits == 0u) return kB128One;
  // 448 = 1.75 2^8; below 2^-126 every k is past 126
  const int e = static_cast<int>(amax_bits >> 23) - 127;
  const int k = min(((amax_bits & 0x7fffffu) <= 0x600000u ? 8 : 7) - e, 126);
  return static_cast<uint32_t>(127 - k);
}

// 2^k for a scale byte 127 - k: what a value is multiplied by before it is rounded (exact: k is
// in [-120, 126]).  NaN for the byte 255.
__device__ __forceinline__ float b128_to_codes(uint32_t byte) {
  return byte == kB128Nan ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - byte) << 23);
}

// Four values times f as E4M3 codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t b128_pack4(float a, float b, float c, float d, float f) {
  return e4m3x2(a * f, b * f) | (e4m3x2(c * f, d * f) << 16);
}

cudaError_t launch_b128_quantize(const void* x, bool f32, int64_t rows, int64_t cols, bool square,
                                 void* q, void* qs, void* qt, void* qts, cudaStream_t s);

}  // namespace mlpb
