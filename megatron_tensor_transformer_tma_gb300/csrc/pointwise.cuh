// The activations' pointwise math, shared by the GEMM epilogues and the 8-bit activation
// checkpoints.
#pragma once

#include <cstdint>

namespace mlpb {

// tanh-form GELU written with s = sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3): since
// 1 + tanh(u) = 2 sigmoid(2u), gelu(z) = z s, the same function without cancellation for
// z << 0, and gelu'(z) = s + z s (1 - s) 2 sqrt(2/pi) (1 + 3 * 0.044715 z^2).  The
// constants are folded so that e^{-2u} = 2^{z (a + b z^2)} is one base-2 exponential:
//   a = -2k log2(e), b = -2k c log2(e),  k = sqrt(2/pi), c = 0.044715.
// For |z| past ~10 the exponential overflows to +inf (s = 0) or underflows to 0 (s = 1),
// and both forms then return their limits (0 and z; 0 and 1): s (1 - s) is exactly 0, and its
// factor, past fp32's range from |z| of about 1.2e13 on, is held inside it, so that no finite z
// meets inf * 0 (8-bit checkpoints, GELU T 8192 F 20480: the gradient takes 183 us with it, 181
// without; the step of the block is the same).
constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluA = -2.0f * kSqrt2OverPi * kLog2e;               // -2k log2(e)
constexpr float kGeluB = -2.0f * kSqrt2OverPi * kGeluCubic * kLog2e;  // -2kc log2(e)
constexpr float kGeluD0 = 2.0f * kSqrt2OverPi;                        // 2k
constexpr float kGeluD2 = 6.0f * kSqrt2OverPi * kGeluCubic;           // 6kc

__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// 2^x (the MUFU base-2 exponential; subnormal results flush to zero).
__device__ __forceinline__ float ex2_f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 values in one 64-bit register (lo in the low half) and the f32x2 arithmetic
// of the sm_100 family: one instruction for both lanes, each rounded as its fp32 form.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// e^{-2u} + 1 for two values of z (one MUFU exponential each), and its reciprocal s.
__device__ __forceinline__ uint64_t gelu_s_x2(uint64_t z, uint64_t z2) {
  float u0, u1, d0, d1;
  f2_unpack(f2_mul(z, f2_fma(z2, f2_pack(kGeluB, kGeluB), f2_pack(kGeluA, kGeluA))), u0, u1);
  f2_unpack(f2_add(f2_pack(ex2_f(u0), ex2_f(u1)), f2_pack(1.0f, 1.0f)), d0, d1);
  return f2_pack(__fdividef(1.0f, d0), __fdividef(1.0f, d1));
}

// gelu(z) = z s for two values.
__device__ __forceinline__ uint64_t gelu_x2(uint64_t z) { return f2_mul(z, gelu_s_x2(z, f2_mul(z, z))); }

// The value with x's sign and the lesser magnitude of x and `most` (x not NaN).
__device__ __forceinline__ float hold_f(float x, float most) {
  asm("min.xorsign.abs.f32 %0, %0, %1;" : "+f"(x) : "f"(most));
  return x;
}

// d = 2k z (1 + 3c z^2) for two values, an infinity as fp32's largest value.
__device__ __forceinline__ uint64_t gelu_factor_x2(uint64_t z, uint64_t z2) {
  constexpr float kMost = 3.4028234663852886e38f;
  float a, b;
  f2_unpack(f2_mul(z, f2_fma(z2, f2_pack(kGeluD2, kGeluD2), f2_pack(kGeluD0, kGeluD0))), a, b);
  return f2_pack(hold_f(a, kMost), hold_f(b, kMost));
}

// gelu'(z) = s + d s (1 - s) for two values.
__device__ __forceinline__ uint64_t gelu_grad_x2(uint64_t z) {
  const uint64_t z2 = f2_mul(z, z);
  const uint64_t s = gelu_s_x2(z, z2);
  const uint64_t d = gelu_factor_x2(z, z2);
  return f2_fma(d, f2_sub(s, f2_mul(s, s)), s);
}

// gelu'(z), and gelu(z) in `gelu`, for two values: one exponential and reciprocal each for both.
__device__ __forceinline__ uint64_t gelu_both_x2(uint64_t z, uint64_t& gelu) {
  const uint64_t z2 = f2_mul(z, z);
  const uint64_t s = gelu_s_x2(z, z2);
  const uint64_t d = gelu_factor_x2(z, z2);
  gelu = f2_mul(z, s);
  return f2_fma(d, f2_sub(s, f2_mul(s, s)), s);
}

}  // namespace mlpb
