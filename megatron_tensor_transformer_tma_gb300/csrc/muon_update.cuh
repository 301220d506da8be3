// The update that is orthogonalised, element by element, and its norm (shared by the kernels that
// begin with them).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "muon.cuh"

namespace mlpb {

// Four consecutive elements, n of them valid: in pairs where these lie on 8 bytes (bf16: 4).
template <typename T>
__device__ __forceinline__ void load_some(const T* x, int n, bool pairs, float (&u)[4]) {
  if (pairs) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      u[e] = u[e + 1] = 0.0f;
      if (e < n) {  // n is even
        if constexpr (sizeof(T) == 2) {
          const float2 f = unpack_bf16x2(*reinterpret_cast<const uint32_t*>(x + e));
          u[e] = f.x;
          u[e + 1] = f.y;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(x + e);
          u[e] = f.x;
          u[e + 1] = f.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = e < n ? static_cast<float>(x[e]) : 0.0f;
  }
}

// G and, unless m is NULL, M of four consecutive elements (n of them valid; `vec`: on 16 bytes).
template <typename T>
__device__ __forceinline__ void load4(const T* g, const float* m, int n, bool vec, bool pairs,
                                      float (&u)[4], float (&v)[4]) {
  if (!vec) {
    load_some(g, n, pairs, u);
  } else if constexpr (sizeof(T) == 2) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(g));
    const float2 x = unpack_bf16x2(w.x), y = unpack_bf16x2(w.y);
    u[0] = x.x; u[1] = x.y; u[2] = y.x; u[3] = y.y;
  } else {
    const float4 x = __ldg(reinterpret_cast<const float4*>(g));
    u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
  }
  if constexpr (sizeof(T) == 4) {
    if (m == nullptr) return;
    if (!vec) {
      load_some(m, n, pairs, v);
    } else {
      const float4 x = *reinterpret_cast<const float4*>(m);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
  }
}

// Their U in u, M written back by the first pass.
template <bool kFirst, typename T>
__device__ __forceinline__ void finish4(float* m, int n, bool vec, float mu, int nesterov,
                                        float (&u)[4], float (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    if (m == nullptr) return;
    if constexpr (kFirst) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmaf(mu, v[e], u[e]);
      if (vec) {
        *reinterpret_cast<float4*>(m) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < n) m[e] = v[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = nesterov ? fmaf(mu, v[e], u[e]) : v[e];
  }
}

// U of four consecutive elements at once.
template <bool kFirst, typename T>
__device__ __forceinline__ void update4(const T* g, float* m, int n, bool vec, float mu,
                                        int nesterov, float (&u)[4], bool pairs = false) {
  float v[4];
  load4(g, m, n, vec, pairs, u, v);
  finish4<kFirst, T>(m, n, vec, mu, nesterov, u, v);
}

// Sums of squares in three ranges (after Blue, 1978), so that neither large nor small values
// leave fp32's range: x small of 2^-40, large of 2^40, the rest.
constexpr float kTiny = 9.094947017729282e-13f;   // 2^-40
constexpr float kHuge = 1.099511627776e12f;       // 2^40
constexpr float kUp = 1.2089258196146292e24f;     // 2^80
constexpr float kDown = 8.271806125530277e-25f;   // 2^-80

__device__ __forceinline__ void add_square(float x, float4& s) {
  const float a = fabsf(x);
  if (a < kTiny) {
    const float y = x * kUp;
    s.x = fmaf(y, y, s.x);
  } else if (a <= kHuge) {
    s.y = fmaf(x, x, s.y);
  } else {  // NaN too
    const float y = x * kDown;
    s.z = fmaf(y, y, s.z);
  }
}

// Four at once: all in the middle range, as a rule.
__device__ __forceinline__ void add_squares4(const float (&u)[4], float4& s) {
  const float a = fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3])));
  const float b = fminf(fminf(fabsf(u[0]), fabsf(u[1])), fminf(fabsf(u[2]), fabsf(u[3])));
  if (b >= kTiny && a <= kHuge) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s.y = fmaf(u[e], u[e], s.y);
    s.z += (u[0] + u[1] + u[2] + u[3]) * 0.0f;  // maxima and minima leave a NaN out
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) add_square(u[e], s);
  }
}

__device__ __forceinline__ double whole_square(float4 p) {
  return static_cast<double>(p.x) * 6.842277657836021e-49 + static_cast<double>(p.y) +
         static_cast<double>(p.z) * 1.461501637330903e48;  // 2^-160, 2^160
}

// x = (u s1) s2 for u / |U|: two factors, since 1 / |U| may be past fp32's range.
__device__ __forceinline__ void norm_factors(double square, float& s1, float& s2) {
  const double norm = sqrt(square);
  s2 = 1.0f;
  if (norm == 0.0) {  // a zero matrix stays zero
    s1 = 0.0f;
  } else if (!(norm < 1e60)) {  // a NaN goes through; with infinities NaN at them, zero elsewhere
    s1 = isnan(norm) ? static_cast<float>(norm) : 0.0f;
  } else {
    int e;
    const double f = frexp(norm, &e);  // norm = f 2^e; e in [-148, 160]
    s1 = ldexpf(1.0f, -(e / 2));
    s2 = ldexpf(static_cast<float>(1.0 / f), -(e - e / 2));
  }
}

}  // namespace mlpb
