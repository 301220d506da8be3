// What stands before the Newton-Schulz products: the momentum, the Frobenius norm of the update
// and its two fp16 parts.  Bound by memory: the norm's pass reads G and M and writes M (12 bytes
// an element), the second reads both again and writes two parts (12 bytes); keeping U instead
// would write and read four bytes more than it saves.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "muon.cuh"

namespace mlpb {

constexpr int kPrepThreads = 256;
constexpr int kPrepMaxParts = 512;

// U of four consecutive elements (n of them valid), M written back by the first pass.
template <bool kFirst, typename T>
__device__ __forceinline__ void update4(const T* g, float* m, int n, bool vec, float mu,
                                        int nesterov, float (&u)[4]) {
  if constexpr (sizeof(T) == 2) {
    if (vec) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(g));
      const float2 x = unpack_bf16x2(w.x), y = unpack_bf16x2(w.y);
      u[0] = x.x; u[1] = x.y; u[2] = y.x; u[3] = y.y;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = e < n ? __bfloat162float(g[e]) : 0.0f;
    }
  } else {
    if (vec) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(g));
      u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = e < n ? g[e] : 0.0f;
    }
    if (m != nullptr) {
      float v[4];
      if (vec) {
        const float4 x = *reinterpret_cast<const float4*>(m);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = e < n ? m[e] : 0.0f;
      }
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

template <typename T>
__global__ void __launch_bounds__(kPrepThreads) muon_norm_kernel(const MuonInput in,
                                                                 float4* __restrict__ part) {
  const int64_t elems = in.rows * in.cols;
  const int64_t base = static_cast<int64_t>(blockIdx.y) * elems;
  const T* g = static_cast<const T*>(in.g) + base;
  float* m = in.m == nullptr ? nullptr : in.m + base;
  const bool vec = elems % 4 == 0;  // tensors are 16-byte aligned, matrices then too
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kPrepThreads * 4;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x) * 4; i < elems;
       i += stride) {
    float u[4];
    const int n = static_cast<int>(min(static_cast<int64_t>(4), elems - i));
    update4<true>(g + i, m == nullptr ? nullptr : m + i, n, vec, in.momentum, in.nesterov, u);
    const float a = fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3])));
    const float b = fminf(fminf(fabsf(u[0]), fabsf(u[1])), fminf(fabsf(u[2]), fabsf(u[3])));
    if (b >= kTiny && a <= kHuge) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s.y = fmaf(u[e], u[e], s.y);
      // max and min leave a NaN out: it is added by the comparisons' failing elsewhere
      s.z += (u[0] + u[1] + u[2] + u[3]) * 0.0f;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) add_square(u[e], s);
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
  }
  __shared__ float4 warps[kPrepThreads / 32];
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kPrepThreads / 32; ++w) {
      s.x += warps[w].x;
      s.y += warps[w].y;
      s.z += warps[w].z;
    }
    part[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = s;
  }
}

// x = (u s1) s2 for u / |U|: two factors, since 1 / |U| may be past fp32's range.  A warp's work;
// the order of the sum is fixed.
__device__ __forceinline__ void norm_factors(const float4* part, int parts, float& s1, float& s2) {
  double t = 0.0;
  for (int i = threadIdx.x & 31; i < parts; i += 32) {
    const float4 p = part[i];
    t += static_cast<double>(p.x) * 6.842277657836021e-49 + static_cast<double>(p.y) +
         static_cast<double>(p.z) * 1.461501637330903e48;  // 2^-160, 2^160
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const double norm = sqrt(t);
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

// X's two parts, eight columns of a row a thread; the pad of both buffers of X is zero.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads)
    muon_split_kernel(const MuonInput in, const float4* __restrict__ part, int parts,
                      __half* __restrict__ xh, __half* __restrict__ xh_other,
                      __half* __restrict__ xl, int ldx) {
  __shared__ float factors[2];
  const int64_t b = blockIdx.y;
  if (threadIdx.x < 32) {
    float f1, f2;
    norm_factors(part + b * parts, parts, f1, f2);
    if (threadIdx.x == 0) {
      factors[0] = f1;
      factors[1] = f2;
    }
  }
  __syncthreads();
  const float s1 = factors[0], s2 = factors[1] * kXScale;
  const int64_t elems = in.rows * in.cols;
  const int groups = ldx / 8;
  const int64_t pieces = in.rows * groups;
  const bool vec = in.cols % 4 == 0;
  const T* g = static_cast<const T*>(in.g) + b * elems;
  float* m = in.m == nullptr ? nullptr : in.m + b * elems;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x; i < pieces;
       i += static_cast<int64_t>(gridDim.x) * kPrepThreads) {
    const int64_t row = i / groups;
    const int64_t col = (i - row * groups) * 8;
    __half hi[8], lo[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t c = col + 4 * h;
      const int n = static_cast<int>(max(static_cast<int64_t>(0),
                                         min(static_cast<int64_t>(4), in.cols - c)));
      float u[4] = {0.f, 0.f, 0.f, 0.f};
      const int64_t o = row * in.cols + c;
      if (n > 0)
        update4<false>(g + o, m == nullptr ? nullptr : m + o, n, vec, in.momentum, in.nesterov, u);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = e < n ? (u[e] * s1) * s2 : 0.0f;
        hi[4 * h + e] = __float2half_rn(x);
        lo[4 * h + e] = __float2half_rn(x - __half2float(hi[4 * h + e]));
      }
    }
    const int64_t o = (b * in.rows + row) * ldx + col;
    *reinterpret_cast<uint4*>(xh + o) = *reinterpret_cast<const uint4*>(hi);
    *reinterpret_cast<uint4*>(xl + o) = *reinterpret_cast<const uint4*>(lo);
    if (col + 8 > in.cols) {  // the pad of the buffer that the first step writes
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e >= in.cols) xh_other[o + e] = __half(0.0f);
    }
  }
}

int muon_partials(int64_t elems, int64_t batch) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kPrepMaxParts, 2432 / batch));
  return static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(most, (elems + 4 * kPrepThreads - 1) /
                                                       (4 * kPrepThreads))));
}

cudaError_t launch_muon_norm(const MuonInput& in, float4* part, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(muon_partials(in.rows * in.cols, in.batch)),
                  static_cast<unsigned>(in.batch));
  if (in.g_f32)
    muon_norm_kernel<float><<<grid, kPrepThreads, 0, s>>>(in, part);
  else
    muon_norm_kernel<__nv_bfloat16><<<grid, kPrepThreads, 0, s>>>(in, part);
  return cudaGetLastError();
}

cudaError_t launch_muon_split(const MuonInput& in, const float4* part, __half* xh,
                              __half* xh_other, __half* xl, int ldx, cudaStream_t s) {
  const int64_t pieces = in.rows * (ldx / 8);
  const int64_t most = std::max<int64_t>(1, 4864 / in.batch);
  const dim3 grid(static_cast<unsigned>(
                      std::min<int64_t>(most, (pieces + kPrepThreads - 1) / kPrepThreads)),
                  static_cast<unsigned>(in.batch));
  const int parts = muon_partials(in.rows * in.cols, in.batch);
  if (in.g_f32)
    muon_split_kernel<float><<<grid, kPrepThreads, 0, s>>>(in, part, parts, xh, xh_other, xl, ldx);
  else
    muon_split_kernel<__nv_bfloat16>
        <<<grid, kPrepThreads, 0, s>>>(in, part, parts, xh, xh_other, xl, ldx);
  return cudaGetLastError();
}

}  // namespace mlpb
