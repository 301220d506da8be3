// What stands before the Newton-Schulz products: the momentum, the Frobenius norm of the update
// and its two fp16 parts.  Bound by memory: the norm's pass reads G and M and writes M (12 bytes
// an element), the second reads both again and writes two parts (12 bytes); keeping U instead
// would write and read four bytes more than it saves.  16 matrices of 1376 x 4096: 154 us
// (7.0 TB/s) and 180 us (6.0 TB/s).
#include <cuda_bf16.h>

#include <algorithm>

#include "muon_update.cuh"

namespace mlpb {

constexpr int kPrepThreads = 256;
constexpr int kPrepMaxParts = kPrepThreads;

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
    add_squares4(u, s);
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

// X's two parts, eight columns of a row a thread; the pad of both buffers of X is zero.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads)
    muon_split_kernel(const MuonInput in, const float4* __restrict__ part, int parts,
                      __half* __restrict__ xh, __half* __restrict__ xh_other,
                      __half* __restrict__ xl, int ldx) {
  __shared__ float factors[2];
  const int64_t b = blockIdx.y;
  {  // a part a thread: muon_partials() is at most the number of threads
    __shared__ double warps[kPrepThreads / 32];
    double t = static_cast<int>(threadIdx.x) < parts ? whole_square(part[b * parts + threadIdx.x])
                                                     : 0.0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kPrepThreads / 32; ++w) t += warps[w];
      norm_factors(t, factors[0], factors[1]);
    }
    __syncthreads();
  }
  const float s1 = factors[0], s2 = factors[1] * kXScale;
  const int64_t elems = in.rows * in.cols;
  const int groups = ldx / 8;
  const int64_t pieces = in.rows * groups;
  const bool vec = in.cols % 4 == 0, pairs = in.cols % 2 == 0;
  const T* g = static_cast<const T*>(in.g) + b * elems;
  float* m = in.m == nullptr ? nullptr : in.m + b * elems;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kPrepThreads;
  const int64_t rows_on = stride / groups;  // no division in the loop
  const int groups_on = static_cast<int>(stride - rows_on * groups);
  int64_t i = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x;
  int64_t row = i / groups;
  int group = static_cast<int>(i - row * groups);
#pragma unroll 2
  for (; i < pieces; i += stride) {
    const int64_t col = static_cast<int64_t>(group) * 8;
    __half hi[8], lo[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t c = col + 4 * h;
      const int n = static_cast<int>(max(static_cast<int64_t>(0),
                                         min(static_cast<int64_t>(4), in.cols - c)));
      float u[4] = {0.f, 0.f, 0.f, 0.f};
      const int64_t o = row * in.cols + c;
      if (n > 0)
        update4<false>(g + o, m == nullptr ? nullptr : m + o, n, vec, in.momentum, in.nesterov, u,
                       pairs);
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
    row += rows_on;
    group += groups_on;
    if (group >= groups) {
      group -= groups;
      ++row;
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
  const int64_t most = std::max<int64_t>(1, 1216 / in.batch);
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
