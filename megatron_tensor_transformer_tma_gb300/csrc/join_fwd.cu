// Forward of the join between two blocks (join.cuh).
#include "../../include/mlpb.h"
#include "join.cuh"

namespace mlpb {

// Mean and 1/sqrt(mean square + eps) of the row in v; LayerNorm by the two-pass method (the
// mean, then the squared deviations from it), so that a common offset costs no digits.
template <int kTpr, bool kSplit>
__device__ __forceinline__ void join_stats(const float (&v)[kJoinVpt][8],
                                           const JoinCols<kSplit, kTpr>& jc, int kind, float inv_h,
                                           float eps, float2* sh, int& par, float& mu, float& rs) {
  mu = 0.f;
  if (kind == MLPB_NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < kJoinVpt; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[k][e];  // zeros past the row's end
    join_sum<kTpr, 1>(s, sh, par);
    mu = s[0] * inv_h;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int k = 0; k < kJoinVpt; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = jc.ok[k][e / 4] ? v[k][e] - mu : 0.f;
      q[0] = fmaf(d, d, q[0]);
    }
  join_sum<kTpr, 1>(q, sh, par);
  rs = rsqrtf(q[0] * inv_h + eps);
}

// 64 registers a thread: 1024 threads an SM.
template <class XT, class YT, int kTpr>
__global__ void __launch_bounds__(join_threads(kTpr), 1024 / join_threads(kTpr))
    join_fwd_kernel(const JoinParams p) {
  constexpr int NT = join_threads(kTpr);
  constexpr int kRows = NT / kTpr;
  constexpr bool kSplit = sizeof(XT) == 4 || sizeof(YT) == 4;
  extern __shared__ __align__(16) uint8_t join_smem[];
  __shared__ float2 sh[2 * NT / 32];
  const int tr = threadIdx.x % kTpr;
  const JoinCols<kSplit, kTpr> jc(tr, p.H);
  const uint32_t x_bytes = NT * join_slot<XT>();
  const uint32_t stage = x_bytes + (p.has_block ? NT * join_slot<YT>() : 0);
  const uint32_t base = smem_u32(join_smem);
  const XT* X = static_cast<const XT*>(p.X);
  const YT* Y = static_cast<const YT*>(p.Y);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const float inv_h = 1.0f / static_cast<float>(p.H);
  const float alpha = p.alpha != nullptr ? *p.alpha : 1.0f;

  auto issue = [&](int b, int64_t row) {
    if (row < p.T) {
      join_copy<XT>(base + b * stage, NT, X + row * p.H, jc);
      if (p.has_block) join_copy<YT>(base + b * stage + x_bytes, NT, Y + row * p.H, jc);
    }
    cp_async_commit();
  };
  for (int b = 0; b < p.nbuf; ++b) issue(b, row0 + b * step);

  int b = 0, par = 0;
  for (int64_t row = row0; row < p.T; row += step) {
    cp_async_wait_ring(p.nbuf);
    const uint8_t* xs = join_smem + b * stage;
    float v[kJoinVpt][8];
    float mu_y = 0.f, rs_y = 0.f, mu_h = 0.f, rs_h = 0.f;
    if (p.has_block) {
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k) join_read<YT>(xs + x_bytes, NT, k, jc, v[k]);
      if (p.post != MLPB_NORM_NONE)
        join_stats<kTpr>(v, jc, p.post, inv_h, p.eps, sh, par, mu_y, rs_y);
      const __nv_bfloat16* gate =
          p.gate == nullptr ? nullptr
          : p.G == 1        ? p.gate
                            : p.gate + (static_cast<uint32_t>(row) /
                                        static_cast<uint32_t>(p.rows_per_group)) *
                                           static_cast<int64_t>(p.H);
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k) {
        if (p.post != MLPB_NORM_NONE) {
          float g[8];
          join_load<__nv_bfloat16, kSplit, kTpr, true>(p.gamma_post, k, jc, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[k][e] = (v[k][e] - mu_y) * rs_y * g[e];
          if (p.beta_post != nullptr) {
            join_load<__nv_bfloat16, kSplit, kTpr, true>(p.beta_post, k, jc, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] += g[e];
          }
        }
        if (gate != nullptr) {
          float g[8];
          join_load<__nv_bfloat16, kSplit, kTpr, true>(gate, k, jc, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[k][e] *= g[e];
        }
        float x[8];
        join_read<XT>(xs, NT, k, jc, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = fmaf(alpha, x[e], v[k][e]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k) join_read<XT>(xs, NT, k, jc, v[k]);
    }
    issue(b, row + p.nbuf * step);  // the slots of this row have been read
    if (++b == p.nbuf) b = 0;
    // The norm is that of the stream as it is stored (rounded, where it is bf16): what a
    // backward that reads Xout differentiates.
    if (p.has_block) {
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k)
        join_store<XT>(static_cast<XT*>(p.Xout) + row * p.H, k, jc, v[k]);
    }
    if (p.pre != MLPB_NORM_NONE) {
      join_stats<kTpr>(v, jc, p.pre, inv_h, p.eps, sh, par, mu_h, rs_h);
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k) {
        float g[8];
        join_load<__nv_bfloat16, kSplit, kTpr, true>(p.gamma_pre, k, jc, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = (v[k][e] - mu_h) * rs_h * g[e];
        if (p.beta_pre != nullptr) {
          join_load<__nv_bfloat16, kSplit, kTpr, true>(p.beta_pre, k, jc, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[k][e] += g[e];
        }
        join_store<__nv_bfloat16>(p.Xn + row * p.H, k, jc, v[k]);
      }
    }
    if (tr == 0)
      *reinterpret_cast<float4*>(p.stats + row * 4) = make_float4(mu_y, rs_y, mu_h, rs_h);
  }
}

template <class XT, class YT, int kTpr>
static cudaError_t join_fwd_launch(JoinParams p, int num_sms, cudaStream_t s) {
  constexpr int NT = join_threads(kTpr);
  const size_t stage = NT * (join_slot<XT>() + (p.has_block ? join_slot<YT>() : 0));
  // Rows in flight: as many stages as let the CTAs that the registers admit share an SM; where
  // that leaves fewer than two, all of an SM's shared memory for one CTA.
  const size_t share = (208u << 10) / (1024 / NT);
  const size_t room = share / stage >= 2 ? share : (208u << 10);
  p.nbuf = static_cast<int>(std::max<size_t>(1, std::min<size_t>(kJoinMaxBuf, room / stage)));
  const size_t smem = p.nbuf * stage;
  auto* kernel = join_fwd_kernel<XT, YT, kTpr>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  int per_sm = 1;
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, NT, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (p.T + NT / kTpr - 1) / (NT / kTpr);
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>(tiles, int64_t(std::max(1, per_sm)) * num_sms));
  kernel<<<grid, NT, smem, s>>>(p);
  return cudaGetLastError();
}

template <class XT, class YT>
static cudaError_t join_fwd_pick(const JoinParams& p, int num_sms, cudaStream_t s) {
  switch (join_tpr(p.H)) {
    case 32: return join_fwd_launch<XT, YT, 32>(p, num_sms, s);
    case 64: return join_fwd_launch<XT, YT, 64>(p, num_sms, s);
    case 128: return join_fwd_launch<XT, YT, 128>(p, num_sms, s);
    case 256: return join_fwd_launch<XT, YT, 256>(p, num_sms, s);
    case 512: return join_fwd_launch<XT, YT, 512>(p, num_sms, s);
    default: return join_fwd_launch<XT, YT, 1024>(p, num_sms, s);
  }
}

cudaError_t launch_join_fwd(const JoinParams& p, bool x32, bool y32, int num_sms, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (x32) return y32 ? join_fwd_pick<float, float>(p, num_sms, s) : join_fwd_pick<float, bf>(p, num_sms, s);
  return y32 ? join_fwd_pick<bf, float>(p, num_sms, s) : join_fwd_pick<bf, bf>(p, num_sms, s);
}

}  // namespace mlpb
