// Forward of the join between two blocks (join.cuh): the kernel and its launcher; join_*.cu
// instantiate them for their types.
#pragma once

#include "../../include/mlpb.h"
#include "join.cuh"

namespace mlpb {

// Adds a value over the wpr warps of a row, in a fixed order.  `sh` holds two places for every
// warp of the CTA; consecutive calls use them in turn (`par`), so one barrier a call is enough:
// who writes a place again has passed a barrier that every reader of it reached after reading.
// After the barrier each lane takes a warp's sum, and shuffles add them.
template <int wpr>
__device__ __forceinline__ float join_sum(float v, float (*sh)[kJoinMaxWarps], int& par) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (wpr > 1) {
    constexpr int kLanes = wpr <= 2 ? 2 : wpr <= 4 ? 4 : wpr <= 8 ? 8 : 16;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, row = warp / wpr;
    float* slot = sh[par] + row * wpr;
    par ^= 1;
    if (lane == 0) slot[warp - row * wpr] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(row + 1), "n"(wpr * 32) : "memory");
    const int l = lane & (kLanes - 1);
    v = l < wpr ? slot[l] : 0.f;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// Mean and 1/sqrt(mean square + eps) of the row in v; LayerNorm by the two-pass method (the
// mean, then the squared deviations from it), so that a common offset costs no digits.
template <bool kBeta, int kWpr, bool kSplit, int kVpt, bool kFull>
__device__ __forceinline__ void join_stats(const JoinVec (&v)[kVpt],
                                           const JoinCols<kSplit, kVpt, kFull>& jc, int kind,
                                           float inv_h, float eps, float (*sh)[kJoinMaxWarps],
                                           int& par, float& mu, float& rs) {
  float s;
  uint64_t acc = 0ull;  // (0, 0)
  mu = 0.f;
  if (kBeta && kind == MLPB_NORM_LAYER) {
#pragma unroll
    for (int k = 0; k < kVpt; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = f2_add(acc, v[k][i]);  // zeros past the row's end
    s = join_add_pair(acc);
    s = join_sum<kWpr>(s, sh, par);
    mu = s * inv_h;
    acc = 0ull;
  }
  const uint64_t m = join_twice(mu);
#pragma unroll
  for (int h = 0; h < 2 * kVpt; ++h)
    if (!kBeta || jc.ok(h)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint64_t d = v[h / 2][2 * (h & 1) + i];
        if (kBeta) d = f2_sub(d, m);
        acc = f2_fma(d, d, acc);
      }
    }
  s = join_add_pair(acc);
  s = join_sum<kWpr>(s, sh, par);
  rs = rsqrtf(s * inv_h + eps);
}

// v = (v - mu) rs g (+ beta)
template <bool kBeta, bool kSplit, int kVpt, bool kFull>
__device__ __forceinline__ void join_affine(JoinVec& v, float mu, float rs, const JoinVec& g,
                                            const __nv_bfloat16* beta, int k,
                                            const JoinCols<kSplit, kVpt, kFull>& jc) {
  const uint64_t m = join_twice(mu), r = join_twice(rs);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2_mul(f2_mul(kBeta ? f2_sub(v[i], m) : v[i], r), g[i]);
  if (kBeta && beta != nullptr) {
    JoinVec b;
    join_unpack(join_param(beta, k, jc), b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_add(v[i], b[i]);
  }
}

// 128 registers a thread: 512 threads an SM.  gamma and the gate stay in them -- gamma_post and a
// common gate as one factor where no beta (kBeta: LayerNorm) comes between them; beta is read
// again for every row.
template <class XT, class YT, int kVpt, int kWpr, bool kBeta, bool kPlain>
__global__ void __launch_bounds__(join_threads(kWpr), 512 / join_threads(kWpr))
    join_fwd_kernel(const JoinParams p) {
  constexpr bool kSplit = sizeof(XT) == 4 || sizeof(YT) == 4;
  using bf = __nv_bfloat16;
  extern __shared__ __align__(16) uint8_t join_smem[];
  __shared__ float sh[2][kJoinMaxWarps];
  constexpr int rows = join_rows(kWpr);
  const int warp = threadIdx.x / 32;
  const bool has_block = kPlain || p.has_block;
  const bool has_post = kPlain || p.post != MLPB_NORM_NONE;
  const bool has_pre = kPlain || p.pre != MLPB_NORM_NONE;
  const JoinCols<kSplit, kVpt, kPlain> jc(kWpr, warp % kWpr, p.H);
  constexpr uint32_t kXs = join_slots<XT, kVpt>();
  const uint32_t slots = kXs + (has_block ? join_slots<YT, kVpt>() : 0);  // a warp's, of a stage
  const uint32_t mine = warp * p.nbuf * slots;
  const uint32_t base = smem_u32(join_smem) + mine;
  const XT* X = static_cast<const XT*>(p.X);
  const YT* Y = static_cast<const YT*>(p.Y);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows + warp / kWpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  const float inv_h = 1.0f / static_cast<float>(p.H);
  const uint64_t alpha = join_twice(p.alpha != nullptr ? *p.alpha : 1.0f);

  auto issue = [&](int b, int64_t row) {
    if (row < p.T) {
      join_copy<XT>(base + b * slots, X + row * p.H, jc);
      if (has_block) join_copy<YT>(base + b * slots + kXs, Y + row * p.H, jc);
    }
    cp_async_commit();
  };
  for (int b = 0; b < p.nbuf; ++b) issue(b, row0 + b * step);

  // With LayerNorm, gamma_pre too is read again for every row where the registers would spill:
  // T8192 H8192 bf16 107 -> 95 us, H4096 59 -> 49, T11061 H2184 80 -> 73.  Where they hardly do,
  // it costs: T16384 H5120 fp32 (five warps, 136 registers) 191 -> 196 us, T4373 H5400 49 -> 53.
  constexpr bool kReread = kBeta && (kPlain ? kWpr != 5 : kWpr <= 4);
  uint4 gpre[kReread ? 1 : kVpt];
  JoinVec gw[kBeta ? 1 : kVpt];                            // gate gamma_post
  uint4 gpost[kBeta ? kVpt : 1], gate[kBeta ? kVpt : 1];  // or each of them
  // the factors of the gate row `g` (every row's where p.G <= 1)
  auto factors = [&](const bf* g) {
#pragma unroll
    for (int k = 0; k < kVpt; ++k) {
      if constexpr (kBeta) {
        gate[k] = join_param(g, k, jc);
      } else {
        JoinVec w;
        join_unpack(join_param(g, k, jc), gw[k]);
        if (has_post) {
          join_unpack(join_param(p.gamma_post, k, jc), w);
#pragma unroll
          for (int i = 0; i < 4; ++i) gw[k][i] = g != nullptr ? f2_mul(gw[k][i], w[i]) : w[i];
        }
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    if constexpr (kBeta) gpost[k] = join_param(p.gamma_post, k, jc);
    if constexpr (!kReread) gpre[k] = join_param(p.gamma_pre, k, jc);
  }
  factors(p.gate);

  int b = 0, par = 0;
  for (int64_t row = row0; row < p.T; row += step) {
    if (p.G > 1)  // this row's gate; used after the first norm
      factors(p.gate + (static_cast<uint32_t>(row) / static_cast<uint32_t>(p.rows_per_group)) *
                           static_cast<int64_t>(p.H));
    cp_async_wait_ring(p.nbuf);
    const uint8_t* st = join_smem + mine + b * slots;
    JoinVec v[kVpt];
    float mu_y = 0.f, rs_y = 0.f, mu_h = 0.f, rs_h = 0.f;
    if (has_block) {
#pragma unroll
      for (int k = 0; k < kVpt; ++k) join_read<YT, false>(st + kXs, k, jc, v[k]);
      if (has_post) join_stats<kBeta, kWpr>(v, jc, p.post, inv_h, p.eps, sh, par, mu_y, rs_y);
#pragma unroll
      for (int k = 0; k < kVpt; ++k) {
        JoinVec t;
        if constexpr (kBeta) {
          if (has_post) {
            join_unpack(gpost[k], t);
            join_affine<kBeta>(v[k], mu_y, rs_y, t, p.beta_post, k, jc);
          }
          if (p.gate != nullptr) {
            join_unpack(gate[k], t);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] = f2_mul(v[k][i], t[i]);
          }
        } else if (has_post) {
          join_affine<kBeta>(v[k], mu_y, rs_y, gw[k], nullptr, k, jc);
        } else if (p.gate != nullptr) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[k][i] = f2_mul(v[k][i], gw[k][i]);
        }
        join_read<XT, false>(st, k, jc, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] = f2_fma(alpha, t[i], v[k][i]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kVpt; ++k) join_read<XT, false>(st, k, jc, v[k]);
    }
    issue(b, row + p.nbuf * step);  // the slots of this row have been read
    if (++b == p.nbuf) b = 0;
    // The norm is that of the stream as it is stored (rounded, where it is bf16): what a
    // backward that reads Xout differentiates.
    if (has_block) {
#pragma unroll
      for (int k = 0; k < kVpt; ++k)
        join_store<XT, true>(static_cast<XT*>(p.Xout) + row * p.H, k, jc, v[k]);
    }
    if (has_pre) {
      join_stats<kBeta, kWpr>(v, jc, p.pre, inv_h, p.eps, sh, par, mu_h, rs_h);
#pragma unroll
      for (int k = 0; k < kVpt; ++k) {
        JoinVec t;
        if constexpr (kReread)
          join_unpack(join_param(p.gamma_pre, k, jc), t);
        else
          join_unpack(gpre[k], t);
        join_affine<kBeta>(v[k], mu_h, rs_h, t, p.beta_pre, k, jc);
        join_store<bf, false>(p.Xn + row * p.H, k, jc, v[k]);
      }
    }
    if (threadIdx.x % (32 * kWpr) == 0)
      *reinterpret_cast<float4*>(p.stats + row * 4) = make_float4(mu_y, rs_y, mu_h, rs_h);
  }
}

template <class XT, class YT, int kVpt, int kWpr, bool kBeta>
static cudaError_t join_fwd_launch(JoinParams p, int num_sms, cudaStream_t s) {
  constexpr int threads = join_threads(kWpr);
  const size_t stage =
      threads / 32 * (join_slots<XT, kVpt>() + (p.has_block ? join_slots<YT, kVpt>() : 0));
  constexpr int ctas = 512 / threads;  // an SM's, by the registers
  const int64_t tiles = (p.T + join_rows(kWpr) - 1) / join_rows(kWpr);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, int64_t(ctas) * num_sms));
  // stages in flight: what lets those CTAs share an SM, and no more than a CTA has turns
  const size_t room = (208u << 10) / ctas;
  p.nbuf = static_cast<int>(std::max<size_t>(1, std::min<size_t>(kJoinMaxBuf, room / stage)));
  p.nbuf = static_cast<int>(std::min<int64_t>(p.nbuf, (tiles + grid - 1) / grid));
  const size_t smem = p.nbuf * stage;
  auto* kernel = join_fwd_kernel<XT, YT, kVpt, kWpr, kBeta, false>;
  if constexpr (kVpt == 4) {
    if (p.has_block && p.post != MLPB_NORM_NONE && p.pre != MLPB_NORM_NONE &&
        p.H == 256 * kVpt * kWpr)
      kernel = join_fwd_kernel<XT, YT, kVpt, kWpr, kBeta, true>;
  }
  const cudaError_t e = join_smem_attr(kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, threads, smem, s>>>(p);
  return cudaGetLastError();
}

template <class XT, class YT, bool kBeta>
static cudaError_t join_fwd_pick(const JoinParams& p, int num_sms, cudaStream_t s) {
  switch (join_fwd_wpr(p.H, kBeta)) {
    case 1:
      return p.H <= 256 ? join_fwd_launch<XT, YT, 1, 1, kBeta>(p, num_sms, s)
                        : join_fwd_launch<XT, YT, 4, 1, kBeta>(p, num_sms, s);
    case 2: return join_fwd_launch<XT, YT, 4, 2, kBeta>(p, num_sms, s);
    case 4: return join_fwd_launch<XT, YT, 4, 4, kBeta>(p, num_sms, s);
    case 5: return join_fwd_launch<XT, YT, 4, 5, kBeta>(p, num_sms, s);
    case 8: return join_fwd_launch<XT, YT, 4, 8, kBeta>(p, num_sms, s);
    default: return join_fwd_launch<XT, YT, 4, 16, kBeta>(p, num_sms, s);
  }
}

template <class XT, class YT>
cudaError_t join_fwd_run(const JoinParams& p, int num_sms, cudaStream_t s) {
  return p.post == MLPB_NORM_LAYER || p.pre == MLPB_NORM_LAYER
             ? join_fwd_pick<XT, YT, true>(p, num_sms, s)
             : join_fwd_pick<XT, YT, false>(p, num_sms, s);
}

}  // namespace mlpb
