// Backward of the join between two blocks (join.cuh): the kernel and its launcher; the
// translation units instantiate it for their types.
//
// Two reductions a row: g = dXn gamma_pre gives mean(g), mean(g xh) and with them
// dh = dXout + rstd_h (g - mean g - xh mean(g xh)); then u = gate dh gamma_post gives
// mean(u), mean(u yh) and dY.
//
// The parameters' gradients need only four sums over rows for each column: sum dXn xh and
// sum dXn (the pre-norm's), and, within one gate group, S1 = sum dh yh and S0 = sum dh:
//   dgate = gamma_post S1 + beta_post S0,  dgamma_post = sum over groups of gate S1,
//   dbeta_post = sum over groups of gate S0.
// They stay in fp32 registers while a CTA walks rows of one group (16 columns a thread: 32
// registers without LayerNorm's two plain sums, 64 with them), and each CTA leaves one row of
// partial sums for a second launch to add up in a fixed order: no atomics, the same bits every
// run.  So a CTA's rows are of one group: a group has blocks_per_group CTAs, or, with more
// groups than CTAs, a CTA walks whole groups and adds each into its own partial row.
#pragma once

#include "../../include/mlpb.h"
#include "join.cuh"

namespace mlpb {

// Adds the kRows rows' accumulators of a column up, over the CTA's groups of threads, in row
// order (the ring's shared memory is free by then: every copy has been waited for, since each
// thread's last wait left only groups of rows past the end, which copied nothing).
template <int kTpr>
__device__ __forceinline__ void join_combine(float (&v)[kJoinVpt][8]) {
  constexpr int NT = join_threads(kTpr), kRows = NT / kTpr;
  if constexpr (kRows > 1) {
    extern __shared__ __align__(16) uint8_t join_smem[];
    float* acc = reinterpret_cast<float*>(join_smem);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinVpt * 8; ++i) acc[i * NT + threadIdx.x] = v[i / 8][i % 8];
    __syncthreads();
    const int tr = threadIdx.x % kTpr;
#pragma unroll
    for (int i = 0; i < kJoinVpt * 8; ++i) {
      float t = 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) t += acc[i * NT + r * kTpr + tr];
      v[i / 8][i % 8] = t;
    }
    __syncthreads();
  }
}

// A row's vector k of fp32 values at `row` (+= with add).
template <bool kSplit, int kTpr>
__device__ __forceinline__ void join_put(float* row, int k, const JoinCols<kSplit, kTpr>& jc,
                                         const float (&v)[8], bool add) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!jc.ok[k][h]) continue;
    float4* q = reinterpret_cast<float4*>(row + jc.c[k][h]);
    float4 o = add ? *q : make_float4(0.f, 0.f, 0.f, 0.f);
    o.x += v[4 * h];
    o.y += v[4 * h + 1];
    o.z += v[4 * h + 2];
    o.w += v[4 * h + 3];
    *q = o;
  }
}

template <class XT, class YT, int kTpr, bool kBeta>
__global__ void __launch_bounds__(join_threads(kTpr), kTpr <= 512 ? 512 / join_threads(kTpr) : 1)
    join_bwd_kernel(const JoinParams p) {
  constexpr int NT = join_threads(kTpr);
  constexpr int kRows = NT / kTpr;
  constexpr bool kSplit = sizeof(XT) == 4 || sizeof(YT) == 4;
  using bf = __nv_bfloat16;
  extern __shared__ __align__(16) uint8_t join_smem[];
  __shared__ float2 sh[2 * NT / 32];
  const int tr = threadIdx.x % kTpr;
  const int sub = threadIdx.x / kTpr;
  const JoinCols<kSplit, kTpr> jc(tr, p.H);
  const bool has_pre = p.pre != MLPB_NORM_NONE, has_post = p.post != MLPB_NORM_NONE;
  const bool need_y = has_post || p.gate != nullptr;
  const bool need_x = p.part_alpha != nullptr;
  const bool late_ring = !p.direct_late;

  // the slots of a stage: Xout, dXn, Y, dXout, X (those that are read)
  uint32_t off = 0;
  const uint32_t o_xout = off;
  off += has_pre ? NT * join_slot<XT>() : 0;
  const uint32_t o_dxn = off;
  off += has_pre ? NT * join_slot<YT>() : 0;
  const uint32_t o_y = off;
  off += need_y ? NT * join_slot<YT>() : 0;
  const uint32_t o_dxout = off;
  off += late_ring && p.dXout ? NT * join_slot<XT>() : 0;
  const uint32_t o_x = off;
  off += late_ring && need_x ? NT * join_slot<XT>() : 0;
  const uint32_t stage = off;
  const uint32_t base = smem_u32(join_smem);

  const float inv_h = 1.0f / static_cast<float>(p.H);
  const float alpha = p.alpha != nullptr ? *p.alpha : 1.0f;
  const XT* Xout = static_cast<const XT*>(p.Xout);
  const XT* X = static_cast<const XT*>(p.X);
  const XT* dXout = static_cast<const XT*>(p.dXout);
  const YT* Y = static_cast<const YT*>(p.Y);
  const YT* dXn = static_cast<const YT*>(p.dXn);

  float a1[kJoinVpt][8], a0[kJoinVpt][8];  // sum dXn xh, sum dXn
  float s1[kJoinVpt][8], s0[kJoinVpt][8];  // sum dh yh, sum dh of the group
  float d_alpha = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinVpt; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a1[k][e] = s1[k][e] = 0.f;
      if (kBeta) a0[k][e] = s0[k][e] = 0.f;
    }

  const int bpg = p.blocks_per_group;
  const int groups = p.G > 0 ? p.G : 1;
  const int walkers = gridDim.x / bpg;  // CTAs apart: groups a CTA steps over
  int par = 0;
  bool first = true;

  for (int g = blockIdx.x / bpg; g < groups; g += walkers) {
    const int64_t r_end = (g + int64_t(1)) * p.rows_per_group;
    const int64_t row0 = g * p.rows_per_group + (blockIdx.x % bpg) * kRows + sub;
    const int64_t step = static_cast<int64_t>(bpg) * kRows;
    const bf* gate = p.gate != nullptr ? p.gate + static_cast<int64_t>(g) * p.H : nullptr;

    auto issue = [&](int b, int64_t row) {
      if (row < r_end) {
        const uint32_t d = base + b * stage;
        if (has_pre) {
          join_copy<XT>(d + o_xout, NT, Xout + row * p.H, jc);
          join_copy<YT>(d + o_dxn, NT, dXn + row * p.H, jc);
        }
        if (need_y) join_copy<YT>(d + o_y, NT, Y + row * p.H, jc);
        if (late_ring && p.dXout) join_copy<XT>(d + o_dxout, NT, dXout + row * p.H, jc);
        if (late_ring && need_x) join_copy<XT>(d + o_x, NT, X + row * p.H, jc);
      }
      cp_async_commit();
    };
    for (int b = 0; b < p.nbuf; ++b) issue(b, row0 + b * step);

    int b = 0;
    for (int64_t row = row0; row < r_end; row += step) {
      cp_async_wait_ring(p.nbuf);
      const uint8_t* st = join_smem + b * stage;
      const float4 stat = __ldg(reinterpret_cast<const float4*>(p.stats + row * 4));
      float m[2] = {0.f, 0.f};
      if (has_pre) {
#pragma unroll
        for (int k = 0; k < kJoinVpt; ++k) {
          float x[8], d[8], w[8];
          join_read<XT>(st + o_xout, NT, k, jc, x);
          join_read<YT>(st + o_dxn, NT, k, jc, d);
          join_load<bf, kSplit, kTpr, true>(p.gamma_pre, k, jc, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xh = (x[e] - stat.z) * stat.w;
            const float q = d[e] * w[e];
            m[0] += q;
            m[1] = fmaf(q, xh, m[1]);
            a1[k][e] = fmaf(d[e], xh, a1[k][e]);
            if (kBeta) a0[k][e] += d[e];
          }
        }
        join_sum<kTpr, 2>(m, sh, par);
        m[0] = p.pre == MLPB_NORM_LAYER ? m[0] * inv_h : 0.f;
        m[1] *= inv_h;
      }
      float dh[kJoinVpt][8], yh[kJoinVpt][8];
      float n[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k) {
        if (p.dXout == nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dh[k][e] = 0.f;
        } else if (late_ring) {
          join_read<XT>(st + o_dxout, NT, k, jc, dh[k]);
        } else {
          join_load<XT, kSplit, kTpr, false>(dXout + row * p.H, k, jc, dh[k]);
        }
        if (has_pre) {
          float x[8], d[8], w[8];
          join_read<XT>(st + o_xout, NT, k, jc, x);
          join_read<YT>(st + o_dxn, NT, k, jc, d);
          join_load<bf, kSplit, kTpr, true>(p.gamma_pre, k, jc, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xh = (x[e] - stat.z) * stat.w;
            dh[k][e] += stat.w * (d[e] * w[e] - m[0] - xh * m[1]);
          }
        }
        if (need_x) {
          float x[8];
          if (late_ring)
            join_read<XT>(st + o_x, NT, k, jc, x);
          else
            join_load<XT, kSplit, kTpr, true>(X + row * p.H, k, jc, x);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (jc.ok[k][e / 4]) d_alpha = fmaf(dh[k][e], x[e], d_alpha);
        }
        if (need_y) {
          join_read<YT>(st + o_y, NT, k, jc, yh[k]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (has_post) yh[k][e] = (yh[k][e] - stat.x) * stat.y;
            s1[k][e] = fmaf(dh[k][e], yh[k][e], s1[k][e]);
            if (kBeta) s0[k][e] += dh[k][e];
          }
        }
      }
      issue(b, row + p.nbuf * step);  // this row's slots have been read
      if (++b == p.nbuf) b = 0;
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k) {
        float dx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] = alpha * dh[k][e];
        join_store<XT>(static_cast<XT*>(p.dX) + row * p.H, k, jc, dx);
        if (p.has_block && gate != nullptr) {
          float w[8];
          join_load<bf, kSplit, kTpr, true>(gate, k, jc, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) dh[k][e] *= w[e];
        }
        if (has_post) {
          float w[8];
          join_load<bf, kSplit, kTpr, true>(p.gamma_post, k, jc, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dh[k][e] *= w[e];  // u, zero past the row's end as gamma is
            n[0] += dh[k][e];
            n[1] = fmaf(dh[k][e], yh[k][e], n[1]);
          }
        }
      }
      if (has_post) {
        join_sum<kTpr, 2>(n, sh, par);
        n[0] = p.post == MLPB_NORM_LAYER ? n[0] * inv_h : 0.f;
        n[1] *= inv_h;
#pragma unroll
        for (int k = 0; k < kJoinVpt; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dh[k][e] = stat.y * (dh[k][e] - n[0] - yh[k][e] * n[1]);
      }
      if (p.has_block) {
#pragma unroll
        for (int k = 0; k < kJoinVpt; ++k) join_store<bf>(p.dY + row * p.H, k, jc, dh[k]);
      }
    }

    // The end of this CTA's rows of the group: S1 and S0 over the CTA, and what they give.
    if (need_y) {
      join_combine<kTpr>(s1);
      if (kBeta) join_combine<kTpr>(s0);
      if (sub == 0) {
        const int64_t slot = static_cast<int64_t>(blockIdx.x) * p.H;
#pragma unroll
        for (int k = 0; k < kJoinVpt; ++k) {
          float w[8], t[8];
          if (gate != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = s1[k][e];
            if (has_post) {
              join_load<bf, kSplit, kTpr, true>(p.gamma_post, k, jc, w);
#pragma unroll
              for (int e = 0; e < 8; ++e) t[e] *= w[e];
            }
            if (kBeta && p.beta_post != nullptr) {
              join_load<bf, kSplit, kTpr, true>(p.beta_post, k, jc, w);
#pragma unroll
              for (int e = 0; e < 8; ++e) t[e] = fmaf(w[e], s0[k][e], t[e]);
            }
            if (bpg > 1)
              join_put(p.part_gate + slot, k, jc, t, false);
            else
              join_put(p.dgate + static_cast<int64_t>(g) * p.H, k, jc, t, p.accumulate != 0);
            join_load<bf, kSplit, kTpr, true>(gate, k, jc, w);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 1.0f;
          }
          if (p.part_gpost != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = w[e] * s1[k][e];
            join_put(p.part_gpost + slot, k, jc, t, !first);
          }
          if (kBeta && p.part_bpost != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = w[e] * s0[k][e];
            join_put(p.part_bpost + slot, k, jc, t, !first);
          }
        }
      }
      first = false;
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s1[k][e] = 0.f;
          if (kBeta) s0[k][e] = 0.f;
        }
    }
  }

  if (has_pre) {
    join_combine<kTpr>(a1);
    if (kBeta) join_combine<kTpr>(a0);
    if (sub == 0) {
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * p.H;
#pragma unroll
      for (int k = 0; k < kJoinVpt; ++k) {
        join_put(p.part_gpre + slot, k, jc, a1[k], false);
        if (kBeta && p.part_bpre != nullptr)
          join_put(p.part_bpre + slot, k, jc, a0[k], false);
      }
    }
  }
  if (need_x) {  // the CTA's part of dalpha, added in warp order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d_alpha += __shfl_xor_sync(0xffffffffu, d_alpha, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x / 32].x = d_alpha;
    __syncthreads();
    if (threadIdx.x == 0) {
      float t = 0.f;
      for (int w = 0; w < NT / 32; ++w) t += sh[w].x;
      p.part_alpha[blockIdx.x] = t;
    }
  }
}

// CTAs of the launch: with few groups, each gets an equal number of CTAs of its own; with
// more groups than CTAs, a CTA walks groups.
template <class XT, class YT, int kTpr, bool kBeta>
static cudaError_t join_bwd_launch(JoinParams p, int grid, cudaStream_t s) {
  constexpr int NT = join_threads(kTpr);
  const bool has_pre = p.pre != MLPB_NORM_NONE;
  const bool need_y = p.post != MLPB_NORM_NONE || p.gate != nullptr;
  const size_t early = NT * ((has_pre ? join_slot<XT>() + join_slot<YT>() : 0) +
                             (need_y ? join_slot<YT>() : 0));
  const size_t late = NT * ((p.dXout != nullptr ? join_slot<XT>() : 0) +
                            (p.part_alpha != nullptr ? join_slot<XT>() : 0));
  const size_t room = (208u << 10) / (NT <= 256 ? 2 : 1);
  p.direct_late = early + late > room;
  const size_t stage = p.direct_late ? early : early + late;
  p.nbuf = static_cast<int>(std::max<size_t>(
      1, std::min<size_t>(kJoinMaxBuf, room / std::max<size_t>(stage, 1))));
  size_t smem = p.nbuf * stage;
  if (NT > kTpr) smem = std::max(smem, static_cast<size_t>(NT) * kJoinVpt * 8 * 4);
  auto* kernel = join_bwd_kernel<XT, YT, kTpr, kBeta>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kernel<<<grid, NT, smem, s>>>(p);
  return cudaGetLastError();
}

template <class XT, class YT, bool kBeta>
static cudaError_t join_bwd_pick(const JoinParams& p, int grid, cudaStream_t s) {
  switch (join_tpr(p.H)) {
    case 32: return join_bwd_launch<XT, YT, 32, kBeta>(p, grid, s);
    case 64: return join_bwd_launch<XT, YT, 64, kBeta>(p, grid, s);
    case 128: return join_bwd_launch<XT, YT, 128, kBeta>(p, grid, s);
    case 256: return join_bwd_launch<XT, YT, 256, kBeta>(p, grid, s);
    case 512: return join_bwd_launch<XT, YT, 512, kBeta>(p, grid, s);
    default: return join_bwd_launch<XT, YT, 1024, kBeta>(p, grid, s);
  }
}

}  // namespace mlpb
