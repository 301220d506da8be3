// Backward of the join between two blocks (join.cuh): the kernel and its launcher; join_*.cu
// instantiate them for their types.
//
// With g = dXn gamma_pre, t = dXout + rstd_h g and w = gate gamma_post,
//   dh = t - rstd_h (mean g + xh mean(g xh)),  u = w dh,  dY = rstd_y (u - mean u - yh mean(u yh))
// (the plain means with LayerNorm only).  mean(u yh) looks as if it had to wait for dh and so for
// the first means, but it is linear in them:
//   sum u yh = sum w yh t - rstd_h (mean g sum w yh + mean(g xh) sum w yh xh),
// and sum u alike.  So a row takes one pass for all its sums (3, or 7 with LayerNorm), one
// reduction, and one pass for what it writes.  (Two reductions, one after the other, cost a
// row of H 8192 about 0.9 us of 3.5.)  xh and t stay in registers between the passes (kKeep);
// with LayerNorm's twice as many column sums, or 32 columns a thread, they are computed again.
//
// The parameters' gradients need only four sums over rows for each column: sum dXn xh and
// sum dXn (the pre-norm's), and, within one gate group, S1 = sum dh yh and S0 = sum dh:
//   dgate = gamma_post S1 + beta_post S0,  dgamma_post = sum over groups of gate S1,
//   dbeta_post = sum over groups of gate S0.
// They stay in fp32 registers while a CTA walks rows of one group (16 columns a thread: 32
// registers without LayerNorm's two plain sums, 64 with them), and each CTA leaves one row of
// partial sums for a second launch to add up in a fixed order: no atomics, the same bits every
// run.  So a CTA's rows are of one group: a group has blocks_per_group CTAs, or, with more
// groups than CTAs, a CTA walks whole groups and adds each into its own partial row.  (Or each
// row of a CTA does, where groups are short: p.split.)
#pragma once

#include "../../include/mlpb.h"
#include "join.cuh"

namespace mlpb {

// Adds a CTA's rows' accumulators of a column up, in row order, for the first row's warps, by way
// of `smem`: the plain instantiations' ring (which is free by then: every copy has been waited
// for, since each thread's last wait left only groups of rows past the end, which copied
// nothing), or memory behind the general ones', whose ring keeps its zeros.
template <int kVpt>
__device__ __forceinline__ void join_combine(JoinVec (&v)[kVpt], int rows, uint8_t* smem) {
  if (rows == 1) return;
  uint64_t* acc = reinterpret_cast<uint64_t*>(smem) + threadIdx.x;
  const int nt = blockDim.x, tpr = nt / rows;
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kVpt * 4; ++i) acc[i * nt] = v[i / 4][i % 4];
  __syncthreads();
  if (threadIdx.x < tpr)
#pragma unroll 1
    for (int r = 1; r < rows; ++r)
#pragma unroll
      for (int i = 0; i < kVpt * 4; ++i)
        v[i / 4][i % 4] = f2_add(v[i / 4][i % 4], acc[i * nt + r * tpr]);
  __syncthreads();
}

// A row's vector k of fp32 values at `row` (+= with add).
template <bool kSplit, int kVpt, bool kFull>
__device__ __forceinline__ void join_put(float* row, int k, const JoinCols<kSplit, kVpt, kFull>& jc,
                                         const JoinVec& v, bool add) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!jc.ok(2 * k + h)) continue;
    float4* q = reinterpret_cast<float4*>(row + jc.c[2 * k + h]);
    float4 o = add ? *q : make_float4(0.f, 0.f, 0.f, 0.f), t;
    f2_unpack(v[2 * h], t.x, t.y);
    f2_unpack(v[2 * h + 1], t.z, t.w);
    o.x += t.x;
    o.y += t.y;
    o.z += t.z;
    o.w += t.w;
    *q = o;
  }
}

// This CTA's number in a cluster of kCl.
template <int kCl>
__device__ __forceinline__ int join_rank() {
  return kCl == 1 ? 0 : static_cast<int>(cluster_ctarank());
}

// Adds NV values over the warps of a row (wpr in each CTA), in a fixed order; one barrier, as
// join_sum.  The shuffles of a warp's sums give away half of the values a lane still has, so that
// 8 values take 9 of them, not 40; a lane then owns one value, and after the barrier adds up every
// eighth (or fourth) warp's.  Two CTAs of a row (kCl) write their warps' sums into both.
template <int kWpr, int kCl, int NV>
__device__ __forceinline__ void join_sums(float (&v)[NV], int wpr,
                                          float (*sh)[kCl * kJoinMaxWarps][8], int& par) {
  constexpr int P = NV <= 4 ? 4 : 8, kLanes = 32 / P;  // lanes of a value
  const int lane = threadIdx.x & 31, own = lane / kLanes;
  float t[P];
#pragma unroll
  for (int i = 0; i < P; ++i) t[i] = i < NV ? v[i] : 0.f;
#pragma unroll
  for (int w = P / 2, o = 16; w >= 1; w >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = up ? t[i] : t[i + w], keep = up ? t[i + w] : t[i];
      t[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) t[0] += __shfl_xor_sync(0xffffffffu, t[0], o);
  if (kCl > 1 || (kWpr != 1 && wpr > 1)) {
    const int warp = threadIdx.x / 32, row = warp / wpr;
    if constexpr (kCl > 1) {
      if (lane % kLanes < kCl) {  // a lane for each CTA
        const uint32_t to = smem_u32(&sh[par][join_rank<kCl>() * wpr + warp][own]);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(to, lane % kLanes)),
                     "f"(t[0])
                     : "memory");
      }
      cluster_sync();
    } else {
      if (lane % kLanes == 0) sh[par][warp][own] = t[0];
      asm volatile("bar.sync %0, %1;" ::"r"(row + 1), "r"(wpr * 32) : "memory");
    }
    t[0] = 0.f;
#pragma unroll
    for (int w0 = 0; w0 < kCl * (kWpr > 0 ? kWpr : -kWpr); w0 += kLanes) {
      const int w = w0 + lane % kLanes;
      if (w < kCl * wpr) t[0] += sh[par][row * wpr + w][own];
    }
    par ^= 1;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) t[0] += __shfl_xor_sync(0xffffffffu, t[0], o);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = __shfl_sync(0xffffffffu, t[0], i * kLanes);
}

// What a thread needs of the parameters for every row: gamma_pre (packed) and w = gate gamma_post
// of its columns, in registers, or (kSmem) in shared memory that is the thread's own: where they
// would not fit, the compiler's spills miss what the ring leaves of L1.
template <int kVpt, bool kSmem>
struct JoinFactors {
  uint4 g[kSmem ? 1 : kVpt];
  JoinVec w[kSmem ? 1 : kVpt];
  uint4* own;
  static constexpr size_t kBytes = kSmem ? 48 * kVpt : 0;  // of a thread
  __device__ __forceinline__ JoinFactors(void* smem)
      : own(static_cast<uint4*>(smem) + threadIdx.x) {}
  __device__ __forceinline__ void set_pre(int k, const uint4& v) {
    if constexpr (kSmem)
      own[3 * k * blockDim.x] = v;
    else
      g[k] = v;
  }
  __device__ __forceinline__ void set_w(int k, const JoinVec& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kSmem)
        reinterpret_cast<uint64_t*>(own + (3 * k + 1 + i / 2) * blockDim.x)[i % 2] = v[i];
      else
        w[k][i] = v[i];
    }
  }
  __device__ __forceinline__ void pre(int k, JoinVec& v) const {
    if constexpr (kSmem)
      join_unpack(own[3 * k * blockDim.x], v);
    else
      join_unpack(g[k], v);
  }
  __device__ __forceinline__ void get_w(int k, JoinVec& v) const {
    if constexpr (kSmem) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const ulonglong2 t =
            *reinterpret_cast<const ulonglong2*>(own + (3 * k + 1 + h) * blockDim.x);
        v[2 * h] = t.x;
        v[2 * h + 1] = t.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = w[k][i];
    }
  }
};

// Whether they are in shared memory.
template <int kWpr, bool kBeta>
constexpr bool join_bwd_smem() {
  return kWpr < 0 || kBeta;
}

template <class XT, class YT, int kVpt, int kWpr, bool kBeta, int kCl>
__global__ void __launch_bounds__(join_threads(kWpr), join_ctas(kWpr))
    join_bwd_kernel(const JoinParams p) {
  constexpr bool kSplit = sizeof(XT) == 4 || sizeof(YT) == 4, kPlain = kWpr > 0;
  constexpr bool kKeep = !kBeta;
  using bf = __nv_bfloat16;
  extern __shared__ __align__(16) uint8_t join_smem[];
  constexpr int kSums = kBeta ? 7 : 3;
  __shared__ float sh[2][kCl * kJoinMaxWarps][8];
  const int wpr = kPlain ? kWpr : p.wpr, rows = kPlain ? join_rows(kWpr) : p.rows;
  const int warp = threadIdx.x / 32, sub = warp / wpr;
  const JoinCols<kSplit, kVpt, kPlain> jc(kCl * wpr, join_rank<kCl>() * wpr + warp % wpr, p.H);
  const bool has_block = kPlain || p.has_block;
  const bool has_pre = kPlain || p.pre != MLPB_NORM_NONE;
  const bool has_post = kPlain || p.post != MLPB_NORM_NONE;
  const bool need_y = has_post || p.gate != nullptr;
  const bool has_dxout = kPlain || p.dXout != nullptr;
  const bool need_x = p.part_alpha != nullptr;

  // a warp's slots of a stage: Xout, dXn, Y, dXout, X (those that are read)
  constexpr uint32_t kXs = join_slots<XT, kVpt>(), kYs = join_slots<YT, kVpt>();
  uint32_t off = 0;
  const uint32_t o_xout = off, o_dxn = off + kXs;
  off += has_pre ? kXs + kYs : 0;
  const uint32_t o_y = off;
  off += need_y ? kYs : 0;
  const uint32_t o_dxout = off;
  off += has_dxout ? kXs : 0;
  const uint32_t o_x = off;
  off += need_x ? kXs : 0;
  const uint32_t slots = off;
  const uint32_t mine = warp * p.nbuf * slots;
  const uint32_t base = smem_u32(join_smem) + mine;

  const float inv_h = 1.0f / static_cast<float>(p.H);
  const uint64_t alpha = join_twice(p.alpha != nullptr ? *p.alpha : 1.0f);
  const XT* Xout = static_cast<const XT*>(p.Xout);
  const XT* X = static_cast<const XT*>(p.X);
  const XT* dXout = static_cast<const XT*>(p.dXout);
  const YT* Y = static_cast<const YT*>(p.Y);
  const YT* dXn = static_cast<const YT*>(p.dXn);

  JoinVec a1[kVpt], a0[kVpt];  // sum dXn xh, sum dXn
  JoinVec s1[kVpt], s0[kVpt];  // sum dh yh, sum dh of the group
  uint64_t d_alpha = 0ull;
  // behind the ring
  using Factors = JoinFactors<kVpt, join_bwd_smem<kWpr, kBeta>()>;
  Factors fac(join_smem + p.ring_bytes);
  uint8_t* comb = kPlain ? join_smem : join_smem + p.ring_bytes + Factors::kBytes * blockDim.x;
  if (!kPlain && p.ragged) join_clear(join_smem, p.ring_bytes);
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    fac.set_pre(k, join_param(p.gamma_pre, k, jc));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a1[k][i] = s1[k][i] = 0ull;
      if (kBeta) a0[k][i] = s0[k][i] = 0ull;
    }
  }

  const int bpg = p.blocks_per_group;
  const int groups = p.G > 0 ? p.G : 1;
  // A group is walked by bpg CTAs (or clusters), whose `at_once` rows are all the group's; or,
  // with p.split, a walker is one row of a CTA.
  constexpr bool kSeveral = !kPlain && kCl == 1 && (kWpr == -12 || kVpt == 1);  // rows of a CTA
  const bool split = kSeveral && p.split;
  const int at_once = split ? 1 : rows, place = split ? 0 : sub;
  const int walker = split ? blockIdx.x * rows + sub : blockIdx.x / kCl;
  const int walkers = (split ? gridDim.x * rows : gridDim.x / kCl) / bpg;  // groups of a turn
  int par = 0;
  bool first = true;
  if constexpr (kCl > 1) cluster_sync();  // the other CTA's shared memory is there

  for (int g = walker / bpg; g < groups; g += walkers) {
    // (below 2^31, and what is added beyond the end below 2^14)
    const uint32_t r_end = (g + 1u) * static_cast<uint32_t>(p.rows_per_group);
    const uint32_t row0 = r_end - static_cast<uint32_t>(p.rows_per_group) +
                          (walker % bpg) * at_once + place;
    const uint32_t step = bpg * at_once;
    const bf* gate = p.gate != nullptr ? p.gate + static_cast<int64_t>(g) * p.H : nullptr;

    auto issue = [&](int b, uint32_t row) {
      if (row < r_end) {
        const uint32_t d = base + b * slots;
        const int64_t o = static_cast<int64_t>(row) * p.H;
        if (has_pre) {
          join_copy<XT>(d + o_xout, Xout + o, jc);
          join_copy<YT>(d + o_dxn, dXn + o, jc);
        }
        if (need_y) join_copy<YT>(d + o_y, Y + o, jc);
        if (has_dxout) join_copy<XT>(d + o_dxout, dXout + o, jc);
        if (need_x) join_copy<XT>(d + o_x, X + o, jc);
      }
      cp_async_commit();
    };
    for (int b = 0; b < p.nbuf; ++b) issue(b, row0 + b * step);
    uint64_t ws = 0ull;
#pragma unroll
    for (int k = 0; k < kVpt; ++k) {
      JoinVec w, t;
      join_unpack(join_param(gate, k, jc), w);
      if (has_post) {
        join_unpack(join_param(p.gamma_post, k, jc), t);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = gate != nullptr ? f2_mul(w[i], t[i]) : t[i];
      }
      fac.set_w(k, w);
      if (kBeta)
#pragma unroll
        for (int i = 0; i < 4; ++i) ws = f2_add(ws, w[i]);
    }

    float w_sum = 0.f;  // sum of w over the row
    if (kBeta && p.post == MLPB_NORM_LAYER) {
      float v[kSums] = {join_add_pair(ws)};
      join_sums<kWpr, kCl>(v, wpr, sh, par);
      w_sum = v[0];
    }

    int b = 0;
    float4 next = make_float4(0.f, 0.f, 0.f, 0.f);  // the next row's statistics, a row ahead
    if (row0 < r_end) next = __ldg(reinterpret_cast<const float4*>(p.stats) + row0);
    for (uint32_t row = row0; row < r_end; row += step) {
      const int64_t at = static_cast<int64_t>(row) * p.H;
      const float4 stat = next;
      if (row + step < r_end)
        next = __ldg(reinterpret_cast<const float4*>(p.stats) + row + step);
      cp_async_wait_ring(p.nbuf);
      uint8_t* st = join_smem + mine + b * slots;
      const uint64_t mu_h = join_twice(stat.z), rs_h = join_twice(stat.w);
      const uint64_t mu_y = join_twice(stat.x), rs_y = join_twice(stat.y);
      // xh and t of vector k, and dXn
      auto start = [&](int k, JoinVec& xh, JoinVec& t, JoinVec& d, uint64_t* g_sum,
                       uint64_t* gx_sum) {
        if (!has_dxout) {
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = 0ull;
        } else {
          join_read<XT, true>(st + o_dxout, k, jc, t);
        }
        if (has_pre) {
          JoinVec w;
          join_read<XT, true>(st + o_xout, k, jc, xh);
          join_read<YT, true>(st + o_dxn, k, jc, d);
          fac.pre(k, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xh[i] = f2_mul(kBeta ? f2_sub(xh[i], mu_h) : xh[i], rs_h);
            const uint64_t q = f2_mul(d[i], w[i]);
            t[i] = f2_fma(rs_h, q, t[i]);
            if (gx_sum != nullptr) {
              *gx_sum = f2_fma(q, xh[i], *gx_sum);
              if (kBeta) *g_sum = f2_add(*g_sum, q);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) xh[i] = d[i] = 0ull;
        }
      };
      auto normed_y = [&](int k, JoinVec& yh) {
        join_read<YT, true>(st + o_y, k, jc, yh);
        if (has_post) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            yh[i] = f2_mul(kBeta ? f2_sub(yh[i], mu_y) : yh[i], rs_y);
        }
      };
      JoinVec kx[kVpt], kt[kVpt];  // kKeep: xh and t
      // sums of g xh, w yh t, w yh xh; g, w t, w xh, w yh
      uint64_t q[7] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int k = 0; k < kVpt; ++k) {
        JoinVec xh, t, d;
        start(k, xh, t, d, &q[3], &q[0]);
        if (has_pre) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a1[k][i] = f2_fma(d[i], xh[i], a1[k][i]);
            if (kBeta) a0[k][i] = f2_add(a0[k][i], d[i]);
          }
        }
        if (has_post) {
          JoinVec yh, gw;
          normed_y(k, yh);
          fac.get_w(k, gw);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t wy = f2_mul(gw[i], yh[i]);
            q[1] = f2_fma(wy, t[i], q[1]);
            q[2] = f2_fma(wy, xh[i], q[2]);
            if (kBeta) {
              q[4] = f2_fma(gw[i], t[i], q[4]);
              q[5] = f2_fma(gw[i], xh[i], q[5]);
              q[6] = f2_add(q[6], wy);
            }
          }
        }
        if (kKeep) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            kx[k][i] = xh[i];
            kt[k][i] = t[i];
          }
        }
      }
      float sum[kSums];
#pragma unroll
      for (int i = 0; i < kSums; ++i) sum[i] = join_add_pair(q[i]);
      if (has_pre || has_post) join_sums<kWpr, kCl>(sum, wpr, sh, par);
      // dh = t + xh cx - cg
      const float cx = -stat.w * sum[0] * inv_h;
      float cg = 0.f, u0 = 0.f, u1 = fmaf(cx, sum[2], sum[1]);  // sums of u, u yh
      if constexpr (kBeta) {
        cg = p.pre == MLPB_NORM_LAYER ? stat.w * sum[3] * inv_h : 0.f;
        u1 = fmaf(-cg, sum[6], u1);
        if (p.post == MLPB_NORM_LAYER) u0 = fmaf(-cg, w_sum, fmaf(cx, sum[5], sum[4]));
      }
      const uint64_t cx2 = join_twice(cx);
      [[maybe_unused]] const uint64_t cg2 = join_twice(cg), c0 = join_twice(u0 * inv_h);
      const uint64_t c1 = join_twice(-u1 * inv_h);
#pragma unroll
      for (int k = 0; k < kVpt; ++k) {
        JoinVec dh;
        if constexpr (kKeep) {
#pragma unroll
          for (int i = 0; i < 4; ++i) dh[i] = f2_fma(kx[k][i], cx2, kt[k][i]);
        } else {
          JoinVec xh, d;
          start(k, xh, dh, d, nullptr, nullptr);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dh[i] = f2_fma(xh[i], cx2, dh[i]);
            if (kBeta) dh[i] = f2_sub(dh[i], cg2);
          }
        }
        if (need_x) {
          JoinVec x;
          join_read<XT, true>(st + o_x, k, jc, x);
#pragma unroll
          for (int i = 0; i < 4; ++i) d_alpha = f2_fma(dh[i], x[i], d_alpha);
        }
        if (p.alpha != nullptr) {
          JoinVec dx;
#pragma unroll
          for (int i = 0; i < 4; ++i) dx[i] = f2_mul(alpha, dh[i]);
          join_store<XT, false>(static_cast<XT*>(p.dX) + at, k, jc, dx);
        } else {
          join_store<XT, false>(static_cast<XT*>(p.dX) + at, k, jc, dh);
        }
        if (need_y) {
          JoinVec yh, gw;
          normed_y(k, yh);
          fac.get_w(k, gw);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s1[k][i] = f2_fma(dh[i], yh[i], s1[k][i]);
            if (kBeta) s0[k][i] = f2_add(s0[k][i], dh[i]);
            dh[i] = f2_mul(dh[i], gw[i]);  // u
          }
          if (has_post) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dh[i] = f2_mul(rs_y, f2_fma(yh[i], c1, kBeta ? f2_sub(dh[i], c0) : dh[i]));
          }
        }
        if (has_block) join_store<bf, false>(p.dY + at, k, jc, dh);
      }
      issue(b, row + p.nbuf * step);  // this row's slots have been read
      if (++b == p.nbuf) b = 0;
    }

    // The end of this CTA's rows of the group: S1 and S0 over the CTA, and what they give.
    if (need_y) {
      join_combine(s1, at_once, comb);
      if (kBeta) join_combine(s0, at_once, comb);
      if (place == 0) {
        const int64_t slot = static_cast<int64_t>(walker) * p.H;
#pragma unroll
        for (int k = 0; k < kVpt; ++k) {
          JoinVec w, t;
          if (gate != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = s1[k][i];
            if (has_post) {
              join_unpack(join_param(p.gamma_post, k, jc), w);
#pragma unroll
              for (int i = 0; i < 4; ++i) t[i] = f2_mul(t[i], w[i]);
            }
            if (kBeta && p.beta_post != nullptr) {
              join_unpack(join_param(p.beta_post, k, jc), w);
#pragma unroll
              for (int i = 0; i < 4; ++i) t[i] = f2_fma(w[i], s0[k][i], t[i]);
            }
            if (bpg > 1)
              join_put(p.part_gate + slot, k, jc, t, false);
            else
              join_put(p.dgate + static_cast<int64_t>(g) * p.H, k, jc, t, p.accumulate != 0);
            join_unpack(join_param(gate, k, jc), w);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = join_twice(1.0f);
          }
          if (p.part_gpost != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = f2_mul(w[i], s1[k][i]);
            join_put(p.part_gpost + slot, k, jc, t, !first);
          }
          if (kBeta && p.part_bpost != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = f2_mul(w[i], s0[k][i]);
            join_put(p.part_bpost + slot, k, jc, t, !first);
          }
        }
      }
      first = false;
#pragma unroll
      for (int k = 0; k < kVpt; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s1[k][i] = 0ull;
          if (kBeta) s0[k][i] = 0ull;
        }
    }
  }

  if (has_pre) {
    join_combine(a1, at_once, comb);
    if (kBeta) join_combine(a0, at_once, comb);
    if (place == 0) {
      const int64_t slot = static_cast<int64_t>(walker) * p.H;
#pragma unroll
      for (int k = 0; k < kVpt; ++k) {
        join_put(p.part_gpre + slot, k, jc, a1[k], false);
        if (kBeta && p.part_bpre != nullptr) join_put(p.part_bpre + slot, k, jc, a0[k], false);
      }
    }
  }
  if (need_x) {  // the CTA's part of dalpha, added in warp order
    float d = join_add_pair(d_alpha);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[0][threadIdx.x / 32][0] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
      float t = 0.f;
      for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) t += sh[0][w][0];
      p.part_alpha[blockIdx.x] = t;
    }
  }
}

template <class XT, class YT, int kVpt, int kWpr, bool kBeta, int kCl = 1>
static cudaError_t join_bwd_launch(JoinParams p, const JoinShape& sh, int grid, cudaStream_t s) {
  const bool has_pre = p.pre != MLPB_NORM_NONE, has_post = p.post != MLPB_NORM_NONE;
  const bool need_y = has_post || p.gate != nullptr;
  const int warps = sh.threads / 32;
  const size_t xs = warps * join_slots<XT, kVpt>(), ys = warps * join_slots<YT, kVpt>();
  const size_t early = (has_pre ? xs + ys : 0) + (need_y ? ys : 0);
  const size_t late = (p.dXout != nullptr ? xs : 0) + (p.part_alpha != nullptr ? xs : 0);
  constexpr size_t kFactors = JoinFactors<kVpt, join_bwd_smem<kWpr, kBeta>()>::kBytes;
  // (the general ones' rows meet in memory of their own)
  const size_t comb = sh.rows > 1 && !p.split ? static_cast<size_t>(sh.threads) * kVpt * 32 : 0;
  const size_t room = (208u << 10) / join_ctas(kWpr) - kFactors * sh.threads -
                      (kWpr < 0 ? comb : 0);
  const size_t stage = early + late;  // 160 KB an SM at most: one fits
  p.nbuf = static_cast<int>(std::max<size_t>(
      1, std::min<size_t>(kJoinMaxBuf, room / std::max<size_t>(stage, 1))));
  size_t smem = p.nbuf * stage;
  if (kWpr > 0) smem = std::max(smem, comb);
  p.ring_bytes = static_cast<int>(smem);
  smem += kFactors * sh.threads + (kWpr < 0 ? comb : 0);
  p.ragged = p.H % (256 * kVpt * kCl * sh.wpr) != 0;
  p.wpr = sh.wpr;
  p.rows = sh.rows;
  auto* kernel = join_bwd_kernel<XT, YT, kVpt, kWpr, kBeta, kCl>;
  const cudaError_t e = join_smem_attr(kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid * kCl));
  cfg.blockDim = dim3(static_cast<unsigned>(sh.threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {kCl, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = kCl > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// `sh` is join_bwd_shape's for this call.
template <class XT, class YT, bool kBeta>
static cudaError_t join_bwd_pick(const JoinParams& p, const JoinShape& sh, bool plain, int grid,
                                 cudaStream_t s) {
  if (plain) {
    switch (sh.wpr) {
      case 2: return join_bwd_launch<XT, YT, 2, 2, kBeta>(p, sh, grid, s);
      case 4: return join_bwd_launch<XT, YT, 2, 4, kBeta>(p, sh, grid, s);
      case 8: return join_bwd_launch<XT, YT, 2, 8, kBeta>(p, sh, grid, s);
      default: return join_bwd_launch<XT, YT, 2, 16, kBeta>(p, sh, grid, s);
    }
  }
  if (sh.vpt == 1) return join_bwd_launch<XT, YT, 1, -16, kBeta>(p, sh, grid, s);
  if (sh.cluster == 1)
    return sh.wpr <= 12 ? join_bwd_launch<XT, YT, 2, -12, kBeta>(p, sh, grid, s)
                        : join_bwd_launch<XT, YT, 2, -16, kBeta>(p, sh, grid, s);
  return sh.wpr <= 12 ? join_bwd_launch<XT, YT, 2, -12, kBeta, 2>(p, sh, grid, s)
                      : join_bwd_launch<XT, YT, 2, -16, kBeta, 2>(p, sh, grid, s);
}

template <class XT, class YT>
cudaError_t join_bwd_run(const JoinParams& p, const JoinShape& sh, bool plain, int grid,
                         cudaStream_t s) {
  return p.post == MLPB_NORM_LAYER || p.pre == MLPB_NORM_LAYER
             ? join_bwd_pick<XT, YT, true>(p, sh, plain, grid, s)
             : join_bwd_pick<XT, YT, false>(p, sh, plain, grid, s);
}

}  // namespace mlpb
