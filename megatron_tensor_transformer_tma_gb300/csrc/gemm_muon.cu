// The products of a Newton-Schulz step (muon.cuh) on the tensor cores, for a batch of matrices.
//
// The pipeline is that of gemm.cuh (pairs of CTAs, 256 x 256 tiles, a 7-stage TMA ring, two
// accumulators in tensor memory, bounded waits), on fp16 operands.  The symmetric products (Gram,
// Poly) compute the tiles on and below the diagonal and write those below it twice, the second
// time transposed: a warp's 32 rows are 32 consecutive elements of each mirrored row.
//   wide (rows <= cols)   Gram  A, B = X        K-major   K = cols
//                         Apply A = D K-major, B = X MN-major, K = rows; beta by row
//   tall                  Gram  A, B = X        MN-major  K = rows
//                         Apply A = X, B = D    K-major   K = cols; beta by column
//   Poly                  A, B = E              K-major   K = n
#include <algorithm>

#include "gemm.cuh"
#include "muon.cuh"

namespace mlpb {

// Instruction descriptor of kind::f16 with fp16 operands (format code 0), fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

struct OrthoTile {
  int b, mp, nt;
};

template <OrthoOp Op>
__device__ __forceinline__ OrthoTile ortho_tile(int u, const OrthoParams& p) {
  OrthoTile t;
  if constexpr (Op == OrthoOp::Gram || Op == OrthoOp::Poly) {
    const int per = p.num_pm * (p.num_pm + 1) / 2;
    t.b = u / per;
    const int i = u - t.b * per;  // row by row below the diagonal
    t.mp = static_cast<int>((sqrtf(8.0f * static_cast<float>(i) + 1.0f) - 1.0f) * 0.5f);
    while (t.mp * (t.mp + 1) / 2 > i) --t.mp;
    while ((t.mp + 1) * (t.mp + 2) / 2 <= i) ++t.mp;
    t.nt = i - t.mp * (t.mp + 1) / 2;
  } else {
    const int per = p.num_pm * p.num_n;
    t.b = u / per;
    tile_coords(u - t.b * per, p.num_pm, p.num_n, 8, t.mp, t.nt);
  }
  return t;
}

template <OrthoOp Op, bool kTall>
struct OrthoMajor {
  static constexpr bool a_mn = Op == OrthoOp::Gram && kTall;
  static constexpr bool b_mn =
      (Op == OrthoOp::Gram && kTall) || ((Op == OrthoOp::Apply || Op == OrthoOp::Last) && !kTall);
};

template <bool kMn, bool kPeer>
__device__ __forceinline__ void ortho_load(uint32_t dst, const CUtensorMap* m, uint32_t bar, int k0,
                                           int row, int b) {
  if constexpr (kMn)
    ld4<kPeer>(dst, m, bar, 0, k0, row >> 6, b);
  else
    ld3<kPeer>(dst, m, bar, k0, row, b);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ void load_half32(const __half* p, float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 u = __ldcg(reinterpret_cast<const uint4*>(p + 8 * q));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_half2(w[e]);
      v[8 * q + 2 * e] = f.x;
      v[8 * q + 2 * e + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store_half32(__half* p, const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    st_global_v4(p + 8 * q,
                 make_uint4(pack_half2(v[8 * q], v[8 * q + 1]),
                            pack_half2(v[8 * q + 2], v[8 * q + 3]),
                            pack_half2(v[8 * q + 4], v[8 * q + 5]),
                            pack_half2(v[8 * q + 6], v[8 * q + 7])));
}

// v[e] of a row's 32 columns from `col` on, without its diagonal element, which is returned (0
// where the chunk has none).
__device__ __forceinline__ float take_diagonal(float (&v)[32], int m, int col) {
  float d = 0.0f;
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (col + e == m) {
      d = v[e];
      v[e] = 0.0f;
    }
  return d;
}

// A symmetric matrix's chunk: row m, columns [col, col + 32), and below the diagonal tiles the
// mirrored column.  Rows have 32 elements from `col` on: they are padded to multiples of 64.
__device__ __forceinline__ void store_symmetric(__half* S, int m, int col, int n, int ld,
                                                bool mirror, const float (&v)[32]) {
  if (m >= n) return;
  store_half32(S + static_cast<size_t>(m) * ld + col, v);
  if (mirror) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (col + e < n) S[static_cast<size_t>(col + e) * ld + m] = __float2half_rn(v[e]);
  }
}

template <OrthoOp Op, bool kTall>
__device__ __forceinline__ void ortho_epilogue(uint32_t tacc, int row, int rank, const OrthoTile& t,
                                               const OrthoParams& p) {
  const int m = (t.mp * 2 + rank) * kBM + row;
  const int n0 = t.nt * kBN;
  if constexpr (Op == OrthoOp::Gram || Op == OrthoOp::Poly) {
    const size_t at = static_cast<size_t>(t.b) * p.n * p.ldn;
    const float* diag = p.diag + static_cast<size_t>(t.b) * p.ldn;
    float dm = 0.0f;
    if (Op == OrthoOp::Poly && m < p.n) dm = __ldg(diag + m);
#pragma unroll 1
    for (int c = 0; c < kBN / 32; ++c) {
      const int col = n0 + c * 32;
      if (col >= p.n) break;
      __syncwarp();  // rows past the end and the diagonal's lanes went ways of their own
      float v[32];
      tmem_load_f32x32(tacc + c * 32, v);
      const bool on = t.mp == t.nt && m >= col && m < col + 32;
      if constexpr (Op == OrthoOp::Gram) {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= kXInv;  // A times 2^12
        if (on) {
          const float d = take_diagonal(v, m, col);
          if (m < p.n) p.diag[static_cast<size_t>(t.b) * p.ldn + m] = d * kXInv;
        }
        store_symmetric(p.e + at, m, col, p.n, p.ldn, t.mp != t.nt, v);
      } else {
        if (on) {
          const float d = take_diagonal(v, m, col);
          if (m < p.n)
            p.beta[static_cast<size_t>(t.b) * p.ldn + m] =
                p.a + dm * fmaf(p.c, dm, p.b) + p.c * (d * kEEInv);
        }
        if (m < p.n) {
          float e16[32];
          load_half32(p.e + at + static_cast<size_t>(m) * p.ldn + col, e16);
          const float* dj = diag + col;  // 16-byte aligned: rows of 64
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 d4 = __ldg(reinterpret_cast<const float4*>(dj + 4 * q));
            const float d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 4 * q + i;
              const float lin = fmaf(p.c, dm + d[i], p.b) * (kXInv * kDScale);
              v[e] = fmaf(lin, e16[e], (p.c * (kEEInv * kDScale)) * v[e]);
            }
          }
        }
        store_symmetric(p.d + at, m, col, p.n, p.ldn, t.mp != t.nt, v);
      }
    }
  } else {
    const bool row_ok = m < p.rows;
    const float* beta = p.beta + static_cast<size_t>(t.b) * p.ldn;
    const float bm = !kTall && row_ok ? __ldg(beta + m) : 0.0f;
    const size_t rm = static_cast<size_t>(t.b) * p.rows + m;
    float keep = 0.0f, step = 0.0f;
    if (Op == OrthoOp::Last && p.w != nullptr) {
      const float lr = __ldg(p.lr);
      keep = 1.0f - lr * p.decay;
      step = lr * p.scale * kXInv;
    }
#pragma unroll 1
    for (int c = 0; c < kBN / 32; ++c) {
      const int col = n0 + c * 32;
      if (col >= p.cols) break;
      __syncwarp();  // rows past the end went a way of their own
      float v[32];
      tmem_load_f32x32(tacc + c * 32, v);
      if (!row_ok) continue;
      float hi[32], lo[32];
      load_half32(p.xh + rm * p.ldx + col, hi);
      load_half32(p.xl + rm * p.ldx + col, lo);
      if constexpr (kTall) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 b4 = __ldg(reinterpret_cast<const float4*>(beta + col + 4 * q));
          const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * q + i;
            const float be = col + e < p.cols ? b[i] : 0.0f;  // what is behind the last is no number
            v[e] = fmaf(be, hi[e] + lo[e], v[e] * (1.0f / kDScale));
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = fmaf(bm, hi[e] + lo[e], v[e] * (1.0f / kDScale));
      }
      if constexpr (Op == OrthoOp::Apply) {  // X' times 2^12, in two parts
#pragma unroll
        for (int e = 0; e < 32; ++e) lo[e] = v[e] - __half2float(__float2half_rn(v[e]));
        store_half32(p.xh_out + rm * p.ldx + col, v);
        store_half32(p.xl + rm * p.ldx + col, lo);
      } else {
        const size_t o = rm * p.cols + col;
        const int nv = min(32, p.cols - col);
        if (p.w == nullptr) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= kXInv;
          if (p.cols % 8 == 0) {
            store_bf16x32(p.out + o, nv, v);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e < nv) p.out[o + e] = __float2bfloat16_rn(v[e]);
          }
        } else if (p.cols % 8 == 0) {
          float w[32];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (4 * q < nv) x = __ldcg(reinterpret_cast<const float4*>(p.w + o + 4 * q));
            w[4 * q] = x.x; w[4 * q + 1] = x.y; w[4 * q + 2] = x.z; w[4 * q + 3] = x.w;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = fmaf(-step, v[e], keep * w[e]);
          store_f32x32(p.w + o, nv, w);
          if (p.wb != nullptr) store_bf16x32(p.wb + o, nv, w);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < nv) {
              const float w = fmaf(-step, v[e], keep * p.w[o + e]);
              p.w[o + e] = w;
              if (p.wb != nullptr) p.wb[o + e] = __float2bfloat16_rn(w);
            }
        }
      }
    }
  }
}

template <OrthoOp Op, bool kTall>
__global__ void __launch_bounds__(kGemmThreads, 1)
    ortho_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const OrthoParams p) {
  constexpr int S = kPairStages;
  constexpr bool a_mn = OrthoMajor<Op, kTall>::a_mn, b_mn = OrthoMajor<Op, kTall>::b_mn;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sA0 = base;
  const uint32_t sB0 = base + S * kPairAStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kPairStageBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + S);
  const uint32_t tfull0 = smem_u32(bars + 2 * S);
  const uint32_t tempty0 = smem_u32(bars + 2 * S + 2);
  const uint32_t drain = smem_u32(bars + 2 * S + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int cid = blockIdx.x / 2;
  const int nclusters = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0u;
    mbar_fence_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full_lead = mapa_shared(full0, 0);
  const uint32_t tempty_lead = mapa_shared(tempty0, 0);
  const WaitCtx wc{abort_flag, p.err, p.wait_ns};

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0, armed_par = 0;
      bool skip_once = p.fault_inject != 0 && cid == 0 && leader;
      for (int u = cid; u < p.units; u += nclusters) {
        const OrthoTile t = ortho_tile<Op>(u, p);
        const int ra = (t.mp * 2 + rank) * kBM, rb = t.nt * kBN + 128 * rank;
        bool ok = true;
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!wait_bounded(empty0 + 8 * stage, phase ^ 1u, wc, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          const uint32_t sa = sA0 + stage * kPairAStage, sb = sB0 + stage * kPairBStage;
          if (skip_once) {
            skip_once = false;  // fault injection: this stage is never armed
          } else if (leader) {
            const uint32_t fb = full0 + 8 * stage;
            mbar_arrive_expect_tx(fb, 2 * kPairStageBytes);
            ortho_load<a_mn, false>(sa, &tmA, fb, kb * kBK, ra, t.b);
            ortho_load<b_mn, false>(sb, &tmB, fb, kb * kBK, rb, t.b);
            armed |= 1u << stage;
            armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          } else {
            const uint32_t fb = full_lead + 8 * stage;
            ortho_load<a_mn, true>(sa, &tmA, fb, kb * kBK, ra, t.b);
            ortho_load<b_mn, true>(sb, &tmB, fb, kb * kBK, rb, t.b);
            armed = 1u;
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
      }
      if (leader) {
        for (int s = 0; s < S; ++s)
          if (armed & (1u << s)) wait_drain(full0 + 8 * s, (armed_par >> s) & 1u, wc);
      } else if (armed != 0u && *abort_flag) {
        // as in gemm.cuh: copies that only the even CTA's barriers observe have long landed
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 20000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------------------------------------------------------- MMA issuer (pair)
      constexpr uint32_t idesc = idesc_f16_f32(2 * kBM, kBN, a_mn, b_mn);
      const uint64_t adesc0 = a_mn ? sdesc(sA0, kChunk, 1024, 2u) : sdesc(sA0, 16, 1024, 2u);
      const uint64_t bdesc0 = b_mn ? sdesc(sB0, kChunk, 1024, 2u) : sdesc(sB0, 16, 1024, 2u);
      constexpr uint32_t kAk = (a_mn ? 2048u : 32u) >> 4, kBk = (b_mn ? 2048u : 32u) >> 4;
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      for (int u = cid; u < p.units; u += nclusters, ++it) {
        const int buf = it & 1;
        const uint32_t acc_par = (it >> 1) & 1;
        if (!wait_bounded(tempty0 + 8 * buf, acc_par ^ 1u, wc, kSiteMmaAccEmpty)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * kBN;
        bool ok = true;
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!wait_bounded(full0 + 8 * stage, phase, wc, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t as = adesc0 + static_cast<uint32_t>(stage) * (kPairAStage >> 4);
          const uint64_t bs = bdesc0 + static_cast<uint32_t>(stage) * (kPairBStage >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_pair(d, as + kk * kAk, bs + kk * kBk, idesc,
                           (kb != 0 || kk != 0) ? 1u : 0u);
          umma_commit_pair_mc(empty0 + 8 * stage, 0x3);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair_mc(tfull0 + 8 * buf, 0x3);
      }
      umma_commit_pair(drain);
      wait_drain(drain, 0, wc);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    int it = 0;
    for (int u = cid; u < p.units; u += nclusters, ++it) {
      const int buf = it & 1;
      const uint32_t acc_par = (it >> 1) & 1;
      int ok = 1;
      if (lane == 0)
        ok = wait_bounded(tfull0 + 8 * buf, acc_par, wc, kSiteEpiAccFull) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      __syncwarp();
      tc_fence_after();
      const OrthoTile t = ortho_tile<Op>(u, p);
      ortho_epilogue<Op, kTall>(
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kBN, row, rank, t, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(tempty0 + 8 * buf);
        else mbar_arrive_remote(tempty_lead + 8 * buf);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

using OrthoKernel = void (*)(const CUtensorMap, const CUtensorMap, const OrthoParams);

static OrthoKernel ortho_kernel_of(OrthoOp op, bool tall) {
  switch (op) {
    case OrthoOp::Gram:
      return tall ? ortho_kernel<OrthoOp::Gram, true> : ortho_kernel<OrthoOp::Gram, false>;
    case OrthoOp::Poly:  // the same for both
      return ortho_kernel<OrthoOp::Poly, false>;
    case OrthoOp::Apply:
      return tall ? ortho_kernel<OrthoOp::Apply, true> : ortho_kernel<OrthoOp::Apply, false>;
    default:
      return tall ? ortho_kernel<OrthoOp::Last, true> : ortho_kernel<OrthoOp::Last, false>;
  }
}

static void ortho_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int clusters,
                         cudaStream_t s) {
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2), 1, 1);
  cfg.blockDim = dim3(kGemmThreads, 1, 1);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

cudaError_t ortho_set_attrs(int* max_clusters) {
  for (OrthoOp op : {OrthoOp::Gram, OrthoOp::Poly, OrthoOp::Apply, OrthoOp::Last})
    for (bool tall : {false, true}) {
      const cudaError_t e =
          cudaFuncSetAttribute(reinterpret_cast<const void*>(ortho_kernel_of(op, tall)),
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
      if (e != cudaSuccess) return e;
    }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  ortho_config(cfg, attr, 2, nullptr);
  return cudaOccupancyMaxActiveClusters(max_clusters, ortho_kernel_of(OrthoOp::Gram, false), &cfg);
}

cudaError_t launch_ortho(OrthoOp op, bool tall, const CUtensorMap& a, const CUtensorMap& b,
                         const OrthoParams& p, int clusters, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  ortho_config(cfg, attr, clusters, s);
  return cudaLaunchKernelEx(&cfg, ortho_kernel_of(op, tall), a, b, p);
}

}  // namespace mlpb
