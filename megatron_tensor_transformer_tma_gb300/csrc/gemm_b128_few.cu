// Products of block-scaled E4M3 matrices with few tiles: few rows of B (tokens of a decoding step),
// or small matrices, C [B rows][A rows] = B A^T.
//
// With few tokens the product is the bytes of A (a weight, one byte an element), so A's rows are
// the MMA's 128 and the tokens its columns (16 to 128), and what matters is that all SMs load
// without a pause: two CTAs an SM, each with a ring of 16 KB tiles of A in flight, and K cut into
// ranges for the CTAs of a cluster (up to eight) until the SMs are full.  The ranges' sums go
// through distributed shared memory: each CTA adds one slice of the tile, in the order of the
// ranges, so that the bits are the same every run, and stores it.
//
// The kernel is launched to begin while the quantization of B's rows ends (pdl_wait): A and its
// scales, which that does not write, are on their way by then.  A CTA (192 threads) has a TMA
// producer, an MMA issuer and four epilogue warps; scales as in gemm_b128.cu.
//
// Bound by the weight's bytes: one token by 5120 x 20480 takes 17.2 us with its quantization in a
// graph of such calls (105 MB: 6.1 TB/s), 16 tokens by 11008 x 4096 11.9.  Depth of the rings
// counts: three and four CTAs an SM, with three and two stages, took 22.8 and 28.8 us where two
// with five took 21.8.
#include <algorithm>

#include "../../include/mlpb.h"
#include "gemm.cuh"
#include "linear8.cuh"

namespace mlpb {

constexpr int kFewThreads = 192;
constexpr int kFewMaxCluster = 8;
constexpr int kFewMaxStages = 8;
constexpr int kFewCtasPerSm = 2;
constexpr int kFewSmem = 232448 / kFewCtasPerSm - 1024;
constexpr int kFewATile = kBM * kB128;

struct FewShape {
  int columns;  // of the MMA: B's rows in a tile, a multiple of 16 up to 128
  int stages;
  __host__ __device__ int stage_bytes() const {
    return kFewATile + columns * kB128 + 2 * kB128Chunk;
  }
};

static FewShape few_shape(int64_t b_rows) {
  FewShape s;
  s.columns = static_cast<int>(std::min<int64_t>(128, (b_rows + 15) / 16 * 16));
  s.stages = std::min(kFewMaxStages, (kFewSmem - 1024 - 256) / s.stage_bytes());
  return s;
}

__device__ __forceinline__ void umma_mx_one(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_copy_scales_one(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

struct FewParams {
  int a_rows, b_rows, num_kb;
  int a_tiles, b_tiles;      // tiles of C: 128 rows of A, `columns` rows of B
  int a_stiles, b_stiles;    // 128-row tiles that the scales have
  int cluster;
  FewShape shape;
  uint32_t tmem_columns;
  int out_f32;
  void* C;
  uint32_t* err;
  uint64_t wait_ns;
  int fault_inject;
};

__global__ void __launch_bounds__(kFewThreads)
    gemm_b128_few_kernel(const __grid_constant__ B128Maps maps, const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int S = p.shape.stages, N = p.shape.columns;
  const uint32_t stage_bytes = static_cast<uint32_t>(p.shape.stage_bytes());
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * stage_bytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kFewMaxStages + 2);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kFewMaxStages;
  const uint32_t tfull = empty0 + 8 * kFewMaxStages, drain = tfull + 8;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / p.cluster;
  const int ta = tile % p.a_tiles, tb = tile / p.a_tiles;
  // this CTA's k-blocks, in whole groups of four, which share words of scales
  const int groups = (p.num_kb + 3) / 4;
  const int kb0 = groups * rank / p.cluster * 4;
  const int kb1 = min(p.num_kb, groups * (rank + 1) / p.cluster * 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(tfull, 1);
    mbar_init(drain, 1);
    *abort_flag = 0u;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc_one(smem_u32(tmem_slot), p.tmem_columns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_next();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtx wc{abort_flag, p.err, p.wait_ns};

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------------- producer
      // stage: A's tile, B's tile, A's scales, B's scales
      const bool skip = p.fault_inject != 0 && blockIdx.x == 0;
      auto load_a = [&](int kb, int stage) {
        const uint32_t st = base + stage * stage_bytes, fb = full0 + 8 * stage;
        const bool scales = (kb & 3) == 0;
        if (skip && kb == kb0) return;  // fault injection: this stage is never armed
        mbar_arrive_expect_tx(fb, static_cast<uint32_t>(kFewATile + N * kB128 +
                                                        (scales ? 2 * kB128Chunk : 0)));
        tma_load_2d(st, &maps.a, fb, kb * kB128, ta * kBM);
        if (scales)
          tma_load_2d(st + kFewATile + N * kB128, &maps.sa, fb, 0, (kb >> 2) * p.a_stiles + ta);
      };
      auto load_b = [&](int kb, int stage) {
        const uint32_t st = base + stage * stage_bytes, fb = full0 + 8 * stage;
        if (skip && kb == kb0) return;
        tma_load_2d(st + kFewATile, &maps.b, fb, kb * kB128, tb * N);
        if ((kb & 3) == 0)
          tma_load_2d(st + kFewATile + N * kB128 + kB128Chunk, &maps.sb, fb, 0,
                      (kb >> 2) * p.b_stiles + tb);
      };
      const int first = min(S, kb1 - kb0);
      for (int i = 0; i < first; ++i) load_a(kb0 + i, i);
      pdl_wait();  // B is written by the kernel before this one
      for (int i = 0; i < first; ++i) load_b(kb0 + i, i);
      uint32_t armed = (1u << first) - 1u, armed_par = 0u;  // the parity of a stage's last use
      if (skip) armed &= ~1u;
      int stage = 0;
      uint32_t phase = 0;  // the parity of a stage's use before
      for (int kb = kb0 + first; kb < kb1; ++kb) {
        if (!wait_bounded(empty0 + 8 * stage, phase, wc, kSiteProducerEmpty)) break;
        load_a(kb, stage);
        load_b(kb, stage);
        armed |= 1u << stage;
        armed_par = (armed_par & ~(1u << stage)) | ((phase ^ 1u) << stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // every copy that was issued lands before shared memory is given up
      for (int s = 0; s < S; ++s)
        if (armed & (1u << s)) wait_drain(full0 + 8 * s, (armed_par >> s) & 1u, wc);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------------- MMA issuer
      // (kind::mxf8f6f4 as in gemm_b128.cu, one CTA: M = 128)
      const uint32_t idesc0 = (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
                              (static_cast<uint32_t>(kBM >> 4) << 24);
      constexpr uint32_t byte1 = (1u << 4) | (1u << 29);
      const uint64_t adesc0 = sdesc(base, 16, 1024, 2u);
      const uint64_t bdesc0 = sdesc(base + kFewATile, 16, 1024, 2u);
      const uint64_t sdesc0 = sdesc(base + kFewATile + N * kB128, 16, 128, 0u);
      const uint32_t scale_col = tmem_base + static_cast<uint32_t>(N);
      int stage = 0;
      uint32_t phase = 0, sbuf = 0;
      bool ok = true;
      pdl_wait();  // the bounded waits count from where B may come
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_bounded(full0 + 8 * stage, phase, wc, kSiteMmaFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t off = static_cast<uint64_t>(stage) * (stage_bytes >> 4);
        const uint32_t byte = kb & 3;
        if (byte == 0u) {
          sbuf ^= 1u;
          tmem_copy_scales_one(scale_col + 8 * sbuf, sdesc0 + off);
          tmem_copy_scales_one(scale_col + 8 * sbuf + 4, sdesc0 + off + (kB128Chunk >> 4));
        }
        const uint32_t sf = scale_col + 8 * sbuf;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_mx_one(tmem_base, adesc0 + off + kk * 2, bdesc0 + off + kk * 2,
                      idesc0 + byte * byte1, sf, sf + 4, (kb != kb0 || kk != 0) ? 1u : 0u);
        umma_commit_one(empty0 + 8 * stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) umma_commit_one(tfull);
      umma_commit_one(drain);
      wait_drain(drain, 0, wc);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    int ok = 1;
    pdl_wait();
    if (lane == 0) ok = wait_bounded(tfull, 0, wc, kSiteEpiAccFull) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    if (ok) {
      tc_fence_after();
      const int m = ta * kBM + row;
      float* sums = reinterpret_cast<float*>(smem);  // the ring is empty: [columns][128]
      for (int c = 0; c < N; c += 16) {
        if (p.cluster == 1 && tb * N + c >= p.b_rows) break;
        __syncwarp();
        uint32_t r[16];
        tmem_ld_32x32b_x16(tacc + c, r);
        tmem_ld_wait();
        if (p.cluster > 1) {
#pragma unroll
          for (int e = 0; e < 16; ++e) sums[(c + e) * kBM + row] = __uint_as_float(r[e]);
        } else if (m < p.a_rows) {
          const int b0 = tb * N + c, rows = min(16, p.b_rows - b0);
          const size_t o = static_cast<size_t>(b0) * p.a_rows + m;
          if (p.out_f32) {
            float* C = static_cast<float*>(p.C) + o;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < rows) C[static_cast<size_t>(e) * p.a_rows] = __uint_as_float(r[e]);
          } else {
            __nv_bfloat16* C = static_cast<__nv_bfloat16*>(p.C) + o;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < rows)
                C[static_cast<size_t>(e) * p.a_rows] = __float2bfloat16_rn(__uint_as_float(r[e]));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.cluster > 1) {
    cluster_sync();  // every range's sums are there
    const int pieces = N * (kBM / 4);  // four rows of A each
    const int b_left = min(N, p.b_rows - tb * N);
    const int q1 = pieces * (rank + 1) / p.cluster;
    for (int q = pieces * rank / p.cluster + threadIdx.x; q < q1; q += kFewThreads) {
      const int t = q / (kBM / 4), m = ta * kBM + (q % (kBM / 4)) * 4;
      if (t >= b_left || m >= p.a_rows) continue;
      float4 s[kFewMaxCluster];
#pragma unroll
      for (int r = 0; r < kFewMaxCluster; ++r)
        if (r < p.cluster) s[r] = ld_cluster4(mapa_shared(base + 16 * q, r));
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < kFewMaxCluster; ++r)
        if (r < p.cluster) {
          v[0] += s[r].x;
          v[1] += s[r].y;
          v[2] += s[r].z;
          v[3] += s[r].w;
        }
      const size_t o = static_cast<size_t>(tb * N + t) * p.a_rows + m;
      if (p.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.C) + o) =
            make_float4(v[0], v[1], v[2], v[3]);
      } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.C) + o) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    }
    cluster_sync();  // nobody reads this CTA's sums any more
  }
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_one(tmem_base, p.tmem_columns);
  }
}

static void few_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int ctas, int cluster,
                       cudaStream_t s) {
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kFewThreads, 1, 1);
  cfg.dynamicSmemBytes = kFewSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

int b128_few_columns(int64_t b_rows) { return few_shape(b_rows).columns; }

cudaError_t b128_few_set_attrs(int* slots) {
  cudaError_t e = cudaFuncSetAttribute(gemm_b128_few_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  if (e != cudaSuccess) return e;
  for (int c = 1, i = 0; c <= kFewMaxCluster; c *= 2, ++i) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    few_config(cfg, attr, c, c, nullptr);
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&slots[i], gemm_b128_few_kernel, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_b128_few(const B128Maps& m, const B128Params& b, const int* slots,
                            cudaStream_t s) {
  FewParams p{};
  // C's rows are B's: the operands trade places
  p.a_rows = b.N;
  p.b_rows = b.M;
  p.num_kb = b.num_kb;
  p.shape = few_shape(b.M);
  p.a_tiles = (b.N + kBM - 1) / kBM;
  p.b_tiles = (b.M + p.shape.columns - 1) / p.shape.columns;
  p.a_stiles = b.b_tiles;
  p.b_stiles = b.a_tiles;
  p.tmem_columns = 32;
  while (p.tmem_columns < static_cast<uint32_t>(p.shape.columns + 16)) p.tmem_columns *= 2;
  p.out_f32 = b.out_f32;
  p.C = b.C;
  p.err = b.err;
  p.wait_ns = b.wait_ns;
  p.fault_inject = b.fault_inject;
  // Ranges of K while every cluster is resident at once with a CTA an SM (what the occupancy call
  // counts for a kernel with tensor memory; two are) and has a group of k-blocks for each.  Two
  // ranges of few k-blocks do not pay for the sums of many columns (128 x 1024 x 1024 9.5 us, 8.5
  // without).
  const int tiles = p.a_tiles * p.b_tiles, groups = (p.num_kb + 3) / 4;
  p.cluster = 1;
  for (int c = 2, i = 1; c <= kFewMaxCluster; c *= 2, ++i)
    if (tiles <= slots[i] && c <= groups) p.cluster = c;
  if (p.cluster == 2 && p.shape.columns > 32 && groups < 8) p.cluster = 1;
  B128Maps swapped;
  swapped.a = m.b;
  swapped.b = m.a;
  swapped.sa = m.sb;
  swapped.sb = m.sa;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  few_config(cfg, attr, tiles * p.cluster, p.cluster, s);
  return cudaLaunchKernelEx(&cfg, gemm_b128_few_kernel, swapped, p);
}

}  // namespace mlpb
