// Products of block-scaled E4M3 matrices on the tensor cores: C = A B^T, scales applied by the
// MMA itself (tcgen05 kind::mxf8f6f4, one scale byte for each row and K = 32; the four MMAs of a
// 128-deep stage take the same byte).
//
// A CTA pair computes a 256 x 256 tile, as in gemm.cuh.  Each CTA (320 threads) has:
//   warp 0      TMA producer: a 6-stage ring of 128 x 128-byte A and B-half tiles, and with every
//               fourth k-block the 512 bytes of scales of the CTA's 128 A rows and the 1024 bytes
//               of all 256 B rows (an SM multiplies its A rows with all of B's), beside the stage;
//   warp 1      in the even CTA: copies scales from both CTAs' shared memory to their tensor
//               memory (tcgen05.cp, in issue order with the MMAs that read them) and issues the
//               MMAs; the scale byte of a k-block is chosen by the instruction descriptor;
//   warps 2..9  epilogue.  The accumulator takes 256 of the 512 columns and scales 32 more, so
//               there is no second one: eight warps take the tile into 128 registers a thread
//               and release it before they convert and store.
//
// An accumulation in the tensor cores cuts off instead of rounding: sums come out too small, by
// 6e-7 of their size after 64 k-blocks and in proportion.  So an fp32 result's sum is taken in
// chunks of 64 k-blocks: dW of 16384 tokens is off by as much as that of 8192.  Chunks are added in
// the epilogue's registers or, where C is added to anyway, in memory, in their order, by TMA, whose
// additions take subnormal values as zeros (16384 x 4096 x 11008 592 us, in registers 547).  128
// sums and the next chunk's are more than 168 registers: 404 bytes a thread are spilled.  That costs
// 3 % (the product alone 485 us without chunks, 499 so compiled and still without), the drain after
// each chunk, which nothing overlaps, 5 % more (523).  A bf16 result's sum is taken at once, however
// long: what is cut off is far below its own rounding.
//
// Measured at 8192 x 5120 x 20480: Y 498-525 us (3270-3450 TFLOP/s), 80-85 % of the cycles with
// the tensor cores active; dX 537, dW (fp32, 64 k-blocks) 545.  What is left is the one
// accumulator's drain between tiles, and the power limit.
#include <algorithm>

#include "../../include/mlpb.h"
#include "gemm.cuh"
#include "linear8.cuh"

namespace mlpb {

constexpr int kMxThreads = 320;
constexpr int kMxEpiWarps = 8;
constexpr int kMxChunk = 64;                   // k-blocks summed in the tensor cores, fp32 results
constexpr int kMxScaleBytes = 3 * kB128Chunk;  // 128 A rows, 256 B rows
constexpr int kMxStagedBelow = 32;             // k-blocks
constexpr int kMxBox = 4096;                    // 32 rows of 128 bytes of a result
constexpr int kMxScaleCol = 256;               // tensor-memory column of the first scales
constexpr int kMxScaleCols = 16;               // 4 of A, 8 of B, twice

// How a tile's results leave.
enum class MxOut {
  Direct,   // from the threads of their rows; behind the next tile's products where K is long
  Staged,   // through shared memory by TMA: two slots of 4 KB a warp, and two stages fewer; the
            // chunks of a long sum one by one, added in memory
  Chunked,  // as Direct, of sums longer than a chunk, which are added in registers
};

template <MxOut O>
struct MxSmem {
  static constexpr int stages = O == MxOut::Staged ? 4 : 6;
  static constexpr int slots = O == MxOut::Staged ? kMxEpiWarps * 2 * kMxBox : 0;
  static constexpr int bytes = stages * (kPairStageBytes + kMxScaleBytes) + slots + 2048 + 256;
  static_assert(bytes <= 232448, "shared memory of a CTA");
};
static_assert(kPairAStage == 128 * 128 && kPairBStage == 128 * 128, "E4M3 tiles");

// Instruction descriptor of kind::mxf8f6f4: E4M3 operands, both K-major, UE8M0 scales; the scale
// bytes' place in their words is added for each k-block.
//   bits 4-5 byte of B's scale word  7-9, 10-12 formats (0 = E4M3)  17-22 N >> 3
//   bit 23 UE8M0  24-28 M >> 4  29-30 byte of A's scale word
__host__ __device__ constexpr uint32_t idesc_mx_e4m3(int M, int N, int byte) {
  return (static_cast<uint32_t>(byte) << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(byte) << 29);
}

__device__ __forceinline__ void umma_mx_pair(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 rows of 16 bytes from both CTAs' shared memory to the four lane quarters of their own
// tensor memory.
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}

template <bool kPeer>
__device__ __forceinline__ void issue_scales(const CUtensorMap* ma, const CUtensorMap* mb,
                                             uint32_t dst, uint32_t bar, int group, int mt, int nt,
                                             const B128Params& p) {
  // tiles past the end are of rows that are not stored
  const int ra = group * p.a_tiles + min(mt, p.a_tiles - 1);
  const int rb = group * p.b_tiles;
  ld2<kPeer>(dst, ma, bar, 0, ra);
  ld2<kPeer>(dst + kB128Chunk, mb, bar, 0, rb + min(2 * nt, p.b_tiles - 1));
  ld2<kPeer>(dst + 2 * kB128Chunk, mb, bar, 0, rb + min(2 * nt + 1, p.b_tiles - 1));
}

template <MxOut O>
__global__ void __launch_bounds__(kMxThreads, 1)
    gemm_b128_kernel(const __grid_constant__ B128Maps maps, const B128Params p) {
  using Sm = MxSmem<O>;
  constexpr int S = Sm::stages;
  constexpr bool kTurns = O != MxOut::Direct;  // sums in chunks
  constexpr bool kChunked = O == MxOut::Chunked;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sA0 = base;
  const uint32_t sB0 = base + S * kPairAStage;
  const uint32_t sc0 = base + S * kPairStageBytes;
  const uint32_t slots = (sc0 + S * kMxScaleBytes + 1023u) & ~1023u;  // boxes begin on 1024 bytes
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (slots + Sm::slots - base));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 3);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + S);
  const uint32_t tfull = smem_u32(bars + 2 * S);
  const uint32_t tempty = smem_u32(bars + 2 * S + 1);
  const uint32_t drain = smem_u32(bars + 2 * S + 2);

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
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * kMxEpiWarps);
    mbar_init(drain, 1);
    *abort_flag = 0u;
    mbar_fence_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
    tma_prefetch_desc(&maps.sa);
    tma_prefetch_desc(&maps.sb);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  pdl_launch_next();
  pdl_wait();  // an operand may come from the kernel before this one
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full_lead = mapa_shared(full0, 0);
  const uint32_t tempty_lead = mapa_shared(tempty, 0);

  const WaitCtx wc{abort_flag, p.err, p.wait_ns};
  const int num_units = p.num_pm * p.num_n;
  // a pair's turns: its tiles, each in chunks of K
  const int chunks = kTurns && p.num_kb > p.chunk ? (p.num_kb + p.chunk - 1) / p.chunk : 1;
  const int turns = (num_units - cid + nclusters - 1) / nclusters * chunks;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0, armed_par = 0;
      bool skip_once = p.fault_inject != 0 && cid == 0 && leader;
      for (int u = cid; u < num_units; u += nclusters) {
        int mp, nt;
        tile_coords(u, p.num_pm, p.num_n, p.raster_group, mp, nt);
        const int mt = mp * 2 + rank;
        bool ok = true;
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!wait_bounded(empty0 + 8 * stage, phase ^ 1u, wc, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          const uint32_t sa = sA0 + stage * kPairAStage, sb = sB0 + stage * kPairBStage;
          const bool scales = (kb & 3) == 0;
          const uint32_t sd = sc0 + stage * kMxScaleBytes;
          if (skip_once) {
            skip_once = false;  // fault injection: this stage is never armed
          } else if (leader) {
            const uint32_t fb = full0 + 8 * stage;
            mbar_arrive_expect_tx(fb, 2 * (kPairStageBytes + (scales ? kMxScaleBytes : 0)));
            ld2<false>(sa, &maps.a, fb, kb * kB128, mt * kBM);
            ld2<false>(sb, &maps.b, fb, kb * kB128, nt * kBN);
            if (scales) issue_scales<false>(&maps.sa, &maps.sb, sd, fb, kb >> 2, mt, nt, p);
            armed |= 1u << stage;
            armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          } else {
            const uint32_t fb = full_lead + 8 * stage;
            ld2<true>(sa, &maps.a, fb, kb * kB128, mt * kBM);
            ld2<true>(sb, &maps.b, fb, kb * kB128, nt * kBN + 128);
            if (scales) issue_scales<true>(&maps.sa, &maps.sb, sd, fb, kb >> 2, mt, nt, p);
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
      static_assert(Sm::bytes < 256 * 1024, "descriptor address field");
      const uint64_t adesc0 = sdesc(sA0, 16, 1024, 2u), bdesc0 = sdesc(sB0, 16, 1024, 2u);
      const uint64_t sdesc0 = sdesc(sc0, 16, 128, 0u);  // 8-row groups of 128 bytes
      constexpr uint32_t idesc0 = idesc_mx_e4m3(2 * kBM, kBN, 0);
      constexpr uint32_t byte1 = idesc_mx_e4m3(2 * kBM, kBN, 1) - idesc0;
      int stage = 0;
      uint32_t phase = 0, sbuf = 0;
      for (int it = 0; it < turns; ++it) {
        const int kb0 = kTurns ? it % chunks * p.chunk : 0;
        const int kb1 = kTurns && chunks > 1 ? min(p.num_kb, kb0 + p.chunk) : p.num_kb;
        if (!wait_bounded(tempty, (it & 1) ^ 1u, wc, kSiteMmaAccEmpty)) break;
        tc_fence_after();
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bounded(full0 + 8 * stage, phase, wc, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t byte = kb & 3;
          if (byte == 0u) {  // the scales of this k-block and of the three after it
            sbuf ^= 1u;
            const uint64_t sd = sdesc0 + static_cast<uint32_t>(stage) * (kMxScaleBytes >> 4);
            const uint32_t t = tmem_base + kMxScaleCol + sbuf * kMxScaleCols;
#pragma unroll
            for (int c = 0; c < 3; ++c)
              tmem_copy_scales_pair(t + 4 * c, sd + c * (kB128Chunk >> 4));
          }
          const uint32_t sfa = tmem_base + kMxScaleCol + sbuf * kMxScaleCols;
          const uint32_t idesc = idesc0 + byte * byte1;
          const uint64_t as = adesc0 + static_cast<uint32_t>(stage) * (kPairAStage >> 4);
          const uint64_t bs = bdesc0 + static_cast<uint32_t>(stage) * (kPairBStage >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_mx_pair(tmem_base, as + kk * 2, bs + kk * 2, idesc, sfa, sfa + 4,
                         (kb != kb0 || kk != 0) ? 1u : 0u);
          umma_commit_pair_mc(empty0 + 8 * stage, 0x3);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair_mc(tfull, 0x3);
      }
      umma_commit_pair(drain);
      wait_drain(drain, 0, wc);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;  // columns [128 half, 128 half + 128) of the tile
    const uint32_t tacc =
        tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 128u * half;
    uint32_t v[4][32];  // the tile's sums
    for (int it = 0; it < turns; ++it) {
      const int chunk = kTurns ? it % chunks : 0;
      const int u = cid + (kTurns ? it / chunks : it) * nclusters;
      int ok = 1;
      if (lane == 0) ok = wait_bounded(tfull, it & 1, wc, kSiteEpiAccFull) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      __syncwarp();
      tc_fence_after();
      if (!kChunked || chunk == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tacc + 32 * c, v[c]);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tacc + 16 * c, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            uint32_t& sum = v[c >> 1][16 * (c & 1) + e];
            sum = __float_as_uint(__uint_as_float(sum) + __uint_as_float(r[e]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(tempty);
        else mbar_arrive_remote(tempty_lead);
      }
      if (kChunked && chunk != chunks - 1) continue;
      int mp, nt;
      tile_coords(u, p.num_pm, p.num_n, p.raster_group, mp, nt);
      const int m0 = (mp * 2 + rank) * kBM + quarter * 32, m = m0 + lane;
      const int n0 = nt * kBN + 128 * half;
      if constexpr (O == MxOut::Staged) {
        if (m0 >= p.M) continue;  // the warp's rows, all of them
        const int width = p.out_f32 ? 32 : 64;  // columns of a box
        const int boxes = min(128 / width, (p.N - n0 + width - 1) / width);
        if (chunk > 0 && lane == 0) bulk_wait<0>();  // the chunk before is in C
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q >= boxes) break;
          const uint32_t box = slots + ((warp - 2) * 2 + (q & 1)) * kMxBox;
          if (lane == 0) bulk_wait_read<1>();  // the slot's last box
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t to = box + lane * 128 + ((j ^ (lane & 7)) << 4);
            uint4 w;
            if (p.out_f32) {
              w = make_uint4(v[q][4 * j], v[q][4 * j + 1], v[q][4 * j + 2], v[q][4 * j + 3]);
            } else {  // boxes 0 and 1: sums of chunks 2 q and 2 q + 1
              const uint32_t* x = &v[(2 * q + j / 4) & 3][8 * (j & 3)];
              w = make_uint4(pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                             pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                             pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                             pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7])));
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(w.x), "r"(w.y),
                         "r"(w.z), "r"(w.w)
                         : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (p.accumulate || chunk > 0) tma_add_2d(&maps.c, box, n0 + q * width, m0);
            else tma_store_2d(&maps.c, box, n0 + q * width, m0);
            bulk_commit();
          }
        }
        // Boxes take the two slots in turns from the first one on, so that a slot's last box is
        // read when at most one later box is not.  A tile at C's right edge that ends with the
        // first slot would break the turns: its boxes are read before the next tile begins.
        if ((boxes & 1) != 0 && lane == 0) bulk_wait_read<0>();
        continue;
      }
      if (m >= p.M) continue;
      const size_t o = static_cast<size_t>(m) * p.N + n0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int nv = p.N - n0 - 32 * c;  // a multiple of 8
        if (nv <= 0) break;
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[c][e]);
        if (p.out_f32) {
          float* C = static_cast<float*>(p.C) + o + 32 * c;
          store_f32x32(C, nv, f);
        } else {
          store_bf16x32(static_cast<__nv_bfloat16*>(p.C) + o + 32 * c, nv, f);
        }
      }
    }
    if (O == MxOut::Staged && lane == 0) bulk_wait_read<0>();
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

template <MxOut O>
static void pair_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int clusters,
                        cudaStream_t s) {
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2), 1, 1);
  cfg.blockDim = dim3(kMxThreads, 1, 1);
  cfg.dynamicSmemBytes = MxSmem<O>::bytes;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // it begins with pdl_wait
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

template <MxOut O>
static cudaError_t launch_out(const B128Maps& m, const B128Params& p, int clusters,
                              cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  pair_config<O>(cfg, attr, clusters, s);
  return cudaLaunchKernelEx(&cfg, gemm_b128_kernel<O>, m, p);
}

template <MxOut O>
static cudaError_t attrs_of() {
  return cudaFuncSetAttribute(gemm_b128_kernel<O>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              MxSmem<O>::bytes);
}

int b128_chunk(bool out_f32) { return out_f32 ? kMxChunk : 1 << 30; }

cudaError_t b128_gemm_set_attrs(int* max_clusters) {
  for (cudaError_t e :
       {attrs_of<MxOut::Direct>(), attrs_of<MxOut::Staged>(), attrs_of<MxOut::Chunked>()})
    if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  pair_config<MxOut::Chunked>(cfg, attr, 2, nullptr);
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(max_clusters, gemm_b128_kernel<MxOut::Chunked>, &cfg);
}

// Staged where the products of a tile (0.13 us a k-block) no longer hide its stores by threads, and
// where C is added to, which the TMA does in memory: loads by threads, of 32 lines
// each, doubled the time (dW 5120 x 5120 of 4096 tokens 237 us, now 114).
bool b128_staged(int num_kb, bool accumulate) { return num_kb < kMxStagedBelow || accumulate; }

cudaError_t launch_b128_gemm(const B128Maps& m, const B128Params& p, int clusters,
                             cudaStream_t s) {
  if (b128_staged(p.num_kb, p.accumulate != 0)) return launch_out<MxOut::Staged>(m, p, clusters, s);
  return p.num_kb > p.chunk ? launch_out<MxOut::Chunked>(m, p, clusters, s)
                            : launch_out<MxOut::Direct>(m, p, clusters, s);
}

}  // namespace mlpb
