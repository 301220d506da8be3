// The whole orthogonalised update of matrices whose smaller side is at most 128, in one launch: a
// matrix lies in the shared memory of a cluster of CTAs from the first step to the last.
//
// With n <= 128 a product is a few million operations on one tile, and the launches, pipeline
// starts and trips through L2 of fifteen tensor-core launches cost far more than the products
// (one 64 x 4096 matrix: 190 us; here profiles give its time in the table below).  Each CTA keeps a
// slab of the longer side, X [n][slab] in two fp16 parts (muon.cuh has the number formats); a tall
// matrix is transposed as it is read and written, since the polynomial of X^T is that of X
// transposed.  A step is
//   1. each CTA's share of X X^T over its slab (mma.sync; 16 warps, 32 x 32 blocks, the slab split
//      between warps where there are fewer than 16 blocks);
//   2. the sum over CTAs, in rank order: each CTA adds one slice through distributed shared memory
//      and writes E and d to all;
//   3. E E, D and beta, by every CTA for itself;
//   4. X <- beta X + D X in place: a warp takes 16 columns, holds them all in registers as operands
//      and overwrites them.
// Two barriers of the cluster a step.  mma.sync instead of tcgen05: fragments go between
// registers and both layouts of shared memory without descriptors, tensor memory or a pipeline to
// start, and the products are not what bounds it.
#include <algorithm>

#include "muon_update.cuh"
#include "ptx.cuh"

namespace mlpb {

constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallMaxN = 128;
constexpr int kSmallMaxCluster = 16;
constexpr size_t kSmallMaxSmem = 232448;

struct SmallShape {
  int np;    // n rounded up to 32
  int ns;    // elements of a row of E and D: np rounded up to 64
  int slab;  // columns of X in a CTA, a multiple of 64
  int splits;  // of the slab in step 1
  __host__ __device__ size_t x_bytes() const { return static_cast<size_t>(np) * slab * 2; }
  __host__ __device__ size_t e_bytes() const { return static_cast<size_t>(np) * ns * 2; }
  // the partial sums, later D
  __host__ __device__ size_t p_bytes() const {
    return static_cast<size_t>(splits) * np * np * 4;
  }
  __host__ __device__ size_t bytes() const {
    return 2 * x_bytes() + e_bytes() + p_bytes() + 2 * kSmallMaxN * 4 + 512;
  }
};

static SmallShape small_shape(int n, int64_t length, int cluster) {
  SmallShape s;
  s.np = (n + 31) / 32 * 32;
  s.ns = (s.np + 63) / 64 * 64;
  s.slab = static_cast<int>((length + cluster * 64 - 1) / (cluster * 64)) * 64;
  const int blocks = (s.np / 32) * (s.np / 32);
  s.splits = std::max(1, kSmallWarps / blocks);
  return s;
}

struct SmallParams {
  MuonInput in;
  SmallShape shape;
  int n, cluster, steps, tall;
  int64_t length;  // of the longer side
  float a, b, c;
  __nv_bfloat16* out;
  float* w;
  __nv_bfloat16* wb;
  const float* lr;
  float decay, scale;
};

// Element (row, col) of a swizzled matrix of fp16: 16-byte pieces of a row change places within
// groups of eight, so that eight rows' pieces of one column lie in different banks.
__device__ __forceinline__ int swz(int row, int col, int stride) {
  return row * stride + ((((col >> 3) ^ (row & 7)) << 3) | (col & 7));
}

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 ld_remote4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void st_remote8(uint32_t cluster_addr, uint2 v) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(cluster_addr), "r"(v.x), "r"(v.y)
               : "memory");
}

__device__ __forceinline__ void st_remote4(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A 32 x 32 block of S S^T at rows i0 and j0 over columns [k0, k1) of a swizzled matrix.
__device__ __forceinline__ void block_product(float (&acc)[2][4][4], uint32_t s, int stride, int i0,
                                              int j0, int k0, int k1, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
  const int ar = lane & 15, ak = (lane >> 4) * 8;                        // rows, then k
  const int br = (lane & 7) + ((lane >> 4) << 3), bk = ((lane >> 3) & 1) * 8;  // k, then rows
  for (int k = k0; k < k1; k += 16) {
    uint32_t a[2][4], b[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) ldm4(s + 2 * swz(i0 + 16 * i + ar, k + ak, stride), a[i]);
#pragma unroll
    for (int j = 0; j < 2; ++j) ldm4(s + 2 * swz(j0 + 16 * j + br, k + bk, stride), b[j]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        mma_f16(acc[i][j], a[i], b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kSmallThreads, 1) muon_small_kernel(const SmallParams p) {
  extern __shared__ __align__(1024) uint8_t small_smem[];
  const SmallShape sh = p.shape;
  const int np = sh.np, ns = sh.ns, slab = sh.slab;
  __half* xh = reinterpret_cast<__half*>(small_smem);
  __half* xl = reinterpret_cast<__half*>(small_smem + sh.x_bytes());
  __half* e = reinterpret_cast<__half*>(small_smem + 2 * sh.x_bytes());
  float* part = reinterpret_cast<float*>(small_smem + 2 * sh.x_bytes() + sh.e_bytes());
  __half* d = reinterpret_cast<__half*>(part);  // once the partial sums have been read
  float* diag = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(part) + sh.p_bytes());
  float* beta = diag + kSmallMaxN;
  float4* squares = reinterpret_cast<float4*>(beta + kSmallMaxN);  // a warp each, then the CTA's
  float* factors = reinterpret_cast<float*>(squares + kSmallWarps + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t matrix = blockIdx.x / p.cluster;
  const int64_t l0 = static_cast<int64_t>(rank) * slab;
  const int width = static_cast<int>(max(static_cast<int64_t>(0),
                                         min(static_cast<int64_t>(slab), p.length - l0)));
  const int64_t elems = p.in.rows * p.in.cols;
  const T* g = static_cast<const T*>(p.in.g) + matrix * elems;
  float* m = p.in.m == nullptr ? nullptr : p.in.m + matrix * elems;
  // this CTA's elements: `runs` runs of `run` consecutive ones, `pitch` apart
  const int runs = p.tall ? 1 : p.n;
  const int run = p.tall ? width * p.n : width;
  const int64_t start = p.tall ? l0 * p.n : l0;
  const int64_t pitch = p.in.cols;  // of a wide matrix
  const int quads = (run + 3) / 4;
  const bool vec = p.in.cols % 4 == 0;  // rows, slabs and matrices then begin on 16 bytes

  // ------------------------------------------------------------ momentum and norm
  float4 sq = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = tid; i < runs * quads; i += kSmallThreads) {
    const int r = i / quads, o = (i - r * quads) * 4;
    const int64_t at = start + r * pitch + o;
    float u[4];
    update4<true>(g + at, m == nullptr ? nullptr : m + at, min(4, run - o), vec, p.in.momentum,
                  p.in.nesterov, u);
    add_squares4(u, sq);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sq.x += __shfl_xor_sync(0xffffffffu, sq.x, o);
    sq.y += __shfl_xor_sync(0xffffffffu, sq.y, o);
    sq.z += __shfl_xor_sync(0xffffffffu, sq.z, o);
  }
  if (lane == 0) squares[warp] = sq;
  // zeros where no element of the matrix lies
  for (int i = tid; i < np * slab / 8; i += kSmallThreads) {
    reinterpret_cast<uint4*>(xh)[i] = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(xl)[i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kSmallWarps; ++w) {
      sq.x += squares[w].x;
      sq.y += squares[w].y;
      sq.z += squares[w].z;
    }
    squares[kSmallWarps] = sq;
  }
  __syncthreads();
  if (p.cluster > 1) cluster_sync();
  if (warp == 0) {
    const uint32_t mine = smem_u32(squares + kSmallWarps);
    double t = 0.0;
    if (lane < p.cluster)
      t = whole_square(ld_remote4(p.cluster > 1 ? mapa_shared(mine, lane) : mine));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) norm_factors(t, factors[0], factors[1]);
  }
  __syncthreads();

  // ------------------------------------------------------------ X in two parts
  {
    const float s1 = factors[0], s2 = factors[1] * kXScale;
    for (int i = tid; i < runs * quads; i += kSmallThreads) {
      const int r = i / quads, o = (i - r * quads) * 4;
      const int64_t at = start + r * pitch + o;
      const int n = min(4, run - o);
      float u[4];
      update4<false>(g + at, m == nullptr ? nullptr : m + at, n, vec, p.in.momentum,
                     p.in.nesterov, u);
      int row = r, col = o;
      if (p.tall) {
        col = o / p.n;
        row = o - col * p.n;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= n) break;
        const float x = (u[k] * s1) * s2;
        const __half h = __float2half_rn(x);
        const int to = swz(row, col, slab);
        xh[to] = h;
        xl[to] = __float2half_rn(x - __half2float(h));
        if (!p.tall) {
          ++col;
        } else if (++row == p.n) {
          row = 0;
          ++col;
        }
      }
    }
  }
  __syncthreads();

  const uint32_t xh_a = smem_u32(xh), e_a = smem_u32(e), d_a = smem_u32(d);
  const int nb = np / 32, blocks = nb * nb;
  const int g8 = lane >> 2, t2 = (lane & 3) * 2;  // a fragment's row and columns
  float keep = 0.0f, rate = 0.0f;
  if (p.w != nullptr) {
    const float lr = __ldg(p.lr);
    keep = 1.0f - lr * p.decay;
    rate = lr * p.scale * kXInv;
  }
  for (int step = 0; step < p.steps; ++step) {
    // ---------------------------------------------------------- 1: this slab's X X^T
    if (warp < blocks * sh.splits) {
      const int block = warp % blocks, split = warp / blocks;
      const int i0 = block / nb * 32, j0 = block % nb * 32;
      const int chunks = slab / 16;
      float acc[2][4][4];
      block_product(acc, xh_a, slab, i0, j0, chunks * split / sh.splits * 16,
                    chunks * (split + 1) / sh.splits * 16, lane);
      float* to = part + split * np * np;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(to + (i0 + 16 * i + g8 + 8 * h) * np + j0 + 8 * j + t2) =
                make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
    }
    __syncthreads();
    if (sh.splits > 1) {
      for (int q = tid; q < np * np / 4; q += kSmallThreads) {
        float4 s = reinterpret_cast<float4*>(part)[q];
        for (int k = 1; k < sh.splits; ++k) {
          const float4 o = reinterpret_cast<float4*>(part)[k * (np * np / 4) + q];
          s.x += o.x;
          s.y += o.y;
          s.z += o.z;
          s.w += o.w;
        }
        reinterpret_cast<float4*>(part)[q] = s;
      }
      __syncthreads();
    }
    // ---------------------------------------------------------- 2: the sum over CTAs
    if (p.cluster > 1) cluster_sync();  // all partial sums are there, and nobody reads E or d
    {
      const int pieces = np * np / 4;
      const int per = (pieces + p.cluster - 1) / p.cluster;
      const uint32_t part_a = smem_u32(part), diag_a = smem_u32(diag);
      for (int q = rank * per + tid; q < min(pieces, (rank + 1) * per); q += kSmallThreads) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < p.cluster; ++r) {
          const float4 o =
              ld_remote4(p.cluster > 1 ? mapa_shared(part_a + 16 * q, r) : part_a + 16 * q);
          s.x += o.x;
          s.y += o.y;
          s.z += o.z;
          s.w += o.w;
        }
        const int row = 4 * q / np, col = 4 * q - row * np;
        float v[4] = {s.x * kXInv, s.y * kXInv, s.z * kXInv, s.w * kXInv};  // A times 2^12
        float on = 0.0f;
        const bool has = row >= col && row < col + 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (row == col + k) {
            on = v[k] * kXInv;
            v[k] = 0.0f;
          }
        const uint2 word = make_uint2(half2_bits(v[0], v[1]), half2_bits(v[2], v[3]));
        const uint32_t to = e_a + 2 * swz(row, col, ns);
        for (int r = 0; r < p.cluster; ++r) {
          st_remote8(p.cluster > 1 ? mapa_shared(to, r) : to, word);
          if (has) st_remote4(p.cluster > 1 ? mapa_shared(diag_a + 4 * row, r) : diag_a + 4 * row, on);
        }
      }
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    // ---------------------------------------------------------- 3: D and beta
    if (warp < blocks) {
      const int i0 = warp / nb * 32, j0 = warp % nb * 32;
      float acc[2][4][4];
      block_product(acc, e_a, ns, i0, j0, 0, np, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = i0 + 16 * i + g8 + 8 * h;
          const float dm = diag[row];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int col = j0 + 8 * j + t2;
            const int at = swz(row, col, ns);
            const float2 e2 = __half22float2(*reinterpret_cast<const __half2*>(e + at));
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float ee = acc[i][j][2 * h + k];
              const float lin = fmaf(p.c, dm + diag[col + k], p.b) * (kXInv * kDScale);
              v[k] = fmaf(lin, k == 0 ? e2.x : e2.y, (p.c * (kEEInv * kDScale)) * ee);
              if (row == col + k) {
                v[k] = 0.0f;
                beta[row] = p.a + dm * fmaf(p.c, dm, p.b) + p.c * (ee * kEEInv);
              }
            }
            *reinterpret_cast<uint32_t*>(d + at) = half2_bits(v[0], v[1]);
          }
        }
    }
    __syncthreads();
    // ---------------------------------------------------------- 4: X <- beta X + D X
    const bool last = step == p.steps - 1;
    const int ksteps = np / 16;
    for (int c0 = warp * 16; c0 < width; c0 += kSmallWarps * 16) {
      uint32_t x[kSmallMaxN / 16][4];  // all rows of 16 columns, as the second operand
#pragma unroll
      for (int k = 0; k < kSmallMaxN / 16; ++k)
        if (k < ksteps)
          ldm4_t(xh_a + 2 * swz(16 * k + (lane & 15), c0 + (lane >> 4) * 8, slab), x[k]);
      __syncwarp();
      for (int r0 = 0; r0 < np; r0 += 16) {
        float acc[2][4] = {};
#pragma unroll
        for (int k = 0; k < kSmallMaxN / 16; ++k)
          if (k < ksteps) {
            uint32_t a[4];
            ldm4(d_a + 2 * swz(r0 + (lane & 15), 16 * k + (lane >> 4) * 8, ns), a);
            mma_f16(acc[0], a, x[k][0], x[k][1]);
            mma_f16(acc[1], a, x[k][2], x[k][3]);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = r0 + g8 + 8 * h;
          const float bm = beta[row];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = c0 + 8 * j + t2;
            const int at = swz(row, col, slab);
            const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(xh + at));
            float v[2] = {hi.x, hi.y};
            if (!last) {
              const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(xl + at));
              v[0] += lo.x;
              v[1] += lo.y;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
              v[k] = fmaf(bm, v[k], acc[j][2 * h + k] * (1.0f / kDScale));
            if (!last) {
              const uint32_t hb = half2_bits(v[0], v[1]);
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hb));
              *reinterpret_cast<uint32_t*>(xh + at) = hb;
              *reinterpret_cast<uint32_t*>(xl + at) = half2_bits(v[0] - back.x, v[1] - back.y);
            } else if (row < p.n) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if (col + k >= width) break;
                const int64_t o = matrix * elems + (p.tall ? (l0 + col + k) * p.n + row
                                                           : row * p.in.cols + l0 + col + k);
                if (p.w == nullptr) {
                  p.out[o] = __float2bfloat16_rn(v[k] * kXInv);
                } else {
                  const float w = fmaf(-rate, v[k], keep * p.w[o]);
                  p.w[o] = w;
                  if (p.wb != nullptr) p.wb[o] = __float2bfloat16_rn(w);
                }
              }
            }
          }
        }
      }
    }
    __syncthreads();
  }
  if (p.cluster > 1) cluster_sync();  // nobody reads this CTA's shared memory any more
}

// CTAs of a cluster for one matrix, or 0 where the matrix does not fit: the fewest that hold it,
// more while there are SMs for them and at least 64 columns for each.
int muon_small_cluster(int n, int64_t length, int64_t batch, int num_sms) {
  if (n > kSmallMaxN) return 0;
  int c = 1;
  while (c <= kSmallMaxCluster && small_shape(n, length, c).bytes() > kSmallMaxSmem) c *= 2;
  if (c > kSmallMaxCluster) return 0;
  while (2 * c <= kSmallMaxCluster && batch * 2 * c <= num_sms && length > 64 * c) c *= 2;
  return c;
}

template <typename T>
static cudaError_t small_attrs() {
  cudaError_t e = cudaFuncSetAttribute(muon_small_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmallMaxSmem));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(muon_small_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                             1);
  return e;
}

static void small_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int64_t batch,
                         int cluster, size_t smem, cudaStream_t s) {
  cfg.gridDim = dim3(static_cast<unsigned>(batch * cluster), 1, 1);
  cfg.blockDim = dim3(kSmallThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

cudaError_t muon_small_set_attrs(int n, int64_t length, int cluster, bool* fits) {
  *fits = false;
  cudaError_t e = small_attrs<float>();
  if (e == cudaSuccess) e = small_attrs<__nv_bfloat16>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  small_config(cfg, attr, 1, cluster, small_shape(n, length, cluster).bytes(), nullptr);
  int clusters = 0;
  e = cudaOccupancyMaxActiveClusters(&clusters, muon_small_kernel<float>, &cfg);
  *fits = e == cudaSuccess && clusters > 0;
  return e;
}

cudaError_t launch_muon_small(const MuonInput& in, const OrthoParams& o, int steps, int cluster,
                              cudaStream_t s) {
  SmallParams p{};
  p.in = in;
  p.tall = in.rows > in.cols ? 1 : 0;
  p.n = static_cast<int>(std::min(in.rows, in.cols));
  p.length = std::max(in.rows, in.cols);
  p.shape = small_shape(p.n, p.length, cluster);
  p.cluster = cluster;
  p.steps = steps;
  p.a = o.a;
  p.b = o.b;
  p.c = o.c;
  p.out = o.out;
  p.w = o.w;
  p.wb = o.wb;
  p.lr = o.lr;
  p.decay = o.decay;
  p.scale = o.scale;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  small_config(cfg, attr, in.batch, cluster, p.shape.bytes(), s);
  return in.g_f32 ? cudaLaunchKernelEx(&cfg, muon_small_kernel<float>, p)
                  : cudaLaunchKernelEx(&cfg, muon_small_kernel<__nv_bfloat16>, p);
}

}  // namespace mlpb
