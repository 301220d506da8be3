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

// A block of S S^T, 16 I x 8 J elements at rows i0 and j0, over columns [k0, k1) of a swizzled
// matrix.  Rows of fragments begin at multiples of 8, so that a lane's swizzle is its own.
template <int I, int J>
__device__ __forceinline__ void block_product(float (&acc)[I][J][4], uint32_t s, int stride, int i0,
                                              int j0, int k0, int k1, int lane) {
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
  const uint32_t a0 = s + 2 * (i0 + (lane & 15)) * stride;  // rows, then columns 8 on
  const uint32_t b0 = s + 2 * (j0 + (lane & 7) + ((lane >> 4) << 3)) * stride;  // the other way
  const int ap = lane >> 4, bp = (lane >> 3) & 1, x = lane & 7;
#pragma unroll 2
  for (int k = k0; k < k1; k += 16) {
    uint32_t a[I][4], b[J / 2][4];
    const uint32_t ao = (((k >> 3) + ap) ^ x) << 4, bo = (((k >> 3) + bp) ^ x) << 4;
#pragma unroll
    for (int i = 0; i < I; ++i) ldm4(a0 + 32 * i * stride + ao, a[i]);
#pragma unroll
    for (int j = 0; j < J / 2; ++j) ldm4(b0 + 32 * j * stride + bo, b[j]);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
        mma_f16(acc[i][j], a[i], b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
  }
}

// D (into d) and beta of the block at (i0, j0) of E.
template <int I, int J>
__device__ __forceinline__ void poly_block(const __half* e, __half* d, const float* diag,
                                           float* beta, int np, int ns, int i0, int j0, int lane,
                                           float pa, float pb, float pc) {
  float acc[I][J][4];
  block_product<I, J>(acc, smem_u32(e), ns, i0, j0, 0, np, lane);
  const int g8 = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int col = j0 + 8 * j + t2;
    const int at0 = (((col >> 3) ^ g8) << 3) + t2;
    const float d0 = diag[col], d1 = diag[col + 1];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = i0 + 16 * i + 8 * h + g8;
        const int at = row * ns + at0;
        const float dm = diag[row];
        const float2 e2 = __half22float2(*reinterpret_cast<const __half2*>(e + at));
        const float ee0 = acc[i][j][2 * h], ee1 = acc[i][j][2 * h + 1];
        float v0 = fmaf(fmaf(pc, dm + d0, pb) * (kXInv * kDScale), e2.x,
                        (pc * (kEEInv * kDScale)) * ee0);
        float v1 = fmaf(fmaf(pc, dm + d1, pb) * (kXInv * kDScale), e2.y,
                        (pc * (kEEInv * kDScale)) * ee1);
        if (row == col || row == col + 1) {
          const float ee = row == col ? ee0 : ee1;
          beta[row] = pa + dm * fmaf(pc, dm, pb) + pc * (ee * kEEInv);
          if (row == col) v0 = 0.0f;
          else v1 = 0.0f;
        }
        *reinterpret_cast<uint32_t*>(d + at) = half2_bits(v0, v1);
      }
  }
}

// This CTA's elements of a matrix, in runs of consecutive ones.
struct SmallRuns {
  int runs, run, quads;  // quads: groups of four of a run, the last one shorter
  int64_t start, pitch;
  bool vec;  // whole groups on 16 bytes
};

// Calls f(address, elements, row, column) for groups of four elements: four addresses a thread
// before their first use, so that the loads of four groups are in flight together.
template <int kBatch, typename Load, typename Use>
__device__ __forceinline__ void for_groups(const SmallRuns& r, int tall, int n, Load load, Use use) {
  const int total = r.runs * r.quads;
  for (int i0 = threadIdx.x; i0 < total; i0 += kBatch * kSmallThreads) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kSmallThreads;
      if (i < total) {
        const int row = tall ? 0 : i / r.quads;
        const int o = (i - row * r.quads) * 4;
        load(k, r.start + row * r.pitch + o, min(4, r.run - o));
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kSmallThreads;
      if (i < total) {
        int row = tall ? 0 : i / r.quads;
        const int o = (i - row * r.quads) * 4;
        int col = o;
        if (tall) {
          col = o / n;
          row = o - col * n;
        }
        use(k, r.start + (tall ? 0 : row * r.pitch) + o, min(4, r.run - o), row, col);
      }
    }
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
  SmallRuns runs;
  runs.runs = p.tall ? 1 : p.n;
  runs.run = p.tall ? width * p.n : width;
  runs.start = p.tall ? l0 * p.n : l0;
  runs.pitch = p.in.cols;
  runs.quads = (runs.run + 3) / 4;
  runs.vec = p.in.cols % 4 == 0;  // rows, slabs and matrices then begin on 16 bytes

  // ------------------------------------------------------------ momentum and norm
  float4 sq = make_float4(0.f, 0.f, 0.f, 0.f);
  {
    float u[4][4];
    for_groups<4>(
        runs, p.tall, p.n,
        [&](int k, int64_t at, int n) {
          update4<true>(g + at, m == nullptr ? nullptr : m + at, n, runs.vec, p.in.momentum,
                        p.in.nesterov, u[k]);
        },
        [&](int k, int64_t, int, int, int) { add_squares4(u[k], sq); });
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sq.x += __shfl_xor_sync(0xffffffffu, sq.x, o);
    sq.y += __shfl_xor_sync(0xffffffffu, sq.y, o);
    sq.z += __shfl_xor_sync(0xffffffffu, sq.z, o);
  }
  if (lane == 0) squares[warp] = sq;
  if (p.n < np || width < slab) {  // zeros where no element of the matrix lies
    for (int i = tid; i < np * slab / 8; i += kSmallThreads) {
      reinterpret_cast<uint4*>(xh)[i] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(xl)[i] = make_uint4(0, 0, 0, 0);
    }
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
    float u[4][4];
    for_groups<4>(
        runs, p.tall, p.n,
        [&](int k, int64_t at, int n) {
          update4<false>(g + at, m == nullptr ? nullptr : m + at, n, runs.vec, p.in.momentum,
                         p.in.nesterov, u[k]);
        },
        [&](int k, int64_t, int n, int row, int col) {
          float x[4], lo[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            x[c] = (u[k][c] * s1) * s2;
            lo[c] = x[c] - __half2float(__float2half_rn(x[c]));
          }
          if (!p.tall) {  // four columns of a row, in one piece; those past the end are zeros
            const int to = swz(row, col, slab);
            *reinterpret_cast<uint2*>(xh + to) =
                make_uint2(half2_bits(x[0], x[1]), half2_bits(x[2], x[3]));
            *reinterpret_cast<uint2*>(xl + to) =
                make_uint2(half2_bits(lo[0], lo[1]), half2_bits(lo[2], lo[3]));
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c >= n) break;
              const int to = swz(row, col, slab);
              xh[to] = __float2half_rn(x[c]);
              xl[to] = __float2half_rn(lo[c]);
              if (++row == p.n) {
                row = 0;
                ++col;
              }
            }
          }
        });
  }
  __syncthreads();

  const uint32_t xh_a = smem_u32(xh), e_a = smem_u32(e), d_a = smem_u32(d);
  const int nb = np / 32, blocks = nb * nb;
  const int pieces = np * np / 4;  // fragments of four: rows g8 and g8 + 8, two columns of each
  // Lanes that share a fragment in the sum over CTAs, as many as there are threads for.
  const int per = (pieces + p.cluster - 1) / p.cluster;
  int share = 1;
  while (2 * share <= p.cluster && 2 * share * per <= kSmallThreads) share *= 2;
  const int g8 = lane >> 2, t2 = (lane & 3) * 2;  // a fragment's row and columns
  float keep = 0.0f, rate = 0.0f;
  if (p.w != nullptr) {
    const float lr = __ldg(p.lr);
    keep = 1.0f - lr * p.decay;
    rate = lr * p.scale;
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
      float4* to = reinterpret_cast<float4*>(part) + split * pieces + block * 256 + lane;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          to[(i * 4 + j) * 32] =
              make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
    }
    __syncthreads();
    if (sh.splits > 1) {
      for (int q = tid; q < pieces; q += kSmallThreads) {
        float4 s = reinterpret_cast<float4*>(part)[q];
#pragma unroll 4
        for (int k = 1; k < sh.splits; ++k) {
          const float4 o = reinterpret_cast<float4*>(part)[k * pieces + q];
          s.x += o.x;
          s.y += o.y;
          s.z += o.z;
          s.w += o.w;
        }
        reinterpret_cast<float4*>(part)[q] = s;
      }
      if (p.cluster == 1) __syncthreads();
    }
    // ---------------------------------------------------------- 2: the sum over CTAs
    if (p.cluster > 1) cluster_sync();  // all partial sums are there, and nobody reads E or d
    {
      const uint32_t part_a = smem_u32(part), diag_a = smem_u32(diag);
      const int of = tid & (share - 1);
      // every lane of a group takes as many rounds: the exchange below needs them all
      for (int q0 = 0; q0 < per; q0 += kSmallThreads / share) {
        const int mine = q0 + tid / share, q = rank * per + mine;
        const bool on = mine < per && q < pieces;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
#pragma unroll 4
          for (int r = of; r < p.cluster; r += share) {
            const float4 o =
                ld_remote4(p.cluster > 1 ? mapa_shared(part_a + 16 * q, r) : part_a + 16 * q);
            s.x += o.x;
            s.y += o.y;
            s.z += o.z;
            s.w += o.w;
          }
        }
        for (int o = 1; o < share; o *= 2) {
          s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
          s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
          s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
          s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
        }
        if (on) {
          const int block = q >> 8, frag = (q >> 5) & 7, l = q & 31;
          const int row = block / nb * 32 + 16 * (frag >> 2) + (l >> 2);
          const int col = block % nb * 32 + 8 * (frag & 3) + (l & 3) * 2;
          float v[4] = {s.x * kXInv, s.y * kXInv, s.z * kXInv, s.w * kXInv};  // A times 2^12
          float dia[2] = {0.f, 0.f};
          bool has[2] = {false, false};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (row + 8 * (k >> 1) == col + (k & 1)) {
              has[k >> 1] = true;
              dia[k >> 1] = v[k] * kXInv;
              v[k] = 0.0f;
            }
          const uint32_t w0 = half2_bits(v[0], v[1]), w1 = half2_bits(v[2], v[3]);
          const uint32_t to = e_a + 2 * swz(row, col, ns), at = diag_a + 4 * row;
          for (int r = of; r < p.cluster; r += share) {
            const uint32_t t = p.cluster > 1 ? mapa_shared(to, r) : to;
            const uint32_t z = p.cluster > 1 ? mapa_shared(at, r) : at;
            st_remote4(t, __uint_as_float(w0));
            st_remote4(t + 16 * ns, __uint_as_float(w1));  // eight rows on: the same swizzle
            if (has[0]) st_remote4(z, dia[0]);
            if (has[1]) st_remote4(z + 32, dia[1]);
          }
        }
      }
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    // ---------------------------------------------------------- 3: D and beta
    if (np <= 64) {  // blocks of 16 x 16: more warps than 32 x 32 have
      const int n16 = np / 16;
      if (warp < n16 * n16)
        poly_block<1, 2>(e, d, diag, beta, np, ns, warp / n16 * 16, warp % n16 * 16, lane, p.a, p.b,
                         p.c);
    } else if (warp < blocks) {
      poly_block<2, 4>(e, d, diag, beta, np, ns, warp / nb * 32, warp % nb * 32, lane, p.a, p.b,
                       p.c);
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
      const int x8 = lane & 7;
      const uint32_t da = d_a + 2 * (lane & 15) * ns;
      // of the fragment's pairs of columns: the row's and the swizzle's part
      const int p0 = g8 * slab + (((c0 >> 3) ^ g8) << 3) + t2;
      const int p1 = g8 * slab + ((((c0 >> 3) + 1) ^ g8) << 3) + t2;
      for (int r0 = 0; r0 < np; r0 += 16) {
        float acc[2][4] = {};
#pragma unroll
        for (int k = 0; k < kSmallMaxN / 16; ++k)
          if (k < ksteps) {
            uint32_t a[4];
            ldm4(da + 2 * r0 * ns + (((2 * k + (lane >> 4)) ^ x8) << 4), a);
            mma_f16(acc[0], a, x[k][0], x[k][1]);
            mma_f16(acc[1], a, x[k][2], x[k][3]);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float bm = beta[r0 + 8 * h + g8];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int at = (r0 + 8 * h) * slab + (j == 0 ? p0 : p1);
            const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(xh + at));
            float v0 = hi.x, v1 = hi.y;
            if (!last) {
              const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(xl + at));
              v0 += lo.x;
              v1 += lo.y;
            }
            v0 = fmaf(bm, v0, acc[j][2 * h] * (1.0f / kDScale));
            v1 = fmaf(bm, v1, acc[j][2 * h + 1] * (1.0f / kDScale));
            if (!last) {
              const uint32_t hb = half2_bits(v0, v1);
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hb));
              *reinterpret_cast<uint32_t*>(xh + at) = hb;
              *reinterpret_cast<uint32_t*>(xl + at) = half2_bits(v0 - back.x, v1 - back.y);
            } else {  // fp32, its two halves in the places of the parts
              const uint32_t b0 = __float_as_uint(v0 * kXInv), b1 = __float_as_uint(v1 * kXInv);
              *reinterpret_cast<uint32_t*>(xh + at) = __byte_perm(b0, b1, 0x7632);
              *reinterpret_cast<uint32_t*>(xl + at) = __byte_perm(b0, b1, 0x5410);
            }
          }
        }
      }
    }
    __syncthreads();
  }
  // ------------------------------------------------------------ the result
  {
    float4 w4[4];
    const int64_t base = matrix * elems;
    for_groups<4>(
        runs, p.tall, p.n,
        [&](int k, int64_t at, int) {
          if (p.w != nullptr && runs.vec) w4[k] = *reinterpret_cast<const float4*>(p.w + base + at);
        },
        [&](int k, int64_t at, int n, int row, int col) {
          float v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int from = swz(row, col, slab);
            v[c] = __uint_as_float(
                (static_cast<uint32_t>(__half_as_ushort(xh[from])) << 16) |
                static_cast<uint32_t>(__half_as_ushort(xl[from])));
            if (c + 1 < n) {
              if (!p.tall) {
                ++col;
              } else if (++row == p.n) {
                row = 0;
                ++col;
              }
            }
          }
          const int64_t o = base + at;
          if (runs.vec) {
            if (p.w != nullptr) {
              const float w[4] = {w4[k].x, w4[k].y, w4[k].z, w4[k].w};
#pragma unroll
              for (int c = 0; c < 4; ++c) v[c] = fmaf(-rate, v[c], keep * w[c]);
              *reinterpret_cast<float4*>(p.w + o) = make_float4(v[0], v[1], v[2], v[3]);
            }
            __nv_bfloat16* half = p.w != nullptr ? p.wb : p.out;
            if (half != nullptr)
              *reinterpret_cast<uint2*>(half + o) =
                  make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c >= n) break;
              if (p.w == nullptr) {
                p.out[o + c] = __float2bfloat16_rn(v[c]);
              } else {
                const float w = fmaf(-rate, v[c], keep * p.w[o + c]);
                p.w[o + c] = w;
                if (p.wb != nullptr) p.wb[o + c] = __float2bfloat16_rn(w);
              }
            }
          }
        });
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
