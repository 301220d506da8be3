// The whole orthogonalised update of matrices whose smaller side is at most 128, in one launch: a
// matrix lies in the shared memory of a cluster of CTAs from the first step to the last.
//
// With n <= 128 a product is a few million operations on one tile, and the launches, pipeline
// starts and trips through L2 of fifteen tensor-core launches cost far more than the products
// (64 x 4096: 194 us).  Each CTA keeps a slab of the longer side, X [n][slab] in two fp16 parts
// (muon.cuh has the number formats); a tall matrix is transposed as it is read and written, since
// the polynomial of X^T is that of X transposed.  A step is
//   1. each CTA's share of X X^T over its slab;
//   2. the sum over CTAs: each CTA adds one slice through distributed shared memory, in an order
//      that is the same every run (lanes share a sum), and writes E and d to all;
//   3. E E, D and beta, by every CTA for itself;
//   4. X <- beta X + D X in place, 512 columns at a time (muon.cuh has what X's parts go with).
// Two barriers of the cluster a step.  The products are single tcgen05 chains of M = 128 (rows past
// n are of whatever lies behind and are not read back) that a thread issues between barriers of the
// CTA: with mma.sync, a sixteenth of the rate here, they were two thirds of the time at n = 128
// (128 x 4096: 102 us).  X, E and D lie in chunks of 64 columns, rows of 128 bytes, swizzled: the
// K-major operand of 1, 3 and 4 (D) and, the same bytes, the MN-major one of 4 (X).
//
// 64 x 4096 42 us, 128 x 4096 70 us, 16 x 64 19 us in a graph: 3 to 12 us a step, the latency of
// three chains, two barriers of the cluster and the trips between shared and tensor memory; bytes
// (0.2 us) and operations (0.1 us) are no bound.
#include <algorithm>

#include "muon_update.cuh"
#include "pointwise.cuh"
#include "ptx.cuh"

namespace mlpb {

constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallMaxN = 128;
constexpr int kSmallMaxCluster = 16;
constexpr size_t kSmallMaxSmem = 232448;
// More than half an SM's shared memory, and more than gemm_b128_few.cu leaves: no other CTA that
// takes tensor memory is on the same SM.  (Two clusters that meet on two SMs could each hold there
// what the other's second CTA waits for.)
constexpr size_t kSmallMinSmem = 122880;
constexpr int kSmallTmem = 512;
constexpr int kSmallBlock = 256;  // columns of a chain of step 4; two in tensor memory

struct SmallShape {
  int np;    // n rounded up to 32
  int slab;  // columns of X in a CTA, a multiple of 64
  __host__ __device__ size_t x_bytes() const { return static_cast<size_t>(np) * slab * 2; }
  __host__ __device__ size_t e_bytes() const {
    return static_cast<size_t>(np) * ((np + 63) / 64) * 128;
  }
  // the partial sums, later D
  __host__ __device__ size_t p_bytes() const {
    const size_t sums = static_cast<size_t>(np) * np * 4;
    return sums > e_bytes() ? sums : e_bytes();
  }
  __host__ __device__ size_t used() const { return 2 * x_bytes() + e_bytes() + p_bytes(); }
  // A chain reads 128 rows of its chunk, whatever np is: what lies behind the last is there too.
  __host__ __device__ size_t bytes() const {
    const size_t b = used() + static_cast<size_t>(128 - np) * 128 + 2 * kSmallMaxN * 4 + 512 + 1024;
    return b > kSmallMinSmem ? b : kSmallMinSmem;
  }
};

static SmallShape small_shape(int n, int64_t length, int cluster) {
  SmallShape s;
  s.np = (n + 31) / 32 * 32;
  s.slab = static_cast<int>((length + cluster * 64 - 1) / (cluster * 64)) * 64;
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
  uint32_t* err;
  uint64_t wait_ns;
};

// Element (row, col) of a matrix in chunks of 64 columns: within a row's 128 bytes 16-byte pieces
// trade places by the row modulo 8.
__device__ __forceinline__ int swz(int row, int col, int np) {
  return ((col >> 6) * np + row) * 64 + ((((col >> 3) & 7) ^ (row & 7)) << 3) + (col & 7);
}

__device__ __forceinline__ void umma_f16_one(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
  tmem_ld_wait();
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r[e]);
}

// S S^T over `depth` columns of a matrix in chunks: 128 rows by np.
__device__ __forceinline__ void chain_square(uint32_t d, uint32_t s, int np, int depth) {
  const uint32_t idesc = idesc_bf16_f32(128, np, false, false) & ~((1u << 7) | (1u << 10));
  const uint64_t desc = sdesc(s, 16, 1024, 2u);
  for (int k = 0; k < depth; k += 16) {
    const uint64_t at = desc + static_cast<uint32_t>(((k >> 6) * np * 128 + (k & 63) * 2) >> 4);
    umma_f16_one(d, at, at, idesc, k > 0 ? 1u : 0u);
  }
}

// D X for `cols` columns (at most 256) of X from column c on: 128 rows.
__device__ __forceinline__ void chain_apply(uint32_t d, uint32_t dm, uint32_t x, int np, int c,
                                            int cols) {
  const uint32_t idesc = idesc_bf16_f32(128, cols, false, true) & ~((1u << 7) | (1u << 10));
  const uint64_t adesc = sdesc(dm, 16, 1024, 2u);
  const uint64_t bdesc =
      sdesc(x + (c >> 6) * np * 128, static_cast<uint32_t>(np) * 128, 1024, 2u);
  for (int k = 0; k < np; k += 16)
    umma_f16_one(d,
                 adesc + static_cast<uint32_t>(((k >> 6) * np * 128 + (k & 63) * 2) >> 4),
                 bdesc + static_cast<uint32_t>((k * 128) >> 4), idesc, k > 0 ? 1u : 0u);
}

__device__ __forceinline__ void st_remote16(uint32_t cluster_addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ void st_remote4(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// i / d for i, d below 2^16, by the reciprocal ceil(2^32 / d) (d > 1).
struct Divisor {
  uint32_t d, m;
  __device__ __forceinline__ explicit Divisor(int by)
      : d(static_cast<uint32_t>(by)),
        m(by > 1 ? 0xffffffffu / static_cast<uint32_t>(by) + 1u : 0u) {}
  __device__ __forceinline__ int div(int i) const {
    return d > 1u ? static_cast<int>(__umulhi(static_cast<uint32_t>(i), m)) : i;
  }
};

// This CTA's elements of a matrix, in runs of consecutive ones.
struct SmallRuns {
  int runs, run, quads;  // quads: groups of four of a run, the last one shorter
  int64_t start, pitch;
  bool vec;  // whole groups on 16 bytes
};

constexpr int kSmallBatch = 8;  // groups of a thread whose loads are in flight together

// Calls load(k, address, elements) for a thread's groups of four elements, a batch at a time, then
// use(k, address, elements, row, column).
template <typename Load, typename Use>
__device__ __forceinline__ void for_groups(const SmallRuns& r, int tall, int n, Load load,
                                           Use use) {
  const int total = r.runs * r.quads;
  const Divisor by(tall ? n : r.quads);
  for (int i0 = threadIdx.x; i0 < total; i0 += kSmallBatch * kSmallThreads) {
#pragma unroll
    for (int k = 0; k < kSmallBatch; ++k) {
      const int i = i0 + k * kSmallThreads;
      if (i < total) {
        const int row = tall ? 0 : by.div(i);
        const int o = (i - row * r.quads) * 4;
        load(k, r.start + row * r.pitch + o, min(4, r.run - o));
      }
    }
#pragma unroll
    for (int k = 0; k < kSmallBatch; ++k) {
      const int i = i0 + k * kSmallThreads;
      if (i < total) {
        int row = tall ? 0 : by.div(i);
        const int o = (i - row * r.quads) * 4;
        const int64_t at = r.start + (tall ? 0 : row * r.pitch) + o;
        int col = o;
        if (tall) {
          col = by.div(o);
          row = o - col * n;
        }
        use(k, at, min(4, r.run - o), row, col);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kSmallThreads, 1) muon_small_kernel(const SmallParams p) {
  extern __shared__ __align__(1024) uint8_t small_raw[];
  const SmallShape sh = p.shape;
  const int np = sh.np, slab = sh.slab;
  uint8_t* smem = small_raw + ((1024u - (smem_u32(small_raw) & 1023u)) & 1023u);
  __half* xh = reinterpret_cast<__half*>(smem);
  __half* xl = reinterpret_cast<__half*>(smem + sh.x_bytes());
  __half* e = reinterpret_cast<__half*>(smem + 2 * sh.x_bytes());
  float* part = reinterpret_cast<float*>(smem + 2 * sh.x_bytes() + sh.e_bytes());
  __half* d = reinterpret_cast<__half*>(part);  // once the partial sums have been read
  float* diag = reinterpret_cast<float*>(smem + sh.used() + static_cast<size_t>(128 - np) * 128);
  float* beta = diag + kSmallMaxN;
  float4* squares = reinterpret_cast<float4*>(beta + kSmallMaxN);  // a warp each, then the CTA's
  float* factors = reinterpret_cast<float*>(squares + kSmallWarps + 1);
  uint64_t* bar_mem = reinterpret_cast<uint64_t*>(factors + 2);
  uint32_t* words = reinterpret_cast<uint32_t*>(bar_mem + 1);  // tensor memory, abort flag

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

  if (tid == 0) {
    mbar_init(smem_u32(bar_mem), 1);
    words[1] = 0u;
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc_one(smem_u32(words), kSmallTmem);

  // ------------------------------------------------------------ momentum and norm
  float4 sq = make_float4(0.f, 0.f, 0.f, 0.f);
  float u[kSmallBatch][4];  // of a thread that has one batch: the second pass uses them again
  const bool kept = runs.runs * runs.quads <= kSmallBatch * kSmallThreads;
  float v[kSmallBatch][4];  // M: all loads of a batch come before its first store
  for_groups(
      runs, p.tall, p.n,
      [&](int k, int64_t at, int n) {
        load4(g + at, m == nullptr ? nullptr : m + at, n, runs.vec, false, u[k], v[k]);
      },
      [&](int k, int64_t at, int n, int, int) {
        finish4<true, T>(m == nullptr ? nullptr : m + at, n, runs.vec, p.in.momentum,
                         p.in.nesterov, u[k], v[k]);
        add_squares4(u[k], sq);
      });
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
      t = whole_square(ld_cluster4(p.cluster > 1 ? mapa_shared(mine, lane) : mine));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) norm_factors(t, factors[0], factors[1]);
  }
  __syncthreads();

  // ------------------------------------------------------------ X in two parts
  {
    const float s1 = factors[0], s2 = factors[1] * kXScale;
    for_groups(
        runs, p.tall, p.n,
        [&](int k, int64_t at, int n) {
          if (!kept)
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
            const int to = swz(row, col, np);
            *reinterpret_cast<uint2*>(xh + to) =
                make_uint2(half2_bits(x[0], x[1]), half2_bits(x[2], x[3]));
            *reinterpret_cast<uint2*>(xl + to) =
                make_uint2(half2_bits(lo[0], lo[1]), half2_bits(lo[2], lo[3]));
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c >= n) break;
              const int to = swz(row, col, np);
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

  tc_fence_after();
  const uint32_t tmem = words[0];
  const uint32_t xh_a = smem_u32(xh), e_a = smem_u32(e), d_a = smem_u32(d);
  const uint32_t bar = smem_u32(bar_mem);
  const WaitCtx wc{words + 1, p.err, p.wait_ns};
  uint32_t parity = 0;
  // A chain between two barriers of the CTA: shared memory as written before it, tensor memory as
  // it leaves it.
  auto chain = [&](auto issue) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *wc.abort_flag == 0u) {  // no more products after an expired wait
      tc_fence_after();
      issue();
      umma_commit_one(bar);
    }
    wait_bounded(bar, parity, wc, kSiteMmaFull);
    parity ^= 1u;
    __syncwarp();
    tc_fence_after();
  };
  const int quarter = warp & 3, group = warp >> 2;  // a thread's row, its warp's share of columns
  const int row = quarter * 32 + lane;
  const uint32_t tacc = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const bool rows_here = quarter * 32 < np;
  // of step 4: parts of the columns, and the lane's part and row
  const int spread_log = np == 32 ? 2 : np == 64 ? 1 : 0, spread = 1 << spread_log;
  const int part_of = quarter * 32 / np, mrow = row - part_of * np;
  // The sum over CTAs: a CTA's rows, in pieces of four columns; lanes that share a piece, as many
  // as there are threads for.
  const int slice = np / p.cluster, per = slice * (np / 4);
  const Divisor by_row(np / 4);
  int share = 1;
  while (2 * share <= p.cluster && 2 * share * per <= kSmallThreads) share *= 2;
  float keep = 0.0f, rate = 0.0f;
  if (p.w != nullptr) {
    const float lr = __ldg(p.lr);
    keep = 1.0f - lr * p.decay;
    rate = lr * p.scale;
  }
  for (int step = 0; step < p.steps; ++step) {
    // ---------------------------------------------------------- 1: this slab's X X^T
    chain([&] { chain_square(tmem, xh_a, np, slab); });
    if (rows_here) {
      for (int c = group * (np / 4); c < (group + 1) * (np / 4); c += 8) {
        float v[8];
        tmem_ld_32x32b_x8(tacc + c, v);
        // rows of np sums, pieces of four in an order that no bank meets twice
        float4* to = reinterpret_cast<float4*>(part) + row * (np / 4);
        to[(c >> 2) ^ (row & 7)] = make_float4(v[0], v[1], v[2], v[3]);
        to[((c >> 2) + 1) ^ (row & 7)] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
    // ---------------------------------------------------------- 2: the sum over CTAs
    // all partial sums are there, and nobody reads E or d
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    {
      const uint32_t part_a = smem_u32(part), diag_a = smem_u32(diag);
      const int of = tid & (share - 1);
      // every lane of a group takes as many rounds: the exchange below needs them all
      for (int q0 = 0; q0 < per; q0 += kSmallThreads / share) {
        const int mine = q0 + tid / share, q = rank * per + mine;
        const bool on = mine < per;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
#pragma unroll 8
          for (int r = of; r < p.cluster; r += share) {
            const float4 o =
                ld_cluster4(p.cluster > 1 ? mapa_shared(part_a + 16 * q, r) : part_a + 16 * q);
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
        if (on && of == 0) {
          const int r0 = by_row.div(q), col = ((q - r0 * (np / 4)) ^ (r0 & 7)) * 4;
          float v[4] = {s.x * kXInv, s.y * kXInv, s.z * kXInv, s.w * kXInv};  // A times 2^12
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (r0 == col + k) {
              diag[r0] = v[k] * kXInv;
              v[k] = 0.0f;
            }
          *reinterpret_cast<uint2*>(e + swz(r0, col, np)) =
              make_uint2(half2_bits(v[0], v[1]), half2_bits(v[2], v[3]));
        }
      }
      if (p.cluster > 1) {  // this CTA's rows of E, 16 bytes a lane, and of d, to the others
        __syncthreads();
        const int chunks = (np + 63) / 64, pieces = slice * 8 * chunks;
        const Divisor by_piece(pieces), by_chunk(slice * 8);
        for (int i = tid; i < pieces * p.cluster; i += kSmallThreads) {
          const int to = by_piece.div(i), piece = i - to * pieces;
          const int chunk = by_chunk.div(piece);
          const uint32_t off = static_cast<uint32_t>((chunk * np + rank * slice) * 128 +
                                                     (piece - chunk * slice * 8) * 16);
          if (to != rank)
            st_remote16(mapa_shared(e_a + off, to),
                        *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(e) + off));
        }
        if (tid < slice * p.cluster) {
          const int to = tid / slice, r0 = rank * slice + tid % slice;
          if (to != rank) st_remote4(mapa_shared(diag_a + 4 * r0, to), diag[r0]);
        }
      }
    }
    if (p.cluster > 1) cluster_sync();
    // ---------------------------------------------------------- 3: D and beta
    chain([&] { chain_square(tmem, e_a, np, np); });
    if (rows_here) {
      const float dm = diag[row];
      for (int c = group * (np / 4); c < (group + 1) * (np / 4); c += 8) {
        float v[8];
        tmem_ld_32x32b_x8(tacc + c, v);
        const int at = swz(row, c, np);
        const uint4 w = *reinterpret_cast<const uint4*>(e + at);
        const uint32_t ew[4] = {w.x, w.y, w.z, w.w};
        const float4 d0 = *reinterpret_cast<const float4*>(diag + c);
        const float4 d1 = *reinterpret_cast<const float4*>(diag + c + 4);
        const float dj[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 e2 = __half22float2(*reinterpret_cast<const __half2*>(&ew[k >> 1]));
          const float ee = v[k];
          v[k] = fmaf(fmaf(p.c, dm + dj[k], p.b) * (kXInv * kDScale), k & 1 ? e2.y : e2.x,
                      (p.c * (kEEInv * kDScale)) * ee);
          if (c + k == row) {
            beta[row] = p.a + dm * fmaf(p.c, dm, p.b) + p.c * (ee * kEEInv);
            v[k] = 0.0f;
          }
        }
        *reinterpret_cast<uint4*>(d + at) =
            make_uint4(half2_bits(v[0], v[1]), half2_bits(v[2], v[3]), half2_bits(v[4], v[5]),
                       half2_bits(v[6], v[7]));
      }
    }
    // ---------------------------------------------------------- 4: X <- beta X + D X
    // A chain fills 128 lanes, D np of them: with np = 32 or 64 each part of the columns has a
    // chain of its own whose D lies np rows lower, so that all warps have lanes to take.
    const bool last = step == p.steps - 1;
    for (int c0 = 0; c0 < slab; c0 += 2 * kSmallBlock) {
      const int cols = min(2 * kSmallBlock, slab - c0), blocks = cols / 64;
      chain([&] {
        for (int j = 0; j < spread; ++j) {
          const int end = (blocks * (j + 1) >> spread_log) * 64;
          for (int c = (blocks * j >> spread_log) * 64; c < end; c += kSmallBlock)
            chain_apply(tmem + c, d_a - j * np * 128, xh_a, np, c0 + c, min(kSmallBlock, end - c));
        }
      });
      if (part_of < spread) {
        const uint64_t bm = f2_pack(beta[mrow], beta[mrow]);
        const uint64_t gm = step >= p.steps - 3 ? bm : f2_pack(p.a, p.a);  // of X's low part
        const uint64_t scale = f2_pack(1.0f / kDScale, 1.0f / kDScale);
        const int end = (blocks * (part_of + 1) >> spread_log) * 64;
        for (int c = (blocks * part_of >> spread_log) * 64 + group * 16; c < end; c += 64) {
          uint32_t acc[16];
          tmem_ld_32x32b_x16(tacc + c, acc);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int at = swz(mrow, c0 + c + 8 * j, np);
            const uint4 hw = *reinterpret_cast<const uint4*>(xh + at);
            const uint4 lw =
                last ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(xl + at);
            const uint32_t h[4] = {hw.x, hw.y, hw.z, hw.w}, l[4] = {lw.x, lw.y, lw.z, lw.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
              const float2 g2 = __half22float2(*reinterpret_cast<const __half2*>(&l[k]));
              const uint64_t a2 = f2_mul(f2_pack(__uint_as_float(acc[8 * j + 2 * k]),
                                                 __uint_as_float(acc[8 * j + 2 * k + 1])),
                                         scale);
              float v0, v1;
              f2_unpack(f2_fma(bm, f2_pack(f.x, f.y), f2_fma(gm, f2_pack(g2.x, g2.y), a2)), v0,
                        v1);
              if (!last) {
                hi[k] = half2_bits(v0, v1);
                const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi[k]));
                lo[k] = half2_bits(v0 - back.x, v1 - back.y);
              } else {  // fp32, its two halves in the places of the parts
                const uint32_t b0 = __float_as_uint(v0 * kXInv), b1 = __float_as_uint(v1 * kXInv);
                hi[k] = __byte_perm(b0, b1, 0x7632);
                lo[k] = __byte_perm(b0, b1, 0x5410);
              }
            }
            *reinterpret_cast<uint4*>(xh + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(xl + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // ------------------------------------------------------------ the result
  {
    float4 w4[kSmallBatch];
    const int64_t base = matrix * elems;
    for_groups(
        runs, p.tall, p.n,
        [&](int k, int64_t at, int n) {
          if (p.w == nullptr) return;
          const float* from = p.w + base + at;
          if (runs.vec)
            w4[k] = *reinterpret_cast<const float4*>(from);
          else
            w4[k] = make_float4(from[0], n > 1 ? from[1] : 0.0f, n > 2 ? from[2] : 0.0f,
                                n > 3 ? from[3] : 0.0f);
        },
        [&](int k, int64_t at, int n, int row, int col) {
          float v[4];
          if (!p.tall) {  // four columns of a row, in one piece
            const int from = swz(row, col, np);
            const uint2 hi = *reinterpret_cast<const uint2*>(xh + from);
            const uint2 lo = *reinterpret_cast<const uint2*>(xl + from);
            v[0] = __uint_as_float(__byte_perm(lo.x, hi.x, 0x5410));
            v[1] = __uint_as_float(__byte_perm(lo.x, hi.x, 0x7632));
            v[2] = __uint_as_float(__byte_perm(lo.y, hi.y, 0x5410));
            v[3] = __uint_as_float(__byte_perm(lo.y, hi.y, 0x7632));
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int from = swz(row, col, np);
              v[c] = __uint_as_float(
                  (static_cast<uint32_t>(__half_as_ushort(xh[from])) << 16) |
                  static_cast<uint32_t>(__half_as_ushort(xl[from])));
              if (c + 1 < n && ++row == p.n) {
                row = 0;
                ++col;
              }
            }
          }
          const int64_t o = base + at;
          if (p.w != nullptr) {
            const float w[4] = {w4[k].x, w4[k].y, w4[k].z, w4[k].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = fmaf(-rate, v[c], keep * w[c]);
          }
          if (runs.vec) {
            if (p.w != nullptr) {
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
                p.w[o + c] = v[c];
                if (p.wb != nullptr) p.wb[o + c] = __float2bfloat16_rn(v[c]);
              }
            }
          }
        });
  }
  if (warp == 0) {
    if (*wc.abort_flag != 0u) {  // the chain that a wait gave up on has long ended by then
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 20000ull) {
      }
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc_one(tmem, kSmallTmem);
  }
  if (p.cluster > 1) cluster_sync();  // nobody reads this CTA's shared memory any more
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

// Whether this kernel ends before the products of gemm_muon.cu would: us, fitted to both at 1 to
// 24 steps of 16 x 64 to 128 x 4096 and 24 x 8300, both ways round, 1 to 300 matrices (as a rule
// within 12 % of what they take).  A round of resident clusters takes 6.5 and 0.34 ns an element of
// a slab (0.85 if it has to be transposed) and each step 1.15 + 0.033 np and 0.14 ns an element;
// the other way takes 7.6 and 0.17 (0.2) ns for each element of the longer sides, and each step 12
// (19 past 64) and 0.32 (0.21).  This one against the other: 64 x 4096 18 / 23 us at one step,
// 43 / 81 at five; 32 of 4096 x 64 109 / 66 and 194 / 223; 16 of 128 x 2000 55 / 48 and 132 / 160;
// 64 of 4096 x 128 564 / 154 and 969 / 451.
static bool small_ends_first(const SmallShape& s, int64_t length, int64_t batch, int64_t resident,
                             bool tall, int steps) {
  const double rounds = static_cast<double>((batch + resident - 1) / resident);
  const double slab = static_cast<double>(s.np) * s.slab;
  const double sides = static_cast<double>(batch * length);
  const double here = rounds * (6.5 + (tall ? 0.00085 : 0.00034) * slab +
                                steps * (1.15 + 0.033 * s.np + 0.00014 * slab));
  const double there = 7.6 + (tall ? 0.0002 : 0.00017) * sides +
                       steps * ((s.np <= 64 ? 12.0 : 19.0) + (tall ? 0.00021 : 0.00032) * sides);
  return here <= there;
}

// CTAs of a cluster for one matrix: the most (at least 64 columns for each) with which all matrices
// are resident at once, or the fewest that hold a matrix; 0 where no cluster holds it or the tiled
// products end sooner.  (A cluster has to find its SMs in one part of the GPU: of 16 CTAs only a
// few are resident together.)
cudaError_t muon_small_cluster(int n, int64_t length, int64_t batch, bool tall, int steps,
                               int* cluster) {
  *cluster = 0;
  int64_t at_once = 0;
  if (n > kSmallMaxN) return cudaSuccess;
  cudaError_t e = small_attrs<float>();
  if (e == cudaSuccess) e = small_attrs<__nv_bfloat16>();
  if (e != cudaSuccess) return e;
  for (int c = 1; c <= kSmallMaxCluster; c *= 2) {
    const size_t smem = small_shape(n, length, c).bytes();
    if (smem > kSmallMaxSmem) continue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    small_config(cfg, attr, 1, c, smem, nullptr);
    int resident = 0;
    e = cudaOccupancyMaxActiveClusters(&resident, muon_small_kernel<float>, &cfg);
    if (e != cudaSuccess) return e;
    if (resident < 1) continue;
    if (*cluster == 0 || (batch <= resident && length > 64 * (c / 2))) {
      *cluster = c;
      at_once = resident;
    }
  }
  if (*cluster > 0 &&
      !small_ends_first(small_shape(n, length, *cluster), length, batch, at_once, tall, steps))
    *cluster = 0;
  return cudaSuccess;
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
  p.err = o.err;
  p.wait_ns = kDefaultWaitNs;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  small_config(cfg, attr, in.batch, cluster, p.shape.bytes(), s);
  return in.g_f32 ? cudaLaunchKernelEx(&cfg, muon_small_kernel<float>, p)
                  : cudaLaunchKernelEx(&cfg, muon_small_kernel<__nv_bfloat16>, p);
}

}  // namespace mlpb
