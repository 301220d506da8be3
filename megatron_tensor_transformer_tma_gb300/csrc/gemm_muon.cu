// The products of a Newton-Schulz step (muon.cuh) on the tensor cores, for a batch of matrices.
//
// The pipeline is that of gemm.cuh (pairs of CTAs, 256 x 256 tiles, a TMA ring, two accumulators
// in tensor memory, bounded waits), on fp16 operands.  The symmetric products (Gram, Poly) compute
// the tiles on and below the diagonal and write those below it twice, the second time transposed.
//   wide (rows <= cols)   Gram  A, B = X        K-major   K = cols
//                         Apply A = D K-major, B = X MN-major, K = rows; beta by row
//   tall                  Gram  A, B = X        MN-major  K = rows
//                         Apply A = X, B = D    K-major   K = cols; beta by column
//   Poly                  A, B = E              K-major   K = n
//
// An element of X' takes 8 bytes in and out beside 2 n operations, as much of the memory's time as
// of the tensor cores' at n = 1376, so the epilogue's tiles go through shared memory by TMA: each
// of eight epilogue warps has a slot for 32 rows by 64 columns, computes in place, stores the box,
// and loads its next box when the store has read it.  (Rows read and written by their threads,
// 16 bytes a lane, took 540 us for 16 matrices of 1376 x 4096, four times the product: every
// access touches 32 lines.)  The ring has 5 stages for that, 4 where W's fp32 boxes come too.
//
// Measured for 16 matrices of 1376 x 4096: Gram 110 us, Poly 51, Apply 205, the last with W 245.
// Gram runs at the rate of large products (84 % tensor-active at 4 x 2560 x 5120) but for its last
// wave; Apply loses 30 of its 205 us to the loads and stores of X's parts: without them it takes
// 165-170, without its arithmetic as long.  Boxes half as wide in two slots a warp took 205, in
// three slots with a stage less 215, the next tile's X prefetched into L2 231.
//
// Few tiles leave pairs idle and the epilogue in the open.  Then tiles are 256 x 128 (the rule is
// at tiling() in muon.cu), and the symmetric products' K is cut into ranges (`split`), whose fp32
// sums go to the workspace for ortho_fold_kernel, which adds them in their order on all SMs and
// does what the epilogue does.  (The warp that comes last doing that in the product's own kernel
// took 8 us for three ranges of 1376 x 1376: a fence, an atomic and a quarter of the SMs.)
#include <algorithm>

#include "gemm.cuh"
#include "muon.cuh"

namespace mlpb {

// Instruction descriptor of kind::f16 with fp16 operands (format code 0), fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

struct OrthoTile {
  int b, mp, nt;     // matrix, tile of 256 rows, tile of BN columns
  int part, parts;   // range of K
  bool mirror;       // below the diagonal: its transpose is stored too
};

template <OrthoOp Op>
constexpr bool kSymmetric = Op == OrthoOp::Gram || Op == OrthoOp::Poly;

template <OrthoOp Op, int BN>
__device__ __forceinline__ OrthoTile ortho_tile(int u, const OrthoParams& p) {
  OrthoTile t;
  t.part = 0;
  t.parts = 1;
  t.mirror = false;
  if constexpr (kSymmetric<Op>) {
    t.parts = p.split;
    t.part = u % p.split;
    u /= p.split;
    // row by row of 256, with R columns tiles in each more: R mp (mp + 1) / 2 tiles before row mp
    constexpr int R = 256 / BN;
    t.b = u / p.per_matrix;
    const int i = u - t.b * p.per_matrix;
    t.mp = static_cast<int>((sqrtf(8.0f / R * static_cast<float>(i) + 1.0f) - 1.0f) * 0.5f);
    while (R * t.mp * (t.mp + 1) / 2 > i) --t.mp;
    while (R * (t.mp + 1) * (t.mp + 2) / 2 <= i) ++t.mp;
    t.nt = i - R * t.mp * (t.mp + 1) / 2;
    t.mirror = t.nt < R * t.mp;
  } else {
    t.b = u / p.per_matrix;
    tile_coords(u - t.b * p.per_matrix, p.num_pm, p.num_n, 8, t.mp, t.nt);
  }
  return t;
}

__device__ __forceinline__ void ortho_range(const OrthoTile& t, int num_kb, int& kb0, int& kb1) {
  kb0 = num_kb * t.part / t.parts;
  kb1 = num_kb * (t.part + 1) / t.parts;
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

// Eight values of a 16-byte piece.
__device__ __forceinline__ void unpack_half8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_half2(w[e]);
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack_half8(const float (&v)[8]) {
  return make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]),
                    pack_half2(v[6], v[7]));
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ void sts2(uint32_t a, uint32_t low) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(low)) : "memory");
}

constexpr int kEpiRows = 32, kEpiCols = 64;
constexpr int kEpiBox = kEpiRows * kEpiCols * 2;  // 4 KB: rows of 128 bytes, 128-byte swizzle

constexpr int kEpiWarps = 8;
constexpr int kOrthoThreads = 64 + 32 * kEpiWarps;

template <OrthoOp Op, int BN>
struct OrthoSmem {
  static constexpr int b_stage = BN / 2 * kBK * 2;
  static constexpr int stage = kPairAStage + b_stage;
  static constexpr int stages = (Op == OrthoOp::Last ? 4 : 5) + (BN == 128 ? 1 : 0);
  // a slot: the first box, and a second one (low part, mirrored box) or W's two
  static constexpr int slot = Op == OrthoOp::Last ? 3 * kEpiBox : 2 * kEpiBox;
  static constexpr int epi = kEpiWarps * slot;
  static constexpr int bytes = stages * stage + epi + 1024 + 512;
  static_assert(bytes <= 232448, "shared memory of a CTA");
  static constexpr bool loads = Op != OrthoOp::Gram;
};

// Boxes of 64 columns that the matrix has in a tile.
template <OrthoOp Op, int BN>
__device__ __forceinline__ int ortho_boxes(const OrthoTile& t, const OrthoParams& p) {
  const int width = kSymmetric<Op> ? p.n : p.cols;
  return min(BN / kEpiCols, (width - t.nt * BN + kEpiCols - 1) / kEpiCols);
}

// Address of the 16-byte piece j of a box's row.
__device__ __forceinline__ uint32_t box_piece(uint32_t box, int row, int j) {
  return box + row * 128 + ((j ^ (row & 7)) << 4);
}

// A warp's boxes in order: of the 64-column boxes of a tile those of its half, tile after tile.
template <OrthoOp Op, int BN>
struct BoxWalk {
  int u, sub, subs;  // the tile, the box in it, the boxes that the matrix has there
  OrthoTile t;
  __device__ __forceinline__ void find(int half, const OrthoParams& p, int step) {
    for (; u < p.units; u += step) {
      t = ortho_tile<Op, BN>(u, p);
      subs = ortho_boxes<Op, BN>(t, p);
      sub = half;
      if (sub < subs) return;
    }
  }
  __device__ __forceinline__ void next(int half, const OrthoParams& p, int step) {
    sub += 2;
    if (sub >= subs) {
      u += step;
      find(half, p, step);
    }
  }
};

// Loads a box's inputs into its slot; one lane.
template <OrthoOp Op, int BN>
__device__ __forceinline__ void load_box(const BoxWalk<Op, BN>& w, int row0, uint32_t slot,
                                         uint32_t bar, const OrthoMaps& m, const OrthoParams& p) {
  const int col = w.t.nt * BN + w.sub * kEpiCols;
  const bool second =
      Op == OrthoOp::Apply || (Op == OrthoOp::Last && p.w != nullptr && !p.ragged);
  constexpr int more = Op == OrthoOp::Last ? 2 : 1;
  mbar_arrive_expect_tx(bar, kEpiBox * (second ? 1 + more : 1));
  tma_load_3d(slot, &m.in0, bar, col, row0, w.t.b);
  if (second) {
    tma_load_3d(slot + kEpiBox, &m.in1, bar, col, row0, w.t.b);
    if (Op == OrthoOp::Last)
      tma_load_3d(slot + 2 * kEpiBox, &m.in1, bar, col + 32, row0, w.t.b);
  }
}

// Vectors along a box's columns are held by the warp, two elements a lane.
struct ColumnPair {
  float lo, hi;  // of columns lane, 32 + lane
  // of column e of the half box that begins with piece j0
  __device__ __forceinline__ float at(int j0, int e) const {
    return __shfl_sync(0xffffffffu, j0 == 0 ? lo : hi, e);
  }
};

// The same box into L2, before its slot is free.
template <OrthoOp Op, int BN>
__device__ __forceinline__ void prefetch_box(const BoxWalk<Op, BN>& w, int row0,
                                             const OrthoMaps& m, const OrthoParams& p) {
  const int col = w.t.nt * BN + w.sub * kEpiCols;
  tma_prefetch_3d(&m.in0, col, row0, w.t.b);
  if (Op == OrthoOp::Apply || (Op == OrthoOp::Last && p.w != nullptr && !p.ragged)) {
    tma_prefetch_3d(&m.in1, col, row0, w.t.b);
    if (Op == OrthoOp::Last) tma_prefetch_3d(&m.in1, col + 32, row0, w.t.b);
  }
}

// Half a box of a symmetric product (pieces j0 to j0 + 3 of the thread's row m); the diagonal's
// element apart.
template <OrthoOp Op>
__device__ __forceinline__ void symmetric_box(float (&v)[32], int j0, uint32_t slot, int lane,
                                              int m, int col, const OrthoTile& t, float dm,
                                              const ColumnPair& dj, const OrthoParams& p) {
  if constexpr (Op == OrthoOp::Gram) {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] *= kXInv;  // A times 2^12
  }
  if (!t.mirror) {
    const int on = m - col - 8 * j0;
    float d = 0.0f;
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (e == on) {
        d = v[e];
        v[e] = 0.0f;
      }
    if (on >= 0 && on < 32 && m < p.n) {
      const size_t at = static_cast<size_t>(t.b) * p.ldn + m;
      if constexpr (Op == OrthoOp::Gram)
        p.diag[at] = d * kXInv;
      else
        p.beta[at] = p.a + dm * fmaf(p.c, dm, p.b) + p.c * (d * kEEInv);
    }
    __syncwarp();
  }
  const float lin = fmaf(p.c, dm, p.b) * (kXInv * kDScale);  // and by the row
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int j = j0 + q;
    float r[8];
    const uint32_t at = box_piece(slot, lane, j);
    if constexpr (Op == OrthoOp::Poly) {
      float e16[8];
      unpack_half8(lds16(at), e16);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] = fmaf(lin + dj.at(j0, 8 * q + i), e16[i], (p.c * (kEEInv * kDScale)) * v[8 * q + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = v[8 * q + i];
    }
    const uint4 h = pack_half8(r);
    sts16(at, h);
    if (t.mirror) {  // its column, 32 consecutive elements of a row across the warp
      const uint32_t w[4] = {h.x, h.y, h.z, h.w};
      const uint32_t to = slot + kEpiBox + 8 * j * 64 + lane * 2;
#pragma unroll
      for (int i = 0; i < 8; ++i) sts2(to + i * 64, w[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// Half a box of X' or of the result.
template <OrthoOp Op, bool kTall>
__device__ __forceinline__ void apply_box(const float (&v)[32], int j0, uint32_t slot, int lane,
                                          float bm, const ColumnPair& bj, float keep, float step,
                                          const OrthoParams& p) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int j = j0 + q;
    const uint32_t at = box_piece(slot, lane, j);
    float x[8], b[8], r[8];
    unpack_half8(lds16(at), x);
    if constexpr (kTall) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = bj.at(j0, 8 * q + i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = bm;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[8 * q + i] * (1.0f / kDScale);
    if constexpr (Op == OrthoOp::Apply) {
      float lo[8];
      unpack_half8(lds16(at + kEpiBox), lo);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = fmaf(p.low_beta ? b[i] : p.a, lo[i], r[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = fmaf(b[i], x[i], r[i]);
    if constexpr (Op == OrthoOp::Apply) {  // X' times 2^12, in two parts
      sts16(at, pack_half8(r));
      if (p.low_out) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] -= __half2float(__float2half_rn(r[i]));
        sts16(at + kEpiBox, pack_half8(r));
      }
    } else {
      // W's pieces: four columns each, columns 32 on in the second box
      const uint32_t w0 = box_piece(slot + kEpiBox * (1 + j / 4), lane, (2 * j) & 7);
      const uint32_t w1 = box_piece(slot + kEpiBox * (1 + j / 4), lane, (2 * j + 1) & 7);
      if (p.w == nullptr || p.ragged) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] *= kXInv;
      } else {
        const uint4 y = lds16(w0), z = lds16(w1);
        const uint32_t q[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = fmaf(-step, r[i], keep * __uint_as_float(q[i]));
      }
      if (p.w != nullptr || p.ragged) {
        sts16(w0, make_uint4(__float_as_uint(r[0]), __float_as_uint(r[1]), __float_as_uint(r[2]),
                             __float_as_uint(r[3])));
        sts16(w1, make_uint4(__float_as_uint(r[4]), __float_as_uint(r[5]), __float_as_uint(r[6]),
                             __float_as_uint(r[7])));
      }
      if (!p.ragged && (p.w == nullptr || p.wb != nullptr))
        sts16(at, make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]),
                             pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7])));
    }
  }
}

// The result's box where rows are no multiple of 16 bytes: from W's boxes row by row.
__device__ __forceinline__ void ragged_rows(uint32_t slot, int lane, int row0, int col,
                                            const OrthoTile& t, float keep, float step,
                                            const OrthoParams& p) {
  // eight rows at a time: all of W's values on their way before the first is used
  constexpr int kRows = 8;
#pragma unroll 1
  for (int r0 = 0; r0 < kEpiRows && row0 + r0 < p.rows; r0 += kRows) {
    float v[kRows][2], w[kRows][2];
    const size_t o = (static_cast<size_t>(t.b) * p.rows + row0 + r0) * p.cols + col + lane;
    auto here = [&](int r, int h) {
      return row0 + r0 + r < p.rows && col + lane + 32 * h < p.cols;
    };
    if (p.w != nullptr) {
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[r][h] = here(r, h) ? p.w[o + static_cast<size_t>(r) * p.cols + 32 * h] : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(v[r][h])
                     : "r"(box_piece(slot + kEpiBox * (1 + h), r0 + r, lane >> 2) +
                           (lane & 3) * 4));
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!here(r, h)) continue;
        const size_t at = o + static_cast<size_t>(r) * p.cols + 32 * h;
        if (p.w == nullptr) {
          p.out[at] = __float2bfloat16_rn(v[r][h]);
        } else {
          const float x = fmaf(-step * 4096.0f, v[r][h], keep * w[r][h]);
          p.w[at] = x;
          if (p.wb != nullptr) p.wb[at] = __float2bfloat16_rn(x);
        }
      }
  }
}

// Where a 32 x 64 box of a range's sums begins: [unit][CTA][epilogue warp][box of its half]
// [16][32].
template <int BN>
__device__ __forceinline__ size_t partial_box(int unit, int rank, int ewarp, int i) {
  return ((static_cast<size_t>(unit) * 2 + rank) * kEpiWarps + ewarp) * (BN / 128) * 512 + i * 512;
}

// One epilogue warp: the 32 accumulator rows of its lane quarter, the boxes of its half.
template <OrthoOp Op, bool kTall, int BN>
__device__ __forceinline__ void ortho_epilogue(uint32_t tmem_base, uint32_t tfull0,
                                               uint32_t tempty0, uint32_t tempty_lead,
                                               uint32_t slot, uint32_t box_bar, int ewarp,
                                               int quarter, int lane, int rank, int cid,
                                               int nclusters, const WaitCtx& wc,
                                               const OrthoMaps& maps, const OrthoParams& p) {
  using Sm = OrthoSmem<Op, BN>;
  const int half = ewarp >> 2;
  const int row = (rank * kBM) + quarter * 32;  // of a tile's 256
  float keep = 0.0f, step = 0.0f;
  if (Op == OrthoOp::Last && p.w != nullptr) {
    const float lr = __ldg(p.lr);
    keep = 1.0f - lr * p.decay;
    step = lr * p.scale * kXInv;
  }
  BoxWalk<Op, BN> ahead;
  ahead.u = cid;
  ahead.find(half, p, nclusters);
  pdl_wait();
  if (kSymmetric<Op> && p.split > 1) ahead.u = p.units;  // no boxes here
  bool coming = false;  // a box on its way into the slot
  if constexpr (Sm::loads) {
    if (ahead.u < p.units) {
      if (lane == 0) load_box<Op, BN>(ahead, ahead.t.mp * 256 + row, slot, box_bar, maps, p);
      coming = true;
      ahead.next(half, p, nclusters);
    }
  }
  int it = 0;
  uint32_t box_parity = 0;
  bool good = true;
  for (int u = cid; u < p.units && good; u += nclusters, ++it) {
    const int buf = it & 1;
    const OrthoTile t = ortho_tile<Op, BN>(u, p);
    const int subs = ortho_boxes<Op, BN>(t, p);
    const int row0 = t.mp * 256 + row, m = row0 + lane;
    const size_t vec = static_cast<size_t>(t.b) * p.ldn;  // of diag and beta
    float dm = 0.0f;  // the row's d or beta
    if (Op == OrthoOp::Poly && m < p.n) dm = __ldcg(p.diag + vec + m);
    if (!kSymmetric<Op> && !kTall && m < p.rows) dm = __ldcg(p.beta + vec + m);
    // d or beta along a box's columns, read a box ahead
    auto columns_of = [&](int col) {
      ColumnPair c{0.0f, 0.0f};
      if (Op == OrthoOp::Poly || (!kSymmetric<Op> && kTall)) {
        const float* at = (Op == OrthoOp::Poly ? p.diag : p.beta) + vec;
        const int width = kSymmetric<Op> ? p.n : p.cols;
        if (col + lane < width) c.lo = __ldcg(at + col + lane);
        if (col + 32 + lane < width) c.hi = __ldcg(at + col + 32 + lane);
        if (Op == OrthoOp::Poly) {  // what of E's factor goes by the column
          c.lo *= p.c * (kXInv * kDScale);
          c.hi *= p.c * (kXInv * kDScale);
        }
      }
      return c;
    };
    ColumnPair next_cj = columns_of(t.nt * BN + half * kEpiCols);
    int ok = 1;
    if (lane == 0)
      ok = wait_bounded(tfull0 + 8 * buf, (it >> 1) & 1, wc, kSiteEpiAccFull) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) break;
    __syncwarp();
    tc_fence_after();
    const uint32_t tacc =
        tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(buf * BN);
    const bool split = kSymmetric<Op> && p.split > 1;
    if (split) {  // this range's sums as they lie in the registers
      float4* part = p.partial + partial_box<BN>(u, rank, ewarp, 0) + lane;
      for (int sub = half, i = 0; sub < subs; sub += 2, ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[32];
          tmem_load_f32x32(tacc + sub * kEpiCols + 32 * h, v);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            part[(i * 16 + 8 * h + e) * 32] =
                make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
    }
    if (half >= subs || split) {  // no box of this tile
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(tempty0 + 8 * buf);
        else mbar_arrive_remote(tempty_lead + 8 * buf);
      }
      continue;
    }
#pragma unroll 1
    for (int sub = half; sub < subs; sub += 2) {
      const int col = t.nt * BN + sub * kEpiCols;
      const ColumnPair cj = next_cj;
      if (sub + 2 < subs) next_cj = columns_of(col + 2 * kEpiCols);
      if constexpr (Sm::loads) {
        if (lane == 0) ok = wait_bounded(box_bar, box_parity, wc, kSiteEpiAccFull) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          good = false;
          break;
        }
        box_parity ^= 1u;
        coming = false;
        if (lane == 0 && ahead.u < p.units)
          prefetch_box<Op, BN>(ahead, ahead.t.mp * 256 + row, maps, p);
      } else {
        if (lane == 0) bulk_wait_read<0>();  // the slot's last store
      }
      __syncwarp();
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tmem_load_f32x32(tacc + sub * kEpiCols + 32 * h, v);
        if (h == 1 && sub + 2 >= subs) {  // the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) mbar_arrive(tempty0 + 8 * buf);
            else mbar_arrive_remote(tempty_lead + 8 * buf);
          }
        }
        if constexpr (kSymmetric<Op>)
          symmetric_box<Op>(v, 4 * h, slot, lane, m, col, t, dm, cj, p);
        else
          apply_box<Op, kTall>(v, 4 * h, slot, lane, dm, cj, keep, step, p);
        __syncwarp();
      }
      if (Op == OrthoOp::Last && p.ragged) {
        __syncwarp();
        ragged_rows(slot, lane, row0, col, t, keep, step, p);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int height = kSymmetric<Op> ? p.n : p.rows;
        if (row0 < height) {
          if constexpr (kSymmetric<Op>) {
            tma_store_3d(&maps.out0, slot, col, row0, t.b);
            if (t.mirror) tma_store_3d(&maps.mirror, slot + kEpiBox, row0, col, t.b);
          } else if constexpr (Op == OrthoOp::Apply) {
            tma_store_3d(&maps.out0, slot, col, row0, t.b);
            if (p.low_out) tma_store_3d(&maps.out1, slot + kEpiBox, col, row0, t.b);
          } else if (!p.ragged) {
            if (p.w == nullptr || p.wb != nullptr) tma_store_3d(&maps.out0, slot, col, row0, t.b);
            if (p.w != nullptr) {
              tma_store_3d(&maps.in1, slot + kEpiBox, col, row0, t.b);
              if (col + 32 < p.cols)
                tma_store_3d(&maps.in1, slot + 2 * kEpiBox, col + 32, row0, t.b);
            }
          }
        }
        bulk_commit();
      }
      if constexpr (Sm::loads) {
        if (ahead.u < p.units) {
          if (lane == 0) {
            bulk_wait_read<0>();
            load_box<Op, BN>(ahead, ahead.t.mp * 256 + row, slot, box_bar, maps, p);
          }
          coming = true;
          ahead.next(half, p, nclusters);
        }
      }
      __syncwarp();
    }
  }
  if (lane == 0) {
    if (Sm::loads && coming) wait_drain(box_bar, box_parity, wc);  // after an expired wait
    bulk_wait_read<0>();  // what follows waits for the whole grid
  }
}

template <OrthoOp Op, bool kTall, int BN>
__global__ void __launch_bounds__(kOrthoThreads, 1)
    ortho_kernel(const __grid_constant__ OrthoMaps maps, const OrthoParams p) {
  using Sm = OrthoSmem<Op, BN>;
  constexpr int S = Sm::stages;
  constexpr bool a_mn = OrthoMajor<Op, kTall>::a_mn, b_mn = OrthoMajor<Op, kTall>::b_mn;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sA0 = base;
  const uint32_t sB0 = base + S * kPairAStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * Sm::stage + Sm::epi);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5 + 8);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + S);
  const uint32_t tfull0 = smem_u32(bars + 2 * S);
  const uint32_t tempty0 = smem_u32(bars + 2 * S + 2);
  const uint32_t drain = smem_u32(bars + 2 * S + 4);
  const uint32_t box0 = smem_u32(bars + 2 * S + 5);  // the epilogue warps' slots

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
      mbar_init(tempty0 + 8 * b, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(box0 + 8 * i, 1);
    *abort_flag = 0u;
    mbar_fence_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
    if (Sm::loads) tma_prefetch_desc(&maps.in0);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  pdl_launch_next();  // the roles wait for the kernel before this one where they first need it
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
      bool first = true;
      for (int u = cid; u < p.units; u += nclusters) {
        const OrthoTile t = ortho_tile<Op, BN>(u, p);
        const int ra = (t.mp * 2 + rank) * kBM, rb = t.nt * BN + BN / 2 * rank;
        int kb0, kb1;
        ortho_range(t, p.num_kb, kb0, kb1);
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bounded(empty0 + 8 * stage, phase ^ 1u, wc, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          const uint32_t sa = sA0 + stage * kPairAStage, sb = sB0 + stage * Sm::b_stage;
          if (first) {
            first = false;
            pdl_wait();
          }
          if (skip_once) {
            skip_once = false;  // fault injection: this stage is never armed
          } else if (leader) {
            const uint32_t fb = full0 + 8 * stage;
            mbar_arrive_expect_tx(fb, 2 * Sm::stage);
            ortho_load<a_mn, false>(sa, &maps.a, fb, kb * kBK, ra, t.b);
            ortho_load<b_mn, false>(sb, &maps.b, fb, kb * kBK, rb, t.b);
            armed |= 1u << stage;
            armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          } else {
            const uint32_t fb = full_lead + 8 * stage;
            ortho_load<a_mn, true>(sa, &maps.a, fb, kb * kBK, ra, t.b);
            ortho_load<b_mn, true>(sb, &maps.b, fb, kb * kBK, rb, t.b);
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
      constexpr uint32_t idesc = idesc_f16_f32(2 * kBM, BN, a_mn, b_mn);
      const uint64_t adesc0 = a_mn ? sdesc(sA0, kChunk, 1024, 2u) : sdesc(sA0, 16, 1024, 2u);
      const uint64_t bdesc0 = b_mn ? sdesc(sB0, kChunk, 1024, 2u) : sdesc(sB0, 16, 1024, 2u);
      constexpr uint32_t kAk = (a_mn ? 2048u : 32u) >> 4, kBk = (b_mn ? 2048u : 32u) >> 4;
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      pdl_wait();  // the bounded waits below count from where the operands may come
      for (int u = cid; u < p.units; u += nclusters, ++it) {
        const int buf = it & 1;
        const uint32_t acc_par = (it >> 1) & 1;
        if (!wait_bounded(tempty0 + 8 * buf, acc_par ^ 1u, wc, kSiteMmaAccEmpty)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * BN;
        const OrthoTile t = ortho_tile<Op, BN>(u, p);
        int kb0, kb1;
        ortho_range(t, p.num_kb, kb0, kb1);
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bounded(full0 + 8 * stage, phase, wc, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t as = adesc0 + static_cast<uint32_t>(stage) * (kPairAStage >> 4);
          const uint64_t bs = bdesc0 + static_cast<uint32_t>(stage) * (Sm::b_stage >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_pair(d, as + kk * kAk, bs + kk * kBk, idesc,
                           (kb != kb0 || kk != 0) ? 1u : 0u);
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
    ortho_epilogue<Op, kTall, BN>(tmem_base, tfull0, tempty0, tempty_lead,
                                  base + S * Sm::stage + (warp - 2) * Sm::slot,
                                  box0 + 8 * (warp - 2), warp - 2, warp & 3, lane, rank, cid,
                                  nclusters, wc, maps, p);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem_base, 2 * BN);
  }
}

// The sums of a symmetric product's ranges: a CTA adds those of one box, in their order, and
// stores what the product's own epilogue would.  A thread has one row's columns 4 g .. 4 g + 3 for
// four g; the box goes through shared memory so that rows and mirrored rows leave whole.
constexpr int kFoldThreads = 128;
constexpr int kFoldBox = kEpiRows * kEpiCols * 4;

template <OrthoOp Op, int BN>
__global__ void __launch_bounds__(kFoldThreads) ortho_fold_kernel(const OrthoParams p) {
  constexpr int kPitch = kEpiCols + 8;
  __shared__ __align__(16) __half box[kEpiRows * kPitch];
  __shared__ __align__(8) uint64_t bar_mem[2];
  __shared__ uint32_t abort_word;
  extern __shared__ __align__(128) uint8_t fold_smem[];
  constexpr int kBoxes = BN / 128;
  int at = blockIdx.x;
  const int i = at % kBoxes;
  at /= kBoxes;
  const int ewarp = at % kEpiWarps;
  at /= kEpiWarps;
  const int rank = at & 1, u = (at >> 1) * p.split;
  const OrthoTile t = ortho_tile<Op, BN>(u, p);
  const int sub = (ewarp >> 2) + 2 * i, quarter = (ewarp + 2) & 3;
  const int row0 = t.mp * 256 + rank * kBM + quarter * kEpiRows;
  const int col0 = t.nt * BN + sub * kEpiCols;
  if (row0 >= p.n || col0 >= p.n) return;
  // Each range's box is 8 KB in one piece: bulk copies, all in flight.  (Loads by threads, sixteen
  // each, took 2.3 us a round: 9 us for sixteen ranges.)
  const uint32_t bar = smem_u32(bar_mem), ring = smem_u32(fold_smem);
  if (threadIdx.x == 0) {
    abort_word = 0u;
    mbar_init(bar, 1);
    mbar_fence_init();
    pdl_wait();
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.split) * kFoldBox);
    for (int r = 0; r < p.split; ++r)
      bulk_load(ring + r * kFoldBox,
                p.partial + partial_box<BN>(u, rank, ewarp, i) + r * partial_box<BN>(1, 0, 0, 0),
                kFoldBox, bar);
  } else {
    pdl_wait();
  }
  pdl_launch_next();
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int m = row0 + lane;
  const size_t vec = static_cast<size_t>(t.b) * p.ldn;
  const size_t mat = static_cast<size_t>(t.b) * p.n * p.ldn;
  const float dm = Op == OrthoOp::Poly && m < p.n ? __ldcg(p.diag + vec + m) : 0.0f;
  const WaitCtx wc{&abort_word, p.err, p.wait_ns};
  // after an expired wait the copies land before shared memory is given up
  if (!wait_bounded(bar, 0, wc, kSiteEpiAccFull)) wait_drain(bar, 0, wc);
  float4 s[4] = {};
  const float4* from = reinterpret_cast<const float4*>(fold_smem) + warp * 32 + lane;
#pragma unroll 4
  for (int r = 0; r < p.split; ++r)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 x = from[r * (kFoldBox / 16) + k * 128];
      s[k].x += x.x;
      s[k].y += x.y;
      s[k].z += x.z;
      s[k].w += x.w;
    }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (warp + 4 * k) * 4, col = col0 + c;
    const float v[4] = {s[k].x, s[k].y, s[k].z, s[k].w};
    float r[4];
    if constexpr (Op == OrthoOp::Gram) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r[e] = v[e] * kXInv;  // A times 2^12
        if (col + e == m) {
          if (m < p.n) p.diag[vec + m] = r[e] * kXInv;
          r[e] = 0.0f;
        }
      }
    } else {
      float e16[4] = {0.f, 0.f, 0.f, 0.f}, dj[4] = {0.f, 0.f, 0.f, 0.f};
      if (m < p.n) {  // rows of 64 elements: inside the buffer
        const __half* from_e = p.e + mat + static_cast<size_t>(m) * p.ldn + col;
        const uint2 w = __ldcg(reinterpret_cast<const uint2*>(from_e));
        const float2 a = unpack_half2(w.x), b = unpack_half2(w.y);
        e16[0] = a.x;
        e16[1] = a.y;
        e16[2] = b.x;
        e16[3] = b.y;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < p.n) dj[e] = __ldcg(p.diag + vec + col + e);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lin = fmaf(p.c, dm + dj[e], p.b) * (kXInv * kDScale);
        r[e] = fmaf(lin, e16[e], (p.c * (kEEInv * kDScale)) * v[e]);
        if (col + e == m) {
          if (m < p.n) p.beta[vec + m] = p.a + dm * fmaf(p.c, dm, p.b) + p.c * (v[e] * kEEInv);
          r[e] = 0.0f;
        }
        if (col + e >= p.n) r[e] = 0.0f;  // E's pad is nobody's
      }
    }
    *reinterpret_cast<uint2*>(box + lane * kPitch + c) =
        make_uint2(pack_half2(r[0], r[1]), pack_half2(r[2], r[3]));
  }
  __syncthreads();
  __half* out = (Op == OrthoOp::Gram ? p.e : p.d) + mat;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int q = threadIdx.x + k * kFoldThreads;
    const int r = q >> 3, c = (q & 7) * 8;  // eight pieces a row
    if (row0 + r < p.n && col0 + c < p.n)
      *reinterpret_cast<uint4*>(out + static_cast<size_t>(row0 + r) * p.ldn + col0 + c) =
          *reinterpret_cast<const uint4*>(box + r * kPitch + c);
  }
  if (!t.mirror) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int q = threadIdx.x + k * kFoldThreads;
    const int c = q >> 2, r = (q & 3) * 8;  // four pieces a mirrored row
    if (col0 + c < p.n && row0 + r < p.n) {
      __half h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = box[(r + e) * kPitch + c];
      *reinterpret_cast<uint4*>(out + static_cast<size_t>(col0 + c) * p.ldn + row0 + r) =
          *reinterpret_cast<const uint4*>(h);
    }
  }
}

template <OrthoOp Op>
static cudaError_t launch_fold(const OrthoParams& p, cudaStream_t s) {
  const int boxes = p.units / p.split * 2 * kEpiWarps * (p.narrow ? 1 : 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(boxes));
  cfg.blockDim = dim3(kFoldThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.split) * kFoldBox;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.narrow ? cudaLaunchKernelEx(&cfg, ortho_fold_kernel<Op, 128>, p)
                  : cudaLaunchKernelEx(&cfg, ortho_fold_kernel<Op, 256>, p);
}

template <OrthoOp Op, bool kTall>
static cudaError_t attr_of() {
  const cudaError_t e =
      cudaFuncSetAttribute(ortho_kernel<Op, kTall, 128>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, OrthoSmem<Op, 128>::bytes);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(ortho_kernel<Op, kTall, 256>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 OrthoSmem<Op, 256>::bytes);
}

// Launched so that it may begin while the kernel before it ends (pdl_wait).
static void ortho_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int clusters, int smem,
                         cudaStream_t s) {
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2), 1, 1);
  cfg.blockDim = dim3(kOrthoThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

template <OrthoOp Op, bool kTall>
static cudaError_t launch_as(const OrthoMaps& m, const OrthoParams& p, int clusters,
                             cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  ortho_config(cfg, attr, clusters,
               p.narrow ? OrthoSmem<Op, 128>::bytes : OrthoSmem<Op, 256>::bytes, s);
  return p.narrow ? cudaLaunchKernelEx(&cfg, ortho_kernel<Op, kTall, 128>, m, p)
                  : cudaLaunchKernelEx(&cfg, ortho_kernel<Op, kTall, 256>, m, p);
}

template <OrthoOp Op>
static cudaError_t fold_attr_of() {
  const int most = kOrthoMaxSplit * kFoldBox;
  const cudaError_t e = cudaFuncSetAttribute(ortho_fold_kernel<Op, 128>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(ortho_fold_kernel<Op, 256>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

cudaError_t ortho_set_attrs(int* max_clusters) {
  for (cudaError_t e :
       {fold_attr_of<OrthoOp::Gram>(), fold_attr_of<OrthoOp::Poly>(),
        attr_of<OrthoOp::Gram, false>(), attr_of<OrthoOp::Gram, true>(),
        attr_of<OrthoOp::Poly, false>(), attr_of<OrthoOp::Apply, false>(),
        attr_of<OrthoOp::Apply, true>(), attr_of<OrthoOp::Last, false>(),
        attr_of<OrthoOp::Last, true>()})
    if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  ortho_config(cfg, attr, 2, OrthoSmem<OrthoOp::Last, 256>::bytes, nullptr);
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(max_clusters, ortho_kernel<OrthoOp::Last, false, 256>,
                                        &cfg);
}

cudaError_t launch_ortho(OrthoOp op, bool tall, const OrthoMaps& m, const OrthoParams& p,
                         int clusters, cudaStream_t s) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (op) {
    case OrthoOp::Gram:
      e = tall ? launch_as<OrthoOp::Gram, true>(m, p, clusters, s)
               : launch_as<OrthoOp::Gram, false>(m, p, clusters, s);
      return e == cudaSuccess && p.split > 1 ? launch_fold<OrthoOp::Gram>(p, s) : e;
    case OrthoOp::Poly:  // the same for both
      e = launch_as<OrthoOp::Poly, false>(m, p, clusters, s);
      return e == cudaSuccess && p.split > 1 ? launch_fold<OrthoOp::Poly>(p, s) : e;
    case OrthoOp::Apply:
      return tall ? launch_as<OrthoOp::Apply, true>(m, p, clusters, s)
                  : launch_as<OrthoOp::Apply, false>(m, p, clusters, s);
    case OrthoOp::Last:
      return tall ? launch_as<OrthoOp::Last, true>(m, p, clusters, s)
                  : launch_as<OrthoOp::Last, false>(m, p, clusters, s);
  }
  return e;
}

}  // namespace mlpb
