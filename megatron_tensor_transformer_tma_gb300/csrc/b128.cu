// Quantization to block-scaled E4M3 (b128.cuh), in the matrix's own layout and transposed.
//
// Reads of 2 (or 4) bytes and writes of one or two bytes an element bound it.  A CTA takes one
// 128 x 128 tile, so that every block of the matrix and of its transpose lies in one CTA and the
// tile is read from memory once.  Four lanes hold a row (four 16-byte pieces each, all in flight
// before the first is used), so that its maximum takes two exchanges; pieces are kept as loaded,
// bf16 in pairs (one instruction for two maxima), and the tile goes through shared memory for the
// columns, of which a thread takes two over 32 rows, and the transposed codes once more, so that
// rows leave whole (written by their threads, each store touched 32 lines: 143 us for T8192 x
// 20480 in both layouts).  That takes 117-132 us (5.1-5.7 TB/s), in rows alone 82-85 (6.0 TB/s, of
// 6.8 that a copy reaches).
#include <algorithm>

#include "b128.cuh"
#include "common.cuh"
#include "plan.h"

namespace mlpb {

constexpr int kQThreads = 256;

// Eight consecutive elements of a row, as loaded.
template <typename T>
struct Piece;

template <>
struct Piece<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = ld_global_v4(p); }
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void keep(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = u;
  }
  // Codes of the eight values times f.
  __device__ __forceinline__ uint2 codes(float f) const;
};

template <>
struct Piece<float> {
  uint4 u, v;
  __device__ __forceinline__ void load(const float* p) {
    u = ld_global_v4(p);
    v = ld_global_v4(p + 4);
  }
  __device__ __forceinline__ void clear() { u = v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void keep(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = u;
    reinterpret_cast<uint4*>(p)[1] = v;
  }
  __device__ __forceinline__ uint2 codes(float f) const {
    return make_uint2(b128_pack4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                 __uint_as_float(u.w), f),
                      b128_pack4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                                 __uint_as_float(v.w), f));
  }
};

// The larger magnitudes of two pairs of bf16 (a NaN's is the largest).
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t w) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A pair of bf16 as two floats.
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint2 Piece<__nv_bfloat16>::codes(float f) const {
  return make_uint2(b128_pack4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y), f),
                    b128_pack4(bf_lo(u.z), bf_hi(u.z), bf_lo(u.w), bf_hi(u.w), f));
}

// Magnitudes as fp32 bits: of pieces of a row, of pairs of a column.
__device__ __forceinline__ uint32_t magnitude(const Piece<__nv_bfloat16> (&p)[4]) {
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m = absmax2(m, p[j].u.x);
    m = absmax2(m, p[j].u.y);
    m = absmax2(m, p[j].u.z);
    m = absmax2(m, p[j].u.w);
  }
  return max(m << 16, m & 0xffff0000u);
}

__device__ __forceinline__ uint32_t magnitude(const Piece<float> (&p)[4]) {
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w[8] = {p[j].u.x, p[j].u.y, p[j].u.z, p[j].u.w,
                           p[j].v.x, p[j].v.y, p[j].v.z, p[j].v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, w[e] & 0x7fffffffu);
  }
  return m;
}

// Two columns' elements of a row, as kept in shared memory.
template <typename T>
struct Pair;

template <>
struct Pair<__nv_bfloat16> {
  uint32_t w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ float lo() const { return bf_lo(w); }
  __device__ __forceinline__ float hi() const { return bf_hi(w); }
};

template <>
struct Pair<float> {
  float2 f;
  __device__ __forceinline__ void load(const float* p) { f = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ float lo() const { return f.x; }
  __device__ __forceinline__ float hi() const { return f.y; }
};

__device__ __forceinline__ void column_magnitudes(const Pair<__nv_bfloat16> (&c)[32],
                                                  uint32_t (&m)[2]) {
  uint32_t a = 0u;
#pragma unroll
  for (int r = 0; r < 32; ++r) a = absmax2(a, c[r].w);
  m[0] = a << 16;
  m[1] = a & 0xffff0000u;
}

__device__ __forceinline__ void column_magnitudes(const Pair<float> (&c)[32], uint32_t (&m)[2]) {
  m[0] = m[1] = 0u;
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    m[0] = max(m[0], __float_as_uint(c[r].f.x) & 0x7fffffffu);
    m[1] = max(m[1], __float_as_uint(c[r].f.y) & 0x7fffffffu);
  }
}

template <typename T>
struct QTile {
  // Strides of 80 (bf16) and 132 (fp32) words: a quarter of a warp's 16-byte stores (two rows of
  // four pieces) and the reads of consecutive pairs of a row meet no bank twice.
  static constexpr int kStride = sizeof(T) == 2 ? 160 : 132;
  T v[kB128 * kStride];
  uint32_t colmax[4][kB128];
  uint32_t rowmax[kQThreads / 32];
};

// The scale byte of row `row` (of the `tiles` x 128 rows that have bytes) and block kb, and those
// of the blocks after the last one that share its word.
__device__ __forceinline__ void put_scale(uint8_t* s, int64_t tiles, int64_t row, int64_t kb,
                                          int64_t blocks, uint32_t byte) {
  uint8_t* w = s + ((kb >> 2) * tiles + (row >> 7)) * kB128Chunk + (row & 31) * 16 +
               ((row & 127) >> 5) * 4;
  w[kb & 3] = static_cast<uint8_t>(byte);
  if (kb == blocks - 1)
    for (int j = (kb & 3) + 1; j < 4; ++j) w[j] = static_cast<uint8_t>(kB128One);
}

template <typename T>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 2 ? 4 : 2)
    b128_quantize_kernel(const T* x, int64_t R, int64_t C, int square,
                         uint8_t* __restrict__ q, uint8_t* __restrict__ qs,
                         uint8_t* __restrict__ qt, uint8_t* __restrict__ qts) {
  extern __shared__ __align__(16) uint8_t q_smem[];
  pdl_wait();         // x may come from the kernel before this one
  pdl_launch_next();  // after it: what the next kernel reads early is final as well
  QTile<T>& sh = *reinterpret_cast<QTile<T>*>(q_smem);
  constexpr int S = QTile<T>::kStride;
  const int64_t cb = blockIdx.x, rb = blockIdx.y;
  const int64_t c0 = cb * kB128, r0 = rb * kB128;
  const int64_t cblocks = gridDim.x, rblocks = gridDim.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ch = (tid & 3) * 8, rr = tid >> 2;  // columns ch + 32 j of rows rr, rr + 64

  Piece<T> p[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = r0 + rr + 64 * i, col = c0 + ch + 32 * j;
      if (row < R && col < C) p[i][j].load(x + row * C + col);
      else p[i][j].clear();
    }
  uint32_t m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m[i] = magnitude(p[i]);
    m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
    m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
  }
  uint32_t all = 0u;
  if (square) {
    all = __reduce_max_sync(0xffffffffu, max(m[0], m[1]));
    if (lane == 0) sh.rowmax[warp] = all;
  }
  if (qt != nullptr) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) p[i][j].keep(sh.v + (rr + 64 * i) * S + ch + 32 * j);
  }
  __syncthreads();
  if (square) {
    all = 0u;
#pragma unroll
    for (int w = 0; w < kQThreads / 32; ++w) all = max(all, sh.rowmax[w]);
  }
  if (q != nullptr) {
    const int64_t ld = b128_ld(C);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = r0 + rr + 64 * i;
      const uint32_t byte = b128_scale_byte(square ? all : m[i]);
      const float f = b128_to_codes(byte);
      if ((tid & 3) == 0) put_scale(qs, rblocks, row, cb, cblocks, row < R ? byte : kB128One);
      if (row < R) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t col = c0 + ch + 32 * j;
          if (col < ld) *reinterpret_cast<uint2*>(q + row * ld + col) = p[i][j].codes(f);
        }
      }
    }
  }
  if (qt == nullptr) return;
  const int j = (tid & 63) * 2, g = tid >> 6;  // two columns, rows [32 g, 32 g + 32)
  Pair<T> c[32];
#pragma unroll
  for (int r = 0; r < 32; ++r) c[r].load(sh.v + (g * 32 + r) * S + j);
  uint32_t mt[2] = {all, all};
  if (!square) {
    column_magnitudes(c, mt);
    *reinterpret_cast<uint2*>(&sh.colmax[g][j]) = make_uint2(mt[0], mt[1]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint2 o = *reinterpret_cast<const uint2*>(&sh.colmax[k][j]);
      mt[0] = max(mt[0], o.x);
      mt[1] = max(mt[1], o.y);
    }
  }
  const int64_t ldt = b128_ld(R);
  const uint32_t b0 = b128_scale_byte(mt[0]), b1 = b128_scale_byte(mt[1]);
  if (g == 0) {
    put_scale(qts, cblocks, c0 + j, rb, rblocks, c0 + j < C ? b0 : kB128One);
    put_scale(qts, cblocks, c0 + j + 1, rb, rblocks, c0 + j + 1 < C ? b1 : kB128One);
  }
  const float f0 = b128_to_codes(b0), f1 = b128_to_codes(b1);
  if (square) __syncthreads();  // the columns have been read (else: above)
  // Rows of the transpose as 128 bytes, in whole pieces of 16 that trade places by pairs of rows.
  uint8_t* codes = reinterpret_cast<uint8_t*>(sh.v);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w0[4], w1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = h * 16 + e * 4;
      w0[e] = b128_pack4(c[r].lo(), c[r + 1].lo(), c[r + 2].lo(), c[r + 3].lo(), f0);
      w1[e] = b128_pack4(c[r].hi(), c[r + 1].hi(), c[r + 2].hi(), c[r + 3].hi(), f1);
    }
    uint8_t* o = codes + j * kB128 + (((g * 2 + h) ^ ((j >> 1) & 7)) << 4);
    *reinterpret_cast<uint4*>(o) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
    *reinterpret_cast<uint4*>(o + kB128) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = i * 32 + (tid >> 3), piece = tid & 7;
    if (c0 + col < C && r0 + piece * 16 < ldt)
      st_global_v4(qt + (c0 + col) * ldt + r0 + piece * 16,
                   *reinterpret_cast<const uint4*>(codes + col * kB128 +
                                                   ((piece ^ ((col >> 1) & 7)) << 4)));
  }
}

template <typename T>
static cudaError_t launch_as(const void* x, int64_t R, int64_t C, bool square, void* q, void* qs,
                             void* qt, void* qts, cudaStream_t s) {
  const int smem = static_cast<int>(sizeof(QTile<T>));
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        b128_quantize_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(b128_blocks(C)), static_cast<unsigned>(b128_blocks(R)));
  cfg.blockDim = dim3(kQThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // it begins with pdl_wait
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, b128_quantize_kernel<T>, static_cast<const T*>(x), R, C,
                            square ? 1 : 0, static_cast<uint8_t*>(q), static_cast<uint8_t*>(qs),
                            static_cast<uint8_t*>(qt), static_cast<uint8_t*>(qts));
}

cudaError_t launch_b128_quantize(const void* x, bool f32, int64_t rows, int64_t cols, bool square,
                                 void* q, void* qs, void* qt, void* qts, cudaStream_t s) {
  if (rows == 0 || cols == 0) return cudaSuccess;
  return f32 ? launch_as<float>(x, rows, cols, square, q, qs, qt, qts, s)
             : launch_as<__nv_bfloat16>(x, rows, cols, square, q, qs, qt, qts, s);
}

static bool b128_in_range(int64_t rows, int64_t cols) {
  return rows <= (int64_t{1} << 20) && cols <= (int64_t{1} << 20) && cols % 8 == 0;
}

}  // namespace mlpb

using namespace mlpb;

extern "C" mlpb_status mlpb_b128_sizes(int64_t rows, int64_t cols, int64_t* ld,
                                       size_t* scale_bytes) {
  if (rows < 0 || cols < 0 || ld == nullptr || scale_bytes == nullptr) return MLPB_EINVAL;
  if (rows > (int64_t{1} << 20) || cols > (int64_t{1} << 20)) return MLPB_EUNSUPPORTED;
  *ld = b128_ld(cols);
  *scale_bytes = static_cast<size_t>(b128_scale_bytes(rows, cols));
  return MLPB_OK;
}

extern "C" mlpb_status mlpb_b128_quantize(const void* x, int32_t x_f32, int64_t rows, int64_t cols,
                                          int32_t square, void* q, void* qs, void* qt, void* qts,
                                          mlpb_stream_t stream) {
  if (rows < 0 || cols < 0 || (x_f32 != 0 && x_f32 != 1) || (square != 0 && square != 1))
    return MLPB_EINVAL;
  if (!b128_in_range(rows, cols)) return MLPB_EUNSUPPORTED;
  if (rows == 0 || cols == 0) return MLPB_OK;
  if (x == nullptr || (q == nullptr && qt == nullptr) || (q == nullptr) != (qs == nullptr) ||
      (qt == nullptr) != (qts == nullptr))
    return MLPB_EINVAL;
  for (const void* p : {x, static_cast<const void*>(q), static_cast<const void*>(qs),
                        static_cast<const void*>(qt), static_cast<const void*>(qts)})
    if (!aligned16(p)) return MLPB_EINVAL;
  return launch_b128_quantize(x, x_f32 != 0, rows, cols, square != 0, q, qs, qt, qts,
                              reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MLPB_OK
             : MLPB_ECUDA;
}
