// Quantization to block-scaled E4M3 (b128.cuh), in the matrix's own layout and transposed.
//
// Reads of 2 (or 4) bytes and writes of one or two bytes an element bound it.  A CTA takes one
// 128 x 128 tile, so that every block of the matrix and of its transpose lies in one CTA and the
// tile is read from memory once: each thread keeps eight 16-byte pieces (eight rows apart in
// groups of 16 lanes a row) in flight, the rows' maxima come from shuffles of 16 lanes, and the
// tile goes through shared memory for the columns, of which a thread takes two over 32 rows
// (32 bytes of two rows of the transpose: whole sectors).
#include <algorithm>

#include "../../include/mlpb.h"
#include "b128.cuh"
#include "common.cuh"

namespace mlpb {

constexpr int kQThreads = 256;

template <typename T>
struct QTile {
  // a row's stride leaves the columns' reads (consecutive words of a row) and the rows' 16-byte
  // writes free of conflicts
  static constexpr int kStride = kB128 + 16 / static_cast<int>(sizeof(T));
  T v[kB128 * kStride];
  uint32_t colmax[4][kB128];
  uint32_t rowmax[kQThreads / 32];
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8], __nv_bfloat16* keep) {
  const uint4 u = ld_global_nc_v4(p);
  *reinterpret_cast<uint4*>(keep) = u;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_bf16x2(w[e]);
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8], float* keep) {
  const uint4 a = ld_global_nc_v4(p), b = ld_global_nc_v4(p + 4);
  reinterpret_cast<uint4*>(keep)[0] = a;
  reinterpret_cast<uint4*>(keep)[1] = b;
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
}

__device__ __forceinline__ float2 pair_at(const __nv_bfloat16* p) {
  return unpack_bf16x2(*reinterpret_cast<const uint32_t*>(p));
}
__device__ __forceinline__ float2 pair_at(const float* p) {
  return *reinterpret_cast<const float2*>(p);
}

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
__global__ void __launch_bounds__(kQThreads)
    b128_quantize_kernel(const T* __restrict__ x, int64_t R, int64_t C, int square,
                         uint8_t* __restrict__ q, uint8_t* __restrict__ qs,
                         uint8_t* __restrict__ qt, uint8_t* __restrict__ qts) {
  extern __shared__ __align__(16) uint8_t q_smem[];
  QTile<T>& sh = *reinterpret_cast<QTile<T>*>(q_smem);
  constexpr int S = QTile<T>::kStride;
  const int64_t cb = blockIdx.x, rb = blockIdx.y;
  const int64_t c0 = cb * kB128, r0 = rb * kB128;
  const int64_t cblocks = gridDim.x, rblocks = gridDim.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ch = (tid & 15) * 8, rr = tid >> 4;  // this thread's columns, its rows mod 16
  const bool col_ok = c0 + ch < C;

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 16 + rr;
    if (col_ok && r0 + r < R) {
      load8(x + (r0 + r) * C + c0 + ch, v[i], sh.v + r * S + ch);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] = 0.0f;
        sh.v[r * S + ch + e] = T(0.0f);
      }
    }
  }
  uint32_t m[8];
  uint32_t all = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = 0u;  // magnitudes order like their bits, NaN above infinity
#pragma unroll
    for (int e = 0; e < 8; ++e) m[i] = max(m[i], __float_as_uint(v[i][e]) & 0x7fffffffu);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
    all = max(all, m[i]);
  }
  if (square) {
    all = max(all, __shfl_xor_sync(0xffffffffu, all, 16));
    if (lane == 0) sh.rowmax[warp] = all;
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
    for (int i = 0; i < 8; ++i) {
      const int r = i * 16 + rr;
      const uint32_t byte = b128_scale_byte(square ? all : m[i]);
      const float f = b128_to_codes(byte);
      if ((tid & 15) == 0) put_scale(qs, rblocks, r0 + r, cb, cblocks, r0 + r < R ? byte : kB128One);
      if (r0 + r < R && c0 + ch < ld)
        *reinterpret_cast<uint2*>(q + (r0 + r) * ld + c0 + ch) =
            make_uint2(b128_pack4(v[i][0], v[i][1], v[i][2], v[i][3], f),
                       b128_pack4(v[i][4], v[i][5], v[i][6], v[i][7], f));
    }
  }
  if (qt == nullptr) return;
  const int j = (tid & 63) * 2, g = tid >> 6;  // two columns, rows [32 g, 32 g + 32)
  const T* col = sh.v + (g * 32) * S + j;
  uint32_t mt[2];
  if (square) {
    mt[0] = mt[1] = all;
  } else {
    mt[0] = mt[1] = 0u;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const float2 f = pair_at(col + r * S);
      mt[0] = max(mt[0], __float_as_uint(f.x) & 0x7fffffffu);
      mt[1] = max(mt[1], __float_as_uint(f.y) & 0x7fffffffu);
    }
    sh.colmax[g][j] = mt[0];
    sh.colmax[g][j + 1] = mt[1];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e)
      mt[e] = max(max(sh.colmax[0][j + e], sh.colmax[1][j + e]),
                  max(sh.colmax[2][j + e], sh.colmax[3][j + e]));
  }
  const int64_t ldt = b128_ld(R);
  const uint32_t b0 = b128_scale_byte(mt[0]), b1 = b128_scale_byte(mt[1]);
  if (g == 0) {
    put_scale(qts, cblocks, c0 + j, rb, rblocks, c0 + j < C ? b0 : kB128One);
    put_scale(qts, cblocks, c0 + j + 1, rb, rblocks, c0 + j + 1 < C ? b1 : kB128One);
  }
  if (c0 + j >= C) return;  // C is even
  const float f0 = b128_to_codes(b0), f1 = b128_to_codes(b1);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (r0 + g * 32 + h * 16 >= ldt) break;
    uint32_t w0[4], w1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float2 f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = pair_at(col + (h * 16 + e * 4 + i) * S);
      w0[e] = b128_pack4(f[0].x, f[1].x, f[2].x, f[3].x, f0);
      w1[e] = b128_pack4(f[0].y, f[1].y, f[2].y, f[3].y, f1);
    }
    uint8_t* o = qt + (c0 + j) * ldt + r0 + g * 32 + h * 16;
    st_global_v4(o, make_uint4(w0[0], w0[1], w0[2], w0[3]));
    st_global_v4(o + ldt, make_uint4(w1[0], w1[1], w1[2], w1[3]));
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
  const dim3 grid(static_cast<unsigned>(b128_blocks(C)), static_cast<unsigned>(b128_blocks(R)));
  b128_quantize_kernel<T><<<grid, kQThreads, smem, s>>>(
      static_cast<const T*>(x), R, C, square ? 1 : 0, static_cast<uint8_t*>(q),
      static_cast<uint8_t*>(qs), static_cast<uint8_t*>(qt), static_cast<uint8_t*>(qts));
  return cudaGetLastError();
}

cudaError_t launch_b128_quantize(const void* x, bool f32, int64_t rows, int64_t cols, bool square,
                                 void* q, void* qs, void* qt, void* qts, cudaStream_t s) {
  if (rows == 0 || cols == 0) return cudaSuccess;
  return f32 ? launch_as<float>(x, rows, cols, square, q, qs, qt, qts, s)
             : launch_as<__nv_bfloat16>(x, rows, cols, square, q, qs, qt, qts, s);
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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
