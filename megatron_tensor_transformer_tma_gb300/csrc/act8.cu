// 8-bit activation checkpoints: fc1's output saved as 8-bit codes with a scale for each 32
// features (act8.cuh), and the activation's backward from those codes.
//
//   save: A = act(Z); codes and scales of Z.          reads 2 B, writes 2 B + 1.03 B a feature
//   grad: zh = decoded codes; dZ = dA act'(zh), and A = act(zh) again for the weight
//         gradient that follows.                      reads 2 B + 1.03 B, writes 2 B + 2 B
//   (SwiGLU: gate and up for every feature of A)
//
// Both are bound by memory, so each tensor moves once: a thread owns 8 features (16 bytes
// of bf16, 8 bytes of codes), four neighbouring threads a block, whose largest magnitude
// takes two shuffles.  A CTA is ux column units by 256 / ux rows, ux the power of two that
// covers a row's units (at most 256), so narrow rows do not idle threads; every thread walks
// kRows rows of its columns, whose loads are issued together.
#include <algorithm>

#include "../../include/mlpb.h"
#include "act8.cuh"
#include "kernels.h"
#include "pointwise.cuh"

namespace mlpb {

constexpr int kAct8Threads = 256;
constexpr int kAct8Rows = 4;  // rows a thread has in flight

// Where a thread works: its 8 features start at column f of A's row, and its vectors of Z
// (or G, then U) at z0 (z1) with their blocks' scale bytes at s0 (s1).  Column units run over
// shard, block and quarter of a block; `in` is false past a short last block.
struct Act8Place {
  bool in;
  int f, z0, z1, s0, s1;
};

template <bool kGated>
__device__ __forceinline__ Act8Place act8_place(int unit, int width, int blocks) {
  const int blk = unit >> 2;                // over all segments of A's row
  const int seg = kGated ? blk / blocks : 0;
  const int b = blk - seg * blocks;
  const int c = b * kActBlock + (unit & 3) * 8;  // within the segment
  Act8Place p;
  p.in = c < width;
  p.f = seg * width + c;
  p.z0 = (kGated ? 2 * seg : seg) * width + c;
  p.z1 = p.z0 + width;
  p.s0 = (kGated ? 2 * seg : seg) * blocks + b;
  p.s1 = p.s0 + blocks;
  return p;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// The codes of this thread's 8 values and its block's scale byte (the same in all four
// threads of the block).  Every thread of the warp calls it; `u` is zero where there is
// nothing.
__device__ __forceinline__ uint2 act8_encode(const uint4& u, const float (&v)[8],
                                             uint32_t& scale) {
  uint32_t m = absmax_bf16x2(absmax_bf16x2(0u, u.x), u.y);
  m = absmax_bf16x2(absmax_bf16x2(m, u.z), u.w);
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  scale = act8_scale_byte(max(m & 0xffffu, m >> 16));
  const float f = act8_to_codes(scale);
  return make_uint2(act8_pack4(v[0], v[1], v[2], v[3], f), act8_pack4(v[4], v[5], v[6], v[7], f));
}

__device__ __forceinline__ void act8_decode(const uint2& q, uint32_t scale, float (&v)[8]) {
  const float s = act8_step(scale);
  float a[4], b[4];
  act8_unpack4(q.x, s, a);
  act8_unpack4(q.y, s, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// `width` features a segment (all F for GELU, a shard's Fs for SwiGLU), `blocks` of 32 in
// each; F features and F1 saved values a row, nb scales a row.
template <bool kGated>
__global__ void __launch_bounds__(kAct8Threads) act8_save_kernel(
    const __nv_bfloat16* __restrict__ Z, __nv_bfloat16* __restrict__ A,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t T, int64_t F, int64_t F1,
    int64_t nb, int width, int blocks, int units, int ux_log2, int col_ctas) {
  const int ux = 1 << ux_log2;
  const int rows_cta = (kAct8Threads >> ux_log2) * kAct8Rows;
  const int64_t rb = blockIdx.x / col_ctas;
  const int unit = (blockIdx.x - static_cast<int>(rb) * col_ctas) * ux + (threadIdx.x & (ux - 1));
  const int64_t r0 = rb * rows_cta + (threadIdx.x >> ux_log2);
  const int step = kAct8Threads >> ux_log2;
  Act8Place p = act8_place<kGated>(unit, width, blocks);
  p.in = p.in && unit < units;
  uint4 g[kAct8Rows], u[kAct8Rows];
#pragma unroll
  for (int i = 0; i < kAct8Rows; ++i) {
    const int64_t r = r0 + i * step;
    g[i] = u[i] = make_uint4(0, 0, 0, 0);
    if (p.in && r < T) {
      g[i] = ld_global_nc_v4(Z + r * F1 + p.z0);
      if constexpr (kGated) u[i] = ld_global_nc_v4(Z + r * F1 + p.z1);
    }
  }
#pragma unroll
  for (int i = 0; i < kAct8Rows; ++i) {
    const int64_t r = r0 + i * step;
    const bool ok = p.in && r < T;
    float a[8], b[8];
    uint32_t sa, sb = 0;
    unpack8(g[i], a);
    const uint2 qa = act8_encode(g[i], a, sa);
    uint2 qb = make_uint2(0, 0);
    if constexpr (kGated) {
      unpack8(u[i], b);
      qb = act8_encode(u[i], b, sb);
    }
    if (!ok) continue;
    *reinterpret_cast<uint2*>(codes + r * F1 + p.z0) = qa;
    if (kGated) *reinterpret_cast<uint2*>(codes + r * F1 + p.z1) = qb;
    if ((unit & 3) == 0) {
      scales[r * nb + p.s0] = static_cast<uint8_t>(sa);
      if (kGated) scales[r * nb + p.s1] = static_cast<uint8_t>(sb);
    }
    if (A != nullptr) {
      if constexpr (kGated) {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = b[e] * (a[e] * sigmoid_f(a[e]));
      } else {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          f2_unpack(gelu_x2(f2_pack(a[e], a[e + 1])), a[e], a[e + 1]);
      }
      st_global_v4(A + r * F + p.f, pack8(a));
    }
  }
}

template <bool kGated>
__global__ void __launch_bounds__(kAct8Threads) act8_grad_kernel(
    const __nv_bfloat16* __restrict__ dA, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, __nv_bfloat16* __restrict__ dZ,
    __nv_bfloat16* __restrict__ A, int64_t T, int64_t F, int64_t F1, int64_t nb, int width,
    int blocks, int units, int ux_log2, int col_ctas) {
  const int ux = 1 << ux_log2;
  const int rows_cta = (kAct8Threads >> ux_log2) * kAct8Rows;
  const int64_t rb = blockIdx.x / col_ctas;
  const int unit = (blockIdx.x - static_cast<int>(rb) * col_ctas) * ux + (threadIdx.x & (ux - 1));
  const int64_t r0 = rb * rows_cta + (threadIdx.x >> ux_log2);
  const int step = kAct8Threads >> ux_log2;
  const Act8Place p = act8_place<kGated>(unit, width, blocks);
  if (!p.in || unit >= units) return;
  uint4 d[kAct8Rows];
  uint2 g[kAct8Rows], u[kAct8Rows];
  uint32_t sg[kAct8Rows], su[kAct8Rows];
#pragma unroll
  for (int i = 0; i < kAct8Rows; ++i) {
    const int64_t r = r0 + i * step;
    d[i] = make_uint4(0, 0, 0, 0);
    g[i] = u[i] = make_uint2(0, 0);
    sg[i] = su[i] = 127u;
    if (r < T) {
      d[i] = ld_global_nc_v4(dA + r * F + p.f);
      g[i] = __ldg(reinterpret_cast<const uint2*>(codes + r * F1 + p.z0));
      sg[i] = __ldg(scales + r * nb + p.s0);
      if constexpr (kGated) {
        u[i] = __ldg(reinterpret_cast<const uint2*>(codes + r * F1 + p.z1));
        su[i] = __ldg(scales + r * nb + p.s1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kAct8Rows; ++i) {
    const int64_t r = r0 + i * step;
    if (r >= T) break;
    float v[8], a[8];
    unpack8(d[i], v);
    act8_decode(g[i], sg[i], a);
    if constexpr (kGated) {
      float b[8], act[8];
      act8_decode(u[i], su[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = sigmoid_f(a[e]);
        act[e] = b[e] * (a[e] * s);
        const float dg = v[e] * b[e] * s * (1.0f + a[e] * (1.0f - s));
        b[e] = v[e] * a[e] * s;  // dU
        a[e] = dg;               // dG
      }
      st_global_v4(dZ + r * F1 + p.z0, pack8(a));
      st_global_v4(dZ + r * F1 + p.z1, pack8(b));
      if (A != nullptr) st_global_v4(A + r * F + p.f, pack8(act));
    } else {
      if (A != nullptr) {
        float act[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          f2_unpack(gelu_x2(f2_pack(a[e], a[e + 1])), act[e], act[e + 1]);
        st_global_v4(A + r * F + p.f, pack8(act));
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        f2_unpack(f2_mul(f2_pack(v[e], v[e + 1]), gelu_grad_x2(f2_pack(a[e], a[e + 1]))), v[e],
                  v[e + 1]);
      st_global_v4(dZ + r * F1 + p.z0, pack8(v));
    }
  }
}

// Sizes of a call: what the kernels index with.
struct Act8Dims {
  bool gated;
  int64_t F1, nb;
  int width, blocks, units, ux_log2, col_ctas;
  unsigned grid;
};

static mlpb_status act8_dims(int32_t act, int64_t T, int64_t F, int32_t tp, Act8Dims* d) {
  if (act != MLPB_ACT_GELU_TANH && act != MLPB_ACT_SWIGLU) return MLPB_EINVAL;
  if (T < 0 || F <= 0 || tp < 1) return MLPB_EINVAL;
  if (F % tp != 0 || (F / tp) % 8 != 0) return MLPB_EUNSUPPORTED;
  if (F > (int64_t(1) << 28) || T > (int64_t(1) << 40)) return MLPB_EUNSUPPORTED;
  d->gated = act == MLPB_ACT_SWIGLU;
  const int64_t width = d->gated ? F / tp : F, segments = d->gated ? tp : 1;
  const int64_t blocks = (width + kActBlock - 1) / kActBlock;
  d->F1 = d->gated ? 2 * F : F;
  d->nb = (d->gated ? 2 : 1) * segments * blocks;
  d->width = static_cast<int>(width);
  d->blocks = static_cast<int>(blocks);
  d->units = static_cast<int>(segments * blocks * 4);
  d->ux_log2 = 2;
  while ((1 << d->ux_log2) < d->units && (1 << d->ux_log2) < kAct8Threads) ++d->ux_log2;
  d->col_ctas = static_cast<int>((d->units + (1 << d->ux_log2) - 1) >> d->ux_log2);
  const int64_t rows_cta = static_cast<int64_t>(kAct8Threads >> d->ux_log2) * kAct8Rows;
  const int64_t grid = (T + rows_cta - 1) / rows_cta * d->col_ctas;
  if (grid > 0x7fffffffll) return MLPB_EUNSUPPORTED;
  d->grid = static_cast<unsigned>(grid);
  return MLPB_OK;
}

}  // namespace mlpb

using namespace mlpb;

extern "C" mlpb_status mlpb_act8_scales(int32_t act, int64_t ffn, int32_t tp, int64_t* per_row) {
  Act8Dims d;
  if (per_row == nullptr) return MLPB_EINVAL;
  const mlpb_status st = act8_dims(act, 0, ffn, tp, &d);
  if (st == MLPB_OK) *per_row = d.nb;
  return st;
}

extern "C" mlpb_status mlpb_act8_save(int32_t act, int64_t tokens, int64_t ffn, int32_t tp,
                                      const void* Z, void* A, void* codes, void* scales,
                                      mlpb_stream_t stream) {
  Act8Dims d;
  const mlpb_status st = act8_dims(act, tokens, ffn, tp, &d);
  if (st != MLPB_OK) return st;
  if (tokens > 0 && (!Z || !codes || !scales)) return MLPB_EINVAL;
  for (const void* p : {Z, static_cast<const void*>(A), static_cast<const void*>(codes)})
    if (p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0) return MLPB_EINVAL;
  if (tokens == 0) return MLPB_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const auto* z = static_cast<const __nv_bfloat16*>(Z);
  auto* a = static_cast<__nv_bfloat16*>(A);
  auto* c = static_cast<uint8_t*>(codes);
  auto* sc = static_cast<uint8_t*>(scales);
  auto* kernel = d.gated ? act8_save_kernel<true> : act8_save_kernel<false>;
  kernel<<<d.grid, kAct8Threads, 0, s>>>(z, a, c, sc, tokens, ffn, d.F1, d.nb, d.width, d.blocks,
                                         d.units, d.ux_log2, d.col_ctas);
  return cudaGetLastError() == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}

extern "C" mlpb_status mlpb_act8_grad(int32_t act, int64_t tokens, int64_t ffn, int32_t tp,
                                      const void* dA, const void* codes, const void* scales,
                                      void* dZ, void* A, mlpb_stream_t stream) {
  Act8Dims d;
  const mlpb_status st = act8_dims(act, tokens, ffn, tp, &d);
  if (st != MLPB_OK) return st;
  if (tokens > 0 && (!dA || !codes || !scales || !dZ)) return MLPB_EINVAL;
  for (const void* p : {dA, codes, static_cast<const void*>(dZ), static_cast<const void*>(A)})
    if (p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0) return MLPB_EINVAL;
  if (tokens == 0) return MLPB_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const auto* da = static_cast<const __nv_bfloat16*>(dA);
  const auto* c = static_cast<const uint8_t*>(codes);
  const auto* sc = static_cast<const uint8_t*>(scales);
  auto* dz = static_cast<__nv_bfloat16*>(dZ);
  auto* a = static_cast<__nv_bfloat16*>(A);
  auto* kernel = d.gated ? act8_grad_kernel<true> : act8_grad_kernel<false>;
  kernel<<<d.grid, kAct8Threads, 0, s>>>(da, c, sc, dz, a, tokens, ffn, d.F1, d.nb, d.width,
                                         d.blocks, d.units, d.ux_log2, d.col_ctas);
  return cudaGetLastError() == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}
