// 8-bit activation checkpoints: fc1's output saved as 8-bit codes with a scale for each 32
// features (act8.cuh), and the activation's backward from those codes.
//
//   save: A = act(Z); codes and scales of Z.          reads 2 B, writes 2 B + 1.03 B a feature
//   grad: zh = decoded codes; dZ = dA act'(zh), and A = act(zh) again for the weight
//         gradient that follows.                      reads 2 B + 1.03 B, writes 2 B + 2 B
//   (SwiGLU: gate and up for every feature of A)
//
// Both are bound by memory, so each tensor moves once: a thread owns 16 features (two 32-byte
// halves of a block; 8 where rows are not 32-byte aligned throughout), neighbouring threads a
// block, whose largest magnitude takes a shuffle or two.  A CTA is ux column units by 256 / ux
// rows, ux the power of two that covers a row's units (at most 256), so narrow rows do not idle
// threads; every thread walks act8_rows() rows of its columns, whose loads are issued together.
//
// Measured, with the rate of the bytes above (a copy reaches 6.8 TB/s): GELU T8192 F20480 save
// 124 us, 6.8 TB/s, grad 183 us, 6.4 TB/s; SwiGLU T16384 F11008 save 214 us, 6.8 TB/s, grad
// 277 us, 6.5 TB/s.
#include <algorithm>

#include "../../include/mlpb.h"
#include "act8.cuh"
#include "kernels.h"
#include "pointwise.cuh"

namespace mlpb {

constexpr int kAct8Threads = 256;

// Rows a thread has in flight (v times 8 features).  Saving: 4 of 8 features or 2 of 16 (one:
// GELU T8192 F20480 124 -> 132 us).  The gradient, which has more streams and registers: 2, or 1
// where gated (SwiGLU T16384 F11008, 16 features: 1 row 277 us, 2 301, 4 347; F11016, 8 features:
// 306, 326, 363).
constexpr int act8_rows(int v, bool grad, bool gated) {
  return grad ? (gated ? 1 : 2) : 4 / v;
}

// Where a thread works: its 8 V features start at column f of A's row, and its vectors of Z
// (or G, then U) at z0 (z1) with their blocks' scale bytes at s0 (s1).  Column units run over
// shard, block and place in a block; `in` is false past a short last block.
struct Act8Place {
  bool in;
  int f, z0, z1, s0, s1;
};

template <int V, bool kGated>
__device__ __forceinline__ Act8Place act8_place(int unit, int width, int blocks) {
  constexpr int kPer = 4 / V;               // units of a block
  const int blk = unit / kPer;              // over all segments of A's row
  const int seg = kGated ? blk / blocks : 0;
  const int b = blk - seg * blocks;
  const int c = b * kActBlock + (unit % kPer) * (8 * V);  // within the segment
  Act8Place p;
  p.in = c < width;
  p.f = seg * width + c;
  p.z0 = (kGated ? 2 * seg : seg) * width + c;
  p.z1 = p.z0 + width;
  p.s0 = (kGated ? 2 * seg : seg) * blocks + b;
  p.s1 = p.s0 + blocks;
  return p;
}

// 16 V bytes: a 16- or a 32-byte access.
template <int V>
struct Act8Words {
  uint32_t w[4 * V];
};

template <int V>
__device__ __forceinline__ Act8Words<V> act8_load(const void* p) {
  Act8Words<V> r;
  if constexpr (V == 1) {
    const uint4 u = ld_global_nc_v4(p);
    r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
  } else {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]),
          "=r"(r.w[6]), "=r"(r.w[7])
        : "l"(p));
  }
  return r;
}

template <int V>
__device__ __forceinline__ void act8_store(void* p, const Act8Words<V>& r) {
  if constexpr (V == 1) {
    st_global_v4(p, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
  } else {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]),
                 "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]),
                 "r"(r.w[7])
                 : "memory");
  }
}

// The 2 V words of codes of 8 V features.
template <int V>
struct Act8Codes {
  uint32_t w[2 * V];
};

template <int V>
__device__ __forceinline__ Act8Codes<V> act8_load_codes(const void* p) {
  Act8Codes<V> r;
  if constexpr (V == 1) {
    const uint2 u = __ldg(static_cast<const uint2*>(p));
    r.w[0] = u.x; r.w[1] = u.y;
  } else {
    const uint4 u = ld_global_nc_v4(p);
    r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
  }
  return r;
}

template <int V>
__device__ __forceinline__ void act8_store_codes(void* p, const Act8Codes<V>& r) {
  if constexpr (V == 1)
    *static_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
  else
    st_global_v4(p, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
}

template <int V>
__device__ __forceinline__ void act8_unpack(const Act8Words<V>& u, float (&v)[8 * V]) {
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) {
    const float2 f = unpack_bf16x2(u.w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <int V>
__device__ __forceinline__ Act8Words<V> act8_pack(const float (&v)[8 * V]) {
  Act8Words<V> r;
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) r.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  return r;
}

// The codes of this thread's values and its block's scale byte (the same in all threads of the
// block).  Every thread of the warp calls it; `u` is zero where there is nothing.
template <int V>
__device__ __forceinline__ Act8Codes<V> act8_encode(const Act8Words<V>& u,
                                                    const float (&v)[8 * V], uint32_t& scale) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) m = absmax_bf16x2(m, u.w[i]);
#pragma unroll
  for (int o = 1; o < 4 / V; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint32_t amax = max(m & 0xffffu, m >> 16);
  scale = act8_scale_byte(amax);
  const float f = act8_to_codes(scale, amax);
  Act8Codes<V> q;
#pragma unroll
  for (int i = 0; i < 2 * V; ++i)
    q.w[i] = act8_pack4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], f);
  return q;
}

template <int V>
__device__ __forceinline__ void act8_decode(const Act8Codes<V>& q, uint32_t scale,
                                            float (&v)[8 * V]) {
  const float s = act8_step(scale);
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) {
    float t[4];
    act8_unpack4(q.w[i], s, t);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = t[j];
  }
}

// `width` features a segment (all F for GELU, a shard's Fs for SwiGLU), `blocks` of 32 in
// each; F features and F1 saved values a row, nb scales a row.
template <int V, bool kGated>
__global__ void __launch_bounds__(kAct8Threads) act8_save_kernel(
    const __nv_bfloat16* __restrict__ Z, __nv_bfloat16* __restrict__ A,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t T, int64_t F, int64_t F1,
    int64_t nb, int width, int blocks, int units, int ux_log2, int col_ctas) {
  constexpr int kRows = act8_rows(V, false, kGated);
  const int ux = 1 << ux_log2;
  const int rows_cta = (kAct8Threads >> ux_log2) * kRows;
  const int64_t rb = blockIdx.x / col_ctas;
  const int unit = (blockIdx.x - static_cast<int>(rb) * col_ctas) * ux + (threadIdx.x & (ux - 1));
  const int64_t r0 = rb * rows_cta + (threadIdx.x >> ux_log2);
  const int step = kAct8Threads >> ux_log2;
  Act8Place p = act8_place<V, kGated>(unit, width, blocks);
  p.in = p.in && unit < units;
  Act8Words<V> g[kRows], u[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + i * step;
    g[i] = u[i] = Act8Words<V>{};
    if (p.in && r < T) {
      g[i] = act8_load<V>(Z + r * F1 + p.z0);
      if constexpr (kGated) u[i] = act8_load<V>(Z + r * F1 + p.z1);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + i * step;
    const bool ok = p.in && r < T;
    float a[8 * V], b[8 * V];
    uint32_t sa, sb = 0;
    act8_unpack<V>(g[i], a);
    const Act8Codes<V> qa = act8_encode<V>(g[i], a, sa);
    Act8Codes<V> qb{};
    if constexpr (kGated) {
      act8_unpack<V>(u[i], b);
      qb = act8_encode<V>(u[i], b, sb);
    }
    if (!ok) continue;
    act8_store_codes<V>(codes + r * F1 + p.z0, qa);
    if constexpr (kGated) act8_store_codes<V>(codes + r * F1 + p.z1, qb);
    if (unit % (4 / V) == 0) {
      scales[r * nb + p.s0] = static_cast<uint8_t>(sa);
      if constexpr (kGated) scales[r * nb + p.s1] = static_cast<uint8_t>(sb);
    }
    if (A != nullptr) {
      if constexpr (kGated) {
#pragma unroll
        for (int e = 0; e < 8 * V; ++e) a[e] = b[e] * (a[e] * sigmoid_f(a[e]));
      } else {
#pragma unroll
        for (int e = 0; e < 8 * V; e += 2)
          f2_unpack(gelu_x2(f2_pack(a[e], a[e + 1])), a[e], a[e + 1]);
      }
      act8_store<V>(A + r * F + p.f, act8_pack<V>(a));
    }
  }
}

template <int V, bool kGated>
__global__ void __launch_bounds__(kAct8Threads) act8_grad_kernel(
    const __nv_bfloat16* __restrict__ dA, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, __nv_bfloat16* __restrict__ dZ,
    __nv_bfloat16* __restrict__ A, int64_t T, int64_t F, int64_t F1, int64_t nb, int width,
    int blocks, int units, int ux_log2, int col_ctas) {
  constexpr int kRows = act8_rows(V, true, kGated);
  const int ux = 1 << ux_log2;
  const int rows_cta = (kAct8Threads >> ux_log2) * kRows;
  const int64_t rb = blockIdx.x / col_ctas;
  const int unit = (blockIdx.x - static_cast<int>(rb) * col_ctas) * ux + (threadIdx.x & (ux - 1));
  const int64_t r0 = rb * rows_cta + (threadIdx.x >> ux_log2);
  const int step = kAct8Threads >> ux_log2;
  const Act8Place p = act8_place<V, kGated>(unit, width, blocks);
  if (!p.in || unit >= units) return;
  Act8Words<V> d[kRows];
  Act8Codes<V> g[kRows], u[kRows];
  uint32_t sg[kRows], su[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + i * step;
    d[i] = Act8Words<V>{};
    g[i] = u[i] = Act8Codes<V>{};
    sg[i] = su[i] = 127u;
    if (r < T) {
      d[i] = act8_load<V>(dA + r * F + p.f);
      g[i] = act8_load_codes<V>(codes + r * F1 + p.z0);
      sg[i] = __ldg(scales + r * nb + p.s0);
      if constexpr (kGated) {
        u[i] = act8_load_codes<V>(codes + r * F1 + p.z1);
        su[i] = __ldg(scales + r * nb + p.s1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + i * step;
    if (r >= T) break;
    float v[8 * V], a[8 * V], act[8 * V];
    act8_unpack<V>(d[i], v);
    act8_decode<V>(g[i], sg[i], a);
    if constexpr (kGated) {
      float b[8 * V];
      act8_decode<V>(u[i], su[i], b);
#pragma unroll
      for (int e = 0; e < 8 * V; ++e) {
        const float s = sigmoid_f(a[e]);
        act[e] = b[e] * (a[e] * s);
        const float dg = v[e] * b[e] * s * (1.0f + a[e] * (1.0f - s));
        b[e] = v[e] * a[e] * s;  // dU
        a[e] = dg;               // dG
      }
      act8_store<V>(dZ + r * F1 + p.z0, act8_pack<V>(a));
      act8_store<V>(dZ + r * F1 + p.z1, act8_pack<V>(b));
    } else {
#pragma unroll
      for (int e = 0; e < 8 * V; e += 2) {
        uint64_t gelu;
        const uint64_t slope = gelu_both_x2(f2_pack(a[e], a[e + 1]), gelu);
        f2_unpack(gelu, act[e], act[e + 1]);
        f2_unpack(f2_mul(f2_pack(v[e], v[e + 1]), slope), v[e], v[e + 1]);
      }
      act8_store<V>(dZ + r * F1 + p.z0, act8_pack<V>(v));
    }
    if (A != nullptr) act8_store<V>(A + r * F + p.f, act8_pack<V>(act));
  }
}

// Sizes of a call: what the kernels index with.
struct Act8Dims {
  bool gated;
  int64_t F1, nb;
  int width, blocks, units, ux_log2, col_ctas;
  unsigned grid;
  bool wide;  // 16 features a thread
};

// `bits`: the pointers of the tensors that are read and written 32 bytes at a time, or'ed.
static mlpb_status act8_dims(int32_t act, int64_t T, int64_t F, int32_t tp, uintptr_t bits,
                             bool grad, Act8Dims* d) {
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
  // 32-byte accesses where every row and segment starts on one: measured at GELU T8192 F20480,
  // save 137 us with 8 features a thread and 124 with 16 (6.8 TB/s), grad 230 and 181 (6.5 TB/s;
  // there one exponential for both outputs counts too; 183 with the slope held finite)
  d->wide = width % 16 == 0 && (bits & 31u) == 0;
  d->units = static_cast<int>(segments * blocks * (d->wide ? 2 : 4));
  d->ux_log2 = 2;
  while ((1 << d->ux_log2) < d->units && (1 << d->ux_log2) < kAct8Threads) ++d->ux_log2;
  d->col_ctas = static_cast<int>((d->units + (1 << d->ux_log2) - 1) >> d->ux_log2);
  const int64_t rows_cta = static_cast<int64_t>(kAct8Threads >> d->ux_log2) *
                           act8_rows(d->wide ? 2 : 1, grad, d->gated);
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
  const mlpb_status st = act8_dims(act, 0, ffn, tp, 0, false, &d);
  if (st == MLPB_OK) *per_row = d.nb;
  return st;
}

extern "C" mlpb_status mlpb_act8_save(int32_t act, int64_t tokens, int64_t ffn, int32_t tp,
                                      const void* Z, void* A, void* codes, void* scales,
                                      mlpb_stream_t stream) {
  Act8Dims d;
  const mlpb_status st = act8_dims(
      act, tokens, ffn, tp, reinterpret_cast<uintptr_t>(Z) | reinterpret_cast<uintptr_t>(A),
      false, &d);
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
  auto* kernel = d.wide ? (d.gated ? act8_save_kernel<2, true> : act8_save_kernel<2, false>)
                        : (d.gated ? act8_save_kernel<1, true> : act8_save_kernel<1, false>);
  kernel<<<d.grid, kAct8Threads, 0, s>>>(z, a, c, sc, tokens, ffn, d.F1, d.nb, d.width, d.blocks,
                                         d.units, d.ux_log2, d.col_ctas);
  return cudaGetLastError() == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}

extern "C" mlpb_status mlpb_act8_grad(int32_t act, int64_t tokens, int64_t ffn, int32_t tp,
                                      const void* dA, const void* codes, const void* scales,
                                      void* dZ, void* A, mlpb_stream_t stream) {
  Act8Dims d;
  const mlpb_status st = act8_dims(act, tokens, ffn, tp,
                                   reinterpret_cast<uintptr_t>(dA) |
                                       reinterpret_cast<uintptr_t>(dZ) |
                                       reinterpret_cast<uintptr_t>(A),
                                   true, &d);
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
  auto* kernel = d.wide ? (d.gated ? act8_grad_kernel<2, true> : act8_grad_kernel<2, false>)
                        : (d.gated ? act8_grad_kernel<1, true> : act8_grad_kernel<1, false>);
  kernel<<<d.grid, kAct8Threads, 0, s>>>(da, c, sc, dz, a, tokens, ffn, d.F1, d.nb, d.width,
                                         d.blocks, d.units, d.ux_log2, d.col_ctas);
  return cudaGetLastError() == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}
