// The join between two blocks of a transformer's residual stream, in one pass each way:
//
//   forward   P = norm_post(Y);  Xout = alpha X + gate * P;  Xn = norm_pre(Xout)
//   backward  dh = dXout + norm_pre'(dXn);  dX = alpha dh;  dY = norm_post'(gate * dh)
//             and the gradients of alpha, gate and the norms' parameters
//
// Both are bound by memory: about 15 and 30 flops an element against 8 and 12 bytes of bf16.
// What carries them: every tensor moves once; a row stays in registers from its first
// reduction to its last; and the next rows are on their way while this one reduces.  The
// copies are cp.async into slots of shared memory that belong to one thread each: the thread
// reads back only what it copied itself, so the data needs no barrier at all, and a row's only
// barriers are those of its reductions.  (A ring of whole rows that the TMA unit fills, as in
// layernorm.cu, needs one more barrier a row, and waits that can expire, for which these calls
// have no handle to report to.)
//
// Per element the arithmetic is 15 (forward) to 25 (backward) instructions in f32x2 pairs, so
// what else a thread does for a row -- addresses, shuffles, barriers -- is spread over as many
// elements as its registers hold: 32 of a row in the forward, 16 in the backward, which keeps
// column sums too.  (8 a thread, with twice to four times the threads: the backward of T 8192
// H 8192 took 95 instructions an element and 290 us.)  And the usual call -- both norms, every
// warp's columns all inside the row: H 1024, 2048, 4096 and 8192, in the forward 5120 and 16384
// too -- has an instantiation of its own (kPlain) without the
// masks and the checks of what there is, which are half of the general one's instructions.  A
// CTA holds several rows where a row needs few warps.
//
// Measured (bandwidth over the bytes that a call cannot do without; the copy that the card
// reaches is 6.8 TB/s): forward T 8192 H 8192 bf16, RMSNorms and a gate, 92 us, 5.8 TB/s;
// backward 155 us, 5.2 TB/s, of which 143 the first pass; backward T 16384 H 4096 fp32,
// LayerNorms, 265 us, 6.6 TB/s.  What keeps the bf16 backward from the last fifth is the chain
// of a row (its reduction among it) with one row an SM in registers.  Ragged widths: RMS
// T 3000 H 7000 30 us forward (83 %), 62 backward (60 %); LayerNorms T 11061 H 2184 73 and 99
// (39 and 43 %), bound by instructions and the chain of their four reductions.  A gate for each
// token restarts a CTA's copies with every row: backward T 8192 H 8192 278 us (letting them run
// on from group to group gained nothing there and cost the others 1-2 %).
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "pointwise.cuh"

namespace mlpb {

constexpr int kJoinMaxBuf = 3;

struct JoinParams {
  int64_t T;
  int H;
  int G;                   // gate groups (0: no gate)
  int64_t rows_per_group;  // T / max(G, 1)
  int post, pre;           // mlpb_norm
  bool has_block;
  float eps;
  int nbuf;
  // the general backward's
  int wpr, rows;   // warps of a row, rows of a CTA
  int ring_bytes;  // of the ring
  bool split;      // its rows walk groups of their own
  bool ragged;     // some of the threads' columns are past the row's end
  // forward (inputs of both)
  const void *X, *Y;
  const float* alpha;
  const __nv_bfloat16 *gate, *gamma_post, *beta_post, *gamma_pre, *beta_pre;
  void* Xout;
  __nv_bfloat16* Xn;
  float* stats;  // [T][4]
  // backward
  const void *dXout, *dXn;
  void* dX;
  __nv_bfloat16* dY;
  float* dgate;          // [G][H], written here when a group has one CTA (blocks_per_group 1)
  float* part_gate;      // [G * blocks_per_group][H] otherwise
  float *part_gpost, *part_bpost, *part_gpre, *part_bpre;  // [walkers][H], NULL: not wanted
  float* part_alpha;     // [gridDim.x]
  int blocks_per_group;  // CTAs of a gate group; 1 when a CTA walks several groups
  int accumulate;        // dgate is added into (blocks_per_group 1)
};

// The warps of a row are a compile-time number (kWpr), but in the backward's general
// instantiations, where they are a runtime one (kWpr -12 or -16: one CTA of up to 12 or 16 warps
// an SM).
constexpr int kJoinMaxWarps = 16;
constexpr int join_rows(int wpr) { return wpr >= 8 ? 1 : 8 / wpr; }
constexpr int join_threads(int wpr) { return wpr < 0 ? -32 * wpr : 32 * wpr * join_rows(wpr); }
constexpr int join_ctas(int wpr) { return wpr < 0 ? 1 : 512 / join_threads(wpr); }  // of an SM

// Warps of a row in the forward: 256 elements each up to H 256, else 1024, rounded up to the next
// of 1, 2, 4, 8 and 16.  Five warps between (three rows an SM instead of two) where LayerNorm's
// instructions bound the call or the row fills them; RMS rows that do not are faster on eight
// (T 7280 bf16: LayerNorms H 4608 77 us against 93, H 5112 85 against 93, RMS H 4608 53 against 50,
// H 5112 55 against 52).
inline int join_fwd_wpr(int64_t H, bool layer) {
  if (H > 4096 && H <= 5120 && (layer || H % 1024 == 0)) return 5;
  return H <= 1024 ? 1 : H <= 2048 ? 2 : H <= 4096 ? 4 : H <= 8192 ? 8 : 16;
}

// How a backward is laid out: vectors of a thread, warps of a row in one CTA, rows and threads of a
// CTA, CTAs that share a row (a cluster, in the backward above H 8192).
struct JoinShape {
  int vpt, wpr, rows, threads, cluster;
};
inline JoinShape join_shape_plain(int vpt, int wpr) {
  return JoinShape{vpt, wpr, join_rows(wpr), join_threads(wpr), 1};
}
// `max` warps of a CTA, more where one row needs more; at most `most` rows: few rows are spread
// over the SMs.
inline JoinShape join_shape_general(int vpt, int64_t H, int max, int64_t most, int cluster = 1) {
  const int columns = 256 * vpt * cluster;
  const int wpr = static_cast<int>((H + columns - 1) / columns);
  const int rows = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(max / wpr, most)));
  return JoinShape{vpt, wpr, rows, 32 * wpr * rows, cluster};
}

// The backward's: plain instantiations, for 16 elements a thread, where whole rows fill an SM's 16
// warps, that is at powers of two from 1024 to 8192 (H 8192 LayerNorms 108 us; other multiples of
// 1024 leave warps idle and are as fast or faster in the general ones: T 6552 H 5120 bf16 RMS 92 us
// against 107, fp32 LayerNorms 126 against 140, but bf16 LayerNorms 126 against 119).  The general
// ones hold as many (8 up to H 256), on 12 warps of 168 registers where a row fits them (with
// LayerNorm 16 of 128 registers spill: T 11061 H 2184, 119 us against 104; RMS T 7122 H 2936, 64
// against 60), and above H 8192 with two CTAs a row (32 elements a thread in one CTA: T 610
// H 9856 44 us against 30, T 1024 H 16384 with LayerNorm over 90 against 88; three CTAs of 12
// warps there 128).
inline bool join_bwd_has_plain(int64_t H) {
  return H >= 1024 && H <= 8192 && (H & (H - 1)) == 0;
}
inline JoinShape join_bwd_shape(int64_t H, bool plain, int64_t most) {
  if (plain) return join_shape_plain(2, static_cast<int>(H / 512));
  return H <= 256 ? join_shape_general(1, H, 16, most)
                  : join_shape_general(2, H, 12, most, H <= 8192 ? 1 : 2);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most nbuf - 1 of this thread's groups are in flight.
__device__ __forceinline__ void cp_async_wait_ring(int nbuf) {
  if (nbuf == 3)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (nbuf == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Which elements of a row a thread holds: kVpt vectors of 8, as halves of 4.  All bf16: a
// vector is 8 consecutive elements (16 bytes).  Where a tensor is fp32 (kSplit), its halves are
// 128 apart, so that a warp's 16-byte accesses to it are consecutive too: a 32-byte sector read
// in two halves by two instructions would cross L2 twice.  Half h starts at c[h], and is all
// inside the row or not at all; with kFull, all are.
//
// What is past the row's end is not copied or stored, and its parameters are zeros.  The forward
// reads zeros in its place, and skips the vectors that a warp has none of (reading them all: T
// 3712 H 4392 41 us against 30).  The backward, whose instructions the masks doubled, reads all,
// from slots that are cleared before the first copy.
template <bool kSplit, int kVpt, bool kFull>
struct JoinCols {
  int c[2 * kVpt], H;
  __device__ __forceinline__ JoinCols(int wpr, int warp, int H_) : H(H_) {  // warp of a row's
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kVpt; ++k) {
      const int v = (k * wpr + warp) * 256;
      c[2 * k] = v + (kSplit ? lane * 4 : lane * 8);
      c[2 * k + 1] = c[2 * k] + (kSplit ? 128 : 4);
    }
  }
  __device__ __forceinline__ bool ok(int h) const { return kFull || c[h] < H; }
};

// Zeros in a CTA's ring, before its first copy.
__device__ __forceinline__ void join_clear(uint8_t* ring, int bytes) {
  for (int i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16)
    *reinterpret_cast<uint4*>(ring + i) = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

// Eight values as four f32x2 pairs (elements 0 and 1, 2 and 3, ...): two to a half.
using JoinVec = uint64_t[4];

__device__ __forceinline__ uint64_t join_pair(uint32_t w) {  // two bf16
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint64_t join_twice(float f) { return f2_pack(f, f); }
__device__ __forceinline__ float join_add_pair(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}
__device__ __forceinline__ void join_unpack(const uint4& u, JoinVec& v) {
  v[0] = join_pair(u.x);
  v[1] = join_pair(u.y);
  v[2] = join_pair(u.z);
  v[3] = join_pair(u.w);
}
__device__ __forceinline__ void join_unpack_half(uint2 u, uint64_t* v) {
  v[0] = join_pair(u.x);
  v[1] = join_pair(u.y);
}
__device__ __forceinline__ void join_unpack_half(float4 u, uint64_t* v) {
  v[0] = f2_pack(u.x, u.y);
  v[1] = f2_pack(u.z, u.w);
}

// Bytes of a warp's slots for one row of a tensor of type E: vector by vector, half by half
// where it is split, the lanes side by side.
template <class E, int kVpt>
constexpr uint32_t join_slots() {
  return 32 * kVpt * 8 * static_cast<uint32_t>(sizeof(E));
}

// Starts the copy of this thread's elements of a row into its slots of the warp's at `dst`.
template <class E, bool kSplit, int kVpt, bool kFull>
__device__ __forceinline__ void join_copy(uint32_t dst, const E* row,
                                          const JoinCols<kSplit, kVpt, kFull>& jc) {
  constexpr int kHalf = 4 * static_cast<int>(sizeof(E));  // bytes of a half
  const uint32_t lane = threadIdx.x & 31;
  if constexpr (!kSplit) {
    static_assert(kHalf == 8, "8 consecutive elements are bf16");
#pragma unroll
    for (int k = 0; k < kVpt; ++k)
      if (jc.ok(2 * k)) cp_async16(dst + (k * 32 + lane) * 16, row + jc.c[2 * k]);
  } else {
#pragma unroll
    for (int h = 0; h < 2 * kVpt; ++h)
      if (jc.ok(h)) {
        if constexpr (kHalf == 16)
          cp_async16(dst + (h * 32 + lane) * 16, row + jc.c[h]);
        else
          cp_async8(dst + (h * 32 + lane) * 8, row + jc.c[h]);
      }
  }
}

// Vector k of the thread's elements from its slots (zeros past the row's end, with `all` what the
// slots hold).
template <class E, bool all, bool kSplit, int kVpt, bool kFull>
__device__ __forceinline__ void join_read(const uint8_t* src, int k,
                                          const JoinCols<kSplit, kVpt, kFull>& jc, JoinVec& v) {
  const uint32_t lane = threadIdx.x & 31;
  if constexpr (!kSplit) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (all || jc.ok(2 * k)) u = *reinterpret_cast<const uint4*>(src + (k * 32 + lane) * 16);
    join_unpack(u, v);
  } else {
    using U = typename std::conditional<sizeof(E) == 4, float4, uint2>::type;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      U u{};
      if (all || jc.ok(2 * k + h))
        u = *reinterpret_cast<const U*>(src + ((2 * k + h) * 32 + lane) * sizeof(U));
      join_unpack_half(u, v + 2 * h);
    }
  }
}

// Vector k of a parameter, packed (zeros past its end, and where there is none).
template <bool kSplit, int kVpt, bool kFull>
__device__ __forceinline__ uint4 join_param(const __nv_bfloat16* p, int k,
                                            const JoinCols<kSplit, kVpt, kFull>& jc) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (p == nullptr) return u;
  if constexpr (!kSplit) {
    if (jc.ok(2 * k)) u = ld_global_nc_v4(p + jc.c[2 * k]);
  } else {
    if (jc.ok(2 * k)) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p + jc.c[2 * k]));
      u.x = a.x;
      u.y = a.y;
    }
    if (jc.ok(2 * k + 1)) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p + jc.c[2 * k + 1]));
      u.z = a.x;
      u.w = a.y;
    }
  }
  return u;
}

// Writes vector k of a row; with kBack, `v` becomes what was stored.
template <class E, bool kBack, bool kSplit, int kVpt, bool kFull>
__device__ __forceinline__ void join_store(E* row, int k, const JoinCols<kSplit, kVpt, kFull>& jc,
                                           JoinVec& v) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(v[i], f[2 * i], f[2 * i + 1]);
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (jc.ok(2 * k + h))
        *reinterpret_cast<float4*>(row + jc.c[2 * k + h]) =
            make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
  } else {
    const uint4 u = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    if constexpr (!kSplit) {
      if (jc.ok(2 * k)) st_global_v4(row + jc.c[2 * k], u);
    } else {
      if (jc.ok(2 * k)) *reinterpret_cast<uint2*>(row + jc.c[2 * k]) = make_uint2(u.x, u.y);
      if (jc.ok(2 * k + 1)) *reinterpret_cast<uint2*>(row + jc.c[2 * k + 1]) = make_uint2(u.z, u.w);
    }
    if constexpr (kBack) join_unpack(u, v);
  }
}

// Lets a kernel have `smem` bytes of dynamic shared memory. 48 KB, the kernel's static arrays
// among them (4 KB at most), need no leave. The leave is always for the same size: one for
// each launch's own would be undone by a second host thread before the first one's launch.
constexpr size_t kJoinMaxSmem = 212u << 10;

template <class K>
cudaError_t join_smem_attr(K* kernel, size_t smem) {
  return smem <= (44u << 10)
             ? cudaSuccess
             : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kJoinMaxSmem));
}

template <class XT, class YT>
cudaError_t join_fwd_run(const JoinParams& p, int num_sms, cudaStream_t s);
template <class XT, class YT>
cudaError_t join_bwd_run(const JoinParams& p, const JoinShape& sh, bool plain, int grid,
                         cudaStream_t s);

}  // namespace mlpb
