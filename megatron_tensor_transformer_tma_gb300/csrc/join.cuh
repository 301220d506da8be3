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
// A row belongs to kTpr threads (32 to 1024, 16 of its elements each); a CTA of 256 or more
// threads holds kRows of them.  The norms' parameters are read again for every row: the data
// bypasses L1 (cp.async.cg, or the streaming reads of one line by one warp), so they stay
// there, and the registers stay free.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace mlpb {

constexpr int kJoinVpt = 2;  // vectors of 8 elements a thread
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
  float *part_gpost, *part_bpost, *part_gpre, *part_bpre;  // [gridDim.x][H], NULL: not wanted
  float* part_alpha;     // [gridDim.x]
  int blocks_per_group;  // CTAs of a gate group; 1 when a CTA walks several groups
  int accumulate;        // dgate is added into (blocks_per_group 1)
  bool direct_late;      // X and dXout are not in the ring (it would not fit)
};

// Threads of a row: 16 elements each, at least a warp (H <= 16384).
inline int join_tpr(int64_t H) {
  int t = 32;
  while (t < 1024 && static_cast<int64_t>(t) * kJoinVpt * 8 < H) t *= 2;
  return t;
}

constexpr int join_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

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

// Which elements of a row a thread holds.  All bf16: 8 consecutive ones a vector (16 bytes).
// Where a tensor is fp32 (kSplit), 4 + 4 of them 128 apart, so that a warp's 16-byte accesses
// to it are consecutive too: a 32-byte sector read in two halves by two instructions would
// cross L2 twice.
template <bool kSplit, int kTpr>
struct JoinCols {
  int c[kJoinVpt][2];
  bool ok[kJoinVpt][2];
  __device__ __forceinline__ JoinCols(int tr, int H) {
#pragma unroll
    for (int k = 0; k < kJoinVpt; ++k) {
      if constexpr (kSplit) {
        c[k][0] = (k * kTpr + (tr & ~31)) * 8 + (tr & 31) * 4;
        c[k][1] = c[k][0] + 128;
      } else {
        c[k][0] = (k * kTpr + tr) * 8;
        c[k][1] = c[k][0] + 4;
      }
      ok[k][0] = c[k][0] < H;
      ok[k][1] = c[k][1] < H;
    }
  }
};

// Bytes of a thread's slots for one row of a tensor of type E.
template <class E>
constexpr int join_slot() {
  return kJoinVpt * 8 * static_cast<int>(sizeof(E));
}

// Starts the copy of this thread's elements of a row into its slots at `dst` (the address of
// thread 0's; `nt` threads side by side).
template <class E, bool kSplit, int kTpr>
__device__ __forceinline__ void join_copy(uint32_t dst, int nt, const E* row,
                                          const JoinCols<kSplit, kTpr>& jc) {
  constexpr int kHalf = 4 * static_cast<int>(sizeof(E));  // bytes of four elements
#pragma unroll
  for (int k = 0; k < kJoinVpt; ++k) {
    if constexpr (!kSplit) {
      static_assert(kHalf == 8, "8 consecutive elements are bf16");
      if (jc.ok[k][0]) cp_async16(dst + (k * nt + threadIdx.x) * 16, row + jc.c[k][0]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t d = dst + ((k * 2 + h) * nt + threadIdx.x) * kHalf;
        if (jc.ok[k][h]) {
          if constexpr (kHalf == 16)
            cp_async16(d, row + jc.c[k][h]);
          else
            cp_async8(d, row + jc.c[k][h]);
        }
      }
    }
  }
}

__device__ __forceinline__ void join_unpack4(uint2 u, float* v) {
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

__device__ __forceinline__ void join_unpack4(float4 u, float* v) {
  v[0] = u.x;
  v[1] = u.y;
  v[2] = u.z;
  v[3] = u.w;
}

// Vector k of the thread's elements from its slots (zeros past the row's end).
template <class E, bool kSplit, int kTpr>
__device__ __forceinline__ void join_read(const uint8_t* src, int nt, int k,
                                          const JoinCols<kSplit, kTpr>& jc, float (&v)[8]) {
  if constexpr (!kSplit) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (jc.ok[k][0])
      u = *reinterpret_cast<const uint4*>(src + (k * nt + threadIdx.x) * 16);
    join_unpack4(make_uint2(u.x, u.y), v);
    join_unpack4(make_uint2(u.z, u.w), v + 4);
  } else {
    using U = typename std::conditional<sizeof(E) == 4, float4, uint2>::type;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      U u{};
      if (jc.ok[k][h])
        u = *reinterpret_cast<const U*>(src + ((k * 2 + h) * nt + threadIdx.x) * sizeof(U));
      join_unpack4(u, v + 4 * h);
    }
  }
}

// Vector k of a row in global memory.  kParam: a read-only parameter; otherwise a tensor that
// this thread may overwrite afterwards.
template <class E, bool kSplit, int kTpr, bool kParam>
__device__ __forceinline__ void join_load(const E* row, int k, const JoinCols<kSplit, kTpr>& jc,
                                          float (&v)[8]) {
  if constexpr (!kSplit) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (jc.ok[k][0]) {
      const uint4* q = reinterpret_cast<const uint4*>(row + jc.c[k][0]);
      u = kParam ? __ldg(q) : *q;
    }
    join_unpack4(make_uint2(u.x, u.y), v);
    join_unpack4(make_uint2(u.z, u.w), v + 4);
  } else {
    using U = typename std::conditional<sizeof(E) == 4, float4, uint2>::type;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      U u{};
      if (jc.ok[k][h]) {
        const U* q = reinterpret_cast<const U*>(row + jc.c[k][h]);
        u = kParam ? __ldg(q) : *q;
      }
      join_unpack4(u, v + 4 * h);
    }
  }
}

// Writes vector k of a row; for bf16 `v` becomes what was stored.
template <class E, bool kSplit, int kTpr>
__device__ __forceinline__ void join_store(E* row, int k, const JoinCols<kSplit, kTpr>& jc,
                                           float (&v)[8]) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (jc.ok[k][h])
        *reinterpret_cast<float4*>(row + jc.c[k][h]) =
            make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
  } else {
    uint2 u[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u[h] = make_uint2(pack_bf16x2(v[4 * h], v[4 * h + 1]), pack_bf16x2(v[4 * h + 2], v[4 * h + 3]));
      join_unpack4(u[h], v + 4 * h);
    }
    if constexpr (!kSplit) {
      if (jc.ok[k][0])
        st_global_v4(row + jc.c[k][0], make_uint4(u[0].x, u[0].y, u[1].x, u[1].y));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (jc.ok[k][h]) *reinterpret_cast<uint2*>(row + jc.c[k][h]) = u[h];
    }
  }
}

// Adds NV (1 or 2) values over the kTpr threads of a row, in a fixed order.  `sh` holds two
// float2 for every warp of the CTA; consecutive calls use them in turn (`par`), so one barrier
// a call is enough: who writes a place again has passed a barrier that every reader of it
// reached after reading.
template <int kTpr, int NV>
__device__ __forceinline__ void join_sum(float (&v)[NV], float2* sh, int& par) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (kTpr > 32) {
    constexpr int kWarps = kTpr / 32;
    const int group = threadIdx.x / kTpr;
    float2* slot = sh + par * (join_threads(kTpr) / 32) + group * kWarps;
    par ^= 1;
    if ((threadIdx.x & 31) == 0)
      slot[(threadIdx.x / 32) % kWarps] = make_float2(v[0], NV > 1 ? v[NV - 1] : 0.f);
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kTpr) : "memory");
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 s = slot[w];
      v[0] += s.x;
      if (NV > 1) v[NV - 1] += s.y;
    }
  }
}

cudaError_t launch_join_fwd(const JoinParams& p, bool x32, bool y32, int num_sms, cudaStream_t s);
cudaError_t launch_join_bwd_bf16(const JoinParams& p, int grid, cudaStream_t s);
cudaError_t launch_join_bwd_split(const JoinParams& p, bool x32, bool y32, int grid,
                                  cudaStream_t s);

}  // namespace mlpb
