// A whole mixture-of-experts MLP for a few tokens (decoding), in one cooperative launch.
//
//   l = X Wr^T, the top k experts of each token by l, w = softmax(l) at them (or w / sum w)
//   a_s = w_s act(W1_e x_t)        for every pair s = (t, e)         bf16 [pairs][Fe]
//   Y_t = sum over t's pairs of W2_e a_s
//
// Bound by memory: up to 64 tokens share each expert's weights, which move once (a few flops a
// byte).  One CTA an SM runs three phases with a barrier over the grid between them:
//   router  a CTA takes an expert's row of Wr and eight tokens at a time;
//   fc1     units of 16 weight rows (8 gate and the same 8 up features, or 16 for GELU) of one
//           expert times that expert's tokens;
//   fc2     units of 16 output columns over all routed experts, so that a column's sum over
//           experts stays in one CTA (no atomics, a fixed order).
// The 16 warps of a CTA split a unit's K in steps of 32, warp w taking steps w, w + 16, ...,
// so that the CTA reads a kilobyte of each row at once; their partial sums meet in shared
// memory at the unit's end.
//
// The products run on mma.sync m16n8k16 with the weights as the 16-row operand and tokens as
// its 8 columns.  tcgen05 has no shape for this: its M is 64 or 128 rows of one operand and it
// would want both operands staged whole in shared memory, while the tensor work here is under a
// tenth of the time even at 64 tokens.  K is permuted the same way in both operands so that a
// lane's fragments are 16 consecutive bytes of a row: what a lane multiplies it copies itself
// (cp.async into slots of its own, as in join.cuh), and the ring of the next steps needs no
// barriers and runs on over the units' ends -- and over the barrier between fc1 and fc2: fc2's
// first weights are on their way while the last CTAs finish fc1.
//
// a is rounded to bf16, as every activation that a GEMM of this library reads; logits, softmax
// and all sums are fp32.
#include <algorithm>
#include <new>

#include "../../include/mlpb.h"
#include "common.cuh"
#include "pointwise.cuh"

namespace mlpb {

constexpr int kMoeThreads = 512;
constexpr int kMoeWarps = kMoeThreads / 32;
constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 256;
constexpr int kMoeMaxTopk = 16;
constexpr int kMoeUnits = 24;  // 16-byte ring units a thread
constexpr int kMoeRing = kMoeUnits * kMoeThreads * 16;
constexpr int kMoeTile = 130;  // floats a warp's 16 x 8 partial tile takes (see moe_reduce)
constexpr int kMoePairs = kMoeMaxTokens * kMoeMaxTopk;

enum MoeSite : uint32_t { kSiteMoeBarrier = 16 };

struct MoeSync {  // device words of a handle, zero between launches
  uint32_t arrived, done, err;
};

struct MoeParams {
  const __nv_bfloat16 *X, *Wr, *W1, *W2;
  __nv_bfloat16* Y;
  int32_t* ids;    // [T][K]
  float* weights;  // [T][K]
  float* logits;   // [T][E] scratch
  __nv_bfloat16* act;  // [T * K][Fe] scratch
  int T, H, Fe, E, K;
  int gated, normalize;
  MoeSync* sync;
  uint64_t wait_ns;
};

struct MoeShared {
  float part[2][kMoeWarps * kMoeTile];
  uint64_t mask[kMoeMaxExperts];      // tokens of an expert
  uint16_t off[kMoeMaxExperts];       // its first pair
  uint16_t active[kMoeMaxExperts];    // routed experts, ascending
  uint16_t ids[kMoePairs];            // [T][K]
  float w[kMoePairs];                 // [T][K]
  uint8_t tok[kMoePairs];             // token of pair s (pairs ordered by expert, then token)
  float wpair[kMoePairs];             // its weight
  int n_active, most;                 // routed experts, most tokens of one
  int abort;
};

constexpr size_t kMoeSmem = kMoeRing + sizeof(MoeShared);

// 16 bytes, or zeros where !ok (src is then any valid address).
__device__ __forceinline__ void moe_copy(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void moe_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void moe_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// c += A B: A 16 x 16 (lane: rows lane/4 and lane/4 + 8), B 16 x 8 (lane: column lane/4).
__device__ __forceinline__ void moe_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A barrier over the grid, number k (1, 2, ...) of the launch.  Bounded: false when it expired
// in any thread 0 (the launch then ends without its results and the handle reports it).
__device__ __forceinline__ bool moe_grid_barrier(const MoeParams& p, MoeShared& sh, uint32_t k) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&p.sync->arrived, 1u);
    const uint32_t want = k * gridDim.x;
    const uint64_t t0 = globaltimer_ns();
    uint32_t seen;
    for (uint32_t i = 1;; ++i) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];"
                   : "=r"(seen)
                   : "l"(&p.sync->arrived)
                   : "memory");
      if (seen >= want) break;
      if ((i & 63u) == 0u && globaltimer_ns() - t0 > p.wait_ns) {
        atomicCAS(&p.sync->err, 0u, kDevErrTimeout | kSiteMoeBarrier);
        sh.abort = 1;
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();
  return sh.abort == 0;
}

// Sum of the 16 warps' partial tiles (16 rows x 8 columns, c as moe_mma leaves it) for the
// value that this thread reads: column n = tid / 64, row r = (tid / 8) % 8 + 8 ((tid / 4) % 2);
// its four neighbours tid % 4 add four warps each and all four return the sum.  The layout --
// row bits 0-1, bit 3, bit 2, then the column, and 130 floats a warp -- keeps a warp's reads
// on 32 different banks.  `buf` alternates between calls: one barrier a call.
__device__ __forceinline__ float moe_reduce(MoeShared& sh, int buf, const float (&c)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, n0 = (lane & 3) * 2;
  float* t = sh.part[buf] + warp * kMoeTile + (g >> 2) * 8 + (g & 3);
  t[n0 * 16] = c[0];
  t[(n0 + 1) * 16] = c[1];
  t[n0 * 16 + 4] = c[2];
  t[(n0 + 1) * 16 + 4] = c[3];
  __syncthreads();
  const int part = threadIdx.x & 3, up = (threadIdx.x >> 2) & 1, f = (threadIdx.x >> 3) & 7;
  const int n = threadIdx.x >> 6;
  const float* s = sh.part[buf] + part * 4 * kMoeTile + n * 16 + (f >> 2) * 8 + up * 4 + (f & 3);
  float v = (s[0] + s[kMoeTile]) + (s[2 * kMoeTile] + s[3 * kMoeTile]);
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v;
}

// ------------------------------------------------------------------ router
__device__ __forceinline__ float moe_dot8(const uint4& a, const uint4& b, float s) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack_bf16x2(x[i]), v = unpack_bf16x2(y[i]);
    s = fmaf(u.x, v.x, s);
    s = fmaf(u.y, v.y, s);
  }
  return s;
}

__device__ void moe_logits(const MoeParams& p, MoeShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tgs = (p.T + 7) / 8;
  int buf = 0;
  for (int u = blockIdx.x; u < p.E * tgs; u += gridDim.x, buf ^= 1) {
    const int tg = u / p.E, e = u - tg * p.E, t0 = tg * 8, nt = min(8, p.T - t0);
    const __nv_bfloat16* w = p.Wr + static_cast<size_t>(e) * p.H;
    const __nv_bfloat16* x = p.X + static_cast<size_t>(t0) * p.H;
    float acc[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[t] = 0.f;
    for (int c = threadIdx.x * 8; c < p.H; c += kMoeThreads * 8) {
      const uint4 a = ld_global_nc_v4(w + c);
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t < nt) acc[t] = moe_dot8(a, ld_global_nc_v4(x + static_cast<size_t>(t) * p.H + c), acc[t]);
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t >= nt) break;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
      if (lane == 0) sh.part[buf][warp * 8 + t] = acc[t];
    }
    __syncthreads();
    if (threadIdx.x < nt) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kMoeWarps; ++k) s += sh.part[buf][k * 8 + threadIdx.x];
      __stcg(p.logits + static_cast<size_t>(t0 + threadIdx.x) * p.E + e, s);
    }
  }
}

// A key that orders like the float: larger floats have larger keys, NaN the least (1).
__device__ __forceinline__ uint32_t moe_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 as +0
  if (l != l) return 1u;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Every CTA routes all tokens itself (a warp a token) from the logits, then lists the pairs by
// expert; CTA 0 writes ids and weights out.
__device__ void moe_route(const MoeParams& p, MoeShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kPer = kMoeMaxExperts / 32;
  for (int t = warp; t < p.T; t += kMoeWarps) {
    float l[kPer];
    uint32_t key[kPer];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 32 + lane;
      const bool in = e < p.E;
      l[i] = in ? __ldcg(p.logits + static_cast<size_t>(t) * p.E + e) : -INFINITY;
      key[i] = in ? moe_key(l[i]) : 0u;
      top = fmaxf(top, l[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * 32 + lane < p.E) sum += expf(l[i] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float mine = 0.f;  // lane k keeps the k-th choice
    int mine_e = 0;
    for (int k = 0; k < p.K; ++k) {
      uint32_t best = 0u;
      int at = 0x7fffffff;
      float val = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (key[i] > best) {  // the lowest index of a lane's equals comes first
          best = key[i];
          at = i * 32 + lane;
          val = l[i];
        }
      const uint32_t all = __reduce_max_sync(0xffffffffu, best);
      const int e = __reduce_min_sync(0xffffffffu, best == all ? at : 0x7fffffff);
      val = __shfl_sync(0xffffffffu, val, e & 31);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * 32 + lane == e) key[i] = 0u;  // taken
      if (lane == k) {
        mine = expf(val - top) / sum;
        mine_e = e;
      }
    }
    if (p.normalize) {
      float s = lane < p.K ? mine : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      mine /= s;
    }
    if (lane < p.K) {
      sh.ids[t * p.K + lane] = static_cast<uint16_t>(mine_e);
      sh.w[t * p.K + lane] = mine;
      if (blockIdx.x == 0) {
        p.ids[t * p.K + lane] = mine_e;
        p.weights[t * p.K + lane] = mine;
      }
    }
  }
  __syncthreads();
  // tokens of each expert, as a bit mask
  for (int e = threadIdx.x; e < p.E; e += kMoeThreads) sh.mask[e] = 0ull;
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * p.K; i += kMoeThreads)
    atomicOr(reinterpret_cast<unsigned long long*>(&sh.mask[sh.ids[i]]), 1ull << (i / p.K));
  __syncthreads();
  if (warp == 0) {  // offsets of the experts' pairs, and the routed experts in order
    int pairs = 0, routed = 0, most = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < p.E ? __popcll(sh.mask[e]) : 0;
      int before = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      const uint32_t on = __ballot_sync(0xffffffffu, n > 0);
      if (e < p.E) sh.off[e] = static_cast<uint16_t>(pairs + before - n);
      if (n > 0) sh.active[routed + __popc(on & ((1u << lane) - 1u))] = static_cast<uint16_t>(e);
      pairs += __shfl_sync(0xffffffffu, before, 31);
      routed += __popc(on);
      most = max(most, static_cast<int>(__reduce_max_sync(0xffffffffu, n)));
    }
    if (lane == 0) {
      sh.n_active = routed;
      sh.most = most;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * p.K; i += kMoeThreads) {
    const int e = sh.ids[i], t = i / p.K;
    const int s = sh.off[e] + __popcll(sh.mask[e] & ((1ull << t) - 1ull));
    sh.tok[s] = static_cast<uint8_t>(t);
    sh.wpair[s] = sh.w[i];
  }
  __syncthreads();
}

// ------------------------------------------------------------------ fc1
// Tiles of eight of an expert's tokens, at most NT; a step's slot is 2 + NT units a thread.
template <int NT>
__device__ void moe_fc1(const MoeParams& p, MoeShared& sh, uint32_t ring, const uint8_t* ring_p,
                        int& buf) {
  constexpr int kDepth = kMoeUnits / (2 + NT);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int rows = p.gated ? 8 : 16;  // features of a unit
  const int fgs = (p.Fe + rows - 1) / rows;
  const int items = sh.n_active * fgs;
  const int ks = (p.H + 31) / 32;
  const int steps = warp < ks ? (ks - warp + kMoeWarps - 1) / kMoeWarps : 0;
  const uint32_t mine = ring + threadIdx.x * 16;
  const uint8_t* mine_p = ring_p + threadIdx.x * 16;
  constexpr uint32_t kUnit = kMoeThreads * 16;

  // the copies' place: unit pi, step pk; its rows and tokens
  int pi = blockIdx.x, pk = warp, pn = 0;
  const __nv_bfloat16 *lo = nullptr, *hi = nullptr;
  bool lo_ok = false, hi_ok = false;
  int tok[NT];
  auto open = [&]() {
    if (pi >= items) return;
    const int a = pi / fgs, f = (pi - a * fgs) * rows + g;
    const int e = sh.active[a];
    if (p.gated) {
      lo = p.W1 + (static_cast<size_t>(e) * 2 * p.Fe + f) * p.H;
      hi = lo + static_cast<size_t>(p.Fe) * p.H;
      lo_ok = hi_ok = f < p.Fe;
    } else {
      lo = p.W1 + (static_cast<size_t>(e) * p.Fe + f) * p.H;
      hi = lo + static_cast<size_t>(8) * p.H;
      lo_ok = f < p.Fe;
      hi_ok = f + 8 < p.Fe;
    }
    pn = __popcll(sh.mask[e]);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      tok[j] = j * 8 + g < pn ? sh.tok[sh.off[e] + j * 8 + g] : -1;
  };
  auto produce = [&](int slot) {
    if (pi < items) {
      const int c = pk * 32 + q * 8;
      const bool in = c < p.H;
      const uint32_t d = mine + slot * (2 + NT) * kUnit;
      moe_copy(d, lo_ok && in ? lo + c : p.X, lo_ok && in);
      moe_copy(d + kUnit, hi_ok && in ? hi + c : p.X, hi_ok && in);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (j * 8 < pn) {
          const bool ok = in && tok[j] >= 0;
          moe_copy(d + (2 + j) * kUnit, ok ? p.X + static_cast<size_t>(tok[j]) * p.H + c : p.X, ok);
        }
      pk += kMoeWarps;
      if (pk >= ks) {
        pk = warp;
        pi += gridDim.x;
        open();
      }
    }
    moe_commit();
  };
  if (steps == 0) pi = items;  // fewer steps than warps: nothing to copy
  open();
#pragma unroll
  for (int s = 0; s < kDepth; ++s) produce(s);

  int slot = 0;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int a = it / fgs, e = sh.active[a], f0 = (it - a * fgs) * rows;
    const int n = __popcll(sh.mask[e]);
    float c[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
    for (int st = 0; st < steps; ++st) {
      moe_wait<kDepth - 1>();
      const uint8_t* s = mine_p + slot * (2 + NT) * kUnit;
      const uint4 l = *reinterpret_cast<const uint4*>(s);
      const uint4 h = *reinterpret_cast<const uint4*>(s + kUnit);
      uint4 x[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (j * 8 < n) x[j] = *reinterpret_cast<const uint4*>(s + (2 + j) * kUnit);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (j * 8 < n) {
          moe_mma(c[j], l.x, h.x, l.y, h.y, x[j].x, x[j].y);
          moe_mma(c[j], l.z, h.z, l.w, h.w, x[j].z, x[j].w);
        }
      produce(slot);  // the slot has been read
      if (++slot == kDepth) slot = 0;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 8 >= n) break;
      float v = moe_reduce(sh, buf, c[j]);
      buf ^= 1;
      const int up = (threadIdx.x >> 2) & 1, f = (threadIdx.x >> 3) & 7;
      const int col = j * 8 + (threadIdx.x >> 6);
      bool write;
      int feat;
      if (p.gated) {
        const float o = __shfl_xor_sync(0xffffffffu, v, 4);  // gate's thread has up
        v = v * sigmoid_f(v) * o;
        feat = f0 + f;
        write = (threadIdx.x & 7) == 0;
      } else {
        float z;
        f2_unpack(gelu_x2(f2_pack(v, v)), v, z);
        feat = f0 + f + 8 * up;
        write = (threadIdx.x & 3) == 0;
      }
      if (write && col < n && feat < p.Fe) {
        const int pair = sh.off[e] + col;
        p.act[static_cast<size_t>(pair) * p.Fe + feat] = __float2bfloat16_rn(v * sh.wpair[pair]);
      }
    }
  }
}

// ------------------------------------------------------------------ fc2
// Columns of the products are all T tokens (NT tiles of 8); an expert's step copies and
// multiplies the tiles in which it has tokens.
template <int NT>
struct MoeFc2 {
  static constexpr int kDepth = kMoeUnits / (2 + NT);
  static constexpr uint32_t kUnit = kMoeThreads * 16;

  const MoeParams& p;
  const MoeShared& sh;
  int g, q, warp, ks, items, steps_total;
  uint32_t mine;
  // place of the copies
  int pi, pa, pk;
  const __nv_bfloat16 *lo, *hi;
  bool lo_ok, hi_ok;
  uint64_t mask;
  int off;

  __device__ MoeFc2(const MoeParams& p_, const MoeShared& sh_, uint32_t ring) : p(p_), sh(sh_) {
    const int lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    g = lane >> 2;
    q = lane & 3;
    ks = (p.Fe + 31) / 32;
    items = (p.H + 15) / 16;
    steps_total = sh.n_active * ks;  // of a unit, over all its warps
    mine = ring + threadIdx.x * 16;
  }
  // the first step of this warp: experts in order, steps of K within each
  __device__ void first(int item) {
    pi = item;
    pk = warp;
    pa = 0;
    settle();
  }
  __device__ void settle() {
    while (pk >= ks) {
      pk -= ks;
      ++pa;
    }
    if (pa >= sh.n_active) {  // the unit's steps are done: on to the next one
      pi += gridDim.x;
      pk = warp;
      pa = 0;
      if (warp >= steps_total) pi = items;  // this warp has no steps at all
      while (pk >= ks && pi < items) {
        pk -= ks;
        ++pa;
      }
    }
    if (pi < items) {
      const int e = sh.active[pa], r = pi * 16 + g;
      lo = p.W2 + (static_cast<size_t>(e) * p.H + r) * p.Fe;
      hi = lo + static_cast<size_t>(8) * p.Fe;
      lo_ok = r < p.H;
      hi_ok = r + 8 < p.H;
      mask = sh.mask[e];
      off = sh.off[e];
    }
  }
  __device__ __forceinline__ void weights(int slot) const {
    const int c = pk * 32 + q * 8;
    const bool in = c < p.Fe;
    const uint32_t d = mine + slot * (2 + NT) * kUnit;
    moe_copy(d, lo_ok && in ? lo + c : p.X, lo_ok && in);
    moe_copy(d + kUnit, hi_ok && in ? hi + c : p.X, hi_ok && in);
  }
  __device__ __forceinline__ void tokens(int slot) const {
    const int c = pk * 32 + q * 8;
    const bool in = c < p.Fe;
    const uint32_t d = mine + slot * (2 + NT) * kUnit;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (((mask >> (8 * j)) & 0xffull) == 0ull) continue;
      const int t = j * 8 + g;
      const bool ok = in && ((mask >> t) & 1ull) != 0ull;
      const int s = off + __popcll(mask & ((1ull << t) - 1ull));
      moe_copy(d + (2 + j) * kUnit, ok ? p.act + static_cast<size_t>(s) * p.Fe + c : p.X, ok);
    }
  }
  __device__ __forceinline__ bool more() const { return pi < items; }
  __device__ __forceinline__ void next() {
    pk += kMoeWarps;
    settle();
  }
};

template <int NT>
__device__ bool moe_fc2(const MoeParams& p, MoeShared& sh, uint32_t ring, const uint8_t* ring_p,
                        int& buf) {
  using F = MoeFc2<NT>;
  constexpr int kDepth = F::kDepth;
  F f(p, sh, ring);
  // the first steps' weights do not wait for fc1
  f.first(blockIdx.x);
#pragma unroll
  for (int s = 0; s < kDepth; ++s) {
    if (f.more()) {
      f.weights(s);
      f.next();
    }
  }
  moe_commit();
  if (!moe_grid_barrier(p, sh, 2)) return false;
  f.first(blockIdx.x);
#pragma unroll
  for (int s = 0; s < kDepth; ++s) {
    if (f.more()) {
      f.tokens(s);
      f.next();
    }
  }
  moe_commit();
  moe_wait<0>();
  const uint8_t* mine_p = ring_p + threadIdx.x * 16;
  const int steps =
      f.warp < f.steps_total ? (f.steps_total - f.warp + kMoeWarps - 1) / kMoeWarps : 0;
  int slot = 0;
  for (int it = blockIdx.x; it < f.items; it += gridDim.x) {
    float c[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
    int a = 0, k = f.warp;
    for (int st = 0; st < steps; ++st, k += kMoeWarps) {
      while (k >= f.ks) {
        k -= f.ks;
        ++a;
      }
      const uint64_t mask = sh.mask[sh.active[a]];
      moe_wait<kDepth - 1>();
      const uint8_t* s = mine_p + slot * (2 + NT) * F::kUnit;
      const uint4 l = *reinterpret_cast<const uint4*>(s);
      const uint4 h = *reinterpret_cast<const uint4*>(s + F::kUnit);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (((mask >> (8 * j)) & 0xffull) != 0ull) {
          const uint4 x = *reinterpret_cast<const uint4*>(s + (2 + j) * F::kUnit);
          moe_mma(c[j], l.x, h.x, l.y, h.y, x.x, x.y);
          moe_mma(c[j], l.z, h.z, l.w, h.w, x.z, x.w);
        }
      if (f.more()) {
        f.weights(slot);
        f.tokens(slot);
        f.next();
      }
      moe_commit();
      if (++slot == kDepth) slot = 0;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 8 >= p.T) break;
      const float v = moe_reduce(sh, buf, c[j]);
      buf ^= 1;
      const int r = it * 16 + ((threadIdx.x >> 3) & 7) + 8 * ((threadIdx.x >> 2) & 1);
      const int t = j * 8 + (threadIdx.x >> 6);
      if ((threadIdx.x & 3) == 0 && t < p.T && r < p.H)
        p.Y[static_cast<size_t>(t) * p.H + r] = __float2bfloat16_rn(v);
    }
  }
  return true;
}

__global__ void __launch_bounds__(kMoeThreads, 1) moe_kernel(const MoeParams p) {
  extern __shared__ __align__(16) uint8_t moe_smem[];
  MoeShared& sh = *reinterpret_cast<MoeShared*>(moe_smem + kMoeRing);
  const uint32_t ring = smem_u32(moe_smem);
  if (threadIdx.x == 0) sh.abort = 0;
  moe_logits(p, sh);
  if (moe_grid_barrier(p, sh, 1)) {
    moe_route(p, sh);
    int buf = 0;
    if (sh.most <= 8)
      moe_fc1<1>(p, sh, ring, moe_smem, buf);
    else if (sh.most <= 16)
      moe_fc1<2>(p, sh, ring, moe_smem, buf);
    else if (sh.most <= 32)
      moe_fc1<4>(p, sh, ring, moe_smem, buf);
    else
      moe_fc1<8>(p, sh, ring, moe_smem, buf);
    moe_wait<0>();
    if (p.T <= 8)
      moe_fc2<1>(p, sh, ring, moe_smem, buf);
    else if (p.T <= 16)
      moe_fc2<2>(p, sh, ring, moe_smem, buf);
    else if (p.T <= 32)
      moe_fc2<4>(p, sh, ring, moe_smem, buf);
    else
      moe_fc2<8>(p, sh, ring, moe_smem, buf);
  }
  moe_wait<0>();
  // the last CTA out leaves the barrier's words as it found them, after an expired wait too
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(&p.sync->done, 1u) == gridDim.x - 1) {
    p.sync->arrived = 0u;
    p.sync->done = 0u;
    __threadfence();
  }
}

static size_t moe_align(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace mlpb

using namespace mlpb;

struct mlpb_moe {
  mlpb_moe_config cfg;
  int device, grid;
  MoeSync* sync;
};

static size_t moe_logits_bytes(const mlpb_moe_config& c) {
  return moe_align(static_cast<size_t>(c.max_tokens) * c.experts * 4);
}

extern "C" mlpb_status mlpb_moe_create(const mlpb_moe_config* cfg, mlpb_moe** out) {
  if (cfg == nullptr || out == nullptr) return MLPB_EINVAL;
  *out = nullptr;
  const mlpb_moe_config& c = *cfg;
  if (c.max_tokens < 1 || c.hidden <= 0 || c.ffn <= 0 || c.experts < 1 || c.topk < 1 ||
      c.topk > c.experts)
    return MLPB_EINVAL;
  if (c.act != MLPB_ACT_GELU_TANH && c.act != MLPB_ACT_SWIGLU) return MLPB_EINVAL;
  if ((c.normalize != 0 && c.normalize != 1) || c.flags != 0) return MLPB_EINVAL;
  if (c.max_tokens > kMoeMaxTokens || c.experts > kMoeMaxExperts || c.topk > kMoeMaxTopk ||
      c.hidden % 8 != 0 || c.ffn % 8 != 0 || c.hidden > (1 << 20) || c.ffn > (1 << 20))
    return MLPB_EUNSUPPORTED;
  mlpb_moe* h = new (std::nothrow) mlpb_moe();
  if (h == nullptr) return MLPB_ENOMEM;
  h->cfg = c;
  h->sync = nullptr;
  int major = 0, minor = 0, sms = 0, per_sm = 0;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, h->device) != cudaSuccess) {
    delete h;
    return MLPB_ECUDA;
  }
  if (major != 10 || minor != 3) {
    delete h;
    return MLPB_EUNSUPPORTED;
  }
  if (cudaFuncSetAttribute(moe_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kMoeSmem)) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, moe_kernel, kMoeThreads, kMoeSmem) !=
          cudaSuccess ||
      per_sm < 1 || cudaMalloc(reinterpret_cast<void**>(&h->sync), sizeof(MoeSync)) != cudaSuccess ||
      cudaMemset(h->sync, 0, sizeof(MoeSync)) != cudaSuccess) {
    if (h->sync) cudaFree(h->sync);
    delete h;
    return MLPB_ECUDA;
  }
  h->grid = sms;
  *out = h;
  return MLPB_OK;
}

extern "C" void mlpb_moe_destroy(mlpb_moe* h) {
  if (h == nullptr) return;
  if (h->sync) cudaFree(h->sync);
  delete h;
}

extern "C" mlpb_status mlpb_moe_workspace_size(const mlpb_moe* h, size_t* bytes) {
  if (h == nullptr || bytes == nullptr) return MLPB_EINVAL;
  const mlpb_moe_config& c = h->cfg;
  *bytes = moe_logits_bytes(c) + moe_align(static_cast<size_t>(c.max_tokens) * c.topk * c.ffn * 2);
  return MLPB_OK;
}

extern "C" mlpb_status mlpb_moe_forward(mlpb_moe* h, int64_t tokens, const void* X, const void* Wr,
                                        const void* W1, const void* W2, void* Y, int32_t* ids,
                                        float* weights, void* workspace, mlpb_stream_t stream) {
  if (h == nullptr || tokens < 0) return MLPB_EINVAL;
  const mlpb_moe_config& c = h->cfg;
  if (tokens > c.max_tokens) return MLPB_EUNSUPPORTED;
  if (!Wr || !W1 || !W2) return MLPB_EINVAL;
  if (tokens > 0 && (!X || !Y || !ids || !weights || !workspace)) return MLPB_EINVAL;
  for (const void* q : {X, Wr, W1, W2, static_cast<const void*>(Y), static_cast<const void*>(workspace)})
    if (q && (reinterpret_cast<uintptr_t>(q) & 15u) != 0) return MLPB_EINVAL;
  if ((reinterpret_cast<uintptr_t>(ids) & 3u) != 0 || (reinterpret_cast<uintptr_t>(weights) & 3u) != 0)
    return MLPB_EINVAL;
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess) return MLPB_ECUDA;
  if (device != h->device) return MLPB_EINVAL;
  if (tokens == 0) return MLPB_OK;
  MoeParams p{};
  p.X = static_cast<const __nv_bfloat16*>(X);
  p.Wr = static_cast<const __nv_bfloat16*>(Wr);
  p.W1 = static_cast<const __nv_bfloat16*>(W1);
  p.W2 = static_cast<const __nv_bfloat16*>(W2);
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.ids = ids;
  p.weights = weights;
  p.logits = static_cast<float*>(workspace);
  p.act = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(workspace) + moe_logits_bytes(c));
  p.T = static_cast<int>(tokens);
  p.H = static_cast<int>(c.hidden);
  p.Fe = static_cast<int>(c.ffn);
  p.E = c.experts;
  p.K = c.topk;
  p.gated = c.act == MLPB_ACT_SWIGLU ? 1 : 0;
  p.normalize = c.normalize;
  p.sync = h->sync;
  p.wait_ns = kDefaultWaitNs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(h->grid));
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = kMoeSmem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the grid's barriers need every CTA resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_kernel, p) == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}

extern "C" mlpb_status mlpb_moe_last_device_error(mlpb_moe* h, mlpb_stream_t stream) {
  if (h == nullptr) return MLPB_EINVAL;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MLPB_ECUDA;
  uint32_t v = 0;
  if (cudaMemcpy(&v, &h->sync->err, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess)
    return MLPB_ECUDA;
  if (v == 0) return MLPB_OK;
  if (cudaMemset(&h->sync->err, 0, sizeof(uint32_t)) != cudaSuccess) return MLPB_ECUDA;
  return MLPB_ETIMEOUT;
}
