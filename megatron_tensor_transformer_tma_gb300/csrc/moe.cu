// A whole mixture-of-experts MLP for a few tokens (decoding), in one cooperative launch.
//
//   l = X Wr^T, the top k experts of each token by l, w = softmax(l) at them (or w / sum w)
//   a_s = act(W1_e x_t),  y_s = W2_e a_s        for every pair s = (t, e)
//   Y_t = sum over t's pairs of w_s y_s
//
// Bound by memory: up to 64 tokens share each expert's weights, which move once (a few flops a
// byte).  One CTA an SM runs four phases with a barrier over the grid between them:
//   router   a CTA takes one, four or sixteen pairs of expert and token at a time;
//   fc1      units of 16 weight rows (8 gate and the same 8 up features, or 16 for GELU) of one
//            expert times that expert's tokens;
//   fc2      the same with 16 output columns a unit, into fp32 rows y_s;
//   combine  the pairs of a token, weighted, in order: no atomics, the same bits every run.
// (fc2 by units that run over all experts needs no y_s and no fourth phase, but has a unit for
// only every 16 output columns: 1.7 for each SM at H 4096, the second round on two thirds of
// them; and its columns are all T tokens, mostly not the expert's.)
//
// A CTA is four groups, each with units and a ring of shared-memory stages (16 rows by 256) of
// its own: a warp that fills the stages with tiled bulk copies (cp.async.bulk.tensor, 8 rows by
// 256 each), and four that multiply, each 64 of a stage's K; their partial sums meet in shared
// memory at the unit's end, while the other groups go on.  (With all sixteen multiplying warps
// at every stage, a stage took 0.4 us whatever it held: one warp's wait, loads, products and
// release after the other.)  Weights depend on the routing only, so the copies run on over the
// ends of units and over the barrier between fc1 and fc2: fc2's first weights arrive while the
// last CTAs finish fc1.  Tokens' fragments (from L2) each lane copies for itself, into a slot of
// its own in the same stage, as far ahead.
// Where an expert has more than 16 tokens, those copies, 512 bytes a token for every 8 KB of
// weights, would leave one stage in a group's ring.  Then the CTA has one ring and works on
// units of 64 rows, 16 for each group, and a stage holds its tokens once for all four: T 64
// H 4096 Fe 1792 4 experts top 2 75 us (with rings of the groups 125; two groups with units of
// 32 rows 154), 16 experts top 4 151 us (170); from 9 tokens on it loses (T 24 57 us against
// 51).
// Two other ways to move the weights measured slower: cp.async of each lane's own fragments was
// bound by instructions, about 200 a kilobyte (T 1: 4.1 TB/s over all); and bulk copies of
// single rows, one a lane, by their issue, about 70 ns each (2.1 TB/s).
//
// The products run on mma.sync m16n8k16 with the weights as the 16-row operand and tokens as
// its 8 columns.  (tcgen05 takes 64 or 128 rows: units four times as large would leave 2 for an
// SM at T 1, and the tensor pipe is busy 5 % of the time there, 12 % at T 16, a quarter with 38
// tokens an expert.)  K is permuted the same way in both operands so that a lane's fragments are
// 16 consecutive bytes of a row.
//
// Measured, over the bytes of the routed experts' weights (a copy reaches 6.8 TB/s): SwiGLU T 1
// H 4096 Fe 1376 top 8: 271 MB in 66 us, 4.1 TB/s; T 16 H 4096 Fe 688 128 experts top 8: 1.39 GB
// in 228 us, 6.1 TB/s; T 64 H 5120 Fe 2560 32 experts top 4: 2.52 GB in 412 us, 6.1 TB/s.  At T 1
// the launch, router, choice and three barriers take 13 us of that, and fc1 ends between 35 and
// 48 us by the part of the chip an SM is in (units claimed one by one instead measured 74 us in
// all).
//
// a is rounded to bf16, as every activation that a GEMM of this library reads; logits are
// pairs of fp32 values, softmax and all other sums fp32.  Every wait is bounded (common.cuh).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <new>
#include <type_traits>

#include "../../include/mlpb.h"
#include "common.cuh"
#include "pointwise.cuh"

namespace mlpb {

constexpr int kMoeThreads = 512;  // the multiplying warps
constexpr int kMoeWarps = kMoeThreads / 32;
constexpr int kMoeGroups = 4;                          // of four of them
constexpr int kMoeBlock = kMoeThreads + 32 * kMoeGroups;  // and a copying warp for each group
constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 256;
constexpr int kMoeMaxTopk = 16;
constexpr int kMoeKc = 256;     // K of a stage, and of a tiled copy
constexpr int kMoeBoxRows = 8;  // rows of a tiled copy
constexpr uint32_t kMoeBox = kMoeKc * kMoeBoxRows * 2;
constexpr uint32_t kMoeStageW = 2 * kMoeBox;  // a stage's weights; its tokens take 512 bytes each
constexpr uint32_t kMoeRing = 48u << 10;      // of one group
constexpr int kMoeMaxStages = 5;
constexpr int kMoeSharedFrom = 17;  // tokens of an expert from which a CTA works on one unit
constexpr int kMoePairs = kMoeMaxTokens * kMoeMaxTopk;

enum MoeSite : uint32_t { kSiteMoeGrid = 16, kSiteMoeEmpty = 17, kSiteMoeFull = 18 };

struct MoeSync {  // device words of a handle, zero between launches
  uint32_t arrived, done, err;
};

struct MoeParams {
  const __nv_bfloat16 *X, *Wr, *W1, *W2;
  __nv_bfloat16* Y;
  int32_t* ids;        // [T][K]
  float* weights;      // [T][K]
  float2* logits;      // [T][E] scratch: fp32 and what that leaves out
  __nv_bfloat16* act;  // [T * K][Fe] scratch: a_s, pairs ordered by expert, then token
  float* pair_y;       // [T * K][H] scratch: y_s
  int T, H, Fe, E, K;
  int gated, normalize;
  MoeSync* sync;
  uint64_t wait_ns;
  uint32_t zero;  // 0, which the compiler does not know (moe_release)
  int fault;      // MLPB_MOE_FAULT_INJECT: 1 a stage is never filled, 2 a CTA misses a barrier
};

struct MoeShared {
  float part[kMoeGroups][2][4 * 128];  // partial tiles of a group's four warps, twice
  uint64_t full[kMoeGroups][kMoeMaxStages], empty[kMoeGroups][kMoeMaxStages];
  uint64_t mask[kMoeMaxExperts];    // tokens of an expert
  uint16_t off[kMoeMaxExperts];     // its first pair
  uint16_t active[kMoeMaxExperts];  // routed experts, ascending
  uint16_t ids[kMoePairs];          // [T][K]
  float w[kMoePairs];               // [T][K]
  uint16_t slot[kMoePairs];         // [T][K]: the pair
  uint8_t tok[kMoePairs];           // token of a pair
  int n_active, most;               // routed experts, most tokens of one
  uint32_t abort;
};

constexpr size_t kMoeSmem = kMoeGroups * kMoeRing + sizeof(MoeShared);
static_assert(kMoeSmem <= 227 * 1024, "shared memory of a CTA");
static_assert(kMoeRing >= kMoeStageW + kMoeMaxTokens * kMoeKc * 2, "a stage at the most tokens");

// c += A B: A 16 x 16 (lane: rows lane/4 and lane/4 + 8), B 16 x 8 (lane: column lane/4).
__device__ __forceinline__ void moe_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Barriers over the grid, number k (1, 2) of the launch: every CTA arrives once, and waits until
// all have.  The wait is bounded: false when it expired here or elsewhere in the CTA (the launch
// then ends without its results and the handle reports it).
__device__ __forceinline__ void moe_grid_arrive(const MoeParams& p) {
  __threadfence();
  atomicAdd(&p.sync->arrived, 1u);
}

__device__ __forceinline__ bool moe_grid_wait(const MoeParams& p, MoeShared& sh, uint32_t k) {
  const uint32_t want = k * gridDim.x;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    uint32_t seen;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];"
                 : "=r"(seen)
                 : "l"(&p.sync->arrived)
                 : "memory");
    if (seen >= want) break;
    if ((i & 63u) == 0u) {
      if (*const_cast<volatile uint32_t*>(&sh.abort)) return false;
      if (globaltimer_ns() - t0 > p.wait_ns) {
        atomicCAS(&p.sync->err, 0u, kDevErrTimeout | kSiteMoeGrid);
        *const_cast<volatile uint32_t*>(&sh.abort) = 1u;
        return false;
      }
    }
  }
  __threadfence();
  return true;
}

// A barrier of the multiplying warps.
__device__ __forceinline__ void moe_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kMoeThreads) : "memory");
}

// The group, and the thread's and the warp's number in it.
__device__ __forceinline__ int moe_group() { return threadIdx.x >> 7; }
__device__ __forceinline__ int moe_thread() { return threadIdx.x & 127; }
__device__ __forceinline__ int moe_warp() { return (threadIdx.x >> 5) & 3; }

// Sum of a group's four partial tiles (16 rows x 8 columns, c as moe_mma leaves it), of which
// each thread returns one value: column thread / 16, row (thread / 2) % 8 + 8 (thread % 2) -- a
// gate and its up are neighbours.  `buf` alternates between calls: one barrier a call.
__device__ __forceinline__ float moe_reduce(MoeShared& sh, int buf, const float (&c)[4]) {
  const int lane = threadIdx.x & 31;
  float* part = sh.part[moe_group()][buf];
  float2* t =
      reinterpret_cast<float2*>(part + moe_warp() * 128 + (lane & 3) * 32 + (lane >> 2) * 2);
  t[0] = make_float2(c[0], c[2]);
  t[8] = make_float2(c[1], c[3]);
  asm volatile("bar.sync %0, 128;" ::"r"(moe_group() + 2) : "memory");
  const float* s = part + moe_thread();
  return (s[0] + s[128]) + (s[256] + s[384]);
}

// ------------------------------------------------------------------ router
__device__ __forceinline__ uint64_t moe_pair(uint32_t w) {
  const float2 f = unpack_bf16x2(w);
  return f2_pack(f.x, f.y);
}

// s += x y for two values; what the sum's rounding loses goes into c.  The product of two bf16
// is exact, so this is the error of one addition, by Knuth's two-sum (no order of magnitudes).
__device__ __forceinline__ void moe_add2(uint64_t x, uint64_t y, uint64_t& s, uint64_t& c) {
  const uint64_t t = f2_fma(x, y, s);
  const uint64_t r = f2_sub(s, t);                          // -(what s took of x y)
  const uint64_t lost = f2_add(f2_sub(s, f2_add(t, r)), f2_fma(x, y, r));
  c = f2_add(c, lost);
  s = t;
}

// Eight products into four sums and what they lose (two f32x2 each).
__device__ __forceinline__ void moe_dot8(const uint4& a, const uint4& b, uint64_t (&s)[2],
                                         uint64_t (&c)[2]) {
  moe_add2(moe_pair(a.x), moe_pair(b.x), s[0], c[0]);
  moe_add2(moe_pair(a.y), moe_pair(b.y), s[1], c[1]);
  moe_add2(moe_pair(a.z), moe_pair(b.z), s[0], c[0]);
  moe_add2(moe_pair(a.w), moe_pair(b.w), s[1], c[1]);
}

// v = v + w, each a sum (x) and what it lost (y).
__device__ __forceinline__ void moe_join(float2& v, float2 w) {
  const float t = v.x + w.x, r = t - v.x;
  v.y += w.y + ((v.x - (t - r)) + (w.x - r));
  v.x = t;
}

// A lane's sums, as one.
__device__ __forceinline__ float2 moe_total(const uint64_t (&s)[2], const uint64_t (&c)[2]) {
  float2 a[2], b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f2_unpack(s[i], a[i].x, b[i].x);
    f2_unpack(c[i], a[i].y, b[i].y);
    moe_join(a[i], b[i]);
  }
  moe_join(a[0], a[1]);
  return a[0];
}

// The sum over the lanes that differ in the bits up to `from`.
__device__ __forceinline__ float2 moe_sum(float2 v, int from) {
#pragma unroll 1
  for (int o = from; o > 0; o >>= 1)
    moe_join(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o),
                            __shfl_xor_sync(0xffffffffu, v.y, o)));
  return v;
}

// A pair of expert and token at a time, K over all sixteen warps; with more pairs than CTAs four
// pairs, K over four warps each, and with many sixteen, a warp each (T 64 H 2048 256 experts 165
// us, four warps 176; T 16 H 4096 128 experts 228, 230).  The code is kept short: it runs once, and
// fetching it takes longer than running it.  A logit is right to about 2^-40 of its terms'
// magnitudes, so that a token's experts are those of its exact logits whatever else is in the call;
// with fp32 sums, whose order depends on the number of pairs, near ties went either way (T 16 227
// us, T 64 H 5120 32 experts 412 against 413; in 64 bits 238 and 422).
__device__ __forceinline__ void moe_logits(const MoeParams& p, MoeShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pairs = p.E * p.T;
  const int ctas = gridDim.x;
  const int w = pairs <= ctas ? kMoeWarps : pairs <= 4 * ctas ? 4 : 1;  // warps of a pair
  const int at_once = kMoeWarps / w, sub = warp & (w - 1);
  int buf = 0;
#pragma unroll 1
  for (int first = blockIdx.x * at_once; first < pairs; first += gridDim.x * at_once, buf ^= 1) {
    const int pair = first + warp / w;
    const int t = pair / p.E, e = pair - t * p.E;
    float2* part = reinterpret_cast<float2*>(sh.part[0][buf]);
    if (pair < pairs) {
      const __nv_bfloat16* a = p.Wr + static_cast<size_t>(e) * p.H;
      const __nv_bfloat16* x = p.X + static_cast<size_t>(t) * p.H;
      uint64_t sums[2] = {0ull, 0ull}, lost[2] = {0ull, 0ull};
#pragma unroll 4
      for (int c = (sub * 32 + lane) * 8; c < p.H; c += w * 256)
        moe_dot8(ld_global_nc_v4(a + c), ld_global_nc_v4(x + c), sums, lost);
      const float2 v = moe_sum(moe_total(sums, lost), 16);
      if (lane == 0) part[warp] = v;
    }
    moe_sync();
    if (pair < pairs && sub == 0) {
      float2 v = moe_sum(lane < w ? part[warp + lane] : make_float2(0.f, 0.f), w / 2);
      if (v.y != v.y) v.y = 0.f;  // an infinite sum's loss reads NaN
      const float l = v.x + v.y;
      if (lane == 0)
        __stcg(p.logits + static_cast<size_t>(t) * p.E + e, make_float2(l, v.y - (l - v.x)));
    }
  }
}

// A key that orders like the float: larger floats have larger keys, NaN the least (1).
__device__ __forceinline__ uint32_t moe_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 as +0
  if (l != l) return 1u;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// A token's choices from its logits, by one warp; kPer experts a lane.  CTA 0 writes ids and
// weights out.
template <int kPer>
__device__ __forceinline__ void moe_choose(const MoeParams& p, MoeShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int t = warp; t < p.T; t += kMoeWarps) {
    float l[kPer];
    uint32_t key[kPer], low[kPer];  // order by the fp32 logit, then by what it leaves out
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 32 + lane;
      const bool in = e < p.E;
      const float2 v = in ? __ldcg(p.logits + static_cast<size_t>(t) * p.E + e)
                          : make_float2(-INFINITY, 0.f);
      l[i] = v.x;
      key[i] = in ? moe_key(v.x) : 0u;
      low[i] = moe_key(v.y);
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
      uint32_t best = 0u, next = 0u;
      int at = 0x7fffffff;
      float val = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (key[i] > best || (key[i] == best && low[i] > next)) {  // a lane's lowest index first
          best = key[i];
          next = low[i];
          at = i * 32 + lane;
          val = l[i];
        }
      const uint32_t all = __reduce_max_sync(0xffffffffu, best);
      if (best != all) next = 0u;
      const uint32_t most = __reduce_max_sync(0xffffffffu, next);
      const int e = __reduce_min_sync(0xffffffffu, next == most ? at : 0x7fffffff);
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
}

// Every CTA routes all tokens itself, then lists the pairs by expert.
__device__ void moe_route(const MoeParams& p, MoeShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (p.E <= 32)
    moe_choose<1>(p, sh);
  else if (p.E <= 64)
    moe_choose<2>(p, sh);
  else if (p.E <= 128)
    moe_choose<4>(p, sh);
  else
    moe_choose<8>(p, sh);
  // tokens of each expert, as a bit mask
  for (int e = threadIdx.x; e < p.E; e += kMoeThreads) sh.mask[e] = 0ull;
  moe_sync();
  for (int i = threadIdx.x; i < p.T * p.K; i += kMoeThreads)
    atomicOr(reinterpret_cast<unsigned long long*>(&sh.mask[sh.ids[i]]), 1ull << (i / p.K));
  moe_sync();
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
  moe_sync();
  for (int i = threadIdx.x; i < p.T * p.K; i += kMoeThreads) {
    const int e = sh.ids[i], t = i / p.K;
    const int s = sh.off[e] + __popcll(sh.mask[e] & ((1ull << t) - 1ull));
    sh.tok[s] = static_cast<uint8_t>(t);
    sh.slot[i] = static_cast<uint16_t>(s);
  }
}

// ------------------------------------------------------------------ the rings
// A group's ring (kTiles 1), or the CTA's (kTiles 4).  A stage: for each tile of 16 rows the
// weights (8 rows by 256, twice), then for each warp of a group 128 bytes (its 64 of K) of up to
// `most` tokens.
template <int kTiles>
struct MoeRing {
  static constexpr uint32_t kWeights = kTiles * kMoeStageW;
  uint32_t base;       // shared-memory address of stage 0
  const uint8_t* ptr;  // the same as a pointer
  uint32_t full, empty;  // its barriers
  uint32_t tokens;       // kTiles 4: of a stage's tokens (full is the weights' alone)
  uint32_t stage_bytes, most;
  int stages;
  __device__ __forceinline__ MoeRing(uint8_t* smem, MoeShared& sh, int group)
      : base(smem_u32(smem + group * kMoeRing)),
        ptr(smem + group * kMoeRing),
        full(smem_u32(sh.full[group])),
        empty(smem_u32(sh.empty[group])),
        tokens(smem_u32(sh.full[kMoeGroups - 1])),
        most(sh.most) {
    stage_bytes = kWeights + most * (kMoeKc * 2);
    stages = min(kMoeMaxStages, static_cast<int>(kTiles * kMoeRing / stage_bytes));
  }
  // Offset in a stage of a lane's slot for the expert's token number t and step i.
  __device__ __forceinline__ uint32_t slot(int i, int t) const {
    return kWeights + ((moe_warp() * 2 + i) * most + t) * 64 + (threadIdx.x & 3) * 16;
  }
};

// Where one side of a ring is.
struct MoePlace {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// The units of fc1 and fc2: expert by expert, `rows` features or output columns each, kTiles
// tiles of weight rows.  Unit u belongs to CTA u mod grid, and there to the groups in turn, or to
// all of them (kTiles 4).
template <int kTiles, bool kFc1>
struct MoeUnits {
  int rows, per, count, kcs, len;  // rows of a unit, units of an expert, of all; stages; K
  __device__ __forceinline__ MoeUnits(const MoeParams& p, const MoeShared& sh) {
    rows = kTiles * (kFc1 && p.gated ? 8 : 16);
    per = ((kFc1 ? p.Fe : p.H) + rows - 1) / rows;
    count = sh.n_active * per;
    len = kFc1 ? p.H : p.Fe;
    kcs = (len + kMoeKc - 1) / kMoeKc;
  }
  static __device__ __forceinline__ int first(int group) {
    return kTiles == 1 ? blockIdx.x + group * gridDim.x : blockIdx.x;
  }
  static __device__ __forceinline__ int step() { return kMoeGroups / kTiles * gridDim.x; }
};

// A wait of many threads: without the clock as long as it is short.
__device__ __forceinline__ bool moe_wait(uint32_t bar, uint32_t parity, const WaitCtx& wc,
                                         uint32_t site) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return wait_bounded(bar, parity, wc, site);
}

// The same for two barriers, asked at once: one after the other, T 64 H 4096 Fe 1792 takes 158 us
// with 16 experts top 4, not 151.
__device__ __forceinline__ bool moe_wait_both(uint32_t a, uint32_t b, uint32_t parity,
                                              const WaitCtx& wc) {
  const bool x = mbar_try_wait(a, parity), y = mbar_try_wait(b, parity);
  if (x && y) return true;
  return moe_wait(a, parity, wc, kSiteMoeFull) && moe_wait(b, parity, wc, kSiteMoeFull);
}

// ------------------------------------------------------------------ the copying threads
// Rows and columns past the matrix read as zeros; rows that belong to another expert, where a
// unit reaches past its own, give outputs that are dropped.
template <int kTiles, bool kFc1>
__device__ __forceinline__ bool moe_fill(const MoeParams& p, const MoeShared& sh,
                                         const MoeRing<kTiles>& ring, const WaitCtx& wc,
                                         const CUtensorMap* m, int group, MoePlace& at,
                                         uint32_t& armed, uint32_t& armed_phase, bool& skip) {
  const MoeUnits<kTiles, kFc1> d(p, sh);
  const bool gated = kFc1 && p.gated;
  for (int u = d.first(group); u < d.count; u += d.step()) {
    const int a = u / d.per, r = (u - a * d.per) * d.rows;
    const int e = sh.active[a];
    const int r0 = (kFc1 ? (gated ? 2 * e : e) * p.Fe : e * p.H) + r;
    const int r1 = r0 + (gated ? p.Fe : 8), tile = gated ? 8 : 16;
    for (int kc = 0; kc < d.kcs; ++kc) {
      if (!moe_wait(ring.empty + 8 * at.stage, at.phase ^ 1u, wc, kSiteMoeEmpty)) return false;
      const uint32_t bar = ring.full + 8 * at.stage;
      const uint32_t dst = ring.base + at.stage * ring.stage_bytes;
      if (skip) {  // fault injection: this stage is never filled
        skip = false;
        at.next(ring.stages);
        continue;
      }
      mbar_arrive_expect_tx(bar, ring.kWeights);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        tma_load_2d(dst + 2 * t * kMoeBox, m, bar, kc * kMoeKc, r0 + t * tile);
        tma_load_2d(dst + (2 * t + 1) * kMoeBox, m, bar, kc * kMoeKc, r1 + t * tile);
      }
      armed |= 1u << at.stage;
      armed_phase = (armed_phase & ~(1u << at.stage)) | (at.phase << at.stage);
      at.next(ring.stages);
    }
  }
  return true;
}

template <int kTiles>
__device__ __forceinline__ void moe_copy_thread(const MoeParams& p, MoeShared& sh,
                                                const MoeRing<kTiles>& ring, const WaitCtx& wc,
                                                const CUtensorMap* m1, const CUtensorMap* m2,
                                                int group) {
  MoePlace at;
  uint32_t armed = 0, armed_phase = 0;
  bool skip = p.fault == 1 && blockIdx.x == 0 && group == 0;
  if (moe_fill<kTiles, true>(p, sh, ring, wc, m1, group, at, armed, armed_phase, skip))
    moe_fill<kTiles, false>(p, sh, ring, wc, m2, group, at, armed, armed_phase, skip);
  // Every copy that was issued has landed, after an expired wait too: these barriers count the
  // copies alone, and a stage is not filled again before all who read it have seen it full.
  for (int s = 0; s < ring.stages; ++s)
    if (armed & (1u << s)) wait_drain(ring.full + 8 * s, (armed_phase >> s) & 1u, wc);
}

// ------------------------------------------------------------------ the multiplying warps
__device__ __forceinline__ void moe_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void moe_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Of 16 bytes, or zeros (src is not read then).
__device__ __forceinline__ void moe_copy16_or_0(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
// Waits for this thread's oldest group of copies when `ahead` (1 to 5) groups are in flight.
__device__ __forceinline__ void moe_wait_oldest(int ahead) {
  if (ahead >= 5)
    asm volatile("cp.async.wait_group 4;" ::: "memory");
  else if (ahead == 4)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (ahead == 3)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (ahead == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A lane's place in step i (0, 1) of a stage: rows lane / 4 and lane / 4 + 8, and 8 of K from
// moe_col() + 32 i.
__device__ __forceinline__ int moe_col() { return moe_warp() * 64 + (threadIdx.x & 3) * 8; }

// A lane's copies of its tokens' fragments -- column lane / 4 of tile j is the expert's token
// number j * 8 + lane / 4 -- one stage after the other, ahead of the products.
template <int NT, bool kFc1>
struct MoeTokens {
  const MoeParams& p;
  const MoeShared& sh;
  const MoeRing<1>& ring;
  const MoeUnits<1, kFc1>& d;
  int u, kc, stage, n;
  const __nv_bfloat16* src;
  int row[NT];  // offsets of the tokens' rows (elements)

  __device__ __forceinline__ MoeTokens(const MoeParams& p_, const MoeShared& sh_,
                                       const MoeRing<1>& ring_, const MoeUnits<1, kFc1>& d_,
                                       int stage_)
      : p(p_), sh(sh_), ring(ring_), d(d_), u(d_.first(moe_group())), kc(0), stage(stage_), n(0) {
    src = (kFc1 ? p.X : p.act) + moe_col();
    open();
  }
  __device__ __forceinline__ void open() {
    if (u >= d.count) return;
    const int e = sh.active[u / d.per], off = sh.off[e], g = (threadIdx.x & 31) >> 2;
    n = __popcll(sh.mask[e]);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int s = off + min(j * 8 + g, n - 1);
      row[j] = kFc1 ? sh.tok[s] * p.H : s * p.Fe;
    }
  }
  __device__ __forceinline__ void issue() {
    if (u < d.count) {
      const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (kc * kMoeKc + moe_col() + i * 32 < d.len) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            if (j * 8 + g < n)
              moe_copy16(ring.base + stage * ring.stage_bytes + ring.slot(i, j * 8 + g),
                         src + row[j] + kc * kMoeKc + i * 32);
        }
      if (++stage == ring.stages) stage = 0;
      if (++kc == d.kcs) {
        kc = 0;
        u += d.step();
        open();
      }
    }
    moe_commit();
  }
};

// Writes a thread's value of a tile (moe_reduce): 16 weight rows from feature or column r0 on,
// the expert's tokens j * 8 to j * 8 + 7.
template <bool kFc1>
__device__ __forceinline__ void moe_result(const MoeParams& p, const MoeShared& sh, int e, int n,
                                           int r0, int j, float v) {
  const int up = moe_thread() & 1, f = (moe_thread() >> 1) & 7;
  const int t = j * 8 + (moe_thread() >> 4);
  const size_t s = sh.off[e] + t;
  if constexpr (kFc1) {
    int feat = r0 + f;
    if (p.gated) {
      const float o = __shfl_xor_sync(0xffffffffu, v, 1);  // the gate's thread gets its up
      v = v * sigmoid_f(v) * o;
    } else {
      float z;
      f2_unpack(gelu_x2(f2_pack(v, v)), v, z);
      feat += 8 * up;
    }
    if (t < n && feat < p.Fe && !(p.gated && up))
      p.act[s * p.Fe + feat] = __float2bfloat16_rn(v);
  } else {
    const int r = r0 + f + 8 * up;
    if (t < n && r < p.H) __stcg(p.pair_y + s * p.H + r, v);
  }
}

// Gives a stage that a warp has read back to those who refill it.  That the reads stand before
// the arrival is not enough: a read of shared memory that was issued may still be under way when
// the warp arrives, and the bulk copies' writes, which go through another proxy, are not ordered
// behind it (with the arrival right after the reads, T 3 H 4096 Fe 8200 took weights of a refill,
// five stages on, in one call of 70 to 500, and T 12 in every call).  So the arrival's address
// takes bits of `sums`, into which the products of everything read have gone, masked by a zero:
// it cannot be issued before the reads have returned.  It costs nothing measurable (a proxy fence
// of every lane instead: T 64 H 5120 Fe 2560 32 experts 423 us against 399).
// A warp that has given up waiting (`dead`) does not arrive: it may not have seen the stage full,
// and a barrier that is armed again before its copies have landed loses count.
template <int NT>
__device__ __forceinline__ void moe_release(uint32_t bar, const float (&sums)[NT][4],
                                            uint32_t zero, bool dead) {
  uint32_t seen = 0u;
#pragma unroll
  for (int j = 0; j < NT; ++j) seen |= __float_as_uint(sums[j][0]);
  __syncwarp();
  if ((threadIdx.x & 31) == 0 && !dead) mbar_arrive(bar + (seen & zero));
}

// fc1 or fc2 with up to NT (1 or 2) tiles of eight of an expert's tokens.  After an expired wait
// (`dead`), a lane waits and arrives no more and works on with what the stages hold: the launch is
// lost and reported, but every barrier that the warps share still meets all of them.
template <int NT, bool kFc1>
__device__ void moe_multiply(const MoeParams& p, MoeShared& sh, const MoeRing<1>& ring,
                             const WaitCtx& wc, MoePlace& at, int& buf, bool& dead) {
  const int g = (threadIdx.x & 31) >> 2;
  const MoeUnits<1, kFc1> d(p, sh);
  MoeTokens<NT, kFc1> tokens(p, sh, ring, d, at.stage);
#pragma unroll 1
  for (int s = 0; s < ring.stages; ++s) tokens.issue();
#pragma unroll 1
  for (int u = d.first(moe_group()); u < d.count; u += d.step()) {
    const int a = u / d.per, e = sh.active[a], r0 = (u - a * d.per) * d.rows;
    const int n = __popcll(sh.mask[e]);
    float c[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
#pragma unroll 1
    for (int kc = 0; kc < d.kcs; ++kc) {
      if (!dead) dead = !moe_wait(ring.full + 8 * at.stage, at.phase, wc, kSiteMoeFull);
      moe_wait_oldest(ring.stages);
      const uint8_t* st = ring.ptr + at.stage * ring.stage_bytes;
      const int left = d.len - kc * kMoeKc - moe_col();
      uint4 l[2], h[2], x[2][NT];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* w = st + g * (kMoeKc * 2) + (moe_col() + i * 32) * 2;
        l[i] = *reinterpret_cast<const uint4*>(w);
        h[i] = *reinterpret_cast<const uint4*>(w + kMoeBox);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          x[i][j] = make_uint4(0, 0, 0, 0);  // past K's end, and past the expert's tokens
          if (j * 8 + g < n && i * 32 < left)
            x[i][j] = *reinterpret_cast<const uint4*>(st + ring.slot(i, j * 8 + g));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (j * 8 < n) {
            moe_mma(c[j], l[i].x, h[i].x, l[i].y, h[i].y, x[i][j].x, x[i][j].y);
            moe_mma(c[j], l[i].z, h[i].z, l[i].w, h[i].w, x[i][j].z, x[i][j].w);
          }
      moe_release(ring.empty + 8 * at.stage, c, p.zero, dead);
      at.next(ring.stages);
      tokens.issue();  // into the slots just read
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 8 >= n) break;
      const float v = moe_reduce(sh, buf, c[j]);
      buf ^= 1;
      moe_result<kFc1>(p, sh, e, n, r0, j, v);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The same for experts with many tokens, by the whole CTA: a unit is four tiles of 16 rows, one
// for each group, and a stage's tokens are there once for all of them.  Of the tokens' tiles of
// eight, group g copies j = g and g + 4, each warp its 64 of K; an asynchronous arrival of every
// thread on a barrier of their own says that they are there.  A stage is filled again one stage
// late, when the slower warps have left it too.
template <bool kFc1>
__device__ void moe_multiply_cta(const MoeParams& p, MoeShared& sh, const MoeRing<4>& ring,
                                 const WaitCtx& wc, MoePlace& at, MoePlace& to, int& buf,
                                 bool& dead) {
  const int g = (threadIdx.x & 31) >> 2;
  const MoeUnits<4, kFc1> d(p, sh);
  const __nv_bfloat16* src = (kFc1 ? p.X : p.act) + moe_col();
  const uint32_t slot = ring.slot(0, g), step = ring.most * 64;
  const uint32_t weights = moe_group() * kMoeStageW + g * (kMoeKc * 2) + moe_col() * 2;
  int cu = d.first(0), ckc = 0, there = 0;  // of the copies: unit, stage in it, tiles (bits)
  const __nv_bfloat16* row[2];
  auto open = [&]() {
    if (cu >= d.count) return;
    const int e = sh.active[cu / d.per], off = sh.off[e], n = __popcll(sh.mask[e]);
    there = 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int t = (moe_group() + 4 * q) * 8 + g, s = off + min(t, n - 1);
      if (t < n) there |= 1 << q;
      row[q] = src + static_cast<size_t>(kFc1 ? sh.tok[s] : s) * d.len;
    }
  };
  auto issue = [&]() {
    if (cu >= d.count) return;
    if (!dead) dead = !moe_wait(ring.empty + 8 * to.stage, to.phase ^ 1u, wc, kSiteMoeEmpty);
    if (dead) return;  // neither copies nor an arrival out of turn
    const uint32_t dst = ring.base + to.stage * ring.stage_bytes + slot + moe_group() * 512;
    const int left = d.len - ckc * kMoeKc - moe_col();
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (there >> q & 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i)  // zeros past K's end
          moe_copy16_or_0(dst + i * step + q * 2048, left > i * 32 ? row[q] + i * 32 : src,
                          left > i * 32);
        row[q] += kMoeKc;
      }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];"
                 ::"r"(ring.tokens + 8 * to.stage)
                 : "memory");
    to.next(ring.stages);
    if (++ckc == d.kcs) {
      ckc = 0;
      cu += d.step();
      open();
    }
  };
  open();
#pragma unroll 1
  for (int s = 0; s < ring.stages - 1; ++s) issue();
#pragma unroll 1
  for (int u = d.first(0); u < d.count; u += d.step()) {
    const int a = u / d.per, e = sh.active[a];
    const int r0 = (u - a * d.per) * d.rows + moe_group() * (d.rows / 4);
    const int n = __popcll(sh.mask[e]);
    // by the number of token tiles, without a branch in a stage
    auto unit = [&](auto tiles) {
      constexpr int NT = decltype(tiles)::value;
      float c[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
#pragma unroll 1
      for (int kc = 0; kc < d.kcs; ++kc) {
        if (!dead)
          dead = !moe_wait_both(ring.full + 8 * at.stage, ring.tokens + 8 * at.stage, at.phase,
                                wc);
        const uint8_t* st = ring.ptr + at.stage * ring.stage_bytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 l = *reinterpret_cast<const uint4*>(st + weights + i * 64);
          const uint4 h = *reinterpret_cast<const uint4*>(st + weights + i * 64 + kMoeBox);
          uint4 x[NT];  // (slots of tokens that the expert does not have: columns that are dropped)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            x[j] = *reinterpret_cast<const uint4*>(st + slot + i * step + j * 512);
#pragma unroll
          for (int j = 0; j < NT; ++j) moe_mma(c[j], l.x, h.x, l.y, h.y, x[j].x, x[j].y);
#pragma unroll
          for (int j = 0; j < NT; ++j) moe_mma(c[j], l.z, h.z, l.w, h.w, x[j].z, x[j].w);
        }
        issue();  // (of an earlier stage; the sums are ready after it)
        moe_release(ring.empty + 8 * at.stage, c, p.zero, dead);
        at.next(ring.stages);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float v = moe_reduce(sh, buf, c[j]);
        buf ^= 1;
        moe_result<kFc1>(p, sh, e, n, r0, j, v);
      }
    };
    switch ((n + 7) >> 3) {
      case 1: unit(std::integral_constant<int, 1>()); break;
      case 2: unit(std::integral_constant<int, 2>()); break;
      case 3: unit(std::integral_constant<int, 3>()); break;
      case 4: unit(std::integral_constant<int, 4>()); break;
      case 5: unit(std::integral_constant<int, 5>()); break;
      case 6: unit(std::integral_constant<int, 6>()); break;
      default: unit(std::integral_constant<int, 8>()); break;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// After a phase: the CTA's results are written, and those of all CTAs.
__device__ __forceinline__ void moe_phase_end(const MoeParams& p, MoeShared& sh, uint32_t barrier) {
  moe_sync();
  if (threadIdx.x == 0) {
    moe_grid_arrive(p);
    moe_grid_wait(p, sh, barrier);
  }
  moe_sync();
}

// fc1 and fc2, by all threads of a CTA.
template <int kTiles>
__device__ __forceinline__ void moe_experts(const MoeParams& p, MoeShared& sh, uint8_t* smem,
                                            const CUtensorMap* m1, const CUtensorMap* m2) {
  constexpr int kRings = kMoeGroups / kTiles;
  const bool multiplies = threadIdx.x < kMoeThreads;
  const int group = multiplies ? moe_group() : (threadIdx.x - kMoeThreads) >> 5;
  const MoeRing<kTiles> ring(smem, sh, kTiles == 1 ? group : 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRings; ++i)
      for (int s = 0; s < ring.stages; ++s) {
        mbar_init(smem_u32(&sh.full[i][s]), 1);  // the copying thread
        mbar_init(smem_u32(&sh.empty[i][s]), kMoeWarps / kRings);
        if (kTiles > 1) mbar_init(ring.tokens + 8 * s, kMoeThreads);
      }
    mbar_fence_init();
  }
  __syncthreads();
  const WaitCtx wc{&sh.abort, &p.sync->err, p.wait_ns};
  if (!multiplies) {
    if ((threadIdx.x & 31) == 0 && group < kRings)
      moe_copy_thread<kTiles>(p, sh, ring, wc, m1, m2, group);
    return;
  }
  MoePlace at;
  int buf = 0;
  bool dead = false;
  if constexpr (kTiles == 1) {
    auto phase = [&](auto fc1) {
      if (sh.most <= 8)
        moe_multiply<1, fc1.value>(p, sh, ring, wc, at, buf, dead);
      else
        moe_multiply<2, fc1.value>(p, sh, ring, wc, at, buf, dead);
    };
    phase(std::true_type());
    moe_phase_end(p, sh, 2);
    phase(std::false_type());
  } else {
    MoePlace to;
    moe_multiply_cta<true>(p, sh, ring, wc, at, to, buf, dead);
    moe_phase_end(p, sh, 2);
    moe_multiply_cta<false>(p, sh, ring, wc, at, to, buf, dead);
  }
  moe_phase_end(p, sh, 3);
}

// Y_t = sum over t's pairs, in the order of its choices, of w y.
__device__ __forceinline__ void moe_combine(const MoeParams& p, const MoeShared& sh) {
  const int per = p.H / 8;
  for (int i = blockIdx.x * kMoeThreads + threadIdx.x; i < p.T * per;
       i += gridDim.x * kMoeThreads) {
    const int t = i / per, c = (i - t * per) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
    for (int k = 0; k < p.K; ++k) {
      const float w = sh.w[t * p.K + k];
      const float4* y = reinterpret_cast<const float4*>(
          p.pair_y + static_cast<size_t>(sh.slot[t * p.K + k]) * p.H + c);
      const float4 a = __ldcg(y), b = __ldcg(y + 1);
      v[0] = fmaf(w, a.x, v[0]); v[1] = fmaf(w, a.y, v[1]);
      v[2] = fmaf(w, a.z, v[2]); v[3] = fmaf(w, a.w, v[3]);
      v[4] = fmaf(w, b.x, v[4]); v[5] = fmaf(w, b.y, v[5]);
      v[6] = fmaf(w, b.z, v[6]); v[7] = fmaf(w, b.w, v[7]);
    }
    st_global_v4(p.Y + static_cast<size_t>(t) * p.H + c,
                 make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
  }
}

__global__ void __launch_bounds__(kMoeBlock, 1)
    moe_kernel(const __grid_constant__ CUtensorMap map_w1,
               const __grid_constant__ CUtensorMap map_w2, const MoeParams p) {
  extern __shared__ __align__(128) uint8_t moe_smem[];
  MoeShared& sh = *reinterpret_cast<MoeShared*>(moe_smem + kMoeGroups * kMoeRing);
  const bool multiplies = threadIdx.x < kMoeThreads;
  if (threadIdx.x == 0) sh.abort = 0u;
  if (multiplies) moe_logits(p, sh);
  __syncthreads();
  if (threadIdx.x == 0) {
    if (p.fault != 2 || blockIdx.x != 0) moe_grid_arrive(p);
    if (!moe_grid_wait(p, sh, 1)) {  // it will not come to the other barriers
      moe_grid_arrive(p);
      moe_grid_arrive(p);
    }
  }
  __syncthreads();
  if (sh.abort == 0u) {
    if (multiplies) moe_route(p, sh);
    __syncthreads();
    if (sh.most < kMoeSharedFrom)
      moe_experts<1>(p, sh, moe_smem, &map_w1, &map_w2);
    else
      moe_experts<4>(p, sh, moe_smem, &map_w1, &map_w2);
    if (multiplies) moe_combine(p, sh);
  }
  // the last CTA out leaves the barriers' word as it found it, after an expired wait too
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
  int faults;  // MLPB_MOE_FAULT_INJECT: launches still to come with one
  MoeSync* sync;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
};

// A row-major bf16 matrix in boxes of 8 rows by 256 columns; what is past its edges reads zero.
static bool moe_map(const mlpb_moe* h, CUtensorMap* m, const void* base, uint64_t rows,
                    uint64_t cols) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * 2};
  const cuuint32_t box[2] = {kMoeKc, kMoeBoxRows}, steps[2] = {1, 1};
  return h->encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                   box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static size_t moe_logits_bytes(const mlpb_moe_config& c) {
  return moe_align(static_cast<size_t>(c.max_tokens) * c.experts * 8);
}

static size_t moe_act_bytes(const mlpb_moe_config& c) {
  return moe_align(static_cast<size_t>(c.max_tokens) * c.topk * c.ffn * 2);
}

extern "C" mlpb_status mlpb_moe_create(const mlpb_moe_config* cfg, mlpb_moe** out) {
  if (cfg == nullptr || out == nullptr) return MLPB_EINVAL;
  *out = nullptr;
  const mlpb_moe_config& c = *cfg;
  if (c.max_tokens < 1 || c.hidden <= 0 || c.ffn <= 0 || c.experts < 1 || c.topk < 1 ||
      c.topk > c.experts)
    return MLPB_EINVAL;
  if (c.act != MLPB_ACT_GELU_TANH && c.act != MLPB_ACT_SWIGLU) return MLPB_EINVAL;
  if ((c.normalize != 0 && c.normalize != 1) || (c.flags & ~MLPB_MOE_FAULT_INJECT) != 0)
    return MLPB_EINVAL;
  if (c.max_tokens > kMoeMaxTokens || c.experts > kMoeMaxExperts || c.topk > kMoeMaxTopk ||
      c.hidden % 8 != 0 || c.ffn % 8 != 0 || c.hidden > (1 << 20) || c.ffn > (1 << 20))
    return MLPB_EUNSUPPORTED;
  mlpb_moe* h = new (std::nothrow) mlpb_moe();
  if (h == nullptr) return MLPB_ENOMEM;
  h->cfg = c;
  h->faults = (c.flags & MLPB_MOE_FAULT_INJECT) != 0 ? 2 : 0;
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
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found{};
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess || fn == nullptr) {
    delete h;
    return MLPB_ECUDA;
  }
  h->encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  if (cudaFuncSetAttribute(moe_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kMoeSmem)) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, moe_kernel, kMoeBlock, kMoeSmem) !=
          cudaSuccess ||
      per_sm < 1 ||
      cudaMalloc(reinterpret_cast<void**>(&h->sync), sizeof(MoeSync)) != cudaSuccess ||
      cudaMemset(h->sync, 0, sizeof(MoeSync)) != cudaSuccess ||
      cudaStreamSynchronize(nullptr) != cudaSuccess) {  // streams that do not wait for it may come
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
  *bytes = moe_logits_bytes(c) + moe_act_bytes(c) +
           moe_align(static_cast<size_t>(c.max_tokens) * c.topk * c.hidden * 4);
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
  for (const void* q :
       {X, Wr, W1, W2, static_cast<const void*>(Y), static_cast<const void*>(workspace)})
    if (q && (reinterpret_cast<uintptr_t>(q) & 15u) != 0) return MLPB_EINVAL;
  if ((reinterpret_cast<uintptr_t>(ids) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(weights) & 3u) != 0)
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
  p.logits = static_cast<float2*>(workspace);
  uint8_t* ws = static_cast<uint8_t*>(workspace) + moe_logits_bytes(c);
  p.act = reinterpret_cast<__nv_bfloat16*>(ws);
  p.pair_y = reinterpret_cast<float*>(ws + moe_act_bytes(c));
  p.T = static_cast<int>(tokens);
  p.H = static_cast<int>(c.hidden);
  p.Fe = static_cast<int>(c.ffn);
  p.E = c.experts;
  p.K = c.topk;
  p.gated = c.act == MLPB_ACT_SWIGLU ? 1 : 0;
  p.normalize = c.normalize;
  p.sync = h->sync;
  p.wait_ns = kDefaultWaitNs;
  if (h->faults > 0) p.fault = 3 - h->faults--;
  CUtensorMap m1, m2;
  const uint64_t f1 = static_cast<uint64_t>(c.ffn) * (p.gated ? 2 : 1);
  if (!moe_map(h, &m1, W1, c.experts * f1, c.hidden) ||
      !moe_map(h, &m2, W2, static_cast<uint64_t>(c.experts) * c.hidden, c.ffn))
    return MLPB_EINVAL;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(h->grid));
  cfg.blockDim = dim3(kMoeBlock);
  cfg.dynamicSmemBytes = kMoeSmem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the grid's barriers need every CTA resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_kernel, m1, m2, p) == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}

extern "C" mlpb_status mlpb_moe_last_device_error(mlpb_moe* h, mlpb_stream_t stream) {
  if (h == nullptr) return MLPB_EINVAL;
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess) return MLPB_ECUDA;
  if (device != h->device) return MLPB_EINVAL;  // `stream` would not be one of the handle's
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, &h->sync->err, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MLPB_ECUDA;
  if (v == 0) return MLPB_OK;
  if (cudaMemsetAsync(&h->sync->err, 0, sizeof(uint32_t), s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MLPB_ECUDA;
  return MLPB_ETIMEOUT;
}
