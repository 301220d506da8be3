// C entry points of the join between two blocks: validation, launch plans, and the second
// pass of the parameters' gradients.
#include "../../include/mlpb.h"
#include "join.cuh"

namespace mlpb {

// One sum of partial rows: out[c] = sum_k part[k][c] over np rows, += with accumulate.
struct JoinSum {
  const float* part;
  float* out;
  int np;
};

struct JoinSums {
  JoinSum s[4];  // dgamma_post, dbeta_post, dgamma_pre, dbeta_pre (those wanted)
  int n;
  const float* part_gate;  // [groups][per_group][H] partial rows of dgate, NULL: none
  float* dgate;
  int groups, per_group;
  const float* part_alpha;  // [np_alpha]
  float* dalpha;
  int np_alpha;
  int H, accumulate;
};

// The second pass: block (x, y) sums 32 columns of sum y (then of the groups' dgate rows): warp
// w takes partial rows w, w + 16, ..., and the warps' sums are added in warp order.  The last
// block in x of row 0 adds dalpha up, in 64 bits.  Bound by latency: 15 MB from L2 in 7 us at
// T 8192 H 8192, eight loads in flight a thread (with eight warps and four loads 9).  Launched
// while the first pass ends, it gains 1 us of 150: not kept.
constexpr int kJoinSumWarps = 16;
__global__ void __launch_bounds__(32 * kJoinSumWarps) join_sums_kernel(const JoinSums p) {
  __shared__ float red[kJoinSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0 && p.dalpha != nullptr && warp == 0) {
      double t = 0.0;
      for (int i = lane; i < p.np_alpha; i += 32) t += static_cast<double>(p.part_alpha[i]);
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane == 0) *p.dalpha = static_cast<float>(p.accumulate ? *p.dalpha + t : t);
    }
    return;
  }
  const int y = blockIdx.y;
  const int64_t H = p.H;
  JoinSum q;
  if (y < p.n) {
    q = p.s[y];
  } else {
    const int g = y - p.n;
    q.part = p.part_gate + static_cast<int64_t>(g) * p.per_group * H;
    q.out = p.dgate + g * H;
    q.np = p.per_group;
  }
  const int c = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (c < p.H) {
    const float* from = q.part + c;
#pragma unroll 1
    for (int k = warp; k < q.np; k += 8 * kJoinSumWarps) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = k + i * kJoinSumWarps;
        v[i] = r < q.np ? from[r * H] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) t += v[i];
    }
  }
  red[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && c < p.H) {
    t = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinSumWarps; ++w) t += red[w][lane];
    q.out[c] = p.accumulate ? q.out[c] + t : t;
  }
}

struct JoinPlan {
  bool plain, split;
  JoinShape shape;
  int grid, blocks_per_group, parts;  // partial rows
  size_t o_gate, o_gpost, o_bpost, o_gpre, o_bpre, o_alpha, bytes;
};

static size_t join_align(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The backward's CTAs (as many as run at once) and its partial rows in the workspace.  Where a
// CTA holds several rows and groups are many and short, its rows walk groups of their own (a gate
// for each token at T 16384 H 512: 59 us, against 329 with one row of the CTA busy; H 1024 101
// against 176); the plain instantiations leave that to the general ones.
static JoinPlan join_plan(const mlpb_join_config& c, bool plain, int num_sms) {
  JoinPlan q{};
  const int64_t groups = std::max<int64_t>(1, c.gate_groups);
  const int64_t per = c.tokens / groups;  // rows of a group
  auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  q.plain = plain;
  for (;;) {
    q.shape = join_bwd_shape(c.hidden, q.plain, ceil_div(c.tokens, num_sms));
    const int rows = q.shape.rows;
    const int target = q.plain ? num_sms * (512 / q.shape.threads) : num_sms / q.shape.cluster;
    const int64_t want = std::max<int64_t>(1, ceil_div(per, rows));
    q.blocks_per_group =
        static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, target / groups)));
    q.grid = static_cast<int>(q.blocks_per_group > 1 ? groups * q.blocks_per_group
                                                     : std::min<int64_t>(groups, target));
    q.parts = q.grid;
    // turns of a walker: a CTA, or each of its rows
    q.split = q.blocks_per_group == 1 && rows > 1 &&
              ceil_div(groups, int64_t(target) * rows) * per < ceil_div(groups, target) * want;
    if (!q.split) break;
    if (q.plain) {
      q.plain = false;
      continue;
    }
    q.grid = static_cast<int>(std::min<int64_t>(ceil_div(groups, rows), target));
    q.parts = static_cast<int>(std::min<int64_t>(groups, int64_t(q.grid) * rows));
    break;
  }
  // (a row for every walker, those without a group too)
  const size_t row = static_cast<size_t>(q.grid) * (q.split ? q.shape.rows : 1) * c.hidden * 4;
  size_t o = 0;
  auto take = [&o](size_t n) {
    const size_t at = o;
    o += join_align(n);
    return at;
  };
  q.o_gate = take(c.gate_groups > 0 && q.blocks_per_group > 1 ? row : 0);
  q.o_gpost = take(c.post_norm != MLPB_NORM_NONE ? row : 0);
  q.o_bpost = take(c.post_norm == MLPB_NORM_LAYER ? row : 0);
  q.o_gpre = take(c.pre_norm != MLPB_NORM_NONE ? row : 0);
  q.o_bpre = take(c.pre_norm == MLPB_NORM_LAYER ? row : 0);
  q.o_alpha = take(static_cast<size_t>(q.grid * q.shape.cluster) * 4);
  q.bytes = std::max<size_t>(o, 256);
  return q;
}

static mlpb_status join_check(const mlpb_join_config* c) {
  if (c == nullptr) return MLPB_EINVAL;
  if (c->tokens < 0 || c->hidden <= 0 || c->gate_groups < 0) return MLPB_EINVAL;
  if (c->has_block != 0 && c->has_block != 1) return MLPB_EINVAL;
  for (int32_t k : {c->post_norm, c->pre_norm})
    if (k != MLPB_NORM_NONE && k != MLPB_NORM_LAYER && k != MLPB_NORM_RMS) return MLPB_EINVAL;
  if ((c->flags & ~(MLPB_JOIN_STREAM_F32 | MLPB_JOIN_BLOCK_F32 | MLPB_JOIN_ACCUMULATE_GRADS)) != 0)
    return MLPB_EINVAL;
  if ((c->post_norm != MLPB_NORM_NONE || c->pre_norm != MLPB_NORM_NONE) &&
      !(c->eps > 0.f && c->eps < 1e30f))
    return MLPB_EINVAL;
  if (!c->has_block && (c->post_norm != MLPB_NORM_NONE || c->gate_groups != 0 ||
                        c->pre_norm == MLPB_NORM_NONE))
    return MLPB_EINVAL;
  if (c->hidden % 8 != 0 || c->hidden > 16384 || c->tokens > 0x7fffffffll)
    return MLPB_EUNSUPPORTED;
  if (c->gate_groups > 0 && (c->tokens % c->gate_groups != 0 || c->gate_groups > c->tokens) &&
      c->tokens > 0)
    return MLPB_EUNSUPPORTED;
  if (c->gate_groups > 0x7fffffffll) return MLPB_EUNSUPPORTED;
  return MLPB_OK;
}

static bool join_sms(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

static JoinParams join_base(const mlpb_join_config& c) {
  JoinParams p{};
  p.T = c.tokens;
  p.H = static_cast<int>(c.hidden);
  p.G = static_cast<int>(c.gate_groups);
  p.rows_per_group = c.tokens / std::max<int64_t>(1, c.gate_groups);
  p.post = c.post_norm;
  p.pre = c.pre_norm;
  p.has_block = c.has_block != 0;
  p.eps = c.eps;
  return p;
}

static bool join_misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return true;
  return false;
}

// A pointer that the configuration asks for is there, and one that it does not is not.
static bool join_present(bool wanted, const void* p) { return wanted == (p != nullptr); }

}  // namespace mlpb

using namespace mlpb;

extern "C" mlpb_status mlpb_join_workspace_size(const mlpb_join_config* cfg, size_t* bytes) {
  const mlpb_status st = join_check(cfg);
  if (st != MLPB_OK) return st;
  if (bytes == nullptr) return MLPB_EINVAL;
  int sms = 0;
  if (!join_sms(&sms)) return MLPB_ECUDA;
  *bytes = join_plan(*cfg, false, sms).bytes;
  if (join_bwd_has_plain(cfg->hidden)) *bytes = std::max(*bytes, join_plan(*cfg, true, sms).bytes);
  return MLPB_OK;
}

extern "C" mlpb_status mlpb_join_fwd(const mlpb_join_config* cfg, const void* X, const void* Y,
                                     const float* res_scale, const void* gate,
                                     const void* gamma_post, const void* beta_post,
                                     const void* gamma_pre, const void* beta_pre, void* Xout,
                                     void* Xn, float* stats, mlpb_stream_t stream) {
  const mlpb_status st = join_check(cfg);
  if (st != MLPB_OK) return st;
  const mlpb_join_config& c = *cfg;
  const bool rows = c.tokens > 0, pre = c.pre_norm != MLPB_NORM_NONE;
  if (!join_present(c.post_norm != MLPB_NORM_NONE, gamma_post) ||
      !join_present(c.post_norm == MLPB_NORM_LAYER, beta_post) || !join_present(pre, gamma_pre) ||
      !join_present(c.pre_norm == MLPB_NORM_LAYER, beta_pre))
    return MLPB_EINVAL;
  if (!c.has_block && (Y || Xout || res_scale)) return MLPB_EINVAL;
  if (!join_present(c.gate_groups > 0, gate) && !(c.gate_groups > 0 && !rows)) return MLPB_EINVAL;
  if (rows && (!X || !stats || (c.has_block && (!Y || !Xout)) || pre != (Xn != nullptr)))
    return MLPB_EINVAL;
  if (join_misaligned({X, Y, gate, gamma_post, beta_post, gamma_pre, beta_pre, Xout, Xn, stats}) ||
      (reinterpret_cast<uintptr_t>(res_scale) & 3u) != 0)
    return MLPB_EINVAL;
  if (!rows) return MLPB_OK;
  int sms = 0;
  if (!join_sms(&sms)) return MLPB_ECUDA;
  using bf = __nv_bfloat16;
  JoinParams p = join_base(c);
  p.X = X;
  p.Y = Y;
  p.alpha = res_scale;
  p.gate = static_cast<const bf*>(gate);
  p.gamma_post = static_cast<const bf*>(gamma_post);
  p.beta_post = static_cast<const bf*>(beta_post);
  p.gamma_pre = static_cast<const bf*>(gamma_pre);
  p.beta_pre = static_cast<const bf*>(beta_pre);
  p.Xout = Xout;
  p.Xn = static_cast<bf*>(Xn);
  p.stats = stats;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool y32 = (c.flags & MLPB_JOIN_BLOCK_F32) != 0;
  const cudaError_t e = (c.flags & MLPB_JOIN_STREAM_F32) != 0
                            ? (y32 ? join_fwd_run<float, float>(p, sms, s)
                                   : join_fwd_run<float, bf>(p, sms, s))
                            : (y32 ? join_fwd_run<bf, float>(p, sms, s)
                                   : join_fwd_run<bf, bf>(p, sms, s));
  return e == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}

extern "C" mlpb_status mlpb_join_bwd(const mlpb_join_config* cfg, const void* X, const void* Y,
                                     const void* Xout, const float* stats, const float* res_scale,
                                     const void* gate, const void* gamma_post,
                                     const void* beta_post, const void* gamma_pre,
                                     const void* dXout, const void* dXn, void* dX, void* dY,
                                     float* dres_scale, float* dgate, float* dgamma_post,
                                     float* dbeta_post, float* dgamma_pre, float* dbeta_pre,
                                     void* workspace, mlpb_stream_t stream) {
  const mlpb_status st = join_check(cfg);
  if (st != MLPB_OK) return st;
  const mlpb_join_config& c = *cfg;
  const bool rows = c.tokens > 0, pre = c.pre_norm != MLPB_NORM_NONE;
  const bool post = c.post_norm != MLPB_NORM_NONE;
  const bool post_ln = c.post_norm == MLPB_NORM_LAYER, pre_ln = c.pre_norm == MLPB_NORM_LAYER;
  if (!join_present(post, gamma_post) || !join_present(post_ln, beta_post) ||
      !join_present(pre, gamma_pre) || !join_present(post, dgamma_post) ||
      !join_present(post_ln, dbeta_post) || !join_present(pre, dgamma_pre) ||
      !join_present(pre_ln, dbeta_pre))
    return MLPB_EINVAL;
  if (!c.has_block && (Y || X || dY || res_scale)) return MLPB_EINVAL;
  if (rows && (join_present(c.gate_groups > 0, gate) == false ||
               join_present(c.gate_groups > 0, dgate) == false))
    return MLPB_EINVAL;
  if (!join_present(res_scale != nullptr, dres_scale)) return MLPB_EINVAL;
  const bool need_y = post || c.gate_groups > 0;
  if (rows && (!dX || !stats || !workspace || (c.has_block && !dY) || (need_y && !Y) ||
               (pre && (!Xout || !dXn)) || (!pre && (dXn || !dXout)) || (res_scale && !X)))
    return MLPB_EINVAL;
  if (join_misaligned({X, Y, Xout, stats, gate, gamma_post, beta_post, gamma_pre, dXout, dXn, dX,
                       dY, dgate, dgamma_post, dbeta_post, dgamma_pre, dbeta_pre, workspace}) ||
      (reinterpret_cast<uintptr_t>(res_scale) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(dres_scale) & 3u) != 0)
    return MLPB_EINVAL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool acc = (c.flags & MLPB_JOIN_ACCUMULATE_GRADS) != 0;
  if (!rows) {  // no rows: zero parameter gradients (adds nothing when accumulating)
    if (acc) return MLPB_OK;
    cudaError_t e = cudaSuccess;
    for (float* q : {dgamma_post, dbeta_post, dgamma_pre, dbeta_pre})
      if (e == cudaSuccess && q) e = launch_fill_zero(q, static_cast<size_t>(c.hidden) * 4, s);
    if (e == cudaSuccess && dgate)
      e = launch_fill_zero(dgate, static_cast<size_t>(c.gate_groups * c.hidden) * 4, s);
    if (e == cudaSuccess && dres_scale) e = cudaMemsetAsync(dres_scale, 0, 4, s);
    return e == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
  }
  int sms = 0;
  if (!join_sms(&sms)) return MLPB_ECUDA;
  using bf = __nv_bfloat16;
  const bool plain = pre && post && dXout != nullptr && join_bwd_has_plain(c.hidden);
  const JoinPlan q = join_plan(c, plain, sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto part = [&](bool on, size_t o) { return on ? reinterpret_cast<float*>(ws + o) : nullptr; };
  JoinParams p = join_base(c);
  p.X = X;
  p.Y = Y;
  p.Xout = const_cast<void*>(Xout);
  p.stats = const_cast<float*>(stats);
  p.alpha = res_scale;
  p.gate = static_cast<const bf*>(gate);
  p.gamma_post = static_cast<const bf*>(gamma_post);
  p.beta_post = static_cast<const bf*>(beta_post);
  p.gamma_pre = static_cast<const bf*>(gamma_pre);
  p.dXout = dXout;
  p.dXn = dXn;
  p.dX = dX;
  p.dY = static_cast<bf*>(dY);
  p.dgate = dgate;
  p.blocks_per_group = q.blocks_per_group;
  p.split = q.split;
  p.accumulate = acc ? 1 : 0;
  p.part_gate = part(c.gate_groups > 0 && q.blocks_per_group > 1, q.o_gate);
  p.part_gpost = part(post, q.o_gpost);
  p.part_bpost = part(post_ln, q.o_bpost);
  p.part_gpre = part(pre, q.o_gpre);
  p.part_bpre = part(pre_ln, q.o_bpre);
  p.part_alpha = part(res_scale != nullptr, q.o_alpha);
  const bool y32 = (c.flags & MLPB_JOIN_BLOCK_F32) != 0;
  cudaError_t e = (c.flags & MLPB_JOIN_STREAM_F32) != 0
                      ? (y32 ? join_bwd_run<float, float>(p, q.shape, q.plain, q.grid, s)
                             : join_bwd_run<float, bf>(p, q.shape, q.plain, q.grid, s))
                      : (y32 ? join_bwd_run<bf, float>(p, q.shape, q.plain, q.grid, s)
                             : join_bwd_run<bf, bf>(p, q.shape, q.plain, q.grid, s));
  if (e != cudaSuccess) return MLPB_ECUDA;
  JoinSums r{};
  auto want = [&](const float* from, float* to) {
    if (from != nullptr) r.s[r.n++] = JoinSum{from, to, q.parts};
  };
  want(p.part_gpost, dgamma_post);
  want(p.part_bpost, dbeta_post);
  want(p.part_gpre, dgamma_pre);
  want(p.part_bpre, dbeta_pre);
  r.part_gate = p.part_gate;
  r.dgate = dgate;
  r.groups = p.part_gate != nullptr ? p.G : 0;
  r.per_group = q.blocks_per_group;
  r.part_alpha = p.part_alpha;
  r.dalpha = dres_scale;
  r.np_alpha = q.grid * q.shape.cluster;
  r.H = p.H;
  r.accumulate = p.accumulate;
  if (r.n + r.groups == 0 && r.dalpha == nullptr) return MLPB_OK;
  const dim3 grid = r.n + r.groups == 0  // dalpha alone: only the last block of the row
                        ? dim3(1)
                        : dim3(static_cast<unsigned>((p.H + 31) / 32 + 1),
                               static_cast<unsigned>(r.n + r.groups));
  join_sums_kernel<<<grid, 32 * kJoinSumWarps, 0, s>>>(r);
  return cudaGetLastError() == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}
