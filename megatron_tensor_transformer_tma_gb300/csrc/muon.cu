// Orthogonalised updates of weights: handle, workspace, tensor maps, the launches of a call.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "common.cuh"
#include "gemm_params.h"
#include "muon.cuh"
#include "plan.h"

using namespace mlpb;

struct mlpb_muon {
  mlpb_muon_config cfg;
  PlanDevice on;
  int max_clusters;
  bool tall, fault_pending;
  int n, ldx, ldn;
  int small;  // CTAs of a cluster that keeps a matrix in shared memory; 0: tiles of tensor cores
};

namespace {

struct Layout {
  float4* part;
  __half *x0, *x1, *xl, *e, *d;
  float *diag, *beta;
  float4* partial;
  size_t bytes;
};

// The tiles of a product over all matrices.
struct Tiling {
  int narrow, num_pm, num_n, per_matrix, split, units, num_kb;
  size_t partial_bytes() const {
    return split > 1 ? static_cast<size_t>(units) * 256 * (narrow ? 128 : 256) * 4 : 0;
  }
};

// Tiles of 256 or 128 columns, and for the symmetric products ranges of K: what is estimated to
// end first, in the time of a k-block (0.26 us).  That is the same for both widths: a ring of five
// or six stages keeps up with 256 columns and no more, so that narrow tiles pay where they are all
// in the first wave and leave half the epilogue (a box of 64 columns for each of its warps: four
// k-blocks) after the last product.  Ranges cost a launch that adds their sums (15 k-blocks) and
// the sums' way through L2 (0.07 us for 256 KB): 1376 x 4096 280 us with ranges in the first
// product alone, 306 with them in both, 288 with none; 2048 x 2048 260, 296 with them.  (Sums that
// met in distributed shared memory, clusters of up to eight pairs, cost the same 4 to 5 us a
// product as the launch and allow fewer ranges: 182 x 5158 121 us against 108.)
Tiling tiling(const mlpb_muon* h, bool symmetric, int64_t rows, int64_t cols, int64_t depth) {
  const int64_t batch = h->cfg.batch;
  Tiling best{};
  double least = 0.0;
  for (int narrow = 0; narrow < 2; ++narrow) {
    const int bn = narrow ? 128 : 256;
    Tiling t;
    t.narrow = narrow;
    t.num_pm = static_cast<int>(cdiv(rows, 256));
    t.num_n = static_cast<int>(cdiv(cols, bn));
    t.num_kb = static_cast<int>(cdiv(depth, kBK));
    t.per_matrix = t.num_pm * t.num_n;
    if (symmetric) {
      const int r = 256 / bn;  // the last row of tiles may lack some at its end
      t.per_matrix = r * t.num_pm * (t.num_pm + 1) / 2 - (r * t.num_pm - t.num_n);
    }
    const int64_t tiles = batch * t.per_matrix;
    const int boxes = narrow ? 1 : 2;
    for (t.split = 1; t.split <= kOrthoMaxSplit; ++t.split) {
      if (t.split > 1 && (!symmetric || tiles * t.split > h->max_clusters ||
                          t.split > t.num_kb))
        break;
      t.units = static_cast<int>(tiles) * t.split;
      double cost = static_cast<double>(cdiv(t.units, h->max_clusters)) *
                        cdiv(t.num_kb, t.split) +
                    4.0 * boxes;
      if (t.split > 1) cost += 15.0 + 0.27 / (narrow ? 2 : 1) * t.units;
      if (best.split == 0 || cost < least) {
        best = t;
        least = cost;
      }
    }
  }
  return best;
}

Tiling gram_tiling(const mlpb_muon* h) {
  return tiling(h, true, h->n, h->n, std::max(h->cfg.rows, h->cfg.cols));
}
Tiling poly_tiling(const mlpb_muon* h) { return tiling(h, true, h->n, h->n, h->n); }
Tiling apply_tiling(const mlpb_muon* h) {
  return tiling(h, false, h->cfg.rows, h->cfg.cols, h->n);
}

Layout layout(const mlpb_muon* h, void* workspace) {
  const mlpb_muon_config& c = h->cfg;
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = base + at;
    at += align256(bytes);
    return p;
  };
  const size_t x = static_cast<size_t>(c.batch * c.rows) * h->ldx * 2;
  const size_t s = static_cast<size_t>(c.batch) * h->n * h->ldn * 2;
  const size_t v = static_cast<size_t>(c.batch) * h->ldn * 4;
  Layout l;
  l.part = reinterpret_cast<float4*>(
      take(static_cast<size_t>(c.batch) * muon_partials(c.rows * c.cols, c.batch) * 16));
  l.x0 = reinterpret_cast<__half*>(take(x));
  l.x1 = reinterpret_cast<__half*>(take(x));
  l.xl = reinterpret_cast<__half*>(take(x));
  l.e = reinterpret_cast<__half*>(take(s));
  l.d = reinterpret_cast<__half*>(take(s));
  l.diag = reinterpret_cast<float*>(take(v));
  l.beta = reinterpret_cast<float*>(take(v));
  l.partial = reinterpret_cast<float4*>(
      take(std::max(gram_tiling(h).partial_bytes(), poly_tiling(h).partial_bytes())));
  l.bytes = at;
  return l;
}

// Matrices [batch][rows][ld] in boxes of some rows by some columns.
struct Matrices {
  const void* base;
  int64_t rows, cols, ld;
};

bool map_box(const mlpb_muon* h, CUtensorMap* m, const Matrices& x, CUtensorMapDataType type,
             uint64_t size, uint32_t box_cols, uint32_t box_rows, bool swizzled) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(x.cols), static_cast<cuuint64_t>(x.rows),
                              static_cast<cuuint64_t>(h->cfg.batch)};
  const cuuint64_t strides[2] = {x.ld * size, static_cast<cuuint64_t>(x.rows) * x.ld * size};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  return h->on.map(m, type, x.base, 3, dims, strides, box,
                   swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

// As operands whose K runs along a row: `size` (128 or 64) rows by 64 columns.
bool map_k(const mlpb_muon* h, CUtensorMap* m, const Matrices& x, int size) {
  return map_box(h, m, x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, kBK, static_cast<uint32_t>(size),
                 true);
}

// With K along a column: `size` / 64 chunks, 64 wide, of 64 rows.
bool map_mn(const mlpb_muon* h, CUtensorMap* m, const Matrices& x, int size) {
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(x.rows),
                              static_cast<cuuint64_t>(x.ld / 64),
                              static_cast<cuuint64_t>(h->cfg.batch)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(x.ld) * 2, 128,
                                 static_cast<cuuint64_t>(x.rows) * x.ld * 2};
  const cuuint32_t box[4] = {64, kBK, static_cast<cuuint32_t>(size / 64), 1};
  return h->on.map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x.base, 4, dims, strides, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
}

// The epilogue's boxes of 32 rows by 64 columns, and mirrored.
bool map_tile(const mlpb_muon* h, CUtensorMap* m, const Matrices& x) {
  return map_box(h, m, x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, 64, 32, true);
}
bool map_mirror(const mlpb_muon* h, CUtensorMap* m, const Matrices& x) {
  return map_box(h, m, x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, 32, 64, false);
}

// The steps, the last of them into what `p` names.
mlpb_status iterate(mlpb_muon* h, const MuonInput& in, OrthoParams p, void* workspace,
                    cudaStream_t s) {
  const mlpb_muon_config& c = h->cfg;
  p.a = c.coef[0];
  p.b = c.coef[1];
  p.c = c.coef[2];
  p.err = h->on.err;
  if (h->small > 0)
    return launch_muon_small(in, p, c.steps, h->small, s) == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
  const Layout l = layout(h, workspace);
  const Matrices x[2] = {{l.x0, c.rows, c.cols, h->ldx}, {l.x1, c.rows, c.cols, h->ldx}};
  const Matrices low{l.xl, c.rows, c.cols, h->ldx};
  const Matrices e{l.e, h->n, h->n, h->ldn}, d{l.d, h->n, h->n, h->ldn};
  OrthoMaps gram[2], poly, apply[2], last;  // by the buffer that X is in
  const Tiling tg = gram_tiling(h), tp = poly_tiling(h), ta = apply_tiling(h);
  // a CTA's rows of B
  const int bg = tg.narrow ? 64 : 128, bp = tp.narrow ? 64 : 128, ba = ta.narrow ? 64 : 128;
  bool ok = map_k(h, &poly.a, e, 128) && map_k(h, &poly.b, e, bp) && map_tile(h, &poly.in0, e) &&
            map_tile(h, &poly.out0, d) && map_mirror(h, &poly.mirror, d);
  poly.in1 = poly.out1 = poly.a;
  const int buffers = c.steps > 1 ? 2 : 1;
  for (int i = 0; i < buffers && ok; ++i) {
    OrthoMaps& g = gram[i];
    OrthoMaps& y = apply[i];
    ok = (h->tall ? map_mn(h, &g.a, x[i], 128) && map_mn(h, &g.b, x[i], bg)
                  : map_k(h, &g.a, x[i], 128) && map_k(h, &g.b, x[i], bg)) &&
         map_tile(h, &g.out0, e) && map_mirror(h, &g.mirror, e);
    g.in0 = g.in1 = g.out1 = g.a;
    ok = ok && (h->tall ? map_k(h, &y.a, x[i], 128) && map_k(h, &y.b, d, ba)
                        : map_k(h, &y.a, d, 128) && map_mn(h, &y.b, x[i], ba)) &&
         map_tile(h, &y.in0, x[i]) && map_tile(h, &y.in1, low) && map_tile(h, &y.out0, x[1 - i]);
    y.out1 = y.mirror = y.in1;
  }
  last = apply[(c.steps - 1) & 1];
  p.ragged = c.cols % 8 != 0 ? 1 : 0;
  if (ok && !p.ragged) {
    if (p.w != nullptr)
      ok = map_box(h, &last.in1, {p.w, c.rows, c.cols, c.cols}, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
                   32, 32, true);
    const void* half = p.w != nullptr ? p.wb : p.out;
    if (ok && half != nullptr)
      ok = map_box(h, &last.out0, {half, c.rows, c.cols, c.cols}, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   2, 64, 32, true);
  }
  if (!ok || launch_muon_norm(in, l.part, s) != cudaSuccess ||
      launch_muon_split(in, l.part, l.x0, l.x1, l.xl, h->ldx, s) != cudaSuccess)
    return MLPB_ECUDA;
  p.batch = static_cast<int>(c.batch);
  p.rows = static_cast<int>(c.rows);
  p.cols = static_cast<int>(c.cols);
  p.n = h->n;
  p.ldn = h->ldn;
  p.diag = l.diag;
  p.beta = l.beta;
  p.wait_ns = kDefaultWaitNs;
  p.fault_inject = h->fault_pending ? 1 : 0;
  h->fault_pending = false;
  p.partial = l.partial;
  p.e = l.e;
  p.d = l.d;
  auto run = [&](OrthoOp op, const Tiling& t, const OrthoMaps& maps) {
    p.narrow = t.narrow;
    p.num_pm = t.num_pm;
    p.num_n = t.num_n;
    p.per_matrix = t.per_matrix;
    p.split = t.split;
    p.units = t.units;
    p.num_kb = t.num_kb;
    const cudaError_t err =
        launch_ortho(op, h->tall, maps, p, std::min(t.units, h->max_clusters), s);
    p.fault_inject = 0;
    return err == cudaSuccess;
  };
  for (int i = 0; i < c.steps; ++i) {
    p.low_out = i < c.steps - 2 ? 1 : 0;
    p.low_beta = i >= c.steps - 3 ? 1 : 0;
    if (!run(OrthoOp::Gram, tg, gram[i & 1]) || !run(OrthoOp::Poly, tp, poly) ||
        !(i == c.steps - 1 ? run(OrthoOp::Last, ta, last) : run(OrthoOp::Apply, ta, apply[i & 1])))
      return MLPB_ECUDA;
  }
  return MLPB_OK;
}

// Whether singular values that start in [0, 1] stay below 2, where the fp16 formats' fixed scales
// hold every operand (b A + c A A below 60).
bool coefficients_fit(const mlpb_muon_config& c) {
  for (int i = 0; i <= 4096; ++i) {
    double s = i / 4096.0;
    for (int k = 0; k < c.steps; ++k) {
      const double q = s * s;
      if (std::fabs(c.coef[1]) * q + std::fabs(c.coef[2]) * q * q > 60.0) return false;
      s = std::fabs(s * (c.coef[0] + q * (c.coef[1] + c.coef[2] * q)));
      if (!(s < 2.0)) return false;
    }
  }
  return true;
}

}  // namespace

extern "C" mlpb_status mlpb_muon_create(const mlpb_muon_config* cfg, mlpb_muon** out) {
  if (cfg == nullptr || out == nullptr) return MLPB_EINVAL;
  *out = nullptr;
  const mlpb_muon_config& c = *cfg;
  if (c.batch < 1 || c.rows < 1 || c.cols < 1 || c.steps < 1 ||
      (c.nesterov != 0 && c.nesterov != 1) || (c.flags & ~MLPB_MUON_FAULT_INJECT) != 0)
    return MLPB_EINVAL;
  for (float f : {c.coef[0], c.coef[1], c.coef[2], c.weight_decay, c.scale})
    if (!std::isfinite(f)) return MLPB_EINVAL;
  if (!(c.momentum >= 0.0f && c.momentum < 1.0f)) return MLPB_EINVAL;
  if (c.batch > 65535 || c.rows > 65536 || c.cols > 65536 || c.steps > 64 ||
      c.batch * cdiv(c.rows, 256) * cdiv(c.cols, 256) > (int64_t{1} << 29) || !coefficients_fit(c))
    return MLPB_EUNSUPPORTED;
  mlpb_muon* h = new (std::nothrow) mlpb_muon();
  if (h == nullptr) return MLPB_ENOMEM;
  h->cfg = c;
  h->tall = c.rows > c.cols;
  h->n = static_cast<int>(std::min(c.rows, c.cols));
  h->ldx = static_cast<int>(cdiv(c.cols, kOrthoLd)) * kOrthoLd;
  h->ldn = static_cast<int>(cdiv(h->n, kOrthoLd)) * kOrthoLd;
  h->fault_pending = (c.flags & MLPB_MUON_FAULT_INJECT) != 0;
  mlpb_status st = h->on.find();
  if (st == MLPB_OK &&
      (muon_small_cluster(h->n, std::max(c.rows, c.cols), c.batch, h->tall, c.steps, &h->small) !=
           cudaSuccess ||
       ortho_set_attrs(&h->max_clusters) != cudaSuccess || h->max_clusters < 1))
    st = MLPB_ECUDA;
  if (st == MLPB_OK) st = h->on.allocate();
  if (st != MLPB_OK) {
    delete h;
    return st;
  }
  *out = h;
  return MLPB_OK;
}

extern "C" void mlpb_muon_destroy(mlpb_muon* h) {
  if (h == nullptr) return;
  h->on.release();
  delete h;
}

extern "C" mlpb_status mlpb_muon_workspace_size(const mlpb_muon* h, size_t* bytes) {
  if (h == nullptr || bytes == nullptr) return MLPB_EINVAL;
  *bytes = h->small > 0 ? 256 : layout(h, nullptr).bytes;
  return MLPB_OK;
}

extern "C" mlpb_status mlpb_muon_orthogonalize(mlpb_muon* h, const void* U, int32_t u_f32, void* O,
                                               void* workspace, mlpb_stream_t stream) {
  if (h == nullptr || !U || !O || !workspace || (u_f32 != 0 && u_f32 != 1)) return MLPB_EINVAL;
  for (const void* q : {U, static_cast<const void*>(O), static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MLPB_EINVAL;
  const mlpb_status st = h->on.current();
  if (st != MLPB_OK) return st;
  MuonInput in{};
  in.g = U;
  in.g_f32 = u_f32;
  in.batch = h->cfg.batch;
  in.rows = h->cfg.rows;
  in.cols = h->cfg.cols;
  OrthoParams p{};
  p.out = static_cast<__nv_bfloat16*>(O);
  return iterate(h, in, p, workspace, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" mlpb_status mlpb_muon_step(mlpb_muon* h, const float* G, float* M, float* W, void* Wb,
                                      const float* lr, void* workspace, mlpb_stream_t stream) {
  if (h == nullptr || !G || !M || !W || !lr || !workspace) return MLPB_EINVAL;
  for (const void* q : {static_cast<const void*>(G), static_cast<const void*>(M),
                        static_cast<const void*>(W), static_cast<const void*>(Wb),
                        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MLPB_EINVAL;
  if ((reinterpret_cast<uintptr_t>(lr) & 3u) != 0) return MLPB_EINVAL;
  const mlpb_status st = h->on.current();
  if (st != MLPB_OK) return st;
  const mlpb_muon_config& c = h->cfg;
  MuonInput in{};
  in.g = G;
  in.m = M;
  in.g_f32 = 1;
  in.nesterov = c.nesterov;
  in.momentum = c.momentum;
  in.batch = c.batch;
  in.rows = c.rows;
  in.cols = c.cols;
  OrthoParams p{};
  p.w = W;
  p.wb = static_cast<__nv_bfloat16*>(Wb);
  p.lr = lr;
  p.decay = c.weight_decay;
  p.scale = c.scale;
  return iterate(h, in, p, workspace, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" mlpb_status mlpb_muon_last_device_error(mlpb_muon* h, mlpb_stream_t stream) {
  if (h == nullptr) return MLPB_EINVAL;
  return h->on.last_error(reinterpret_cast<cudaStream_t>(stream));
}
