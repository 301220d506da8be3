// A linear layer on block-scaled E4M3 operands: handle, workspace, tensor maps, launches.
#include <algorithm>
#include <new>

#include "common.cuh"
#include "linear8.cuh"
#include "plan.h"

using namespace mlpb;

struct mlpb_linear8 {
  mlpb_linear8_config cfg;
  PlanDevice on;
  int max_clusters;
  int few_slots[kFewSlots];
  bool fault_pending;
};

namespace {

size_t code_bytes(int64_t rows, int64_t cols) {
  return align256(static_cast<size_t>(rows * b128_ld(cols)));
}

size_t scale_bytes(int64_t rows, int64_t cols) {
  return static_cast<size_t>(b128_scale_bytes(rows, cols));
}

// A quantized matrix: codes [rows][ld] and scales.
struct Quantized {
  uint8_t *codes, *scales;
  int64_t rows, cols;
};

Quantized quantized(const void* codes, const void* scales, int64_t rows, int64_t cols) {
  return Quantized{static_cast<uint8_t*>(const_cast<void*>(codes)),
                   static_cast<uint8_t*>(const_cast<void*>(scales)), rows, cols};
}

// The next one of the workspace.
Quantized take(uint8_t*& at, int64_t rows, int64_t cols) {
  Quantized q{at, at + code_bytes(rows, cols), rows, cols};
  at += code_bytes(rows, cols) + scale_bytes(rows, cols);
  return q;
}

bool encode(const mlpb_linear8* h, CUtensorMap* m, CUtensorMapDataType type, const void* base,
            uint64_t inner, uint64_t outer, uint64_t stride, uint32_t box_inner,
            uint32_t box_outer, CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[2] = {inner, outer}, strides[1] = {stride};
  const cuuint32_t box[2] = {box_inner, box_outer};
  return h->on.map(m, type, base, 2, dims, strides, box, swizzle);
}

// Codes in tiles of `rows` (128) rows by 128 bytes; what is past the edges reads zero.
bool map_codes(const mlpb_linear8* h, CUtensorMap* m, const Quantized& q, int rows) {
  const uint64_t ld = static_cast<uint64_t>(b128_ld(q.cols));
  return encode(h, m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.codes, ld, static_cast<uint64_t>(q.rows), ld,
                kB128, static_cast<uint32_t>(rows), CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scales as rows of 512 bytes: group of four blocks by group, 128-row tile by tile.
bool map_scales(const mlpb_linear8* h, CUtensorMap* m, const Quantized& q) {
  return encode(h, m, CU_TENSOR_MAP_DATA_TYPE_UINT32, q.scales, kB128Chunk / 4,
                static_cast<uint64_t>(b128_scale_bytes(q.rows, q.cols) / kB128Chunk), kB128Chunk,
                kB128Chunk / 4, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Whether a product goes to the kernel for few tiles.  It does
//   - with at most 128 rows of C, where the bytes of B are all that counts;
//   - where its own tiles (128 of B's rows by at most 128 of A's) are few enough for K to be cut
//     into ranges, so that SMs work that would have no tile of a pair: the more k-blocks, the more
//     it gains (forward of 256 x 1024 with its quantization 6.8 against 7.2 us at 4 k-blocks,
//     10.7 / 15.2 at 24, 18.1 / 33.3 at 86; 512 x 2048 27.4 / 35.1 at 86);
//   - with no more tiles of 256 x 256 than pairs of SMs, up to 32 k-blocks: it starts and ends
//     sooner (a tile of 128 x 128 and one CTA, in place of a pair's), and a k-block costs it more,
//     half the bytes for a quarter of the products.  Between 12 and 40 k-blocks it is 11 % ahead to
//     7 % behind, mostly within 5 (512 x 4096 7.1 / 8.0 at 4, 13.0 / 12.7 at 16, 22.2 / 21.8 at 40,
//     41.0 / 35.8 at 86; 1024 x 4096 10.5 / 11.8 at 8, 18.9 / 18.9 at 24, 28.5 / 26.5 at 48;
//     512 x 5120 18.4 / 18.8 at 28, 29.3 / 28.5 at 56).
// Not where C is added to, which the other kernel does in memory (2048 x 2048 at 8 19.2 against
// 14.9), nor where an fp32 sum is long enough for chunks, which this one does not have.
bool few_tiles(const mlpb_linear8* h, int64_t m, int64_t n, int64_t k, bool f32, bool accumulate) {
  const int64_t blocks = b128_blocks(k);
  if (accumulate || blocks > b128_chunk(f32)) return false;
  if (m <= 128) return true;
  const int64_t tiles = cdiv(m, 128) * cdiv(n, 128), pairs = cdiv(m, 256) * cdiv(n, 256);
  return tiles <= h->few_slots[1] || (pairs <= h->max_clusters && blocks <= 32);
}

// C [a.rows][b.rows] (+)= A B^T over the columns that both have.
mlpb_status product(mlpb_linear8* h, const Quantized& a, const Quantized& b, void* C, bool f32,
                    bool accumulate, cudaStream_t s) {
  B128Maps m{};
  const bool few = few_tiles(h, a.rows, b.rows, a.cols, f32, accumulate);
  if (!map_codes(h, &m.a, a, few ? b128_few_columns(a.rows) : kB128) ||
      !map_codes(h, &m.b, b, kB128) || !map_scales(h, &m.sa, a) ||
      !map_scales(h, &m.sb, b))
    return MLPB_ECUDA;
  if (!few && b128_staged(static_cast<int>(b128_blocks(a.cols)), accumulate) &&
      !encode(h, &m.c,
              f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, C,
              static_cast<uint64_t>(b.rows), static_cast<uint64_t>(a.rows),
              static_cast<uint64_t>(b.rows) * (f32 ? 4 : 2), f32 ? 32 : 64, 32,
              CU_TENSOR_MAP_SWIZZLE_128B))
    return MLPB_ECUDA;
  B128Params p{};
  p.M = static_cast<int>(a.rows);
  p.N = static_cast<int>(b.rows);
  p.num_pm = static_cast<int>(cdiv(a.rows, 256));
  p.num_n = static_cast<int>(cdiv(b.rows, 256));
  p.num_kb = static_cast<int>(b128_blocks(a.cols));
  p.a_tiles = static_cast<int>(b128_blocks(a.rows));
  p.b_tiles = static_cast<int>(b128_blocks(b.rows));
  p.out_f32 = f32 ? 1 : 0;
  p.accumulate = accumulate ? 1 : 0;
  p.chunk = b128_chunk(f32);
  // as the short-K products of the block: larger groups of tiles keep more of A in L2 (2 % at 40
  // k-blocks; none or a loss from 64 on)
  p.raster_group = p.num_kb <= 48 ? 16 : 8;
  p.C = C;
  p.err = h->on.err;
  p.wait_ns = kDefaultWaitNs;
  p.fault_inject = h->fault_pending ? 1 : 0;
  h->fault_pending = false;
  if (few)
    return launch_b128_few(m, p, h->few_slots, s) == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
  const int clusters = std::min(p.num_pm * p.num_n, h->max_clusters);
  return launch_b128_gemm(m, p, clusters, s) == cudaSuccess ? MLPB_OK : MLPB_ECUDA;
}

mlpb_status quantize(const void* x, bool f32, int64_t rows, int64_t cols, const Quantized* q,
                     const Quantized* qt, cudaStream_t s) {
  return launch_b128_quantize(x, f32, rows, cols, false, q ? q->codes : nullptr,
                              q ? q->scales : nullptr, qt ? qt->codes : nullptr,
                              qt ? qt->scales : nullptr, s) == cudaSuccess
             ? MLPB_OK
             : MLPB_ECUDA;
}

}  // namespace

extern "C" mlpb_status mlpb_linear8_create(const mlpb_linear8_config* cfg, mlpb_linear8** out) {
  if (cfg == nullptr || out == nullptr) return MLPB_EINVAL;
  *out = nullptr;
  const mlpb_linear8_config& c = *cfg;
  if (c.max_tokens < 1 || c.inputs < 1 || c.outputs < 1 ||
      (c.flags & ~(MLPB_LINEAR8_OUT_F32 | MLPB_LINEAR8_FAULT_INJECT)) != 0)
    return MLPB_EINVAL;
  constexpr int64_t most = int64_t{1} << 20;
  if (c.max_tokens > most || c.inputs > most || c.outputs > most || c.inputs % 8 != 0 ||
      c.outputs % 8 != 0)
    return MLPB_EUNSUPPORTED;
  mlpb_linear8* h = new (std::nothrow) mlpb_linear8();
  if (h == nullptr) return MLPB_ENOMEM;
  h->cfg = c;
  h->fault_pending = (c.flags & MLPB_LINEAR8_FAULT_INJECT) != 0;
  mlpb_status st = h->on.find();
  if (st == MLPB_OK && (b128_gemm_set_attrs(&h->max_clusters) != cudaSuccess ||
                        h->max_clusters < 1 || b128_few_set_attrs(h->few_slots) != cudaSuccess ||
                        h->few_slots[0] < 1))
    st = MLPB_ECUDA;
  if (st == MLPB_OK) st = h->on.allocate();
  if (st != MLPB_OK) {
    delete h;
    return st;
  }
  *out = h;
  return MLPB_OK;
}

extern "C" void mlpb_linear8_destroy(mlpb_linear8* h) {
  if (h == nullptr) return;
  h->on.release();
  delete h;
}

extern "C" mlpb_status mlpb_linear8_workspace_size(const mlpb_linear8* h, size_t* bytes) {
  if (h == nullptr || bytes == nullptr) return MLPB_EINVAL;
  const mlpb_linear8_config& c = h->cfg;
  const size_t x = code_bytes(c.max_tokens, c.inputs) + scale_bytes(c.max_tokens, c.inputs);
  const size_t dy = code_bytes(c.max_tokens, c.outputs) + scale_bytes(c.max_tokens, c.outputs) +
                    code_bytes(c.outputs, c.max_tokens) + scale_bytes(c.outputs, c.max_tokens);
  *bytes = std::max(x, dy);
  return MLPB_OK;
}

extern "C" mlpb_status mlpb_linear8_forward(mlpb_linear8* h, int64_t tokens, const void* X,
                                            const void* Wq, const void* Ws, void* Y, void* Xt,
                                            void* Xts, void* workspace, mlpb_stream_t stream) {
  if (h == nullptr || tokens < 0) return MLPB_EINVAL;
  const mlpb_linear8_config& c = h->cfg;
  if (tokens > c.max_tokens) return MLPB_EUNSUPPORTED;
  if (!Wq || !Ws || (Xt == nullptr) != (Xts == nullptr)) return MLPB_EINVAL;
  if (tokens > 0 && (!X || !Y || !workspace)) return MLPB_EINVAL;
  for (const void* q : {X, Wq, Ws, static_cast<const void*>(Y), static_cast<const void*>(Xt),
                        static_cast<const void*>(Xts), static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MLPB_EINVAL;
  mlpb_status st = h->on.current();
  if (st != MLPB_OK || tokens == 0) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  const Quantized x = take(at, tokens, c.inputs);
  const Quantized w = quantized(Wq, Ws, c.outputs, c.inputs);
  const Quantized xt = quantized(Xt, Xts, c.inputs, tokens);
  st = quantize(X, false, tokens, c.inputs, &x, Xt ? &xt : nullptr, s);
  if (st != MLPB_OK) return st;
  return product(h, x, w, Y, (c.flags & MLPB_LINEAR8_OUT_F32) != 0, false, s);
}

extern "C" mlpb_status mlpb_linear8_backward(mlpb_linear8* h, int64_t tokens, const void* dY,
                                             const void* Wt, const void* Wts, const void* Xt,
                                             const void* Xts, void* dX, float* dW,
                                             int32_t accumulate, void* workspace,
                                             mlpb_stream_t stream) {
  if (h == nullptr || tokens < 0 || (accumulate != 0 && accumulate != 1)) return MLPB_EINVAL;
  const mlpb_linear8_config& c = h->cfg;
  if (tokens > c.max_tokens) return MLPB_EUNSUPPORTED;
  if (tokens > 0 && (!dY || !workspace || (!dX && !dW) || (dX && (!Wt || !Wts)) ||
                     (dW && (!Xt || !Xts))))
    return MLPB_EINVAL;
  for (const void* q :
       {dY, Wt, Wts, Xt, Xts, static_cast<const void*>(dX), static_cast<const void*>(dW),
        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MLPB_EINVAL;
  mlpb_status st = h->on.current();
  if (st != MLPB_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (dW != nullptr && accumulate == 0 &&
        cudaMemsetAsync(dW, 0, static_cast<size_t>(c.inputs * c.outputs) * 4, s) != cudaSuccess)
      return MLPB_ECUDA;
    return MLPB_OK;
  }
  uint8_t* at = static_cast<uint8_t*>(workspace);
  const Quantized dy = take(at, tokens, c.outputs), dyt = take(at, c.outputs, tokens);
  st = quantize(dY, false, tokens, c.outputs, dX ? &dy : nullptr, dW ? &dyt : nullptr, s);
  if (st == MLPB_OK && dX != nullptr)
    st = product(h, dy, quantized(Wt, Wts, c.inputs, c.outputs), dX,
                 (c.flags & MLPB_LINEAR8_OUT_F32) != 0, false, s);
  if (st == MLPB_OK && dW != nullptr)
    st = product(h, dyt, quantized(Xt, Xts, c.inputs, tokens), dW, true, accumulate != 0, s);
  return st;
}

extern "C" mlpb_status mlpb_linear8_last_device_error(mlpb_linear8* h, mlpb_stream_t stream) {
  if (h == nullptr) return MLPB_EINVAL;
  return h->on.last_error(reinterpret_cast<cudaStream_t>(stream));
}
