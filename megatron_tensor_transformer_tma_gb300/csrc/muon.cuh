// Newton-Schulz orthogonalisation on the tensor cores: number formats, launch parameters.
//
// X <- a X + (b A + c A A) X with A = X X^T (or X <- a X + X (b A + c A A), A = X^T X, when X has
// more rows than columns).  With n the smaller side, two of the three products are symmetric
// n x n matrices, of which only the tiles on and below the diagonal are computed.
//
// Operands are fp16, which has eight times bf16's precision at the same rate; values have fixed
// scales, since singular values stay below 2 (the host checks the coefficients).  What would cost
// precision is kept out of the products:
//   - X is hi + lo, two fp16 parts (22 bits); the product takes hi, a X both.  (The last step's X
//     is hi alone: what it loses is not amplified any more.)
//   - The diagonal d of A is fp32 and its part E off the diagonal fp16:
//       A A = E E + (d_i + d_j) E_ij + delta_ij d_i^2,
//     so the identity that A comes near is not rounded.  Likewise b A + c A A + a I is
//     D + diag(beta) and X' = beta hi + D hi + a lo: a X and most of (b A + c A A) X cancel
//     (3.4 - 2.7 near the end), and do so in fp32.
//   - What the product does not see of lo, (b A + c A A) lo, lies along the large singular values,
//     which stay as they are.  beta lo in place of a lo would leave out D lo alone, less where A is
//     near the identity; but where few directions dominate, D + diag(beta) - a I has a low rank,
//     which D has not, and what it leaves out falls into all the others, which later steps amplify
//     a times each: 4 % of O for rank one at 2 x 40, more than O in 12 steps.  So lo goes with beta
//     in the last two steps that have one, and with a before.
// Against 64 bits the result of five steps is off by 3e-4 to 1.4e-3 of its size, and by up to 4e-3
// below n = 32 or where one singular value dominates (Gaussian matrices, gradients, low ranks and
// singular values that fall to 1e-4 of the largest, from n = 64 on: 3e-4 to 1.2e-3).  12 steps:
// 1e-3 to 1e-2, but what lies below 2^-22 of |U| grows a times a step, to 0.1 of O for rank one.
// With the diagonals in the products even spectra are off by 1e-3 to 3e-3, with bf16 operands by
// 1e-2 to 2e-2.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace mlpb {

constexpr float kXScale = 4096.0f;    // X, E are stored times 2^12
constexpr float kXInv = 1.0f / 4096.0f;
constexpr float kDScale = 1024.0f;    // D times 2^10
constexpr float kEEInv = kXInv * kXInv;            // a product's scale: 2^-24
constexpr int kOrthoMaxSplit = 16;  // ranges of K
constexpr int kOrthoLd = 64;  // rows of X, E and D are padded to multiples of 64 (X's with zeros)

enum class OrthoOp : int {
  Gram = 0,  // E, d from X
  Poly,      // D, beta from E, d
  Apply,     // X' from D, beta, X
  Last,      // as Apply, into the result
};

struct OrthoParams {
  int batch, rows, cols, n;  // n = min(rows, cols)
  int ldn;                   // elements of a row of E, D, diag and beta
  int narrow;                // tiles of 128 columns, not 256
  int num_pm, num_n;         // 256-row tiles and column tiles of a matrix
  int per_matrix;            // tiles of a matrix (on and below the diagonal for Gram, Poly)
  int split;                 // Gram, Poly: ranges of K; then no more units than pairs
  int units;                 // tiles of all matrices, times split
  int num_kb;                // 64-deep k-blocks
  float4* partial;           // the ranges' sums
  __half *e, *d;             // [batch][n][ldn], for the sums of ranges
  float a, b, c;
  float* diag;  // d [batch][ldn]
  float* beta;  // [batch][ldn]
  int low_out;  // Apply: X' has a low part (the last step's X is the high part alone)
  int low_beta;  // Apply: the low part of X goes with beta, not with a
  // Last: O bf16, or the weight's update W <- (1 - lr wd) W - lr scale O
  __nv_bfloat16* out;
  float* w;
  __nv_bfloat16* wb;  // a bf16 copy of the updated W, or NULL
  int ragged;         // rows of out, w, wb that no tensor map takes (cols % 8 != 0)
  const float* lr;
  float decay, scale;
  uint32_t* err;
  uint64_t wait_ns;
  int fault_inject;
};

// The operands' maps, and those of the epilogue's boxes of 32 rows by 64 columns (W: 32 by 32).
struct OrthoMaps {
  CUtensorMap a, b;
  CUtensorMap in0;     // Poly: E;  Apply, Last: X
  CUtensorMap in1;     // Apply: its low part;  Last: W
  CUtensorMap out0;    // Gram: E;  Poly: D;  Apply: X';  Last: O or W's bf16 copy
  CUtensorMap out1;    // Apply: its low part
  CUtensorMap mirror;  // Gram: E;  Poly: D in boxes of 64 rows by 32 columns
};

cudaError_t ortho_set_attrs(int* max_clusters);
cudaError_t launch_ortho(OrthoOp op, bool tall, const OrthoMaps& m, const OrthoParams& p,
                         int clusters, cudaStream_t s);

// muon_prepare.cu.  U = G + momentum M' with M' = momentum M + G (nesterov), or M', or (M NULL) G
// itself; X = U / |U| in two fp16 parts.
struct MuonInput {
  const void* g;  // fp32, or bf16 (M NULL)
  float* m;
  int g_f32, nesterov;
  float momentum;
  int64_t batch, rows, cols;
};
int muon_partials(int64_t elems, int64_t batch);
cudaError_t launch_muon_norm(const MuonInput& in, float4* part, cudaStream_t s);
cudaError_t launch_muon_split(const MuonInput& in, const float4* part, __half* xh, __half* xh_other,
                              __half* xl, int ldx, cudaStream_t s);

// muon_small.cu: the whole update in one launch, for n <= 128 and lengths that a cluster's shared
// memory holds; 0 CTAs: it does not, or takes longer.
cudaError_t muon_small_cluster(int n, int64_t length, int64_t batch, bool tall, int steps,
                               int* cluster);
cudaError_t launch_muon_small(const MuonInput& in, const OrthoParams& o, int steps, int cluster,
                              cudaStream_t s);

}  // namespace mlpb
