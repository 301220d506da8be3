// Launch parameters of the products of block-scaled E4M3 operands (linear8.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "b128.cuh"

namespace mlpb {

// C [M][N] (+)= A B^T for A [M][K] and B [N][K] in block-scaled E4M3.
struct B128Params {
  int M, N;
  int num_pm, num_n, num_kb;  // pairs of M tiles, N tiles, 128-deep k-blocks
  int a_tiles, b_tiles;       // 128-row tiles that the scales have
  int raster_group;
  int out_f32;     // C is fp32 (else bf16)
  int accumulate;  // C += (fp32)
  int chunk;       // k-blocks of a sum in the tensor cores, a power of two
  void* C;
  uint32_t* err;
  uint64_t wait_ns;
  int fault_inject;
};

struct B128Maps {
  CUtensorMap a, b, sa, sb;
  CUtensorMap c;  // C in boxes of 32 rows by 128 bytes, where b128_staged says so
};

// k-blocks of a sum in the tensor cores for an fp32 result (bf16: all of them).
int b128_chunk(bool out_f32);
bool b128_staged(int num_kb, bool accumulate);
cudaError_t b128_gemm_set_attrs(int* max_clusters);
cudaError_t launch_b128_gemm(const B128Maps& m, const B128Params& p, int clusters, cudaStream_t s);

// gemm_b128_few.cu: the same with few tiles, C written (not added to).  `slots`: clusters of 1, 2,
// 4 and 8 CTAs that are resident at once with a CTA an SM; the box of m.a has b128_few_columns(M)
// rows.
constexpr int kFewSlots = 4;
int b128_few_columns(int64_t b_rows);
cudaError_t b128_few_set_attrs(int* slots);
cudaError_t launch_b128_few(const B128Maps& m, const B128Params& p, const int* slots,
                            cudaStream_t s);

}  // namespace mlpb
