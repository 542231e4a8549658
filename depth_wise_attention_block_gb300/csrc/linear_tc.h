// Tensor-core matrix products (linear_tc.cu) as linear.cu calls them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace attnres {

struct LinearEpilogue;

// A matrix [rows, cols] in memory (row stride ld): an operand whose rows
// (mn = false) or columns (mn = true) run along the product's side.  `prep`:
// where its copy for the tensor cores lies (launch_tc_prep), or null when TMA
// takes the matrix as it is.
struct TcOperand {
  const void* ptr;
  int64_t ld;
  int64_t rows, cols;
  bool mn;
  void* prep;
};

struct TcPlan {
  enum Shape { kWide, kPairs, kNarrow };
  Shape shape;    // narrow: B's rows along the lanes (few rows of A)
  int bn;         // columns of a tile
  int ksplit;     // CTAs of a cluster that share a tile's contraction
  int part_rows;  // partial rows of the column sums (kEpiDz)
  bool fused;     // fp32, narrow: B enters as it is, its terms are made on the way
};
// np: 1 (bf16) or 3 (fp32, three bf16 terms)
TcPlan tc_plan(int64_t M, int N, int64_t K, int np, int sm_count);
inline TcPlan tc_plan_unfused(TcPlan p) {
  p.fused = false;
  return p;
}
bool tc_rows_ok(const void* ptr, int64_t ld);                     // bf16 rows TMA takes as they are
int64_t tc_prep_bytes(int64_t rows, int64_t cols, int np);
cudaError_t launch_tc_prep(const TcOperand* ops, int n, int np, cudaStream_t stream);  // n <= 2
cudaError_t launch_tc_gemm(const TcPlan& plan, const TcOperand& A, const TcOperand& B, int64_t M, int N, int64_t K, int np,
                           int mode, const LinearEpilogue& epi, int* dev_err, cudaStream_t stream);

}  // namespace attnres
