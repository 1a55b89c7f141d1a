// The product of 8-bit matrices, between its entry point (ops_fp8.cu) and its
// kernels (ops_fp8_gemm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rot {
namespace ops {

// C = A B^T (rot_fp8_gemm's checked arguments, K > 0).  The scale of row r and
// K block j of A is sa[j * ldsa + (r >> ash)].
struct Prod {
  const uint8_t *a, *b, *sa, *sb;
  void* c;
  int64_t lda, ldb, ldsa, ldsb, ldc;
  int M, N, K, ctype, accumulate;
  int a5, b5;    // operands in E5M2
  int ash, bsh;  // 0 (a scale per row) or 7 (per 128 rows)
  float* part;   // workspace
};

uint64_t fp8_work_bytes(int64_t M, int64_t N, int64_t K);
int fp8_product(const Prod& p, int* status, cudaStream_t stream);

}  // namespace ops
}  // namespace rot
