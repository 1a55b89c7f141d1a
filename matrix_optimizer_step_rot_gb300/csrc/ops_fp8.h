// The product of 8-bit matrices, between its entry point (ops_fp8.cu) and its
// kernels (ops_fp8_gemm.cu).
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
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

// Products with few rows of A (ops_fp8_few.cu): fp8_few where that kernel
// takes them in 8 bits (their scales in p), fp8_self_rounded where it takes
// them in a float type too and rounds them as rot_fp8_quantize does.
bool fp8_few(int64_t M, int64_t N, int64_t K);
bool fp8_self_rounded(int64_t M, int64_t N, int64_t K);
int fp8_few_product(const Prod& p, const void* x, int64_t ldx, int32_t xtype, cudaStream_t stream);

uint64_t fp8_work_bytes(int64_t M, int64_t N, int64_t K);
int fp8_product(const Prod& p, int* status, cudaStream_t stream);
// Two products in one launch of the large kernel, where neither needs parts;
// neither may be an operand of the other, and the second one's C is float32.
bool fp8_takes_two(int64_t M0, int64_t N0, int64_t K0, int64_t M1, int64_t N1, int64_t K1);
int fp8_two_products(const Prod& p, const Prod& q, int* status, cudaStream_t stream);

// The scale's byte for a block whose largest finite magnitude is `amax`: the
// least e >= -127 with amax <= max 2^e.  max is 1.75 2^top (448: top 8;
// 57344: top 15), amax is m 2^k with m in [1, 2), so e = k - top, plus one
// where m > 1.75.  Subnormal amax (and 0) end at -127.
__device__ __forceinline__ int scale_byte(float amax, bool e5m2) {
  const uint32_t bits = __float_as_uint(amax);
  const int k = (int)(bits >> 23) - 127;
  const int e = k - (e5m2 ? 15 : 8) + ((bits & 0x7FFFFFu) > 0x600000u);
  return max(e, -127) + 127;
}
// 2^-(byte - 127), a normal number for every byte up to 253 (scale_byte ends
// at 247)
__device__ __forceinline__ float inverse_scale(int byte) {
  return __uint_as_float((uint32_t)(254 - byte) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// 8 bits of x * inv (at most max in magnitude by choice of inv); NaN and
// infinities become NaN.
__device__ __forceinline__ uint32_t to_f8(float x, float inv, bool e5m2) {
  float v = x * inv;
  if (!(fabsf(x) < INFINITY)) v = NAN;
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, e5m2 ? __NV_E5M2 : __NV_E4M3);
}

}  // namespace ops
}  // namespace rot
