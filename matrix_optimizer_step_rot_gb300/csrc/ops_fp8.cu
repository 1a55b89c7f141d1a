// 8-bit matrices with power-of-two block scales (include/rot_ops.h):
// quantisation, and the product's entry point (its kernels: ops_fp8_gemm.cu).
#include <cuda_fp8.h>

#include <algorithm>

#include "ops_common.cuh"
#include "ops_fp8.h"
#include "profile.h"

namespace rot {
namespace ops {
namespace {

// ---------------------------------------------------------------------------
// quantisation
// ---------------------------------------------------------------------------

struct Quant {
  const void* x;
  uint8_t *q, *s, *qt, *st;
  int64_t ldx, rows, cols, ldq, lds, ldqt, ldst;
  int e5m2, square;  // square: blocks of 128 x 128
};

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

constexpr int kQ = 128;  // a block's edge

// A 128 x 128 tile per CTA, 256 threads: thread (g = t / 16, v = t % 16) holds
// rows 8 g .. 8 g + 7 of columns 8 v .. 8 v + 7, so both orientations' 8-bit
// runs of eight are in one thread.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) quantize_kernel(const Quant a) {
  __shared__ float colmax[16][kQ];
  __shared__ uint8_t colscale[kQ];
  __shared__ float wide[8];
  const int64_t tiles_c = (a.cols + kQ - 1) / kQ;
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x % tiles_c;  // tile row, column
  const int64_t r0 = tr * kQ, c0 = tc * kQ;
  const int g = threadIdx.x / 16, v = threadIdx.x % 16;
  const int64_t r = r0 + 8 * g, c = c0 + 8 * v;
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[i][k] = 0.f;
    if (r + i >= a.rows) continue;
    const T* p = (const T*)a.x + (r + i) * a.ldx + c;
    if (VEC && c + 8 <= a.cols) {
      constexpr int U = 16 / sizeof(T);
#pragma unroll
      for (int k = 0; k < 8; k += U) {
        float f[U];
        load_run(p + k, f);
#pragma unroll
        for (int j = 0; j < U; ++j) x[i][k + j] = f[j];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < a.cols) x[i][k] = to_f32(p[k]);
    }
  }
  float rm[8], cm[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) rm[k] = cm[k] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float m = finite_abs(x[i][k]);
      rm[i] = fmaxf(rm[i], m);
      cm[k] = fmaxf(cm[k], m);
    }
  int rb[8], cb[8];  // scale bytes of this thread's rows and columns
  if (a.square) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, rm[i]);
    m = warp_max(m);
    if (threadIdx.x % 32 == 0) wide[threadIdx.x / 32] = m;
    __syncthreads();
    m = wide[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, wide[i]);
    const int b = scale_byte(m, a.e5m2);
#pragma unroll
    for (int i = 0; i < 8; ++i) rb[i] = cb[i] = b;
    if (threadIdx.x == 0) {
      if (a.q) a.s[tc * a.lds + tr] = (uint8_t)b;
      if (a.qt) a.st[tr * a.ldst + tc] = (uint8_t)b;
    }
  } else {
    if (a.q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float m = rm[i];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        rb[i] = scale_byte(m, a.e5m2);
        if (v == 0 && r + i < a.rows)
          a.s[tc * a.lds + r + i] = (uint8_t)rb[i];
      }
    }
    if (a.qt) {
#pragma unroll
      for (int k = 0; k < 8; ++k) colmax[g][8 * v + k] = cm[k];
      __syncthreads();
      if (threadIdx.x < kQ) {
        float m = colmax[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < 16; ++i) m = fmaxf(m, colmax[i][threadIdx.x]);
        const int b = scale_byte(m, a.e5m2);
        colscale[threadIdx.x] = (uint8_t)b;
        if (c0 + threadIdx.x < a.cols)
          a.st[tr * a.ldst + c0 + threadIdx.x] = (uint8_t)b;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) cb[k] = colscale[8 * v + k];
    }
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r + i >= a.rows) continue;
      const float inv = inverse_scale(rb[i]);
      uint8_t* p = a.q + (r + i) * a.ldq + c;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < a.cols) p[k] = (uint8_t)to_f8(x[i][k], inv, a.e5m2);
    }
  }
  if (a.qt) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (c + k >= a.cols) continue;
      const float inv = inverse_scale(cb[k]);
      uint8_t* p = a.qt + (c + k) * a.ldqt + r;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + i < a.rows) p[i] = (uint8_t)to_f8(x[i][k], inv, a.e5m2);
    }
  }
}

template <class T>
int launch_quantize(const Quant& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(((a.cols + kQ - 1) / kQ) * ((a.rows + kQ - 1) / kQ));
  const bool vec = rows16(a.x, a.ldx, sizeof(T));
  const double n = (double)a.rows * a.cols;
  ProfScope prof(ROT_PROF_ELEMENTWISE, n * (sizeof(T) + (a.q != nullptr) + (a.qt != nullptr)), s);
  auto k = vec ? quantize_kernel<T, true> : quantize_kernel<T, false>;
  k<<<grid, 256, 0, s>>>(a);
  return launched();
}

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m; }
constexpr int64_t kMost = (int64_t(1) << 31) - 256;

bool bad_operand(const void* d, int64_t ld, int32_t fmt, const uint8_t* s, int64_t lds,
                 int32_t block_rows, int64_t rows, int64_t K) {
  if (fmt != ROT_TYPE_E4M3 && fmt != ROT_TYPE_E5M2) return true;
  if (block_rows != 1 && block_rows != kQ) return true;
  if (ld < K || ld % 16 || lds < up(rows, block_rows)) return true;
  return rows > 0 && K > 0 && (!d || !s || !aligned16(d));
}

}  // namespace
}  // namespace ops
}  // namespace rot

using namespace rot;
using namespace rot::ops;

extern "C" {

int rot_fp8_quantize(const void* x, int64_t ldx, int64_t rows, int64_t cols, int32_t type,
                     int32_t format, int32_t block_rows, void* data, int64_t ldq, uint8_t* scale,
                     int64_t lds, void* data_t, int64_t ldqt, uint8_t* scale_t, int64_t ldst,
                     void* stream) {
  if (rows < 0 || cols < 0 || rows > kMost || cols > kMost || !float_type(type)) return ROT_EINVAL;
  if (format != ROT_TYPE_E4M3 && format != ROT_TYPE_E5M2) return ROT_EINVAL;
  if ((block_rows != 1 && block_rows != kQ) || ldx < cols) return ROT_EINVAL;
  if (data && (!scale || ldq < cols || lds < up(rows, block_rows))) return ROT_EINVAL;
  if (data_t && (!scale_t || ldqt < rows || ldst < up(cols, block_rows))) return ROT_EINVAL;
  if (rows == 0 || cols == 0) return ROT_OK;
  if (!x || (!data && !data_t)) return ROT_EINVAL;
  if (up(rows, kQ) * up(cols, kQ) > 0x7FFFFFFF) return ROT_EINVAL;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  Quant a = {x, (uint8_t*)data, scale, (uint8_t*)data_t, scale_t, ldx, rows, cols, ldq, lds, ldqt,
             ldst, format == ROT_TYPE_E5M2, block_rows == kQ};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return guarded([&] {
    if (type == ROT_TYPE_F32) return launch_quantize<float>(a, s);
    if (type == ROT_TYPE_F16) return launch_quantize<__half>(a, s);
    return launch_quantize<__nv_bfloat16>(a, s);
  });
}

uint64_t rot_fp8_gemm_work_bytes(int64_t M, int64_t N, int64_t K) {
  return fp8_work_bytes(M, N, K);
}

int rot_fp8_gemm(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda, int32_t a_format,
                 const uint8_t* a_scale, int64_t a_lds, int32_t a_block_rows, const void* b,
                 int64_t ldb, int32_t b_format, const uint8_t* b_scale, int64_t b_lds,
                 int32_t b_block_rows, void* c, int64_t ldc, int32_t ctype, int32_t accumulate,
                 void* work, uint64_t work_bytes, int32_t* status, void* stream) {
  if (M < 0 || N < 0 || K < 0 || M > kMost || N > kMost || K > kMost) return ROT_EINVAL;
  if (bad_operand(a, lda, a_format, a_scale, a_lds, a_block_rows, M, K) ||
      bad_operand(b, ldb, b_format, b_scale, b_lds, b_block_rows, N, K))
    return ROT_EINVAL;
  if (!float_type(ctype) || (accumulate && ctype != ROT_TYPE_F32) || ldc < N) return ROT_EINVAL;
  if (M == 0 || N == 0 || (K == 0 && accumulate)) return ROT_OK;
  const uint64_t need = rot_fp8_gemm_work_bytes(M, N, K);
  if (!c || (need && (!work || work_bytes < need || (reinterpret_cast<uintptr_t>(work) & 255))))
    return ROT_EINVAL;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  Prod p = {(const uint8_t*)a, (const uint8_t*)b, a_scale, b_scale, c, lda, ldb, a_lds, b_lds, ldc,
            (int)M, (int)N, (int)K, ctype, accumulate, a_format == ROT_TYPE_E5M2,
            b_format == ROT_TYPE_E5M2, a_block_rows == 1 ? 0 : 7, b_block_rows == 1 ? 0 : 7,
            static_cast<float*>(work)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0)  // all bits zero is 0 in every type
    return cudaMemset2DAsync(c, ldc * type_bytes(ctype), 0, N * type_bytes(ctype), M, s) ==
                   cudaSuccess
               ? ROT_OK
               : ROT_ECUDA;
  return guarded([&] { return fp8_product(p, reinterpret_cast<int*>(status), s); });
}

}  // extern "C"
