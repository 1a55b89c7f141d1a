// Layer norm (include/rot_ops.h): what the forward and the backward pass share.
#pragma once

#include "ops_common.cuh"

namespace rot {
namespace ops {

struct NormFwd {
  const void *x, *res, *w, *b;
  void *h, *y;
  float *mean, *rstd;
  int64_t ldx, ldr, ldh, ldy, rows;
  int cols;
  int w32;  // weight and bias are float32 (otherwise of the row's type)
  float eps;
  Drop d;
};

struct NormBwd {
  const void *dy, *h, *w, *dh;
  const float *mean, *rstd;
  void *dres, *dx;
  float* part;  // [parts][2][cols]: dweight, dbias
  int64_t lddy, ldh, lddh, lddres, lddx, rows;
  int cols;
  int w32;
  Drop d;
};

template <class T, int U>
__device__ __forceinline__ Vec<U> load_weight(const void* w, bool w32, int c) {
  if (!w32) return unpack(raw_run<T, U>(w, c));
  Vec<U> f;
  if constexpr (U > 1) {
#pragma unroll
    for (int k = 0; k < U / 2; k += 2) {
      const float4 v = *reinterpret_cast<const float4*>((const float*)w + c + 2 * k);
      f.p[k] = make_float2(v.x, v.y), f.p[k + 1] = make_float2(v.z, v.w);
    }
  } else {
    f.p[0] = ((const float*)w)[c];
  }
  return f;
}

// 1 / sqrt(v): the approximation and one Newton step (as exact as the two
// rounded operations, at a few instructions); the plain operations at the ends
// of the range.
__device__ __forceinline__ float inverse_root(float v) {
  const float r = rsqrtf(v);
  if (!(v > 1e-36f && v < 1e36f)) return 1.f / sqrtf(v);
  return r * fmaf(-0.5f * v * r, r, 1.5f);
}

// Waits for the TPR threads of this thread's row (a block may hold several).
template <int TPR, int BLOCK>
__device__ __forceinline__ void row_barrier() {
  if constexpr (TPR == BLOCK)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / TPR), "n"(TPR) : "memory");
}

// Sums of two values over the TPR threads of a row, in one exchange; `red`
// holds a pair per warp of the block.  Calls in a row need different `red`
// arrays (a thread may still read the last one).
template <int TPR, int BLOCK>
__device__ __forceinline__ float2 row_sum2(float x, float y, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float2 v = make_float2(__shfl_xor_sync(0xffffffffu, x, o),
                                 __shfl_xor_sync(0xffffffffu, y, o));
    const float2 w = add2(make_float2(x, y), v);
    x = w.x, y = w.y;
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(x, y);
    row_barrier<TPR, BLOCK>();
    const float4* p = reinterpret_cast<const float4*>(red + warp / W * W);
    float2 sum = both(0.f);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const float4 v = p[i];
      sum = add2(sum, add2(make_float2(v.x, v.y), make_float2(v.z, v.w)));
    }
    return sum;
  }
  return make_float2(x, y);
}
template <int TPR, int BLOCK>
__device__ __forceinline__ float row_sum(float x, float* red) {
  x = warp_sum(x);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = x;
    row_barrier<TPR, BLOCK>();
    const float4* p = reinterpret_cast<const float4*>(red + warp / W * W);
    float2 sum = both(0.f);
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const float4 v = p[i];
      sum = add2(sum, add2(make_float2(v.x, v.y), make_float2(v.z, v.w)));
    }
    return sum.x + sum.y;
  }
  return x;
}

constexpr int block_of(int tpr) { return tpr > 128 ? tpr : 128; }

// Threads per row that hold `cols` in shares of at most `share` elements; 0:
// too wide.
inline int row_threads(int cols, int share) {
  for (int t : {32, 128, 256, 512, 1024})
    if (cols <= t * share) return t;
  return 0;
}

// Partial sums of the weight gradient kept at most (the workspace's size does
// not depend on the GPU).
constexpr int kMaxParts = 608;

int norm_forward(int32_t type, const NormFwd& a, cudaStream_t s);
int norm_backward(int32_t type, const NormBwd& a, float* dweight, float* dbias, cudaStream_t s);

}  // namespace ops
}  // namespace rot
