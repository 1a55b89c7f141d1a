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
    if constexpr (W == 2) return red[warp & ~1] + red[warp | 1];
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

// Rows that are not 16-byte aligned go element by element (runs of U = 1): a
// warp takes 32 N consecutive ones, lane by lane, so that accesses stay
// together and the warp shares the dropout's generator calls (keep_bits).
// Shares of a warp are then large: 64 threads per row as well, and for short
// rows shares of 4.
constexpr int kSingles = 8, kFewSingles = 4;
inline int row_threads_single(int cols) {
  return cols > 32 * kSingles && cols <= 64 * kSingles ? 64 : row_threads(cols, kSingles);
}
// First element of run n of a row's thread t.
template <int U, int TPR, int N>
__device__ __forceinline__ int column_of(int n, int t) {
  return U > 1 ? (n * TPR + t) * U : (t / 32 * N + n) * 32 + t % 32;
}
// Whether the warp of thread t has elements of the row at all.
template <int U, int N>
__device__ __forceinline__ bool has_columns(int t, int cols) {
  return U > 1 || t / 32 * N * 32 < cols;
}
// A thread's runs of the row at element o of p.  Single elements are 32 apart,
// so that one address serves them all; those past the row's end read as 0.
template <class T, int U, int N>
__device__ __forceinline__ void get_runs(Run<T, U> (&r)[N], const void* p, int64_t o,
                                         const int (&c)[N], const bool (&in)[N]) {
  if constexpr (U > 1) {
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = raw_run<T, U>(p, o + c[n]);
  } else {
    const T* q = (const T*)p + o + c[0];
#pragma unroll
    for (int n = 0; n < N; ++n) r[n].v[0] = in[n] ? q[32 * n] : from_f32<T>(0.f);
  }
}
template <class T, int U, int N>
__device__ __forceinline__ void put_runs(void* p, int64_t o, const int (&c)[N],
                                         const bool (&in)[N], const Vec<U> (&f)[N]) {
  T* q = (T*)p + o + c[0];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!in[n]) continue;
    if constexpr (U > 1)
      put_run(p, o + c[n], pack<T>(f[n]));
    else
      q[32 * n] = from_f32<T>(f[n].p[0]);
  }
}
template <class T, int U, int N>
__device__ __forceinline__ void get_weights(Vec<U> (&f)[N], const void* w, bool w32,
                                            const int (&c)[N], const bool (&in)[N]) {
  if constexpr (U > 1) {
#pragma unroll
    for (int n = 0; n < N; ++n) f[n] = load_weight<T, U>(w, w32, c[n]);
  } else if (w32) {
    const float* q = (const float*)w + c[0];
#pragma unroll
    for (int n = 0; n < N; ++n) f[n].p[0] = in[n] ? q[32 * n] : 0.f;
  } else {
    const T* q = (const T*)w + c[0];
#pragma unroll
    for (int n = 0; n < N; ++n) f[n].p[0] = in[n] ? to_f32(q[32 * n]) : 0.f;
  }
}
// Dropout of the N runs of a thread of a row.
template <int U, int N>
__device__ __forceinline__ void drop_runs(const Drop& d, uint64_t row0, const int (&c)[N],
                                          int t, int cols, Vec<U> (&f)[N]) {
  if constexpr (U > 1) {
#pragma unroll
    for (int n = 0; n < N; ++n) drop_run(d, row0 + c[n], f[n]);
  } else {
    const int c0 = t / 32 * N * 32;
    const uint32_t bits = keep_bits<N>(d, row0 + c0, cols - c0);
#pragma unroll
    for (int n = 0; n < N; ++n) f[n].p[0] = kept(d, bits >> n & 1, f[n].p[0]);
  }
}

// Partial sums of the weight gradient kept at most (the workspace's size does
// not depend on the GPU).
constexpr int kMaxParts = 608;

int norm_forward(int32_t type, const NormFwd& a, cudaStream_t s);
int norm_backward(int32_t type, const NormBwd& a, float* dweight, float* dbias, cudaStream_t s);

}  // namespace ops
}  // namespace rot
