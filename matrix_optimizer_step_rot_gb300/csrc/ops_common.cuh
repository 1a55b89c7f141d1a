// Shared by the operators' kernels (include/rot_ops.h): element types, wide
// loads and stores, sums over the threads of a row, the dropout generator.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "rot_internal.h"
#include "rot_ops.h"

namespace rot {
namespace ops {

// Runs an entry point's body: no C++ exception leaves it (the launch
// instrumentation keeps host containers).
template <class F>
int guarded(F&& body) {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return ROT_ENOMEM;
  } catch (...) {
    return ROT_ECUDA;
  }
}

inline int launched() { return cudaGetLastError() == cudaSuccess ? ROT_OK : ROT_ECUDA; }

inline bool float_type(int32_t t) {
  return t == ROT_TYPE_F32 || t == ROT_TYPE_F16 || t == ROT_TYPE_BF16;
}
inline int type_bytes(int32_t t) { return t == ROT_TYPE_F32 ? 4 : t <= ROT_TYPE_BF16 ? 2 : 1; }

__host__ __device__ inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether 16-byte accesses reach every row's elements: base and row pitch are
// multiples of 16 bytes (a null matrix does not matter).
__host__ __device__ inline bool rows16(const void* p, int64_t ld, int es) {
  return !p || (aligned16(p) && (ld * es) % 16 == 0);
}

// The number of SMs of the current device (set up once, as rot.h states).
inline int sm_count() {
  static const int n = [] {
    int dev = 0, k = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&k, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      k = 0;
    }
    return k > 0 ? k : 1;
  }();
  return n;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// A run of U elements as one access: U = 1, or 16 bytes' worth.
template <class T, int U>
struct alignas(sizeof(T) * U) Run {
  T v[U];
};

template <class T, int U>
__device__ __forceinline__ void load_run(const T* p, float (&f)[U]) {
  const Run<T, U> r = *reinterpret_cast<const Run<T, U>*>(p);
#pragma unroll
  for (int i = 0; i < U; ++i) f[i] = to_f32(r.v[i]);
}

template <class T, int U>
__device__ __forceinline__ void store_run(T* p, const float (&f)[U]) {
  Run<T, U> r;
#pragma unroll
  for (int i = 0; i < U; ++i) r.v[i] = from_f32<T>(f[i]);
  *reinterpret_cast<Run<T, U>*>(p) = r;
}

// Dropout of one call: whether it drops at all, 1 / (1 - p), and what the
// generator takes.  An element is kept where its word is above `bar`, round(p
// 2^32) - 1 (p = 1: above 2^32 - 1, which no word is).  Philox4x32-10 (Salmon,
// Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011)
// is ten rounds of two 32 x 32 -> 64 products; the rounds' keys depend on the
// seed alone, so the host works them out and the kernels read them as
// parameters.
struct Drop {
  int on = 0;
  uint32_t bar = 0;
  float scale = 1.f;
  uint32_t offset[2] = {};
  uint32_t key[10][2] = {};
};
struct Words {
  uint32_t w[4];
};
__device__ __forceinline__ Words philox(const Drop& d, uint64_t counter) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32);
  uint32_t c2 = d.offset[0], c3 = d.offset[1];
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ d.key[r][0];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ d.key[r][1];
    c3 = (uint32_t)a;
  }
  return {{c0, c1, c2, c3}};
}
Drop make_drop(double p, uint64_t seed, uint64_t offset);

// f[k] (elements i0 .. i0 + U - 1 of the row-major order) <- dropped values.
// Runs of 4 or more start on a multiple of 4.
template <int U>
__device__ __forceinline__ void drop_run(const Drop& d, uint64_t i0, float (&f)[U]) {
  if (!d.on) return;
  if constexpr (U % 4 == 0) {
#pragma unroll
    for (int q = 0; q < U / 4; ++q) {
      const Words w = philox(d, i0 / 4 + q);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        f[4 * q + k] = w.w[k] > d.bar ? __fmul_rn(f[4 * q + k], d.scale) : 0.f;
    }
  } else {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const Words w = philox(d, (i0 + k) / 4);
      const uint32_t s = (uint32_t)(i0 + k) & 3u;
      const uint32_t word = s == 0 ? w.w[0] : s == 1 ? w.w[1] : s == 2 ? w.w[2] : w.w[3];
      f[k] = word > d.bar ? __fmul_rn(f[k], d.scale) : 0.f;
    }
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

}  // namespace ops
}  // namespace rot
