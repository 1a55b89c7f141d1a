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

// Launches a kernel that begins with wait_for_prior(): its blocks may start
// (set-up, no reads of earlier results) while the stream's kernel before it
// ends.
template <class... P, class... A>
int launch_behind(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                  cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  if (cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...) == cudaSuccess) return ROT_OK;
  cudaGetLastError();
  return ROT_ECUDA;
}
// Waits until the stream's earlier kernels have ended and their writes are
// visible.
__device__ __forceinline__ void wait_for_prior() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

// Pairs of float32 operations as one instruction (each half rounds as the
// single operation does).
__device__ __forceinline__ unsigned long long bits2(float2 x) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.x), "f"(x.y));
  return r;
}
__device__ __forceinline__ float2 float2_of(unsigned long long x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
// the same on one value, for runs of one element
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float add2(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float mul2(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
template <class E>
__device__ __forceinline__ E all_of(float x);
template <>
__device__ __forceinline__ float2 all_of<float2>(float x) { return make_float2(x, x); }
template <>
__device__ __forceinline__ float all_of<float>(float x) { return x; }
__device__ __forceinline__ float total(float2 x) { return x.x + x.y; }
__device__ __forceinline__ float total(float x) { return x; }

// A run of U elements as float32, in pairs or one alone.
template <int U>
struct Vec {
  using E = float2;
  static constexpr int P = U / 2;
  E p[P];
};
template <>
struct Vec<1> {
  using E = float;
  static constexpr int P = 1;
  E p[1];
};
__device__ __forceinline__ float2 unpack2(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ float2 unpack2(__half a, __half b) {
  return __half22float2(__halves2half2(a, b));
}
__device__ __forceinline__ float2 unpack2(__nv_bfloat16 a, __nv_bfloat16 b) {
  return __bfloat1622float2(__halves2bfloat162(a, b));
}
template <class T, int U>
__device__ __forceinline__ Vec<U> unpack(const Run<T, U>& r) {
  Vec<U> v;
  if constexpr (U == 1) {
    v.p[0] = to_f32(r.v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < U / 2; ++i) v.p[i] = unpack2(r.v[2 * i], r.v[2 * i + 1]);
  }
  return v;
}
__device__ __forceinline__ void pack2(float2 x, float& a, float& b) { a = x.x, b = x.y; }
__device__ __forceinline__ void pack2(float2 x, __half& a, __half& b) {
  const __half2 h = __float22half2_rn(x);
  a = __low2half(h), b = __high2half(h);
}
__device__ __forceinline__ void pack2(float2 x, __nv_bfloat16& a, __nv_bfloat16& b) {
  const __nv_bfloat162 h = __float22bfloat162_rn(x);
  a = __low2bfloat16(h), b = __high2bfloat16(h);
}
template <class T, int U>
__device__ __forceinline__ Run<T, U> pack(const Vec<U>& v) {
  Run<T, U> r;
  if constexpr (U == 1) {
    r.v[0] = from_f32<T>(v.p[0]);
  } else {
#pragma unroll
    for (int i = 0; i < U / 2; ++i) pack2(v.p[i], r.v[2 * i], r.v[2 * i + 1]);
  }
  return r;
}
template <class T, int U>
__device__ __forceinline__ Run<T, U> raw_run(const void* p, int64_t o) {
  return *reinterpret_cast<const Run<T, U>*>((const T*)p + o);
}
template <class T, int U>
__device__ __forceinline__ void put_run(void* p, int64_t o, const Run<T, U>& r) {
  *reinterpret_cast<Run<T, U>*>((T*)p + o) = r;
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
  // round 0 with its constants (offset and key) worked in: {hi(offset low *
  // M1) ^ key, lo of the same, offset high ^ key}
  uint32_t first[3] = {};
  uint32_t key[9][2] = {};  // of rounds 1 to 9
};
struct Words {
  uint32_t w[4];
};
__device__ __forceinline__ uint2 mul_wide(uint32_t a, uint32_t b) {  // (low, high)
  uint2 r;
  asm("{\n\t.reg .b64 t;\n\tmul.wide.u32 t, %2, %3;\n\tmov.b64 {%0, %1}, t;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u;
__device__ __forceinline__ Words philox(const Drop& d, uint64_t counter) {
  const uint2 first = mul_wide((uint32_t)counter, kPhiloxM0);
  uint32_t c0 = d.first[0] ^ (uint32_t)(counter >> 32), c1 = d.first[1];
  uint32_t c2 = first.y ^ d.first[2], c3 = first.x;
#pragma unroll
  for (int r = 0; r < 9; ++r) {
    const uint2 a = mul_wide(c0, kPhiloxM0), b = mul_wide(c2, kPhiloxM1);
    c0 = b.y ^ c1 ^ d.key[r][0];
    c1 = b.x;
    c2 = a.y ^ c3 ^ d.key[r][1];
    c3 = a.x;
  }
  return {{c0, c1, c2, c3}};
}
Drop make_drop(double p, uint64_t seed, uint64_t offset);

// Elements i0 .. i0 + U - 1 of the row-major order <- dropped values.  Runs of
// 4 or more start on a multiple of 4.
template <int U>
__device__ __forceinline__ void drop_run(const Drop& d, uint64_t i0, Vec<U>& f) {
  if (!d.on) return;
  if constexpr (U % 4 == 0) {
#pragma unroll
    for (int q = 0; q < U / 4; ++q) {
      const Words w = philox(d, i0 / 4 + q);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 s = mul2(f.p[2 * q + k], both(d.scale));
        f.p[2 * q + k].x = w.w[2 * k] > d.bar ? s.x : 0.f;
        f.p[2 * q + k].y = w.w[2 * k + 1] > d.bar ? s.y : 0.f;
      }
    }
  } else {
    static_assert(U == 1, "runs of one element or of a multiple of four");
    const Words w = philox(d, i0 / 4);
    const uint32_t s = (uint32_t)i0 & 3u;
    const uint32_t word = s == 0 ? w.w[0] : s == 1 ? w.w[1] : s == 2 ? w.w[2] : w.w[3];
    f.p[0] = word > d.bar ? __fmul_rn(f.p[0], d.scale) : 0.f;
  }
}

// Dropout of a warp's 32 N consecutive elements from i0, whatever i0 mod 4 is:
// element n * 32 + lane of this lane is kept where bit n is set.  Each lane
// takes every 32nd of the N * 8 generator calls (one more where i0 lies within
// a call) and the others fetch its four answers: N / 4 calls per N elements
// instead of one each.  The whole warp calls it; only the first `count`
// answers (or all) are asked for.
template <int N>
__device__ __forceinline__ uint32_t keep_bits(const Drop& d, uint64_t i0, int count = 32 * N) {
  static_assert(N % 4 == 0 && N <= 16, "whole generator calls, at most five answers");
  const int lane = threadIdx.x & 31;
  const uint32_t phase = (uint32_t)i0 & 3u;
  uint32_t mine = 0;
#pragma unroll
  for (int r = 0; r < N / 4 + 1; ++r) {
    if (r == N / 4 && (int)phase + min(count, 32 * N) <= 32 * N) break;
    const Words w = philox(d, (i0 >> 2) + r * 32 + lane);
#pragma unroll
    for (int k = 0; k < 4; ++k) mine |= (w.w[k] > d.bar ? 1u : 0u) << (4 * r + k);
  }
  uint32_t bits = 0;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t e = phase + n * 32 + lane;
    const uint32_t v = __shfl_sync(0xffffffffu, mine, (e >> 2) & 31);
    bits |= (v >> ((e >> 7) * 4 + (e & 3)) & 1u) << n;
  }
  return bits;
}
__device__ __forceinline__ float kept(const Drop& d, bool keep, float x) {
  return keep ? __fmul_rn(x, d.scale) : 0.f;
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
