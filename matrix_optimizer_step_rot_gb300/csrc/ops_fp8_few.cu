// y = x W^T for a few rows of x (rot_fp8_linear and rot_fp8_gemm with at most
// kFewRows rows): bound by reading W once.
//
// The tensor-core kernel's 128-row tiles would be almost empty, and splitting
// K over its CTAs costs a second launch.  Here every warp takes R rows of W
// (columns of y), a lane 16 bytes of each at a time with those of D steps on
// their way, and multiplies them by
// the matching 16 elements of x, which each CTA keeps in shared memory, rounded
// to 8 bits by itself (so a layer is one launch) or as they come in 8 bits.
// 8-bit values are exact in 16-bit floats and their products in float32; 16
// products are summed, then join under the two scales' exponent.  `share`
// warps split a row's K where y is too narrow to give every warp rows of its
// own; their sums are added in a fixed order.
#include <cuda_fp8.h>

#include <algorithm>

#include "ops_common.cuh"
#include "ops_fp8.h"
#include "profile.h"

namespace rot {
namespace ops {
namespace {

constexpr int kFewRows = 2;
constexpr int kCols = 4;         // rows of W per warp, R
constexpr int kWarps = 8;        // per CTA
constexpr int kSpan = 32 * 16;   // elements of K per step of a warp
constexpr int kMaxShared = 96 << 10;

struct Few {
  const uint8_t *w, *sw;         // W: N x K, as rot_fp8_gemm's B
  const void* x;                 // M x K: float type, or 8-bit with scales sx
  const uint8_t* sx;
  void* y;
  int64_t ldw, ldsw, ldx, ldsx, ldy;
  int M, N, K, xtype, ytype, w5, wsh, xsh, accumulate, share;
};

// 16 8-bit values as 8 pairs of 16-bit floats.
__device__ __forceinline__ void halves_of(uint4 v, bool e5m2, __half2 (&h)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    h[i] = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))),
                                              e5m2 ? __NV_E5M2 : __NV_E4M3));
}

// v 2^e for any e that two scale bytes give, NaN where one of them is 255.
__device__ __forceinline__ float scaled(float v, int ea, int eb) {
  const int e = ea + eb - 254;
  if (e >= -126 && e <= 127 && ea != 255 && eb != 255)
    return v * __uint_as_float((uint32_t)(e + 127) << 23);
  if (ea == 255 || eb == 255) return NAN;
  return ldexpf(v, e);
}

// Row m of x by the whole CTA: 16 elements per thread and turn, eight threads
// to a block of 128; scale and 8-bit values as the quantisation kernel makes
// them.
template <class T>
__device__ __forceinline__ void round_row(const Few& a, int m, __half* xs, uint8_t* sx, int kpad) {
  const T* x = (const T*)a.x + m * a.ldx;
  const bool run16 = aligned16(x);
  constexpr int U = 16 / sizeof(T);
  for (int k0 = 0; k0 < kpad; k0 += 32 * kWarps * 16) {  // (whole warps or none: kpad is a multiple of 128)
    const int k = k0 + threadIdx.x * 16;
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = 0.f;
    if (run16 && k + 16 <= a.K) {
#pragma unroll
      for (int i = 0; i < 16; i += U) {
        float v[U];
        load_run(x + k + i, v);
#pragma unroll
        for (int j = 0; j < U; ++j) f[i + j] = v[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k + i < a.K) f[i] = to_f32(x[k + i]);
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(f[i]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (k < kpad) {
      const int b = scale_byte(amax, false);
      const float inv = inverse_scale(b);
      __half2 h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        h[i] = __half2(__nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(to_f8(f[2 * i], inv, false) | to_f8(f[2 * i + 1], inv, false) << 8),
            __NV_E4M3));
      uint4* p = reinterpret_cast<uint4*>(xs + m * kpad + k);
      p[0] = *reinterpret_cast<const uint4*>(&h[0]);
      p[1] = *reinterpret_cast<const uint4*>(&h[4]);
      if (threadIdx.x % 8 == 0) sx[m * (kpad / 128) + k / 128] = (uint8_t)b;
    }
  }
}

// 16 elements of row m of x, from element k.
__device__ __forceinline__ void x_run(const __half* xs, int o, float2 (&f)[8]) {
  const uint4* p = reinterpret_cast<const uint4*>(xs + o);
  const uint4 lo = p[0], hi = p[1];
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
}
__device__ __forceinline__ void w_run(uint4 v, bool e5m2, float2 (&f)[8]) {
  __half2 h[8];
  halves_of(v, e5m2, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __half22float2(h[i]);
}
__device__ __forceinline__ float dot16(const float2 (&a)[8], const float2 (&b)[8]) {
  float2 q = mul2(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) q = fma2(a[i], b[i], q);
  return total(q);
}

template <int M>
__global__ void __launch_bounds__(32 * kWarps, 2) fp8_few_kernel(const __grid_constant__ Few a) {
  constexpr int D = 2, R = kCols;
  extern __shared__ __align__(16) uint8_t dyn[];
  const int kpad = (a.K + 127) / 128 * 128, blocks = kpad / 128;
  __half* xs = reinterpret_cast<__half*>(dyn);          // [M][kpad]
  uint8_t* sx = dyn + (size_t)M * kpad * 2;             // [M][blocks]
  __shared__ float join[kWarps][R][M];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % a.share, group = warp / a.share;
  const int n0 = (blockIdx.x * (kWarps / a.share) + group) * R;
  const int steps = (a.K + kSpan - 1) / kSpan;
  const int per = (steps + a.share - 1) / a.share;
  const int s0 = part * per, s1 = min(steps, s0 + per);

  wait_for_prior();  // (x and W may both come from the kernel before)
  // 16 bytes of every row of W, and their scales, of D steps
  uint4 wv[D][R];
  int we[D][R];
  const uint8_t* wp = a.w + (int64_t)n0 * a.ldw + lane * 16;
  auto fetch = [&](int s, uint4 (&v)[R], int (&e)[R]) {
    const int k = s * kSpan + lane * 16;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r] = make_uint4(0u, 0u, 0u, 0u);
      e[r] = 127;
      if (s < s1 && k < a.K && n0 + r < a.N) {
        const uint8_t* p = wp + r * a.ldw + s * kSpan;
        e[r] = a.sw[(k / 128) * a.ldsw + ((n0 + r) >> a.wsh)];
        if (k + 16 <= a.K) {
          v[r] = *reinterpret_cast<const uint4*>(p);
        } else {  // (what lies past the last column is not part of the row)
          uint32_t b[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
          for (int i = 0; i < a.K - k; ++i) {
            const uint32_t byte = (uint32_t)p[i] << (8 * (i & 3));
            b[0] |= i / 4 == 0 ? byte : 0u;
            b[1] |= i / 4 == 1 ? byte : 0u;
            b[2] |= i / 4 == 2 ? byte : 0u;
            b[3] |= i / 4 == 3 ? byte : 0u;
          }
          v[r] = make_uint4(b[0], b[1], b[2], b[3]);
        }
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(s0 + d, wv[d], we[d]);
  if (a.xtype >= ROT_TYPE_E4M3) {
    for (int i = threadIdx.x; i < M * kpad; i += 32 * kWarps) {
      const int m = i / kpad, k = i - m * kpad;
      const uint8_t v = m < a.M && k < a.K ? ((const uint8_t*)a.x)[m * a.ldx + k] : 0;
      xs[i] = __half(__nv_cvt_fp8_to_halfraw(v, a.xtype == ROT_TYPE_E5M2 ? __NV_E5M2 : __NV_E4M3));
    }
    for (int i = threadIdx.x; i < M * blocks; i += 32 * kWarps) {
      const int m = i / blocks, b = i - m * blocks;
      sx[i] = m < a.M ? a.sx[b * a.ldsx + (m >> a.xsh)] : 127;
    }
  } else {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (m >= a.M) {
        for (int i = threadIdx.x; i < kpad; i += 32 * kWarps) xs[m * kpad + i] = __float2half_rn(0.f);
        for (int i = threadIdx.x; i < blocks; i += 32 * kWarps) sx[m * blocks + i] = 127;
      } else if (a.xtype == ROT_TYPE_F32) {
        round_row<float>(a, m, xs, sx, kpad);
      } else if (a.xtype == ROT_TYPE_F16) {
        round_row<__half>(a, m, xs, sx, kpad);
      } else {
        round_row<__nv_bfloat16>(a, m, xs, sx, kpad);
      }
    }
  }
  __syncthreads();

  float acc[R][M];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) acc[r][m] = 0.f;
  for (int sd = s0; sd < s1; sd += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int s = sd + d, k = s * kSpan + lane * 16;
      uint4 w[R];
      int e[R];
#pragma unroll
      for (int r = 0; r < R; ++r) w[r] = wv[d][r], e[r] = we[d][r];
      fetch(s + D, wv[d], we[d]);
      if (s >= s1 || k >= a.K) continue;
      float2 xf[M][8];
#pragma unroll
      for (int m = 0; m < M; ++m) x_run(xs, m * kpad + k, xf[m]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float2 wf[8];
        w_run(w[r], a.w5, wf);
#pragma unroll
        for (int m = 0; m < M; ++m)
          acc[r][m] += scaled(dot16(wf, xf[m]), e[r], sx[m * blocks + k / 128]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float v = warp_sum(acc[r][m]);
      if (lane == 0) join[warp][r][m] = v;
    }
  __syncthreads();
  // one thread per result of the CTA
  for (int i = threadIdx.x; i < kWarps / a.share * R * M; i += 32 * kWarps) {
    const int m = i % M, r = i / M % R, g = i / (M * R);
    const int n = (blockIdx.x * (kWarps / a.share) + g) * R + r;
    if (m >= a.M || n >= a.N) continue;
    float v = 0.f;
    for (int q = 0; q < a.share; ++q) v += join[g * a.share + q][r][m];
    const int64_t o = m * a.ldy + n;
    if (a.ytype == ROT_TYPE_F32)
      ((float*)a.y)[o] = a.accumulate ? ((float*)a.y)[o] + v : v;
    else if (a.ytype == ROT_TYPE_F16)
      ((__half*)a.y)[o] = __float2half_rn(v);
    else
      ((__nv_bfloat16*)a.y)[o] = __float2bfloat16_rn(v);
  }
}

template <int M>
int launch_few(const Few& a, cudaStream_t s) {
  static const cudaError_t attr = cudaFuncSetAttribute(
      fp8_few_kernel<M>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
  if (attr != cudaSuccess) return ROT_ECUDA;
  const int kpad = (a.K + 127) / 128 * 128;
  const size_t smem = ((size_t)M * kpad * 2 + M * (kpad / 128) + 15) / 16 * 16;
  const int per_cta = kWarps / a.share * kCols;
  ProfScope prof(ROT_PROF_GEMM_F8, 2.0 * a.M * (double)a.N * a.K, s);
  return launch_behind(fp8_few_kernel<M>, (unsigned)((a.N + per_cta - 1) / per_cta), 32 * kWarps,
                       smem, s, a);
}

}  // namespace

// Where the kernel above takes a product: few rows, whose 16-bit copy fits
// shared memory twice per SM.
bool fp8_few(int64_t M, int64_t K) {
  const int64_t kpad = (K + 127) / 128 * 128;
  return M <= kFewRows && M * (kpad * 2 + kpad / 128) + 15 <= kMaxShared;
}

int fp8_few_product(const Prod& p, const void* x, int64_t ldx, int32_t xtype, cudaStream_t s) {
  Few a;
  a.w = p.b, a.sw = p.sb, a.x = x, a.sx = p.sa, a.y = p.c;
  a.ldw = p.ldb, a.ldsw = p.ldsb, a.ldx = ldx, a.ldsx = p.ldsa, a.ldy = p.ldc;
  a.M = p.M, a.N = p.N, a.K = p.K, a.xtype = xtype, a.ytype = p.ctype;
  a.w5 = p.b5, a.wsh = p.bsh, a.xsh = p.ash, a.accumulate = p.accumulate;
  // warps per row of W, while there are SMs (16 warps each) without work and K for them
  a.share = 1;
  const int steps = (p.K + kSpan - 1) / kSpan;
  while (a.share < kWarps && a.share < steps &&
         (int64_t)(p.N + kCols - 1) / kCols * a.share * 2 <= 16ll * sm_count())
    a.share *= 2;
  return p.M <= 1 ? launch_few<1>(a, s) : launch_few<2>(a, s);
}

}  // namespace ops
}  // namespace rot
