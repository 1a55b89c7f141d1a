// 8-bit matrices with power-of-two block scales (include/rot_ops.h):
// quantisation, and the product's entry point (its kernels: ops_fp8_gemm.cu).
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

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
  int wide;          // q's rows are 16-byte aligned
};
// Two matrices in one launch: CTAs up to `first` take the one, the others the
// other.
struct QuantPair {
  Quant m[2];
  unsigned first;
};

// Two values as 8-bit floats, the first in the low byte.
template <bool E5>
__device__ __forceinline__ uint32_t pair_f8(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, E5 ? __NV_E5M2 : __NV_E4M3);
}

// Element k of values as loaded: 16-bit ones two to a word (even k in the low
// half).
template <class T>
__device__ __forceinline__ float element(const uint32_t* w, int k) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(w[k]);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    return __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
  } else {
    const uint32_t v = w[k / 2];
    return __half2float(__ushort_as_half((unsigned short)(k & 1 ? v >> 16 : v & 0xFFFFu)));
  }
}
template <class T>
__device__ __forceinline__ uint32_t magnitude_bits(const uint32_t* w, int k) {
  return sizeof(T) == 4 ? w[k] & 0x7FFFFFFFu : w[k / 2] >> (16 * (k & 1)) & 0x7FFFu;
}
// the largest magnitudes of two words (of each half, for 16-bit values)
template <class T>
__device__ __forceinline__ uint32_t word_max(uint32_t m, uint32_t w) {
  return sizeof(T) == 4 ? max(m, w & 0x7FFFFFFFu) : __vmaxu2(m, w & 0x7FFF7FFFu);
}
template <class T>
__device__ __forceinline__ uint32_t halves_max(uint32_t m) {
  return sizeof(T) == 4 ? m : max(m & 0xFFFFu, m >> 16);
}
// Run of N elements from p as words (N * sizeof(T) a multiple of 16), elements
// from n on as 0.
template <class T, int N, bool VEC>
__device__ __forceinline__ void load_words(const T* p, int64_t n, uint32_t* w) {
  constexpr int W = N * sizeof(T) / 4;
  if (VEC && n >= N) {
#pragma unroll
    for (int k = 0; k < W; k += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + k);
      w[k] = q.x, w[k + 1] = q.y, w[k + 2] = q.z, w[k + 3] = q.w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = 0u;
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k < n) {
      if constexpr (sizeof(T) == 4)
        w[k] = __float_as_uint(p[k]);
      else
        w[k / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[k] << (16 * (k & 1));
    }
}
// Four values under a scale as 8-bit floats.  The conversion saturates
// infinities; with FIX they become NaN by hand, as NaN stays.
template <bool E5, bool FIX>
__device__ __forceinline__ uint32_t four_f8(float f0, float f1, float f2, float f3, float s) {
  float2 lo = mul2(make_float2(f0, f1), both(s)), hi = mul2(make_float2(f2, f3), both(s));
  if (FIX) {
    if (!(fabsf(f0) < INFINITY)) lo.x = NAN;
    if (!(fabsf(f1) < INFINITY)) lo.y = NAN;
    if (!(fabsf(f2) < INFINITY)) hi.x = NAN;
    if (!(fabsf(f3) < INFINITY)) hi.y = NAN;
  }
  return pair_f8<E5>(lo.x, lo.y) | pair_f8<E5>(hi.x, hi.y) << 16;
}

// |x| as an ordered whole number of the type's bits, and back as a float.
template <class T>
__device__ __forceinline__ float magnitude(uint32_t bits) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(bits << 16);
  return __half2float(__ushort_as_half((unsigned short)bits));
}
template <class T>
constexpr uint32_t kInfBits = sizeof(T) == 4                             ? 0x7F800000u
                              : std::is_same<T, __nv_bfloat16>::value ? 0x7F80u
                                                                      : 0x7C00u;

constexpr int kQ = 128;      // a block's edge
constexpr int kPitch = 144;  // bytes between the staged rows of the transposed tile

// Rows alone, one scale for each row and 128 columns: HBM bound, nothing to
// exchange but the maxima of eight threads, which hold 16 elements of a block
// each.  8192 x 4096 in bfloat16: 19 us, 5.2 TB/s.
template <class T, bool VEC, bool E5>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __grid_constant__ Quant a) {
  const uint32_t blocks = (uint32_t)((a.cols + 127) / 128), total = (uint32_t)a.rows * blocks;
  const int v = threadIdx.x % 8;
  for (uint32_t b = blockIdx.x * 32 + threadIdx.x / 8; b < (total + 3) / 4 * 4;
       b += gridDim.x * 32) {  // (whole warps: four blocks each)
    const uint32_t at = min(b, total - 1), r = at / blocks, j = at - r * blocks;
    const int64_t row = r, c = (int64_t)j * 128 + 16 * v;
    uint32_t x[4 * sizeof(T)];
    load_words<T, 16, VEC>((const T*)a.x + row * a.ldx + c, a.cols - c, x);
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < (int)(4 * sizeof(T)); ++i) most = word_max<T>(most, x[i]);
    most = halves_max<T>(most);
    const bool odd = most >= kInfBits<T>;  // a NaN or an infinity among the 16
    if (odd) {
      most = 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t m = magnitude_bits<T>(x, i);
        most = max(most, m >= kInfBits<T> ? 0u : m);
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (b >= total) continue;
    const int e = scale_byte(magnitude<T>(most), E5);
    const float inv = inverse_scale(e);
    if (v == 0) a.s[j * a.lds + row] = (uint8_t)e;
    uint32_t w[4];
    auto convert = [&](auto fix) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = four_f8<E5, decltype(fix)::value>(element<T>(x, 4 * i), element<T>(x, 4 * i + 1),
                                                 element<T>(x, 4 * i + 2), element<T>(x, 4 * i + 3),
                                                 inv);
    };
    if (odd)
      convert(std::true_type());
    else
      convert(std::false_type());
    uint8_t* o = a.q + row * a.ldq + c;
    if (c + 16 <= a.cols && a.wide) {
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < a.cols) o[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
    }
  }
}

// HBM bound (one read of x, one or two bytes written per element); 4099 x 6144
// in both orientations: 21 us, 4.8 TB/s.  A 128 x
// 128 tile per CTA, 256 threads: thread (g = t / 16, v = t % 16) holds rows
// 8 g .. 8 g + 7 of columns 8 v .. 8 v + 7, so both orientations' runs of
// eight are in one thread.  Maxima are taken on the bits of |x|; a row's 16
// threads join by shuffles, a column's through shared memory.  The rows go
// out as 8 bytes per thread (128 per row), the transposed tile through shared
// memory as 16.
template <class T, bool VEC, bool E5>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 2 : 4)
    quantize_kernel(const __grid_constant__ QuantPair pair) {
  const Quant& a = pair.m[blockIdx.x >= pair.first];
  const unsigned block = blockIdx.x - (blockIdx.x >= pair.first ? pair.first : 0u);
  __shared__ __align__(16) uint32_t colmax[16][kQ];
  __shared__ __align__(16) uint8_t colscale[kQ];
  __shared__ uint32_t wide[8];
  __shared__ __align__(16) uint8_t tile[kQ * kPitch];
  constexpr int W = 8 * sizeof(T) / 4;
  const int64_t tiles_c = (a.cols + kQ - 1) / kQ;
  const int64_t tr = block / tiles_c, tc = block % tiles_c;  // tile row, column
  const int64_t r0 = tr * kQ, c0 = tc * kQ;
  const int g = threadIdx.x / 16, v = threadIdx.x % 16;
  const int64_t r = r0 + 8 * g, c = c0 + 8 * v;
  uint32_t x[8][W];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load_words<T, 8, VEC>((const T*)a.x + (r + i) * a.ldx + c, r + i < a.rows ? a.cols - c : 0, x[i]);
  // largest |x| of each row and column of the piece
  uint32_t rm[8], cm[8];
  bool odd;  // a NaN or an infinity in the piece
  {
    uint32_t cw[W], all = 0u;
#pragma unroll
    for (int k = 0; k < W; ++k) cw[k] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0u;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        m = word_max<T>(m, x[i][k]);
        cw[k] = word_max<T>(cw[k], x[i][k]);
      }
      rm[i] = halves_max<T>(m);
      all = max(all, rm[i]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      cm[k] = sizeof(T) == 4 ? cw[k % W] : (k & 1 ? cw[k / 2 % W] >> 16 : cw[k / 2 % W] & 0xFFFFu);
    odd = all >= kInfBits<T>;
    if (odd) {  // over the finite ones
#pragma unroll
      for (int k = 0; k < 8; ++k) rm[k] = cm[k] = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t b = magnitude_bits<T>(x[i], k);
          if (b >= kInfBits<T>) b = 0u;
          rm[i] = max(rm[i], b);
          cm[k] = max(cm[k], b);
        }
    }
  }
  // a whole tile, every access wide
  const bool whole = a.wide && r0 + kQ <= a.rows && c0 + kQ <= a.cols;
  auto put_rows = [&](const float (&ri)[8]) {
    auto convert = [&](int i, uint32_t (&o)[2], auto fix) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 4 * h;
        o[h] = four_f8<E5, decltype(fix)::value>(element<T>(x[i], k), element<T>(x[i], k + 1),
                                                 element<T>(x[i], k + 2), element<T>(x[i], k + 3),
                                                 ri[i]);
      }
    };
    uint8_t* p = a.q + r * a.ldq + c;
    if (whole && !odd) {
#pragma unroll
      for (int i = 0; i < 8; ++i, p += a.ldq) {
        uint32_t o[2];
        convert(i, o, std::false_type());
        *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i, p += a.ldq) {
      if (r + i >= a.rows) continue;
      uint32_t o[2];
      convert(i, o, std::true_type());
      if (a.wide && c + 8 <= a.cols) {
        *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
        continue;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < a.cols) p[k] = (uint8_t)(o[k / 4] >> (8 * (k & 3)));
    }
  };
  float ri[8], ci[8];  // inverse scales of this thread's rows and columns
  if (a.square) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x % 32 == 0) wide[threadIdx.x / 32] = m;
    __syncthreads();
    m = wide[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, wide[i]);
    const int b = scale_byte(magnitude<T>(m), E5);
#pragma unroll
    for (int i = 0; i < 8; ++i) ri[i] = ci[i] = inverse_scale(b);
    if (threadIdx.x == 0) {
      if (a.q) a.s[tc * a.lds + tr] = (uint8_t)b;
      if (a.qt) a.st[tr * a.ldst + tc] = (uint8_t)b;
    }
    if (a.q) put_rows(ri);
  } else {
    if (a.qt) {
      uint4* p = reinterpret_cast<uint4*>(&colmax[g][8 * v]);
      p[0] = make_uint4(cm[0], cm[1], cm[2], cm[3]);
      p[1] = make_uint4(cm[4], cm[5], cm[6], cm[7]);
      __syncthreads();
      if (threadIdx.x < kQ) {
        uint32_t m = colmax[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < 16; ++i) m = max(m, colmax[i][threadIdx.x]);
        const int b = scale_byte(magnitude<T>(m), E5);
        colscale[threadIdx.x] = (uint8_t)b;
        if (c0 + threadIdx.x < a.cols) a.st[tr * a.ldst + c0 + threadIdx.x] = (uint8_t)b;
      }
    }
    if (a.q) {
      // the largest of each row over its 16 threads, two rows to a word where
      // they fit; thread v works out row v's scale for all of them
      uint32_t mine = 0u;
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t m = rm[i];
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (v == i) mine = m;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t m = rm[2 * i] | rm[2 * i + 1] << 16;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (v / 2 == i) mine = v & 1 ? m >> 16 : m & 0xFFFFu;
        }
      }
      const int b = scale_byte(magnitude<T>(mine), E5);
      if (v < 8 && r + v < a.rows) a.s[tc * a.lds + r + v] = (uint8_t)b;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        ri[i] = inverse_scale(__shfl_sync(0xffffffffu, b, (threadIdx.x & 16) + i));
      put_rows(ri);
    }
    if (a.qt) {
      __syncthreads();
      const uint2 b = *reinterpret_cast<const uint2*>(&colscale[8 * v]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        ci[k] = inverse_scale((int)((k < 4 ? b.x : b.y) >> (8 * (k & 3)) & 0xFFu));
    }
  }
  if (a.qt) {
    // column 8 v + k is staged as row 16 k + v, so that a warp's writes spread
    // over the banks
    auto stage = [&](auto fix) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = 4 * h;
          o[h] = four_f8<E5, decltype(fix)::value>(element<T>(x[i], k), element<T>(x[i + 1], k),
                                                   element<T>(x[i + 2], k),
                                                   element<T>(x[i + 3], k), ci[k]);
        }
        *reinterpret_cast<uint2*>(&tile[(16 * k + v) * kPitch + 8 * g]) = make_uint2(o[0], o[1]);
      }
    };
    if (odd)
      stage(std::true_type());
    else
      stage(std::false_type());
    __syncthreads();
    const bool run16 = rows16(a.qt, a.ldqt, 1);
    const int64_t rr = r0 + 16 * (threadIdx.x % 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = threadIdx.x / 8 + 32 * i;
      if (c0 + col >= a.cols || rr >= a.rows) continue;
      const uint4 o = *reinterpret_cast<const uint4*>(
          &tile[(16 * (col % 8) + col / 8) * kPitch + 16 * (threadIdx.x % 8)]);
      uint8_t* p = a.qt + (c0 + col) * a.ldqt + rr;
      if (run16 && rr + 16 <= a.rows) {
        *reinterpret_cast<uint4*>(p) = o;
      } else {
        const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (rr + k < a.rows) p[k] = (uint8_t)(w[k / 4] >> (8 * (k & 3)));
      }
    }
  }
}

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m; }
constexpr int64_t kMost = (int64_t(1) << 31) - 256;

inline int64_t tiles_of(const Quant& a) { return up(a.rows, kQ) * up(a.cols, kQ); }
template <class T>
bool vec_of(const Quant& a) {
  return rows16(a.x, a.ldx, sizeof(T));
}
template <class T>
double bytes_of(const Quant& a) {
  return (double)a.rows * a.cols * (sizeof(T) + (a.q != nullptr) + (a.qt != nullptr));
}

template <class T>
int launch_tiles(const QuantPair& p, unsigned grid, cudaStream_t s) {
  const bool vec = vec_of<T>(p.m[0]);
  auto k = p.m[0].e5m2 ? (vec ? quantize_kernel<T, true, true> : quantize_kernel<T, false, true>)
                       : (vec ? quantize_kernel<T, true, false> : quantize_kernel<T, false, false>);
  k<<<grid, 256, 0, s>>>(p);
  return launched();
}

template <class T>
int launch_quantize(const Quant& a, cudaStream_t s) {
  const unsigned grid = (unsigned)tiles_of(a);
  const bool vec = vec_of<T>(a);
  ProfScope prof(ROT_PROF_ELEMENTWISE, bytes_of<T>(a), s);
  const int64_t row_blocks = a.rows * ((a.cols + 127) / 128);
  if (!a.qt && !a.square && row_blocks < (1ll << 30)) {
    const int64_t most = (row_blocks + 31) / 32;
    const unsigned ctas = (unsigned)std::min<int64_t>(most, 16ll * sm_count());
    auto k = a.e5m2 ? (vec ? quantize_rows_kernel<T, true, true> : quantize_rows_kernel<T, false, true>)
                    : (vec ? quantize_rows_kernel<T, true, false> : quantize_rows_kernel<T, false, false>);
    k<<<ctas, 256, 0, s>>>(a);
    return launched();
  }
  return launch_tiles<T>({{a, a}, grid}, grid, s);
}

// Both orientations' tiles of a (and of b) in one launch where they load
// alike: small matrices' launches are most of their time (436 x 2714 and 436 x
// 203: 6 us, 18 in two).
template <class T>
int launch_both(const Quant& a, const Quant& b, cudaStream_t s) {
  const int64_t grid = tiles_of(a) + tiles_of(b);
  if (vec_of<T>(a) != vec_of<T>(b) || grid > 0x7FFFFFFF) {
    const int e = launch_quantize<T>(a, s);
    return e != ROT_OK ? e : launch_quantize<T>(b, s);
  }
  ProfScope prof(ROT_PROF_ELEMENTWISE, bytes_of<T>(a) + bytes_of<T>(b), s);
  return launch_tiles<T>({{a, b}, (unsigned)tiles_of(a)}, (unsigned)grid, s);
}

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
             ldst, format == ROT_TYPE_E5M2, block_rows == kQ, rows16(data, ldq, 1)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return guarded([&] {
    if (type == ROT_TYPE_F32) return launch_quantize<float>(a, s);
    if (type == ROT_TYPE_F16) return launch_quantize<__half>(a, s);
    return launch_quantize<__nv_bfloat16>(a, s);
  });
}

uint64_t rot_fp8_gemm_work_bytes(int64_t M, int64_t N, int64_t K) {
  return fp8_few(M, N, K) ? 0 : fp8_work_bytes(M, N, K);
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
  return guarded([&] {
    if (fp8_few(M, N, K)) return fp8_few_product(p, a, lda, a_format, s);
    return fp8_product(p, reinterpret_cast<int*>(status), s);
  });
}

namespace {

// An 8-bit matrix in a workspace: rows x cols, one scale per row and 128
// columns.
struct Held {
  uint8_t *q, *s;
  int64_t ld, lds;
};
struct Carve {
  char* base;
  uint64_t at = 0;
  char* take(uint64_t bytes) {
    char* p = base ? base + at : nullptr;
    at += align256(bytes);
    return p;
  }
  Held matrix(int64_t rows, int64_t cols) {
    Held h;
    h.ld = up(cols, kQ) * kQ;  // (rows of whole 128-byte lines, as the product's loads take them)
    h.lds = rows;
    h.q = reinterpret_cast<uint8_t*>(take((uint64_t)rows * h.ld));
    h.s = reinterpret_cast<uint8_t*>(take((uint64_t)rows * up(cols, kQ)));
    return h;
  }
};

bool bad_layer(int64_t tokens, int64_t inner, int64_t outer) {
  return tokens < 0 || inner < 0 || outer < 0 || tokens > kMost || inner > kMost || outer > kMost;
}
bool bad_work(const void* work, uint64_t have, uint64_t need) {
  return need > 0 && (!work || have < need || (reinterpret_cast<uintptr_t>(work) & 255));
}

}  // namespace

uint64_t rot_fp8_linear_work_bytes(int64_t tokens, int64_t inner, int64_t outer) {
  if (bad_layer(tokens, inner, outer) || outer == 0 || fp8_self_rounded(tokens, outer, inner)) return 0;
  Carve c = {nullptr};
  c.matrix(tokens, inner);
  c.take(rot_fp8_gemm_work_bytes(tokens, outer, inner));
  return c.at;
}

int rot_fp8_linear(int64_t tokens, int64_t inner, int64_t outer, const void* x, int64_t ldx,
                   int32_t type, const void* w, int64_t ldw, int32_t w_format,
                   const uint8_t* w_scale, int64_t w_lds, int32_t w_block_rows, void* y,
                   int64_t ldy, void* work, uint64_t work_bytes, int32_t* status, void* stream) {
  if (bad_layer(tokens, inner, outer) || !float_type(type) || ldx < inner || ldy < outer ||
      (tokens > 0 && inner > 0 && !x) ||
      bad_operand(w, ldw, w_format, w_scale, w_lds, w_block_rows, outer, inner) ||
      (tokens > 0 && outer > 0 && !y) ||
      bad_work(work, work_bytes, rot_fp8_linear_work_bytes(tokens, inner, outer)))
    return ROT_EINVAL;
  if (tokens == 0 || outer == 0) return ROT_OK;
  if (fp8_self_rounded(tokens, outer, inner) && inner > 0) {
    const int dev = check_device();
    if (dev != ROT_OK) return dev;
    Prod p = {nullptr, (const uint8_t*)w, nullptr, w_scale, y, 0, ldw, 0, w_lds, ldy,
              (int)tokens, (int)outer, (int)inner, type, 0, 0, w_format == ROT_TYPE_E5M2,
              0, w_block_rows == 1 ? 0 : 7, nullptr};
    return guarded([&] { return fp8_few_product(p, x, ldx, type, static_cast<cudaStream_t>(stream)); });
  }
  Carve c = {static_cast<char*>(work)};
  const Held q = c.matrix(tokens, inner);
  const uint64_t more = rot_fp8_gemm_work_bytes(tokens, outer, inner);
  int e = rot_fp8_quantize(x, ldx, tokens, inner, type, ROT_TYPE_E4M3, 1, q.q, q.ld, q.s, q.lds,
                           nullptr, 0, nullptr, 0, stream);
  if (e != ROT_OK) return e;
  return rot_fp8_gemm(tokens, outer, inner, q.q, q.ld, ROT_TYPE_E4M3, q.s, q.lds, 1, w, ldw,
                      w_format, w_scale, w_lds, w_block_rows, y, ldy, type, 0, c.take(more), more,
                      status, stream);
}

uint64_t rot_fp8_linear_backward_work_bytes(int64_t tokens, int64_t inner, int64_t outer) {
  if (bad_layer(tokens, inner, outer)) return 0;
  Carve c = {nullptr};
  c.matrix(tokens, outer);
  c.matrix(outer, tokens);
  c.matrix(inner, tokens);
  c.take(std::max(rot_fp8_gemm_work_bytes(tokens, inner, outer), rot_fp8_gemm_work_bytes(outer, inner, tokens)));
  return c.at;
}

int rot_fp8_linear_backward(int64_t tokens, int64_t inner, int64_t outer, const void* dy,
                            int64_t lddy, const void* x, int64_t ldx, int32_t type,
                            const void* wt, int64_t ldwt, int32_t wt_format,
                            const uint8_t* wt_scale, int64_t wt_lds, int32_t wt_block_rows,
                            void* dx, int64_t lddx, float* dw, int64_t lddw, int32_t accumulate,
                            void* work, uint64_t work_bytes, int32_t* status, void* stream) {
  if (bad_layer(tokens, inner, outer) || !float_type(type) || lddy < outer || ldx < inner ||
      lddx < inner || lddw < inner || (tokens > 0 && outer > 0 && !dy) ||
      (tokens > 0 && inner > 0 && (!x || !dx)) || (inner > 0 && outer > 0 && !dw) ||
      bad_operand(wt, ldwt, wt_format, wt_scale, wt_lds, wt_block_rows, inner, outer) ||
      bad_work(work, work_bytes, rot_fp8_linear_backward_work_bytes(tokens, inner, outer)))
    return ROT_EINVAL;
  Carve c = {static_cast<char*>(work)};
  const Held d = c.matrix(tokens, outer), dt = c.matrix(outer, tokens), xt = c.matrix(inner, tokens);
  const uint64_t more =
      std::max(rot_fp8_gemm_work_bytes(tokens, inner, outer), rot_fp8_gemm_work_bytes(outer, inner, tokens));
  char* part = c.take(more);
  int e = ROT_OK;
  if (tokens > 0 && inner > 0 && outer > 0) {
    if (up(tokens, kQ) * up(std::max(inner, outer), kQ) > 0x7FFFFFFF) return ROT_EINVAL;
    e = check_device();
    if (e != ROT_OK) return e;
    const Quant qd = {dy, d.q, d.s, dt.q, dt.s, lddy, tokens, outer, d.ld, d.lds, dt.ld, dt.lds,
                      0, 0, rows16(d.q, d.ld, 1)};
    const Quant qx = {x, nullptr, nullptr, xt.q, xt.s, ldx, tokens, inner, 0, 0, xt.ld, xt.lds,
                      0, 0, 0};
    e = guarded([&] {
      cudaStream_t s = static_cast<cudaStream_t>(stream);
      if (type == ROT_TYPE_F32) return launch_both<float>(qd, qx, s);
      if (type == ROT_TYPE_F16) return launch_both<__half>(qd, qx, s);
      return launch_both<__nv_bfloat16>(qd, qx, s);
    });
  }
  if (e != ROT_OK) return e;
  // Neither product fills its last round of SMs (4099 x 2048 x 6144: 2.4 and
  // 3.5 rounds): in one launch the second starts where the first leaves them (82
  // us for both, 101 in two launches).
  if (fp8_takes_two(tokens, inner, outer, outer, inner, tokens)) {
    const Prod px = {d.q, (const uint8_t*)wt, d.s, wt_scale, dx, d.ld, ldwt, d.lds, wt_lds, lddx,
                     (int)tokens, (int)inner, (int)outer, type, 0, 0, wt_format == ROT_TYPE_E5M2,
                     0, wt_block_rows == 1 ? 0 : 7, nullptr};
    const Prod pw = {dt.q, xt.q, dt.s, xt.s, dw, dt.ld, xt.ld, dt.lds, xt.lds, lddw,
                     (int)outer, (int)inner, (int)tokens, ROT_TYPE_F32, accumulate, 0, 0,
                     0, 0, nullptr};
    return guarded([&] {
      return fp8_two_products(px, pw, reinterpret_cast<int*>(status),
                              static_cast<cudaStream_t>(stream));
    });
  }
  e = rot_fp8_gemm(tokens, inner, outer, d.q, d.ld, ROT_TYPE_E4M3, d.s, d.lds, 1, wt, ldwt,
                   wt_format, wt_scale, wt_lds, wt_block_rows, dx, lddx, type, 0, part, more, status,
                   stream);
  if (e != ROT_OK) return e;
  return rot_fp8_gemm(outer, inner, tokens, dt.q, dt.ld, ROT_TYPE_E4M3, dt.s, dt.lds, 1, xt.q,
                      xt.ld, ROT_TYPE_E4M3, xt.s, xt.lds, 1, dw, lddw, ROT_TYPE_F32, accumulate,
                      part, more, status, stream);
}

}  // extern "C"
