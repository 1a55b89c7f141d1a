// AdamW over many tensors and the norm of their gradients (include/rot_ops.h).
// Bound by HBM: every array is read once and written once.
//
// A launch takes a table of tensors as its parameter (nothing is copied to the
// device, and a captured launch keeps its table).  A block takes kChunk
// elements of one tensor, found by bisection in the tensors' first chunks.  A
// warp takes 128 consecutive elements at a time, four to a lane: the elements
// that share a scale in 8 bits, and one call of the generator to a lane.
#include <algorithm>
#include <cmath>
#include <vector>

#include "ops_common.cuh"
#include "profile.h"

namespace rot {
namespace ops {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAhead = 4;                        // times 128 elements that a warp loads at once
constexpr int kChunk = kWarps * kAhead * 128;    // elements to a block

// What is stepped: p itself, rounded at random to bfloat16, or a float32
// master with p as its 16-bit copy.
enum Kept { kF32 = 0, kBf16Random = 1, kBf16Master = 2, kF16Master = 3 };

struct Entry {
  void* p;
  const void* g;
  void *m, *v;
  uint8_t *ms, *vs;
  float* master;
  int64_t n;
  uint64_t word;   // the generator's counter of its first element (index / 4)
  int32_t g_type;
  int32_t whole;   // vector accesses reach all its arrays
};

struct Hyper {
  float lr, beta1, rest1, beta2, rest2, eps, decay;  // decay: 1 - lr weight_decay
  float step_size, inv_root;                         // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float log1, log2, weight_decay, scale, max_norm;
  const float* lr_device;
  const int64_t* step_device;
  const float* norm;
  uint64_t step;
  uint32_t key[10][2];
};

template <int CAP>
struct Table {
  Hyper h;
  int32_t count;
  uint32_t first[CAP];  // chunk that each tensor begins with
  Entry e[CAP];
};
constexpr int kFew = 12, kMany = 360;
static_assert(sizeof(Table<kMany>) <= 32764, "a kernel's parameters");

template <int CAP>
__device__ __forceinline__ int tensor_of(const uint32_t (&first)[CAP], int count, uint32_t chunk) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Four elements from i on, of which `left` are there (the rest 0).
template <class T>
__device__ __forceinline__ Run<T, 4> four(const void* p, int64_t i, int left, bool whole) {
  const T* q = (const T*)p + i;
  if (whole && left >= 4) return *reinterpret_cast<const Run<T, 4>*>(q);
  Run<T, 4> r{};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < left) r.v[k] = q[k];
  return r;
}
template <class T>
__device__ __forceinline__ void put_four(void* p, int64_t i, int left, bool whole,
                                         const Run<T, 4>& r) {
  T* q = (T*)p + i;
  if (whole && left >= 4) {
    *reinterpret_cast<Run<T, 4>*>(q) = r;
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < left) q[k] = r.v[k];
}

// Four gradients as they came, of any type.
struct Raw4 {
  uint32_t w[4];
};
__device__ __forceinline__ Raw4 four_raw(const Entry& e, int64_t i, int left) {
  Raw4 r{};
  if (e.g_type == ROT_TYPE_F32) {
    const Run<uint32_t, 4> f = four<uint32_t>(e.g, i, left, e.whole);
#pragma unroll
    for (int k = 0; k < 4; ++k) r.w[k] = f.v[k];
  } else {
    const Run<uint16_t, 4> f = four<uint16_t>(e.g, i, left, e.whole);
    r.w[0] = f.v[0] | (uint32_t)f.v[1] << 16;
    r.w[1] = f.v[2] | (uint32_t)f.v[3] << 16;
  }
  return r;
}
__device__ __forceinline__ void floats_of(const Raw4& r, int type, float (&f)[4]) {
  if (type == ROT_TYPE_F32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(r.w[k]);
  } else if (type == ROT_TYPE_BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      f[k] = __uint_as_float(k & 1 ? r.w[k / 2] & 0xffff0000u : r.w[k / 2] << 16);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      f[k] = __half2float(__ushort_as_half((unsigned short)(r.w[k / 2] >> (k & 1 ? 16 : 0))));
  }
}

// ---- 8 bits ----

// 2^(byte - 127) (byte 0: subnormal; 255: NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 1u << 22 : byte == 255 ? 0x7fc00000u : byte << 23);
}
__device__ __forceinline__ void values8(uint32_t q, float scale, float (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(h)
        : "r"(k ? q >> 16 : q & 0xffffu));
    f[2 * k] = __half2float(__ushort_as_half((unsigned short)h)) * scale;
    f[2 * k + 1] = __half2float(__ushort_as_half((unsigned short)(h >> 16))) * scale;
  }
}

// Four numbers of a warp's 128 in E4M3, rounded by each one's 16 random bits
// (the low half of its word), and the scale byte.  root: nothing above 0
// becomes 0.
//
// A number's bits times 2^-120 as float32 are E4M3's above 20 more (their
// least exponents meet there, below it both count in fixed steps), so that an
// addition to the bits and a shift round it at any size.
template <bool ROOT>
__device__ __forceinline__ uint32_t rounded8(const float (&x)[4], const uint32_t (&word)[4],
                                             uint32_t& byte) {
  uint32_t b[4], top = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    b[k] = __float_as_uint(x[k]);
    top = max(top, b[k] & 0x7fffffffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const bool odd = top >= 0x7f800000u;  // NaN or infinity among the 128
  if (odd) {
    top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = b[k] & 0x7fffffffu;
      if (a < 0x7f800000u) top = max(top, a);
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  // top = (1 + f) 2^(t - 127) <= 448 2^(byte - 127), 448 = 1.75 2^8
  const int t = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
  byte = (uint32_t)max(t, 0);
  const float back = __uint_as_float((254u - byte) << 23);
  uint32_t out = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t y = __float_as_uint(x[k] * back * 0x1p-120f);
    const uint32_t s = y + ((word[k] & 0xffffu) << 4) + 8u;
    uint32_t code = s >> 20 & 0x7fu;
    if (ROOT) code = max(code, (uint32_t)(x[k] > 0.f));
    code |= y >> 24 & 0x80u;
    if (odd && (b[k] & 0x7fffffffu) >= 0x7f800000u) code = 0x7fu;
    out |= code << (8 * k);
  }
  return out;
}

__device__ __forceinline__ void words_of(const Hyper& h, uint64_t counter, uint64_t offset,
                                         uint32_t (&w)[4]) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint2 a = mul_wide(c0, kPhiloxM0), b = mul_wide(c2, kPhiloxM1);
    c0 = b.y ^ c1 ^ h.key[r][0];
    c1 = b.x;
    c2 = a.y ^ c3 ^ h.key[r][1];
    c3 = a.x;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

template <Kept KEPT>
struct Stepped {
  using T = float;
};
template <>
struct Stepped<kBf16Random> {
  using T = uint16_t;
};

template <Kept KEPT, bool EIGHT, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<CAP> a) {
  using P = typename Stepped<KEPT>::T;
  constexpr bool kWords = EIGHT || KEPT == kBf16Random;
  const Hyper& h = a.h;
  const Entry& e = a.e[tensor_of(a.first, a.count, blockIdx.x)];
  const int64_t start =
      (int64_t)(blockIdx.x - a.first[&e - a.e]) * kChunk + (threadIdx.x >> 5) * 128;
  const int lane = threadIdx.x & 31;
  void* const at = KEPT >= kBf16Master ? (void*)e.master : e.p;
  Raw4 rg[kAhead];
  Run<P, 4> rp[kAhead];
  Run<float, 4> rm[EIGHT ? 1 : kAhead], rv[EIGHT ? 1 : kAhead];
  uint32_t qm[EIGHT ? kAhead : 1], qv[EIGHT ? kAhead : 1];
  uint32_t sm[EIGHT ? kAhead : 1], sv[EIGHT ? kAhead : 1];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int64_t i = start + k * kWarps * 128 + lane * 4;
    const int left = (int)max((int64_t)0, min((int64_t)4, e.n - i));
    rg[k] = four_raw(e, i, left);
    rp[k] = four<P>(at, i, left, e.whole);
    if constexpr (EIGHT) {
      const Run<uint8_t, 4> x = four<uint8_t>(e.m, i, left, e.whole);
      const Run<uint8_t, 4> y = four<uint8_t>(e.v, i, left, e.whole);
      qm[k] = x.v[0] | x.v[1] << 8 | x.v[2] << 16 | (uint32_t)x.v[3] << 24;
      qv[k] = y.v[0] | y.v[1] << 8 | y.v[2] << 16 | (uint32_t)y.v[3] << 24;
      sm[k] = left > 0 ? e.ms[i / 128] : 0u;
      sv[k] = left > 0 ? e.vs[i / 128] : 0u;
    } else {
      rm[k] = four<float>(e.m, i, left, e.whole);
      rv[k] = four<float>(e.v, i, left, e.whole);
    }
  }
  float scale = h.scale;
  if (h.norm) {
    const float norm = fabsf(scale) * *h.norm;
    if (!isfinite(norm)) return;  // (the same for every thread)
    if (norm > h.max_norm) scale *= h.max_norm / norm;
  }
  float decay = h.decay, step_size = h.step_size, inv_root = h.inv_root;
  uint64_t t = h.step;
  if (h.lr_device || h.step_device) {
    const float lr = h.lr_device ? *h.lr_device : h.lr;
    if (h.step_device) t = (uint64_t)*h.step_device;
    if ((int64_t)t < 1) return;
    // 1 - beta^t = -(e^(t log beta) - 1)
    step_size = lr / -expm1f((float)(int64_t)t * h.log1);
    inv_root = 1.f / sqrtf(-expm1f((float)(int64_t)t * h.log2));
    decay = 1.f - lr * h.weight_decay;
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int64_t i = start + k * kWarps * 128 + lane * 4;
    const int left = (int)max((int64_t)0, min((int64_t)4, e.n - i));
    if (i - lane * 4 >= e.n) break;  // (the same for a warp)
    float g[4], m[4], v[4], r[4], p[4];
    floats_of(rg[k], e.g_type, g);
    if constexpr (EIGHT) {
      values8(qm[k], scale_of(sm[k]), m);
      values8(qv[k], scale_of(sv[k]), v);
    }
    uint32_t w[4];
    if constexpr (kWords) words_of(h, e.word + (uint64_t)i / 4, t, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!EIGHT) m[j] = rm[k].v[j], v[j] = rv[k].v[j];
      if constexpr (KEPT == kBf16Random)
        p[j] = __uint_as_float((uint32_t)rp[k].v[j] << 16);
      else
        p[j] = rp[k].v[j];
      if constexpr (EIGHT) v[j] = __fmul_rn(v[j], v[j]);
      g[j] = __fmul_rn(g[j], scale);
      // (products and sums rounded one by one: the 8-bit scales' borders are
      // then where the formula's float32 steps put them)
      m[j] = __fadd_rn(__fmul_rn(h.beta1, m[j]), __fmul_rn(h.rest1, g[j]));
      v[j] = __fadd_rn(__fmul_rn(h.beta2, v[j]), __fmul_rn(__fmul_rn(h.rest2, g[j]), g[j]));
      r[j] = __fsqrt_rn(v[j]);
      p[j] = p[j] * decay - __fdividef(step_size * m[j], r[j] * inv_root + h.eps);
    }
    if constexpr (EIGHT) {
      uint32_t bm, bv;
      const uint32_t nm = rounded8<false>(m, w, bm), nv = rounded8<true>(r, w, bv);
      Run<uint8_t, 4> x, y;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x.v[j] = (uint8_t)(nm >> 8 * j), y.v[j] = (uint8_t)(nv >> 8 * j);
      put_four<uint8_t>(e.m, i, left, e.whole, x);
      put_four<uint8_t>(e.v, i, left, e.whole, y);
      if (lane == 0) e.ms[i / 128] = (uint8_t)bm, e.vs[i / 128] = (uint8_t)bv;
    } else {
      Run<float, 4> x, y;
#pragma unroll
      for (int j = 0; j < 4; ++j) x.v[j] = m[j], y.v[j] = v[j];
      put_four<float>(e.m, i, left, e.whole, x);
      put_four<float>(e.v, i, left, e.whole, y);
    }
    if constexpr (KEPT == kBf16Random) {
      Run<uint16_t, 4> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t bits = __float_as_uint(p[j]);
        const bool fine = (bits & 0x7fffffffu) < 0x7f800000u;
        // (not finite: to nearest, which keeps a NaN one)
        o.v[j] = fine ? (uint16_t)((bits + (w[j] >> 16)) >> 16)
                      : __bfloat16_as_ushort(__float2bfloat16_rn(p[j]));
      }
      put_four<uint16_t>(e.p, i, left, e.whole, o);
    } else {
      Run<float, 4> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o.v[j] = p[j];
      put_four<float>(at, i, left, e.whole, o);
      if constexpr (KEPT == kBf16Master) {
        Run<__nv_bfloat16, 4> c;
#pragma unroll
        for (int j = 0; j < 4; ++j) c.v[j] = __float2bfloat16_rn(p[j]);
        put_four<__nv_bfloat16>(e.p, i, left, e.whole, c);
      } else if constexpr (KEPT == kF16Master) {
        Run<__half, 4> c;
#pragma unroll
        for (int j = 0; j < 4; ++j) c.v[j] = __float2half_rn(p[j]);
        put_four<__half>(e.p, i, left, e.whole, c);
      }
    }
  }
}

template <Kept KEPT, bool EIGHT, int CAP>
int launch_table(const Hyper& h, const Entry* e, int count, cudaStream_t s) {
  Table<CAP> t;
  t.h = h, t.count = count;
  uint64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    t.first[i] = (uint32_t)chunks;
    t.e[i] = e[i];
    chunks += (e[i].n + kChunk - 1) / kChunk;
  }
  adamw_kernel<KEPT, EIGHT, CAP><<<(unsigned)chunks, kThreads, 0, s>>>(t);
  return launched();
}

// Launches of at most kMany tensors (of 2^40 elements in all).
template <Kept KEPT, bool EIGHT>
int launch_adamw(const Hyper& h, const std::vector<Entry>& all, cudaStream_t s) {
  constexpr double each = KEPT == kF32 ? 8 : KEPT == kBf16Random ? 4 : 10;
  for (size_t at = 0; at < all.size();) {
    size_t end = at;
    double bytes = 0.0;
    while (end < all.size() && end - at < kMany) {
      bytes += all[end].n * (each + (all[end].g_type == ROT_TYPE_F32 ? 4 : 2) +
                             (EIGHT ? 4.03125 : 16.0));
      ++end;
    }
    ProfScope prof(ROT_PROF_ELEMENTWISE, bytes, s);
    const int n = (int)(end - at);
    const int e = n <= kFew ? launch_table<KEPT, EIGHT, kFew>(h, &all[at], n, s)
                            : launch_table<KEPT, EIGHT, kMany>(h, &all[at], n, s);
    if (e != ROT_OK) return e;
    at = end;
  }
  return ROT_OK;
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
int word_bytes(int32_t type) { return type == ROT_TYPE_F32 ? 16 : 8; }

// ---- norm ----

struct Square {
  const void* g;
  int64_t n;
  int32_t type, whole;
};
constexpr int kSquares = 1000, kSquareChunk = 8192, kSquareBlocks = 1024;
struct SquareTable {
  float* part;
  int32_t count;
  uint32_t chunks;
  uint32_t first[kSquares];
  Square e[kSquares];
};
static_assert(sizeof(SquareTable) <= 32764, "a kernel's parameters");

template <class T>
__device__ __forceinline__ float squares(const Square& e, int64_t i0, int64_t end) {
  constexpr int U = 16 / sizeof(T), N = kSquareChunk / (U * kThreads);
  const T* g = (const T*)e.g;
  float2 sum[2] = {both(0.f), both(0.f)};
  if (e.whole && end - i0 == kSquareChunk) {
    Run<T, U> r[N];
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = raw_run<T, U>(g, i0 + (n * kThreads + threadIdx.x) * U);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Vec<U> v = unpack<T, U>(r[n]);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) sum[k & 1] = fma2(v.p[k], v.p[k], sum[k & 1]);
    }
  } else {
    for (int64_t i = i0 + threadIdx.x; i < end; i += kThreads) {
      const float x = to_f32(g[i]);
      sum[0].x = fmaf(x, x, sum[0].x);
    }
  }
  return total(add2(sum[0], sum[1]));
}

// A block sums the squares of a run of chunks.
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ SquareTable a) {
  __shared__ float red[kWarps];
  const uint32_t c0 = (uint32_t)((uint64_t)a.chunks * blockIdx.x / gridDim.x);
  const uint32_t c1 = (uint32_t)((uint64_t)a.chunks * (blockIdx.x + 1) / gridDim.x);
  float sum = 0.f;
  int t = tensor_of(a.first, a.count, c0);
  for (uint32_t c = c0; c < c1; ++c) {
    while (t + 1 < a.count && a.first[t + 1] <= c) ++t;
    const Square& e = a.e[t];
    const int64_t i0 = (int64_t)(c - a.first[t]) * kSquareChunk;
    const int64_t end = min(i0 + kSquareChunk, e.n);
    if (e.type == ROT_TYPE_F32)
      sum += squares<float>(e, i0, end);
    else if (e.type == ROT_TYPE_BF16)
      sum += squares<__nv_bfloat16>(e, i0, end);
    else
      sum += squares<__half>(e, i0, end);
  }
  sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) sum += red[w];
    a.part[blockIdx.x] = sum;
  }
}

// The root of the parts' sum, in a fixed order.
__global__ void __launch_bounds__(1024) norm_root_kernel(const float* part, int parts,
                                                         float* norm) {
  __shared__ double red[32];
  wait_for_prior();
  double sum = 0.0;
  for (int p = threadIdx.x; p < parts; p += 1024) sum += (double)part[p];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) sum += red[w];
    *norm = (float)sqrt(sum);
  }
}

constexpr int64_t kMostElements = int64_t(1) << 40;  // of a call

}  // namespace
}  // namespace ops
}  // namespace rot

using namespace rot;
using namespace rot::ops;

extern "C" {

int rot_adamw_step(const rot_adamw_tensor* tensors, int32_t count, const rot_adamw_hyper* hyper,
                   void* stream) {
  if (count < 0 || (count > 0 && !tensors) || !hyper) return ROT_EINVAL;
  const rot_adamw_hyper& y = *hyper;
  for (double x : {y.lr, y.eps, y.weight_decay})
    if (!(x >= 0.0)) return ROT_EINVAL;
  for (double x : {y.beta1, y.beta2})
    if (!(x >= 0.0 && x < 1.0)) return ROT_EINVAL;
  if (!std::isfinite(y.scale) || (y.norm && !(y.max_norm > 0.0))) return ROT_EINVAL;
  if (!y.step_device && y.step < 1) return ROT_EINVAL;
  return guarded([&]() -> int {
    std::vector<Entry> of[4][2];
    std::vector<const void*> written;
    uint64_t words = 0;
    int64_t room = kMostElements;
    for (int32_t i = 0; i < count; ++i) {
      const rot_adamw_tensor& t = tensors[i];
      if (t.n < 0 || t.n > room || !float_type(t.p_type) || !float_type(t.g_type))
        return ROT_EINVAL;
      const bool eight = t.m_scale != nullptr;
      if (eight != (t.v_scale != nullptr)) return ROT_EINVAL;
      if (t.p_type == ROT_TYPE_F32 ? t.master != nullptr
                                   : t.p_type == ROT_TYPE_F16 && !t.master && t.n > 0)
        return ROT_EINVAL;
      room -= t.n;
      const uint64_t word = words;
      words += (uint64_t)((t.n + 127) / 128) * 32;
      if (t.n == 0) continue;
      const int state = eight ? 1 : 4;
      if (!t.p || !t.g || !t.m || !t.v || !aligned(t.p, type_bytes(t.p_type)) ||
          !aligned(t.g, type_bytes(t.g_type)) || !aligned(t.m, state) || !aligned(t.v, state) ||
          !aligned(t.master, 4))
        return ROT_EINVAL;
      for (const void* p : {(const void*)t.p, (const void*)t.m, (const void*)t.v,
                            (const void*)t.m_scale, (const void*)t.v_scale,
                            (const void*)t.master})
        if (p) written.push_back(p);
      const int kept = t.p_type == ROT_TYPE_F32    ? kF32
                       : t.p_type == ROT_TYPE_F16 ? kF16Master
                       : t.master                  ? kBf16Master
                                                   : kBf16Random;
      Entry e;
      e.p = t.p, e.g = t.g, e.m = t.m, e.v = t.v, e.ms = t.m_scale, e.vs = t.v_scale;
      e.master = t.master, e.n = t.n, e.word = word, e.g_type = t.g_type;
      e.whole = aligned(t.p, word_bytes(t.p_type)) && aligned(t.g, word_bytes(t.g_type)) &&
                aligned(t.m, 4 * state) && aligned(t.v, 4 * state) && aligned(t.master, 16);
      of[kept][eight].push_back(e);
    }
    std::sort(written.begin(), written.end());
    if (std::adjacent_find(written.begin(), written.end()) != written.end()) return ROT_EINVAL;
    if (written.empty()) return ROT_OK;
    const int dev = check_device();
    if (dev != ROT_OK) return dev;
    Hyper h;
    h.lr = (float)y.lr, h.eps = (float)y.eps, h.weight_decay = (float)y.weight_decay;
    h.beta1 = (float)y.beta1, h.rest1 = (float)(1.0 - y.beta1);
    h.beta2 = (float)y.beta2, h.rest2 = (float)(1.0 - y.beta2);
    h.decay = (float)(1.0 - y.lr * y.weight_decay);
    const double t = (double)std::max<int64_t>(y.step, 1);
    h.step_size = (float)(y.lr / (1.0 - std::pow(y.beta1, t)));
    h.inv_root = (float)(1.0 / std::sqrt(1.0 - std::pow(y.beta2, t)));
    h.log1 = (float)std::log(y.beta1), h.log2 = (float)std::log(y.beta2);
    h.scale = (float)y.scale, h.max_norm = (float)y.max_norm;
    h.lr_device = y.lr_device, h.step_device = y.step_device, h.norm = y.norm;
    h.step = (uint64_t)y.step;
    uint32_t k0 = (uint32_t)y.seed, k1 = (uint32_t)(y.seed >> 32);
    for (auto& key : h.key) {
      key[0] = k0, key[1] = k1;
      k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int code = ROT_OK;
    (code = launch_adamw<kF32, false>(h, of[kF32][0], s)) ||
        (code = launch_adamw<kF32, true>(h, of[kF32][1], s)) ||
        (code = launch_adamw<kBf16Random, false>(h, of[kBf16Random][0], s)) ||
        (code = launch_adamw<kBf16Random, true>(h, of[kBf16Random][1], s)) ||
        (code = launch_adamw<kBf16Master, false>(h, of[kBf16Master][0], s)) ||
        (code = launch_adamw<kBf16Master, true>(h, of[kBf16Master][1], s)) ||
        (code = launch_adamw<kF16Master, false>(h, of[kF16Master][0], s)) ||
        (code = launch_adamw<kF16Master, true>(h, of[kF16Master][1], s));
    return code;
  });
}

uint64_t rot_gradient_norm_work_bytes(int32_t count) {
  if (count < 0) return 0;
  const uint64_t launches = std::max<uint64_t>(1, ((uint64_t)count + kSquares - 1) / kSquares);
  return align256(4ull * kSquareBlocks * launches);
}

int rot_gradient_norm(const rot_gradient* gradients, int32_t count, float* norm, void* work,
                      uint64_t work_bytes, void* stream) {
  if (count < 0 || (count > 0 && !gradients) || !norm || !work ||
      (reinterpret_cast<uintptr_t>(work) & 255) ||
      work_bytes < rot_gradient_norm_work_bytes(count))
    return ROT_EINVAL;
  int64_t room = kMostElements;
  for (int32_t i = 0; i < count; ++i) {
    const rot_gradient& g = gradients[i];
    if (g.n < 0 || g.n > room || !float_type(g.type) ||
        (g.n > 0 && (!g.g || !aligned(g.g, type_bytes(g.type)))))
      return ROT_EINVAL;
    room -= g.n;
  }
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return guarded([&]() -> int {
    int parts = 0;
    const unsigned most = (unsigned)std::min(kSquareBlocks, 6 * sm_count());
    for (int32_t at = 0; at < count;) {
      SquareTable t;
      t.part = static_cast<float*>(work) + parts;
      t.count = 0;
      uint64_t chunks = 0;
      double bytes = 0.0;
      for (; at < count && t.count < kSquares; ++at) {
        const rot_gradient& g = gradients[at];
        if (g.n == 0) continue;
        t.first[t.count] = (uint32_t)chunks;
        t.e[t.count++] = {g.g, g.n, g.type, aligned(g.g, 16)};
        chunks += (uint64_t)(g.n + kSquareChunk - 1) / kSquareChunk;
        bytes += (double)g.n * type_bytes(g.type);
      }
      if (t.count == 0) break;
      t.chunks = (uint32_t)chunks;
      const unsigned blocks = (unsigned)std::min<uint64_t>(chunks, most);
      ProfScope prof(ROT_PROF_ELEMENTWISE, bytes, s);
      squares_kernel<<<blocks, kThreads, 0, s>>>(t);
      const int e = launched();
      if (e != ROT_OK) return e;
      parts += (int)blocks;
    }
    ProfScope prof(ROT_PROF_ELEMENTWISE, 0.0, s);
    return launch_behind(norm_root_kernel, 1, 1024, 0, s, (const float*)work, parts, norm);
  });
}

}  // extern "C"
