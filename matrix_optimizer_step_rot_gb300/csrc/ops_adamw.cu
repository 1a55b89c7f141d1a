// AdamW over many tensors and the norm of their gradients (include/rot_ops.h).
// Bound by HBM: every array is read once and written once.
//
// A launch takes a table of tensors as its parameter (nothing is copied to the
// device, and a captured launch keeps its table).  A block takes a chunk of one
// tensor, found by bisection in the tensors' first chunks.  A lane takes four
// or eight consecutive elements: whole calls of the generator, and 16 lanes
// share a scale.
//
// 352 million elements: float32 with the norm before it 1585 us (7.1 TB/s);
// bfloat16 with 8-bit states 705 us (5.0 TB/s), where 57 instructions an element
// bound it (the generator takes 10 of them); 205 million with float32 masters,
// 8-bit states and the norm 592 us (6.3 TB/s).
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <vector>

#include "ops_common.cuh"
#include "profile.h"

namespace rot {
namespace ops {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;  // of the gradients' squares
// A block's threads, the elements that a lane takes at once and how often.
// (8-bit states, 352 million elements in bfloat16: 64 threads 703 us, 128 917,
// 256 1519; eight turns 703 us, two 820, sixteen 688; an embedding of 205 million
// with masters and the norm 592 us, 663, 938; 604, 596.  Blocks per SM: one more
// is 5 and 12% slower, one fewer 1% faster and 4% slower.)
constexpr int threads_of(bool eight) { return eight ? 64 : 256; }
constexpr int lane_elements(bool eight) { return eight ? 8 : 4; }
constexpr int times_of(bool eight) { return eight ? 8 : 4; }
constexpr int chunk_of(bool eight) {
  return threads_of(eight) * times_of(eight) * lane_elements(eight);
}

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

// A step that is counted on the device, and its constants.
struct Counted {
  int64_t t;  // 0: not taken
  float decay, step_size, inv_root, none;
};
static_assert(sizeof(Counted) <= ROT_ADAMW_COUNT_BYTES, "rot_ops.h states it");

struct Hyper {
  float lr, beta1, rest1, beta2, rest2, eps, decay;  // decay: 1 - lr weight_decay
  float step_size, inv_root;                         // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float log1, log2, weight_decay, scale, max_norm, one;
  const float* lr_device;
  const int64_t* step_device;
  const float* norm;
  const Counted* counted;
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

// A block's chunk: its arrays from there on, and how much of them there is (at
// most a chunk).  The same for every thread, so that an address is a uniform
// register and 32 bits.
struct Here {
  void* p;
  const void* g;
  void *m, *v;
  uint8_t *ms, *vs;
  float* master;
  uint64_t word;
  int32_t n, g_type;
};
template <Kept KEPT, bool EIGHT>
__device__ __forceinline__ Here here_of(const Entry& e, uint32_t chunk) {
  constexpr int P = KEPT == kF32 ? 4 : 2, S = EIGHT ? 1 : 4;
  const int64_t at = (int64_t)chunk * chunk_of(EIGHT);
  Here h;
  h.p = (char*)e.p + at * P;
  h.g = (const char*)e.g + at * (e.g_type == ROT_TYPE_F32 ? 4 : 2);
  h.m = (char*)e.m + at * S, h.v = (char*)e.v + at * S;
  h.ms = e.ms + at / 128, h.vs = e.vs + at / 128;
  h.master = e.master + at;
  h.word = e.word + (uint64_t)at / 4;
  h.n = (int32_t)min((int64_t)chunk_of(EIGHT), e.n - at);
  h.g_type = e.g_type;
  return h;
}

// What a call's constants come to on the device.
struct Now {
  float scale, decay, step_size, inv_root;
  uint64_t t;
  uint32_t first[3];  // the generator's round 0 with the step and the key worked in
};

// N elements of `ES` bytes as they lie in memory, 32 bits at a time.  FULL: all
// there and reached by accesses of 16 bytes (or all of them), else `left` of
// them one by one (the rest 0).
template <int W>
struct Piece {
  uint32_t w[W];
};
template <int ES>
using Bits = std::conditional_t<ES == 4, uint32_t, std::conditional_t<ES == 2, uint16_t, uint8_t>>;

template <int ES, int N, bool FULL>
__device__ __forceinline__ Piece<N * ES / 4> some(const void* p, uint32_t i, int left) {
  using T = Bits<ES>;
  constexpr int W = N * ES / 4;
  const T* q = (const T*)p + i;
  Piece<W> r;
  if constexpr (!FULL) {
#pragma unroll
    for (int k = 0; k < W; ++k) r.w[k] = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < left) r.w[k * ES / 4] |= (uint32_t)q[k] << (k * ES % 4 * 8);
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(q);
    r.w[0] = x.x, r.w[1] = x.y;
  } else {
    static_assert(W % 4 == 0, "whole accesses");
#pragma unroll
    for (int k = 0; k < W; k += 4) {
      const uint4 x = reinterpret_cast<const uint4*>(q)[k / 4];
      r.w[k] = x.x, r.w[k + 1] = x.y, r.w[k + 2] = x.z, r.w[k + 3] = x.w;
    }
  }
  return r;
}
template <int ES, int N, bool FULL>
__device__ __forceinline__ void put_some(void* p, uint32_t i, int left, const Piece<N * ES / 4>& r) {
  using T = Bits<ES>;
  constexpr int W = N * ES / 4;
  T* q = (T*)p + i;
  if constexpr (!FULL) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < left) q[k] = (T)(r.w[k * ES / 4] >> (k * ES % 4 * 8));
  } else if constexpr (W == 2) {
    *reinterpret_cast<uint2*>(q) = make_uint2(r.w[0], r.w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < W; k += 4)
      reinterpret_cast<uint4*>(q)[k / 4] =
          make_uint4(r.w[k], r.w[k + 1], r.w[k + 2], r.w[k + 3]);
  }
}
__device__ __forceinline__ float2 f32_pair(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
template <int N>
__device__ __forceinline__ Piece<N> words_of(const float2 (&x)[N / 2]) {
  Piece<N> r;
#pragma unroll
  for (int k = 0; k < N / 2; ++k)
    r.w[2 * k] = __float_as_uint(x[k].x), r.w[2 * k + 1] = __float_as_uint(x[k].y);
  return r;
}

// 16-bit numbers in pairs.
__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 f16_pair(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// ---- 8 bits ----

// 2^(byte - 127) (byte 0: subnormal; 255: NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 1u << 22 : byte == 255 ? 0x7fc00000u : byte << 23);
}
// Four E4M3 numbers.
__device__ __forceinline__ void numbers8(uint32_t q, float2& a, float2& b) {
  uint32_t h, k;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(h), "=r"(k)
      : "r"(q));
  a = f16_pair(h), b = f16_pair(k);
}

// The largest of three sizes; NaN if there is one.
__device__ __forceinline__ float top_of(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float top_of(const float2 (&x)[4]) {
  return top_of(top_of(top_of(x[0].x, x[0].y, x[1].x), x[1].y, x[2].x),
                top_of(x[2].y, x[3].x, x[3].y), 0.f);
}

// The scale byte for a largest size of these bits, 8 more than it (0 below
// that): size = (1 + f) 2^(t - 127) <= 448 2^(byte - 127), 448 = 1.75 2^8.
// 255 and more: NaN or infinity.
__device__ __forceinline__ uint32_t byte8_of(uint32_t size) { return (size + 0x1fffffu) >> 23; }

// A number in E4M3, in the upper byte, rounded by `part` (its 16 random bits 4
// up, and 8 for the half).  y: the number under its scale, times 2^-120: its
// bits as float32 are E4M3's above 20 more (their least exponents meet there,
// below it both count in fixed steps), so that an addition to the bits and a
// shift round it at any size.  ROOT: x is not negative, and not rounded to 0
// where it is not 0 (its bits are then above 2^20).
template <bool ROOT>
__device__ __forceinline__ uint32_t code8(float x, float y, uint32_t part) {
  const uint32_t b = __float_as_uint(y);
  if constexpr (ROOT) return __viaddmax_u32(b, part, min(__float_as_uint(x), 1u << 20)) << 4;
  return ((b + part) << 4 & 0x7fffffffu) | (b & 0x80000000u);
}
__device__ __forceinline__ uint32_t packed8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x73), __byte_perm(c, d, 0x73), 0x5410);
}

// Eight numbers of a half warp's 128 in E4M3.
template <bool ROOT>
__device__ __forceinline__ uint2 rounded8(const float2 (&x)[4], const uint32_t (&part)[8],
                                          uint32_t byte) {
  const float2 back = both(__uint_as_float((134u - byte) << 23));
  uint32_t c[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 y = mul2(x[k], back);
    c[2 * k] = code8<ROOT>(x[k].x, y.x, part[2 * k]);
    c[2 * k + 1] = code8<ROOT>(x[k].y, y.y, part[2 * k + 1]);
  }
  return make_uint2(packed8(c[0], c[1], c[2], c[3]), packed8(c[4], c[5], c[6], c[7]));
}
// The same where there is a NaN or an infinity among the 128 or their scale is
// large (2^(127 - byte) 2^-120 is no normal number).
template <bool ROOT>
__device__ __noinline__ uint3 rounded8_any(float2 x0, float2 x1, float2 x2, float2 x3, uint4 p0,
                                           uint4 p1) {
  const float x[8] = {x0.x, x0.y, x1.x, x1.y, x2.x, x2.y, x3.x, x3.y};
  const uint32_t part[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
  const uint32_t half = 0xffffu << (threadIdx.x & 16);
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t a = __float_as_uint(x[k]) & 0x7fffffffu;
    if (a < 0x7f800000u) top = max(top, a);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(half, top, o));
  const uint32_t byte = (uint32_t)max((int)byte8_of(top) - 8, 0);
  uint32_t c[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float y = x[k] * __uint_as_float((254u - byte) << 23) * 0x1p-120f;
    c[k] = (__float_as_uint(x[k]) & 0x7fffffffu) < 0x7f800000u ? code8<ROOT>(x[k], y, part[k])
                                                               : 0x7f000000u;
  }
  return make_uint3(packed8(c[0], c[1], c[2], c[3]), packed8(c[4], c[5], c[6], c[7]), byte);
}

__device__ __forceinline__ void random_of(const Hyper& h, const Now& c, uint64_t counter,
                                          uint32_t* w) {
  const uint2 a0 = mul_wide((uint32_t)counter, kPhiloxM0);
  uint32_t c0 = c.first[0] ^ (uint32_t)(counter >> 32), c1 = c.first[1];
  uint32_t c2 = a0.y ^ c.first[2], c3 = a0.x;
#pragma unroll
  for (int r = 1; r < 10; ++r) {
    const uint2 a = mul_wide(c0, kPhiloxM0), b = mul_wide(c2, kPhiloxM1);
    c0 = b.y ^ c1 ^ h.key[r][0];
    c1 = b.x;
    c2 = a.y ^ c3 ^ h.key[r][1];
    c3 = a.x;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

// Two numbers in bfloat16, each rounded by 16 bits (of the second the upper):
// added below the last place kept, and cut off there.
__device__ __forceinline__ uint32_t rounded_bf16(float2 x, uint32_t random) {
  uint32_t r;
  asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(r) : "f"(x.y), "f"(x.x), "r"(random));
  return r;
}

// x + y of products that keep their own rounding.  `one` comes with the
// parameters: with a plain sum behind a product the moments' codes were not
// those of steps rounded one by one.
__device__ __forceinline__ float2 plus2(float2 x, float one, float2 y) {
  return fma2(x, both(one), y);
}

// The roots of x, which are 0 or positive, to the nearest number but where they
// lie within 2^-20 of a last place of the middle of two (39 of 2^25 significands
// and exponents): Newton's iteration with the residual in one rounding
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", IBM Journal of Research and Development 34, 1990), r = s - (s^2 -
// x) / (2 s).  s, x times an approximate reciprocal root, is within two last
// places; the residual is exact, and its quotient good to 2^-20 of a last place.
// Where an x of the lane is too small for that (the residual would not be exact
// below 2^-100; 0 is among them) or not finite, the library's function.  top:
// the largest.
template <int H>
__device__ __forceinline__ void roots(const float2 (&x)[H], float2 (&r)[H], float& top) {
  float low = 0x1p127f;
  top = 0.f;
#pragma unroll
  for (int k = 0; k < H; ++k) {
    float2 y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x[k].x));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x[k].y));
    const float2 s = mul2(x[k], y);
    r[k] = fma2(fma2(s, s, mul2(x[k], both(-1.f))), mul2(y, both(-0.5f)), s);
    asm("min.f32 %0, %1, %2, %3;" : "=f"(low) : "f"(low), "f"(x[k].x), "f"(x[k].y));
    top = top_of(r[k].x, r[k].y, top);
  }
  if (low >= 0x1p-100f && top < __int_as_float(0x7f800000)) return;
  top = 0.f;
#pragma unroll
  for (int k = 0; k < H; ++k) {
    r[k] = make_float2(__fsqrt_rn(x[k].x), __fsqrt_rn(x[k].y));
    top = top_of(r[k].x, r[k].y, top);
  }
}
__device__ __forceinline__ float inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A lane's elements of one turn as they lie in memory.
template <Kept KEPT, bool EIGHT, bool WIDE>
struct Raw {
  static constexpr int N = lane_elements(EIGHT);
  static constexpr int G = WIDE ? 4 : 2, P = KEPT == kBf16Random ? 2 : 4, S = EIGHT ? 1 : 4;
  Piece<N * G / 4> g;
  Piece<N * P / 4> p;
  Piece<N * S / 4> m, v;
  uint32_t sm, sv;  // (8 bits: the scales' bytes)

  template <bool FULL>
  __device__ __forceinline__ void load(const Here& e, uint32_t i, int left) {
    g = some<G, N, FULL>(e.g, i, left);
    p = some<P, N, FULL>(KEPT >= kBf16Master ? (const void*)e.master : e.p, i, left);
    m = some<S, N, FULL>(e.m, i, left);
    v = some<S, N, FULL>(e.v, i, left);
    if constexpr (EIGHT) {
      sm = FULL || left > 0 ? e.ms[i >> 7] : 0u;
      sv = FULL || left > 0 ? e.vs[i >> 7] : 0u;
    }
  }
};

// A lane's N elements from i on: one step, and the results stored.
template <Kept KEPT, bool EIGHT, bool WIDE, bool FULL>
__device__ __forceinline__ void step_lane(const Hyper& h, const Now& c, const Here& e,
                                          const Raw<KEPT, EIGHT, WIDE>& raw, uint32_t i, int left) {
  constexpr int N = lane_elements(EIGHT), H = N / 2;
  constexpr bool kWords = EIGHT || KEPT == kBf16Random;
  float2 g[H], m[H], v[H], r[H], p[H];
#pragma unroll
  for (int k = 0; k < H; ++k) {
    if constexpr (WIDE)
      g[k] = f32_pair(raw.g.w[2 * k], raw.g.w[2 * k + 1]);
    else
      g[k] = bf16_pair(raw.g.w[k]);
    if constexpr (KEPT == kBf16Random)
      p[k] = bf16_pair(raw.p.w[k]);
    else
      p[k] = f32_pair(raw.p.w[2 * k], raw.p.w[2 * k + 1]);
    if constexpr (!EIGHT) {
      m[k] = f32_pair(raw.m.w[2 * k], raw.m.w[2 * k + 1]);
      v[k] = f32_pair(raw.v.w[2 * k], raw.v.w[2 * k + 1]);
    }
  }
  if constexpr (!WIDE) {
    if (e.g_type == ROT_TYPE_F16) {  // (the same for every thread)
#pragma unroll
      for (int k = 0; k < H; ++k) g[k] = f16_pair(raw.g.w[k]);
    }
  }
  float ms = h.beta1;
  if constexpr (EIGHT) {
    ms *= scale_of(raw.sm);
    const float2 vs = both(scale_of(raw.sv));
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      numbers8(raw.m.w[k], m[2 * k], m[2 * k + 1]);
      numbers8(raw.v.w[k], v[2 * k], v[2 * k + 1]);
    }
#pragma unroll
    for (int k = 0; k < H; ++k) v[k] = mul2(v[k], vs), v[k] = mul2(v[k], v[k]);
  }
#pragma unroll
  for (int k = 0; k < H; ++k) {
    // (every step rounds as the formula's float32 steps do: what comes next is
    // rounded to 3 bits at places that an error of one last place may cross)
    g[k] = mul2(g[k], both(c.scale));
    m[k] = plus2(mul2(m[k], both(ms)), h.one, mul2(g[k], both(h.rest1)));
    v[k] = plus2(mul2(v[k], both(h.beta2)), h.one, mul2(mul2(g[k], both(h.rest2)), g[k]));
  }
  float top;
  roots(v, r, top);
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const float2 under = fma2(r[k], both(c.inv_root), both(h.eps));
    const float2 u = mul2(m[k], both(-c.step_size));
    p[k] = fma2(u, make_float2(inverse(under.x), inverse(under.y)), mul2(p[k], both(c.decay)));
  }
  uint32_t w[N];
  if constexpr (kWords) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) random_of(h, c, e.word + ((i >> 2) + k), w + 4 * k);
  }
  if constexpr (EIGHT) {
    uint32_t part[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) part[k] = (w[k] & 0xffffu) * 16u + 8u;
    uint32_t t = byte8_of(__float_as_uint(top_of(m))) | byte8_of(__float_as_uint(top)) << 16;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
    const uint32_t tm = t & 0xffffu, tv = t >> 16;
    uint32_t bm, bv;
    uint2 nm, nv;
    if (max(tm, tv) <= 133 + 8) {  // (the same for a half warp)
      bm = (uint32_t)max((int)tm - 8, 0), bv = (uint32_t)max((int)tv - 8, 0);
      nm = rounded8<false>(m, part, bm), nv = rounded8<true>(r, part, bv);
    } else {
      const uint4 p0 = make_uint4(part[0], part[1], part[2], part[3]);
      const uint4 p1 = make_uint4(part[4], part[5], part[6], part[7]);
      const uint3 am = rounded8_any<false>(m[0], m[1], m[2], m[3], p0, p1);
      const uint3 av = rounded8_any<true>(r[0], r[1], r[2], r[3], p0, p1);
      nm = make_uint2(am.x, am.y), bm = am.z;
      nv = make_uint2(av.x, av.y), bv = av.z;
    }
    put_some<1, 8, FULL>(e.m, i, left, {{nm.x, nm.y}});
    put_some<1, 8, FULL>(e.v, i, left, {{nv.x, nv.y}});
    if ((threadIdx.x & 15) == 0 && (FULL || left > 0))
      e.ms[i >> 7] = (uint8_t)bm, e.vs[i >> 7] = (uint8_t)bv;
  } else {
    put_some<4, N, FULL>(e.m, i, left, words_of<N>(m));
    put_some<4, N, FULL>(e.v, i, left, words_of<N>(v));
  }
  if constexpr (KEPT == kBf16Random) {
    Piece<H> q;
#pragma unroll
    for (int k = 0; k < H; ++k)
      q.w[k] = rounded_bf16(p[k], __byte_perm(w[2 * k], w[2 * k + 1], 0x7632));
    put_some<2, N, FULL>(e.p, i, left, q);
  } else if constexpr (KEPT == kF32) {
    put_some<4, N, FULL>(e.p, i, left, words_of<N>(p));
  } else {
    put_some<4, N, FULL>(e.master, i, left, words_of<N>(p));
    Piece<H> q;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      if constexpr (KEPT == kBf16Master) {
        const __nv_bfloat162 x = __float22bfloat162_rn(p[k]);
        q.w[k] = *reinterpret_cast<const uint32_t*>(&x);
      } else {
        const __half2 x = __float22half2_rn(p[k]);
        q.w[k] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    put_some<2, N, FULL>(e.p, i, left, q);
  }
}

// A warp's turns from its lane's element i on: `full` of them whole (and every
// array reached by vector accesses), and what is left of its share.
template <Kept KEPT, bool EIGHT, bool WIDE>
__device__ __forceinline__ void step_warp(const Hyper& h, const Now& c, const Here& e, uint32_t i,
                                          int full) {
  constexpr int N = lane_elements(EIGHT), kStep = 32 * N, kTimes = times_of(EIGHT);
  const uint32_t end = i + kTimes * kStep;
  if (EIGHT || full < kTimes) {  // the next turn's elements are on their way meanwhile
    Raw<KEPT, EIGHT, WIDE> a, b;
    if (full > 0) a.template load<true>(e, i, N);
#pragma unroll 1
    while (full > 0) {
      if (full > 1) b.template load<true>(e, i + kStep, N);
      step_lane<KEPT, EIGHT, WIDE, true>(h, c, e, a, i, N);
      i += kStep;
      if (--full == 0) break;
      if (full > 1) a.template load<true>(e, i + kStep, N);
      step_lane<KEPT, EIGHT, WIDE, true>(h, c, e, b, i, N);
      i += kStep;
      --full;
    }
  } else {  // all turns' elements first
    Raw<KEPT, EIGHT, WIDE> raw[kTimes];
#pragma unroll
    for (int k = 0; k < kTimes; ++k) raw[k].template load<true>(e, i + k * kStep, N);
#pragma unroll
    for (int k = 0; k < kTimes; ++k, i += kStep)
      step_lane<KEPT, EIGHT, WIDE, true>(h, c, e, raw[k], i, N);
  }
#pragma unroll 1
  for (; i < end; i += kStep) {
    const int left = max(0, min(N, e.n - (int)i));
    if (!__any_sync(0xffffffffu, left > 0)) return;
    Raw<KEPT, EIGHT, WIDE> raw;
    raw.template load<false>(e, i, left);
    step_lane<KEPT, EIGHT, WIDE, false>(h, c, e, raw, i, left);
  }
}

// 1 - lr weight_decay, lr / (1 - beta1^t) and 1 / sqrt(1 - beta2^t), on the host
// and on the device.
struct Rates {
  double lr, beta1, beta2, weight_decay;
};
__host__ __device__ inline void constants_of(const Rates& y, int64_t t, float& decay,
                                             float& step_size, float& inv_root) {
  const double lost = y.lr * y.weight_decay;
  decay = (float)(1.0 - lost);
  step_size = (float)(y.lr / (1.0 - pow(y.beta1, (double)t)));
  inv_root = (float)(1.0 / sqrt(1.0 - pow(y.beta2, (double)t)));
}

// Counts the step that begins, unless it is not taken.  One thread, since the
// constants are float64 (in the step's own blocks a few hundred slow operations
// each).  113 vectors: 18.9 us a call, 14.3 without it.
__global__ void count_kernel(const Rates rates, const float* lr_device, const float scale,
                             const float* norm, int64_t* taken, Counted* out) {
  wait_for_prior();
  Counted c = {};
  if (!norm || isfinite(fabsf(scale) * *norm)) c.t = *taken + 1;
  if (c.t < 1) c.t = 0;
  if (c.t) {
    *taken = c.t;
    Rates r = rates;
    if (lr_device) r.lr = *lr_device;
    constants_of(r, c.t, c.decay, c.step_size, c.inv_root);
  }
  *out = c;
}

template <Kept KEPT, bool EIGHT, int CAP>
__global__ void __launch_bounds__(threads_of(EIGHT), EIGHT ? KEPT == kBf16Random ? 10 : 11 : 2)
    adamw_kernel(const __grid_constant__ Table<CAP> a) {
  const Hyper& h = a.h;
  const int of = tensor_of(a.first, a.count, blockIdx.x);
  const Here e = here_of<KEPT, EIGHT>(a.e[of], blockIdx.x - a.first[of]);
  Now c = {h.scale, h.decay, h.step_size, h.inv_root, h.step, {}};
  wait_for_prior();
  if (h.norm) {
    const float norm = fabsf(c.scale) * *h.norm;
    if (!isfinite(norm)) return;
    if (norm > h.max_norm) c.scale *= h.max_norm / norm;
  }
  if (h.counted) {
    const Counted n = *h.counted;
    if (n.t < 1) return;
    c.t = (uint64_t)n.t;
    c.decay = n.decay, c.step_size = n.step_size, c.inv_root = n.inv_root;
  } else if (h.lr_device || h.step_device) {
    const float lr = h.lr_device ? *h.lr_device : h.lr;
    if (h.step_device) c.t = (uint64_t)*h.step_device;
    if ((int64_t)c.t < 1) return;
    // 1 - beta^t = -(e^(t log beta) - 1)
    c.step_size = lr / -expm1f((float)(int64_t)c.t * h.log1);
    c.inv_root = 1.f / sqrtf(-expm1f((float)(int64_t)c.t * h.log2));
    c.decay = 1.f - lr * h.weight_decay;
  }
  const uint2 b = mul_wide((uint32_t)c.t, kPhiloxM1);
  c.first[0] = b.y ^ h.key[0][0], c.first[1] = b.x;
  c.first[2] = (uint32_t)(c.t >> 32) ^ h.key[0][1];
  constexpr int kStep = 32 * lane_elements(EIGHT), kTimes = times_of(EIGHT);
  const int begin = (threadIdx.x >> 5) * (kTimes * kStep);
  const int full = a.e[of].whole ? max(0, min(kTimes, (e.n - begin) / kStep)) : 0;
  const uint32_t i = begin + (threadIdx.x & 31) * lane_elements(EIGHT);
  if (e.g_type == ROT_TYPE_F32)
    step_warp<KEPT, EIGHT, true>(h, c, e, i, full);
  else
    step_warp<KEPT, EIGHT, false>(h, c, e, i, full);
}

template <Kept KEPT, bool EIGHT, int CAP>
int launch_table(const Hyper& h, const Entry* e, int count, cudaStream_t s) {
  Table<CAP> t;
  t.h = h, t.count = count;
  uint64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    t.first[i] = (uint32_t)chunks;
    t.e[i] = e[i];
    chunks += (e[i].n + chunk_of(EIGHT) - 1) / chunk_of(EIGHT);
  }
  return launch_behind(adamw_kernel<KEPT, EIGHT, CAP>, (unsigned)chunks, threads_of(EIGHT), 0, s, t);
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

// The addresses that a call writes: each one once.  (A table twice as large: a
// list of 300 tensors takes 58 us of the host with their addresses sorted.)
class Written {
 public:
  explicit Written(size_t most) {
    size_t size = 16;
    while (size < 2 * most) size *= 2;
    at_.resize(size);
  }
  bool again(const void* p) {  // whether p was there
    const uintptr_t x = reinterpret_cast<uintptr_t>(p);
    size_t i = (size_t)((uint64_t)x * 0x9E3779B97F4A7C15u >> 32) & (at_.size() - 1);
    for (; at_[i]; i = (i + 1) & (at_.size() - 1))
      if (at_[i] == x) return true;
    at_[i] = x;
    return false;
  }

 private:
  std::vector<uintptr_t> at_;
};

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// ---- norm ----

struct Square {
  const void* g;
  int64_t n;
  int32_t type, whole;
};
constexpr int kSquares = 1000, kSquareChunk = 8192, kSquareBlocks = 1024;
struct SquareTable {
  double* part;
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
  __shared__ double red[kWarps];
  wait_for_prior();
  const uint32_t c0 = (uint32_t)((uint64_t)a.chunks * blockIdx.x / gridDim.x);
  const uint32_t c1 = (uint32_t)((uint64_t)a.chunks * (blockIdx.x + 1) / gridDim.x);
  double sum = 0.0;  // (a thread's 32 elements of a chunk are summed in float32)
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
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) sum += red[w];
    a.part[blockIdx.x] = sum;
  }
}

// The root of the parts' sum, in a fixed order.
__global__ void __launch_bounds__(1024) norm_root_kernel(const double* part, int parts,
                                                         float* norm) {
  __shared__ double red[32];
  wait_for_prior();
  double sum = 0.0;
  for (int p = threadIdx.x; p < parts; p += 1024) sum += part[p];
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

// taken: null, or the device's count of the steps, with `counted` as workspace.
int adamw_step(const rot_adamw_tensor* tensors, int32_t count, const rot_adamw_hyper* hyper,
               int64_t* taken, Counted* counted, void* stream) {
  if (count < 0 || (count > 0 && !tensors) || !hyper) return ROT_EINVAL;
  const rot_adamw_hyper& y = *hyper;
  for (double x : {y.lr, y.eps, y.weight_decay})
    if (!(x >= 0.0)) return ROT_EINVAL;
  for (double x : {y.beta1, y.beta2})
    if (!(x >= 0.0 && x < 1.0)) return ROT_EINVAL;
  if (!std::isfinite(y.scale) || (y.norm && !(y.max_norm > 0.0))) return ROT_EINVAL;
  if (!taken && !y.step_device && y.step < 1) return ROT_EINVAL;
  if (!aligned(y.lr_device, 4) || (!taken && !aligned(y.step_device, 8)) || !aligned(y.norm, 4))
    return ROT_EINVAL;
  return guarded([&]() -> int {
    std::vector<Entry> of[4][2];
    Written written(6 * (size_t)count);
    bool some = false;
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
        if (p && written.again(p)) return ROT_EINVAL;
      some = true;
      const int kept = t.p_type == ROT_TYPE_F32    ? kF32
                       : t.p_type == ROT_TYPE_F16 ? kF16Master
                       : t.master                  ? kBf16Master
                                                   : kBf16Random;
      Entry e;
      e.p = t.p, e.g = t.g, e.m = t.m, e.v = t.v, e.ms = t.m_scale, e.vs = t.v_scale;
      e.master = t.master, e.n = t.n, e.word = word, e.g_type = t.g_type;
      const int lane = lane_elements(eight);
      auto fits = [&](const void* p, int es) { return aligned(p, std::min(16, lane * es)); };
      e.whole = fits(t.p, type_bytes(t.p_type)) && fits(t.g, type_bytes(t.g_type)) &&
                fits(t.m, state) && fits(t.v, state) && fits(t.master, 4);
      std::vector<Entry>& list = of[kept][eight];
      if (list.empty()) list.reserve(count - i);
      list.push_back(e);
    }
    if (!some && !taken) return ROT_OK;
    const int dev = check_device();
    if (dev != ROT_OK) return dev;
    Hyper h;
    h.lr = (float)y.lr;
    // (the quotient's approximate reciprocal takes subnormal numbers for 0)
    h.eps = y.eps > 0.0 ? std::max((float)y.eps, 0x1p-126f) : 0.f;
    h.weight_decay = (float)y.weight_decay;
    h.beta1 = (float)y.beta1, h.rest1 = (float)(1.0 - y.beta1);
    h.beta2 = (float)y.beta2, h.rest2 = (float)(1.0 - y.beta2);
    const Rates rates = {y.lr, y.beta1, y.beta2, y.weight_decay};
    constants_of(rates, std::max<int64_t>(y.step, 1), h.decay, h.step_size, h.inv_root);
    h.log1 = (float)std::log(y.beta1), h.log2 = (float)std::log(y.beta2);
    h.scale = (float)y.scale, h.max_norm = (float)y.max_norm, h.one = 1.f;
    h.lr_device = y.lr_device, h.step_device = y.step_device, h.norm = y.norm;
    h.counted = counted, h.step = (uint64_t)y.step;
    uint32_t k0 = (uint32_t)y.seed, k1 = (uint32_t)(y.seed >> 32);
    for (auto& key : h.key) {
      key[0] = k0, key[1] = k1;
      k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int code = ROT_OK;
    if (taken) {
      ProfScope prof(ROT_PROF_ELEMENTWISE, 0.0, s);
      code = launch_behind(count_kernel, 1, 1, 0, s, rates, y.lr_device, h.scale, y.norm, taken,
                           counted);
    }
    code || (code = launch_adamw<kF32, false>(h, of[kF32][0], s)) ||
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

}  // namespace
}  // namespace ops
}  // namespace rot

using namespace rot;
using namespace rot::ops;

extern "C" {

int rot_adamw_step(const rot_adamw_tensor* tensors, int32_t count, const rot_adamw_hyper* hyper,
                   void* stream) {
  return adamw_step(tensors, count, hyper, nullptr, nullptr, stream);
}

int rot_adamw_step_counted(const rot_adamw_tensor* tensors, int32_t count,
                           const rot_adamw_hyper* hyper, int64_t* taken, void* work, void* stream) {
  if (!taken || !aligned(taken, 8) || !work || !aligned(work, 16)) return ROT_EINVAL;
  return adamw_step(tensors, count, hyper, taken, static_cast<Counted*>(work), stream);
}

uint64_t rot_gradient_norm_work_bytes(int32_t count) {
  if (count < 0) return 0;
  const uint64_t launches = std::max<uint64_t>(1, ((uint64_t)count + kSquares - 1) / kSquares);
  return align256(8ull * kSquareBlocks * launches);
}

int rot_gradient_norm(const rot_gradient* gradients, int32_t count, float* norm, void* work,
                      uint64_t work_bytes, void* stream) {
  if (count < 0 || (count > 0 && !gradients) || !norm || !aligned(norm, 4) || !work ||
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
      t.part = static_cast<double*>(work) + parts;
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
      const int e = launch_behind(squares_kernel, blocks, kThreads, 0, s, t);
      if (e != ROT_OK) return e;
      parts += (int)blocks;
    }
    ProfScope prof(ROT_PROF_ELEMENTWISE, 0.0, s);
    return launch_behind(norm_root_kernel, 1, 1024, 0, s, (const double*)work, parts, norm);
  });
}

}  // extern "C"
