// Rotary positions and the norm of queries and keys (include/rot_ops.h): one
// kernel for the rotation, the norm with it, and the norm's backward pass.
// Bound by HBM: every array is read once and written once.
//
// A row is one head of one token.  A group of 2^k lanes takes it, a lane two
// runs of V elements: those whose elements turn together.  For pairs (i, i +
// rotated / 2) these are runs of the two halves, interleaved two runs next to
// each other; either way a lane holds a[j] and b[j] of the pairs u V + j, u
// its place in the group, and all arithmetic is the same.  What is not rotated
// follows in runs of its own.
//
// A warp takes a token's heads in passes of as many as it has groups, queries
// first, then keys (or a part of the passes, where there are few tokens): the
// token's angles are worked out once, a pair to a lane, and shared through
// shared memory, where the weights lie, too.  Warps stay for several tokens.
// Rows come by asynchronous copies a few passes ahead; a lane copies and reads
// its own runs alone, so that no lane waits for another's.  (Single 16-bit
// elements, which such copies do not take: the next pass's in registers.)
//
// 16384 tokens of 16 and 8 heads of 128 in bfloat16: rotation 34.9 us, norm and
// rotation 34.0 (5.9 TB/s of 201 MB), backward 54.8 (5.5 TB/s of 302 MB), of
// which the join is 3.  With queries and keys on warps of their own (angles
// twice) and one pass of register loads ahead: 48, 66 and 141.
#pragma once

#include <algorithm>

#include "ops_common.cuh"
#include "profile.h"

namespace rot {
namespace ops {

enum HeadsMode { kRotate = 0, kNorm = 1, kNormGrad = 2 };

constexpr int kHeadWarps = 4;     // per block
constexpr int kHeadParts = 1024;  // most blocks of a backward pass: its partial sums
// Blocks per SM that stay, and that the registers are made to fit; passes that
// are on their way.  (16384 tokens, norm and rotation 34.2 us and 54.8 backward:
// forward 6 blocks, of 80 registers, 41.0 us, 4 34.8; backward 4 blocks, of 128
// registers, spill, 84 us, 2 66; 2 passes on their way 34.8 and 55.5 us, 4 34.3
// and 54.9.)
constexpr int head_blocks(HeadsMode mode, int runs) {
  return mode == kNormGrad ? (runs > 2 ? 2 : 3) : (runs > 2 ? 3 : 5);
}
constexpr int kHeadAhead = 3;

struct HeadStrides {
  int64_t batch = 0, token = 0, head = 0;
};

// Queries or keys.
struct HeadSide {
  const void* x = nullptr;
  const void* dy = nullptr;  // backward
  void* out = nullptr;
  const void* w = nullptr;  // null: no norm
  HeadStrides xs, ds, os;
  int32_t heads = 0;
};

// How far apart in items a warp's are: batch entries, tokens, items of a token.
struct HeadStep {
  uint32_t b = 0, t = 0;
  int32_t chunk = 0;
};

struct HeadArgs {
  HeadSide side[2];
  int32_t passes0 = 0, passes = 0;  // of a token's queries, and of both
  int32_t chunk = 0;                // passes to an item
  int32_t chunks = 1;               // items of a token
  uint32_t items = 0;               // of all
  HeadStep step;
  uint32_t tokens = 1;              // of a batch entry
  int32_t dim = 0, rotated = 0, units = 0, log_group = 0;
  const uint64_t* turns = nullptr;
  const void* positions = nullptr;
  int32_t position_bytes = 8;
  int64_t pbs = 0, pts = 0, start = 0;
  float cos_scale = 1.f, sin_scale = 1.f;  // the magnitude; sin's sign turns the other way
  int32_t w32 = 0;
  float eps = 0.f;
  float* part = nullptr;  // backward: [blocks][2][dim]
  const void* safe = nullptr;  // an address that may be read
  int32_t blocks = 0;     // of the launch
};

// Where a unit's two runs lie, and whether they are there and rotated.
struct Unit {
  int a = 0, b = 0;
  bool has_a = false, has_b = false, rot_a = false, rot_b = false;
};

template <int V, bool IL>
__device__ __forceinline__ Unit unit_of(int u, int units, int dim, int rotated, bool il) {
  Unit t;
  t.has_a = u < units;
  if (IL || (V == 1 && il)) {
    t.a = 2 * u * V, t.b = t.a + V;
    t.rot_a = t.a < rotated, t.rot_b = t.b < rotated;
  } else {
    const int half = rotated / 2, turned = half / V;
    if (u < turned) {
      t.a = u * V, t.b = half + u * V;
      t.rot_a = t.rot_b = true;
    } else {
      t.a = rotated + 2 * (u - turned) * V, t.b = t.a + V;
    }
  }
  t.has_b = t.has_a && t.b < dim;
  return t;
}

// A run as it lies in memory, 32 bits at a time (V = 1: one element).
template <class T, int V>
struct Piece {
  static constexpr int N = V * (int)sizeof(T) < 4 ? 1 : V * (int)sizeof(T) / 4;
  uint32_t w[N];
};
__device__ __forceinline__ float2 two_of(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 two_of(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t word_of(float2 x, __nv_bfloat16) {
  const __nv_bfloat162 r = __float22bfloat162_rn(x);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t word_of(float2 x, __half) {
  const __half2 r = __float22half2_rn(x);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The lane's runs as a[] and b[] of its pairs, and back.
template <class T, int V, bool IL>
__device__ __forceinline__ void pairs_of(const Piece<T, V>& ra, const Piece<T, V>& rb, Vec<V>& a,
                                         Vec<V>& b) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 4)
      a.p[0] = __uint_as_float(ra.w[0]), b.p[0] = __uint_as_float(rb.w[0]);
    else
      a.p[0] = two_of(ra.w[0], T()).x, b.p[0] = two_of(rb.w[0], T()).x;
  } else {
    static_assert(V % 4 == 0 || !IL, "a pack comes from one run");
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if constexpr (!IL && sizeof(T) == 4) {
        a.p[i] = make_float2(__uint_as_float(ra.w[2 * i]), __uint_as_float(ra.w[2 * i + 1]));
        b.p[i] = make_float2(__uint_as_float(rb.w[2 * i]), __uint_as_float(rb.w[2 * i + 1]));
      } else if constexpr (!IL) {
        a.p[i] = two_of(ra.w[i], T()), b.p[i] = two_of(rb.w[i], T());
      } else {
        const Piece<T, V>& r = i < V / 4 ? ra : rb;
        if constexpr (sizeof(T) == 4) {
          const int k = 4 * i % V;
          a.p[i] = make_float2(__uint_as_float(r.w[k]), __uint_as_float(r.w[k + 2]));
          b.p[i] = make_float2(__uint_as_float(r.w[k + 1]), __uint_as_float(r.w[k + 3]));
        } else {
          const int k = 2 * i % (V / 2);
          const float2 x = two_of(r.w[k], T()), y = two_of(r.w[k + 1], T());
          a.p[i] = make_float2(x.x, y.x), b.p[i] = make_float2(x.y, y.y);
        }
      }
    }
  }
}
template <class T, int V, bool IL>
__device__ __forceinline__ void runs_of(const Vec<V>& a, const Vec<V>& b, Piece<T, V>& ra,
                                        Piece<T, V>& rb) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 4)
      ra.w[0] = __float_as_uint(a.p[0]), rb.w[0] = __float_as_uint(b.p[0]);
    else
      ra.w[0] = word_of(make_float2(a.p[0], 0.f), T()), rb.w[0] = word_of(make_float2(b.p[0], 0.f), T());
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if constexpr (!IL && sizeof(T) == 4) {
        ra.w[2 * i] = __float_as_uint(a.p[i].x), ra.w[2 * i + 1] = __float_as_uint(a.p[i].y);
        rb.w[2 * i] = __float_as_uint(b.p[i].x), rb.w[2 * i + 1] = __float_as_uint(b.p[i].y);
      } else if constexpr (!IL) {
        ra.w[i] = word_of(a.p[i], T()), rb.w[i] = word_of(b.p[i], T());
      } else {
        Piece<T, V>& r = i < V / 4 ? ra : rb;
        if constexpr (sizeof(T) == 4) {
          const int k = 4 * i % V;
          r.w[k] = __float_as_uint(a.p[i].x), r.w[k + 1] = __float_as_uint(b.p[i].x);
          r.w[k + 2] = __float_as_uint(a.p[i].y), r.w[k + 3] = __float_as_uint(b.p[i].y);
        } else {
          const int k = 2 * i % (V / 2);
          r.w[k] = word_of(make_float2(a.p[i].x, b.p[i].x), T());
          r.w[k + 1] = word_of(make_float2(a.p[i].y, b.p[i].y), T());
        }
      }
    }
  }
}

// V consecutive floats of shared memory.
template <int V>
__device__ __forceinline__ Piece<float, V> floats_at(const float* w) {
  Piece<float, V> r;
  if constexpr (V == 1) {
    r.w[0] = __float_as_uint(w[0]);
  } else if constexpr (V == 2) {
    const uint2 f = *reinterpret_cast<const uint2*>(w);
    r.w[0] = f.x, r.w[1] = f.y;
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const uint4 f = *reinterpret_cast<const uint4*>(w + j);
      r.w[j] = f.x, r.w[j + 1] = f.y, r.w[j + 2] = f.z, r.w[j + 3] = f.w;
    }
  }
  return r;
}

// Cosine and sine of `turn` 2^-32 turns (a whole number; half a turn is the
// end of its range): the nearest quarter turn off, the sums of their Taylor
// series on what is left, at most pi / 4 (the first terms left out are below
// 2e-9).
__device__ __forceinline__ void cos_sin(int32_t turn, float& c, float& s) {
  const uint32_t quarter = ((uint32_t)turn + 0x20000000u) >> 30;
  const float x = (float)(int32_t)((uint32_t)turn - (quarter << 30)) * 0x1.921fb6p-30f;
  const float y = x * x;
  float ps = 1.f / 362880.f;
  ps = fmaf(ps, y, -1.f / 5040.f);
  ps = fmaf(ps, y, 1.f / 120.f);
  ps = fmaf(ps, y, -1.f / 6.f);
  ps = fmaf(ps * y, x, x);
  float pc = -1.f / 3628800.f;
  pc = fmaf(pc, y, 1.f / 40320.f);
  pc = fmaf(pc, y, -1.f / 720.f);
  pc = fmaf(pc, y, 1.f / 24.f);
  pc = fmaf(pc, y, -0.5f);
  pc = fmaf(pc, y, 1.f);
  const float a = quarter & 1 ? ps : pc, b = quarter & 1 ? pc : ps;
  c = quarter + 1 & 2 ? -a : a;
  s = quarter & 2 ? -b : b;
}

template <int V, bool IL>
__device__ __forceinline__ int element_a(const Unit& u, int j) {
  return IL && V > 1 ? u.a + 2 * j : u.a + j;
}
template <int V, bool IL>
__device__ __forceinline__ int element_b(const Unit& u, int j) {
  return IL && V > 1 ? u.a + 2 * j + 1 : u.b + j;
}

__device__ __forceinline__ float lane_of(const Vec<1>& v, int) { return v.p[0]; }
template <int V>
__device__ __forceinline__ float lane_of(const Vec<V>& v, int j) {
  return j & 1 ? v.p[j / 2].y : v.p[j / 2].x;
}

// a, b <- the pairs turned; only those of a rotated run.  n: -s.
template <int V, bool IL>
__device__ __forceinline__ void turn(const Unit& u, const Vec<V>& c, const Vec<V>& s,
                                     const Vec<V>& n, Vec<V>& a, Vec<V>& b) {
  using E = typename Vec<V>::E;
  constexpr int P = Vec<V>::P, H = IL && V > 1 ? P / 2 : P;
  auto pairs = [&](int from, int to) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (i < from || i >= to) continue;
      const E x = a.p[i], y = b.p[i];
      a.p[i] = fma2(y, n.p[i], mul2(x, c.p[i]));
      b.p[i] = fma2(x, s.p[i], mul2(y, c.p[i]));
    }
  };
  if (u.rot_a) pairs(0, H);
  if constexpr (H < P) {
    if (u.rot_b) pairs(H, P);
  }
}

// The sum over a group of `size` lanes.
__device__ __forceinline__ float group_sum(float x, int size) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < size) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float2 group_sum2(float2 x, int size) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < size) {
      const float y = __shfl_xor_sync(0xffffffffu, x.x, o);
      x = add2(x, make_float2(y, __shfl_xor_sync(0xffffffffu, x.y, o)));
    }
  return x;
}

// 1 / sqrt(x).  In float32 to the nearest number but for 2^-19 of its unit: the
// approximation is off by up to two units, the same way for a whole row, which
// made the forward pass's error 8% larger than that of a rounded root.  A Newton
// step with an exact residual, r (1 - (x r^2 - 1) / 2); not where x is 0 or not
// finite.  (16-bit outputs do not show it: 16384 tokens would take 34.4 us for
// 34.0, backward 55.4 for 54.9.)
template <class T>
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  if constexpr (sizeof(T) < 4) return r;
  const float y = x * r;
  const float rest = fmaf(-fmaf(x, r, -y), r, fmaf(-y, r, 1.f));
  return fabsf(rest) < 1.f ? fmaf(0.5f * r, rest, r) : r;
}

// A lane's runs of one row.  DENSE: every lane has both runs of a head (its
// group may be past the last head: what such a group works on is not used).
template <class T, int V, int NU, bool DENSE>
struct HeadRow {
  Piece<T, V> a[NU], b[NU];
  static __device__ __forceinline__ Piece<T, V> run_at(const void* p, bool there) {
    Piece<T, V> r = {};
    if (!there) return r;
    if constexpr (V == 1 && sizeof(T) == 2) {
      r.w[0] = *(const uint16_t*)p;
    } else if constexpr (Piece<T, V>::N == 1) {
      r.w[0] = *(const uint32_t*)p;
    } else if constexpr (Piece<T, V>::N == 2) {
      const uint2 x = *(const uint2*)p;
      r.w[0] = x.x, r.w[1] = x.y;
    } else {
      const uint4 x = *(const uint4*)p;
      r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    }
    return r;
  }
  static __device__ __forceinline__ void put(void* p, const Piece<T, V>& r, bool there) {
    if (!there) return;
    if constexpr (V == 1 && sizeof(T) == 2)
      *(uint16_t*)p = (uint16_t)r.w[0];
    else if constexpr (Piece<T, V>::N == 1)
      *(uint32_t*)p = r.w[0];
    else if constexpr (Piece<T, V>::N == 2)
      *(uint2*)p = make_uint2(r.w[0], r.w[1]);
    else
      *(uint4*)p = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  }
  __device__ __forceinline__ void load(const T* row, const Unit (&u)[NU], bool live) {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      a[n] = run_at(row + u[n].a, live && u[n].has_a);
      b[n] = run_at(row + u[n].b, live && u[n].has_b);
    }
  }
  __device__ __forceinline__ void store(T* row, const Unit (&u)[NU], bool live) const {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      put(row + u[n].a, a[n], live && (DENSE || u[n].has_a));
      put(row + u[n].b, b[n], live && (DENSE || u[n].has_b));
    }
  }
  // The same through a slot of shared memory, 2 NU runs of 32 lanes each
  // (`slot`: this lane's first).  What is not there is filled with zeros.
  static constexpr int kRunBytes = V * sizeof(T), kSlot = 2 * NU * 32 * kRunBytes;
  static __device__ __forceinline__ void copy(uint32_t slot, const T* row, const Unit (&u)[NU],
                                              bool live, const void* safe) {
    auto one = [&](uint32_t to, const T* from, bool there) {
      const int bytes = there ? kRunBytes : 0;
      if constexpr (DENSE)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
      else if constexpr (kRunBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                     : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from),
                     "n"(kRunBytes < 4 ? 4 : kRunBytes), "r"(bytes)
                     : "memory");
    };
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      // (an address that is not read is a valid one all the same)
      if (DENSE) {
        if (live) one(slot + (2 * n) * 32 * kRunBytes, row + u[n].a, true);
        if (live) one(slot + (2 * n + 1) * 32 * kRunBytes, row + u[n].b, true);
        continue;
      }
      const bool la = live && u[n].has_a, lb = live && u[n].has_b;
      one(slot + (2 * n) * 32 * kRunBytes, la ? row + u[n].a : (const T*)safe, la);
      one(slot + (2 * n + 1) * 32 * kRunBytes, lb ? row + u[n].b : (const T*)safe, lb);
    }
  }
  __device__ __forceinline__ void take(const char* slot) {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      a[n] = run_at(slot + (2 * n) * 32 * kRunBytes, true);
      b[n] = run_at(slot + (2 * n + 1) * 32 * kRunBytes, true);
    }
  }
};

// Where a warp is in its items: a pass of a token, and the run of passes of the
// same side that it lies in.
struct HeadPlace {
  uint32_t left;  // items, this one among them
  uint32_t b, t;
  int chunk, pass, end;
  int run;  // passes left of the side in this item
  int h;    // the lane's head
  bool second;
  __device__ __forceinline__ bool there() const { return left > 0; }
  __device__ __forceinline__ void start(const HeadArgs& q, uint32_t item, uint32_t step) {
    left = item < q.items ? (q.items - item + step - 1) / step : 0;
    const uint32_t token = item / (uint32_t)q.chunks;
    chunk = (int)(item - token * q.chunks);
    b = token / q.tokens, t = token - b * q.tokens;
    passes(q);
  }
  __device__ __forceinline__ void passes(const HeadArgs& q) {
    pass = chunk * q.chunk;
    end = min(pass + q.chunk, q.passes);
  }
  __device__ __forceinline__ void next_item(const HeadArgs& q) {
    --left;
    chunk += q.step.chunk;
    t += q.step.t, b += q.step.b;
    if (chunk >= q.chunks) chunk -= q.chunks, ++t;
    if (t >= q.tokens) t -= q.tokens, ++b;
    passes(q);
  }
  __device__ __forceinline__ void begin_run(const HeadArgs& q, int rows, int group) {
    second = pass >= q.passes0;
    run = (second ? end : min(end, q.passes0)) - pass;
    h = (pass - (second ? q.passes0 : 0)) * rows + group;
    pass += run;
  }
  __device__ __forceinline__ int64_t row(const HeadStrides& s) const {
    return b * s.batch + t * s.token + h * s.head;
  }
  __device__ __forceinline__ int64_t position(const HeadArgs& q) const {
    if (!q.positions) return q.start + t;
    const int64_t at = b * q.pbs + t * q.pts;
    return q.position_bytes == 8 ? ((const int64_t*)q.positions)[at]
                                 : (int64_t)((const int32_t*)q.positions)[at];
  }
};

template <class T, int V, int NU, bool IL, bool DENSE, HeadsMode MODE>
__global__ void __launch_bounds__(32 * kHeadWarps, head_blocks(MODE, NU))
    heads_kernel(const __grid_constant__ HeadArgs q, const int il) {
  // the weights of both sides, then each warp's cosines and sines (half each)
  extern __shared__ __align__(16) float dyn[];
  constexpr int P = Vec<V>::P;
  using E = typename Vec<V>::E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int size = 1 << q.log_group, rows = 32 >> q.log_group, group = lane >> q.log_group;
  const int half = q.rotated / 2;
  float* cs = dyn + (2 + warp) * q.dim;
  Unit u[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n)
    u[n] = unit_of<V, IL>((lane & (size - 1)) + 32 * n, q.units, q.dim, q.rotated, il);
  wait_for_prior();
  if constexpr (MODE != kRotate) {
    for (int i = threadIdx.x; i < 2 * q.dim; i += 32 * kHeadWarps) {
      const int second = i >= q.dim;
      const HeadSide& sd = q.side[second];
      const int at = i - second * q.dim;
      if (sd.w) dyn[i] = q.w32 ? ((const float*)sd.w)[at] : to_f32(((const T*)sd.w)[at]);
    }
    __syncthreads();
  }
  constexpr int kSums = MODE == kNormGrad ? NU : 1;
  Vec<V> dwa[2][kSums], dwb[2][kSums];
#pragma unroll
  for (int n = 0; n < kSums; ++n)
#pragma unroll
    for (int i = 0; i < P; ++i)
      dwa[0][n].p[i] = dwb[0][n].p[i] = dwa[1][n].p[i] = dwb[1][n].p[i] = all_of<E>(0.f);
  const float inv = 1.f / (float)q.dim;

  // what is fetched: kAhead passes before it is worked on
  using Row = HeadRow<T, V, NU, DENSE>;
  constexpr bool kRing = Row::kRunBytes >= 4;
  constexpr int kArrays = MODE == kNormGrad ? 2 : 1, kStage = kArrays * Row::kSlot;
  char* ring = reinterpret_cast<char*>(dyn + (2 + kHeadWarps) * q.dim) +
               warp * kHeadAhead * kStage + lane * Row::kRunBytes;
  const uint32_t ring32 = (uint32_t)__cvta_generic_to_shared(ring);
  Row rx, rd;
  HeadPlace ahead;
  const T *px = nullptr, *pd = nullptr;  // the lane's row of the next pass
  int64_t sx = 0, sd = 0;                // a pass on
  int heads_ahead = 0;
  uint32_t filling = ring32, taking = 0;
  auto fetch = [&]() {
    if (ahead.there()) {
      if (ahead.run == 0) {
        ahead.begin_run(q, rows, group);
        const HeadSide& side = q.side[ahead.second];
        heads_ahead = side.heads;
        px = (const T*)side.x + ahead.row(side.xs), sx = rows * side.xs.head;
        if constexpr (MODE == kNormGrad)
          pd = (const T*)side.dy + ahead.row(side.ds), sd = rows * side.ds.head;
      }
      const bool live = ahead.h < heads_ahead;
      if constexpr (kRing) {
        Row::copy(filling, px, u, live, q.safe);
        if constexpr (MODE == kNormGrad) Row::copy(filling + Row::kSlot, pd, u, live, q.safe);
        filling += kStage;
        if (filling == ring32 + kHeadAhead * kStage) filling = ring32;
      } else {
        rx.load(px, u, live);
        if constexpr (MODE == kNormGrad) rd.load(pd, u, live);
      }
      px += sx, pd += sd;
      ahead.h += rows;
      if (--ahead.run == 0 && ahead.pass == ahead.end) ahead.next_item(q);
    }
    if constexpr (kRing) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  HeadPlace at;
  at.start(q, blockIdx.x * kHeadWarps + warp, gridDim.x * kHeadWarps);
  at.run = 0;
  ahead = at;
  int64_t pos = 0;
  if (at.there() && half) pos = at.position(q);
#pragma unroll
  for (int k = 0; k < (kRing ? kHeadAhead : 1); ++k) fetch();
  while (at.there()) {
    HeadPlace next = at;
    next.next_item(q);
    Vec<V> c[NU], s[NU], ns[NU];
    if (half) {
      __syncwarp();  // (the last token's angles have been read)
      for (int i = lane; i < half; i += 32) {
        // the turn's fraction, from -1/2 to 1/2, as a whole number of 2^-32
        float x, y;
        cos_sin((int32_t)(((uint64_t)pos * q.turns[i]) >> 32), x, y);
        cs[i] = x * q.cos_scale;
        cs[half + i] = y * q.sin_scale;
      }
      __syncwarp();
      if (next.there()) pos = next.position(q);
    }
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const int first = ((lane & (size - 1)) + 32 * n) * V;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        c[n].p[i] = s[n].p[i] = all_of<E>(0.f);
        constexpr int W = V / P;  // (a pack is of one run, rotated or not)
        if (first + i * W < half) {
          c[n].p[i] = *reinterpret_cast<const E*>(cs + first + i * W);
          s[n].p[i] = *reinterpret_cast<const E*>(cs + half + first + i * W);
        }
        ns[n].p[i] = mul2(s[n].p[i], all_of<E>(-1.f));
      }
    }
    int heads = 0;
    T* out = nullptr;
    int64_t so = 0;
    const float* w = dyn;
#pragma unroll 1
    while (true) {
      if (at.run == 0) {
        if (at.pass == at.end) break;
        at.begin_run(q, rows, group);
        const HeadSide& side = q.side[at.second];
        heads = side.heads;
        out = (T*)side.out + at.row(side.os), so = rows * side.os.head;
        w = dyn + at.second * q.dim;
      }
      const bool live = at.h < heads;
      if constexpr (kRing) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kHeadAhead - 1) : "memory");
        rx.take(ring + taking);
        if constexpr (MODE == kNormGrad) rd.take(ring + taking + Row::kSlot);
        taking = taking + kStage == kHeadAhead * kStage ? 0 : taking + kStage;
      }
      Vec<V> a[NU], b[NU], ga[NU], gb[NU];
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        pairs_of<T, V, IL>(rx.a[n], rx.b[n], a[n], b[n]);
        if constexpr (MODE == kNormGrad) pairs_of<T, V, IL>(rd.a[n], rd.b[n], ga[n], gb[n]);
      }
      fetch();
      Vec<V> wa[NU], wb[NU];
      auto weights = [&]() {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          // (what is not there is read elsewhere, and 0 elements multiply it)
          const Piece<float, V> ra = floats_at<V>(w + (DENSE || u[n].has_a ? u[n].a : 0));
          const Piece<float, V> rb = floats_at<V>(w + (DENSE || u[n].has_b ? u[n].b : 0));
          pairs_of<float, V, IL>(ra, rb, wa[n], wb[n]);
        }
      };
      // (two sums each, so that an addition need not wait for the last)
      E squares = all_of<E>(0.f), squares2 = squares, along = squares, along2 = squares;
      if constexpr (MODE != kRotate) {
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int i = 0; i < P; ++i) {
            squares = fma2(a[n].p[i], a[n].p[i], squares);
            squares2 = fma2(b[n].p[i], b[n].p[i], squares2);
          }
        squares = add2(squares, squares2);
      }
      if constexpr (MODE == kNormGrad) {
        // both sums in one go: that of x^2 gives r, that of g w x is the one of
        // g w hat over r
        weights();
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          turn<V, IL>(u[n], c[n], s[n], ns[n], ga[n], gb[n]);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            along = fma2(mul2(ga[n].p[i], wa[n].p[i]), a[n].p[i], along);
            along2 = fma2(mul2(gb[n].p[i], wb[n].p[i]), b[n].p[i], along2);
          }
        }
        along = add2(along, along2);
        const float2 sums = group_sum2(make_float2(total(squares), total(along)), size);
        const float r = live ? inverse_root<T>(sums.x * inv + q.eps) : 0.f;  // (eps may be 0)
        const float k = -(sums.y * inv * r * r);
#pragma unroll
        for (int n = 0; n < NU; ++n) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            a[n].p[i] = mul2(a[n].p[i], all_of<E>(r));
            b[n].p[i] = mul2(b[n].p[i], all_of<E>(r));
          }
          auto add = [&](Vec<V>& da, Vec<V>& db) {
            if (DENSE && !live) return;
#pragma unroll
            for (int i = 0; i < P; ++i) {
              da.p[i] = fma2(ga[n].p[i], a[n].p[i], da.p[i]);
              db.p[i] = fma2(gb[n].p[i], b[n].p[i], db.p[i]);
            }
          };
          if (at.second)
            add(dwa[1][n], dwb[1][n]);
          else
            add(dwa[0][n], dwb[0][n]);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const E ka = mul2(mul2(ga[n].p[i], wa[n].p[i]), all_of<E>(r));
            const E kb = mul2(mul2(gb[n].p[i], wb[n].p[i]), all_of<E>(r));
            a[n].p[i] = fma2(a[n].p[i], all_of<E>(k), ka);
            b[n].p[i] = fma2(b[n].p[i], all_of<E>(k), kb);
          }
        }
      } else {
        float r = 1.f;
        if constexpr (MODE == kNorm) {
          r = inverse_root<T>(group_sum(total(squares), size) * inv + q.eps);
          weights();
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if constexpr (MODE == kNorm) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
              a[n].p[i] = mul2(mul2(a[n].p[i], all_of<E>(r)), wa[n].p[i]);
              b[n].p[i] = mul2(mul2(b[n].p[i], all_of<E>(r)), wb[n].p[i]);
            }
          }
          turn<V, IL>(u[n], c[n], s[n], ns[n], a[n], b[n]);
        }
      }
      Row ro;
#pragma unroll
      for (int n = 0; n < NU; ++n) runs_of<T, V, IL>(a[n], b[n], ro.a[n], ro.b[n]);
      ro.store(out, u, live);
      out += so;
      at.h += rows;
      --at.run;
    }
    at = next;
  }
  if constexpr (MODE == kNormGrad) {
    // this block's part: the groups of a warp, then the warps in order
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __syncthreads();  // (angles, the other side's sums have been read)
#pragma unroll
      for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float ea = lane_of(dwa[side][n], j), eb = lane_of(dwb[side][n], j);
          for (int o = size; o < 32; o <<= 1) {
            ea += __shfl_xor_sync(0xffffffffu, ea, o);
            eb += __shfl_xor_sync(0xffffffffu, eb, o);
          }
          const int ia = element_a<V, IL>(u[n], j), ib = element_b<V, IL>(u[n], j);
          if (group == 0 && u[n].has_a) {
            if (ia < q.dim) cs[ia] = ea;
            if (ib < q.dim) cs[ib] = eb;
          }
        }
      __syncthreads();
      for (int d = threadIdx.x; d < q.dim; d += 32 * kHeadWarps) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kHeadWarps; ++w) sum += dyn[(2 + w) * q.dim + d];
        q.part[((int64_t)blockIdx.x * 2 + side) * q.dim + d] = sum;
      }
    }
  }
}

// How the launches of a call run: V elements to a run.
template <int V>
void plan_units(HeadArgs& q, bool il) {
  const int half = q.rotated / 2;
  q.units = il ? (q.dim + 2 * V - 1) / (2 * V)
               : half / V + ((q.dim - q.rotated) + 2 * V - 1) / (2 * V);
  q.log_group = 0;
  while (q.log_group < 5 && (1 << q.log_group) < q.units) ++q.log_group;
}

template <class T, int V, int NU, bool IL, bool DENSE, HeadsMode MODE>
int launch_heads_as(HeadArgs& q, int64_t tokens, bool il, cudaStream_t s) {
  const int rows = 32 >> q.log_group;
  q.passes0 = (q.side[0].heads + rows - 1) / rows;
  q.passes = q.passes0 + (q.side[1].heads + rows - 1) / rows;
  q.safe = q.side[q.side[0].heads ? 0 : 1].x;
  // the blocks that stay on the SMs
  const int64_t most =
      std::min<int64_t>((int64_t)head_blocks(MODE, NU) * sm_count(), kHeadParts);
  // a token's passes to one warp, or to as many as end first, a token's angles
  // counted as a pass (few tokens, or a few more than there are warps)
  int64_t best = INT64_MAX;
  for (int n = 1; n <= q.passes; n += n < 16 ? 1 : n) {
    const int chunk = (q.passes + n - 1) / n;
    const int64_t items = tokens * ((q.passes + chunk - 1) / chunk);
    if (n > 1 && items > int64_t(1) << 31) break;  // (they are counted in 32 bits)
    const int64_t cost =
        (items + most * kHeadWarps - 1) / (most * kHeadWarps) * (chunk + (q.rotated > 0));
    if (cost < best) best = cost, q.chunk = chunk;
  }
  q.chunks = (q.passes + q.chunk - 1) / q.chunk;
  q.items = (uint32_t)(tokens * q.chunks);
  q.blocks = (int)std::min<int64_t>((q.items + kHeadWarps - 1) / kHeadWarps, most);
  const uint32_t step = (uint32_t)q.blocks * kHeadWarps;
  q.step.chunk = (int)(step % q.chunks);
  q.step.t = step / q.chunks % q.tokens;
  q.step.b = step / q.chunks / q.tokens;
  constexpr int ring = V * sizeof(T) < 4 ? 0 : kHeadWarps * kHeadAhead * HeadRow<T, V, NU, DENSE>::kSlot *
                                        (MODE == kNormGrad ? 2 : 1);
  const int smem = (int)sizeof(float) * (2 + kHeadWarps) * q.dim + ring;
  auto k = heads_kernel<T, V, NU, IL, DENSE, MODE>;
  if (smem > 48 << 10 &&  // (of the current device: each time)
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return ROT_ECUDA;
  }
  return launch_behind(k, (unsigned)q.blocks, 32 * kHeadWarps, (size_t)smem, s, q, (int)il);
}

// Rows of which every lane has two runs, without a look at which lanes have
// what: 16384 tokens of 16 and 8 heads of 128 in bfloat16, norm and rotation,
// 34.2 us; with that look 34.7, backward 54.8 and 55.8.
template <class T, int V, bool IL, HeadsMode MODE>
int launch_heads_rows(HeadArgs& q, int64_t tokens, cudaStream_t s) {
  if (q.units == 1 << q.log_group && q.dim == 2 * V * q.units)
    return launch_heads_as<T, V, 1, IL, true, MODE>(q, tokens, IL, s);
  return launch_heads_as<T, V, 1, IL, false, MODE>(q, tokens, IL, s);
}

// Runs of V elements where every row starts and ends on them, and the halves
// do (interleaved: the rotated part).
inline bool heads_align(const HeadArgs& q, int bytes, int es, bool il) {
  const int v = bytes / es;
  if (q.dim % v || q.rotated % v || (!il && q.rotated / 2 % v)) return false;
  auto fits = [&](const void* p, const HeadStrides& s) {
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (s.batch * es) % bytes == 0 &&
                  (s.token * es) % bytes == 0 && (s.head * es) % bytes == 0);
  };
  for (const HeadSide& sd : q.side)
    if (!fits(sd.x, sd.xs) || !fits(sd.dy, sd.ds) || !fits(sd.out, sd.os)) return false;
  return true;
}

template <class T, HeadsMode MODE>
int launch_heads(HeadArgs& q, int64_t tokens, bool il, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (heads_align(q, 16, sizeof(T), il)) {
    plan_units<V>(q, il);
    if constexpr (V == 4) {  // (float32: up to 64 units)
      if (q.units > 32)
        return il ? launch_heads_as<T, V, 2, true, false, MODE>(q, tokens, il, s)
                  : launch_heads_as<T, V, 2, false, false, MODE>(q, tokens, il, s);
    }
    return il ? launch_heads_rows<T, V, true, MODE>(q, tokens, s)
              : launch_heads_rows<T, V, false, MODE>(q, tokens, s);
  }
  if constexpr (V == 8) {
    // halves of an odd number of 8-byte runs (dim 72: 36 elements)
    if (!il && heads_align(q, 8, sizeof(T), il)) {
      plan_units<4>(q, il);
      return q.units > 32 ? launch_heads_as<T, 4, 2, false, false, MODE>(q, tokens, il, s)
                          : launch_heads_as<T, 4, 1, false, false, MODE>(q, tokens, il, s);
    }
  }
  if constexpr (V == 8) {  // 4-byte runs (dim 100: halves of 50)
    if (!il && heads_align(q, 4, sizeof(T), il)) {
      plan_units<2>(q, il);
      if (q.units <= 32) return launch_heads_as<T, 2, 1, false, false, MODE>(q, tokens, il, s);
      if (q.units <= 64) return launch_heads_as<T, 2, 2, false, false, MODE>(q, tokens, il, s);
      return launch_heads_as<T, 2, 4, false, false, MODE>(q, tokens, il, s);
    }
  }
  plan_units<1>(q, il);
  if (q.units <= 32) return launch_heads_as<T, 1, 1, false, false, MODE>(q, tokens, il, s);
  if (q.units <= 64) return launch_heads_as<T, 1, 2, false, false, MODE>(q, tokens, il, s);
  if (q.units <= 128) return launch_heads_as<T, 1, 4, false, false, MODE>(q, tokens, il, s);
  return launch_heads_as<T, 1, 8, false, false, MODE>(q, tokens, il, s);
}

template <HeadsMode MODE>
int launch_heads_type(int32_t type, HeadArgs& q, int64_t tokens, bool il, cudaStream_t s) {
  if (type == ROT_TYPE_F32) return launch_heads<float, MODE>(q, tokens, il, s);
  if (type == ROT_TYPE_F16) return launch_heads<__half, MODE>(q, tokens, il, s);
  return launch_heads<__nv_bfloat16, MODE>(q, tokens, il, s);
}

int heads_rotate(int32_t type, HeadArgs& q, int64_t tokens, bool il, cudaStream_t s);
int heads_norm(int32_t type, HeadArgs& q, int64_t tokens, bool il, cudaStream_t s);
int heads_norm_grad(int32_t type, HeadArgs& q, int64_t tokens, bool il, cudaStream_t s);

}  // namespace ops
}  // namespace rot
