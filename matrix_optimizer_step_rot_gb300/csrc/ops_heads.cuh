// Rotary positions and the norm of queries and keys (include/rot_ops.h): one
// kernel for the rotation, the norm with it, and the norm's backward pass.
// Bound by HBM: each element is read once (twice two arrays backward) and
// written once.
//
// A row is one head of one token.  A group of 2^k lanes takes it, a lane two
// runs of V elements: those whose elements turn together.  For pairs (i, i +
// rotated / 2) these are runs of the two halves, interleaved two runs next to
// each other; either way a lane holds a[j] and b[j] of the pairs u V + j, u
// its place in the group, and all arithmetic is the same.  What is not rotated
// follows in runs of its own.
//
// A warp takes a token's heads one after the other (or a part of them, where
// there are few tokens): the token's angles are worked out once, a pair to a
// lane, and shared through shared memory.  A row's loads are issued before the
// row ahead of it is worked on.
#pragma once

#include <algorithm>

#include "ops_common.cuh"
#include "profile.h"

namespace rot {
namespace ops {

enum HeadsMode { kRotate = 0, kNorm = 1, kNormGrad = 2 };

constexpr int kHeadWarps = 4;         // per block
constexpr int kHeadParts = 1024;      // most blocks of a backward pass: its partial sums
constexpr int kHeadBlocksPerSm = 5;   // backward

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
  int32_t chunk = 1;     // heads to a warp
  uint32_t chunks = 1;   // of a token
  uint32_t items = 0;    // chunks of all tokens
};

struct HeadArgs {
  HeadSide side[2];
  uint32_t blocks0 = 0, blocks1 = 0;  // of the sides
  uint32_t tokens = 1;   // of a batch entry
  int32_t dim = 0, rotated = 0, units = 0, log_group = 0;
  const uint64_t* turns = nullptr;
  const void* positions = nullptr;
  int32_t position_bytes = 8;
  int64_t pbs = 0, pts = 0, start = 0;
  float cos_scale = 1.f, sin_scale = 1.f;  // the magnitude; sin's sign turns the other way
  int32_t w32 = 0;
  float eps = 0.f;
  float* part = nullptr;  // backward: [blocks][dim]
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

// The lane's runs as a[] and b[] of its pairs, and back.
template <class T, int V, bool IL>
__device__ __forceinline__ void pairs_of(const Run<T, V>& ra, const Run<T, V>& rb, Vec<V>& a,
                                         Vec<V>& b) {
  if constexpr (IL && V > 1) {
    static_assert(V % 4 == 0, "a pack comes from one run");
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const Run<T, V>& r = i < V / 4 ? ra : rb;
      const int k = 4 * i % V;
      a.p[i] = unpack2(r.v[k], r.v[k + 2]);
      b.p[i] = unpack2(r.v[k + 1], r.v[k + 3]);
    }
  } else {
    a = unpack<T, V>(ra), b = unpack<T, V>(rb);
  }
}
template <class T, int V, bool IL>
__device__ __forceinline__ void runs_of(const Vec<V>& a, const Vec<V>& b, Run<T, V>& ra,
                                        Run<T, V>& rb) {
  if constexpr (IL && V > 1) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      Run<T, V>& r = i < V / 4 ? ra : rb;
      const int k = 4 * i % V;
      pack2(make_float2(a.p[i].x, b.p[i].x), r.v[k], r.v[k + 1]);
      pack2(make_float2(a.p[i].y, b.p[i].y), r.v[k + 2], r.v[k + 3]);
    }
  } else {
    ra = pack<T, V>(a), rb = pack<T, V>(b);
  }
}

// V consecutive elements of a weight vector of float32 or T.
template <class T, int V>
__device__ __forceinline__ Run<float, V> weights_at(const void* w, int w32, int at) {
  Run<float, V> r;
#pragma unroll
  for (int j = 0; j < V; ++j)
    r.v[j] = w32 ? ((const float*)w)[at + j] : to_f32(((const T*)w)[at + j]);
  return r;
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

// a, b <- the pairs turned; only those of a rotated run.
template <int V, bool IL>
__device__ __forceinline__ void turn(const Unit& u, const Vec<V>& c, const Vec<V>& s, Vec<V>& a,
                                     Vec<V>& b) {
  using E = typename Vec<V>::E;
  constexpr int P = Vec<V>::P, H = IL && V > 1 ? P / 2 : P;
  auto pairs = [&](int from, int to) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (i < from || i >= to) continue;
      const E x = a.p[i], y = b.p[i];
      const E ms = mul2(s.p[i], all_of<E>(-1.f));
      a.p[i] = fma2(y, ms, mul2(x, c.p[i]));
      b.p[i] = fma2(x, s.p[i], mul2(y, c.p[i]));
    }
  };
  if (u.rot_a) pairs(0, H);
  if constexpr (H < P) {
    if (u.rot_b) pairs(H, P);
  }
}

template <class T, int V, int NU>
struct HeadRow {
  Run<T, V> a[NU], b[NU];
  __device__ __forceinline__ void load(const T* row, const Unit (&u)[NU], bool live) {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      a[n] = b[n] = Run<T, V>{};
      if (live && u[n].has_a) a[n] = *reinterpret_cast<const Run<T, V>*>(row + u[n].a);
      if (live && u[n].has_b) b[n] = *reinterpret_cast<const Run<T, V>*>(row + u[n].b);
    }
  }
  __device__ __forceinline__ void store(T* row, const Unit (&u)[NU], bool live) const {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      if (live && u[n].has_a) *reinterpret_cast<Run<T, V>*>(row + u[n].a) = a[n];
      if (live && u[n].has_b) *reinterpret_cast<Run<T, V>*>(row + u[n].b) = b[n];
    }
  }
};

template <class T, int V, int NU, bool IL, HeadsMode MODE>
__global__ void __launch_bounds__(32 * kHeadWarps)
    heads_kernel(const __grid_constant__ HeadArgs q, const int il) {
  extern __shared__ __align__(16) float dyn[];
  constexpr int P = Vec<V>::P;
  using E = typename Vec<V>::E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool second = blockIdx.x >= q.blocks0;
  const HeadSide& sd = q.side[second];
  const uint32_t blocks = second ? gridDim.x - q.blocks0 : q.blocks0;
  const uint32_t block = second ? blockIdx.x - q.blocks0 : blockIdx.x;
  const int group = lane >> q.log_group, size = 1 << q.log_group, rows = 32 >> q.log_group;
  const int half = q.rotated / 2;
  float* cs = dyn + warp * q.dim;  // half cosines, half sines
  Unit u[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n)
    u[n] = unit_of<V, IL>((lane & (size - 1)) + 32 * n, q.units, q.dim, q.rotated, il);
  Vec<V> wa[NU], wb[NU], dwa[NU], dwb[NU];
  if constexpr (MODE != kRotate) {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      Run<float, V> ra{}, rb{};
      if (u[n].has_a) ra = weights_at<T, V>(sd.w, q.w32, u[n].a);
      if (u[n].has_b) rb = weights_at<T, V>(sd.w, q.w32, u[n].b);
      pairs_of<float, V, IL>(ra, rb, wa[n], wb[n]);
#pragma unroll
      for (int i = 0; i < P; ++i) dwa[n].p[i] = dwb[n].p[i] = all_of<E>(0.f);
    }
  }
  const float inv = 1.f / (float)q.dim;
  for (uint32_t item = block * kHeadWarps + warp; item < sd.items; item += blocks * kHeadWarps) {
    const uint32_t token = item / sd.chunks, b = token / q.tokens, t = token - b * q.tokens;
    const int h0 = (int)(item - token * sd.chunks) * sd.chunk + group;
    const int end = min(h0 - group + sd.chunk, sd.heads);
    const T* x = (const T*)sd.x + b * sd.xs.batch + t * sd.xs.token + h0 * sd.xs.head;
    const T* dy = (const T*)sd.dy + b * sd.ds.batch + t * sd.ds.token + h0 * sd.ds.head;
    T* out = (T*)sd.out + b * sd.os.batch + t * sd.os.token + h0 * sd.os.head;
    HeadRow<T, V, NU> rx, rd;
    rx.load(x, u, h0 < end);
    if constexpr (MODE == kNormGrad) rd.load(dy, u, h0 < end);
    if (half) {
      int64_t pos = q.start + t;
      if (q.positions) {
        const int64_t at = b * q.pbs + t * q.pts;
        pos = q.position_bytes == 8 ? ((const int64_t*)q.positions)[at]
                                    : (int64_t)((const int32_t*)q.positions)[at];
      }
      __syncwarp();  // (the last token's angles have been read)
      for (int i = lane; i < half; i += 32) {
        // the turn's fraction, from -1/2 to 1/2, as a whole number of 2^-32
        const int32_t turn = (int32_t)(((uint64_t)pos * q.turns[i]) >> 32);
        float s, c;
        sincospif((float)turn * 0x1p-31f, &s, &c);
        cs[i] = c * q.cos_scale;
        cs[half + i] = s * q.sin_scale;
      }
      __syncwarp();
    }
    Vec<V> c[NU], s[NU];
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
      }
    }
    for (int h = h0; h - group < end; h += rows) {
      const bool live = h < end;
      Vec<V> a[NU], b2[NU], ga[NU], gb[NU];
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        pairs_of<T, V, IL>(rx.a[n], rx.b[n], a[n], b2[n]);
        if constexpr (MODE == kNormGrad) pairs_of<T, V, IL>(rd.a[n], rd.b[n], ga[n], gb[n]);
      }
      x += rows * sd.xs.head;
      rx.load(x, u, h + rows < end);
      if constexpr (MODE == kNormGrad) {
        dy += rows * sd.ds.head;
        rd.load(dy, u, h + rows < end);
      }
      float rstd = 1.f;
      if constexpr (MODE != kRotate) {
        E sum = all_of<E>(0.f);
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int i = 0; i < P; ++i)
            sum = fma2(a[n].p[i], a[n].p[i], fma2(b2[n].p[i], b2[n].p[i], sum));
        float ss = total(sum);
        for (int o = size >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rstd = live ? __frsqrt_rn(ss * inv + q.eps) : 0.f;  // (eps may be 0)
      }
      if constexpr (MODE == kNormGrad) {
        E along = all_of<E>(0.f);
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          turn<V, IL>(u[n], c[n], s[n], ga[n], gb[n]);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            a[n].p[i] = mul2(a[n].p[i], all_of<E>(rstd));
            b2[n].p[i] = mul2(b2[n].p[i], all_of<E>(rstd));
            dwa[n].p[i] = fma2(ga[n].p[i], a[n].p[i], dwa[n].p[i]);
            dwb[n].p[i] = fma2(gb[n].p[i], b2[n].p[i], dwb[n].p[i]);
            ga[n].p[i] = mul2(ga[n].p[i], wa[n].p[i]);
            gb[n].p[i] = mul2(gb[n].p[i], wb[n].p[i]);
            along = fma2(ga[n].p[i], a[n].p[i], fma2(gb[n].p[i], b2[n].p[i], along));
          }
        }
        float m = total(along);
        for (int o = size >> 1; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        m *= -inv;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int i = 0; i < P; ++i) {
            a[n].p[i] = mul2(fma2(a[n].p[i], all_of<E>(m), ga[n].p[i]), all_of<E>(rstd));
            b2[n].p[i] = mul2(fma2(b2[n].p[i], all_of<E>(m), gb[n].p[i]), all_of<E>(rstd));
          }
      } else {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if constexpr (MODE == kNorm) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
              a[n].p[i] = mul2(mul2(a[n].p[i], all_of<E>(rstd)), wa[n].p[i]);
              b2[n].p[i] = mul2(mul2(b2[n].p[i], all_of<E>(rstd)), wb[n].p[i]);
            }
          }
          turn<V, IL>(u[n], c[n], s[n], a[n], b2[n]);
        }
      }
      HeadRow<T, V, NU> ro;
#pragma unroll
      for (int n = 0; n < NU; ++n) runs_of<T, V, IL>(a[n], b2[n], ro.a[n], ro.b[n]);
      ro.store(out, u, live);
      out += rows * sd.os.head;
    }
  }
  if constexpr (MODE == kNormGrad) {
    // this block's part: the groups of a warp, then the warps in order
    __syncthreads();  // (the angles have been read)
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float ea = lane_of(dwa[n], j), eb = lane_of(dwb[n], j);
        for (int o = size; o < 32; o <<= 1) {
          ea += __shfl_xor_sync(0xffffffffu, ea, o);
          eb += __shfl_xor_sync(0xffffffffu, eb, o);
        }
        const int at = element_a<V, IL>(u[n], j), bt = element_b<V, IL>(u[n], j);
        if (group == 0 && u[n].has_a) {
          if (at < q.dim) cs[at] = ea;
          if (bt < q.dim) cs[bt] = eb;
        }
      }
    __syncthreads();
    for (int d = threadIdx.x; d < q.dim; d += 32 * kHeadWarps) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kHeadWarps; ++w) sum += dyn[w * q.dim + d];
      q.part[(int64_t)blockIdx.x * q.dim + d] = sum;
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

template <class T, int V, int NU, bool IL, HeadsMode MODE>
int launch_heads_as(HeadArgs& q, int64_t tokens, bool il, cudaStream_t s) {
  const int rows = 32 >> q.log_group;
  uint32_t blocks[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    HeadSide& sd = q.side[i];
    if (!sd.heads) continue;
    const int passes = (sd.heads + rows - 1) / rows;
    // few tokens: their heads to several warps, so that there are 8 for each SM
    const int64_t most = std::max<int64_t>(1, 8ll * sm_count() / std::max<int64_t>(tokens, 1));
    const int64_t chunks = std::min<int64_t>(passes, most);
    sd.chunk = (int)((passes + chunks - 1) / chunks) * rows;
    sd.chunks = (uint32_t)((sd.heads + sd.chunk - 1) / sd.chunk);
    sd.items = (uint32_t)(tokens * sd.chunks);
    blocks[i] = (sd.items + kHeadWarps - 1) / kHeadWarps;
  }
  if (MODE == kNormGrad) {
    // persistent blocks, the sides' shares as their heads'
    const uint32_t most = (uint32_t)std::min(kHeadParts, kHeadBlocksPerSm * sm_count());
    if (blocks[0] + blocks[1] > most) {
      const int64_t heads = q.side[0].heads + q.side[1].heads;
      const uint32_t first = (uint32_t)std::max<int64_t>(1, (int64_t)most * q.side[0].heads / heads);
      blocks[0] = std::min(blocks[0], q.side[1].heads ? std::min(first, most - 1) : most);
      blocks[1] = std::min(blocks[1], most - blocks[0]);
    }
  }
  q.blocks0 = blocks[0], q.blocks1 = blocks[1];
  heads_kernel<T, V, NU, IL, MODE>
      <<<blocks[0] + blocks[1], 32 * kHeadWarps, sizeof(float) * kHeadWarps * q.dim, s>>>(q, il);
  return launched();
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
        return il ? launch_heads_as<T, V, 2, true, MODE>(q, tokens, il, s)
                  : launch_heads_as<T, V, 2, false, MODE>(q, tokens, il, s);
    }
    return il ? launch_heads_as<T, V, 1, true, MODE>(q, tokens, il, s)
              : launch_heads_as<T, V, 1, false, MODE>(q, tokens, il, s);
  }
  if constexpr (V == 8) {
    // halves of an odd number of 8-byte runs (dim 72: 36 elements)
    if (!il && heads_align(q, 8, sizeof(T), il)) {
      plan_units<4>(q, il);
      return q.units > 32 ? launch_heads_as<T, 4, 2, false, MODE>(q, tokens, il, s)
                          : launch_heads_as<T, 4, 1, false, MODE>(q, tokens, il, s);
    }
  }
  plan_units<1>(q, il);
  if (q.units <= 32) return launch_heads_as<T, 1, 1, false, MODE>(q, tokens, il, s);
  if (q.units <= 64) return launch_heads_as<T, 1, 2, false, MODE>(q, tokens, il, s);
  if (q.units <= 128) return launch_heads_as<T, 1, 4, false, MODE>(q, tokens, il, s);
  return launch_heads_as<T, 1, 8, false, MODE>(q, tokens, il, s);
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
