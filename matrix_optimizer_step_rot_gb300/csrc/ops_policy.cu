// Log-probabilities of tokens and the clipped policy loss with its gradient
// (include/rot_ops.h).  Bound by HBM: one read of the logits, one write of
// their gradient.  Log-probabilities alone, 2049 x 100277 in bfloat16: 75 us,
// 5.5 TB/s.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "ops_common.cuh"
#include "profile.h"

namespace rot {
namespace ops {
namespace {

struct Policy {
  const void* logits;
  const int64_t* targets;
  const float *old, *ref, *adv, *weights;
  float *logp, *terms;
  void* d;  // gradient, or null
  int64_t ldl, ldd, tokens;
  int vocab;
  int loss;  // terms (and the gradient) as well, not log-probabilities alone
  float lo, hi, kl, scale;
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kAhead = 4;  // 16-byte loads of a thread in flight
// Up to here a float32 product is within 1/4 of x log2(e), so that the largest
// exponential of a row is within 2^-0.75 and 2^0.75.
constexpr float kMostScale = 4194304.f;  // 2^22

// Sum of exponentials on a running scale: the sum of 2^(x log2(e) - o) with a
// whole number o near the largest x log2(e), so that o is exact, no rounding
// of it enters the sum, and sums on different scales join by powers of two.
// One fused multiply-add and one exponential per element.
struct ScaledSum {
  float o, s;  // o = -inf: nothing but -inf yet
};
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// what is subtracted: 0 for o = -inf, so that 2^(-inf - o) stays 0
__device__ __forceinline__ float base_of(float o) { return o == -INFINITY ? 0.f : o; }
__device__ __forceinline__ ScaledSum join(ScaledSum a, ScaledSum b) {
  ScaledSum r;
  r.o = fmaxf(a.o, b.o);
  const float o = base_of(r.o);
  r.s = a.s * exp2_fast(a.o - o) + b.s * exp2_fast(b.o - o);
  return r;
}

// 2^((x - m) log2(e) - o) of both halves.
__device__ __forceinline__ float2 exp_pair(float2 x, float m, float o) {
  const float2 t = fma2(add2(x, both(-m)), both(kLog2e), both(-o));
  return make_float2(exp2_fast(t.x), exp2_fast(t.y));
}

// The largest of a run (NaN are passed over: their exponentials carry them on).
template <int U>
__device__ __forceinline__ float largest(const Run<float, U>& r) {
  float m = r.v[0];
#pragma unroll
  for (int k = 1; k < U; ++k) m = fmaxf(m, r.v[k]);
  return m;
}
__device__ __forceinline__ float largest(const Run<__half, 8>& r) {
  __half2 m = __halves2half2(r.v[0], r.v[1]);
#pragma unroll
  for (int k = 2; k < 8; k += 2) m = __hmax2(m, __halves2half2(r.v[k], r.v[k + 1]));
  return to_f32(__hmax(__low2half(m), __high2half(m)));
}
__device__ __forceinline__ float largest(const Run<__nv_bfloat16, 8>& r) {
  __nv_bfloat162 m = __halves2bfloat162(r.v[0], r.v[1]);
#pragma unroll
  for (int k = 2; k < 8; k += 2) m = __hmax2(m, __halves2bfloat162(r.v[k], r.v[k + 1]));
  return to_f32(__hmax(__low2bfloat16(m), __high2bfloat16(m)));
}

// n runs more.
template <class T, int U, int N>
__device__ __forceinline__ void add_runs(ScaledSum& t, const Run<T, U> (&r)[N]) {
  float m = largest(r[0]);
#pragma unroll
  for (int j = 1; j < N; ++j) m = fmaxf(m, largest(r[j]));
  const float o1 = fmaxf(t.o, rintf(m * kLog2e)), o = base_of(o1);
  float2 s[2] = {make_float2(t.s * exp2_fast(t.o - o), 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const Vec<U> f = unpack(r[j]);
#pragma unroll
    for (int k = 0; k < U / 2; ++k) {
      const float2 e = fma2(f.p[k], both(kLog2e), both(-o));
      s[k & 1] = add2(s[k & 1], make_float2(exp2_fast(e.x), exp2_fast(e.y)));
    }
  }
  t.o = o1;
  t.s = total(add2(s[0], s[1]));
}

// One CTA's share of a row: 16-byte runs v0 .. v1 - 1, run i starting at
// element head + i U; the elements before the first run and after the last
// one belong to the first and last CTA of the row.
struct Share {
  int head, runs, v0, v1;
};
template <class T, int U>
__device__ __forceinline__ Share share_of(const T* z, int vocab, int rank, int ranks) {
  Share s;
  s.head = min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) % 16 / sizeof(T)));
  s.runs = (vocab - s.head) / U;
  const int per = (s.runs + ranks - 1) / ranks;
  s.v0 = min(s.runs, rank * per);
  s.v1 = min(s.runs, s.v0 + per);
  return s;
}
// Edge element of this thread, or -1: the first CTA's threads take the head,
// the last one's the tail (each shorter than a run).
template <int U>
__device__ __forceinline__ int edge_of(const Share& s, int vocab, int rank, int ranks) {
  const int t = threadIdx.x;
  if (rank == 0 && t < s.head) return t;
  const int tail = s.head + s.runs * U;
  if (rank == ranks - 1 && t >= 16 && t - 16 < vocab - tail) return tail + t - 16;
  return -1;
}

// The log-probability (x log2(e) - o - log2(s)) ln 2 as a float32 and what its
// rounding leaves.  log2(e) is the float32 that the sum's exponents were formed
// with: whatever all of a row's logits have in common then cancels, and what
// that float32 lacks is 1.3e-8 of the distance between logits alone.  The
// product, both differences and the product with ln 2 carry their rounding
// errors along (Knuth's exact sum of two), and s = 2^k f has its whole exponents
// taken off exactly, so that a ratio loses nothing to a logp of 10 being rounded
// to 2^-21.
__device__ __forceinline__ float rounded_off(float a, float b, float sum) {
  const float t = sum - a;
  return (a - (sum - t)) + (b - t);
}
__device__ __forceinline__ float log_prob(float x, float o, float s, float& rest) {
  constexpr float kLn2Rest = -1.9046542999e-9f;
  const float hi = x * kLog2e;
  rest = 0.f;
  // (x log2(e) is beyond float32's range before x is: a float32's or bfloat16's
  // lowest value as a mask stays finite)
  if (!(fabsf(hi) < INFINITY) || !(s < INFINITY)) return x - kLn2 * (o + log2f(s));
  const float lo = fmaf(x, kLog2e, -hi);
  const int k = (__float_as_int(s) - 0x3F400000) >> 23;  // f in [0.75, 1.5)
  const float f = __int_as_float(__float_as_int(s) - (k << 23));
  const float whole = -(o + (float)k), d = hi + whole;
  const float r = (lo + rounded_off(hi, whole, d)) - log2f(f);
  const float t = d + r, e = rounded_off(d, r, t);
  const float p = kLn2 * t, q = fmaf(kLn2, t, -p) + (kLn2Rest * t + kLn2 * e);
  const float logp = p + q;
  rest = q - (logp - p);
  return logp;
}

// exp(r) - 1 - r, em = exp(r) - 1.  Near 0 (a policy next to its reference) the
// two agree to r^2 / 2 and their difference keeps few bits: the Taylor series up
// to r^8 / 8!, what follows being below 2^-24 of it for |r| < 1/2.
__device__ __forceinline__ float penalty(float r, float em) {
  if (!(fabsf(r) < 0.5f)) return em - r;
  float s = 1.f / 40320.f;
  s = fmaf(s, r, 1.f / 5040.f);
  s = fmaf(s, r, 1.f / 720.f);
  s = fmaf(s, r, 1.f / 120.f);
  s = fmaf(s, r, 1.f / 24.f);
  s = fmaf(s, r, 1.f / 6.f);
  s = fmaf(s, r, 0.5f);
  return r * r * s;
}

// The token's term and the slope d(loss)/d(logp), from its log-probability
// logp + rest.
__device__ __forceinline__ void term_of(const Policy& a, float w, float adv, float old, float ref,
                                        float logp, float rest, float& term, float& slope) {
  const float ratio = expf((logp - old) + rest);
  // (comparisons, not fminf and fmaxf: NaN has to stay)
  const float lo = 1.f - a.lo, hi = 1.f + a.hi;
  const float clipped = ratio < lo ? lo : ratio > hi ? hi : ratio;
  // (an advantage of 0 takes any ratio out, one beyond float32's range too)
  const float plain = adv == 0.f && ratio == INFINITY ? 0.f : ratio * adv;
  const float bounded = clipped * adv;
  const bool through = plain <= bounded;
  // min(plain, bounded) and its derivative's share; a NaN on either side stays
  float v = -(plain != plain || through ? plain : bounded);
  float g = plain != plain || through ? -plain : 0.f;
  if (a.ref) {
    const float r = (ref - logp) - rest, em = expm1f(r);
    v += a.kl * penalty(r, em);
    g -= a.kl * em;
  }
  term = w * v;
  slope = w * g;
}

// The sums of a warp's lanes on one scale; the same in every lane.
__device__ __forceinline__ ScaledSum join_warp(ScaledSum t) {
  ScaledSum r;
  r.o = warp_max(t.o);
  r.s = warp_sum(t.s * exp2_fast(t.o - base_of(r.o)));
  return r;
}

// A run that is not read again.
template <class T, int U>
__device__ __forceinline__ Run<T, U> last_read(const Run<T, U>* p) {
  const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
  return *reinterpret_cast<const Run<T, U>*>(&v);
}

// The row's sum over the CTA's warps and the row's CTAs; the same in every
// thread.  A barrier on memory for all of them: the gradient may be written where
// others have read the logits before (shuffles alone do not order that).
template <int kRow>
__device__ __forceinline__ ScaledSum join_row(ScaledSum t, ScaledSum* red, ScaledSum* mine,
                                              int ranks) {
  constexpr int W = kRow / 32;
  const int lane = threadIdx.x & 31;
  t = join_warp(t);
  if constexpr (W > 1) {
    __syncthreads();  // (red may still be read from a call before)
    if (lane == 0) red[threadIdx.x >> 5] = t;
    __syncthreads();
    const ScaledSum none = {-INFINITY, 0.f};
    t = join_warp(lane < W ? red[lane] : none);
  } else {
    __syncwarp();
  }
  if (ranks > 1) {
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    if (threadIdx.x == 0) *mine = t;
    cluster.sync();
    t = *cluster.map_shared_rank(mine, 0);
    for (int r = 1; r < ranks; ++r) t = join(t, *cluster.map_shared_rank(mine, r));
    cluster.sync();  // (no CTA leaves, or writes again, while another reads)
  }
  return t;
}

// A row per cluster of `ranks` CTAs: a pass for the sum, four 16-byte loads per
// thread in flight, and for the gradient a second one, which goes through the
// row backwards, to meet what L2 and L1 still have.  What is not needed again
// (the second pass's reads, the gradient) leaves the caches first.
//
// 4096 rows of 128 KB, a fifth of them masked: 168 us (5.8 TB/s) on 512
// threads, two rows per SM; four rows of 256 threads each, 6 us more, since
// L2 no longer keeps them all.  A share of the row held in shared memory by a
// CTA of a cluster, read once: 191 to 259 us over shares and CTA counts; the
// row's two cluster barriers leave too little in flight.
template <class T, int kRow>
__global__ void __launch_bounds__(kRow, 1024 / kRow)
    policy_kernel(const __grid_constant__ Policy a, int ranks) {
  constexpr int U = 16 / sizeof(T);
  __shared__ ScaledSum red[kRow / 32];
  __shared__ ScaledSum mine;
  const int rank = ranks > 1 ? blockIdx.x % ranks : 0;
  const int64_t t = ranks > 1 ? blockIdx.x / ranks : blockIdx.x;
  const T* z = (const T*)a.logits + t * a.ldl;
  T* d = a.d ? (T*)a.d + t * a.ldd : nullptr;
  const Share sh = share_of<T, U>(z, a.vocab, rank, ranks);
  const int edge = edge_of<U>(sh, a.vocab, rank, ranks);
  // whether the gradient's runs are 16-byte aligned where the logits' are
  const bool run16 = d && aligned16(d + sh.head);
  const float w = a.weights ? a.weights[t] : 1.f;
  auto put = [&](int i, const Run<T, U>& r) {
    T* q = d + sh.head + i * U;
    if (run16) {
      __stcs(reinterpret_cast<uint4*>(q), *reinterpret_cast<const uint4*>(&r));
    } else {
#pragma unroll
      for (int k = 0; k < U; ++k) q[k] = r.v[k];
    }
  };
  if (w == 0.f) {  // (the same for every CTA of the row)
    if (threadIdx.x == 0 && rank == 0) {
      a.logp[t] = 0.f;
      if (a.loss) a.terms[t] = 0.f;
    }
    if (d) {
      Run<T, U> zero;
#pragma unroll
      for (int k = 0; k < U; ++k) zero.v[k] = from_f32<T>(0.f);
      for (int i = sh.v0 + threadIdx.x; i < sh.v1; i += kRow) put(i, zero);
      if (edge >= 0) d[edge] = from_f32<T>(0.f);
    }
    return;
  }
  const Run<T, U>* runs = reinterpret_cast<const Run<T, U>*>(z + sh.head);
  const int64_t target = a.targets[t];
  const bool valid = target >= 0 && target < a.vocab;
  // (read before anything is written: the gradient may take the logits' place)
  const float zt = valid ? to_f32(z[target]) : NAN;
  const float adv = a.loss ? a.adv[t] : 0.f, old = a.loss ? a.old[t] : 0.f;
  const float ref = a.ref ? a.ref[t] : 0.f;
  ScaledSum sum = {-INFINITY, 0.f};
  int i0 = sh.v0 + threadIdx.x;
  for (; i0 + (kAhead - 1) * kRow < sh.v1; i0 += kAhead * kRow) {
    Run<T, U> r[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) r[j] = runs[i0 + j * kRow];
    add_runs(sum, r);
  }
  for (; i0 < sh.v1; i0 += kRow) {
    const Run<T, U> r[1] = {runs[i0]};
    add_runs(sum, r);
  }
  if (edge >= 0) {
    const float x = to_f32(z[edge]) * kLog2e;
    const ScaledSum one = {rintf(x), exp2_fast(x - base_of(rintf(x)))};
    sum = join(sum, one);
  }
  sum = join_row<kRow>(sum, red, &mine, ranks);
  // Where x log2(e) is beyond float32's range, or rounds by more than a half (o
  // is then no longer near the largest one, and the exponentials may all be 0 or
  // infinite), or with nothing but -inf, the scale says nothing: the row's
  // largest element takes its part, 2^((x - m) log2(e)).  (the same for every
  // thread of the row)
  float m = 0.f;
  if (!(fabsf(sum.o) <= kMostScale) || !(sum.s < INFINITY)) {
    ScaledSum top = {-INFINITY, 0.f};  // o: the maximum
    for (int i = sh.v0 + threadIdx.x; i < sh.v1; i += kRow) top.o = fmaxf(top.o, largest(runs[i]));
    if (edge >= 0) top.o = fmaxf(top.o, to_f32(z[edge]));
    m = join_row<kRow>(top, red, &mine, ranks).o;
    sum.o = 0.f, sum.s = 0.f;
    for (int i = sh.v0 + threadIdx.x; i < sh.v1; i += kRow) {
      const Vec<U> f = unpack(runs[i]);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) sum.s += total(exp_pair(f.p[k], m, 0.f));
    }
    if (edge >= 0) sum.s += exp_pair(both(to_f32(z[edge])), m, 0.f).x;
    sum = join_row<kRow>(sum, red, &mine, ranks);
  }
  // every thread: the same numbers from the same inputs
  float rest, term = 0.f, slope = 0.f;
  const float logp = log_prob(zt - m, sum.o, sum.s, rest);
  if (a.loss) term_of(a, w, adv, old, ref, logp, rest, term, slope);
  if (threadIdx.x == 0 && rank == 0) {
    a.logp[t] = logp;
    if (a.loss) a.terms[t] = term;
  }
  if (!d) return;
  slope *= a.scale;
  const float f = -slope / sum.s;
  if (edge >= 0) {
    const float g = exp_pair(both(to_f32(z[edge])), m, sum.o).x * f;
    d[edge] = from_f32<T>(edge == target ? g + slope : g);
  }
  const int64_t at = valid ? target - sh.head : -1;  // within the runs
  auto grad_run = [&](int i, const Run<T, U>& r) {
    Vec<U> v = unpack(r);
#pragma unroll
    for (int k = 0; k < U / 2; ++k) v.p[k] = mul2(exp_pair(v.p[k], m, sum.o), both(f));
    const int64_t k0 = at - (int64_t)i * U;
    if (k0 >= 0 && k0 < U) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k == k0) (k & 1 ? v.p[k / 2].y : v.p[k / 2].x) += slope;
    }
    put(i, pack<T>(v));
  };
  int i1 = sh.v1 - 1 - (int)threadIdx.x;
  for (; i1 - (kAhead - 1) * kRow >= sh.v0; i1 -= kAhead * kRow) {
    Run<T, U> r[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) r[j] = last_read(runs + i1 - j * kRow);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) grad_run(i1 - j * kRow, r[j]);
  }
  for (; i1 >= sh.v0; i1 -= kRow) grad_run(i1, last_read(runs + i1));
}

// loss = sum of the terms, always in the same order.  A thread adds 16 terms
// at a time as a float32 and the rounding errors of its sums (Knuth's exact
// sum of two), and only such results in double: 16384 terms in 6 us, and in
// 13 with each addition in double, of which an SM makes few.
__global__ void __launch_bounds__(1024) policy_sum_kernel(const float* terms, int64_t tokens,
                                                          float* loss) {
  __shared__ double red[32];
  wait_for_prior();
  double sum = 0.0;
  for (int64_t i0 = threadIdx.x; i0 < tokens; i0 += 16 * 1024) {
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = i0 + k * 1024 < tokens ? terms[i0 + k * 1024] : 0.f;
    float s = v[0], rest = 0.f;
#pragma unroll
    for (int k = 1; k < 16; ++k) {
      const float t = __fadd_rn(s, v[k]), b = __fsub_rn(t, s);
      rest += __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(v[k], b));
      s = t;
    }
    // (a sum beyond float32's range has no errors to speak of: term by term)
    if (fabsf(s) < INFINITY) {
      sum += (double)s + (double)rest;
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) sum += v[k];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int i = 0; i < 32; ++i) sum += red[i];
    *loss = (float)sum;
  }
}

// CTAs per row: while the rows leave SMs without work, shares of a row down to
// 8 KB.  (With rows enough, two CTAs per row cost more in their barriers than
// a fuller last round gains: 2049 rows of 200 KB in 120 us against 95.)
inline int ranks_of(const Policy& a, int es, int per_sm) {
  int r = 1;
  while (r < 8 && a.tokens * r * 2 <= per_sm * sm_count() &&
         (int64_t)a.vocab * es > r * (16 << 10))
    r *= 2;
  return r;
}

template <class T, int kRow>
int launch_rows(const Policy& a, cudaStream_t s) {
  for (int64_t t0 = 0; t0 < a.tokens; t0 += 1 << 27) {
    Policy b = a;
    b.tokens = std::min<int64_t>(a.tokens - t0, 1 << 27);
    b.logits = (const T*)a.logits + t0 * a.ldl;
    if (a.d) b.d = (T*)a.d + t0 * a.ldd;
    b.targets += t0, b.logp += t0;
    if (a.weights) b.weights += t0;
    if (a.loss) b.old += t0, b.adv += t0, b.terms += t0;
    if (a.ref) b.ref += t0;
    ProfScope prof(ROT_PROF_ELEMENTWISE,
                   (double)b.tokens * a.vocab * sizeof(T) * (a.d ? 2 : 1), s);
    const int ranks = ranks_of(b, sizeof(T), 1024 / kRow);
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(b.tokens * ranks));
    c.blockDim = dim3(kRow);
    c.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ranks, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = ranks > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&c, policy_kernel<T, kRow>, b, ranks) != cudaSuccess) {
      cudaGetLastError();
      return ROT_ECUDA;
    }
  }
  return ROT_OK;
}

// Threads of a row: 512 (log-probabilities alone 256), so that few rows share
// the caches at once; but with rows for more than one round of those, fewer
// for short rows, whose time is that of a few dependent steps and the more of
// which an SM then holds.  With the gradient, in us on 32, 128 and 512 threads:
// 16384 rows of 2 KB 20, 52 and 190, of 8 KB 49, 69 and 212; 8192 of 16 KB 52,
// 55 and 135; 4096 of 64 KB 106 on 128 and 123 on 512; but 600 of 8 KB 8.4,
// 6.2 and 10.1.
template <class T>
int launch_type(const Policy& a, cudaStream_t s) {
  const int64_t bytes = (int64_t)a.vocab * sizeof(T);
  if (bytes <= (8 << 10) && a.tokens > 8 * sm_count()) return launch_rows<T, 32>(a, s);
  if (bytes <= (64 << 10) && a.tokens > 2 * sm_count()) return launch_rows<T, 128>(a, s);
  return a.d ? launch_rows<T, 512>(a, s) : launch_rows<T, 256>(a, s);
}
int launch_policy(const Policy& a, int32_t type, cudaStream_t s) {
  if (type == ROT_TYPE_F32) return launch_type<float>(a, s);
  if (type == ROT_TYPE_F16) return launch_type<__half>(a, s);
  return launch_type<__nv_bfloat16>(a, s);
}

bool bad_logits(const void* logits, int64_t ldl, const int64_t* targets, const float* logp,
                int64_t tokens, int64_t vocab, int32_t type) {
  if (tokens < 0 || vocab < 1 || vocab > (1 << 30) || ldl < vocab || !float_type(type)) return true;
  return tokens > 0 && (!logits || !targets || !logp);
}

}  // namespace
}  // namespace ops
}  // namespace rot

using namespace rot;
using namespace rot::ops;

extern "C" {

int rot_token_logprobs(const void* logits, int64_t ldl, const int64_t* targets,
                       const float* weights, float* logp, int64_t tokens, int64_t vocab,
                       int32_t type, void* stream) {
  if (bad_logits(logits, ldl, targets, logp, tokens, vocab, type)) return ROT_EINVAL;
  if (tokens == 0) return ROT_OK;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  Policy a = {};
  a.logits = logits, a.ldl = ldl, a.targets = targets, a.weights = weights, a.logp = logp;
  a.tokens = tokens, a.vocab = (int)vocab;
  return guarded([&] { return launch_policy(a, type, static_cast<cudaStream_t>(stream)); });
}

int rot_policy_loss(const void* logits, int64_t ldl, const int64_t* targets, const float* old_logp,
                    const float* ref_logp, const float* advantages, const float* weights,
                    float* loss, float* logp, float* terms, void* dlogits, int64_t lddl,
                    int64_t tokens, int64_t vocab, int32_t type, float clip_low, float clip_high,
                    float kl_coef, float grad_scale, void* stream) {
  if (bad_logits(logits, ldl, targets, logp, tokens, vocab, type) || !loss) return ROT_EINVAL;
  if (tokens > 0 && (!old_logp || !advantages || !weights || !terms)) return ROT_EINVAL;
  if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) || !(kl_coef >= 0.f))
    return ROT_EINVAL;
  if ((!ref_logp && kl_coef != 0.f) || (dlogits && lddl < vocab)) return ROT_EINVAL;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Policy a = {};
  a.logits = logits, a.ldl = ldl, a.targets = targets, a.weights = weights, a.logp = logp;
  a.tokens = tokens, a.vocab = (int)vocab;
  // (no penalty: its exponential may be infinite, and 0 times that is not 0)
  a.ref = kl_coef != 0.f ? ref_logp : nullptr;
  a.old = old_logp, a.adv = advantages, a.terms = terms, a.d = dlogits;
  a.ldd = lddl, a.loss = 1, a.lo = clip_low, a.hi = clip_high, a.kl = kl_coef;
  a.scale = grad_scale;
  return guarded([&] {
    const int e = launch_policy(a, type, s);
    if (e != ROT_OK) return e;
    ProfScope prof(ROT_PROF_ELEMENTWISE, 4.0 * tokens, s);
    return launch_behind(policy_sum_kernel, 1, 1024, 0, s, terms, tokens, loss);
  });
}

}  // extern "C"
