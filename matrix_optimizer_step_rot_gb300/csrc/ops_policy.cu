// Log-probabilities of tokens and the clipped policy loss with its gradient
// (include/rot_ops.h).  Bound by HBM: one read of the logits, one write of
// their gradient.
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

constexpr int kRow = 512;  // threads per CTA
constexpr int kAhead = 4;  // 16-byte loads of a thread in flight

// Running maximum and sum of exp(x - maximum).
struct MaxSum {
  float m, s;
};
// a reference point that keeps exp(-inf - m) at 0 while only -inf was seen
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  MaxSum r;
  r.m = fmaxf(a.m, b.m);
  const float o = base_of(r.m);
  r.s = a.s * __expf(a.m - o) + b.s * __expf(b.m - o);
  return r;
}

// exp of both halves: the difference first, so that values at the ends of
// float32's range cannot overflow on the way.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 exp_less(float2 x, float m) {
  const float2 t = mul2(add2(x, both(-m)), both(kLog2e));
  return make_float2(exp2_fast(t.x), exp2_fast(t.y));
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
  if (rank == ranks - 1 && t >= 32 && t - 32 < vocab - tail) return tail + t - 32;
  return -1;
}

// The token's term and the slope d(loss)/d(logp), from its log-probability.
__device__ __forceinline__ void term_of(const Policy& a, int64_t t, float w, float logp,
                                        float& term, float& slope) {
  const float adv = a.adv[t], ratio = expf(logp - a.old[t]);
  // (comparisons, not fminf and fmaxf: NaN has to stay)
  const float lo = 1.f - a.lo, hi = 1.f + a.hi;
  const float clipped = ratio < lo ? lo : ratio > hi ? hi : ratio;
  const float plain = ratio * adv, bounded = clipped * adv;
  const bool through = plain <= bounded;
  // min(plain, bounded) and its derivative's share; a NaN on either side stays
  float v = -(plain != plain || through ? plain : bounded);
  float g = plain != plain || through ? -plain : 0.f;
  if (a.ref) {
    const float r = a.ref[t] - logp, em = expm1f(r);
    v += a.kl * (em - r);
    g -= a.kl * em;
  }
  term = w * v;
  slope = w * g;
}

// A row per cluster of `ranks` CTAs (1 where there are rows enough for the
// SMs; more, and the row's parts joined through distributed shared memory,
// where there are few).  A pass for maximum and sum, four 16-byte loads per
// thread in flight; for the gradient a second pass, which finds the row in L2.
template <class T>
__global__ void __launch_bounds__(kRow, 2) policy_kernel(const __grid_constant__ Policy a,
                                                         int ranks) {
  constexpr int U = 16 / sizeof(T);
  __shared__ MaxSum red[kRow / 32];
  __shared__ MaxSum mine;
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
      *reinterpret_cast<Run<T, U>*>(q) = r;
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
  MaxSum ms = {-INFINITY, 0.f};
  if (edge >= 0) {
    ms.m = to_f32(z[edge]);
    ms.s = __expf(ms.m - base_of(ms.m));
  }
  for (int i0 = sh.v0 + threadIdx.x; i0 < sh.v1; i0 += kRow * kAhead) {
    Run<T, U> r[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j * kRow < sh.v1) r[j] = runs[i0 + j * kRow];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j * kRow >= sh.v1) break;
      const Vec<U> f = unpack(r[j]);
      float m = ms.m;
#pragma unroll
      for (int k = 0; k < U / 2; ++k) m = fmaxf(fmaxf(m, f.p[k].x), f.p[k].y);
      const float o = base_of(m);
      float2 s = make_float2(ms.s * exp2_fast((ms.m - o) * kLog2e), 0.f);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) s = add2(s, exp_less(f.p[k], o));
      ms.m = m;
      ms.s = s.x + s.y;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    MaxSum b;
    b.m = __shfl_xor_sync(0xffffffffu, ms.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, ms.s, o);
    ms = join(ms, b);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ms;
  __syncthreads();
  ms = red[0];
#pragma unroll
  for (int i = 1; i < kRow / 32; ++i) ms = join(ms, red[i]);
  if (ranks > 1) {
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    if (threadIdx.x == 0) mine = ms;
    cluster.sync();
    ms = *cluster.map_shared_rank(&mine, 0);
    for (int r = 1; r < ranks; ++r) ms = join(ms, *cluster.map_shared_rank(&mine, r));
    cluster.sync();  // (no CTA leaves while another reads its shared memory)
  }
  // every thread: the same numbers from the same inputs
  const float sum = ms.m == -INFINITY ? NAN : ms.s;  // (-inf throughout: no distribution)
  const int64_t target = a.targets[t];
  const bool valid = target >= 0 && target < a.vocab;
  const float zt = valid ? to_f32(z[target]) : NAN;
  const float logp = zt - ms.m - logf(sum);
  float term = 0.f, slope = 0.f;
  if (a.loss) term_of(a, t, w, logp, term, slope);
  if (threadIdx.x == 0 && rank == 0) {
    a.logp[t] = logp;
    if (a.loss) a.terms[t] = term;
  }
  if (!d) return;
  slope *= a.scale;
  const float f = -slope / sum;
  // (in place, the target's logit must be read by every thread before it is overwritten)
  if (ranks > 1)
    cooperative_groups::this_cluster().sync();
  else
    __syncthreads();
  if (edge >= 0) {
    const float g = __expf(to_f32(z[edge]) - ms.m) * f;
    d[edge] = from_f32<T>(edge == target ? g + slope : g);
  }
  const int64_t at = valid ? target - sh.head : -1;  // within the runs
  for (int i0 = sh.v0 + threadIdx.x; i0 < sh.v1; i0 += kRow * kAhead) {
    Run<T, U> r[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j * kRow < sh.v1) r[j] = runs[i0 + j * kRow];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kRow;
      if (i >= sh.v1) break;
      Vec<U> v = unpack(r[j]);
#pragma unroll
      for (int k = 0; k < U / 2; ++k) v.p[k] = mul2(exp_less(v.p[k], ms.m), both(f));
      const int64_t k0 = at - (int64_t)i * U;
      if (k0 >= 0 && k0 < U) {
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (k == k0) (k & 1 ? v.p[k / 2].y : v.p[k / 2].x) += slope;
      }
      put(i, pack<T>(v));
    }
  }
}

// loss = sum of the terms, always in the same order.
__global__ void __launch_bounds__(1024) policy_sum_kernel(const float* terms, int64_t tokens,
                                                          float* loss) {
  __shared__ double red[32];
  wait_for_prior();
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < tokens; i += 1024) sum += terms[i];
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

// CTAs per row: while the rows leave SMs (two CTAs each) without work, shares
// of a row down to 16 KB.
inline int ranks_of(const Policy& a, int es) {
  int r = 1;
  while (r < 8 && a.tokens * r * 2 <= 2 * sm_count() && (int64_t)a.vocab * es > r * 32768) r *= 2;
  return r;
}

template <class T>
int launch_rows(const Policy& a, cudaStream_t s) {
  for (int64_t t0 = 0; t0 < a.tokens; t0 += 1 << 30) {
    Policy b = a;
    b.tokens = std::min<int64_t>(a.tokens - t0, 1 << 30);
    b.logits = (const T*)a.logits + t0 * a.ldl;
    if (a.d) b.d = (T*)a.d + t0 * a.ldd;
    b.targets += t0, b.logp += t0;
    if (a.weights) b.weights += t0;
    if (a.loss) b.old += t0, b.adv += t0, b.terms += t0;
    if (a.ref) b.ref += t0;
    ProfScope prof(ROT_PROF_ELEMENTWISE,
                   (double)b.tokens * a.vocab * sizeof(T) * (a.d ? 2 : 1), s);
    const int ranks = ranks_of(b, sizeof(T));
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(b.tokens * ranks));
    c.blockDim = dim3(kRow);
    c.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ranks, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = ranks > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&c, policy_kernel<T>, b, ranks) != cudaSuccess) {
      cudaGetLastError();
      return ROT_ECUDA;
    }
  }
  return ROT_OK;
}

int launch_policy(const Policy& a, int32_t type, cudaStream_t s) {
  if (type == ROT_TYPE_F32) return launch_rows<float>(a, s);
  if (type == ROT_TYPE_F16) return launch_rows<__half>(a, s);
  return launch_rows<__nv_bfloat16>(a, s);
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
  a.old = old_logp, a.ref = ref_logp, a.adv = advantages, a.terms = terms, a.d = dlogits;
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
