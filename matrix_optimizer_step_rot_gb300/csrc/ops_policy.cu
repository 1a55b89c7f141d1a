// Log-probabilities of tokens and the clipped policy loss with its gradient
// (include/rot_ops.h).  Bound by HBM: one read of the logits, one write of
// their gradient.
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

constexpr int kRow = 512;  // threads per row

// Running maximum and sum of exp(x - maximum).
struct MaxSum {
  float m = -INFINITY, s = 0.f;
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

// One block per row: a pass for maximum and sum, a pass for the gradient.
template <class T, int U>
__global__ void __launch_bounds__(kRow) policy_kernel(const Policy a) {
  __shared__ MaxSum red[kRow / 32];
  __shared__ float sh[3];
  const int64_t t = blockIdx.x;
  const T* z = (const T*)a.logits + t * a.ldl;
  T* d = a.d ? (T*)a.d + t * a.ldd : nullptr;
  const float w = a.weights ? a.weights[t] : 1.f;
  const int runs = a.vocab / U;  // (U > 1: rows of a multiple of U)
  if (w == 0.f) {
    if (threadIdx.x == 0) {
      a.logp[t] = 0.f;
      if (a.loss) a.terms[t] = 0.f;
    }
    if (d) {
      const float zero[U] = {};
      for (int i = threadIdx.x; i < runs; i += kRow) store_run(d + i * U, zero);
    }
    return;
  }
  MaxSum ms;
  for (int i = threadIdx.x; i < runs; i += kRow) {
    float f[U];
    load_run(z + i * U, f);
    float m = ms.m;
#pragma unroll
    for (int k = 0; k < U; ++k) m = fmaxf(m, f[k]);
    const float o = base_of(m);
    ms.s *= __expf(ms.m - o);
    ms.m = m;
#pragma unroll
    for (int k = 0; k < U; ++k) ms.s += __expf(f[k] - o);
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
  const int64_t target = a.targets[t];
  const bool valid = target >= 0 && target < a.vocab;
  if (threadIdx.x == 0) {
    ms = red[0];
    for (int i = 1; i < kRow / 32; ++i) ms = join(ms, red[i]);
    // (an empty row, -inf throughout, has no distribution)
    const float sum = ms.m == -INFINITY ? NAN : ms.s;
    const float logp = valid ? to_f32(z[target]) - ms.m - logf(sum) : NAN;
    float term = 0.f, slope = 0.f;
    a.logp[t] = logp;
    if (a.loss) {
      term_of(a, t, w, logp, term, slope);
      a.terms[t] = term;
    }
    sh[0] = ms.m;
    sh[1] = slope * a.scale;
    sh[2] = 1.f / sum;
  }
  __syncthreads();
  if (!d) return;
  const float m = sh[0], slope = sh[1], f = -slope * sh[2];
  for (int i = threadIdx.x; i < runs; i += kRow) {
    float x[U];
    load_run(z + i * U, x);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      x[k] = __expf(x[k] - m) * f;
      if (i * U + k == target) x[k] += slope;
    }
    store_run(d + i * U, x);
  }
}

// loss = sum of the terms, always in the same order.
__global__ void __launch_bounds__(1024) policy_sum_kernel(const float* terms, int64_t tokens,
                                                          float* loss) {
  __shared__ double red[32];
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

template <class T>
int launch_rows(const Policy& a, cudaStream_t s) {
  constexpr int U = 16 / sizeof(T);
  const bool vec = a.vocab % U == 0 && rows16(a.logits, a.ldl, sizeof(T)) &&
                   rows16(a.d, a.ldd, sizeof(T));
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
    auto k = vec ? policy_kernel<T, U> : policy_kernel<T, 1>;
    k<<<(unsigned)b.tokens, kRow, 0, s>>>(b);
    const int e = launched();
    if (e != ROT_OK) return e;
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
    policy_sum_kernel<<<1, 1024, 0, s>>>(terms, tokens, loss);
    return launched();
  });
}

}  // extern "C"
