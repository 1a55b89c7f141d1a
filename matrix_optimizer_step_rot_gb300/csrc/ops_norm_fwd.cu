// Layer norm forward (include/rot_ops.h): y and the hidden stream from x and
// the residual.  Bound by HBM: one read of each input, one write of each
// output; with dropout the generator's arithmetic is nearly as long.
//
// 16384 x 4096 in bfloat16 with residual and dropout: 98 us, 5.5 TB/s.
#include <algorithm>

#include "ops_norm.cuh"
#include "profile.h"

namespace rot {
namespace ops {
namespace {

// A row in the registers of TPR threads, N runs of U elements each; of 16-byte
// runs every one but the last lies within the row for every thread (the host
// picks N).  All
// loads come first (a store may alias a later load as far as the compiler
// knows), and what each run needs is computed without branches in between, so
// that the runs' arithmetic overlaps: past the row's end a thread takes its
// first element again, counts it as 0 and stores nothing.
template <class T, int U, int TPR, int N, bool DROP>
__global__ void __launch_bounds__(block_of(TPR), TPR == 1024 ? 1 : 640 / block_of(TPR))
    norm_fwd_kernel(const __grid_constant__ NormFwd a) {
  constexpr int kBlock = block_of(TPR), RPB = kBlock / TPR;
  using E = typename Vec<U>::E;
  constexpr int P = Vec<U>::P;
  __shared__ __align__(16) float red[2][kBlock / 32];
  const int t = threadIdx.x % TPR;
  const float inv = 1.f / (float)a.cols;
  const int64_t wanted = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = wanted < a.rows;
  const int64_t row = live ? wanted : a.rows - 1;
  int c[N];
  bool in[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    c[n] = (n * TPR + t) * U;
    in[n] = (U > 1 && n < N - 1) || c[n] < a.cols;
    if (!in[n]) c[n] = 0;
  }
  Run<T, U> x[N], r[N];
#pragma unroll
  for (int n = 0; n < N; ++n) x[n] = raw_run<T, U>(a.x, row * a.ldx + c[n]);
  if (a.res) {
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = raw_run<T, U>(a.res, row * a.ldr + c[n]);
  }
  Vec<U> h[N];
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = unpack(x[n]);
  if (DROP) {
#pragma unroll
    for (int n = 0; n < N; ++n) drop_run(a.d, (uint64_t)row * a.cols + c[n], h[n]);
  }
  if (a.h) {
    if (a.res) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const Vec<U> v = unpack(r[n]);
#pragma unroll
        for (int k = 0; k < P; ++k) h[n].p[k] = add2(v.p[k], h[n].p[k]);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Run<T, U> stored = pack<T>(h[n]);
      if (live && in[n]) put_run(a.h, row * a.ldh + c[n], stored);
      h[n] = unpack(stored);  // the norm reads what is stored
    }
  }
  E sum = all_of<E>(0.f);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if (!in[n]) h[n].p[k] = all_of<E>(0.f);
      sum = add2(sum, h[n].p[k]);
    }
  const float mean = row_sum<TPR, kBlock>(total(sum), red[0]) * inv;
  E sq = all_of<E>(0.f);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const float less = in[n] ? -mean : 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      h[n].p[k] = add2(h[n].p[k], all_of<E>(less));
      sq = fma2(h[n].p[k], h[n].p[k], sq);
    }
  }
  const float rstd = inverse_root(row_sum<TPR, kBlock>(total(sq), red[1]) * inv + a.eps);
  if (!live) return;
  if (t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const Vec<U> w = load_weight<T, U>(a.w, a.w32, c[n]);
#pragma unroll
    for (int k = 0; k < P; ++k) h[n].p[k] = mul2(mul2(h[n].p[k], all_of<E>(rstd)), w.p[k]);
  }
  if (a.b) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Vec<U> b = load_weight<T, U>(a.b, a.w32, c[n]);
#pragma unroll
      for (int k = 0; k < P; ++k) h[n].p[k] = add2(h[n].p[k], b.p[k]);
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (in[n]) put_run(a.y, row * a.ldy + c[n], pack<T>(h[n]));
}

// Rows too wide for the registers: a block per row, three passes over it (the
// second and third out of L2).
template <class T>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const __grid_constant__ NormFwd a) {
  __shared__ __align__(16) float red[2][32];
  const float inv = 1.f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* src = a.h ? (const T*)a.h + row * a.ldh : (const T*)a.x + row * a.ldx;
    float sum = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += 1024) {
      Vec<1> f = {{to_f32(((const T*)a.x)[row * a.ldx + c])}};
      if (a.h) {
        const float r = a.res ? to_f32(((const T*)a.res)[row * a.ldr + c]) : 0.f;
        drop_run(a.d, (uint64_t)row * a.cols + c, f);
        const T v = from_f32<T>(a.res ? __fadd_rn(r, f.p[0]) : f.p[0]);
        ((T*)a.h)[row * a.ldh + c] = v;
        f.p[0] = to_f32(v);
      }
      sum += f.p[0];
    }
    const float mean = row_sum<1024, 1024>(sum, red[0]) * inv;
    float sq = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += 1024) {
      const float f = to_f32(src[c]) - mean;
      sq += f * f;
    }
    const float rstd = inverse_root(row_sum<1024, 1024>(sq, red[1]) * inv + a.eps);
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < a.cols; c += 1024) {
      const float w = load_weight<T, 1>(a.w, a.w32, c).p[0];
      const float b = a.b ? load_weight<T, 1>(a.b, a.w32, c).p[0] : 0.f;
      ((T*)a.y)[row * a.ldy + c] = from_f32<T>((to_f32(src[c]) - mean) * rstd * w + b);
    }
  }
}

// A thread's share of a row: up to four 16-byte runs (so that what a thread
// does once per row weighs little), or 8 elements one by one where the rows
// are not 16-byte aligned.
template <int U>
constexpr int kMostRuns = U > 1 ? 4 : 8;

template <class T, int U, int TPR, int N, bool DROP>
int launch_runs(const NormFwd& a, unsigned grid, cudaStream_t s) {
  // (at or below a quarter of TPR * 4 runs the next smaller TPR takes the row:
  // those counts need no kernel)
  constexpr int least = U == 1 ? N : TPR == 32 ? 1 : TPR == 128 ? 2 : 3;
  if constexpr (N > least) {
    if (a.cols <= (N - 1) * TPR * U) return launch_runs<T, U, TPR, N - 1, DROP>(a, grid, s);
  }
  norm_fwd_kernel<T, U, TPR, N, DROP><<<grid, block_of(TPR), 0, s>>>(a);
  return launched();
}

template <class T, int U, bool DROP>
int launch_rows(const NormFwd& a, cudaStream_t s) {
  constexpr int N = kMostRuns<U>;
  const int tpr = row_threads(a.cols, U * N);
  const int64_t per = tpr == 32 ? 4 : 1, blocks = (a.rows + per - 1) / per;
  if (blocks > 0x7FFFFFFF) return ROT_EINVAL;
  const unsigned grid = (unsigned)blocks;
  switch (tpr) {
    case 32: return launch_runs<T, U, 32, N, DROP>(a, grid, s);
    case 128: return launch_runs<T, U, 128, N, DROP>(a, grid, s);
    case 256: return launch_runs<T, U, 256, N, DROP>(a, grid, s);
    case 512: return launch_runs<T, U, 512, N, DROP>(a, grid, s);
    case 1024: return launch_runs<T, U, 1024, N, DROP>(a, grid, s);
  }
  norm_fwd_wide_kernel<T><<<grid, 1024, 0, s>>>(a);
  return launched();
}

template <class T>
int run(const NormFwd& a, cudaStream_t s) {
  constexpr int U = 16 / sizeof(T);
  ProfScope prof(ROT_PROF_ELEMENTWISE,
                 (double)a.rows * a.cols * sizeof(T) * (2 + (a.res != nullptr) + (a.h != nullptr)), s);
  const bool vec = a.cols % U == 0 && rows16(a.x, a.ldx, sizeof(T)) &&
                   rows16(a.res, a.ldr, sizeof(T)) && rows16(a.h, a.ldh, sizeof(T)) &&
                   rows16(a.y, a.ldy, sizeof(T)) && aligned16(a.w) && (!a.b || aligned16(a.b));
  if (vec) return a.d.on ? launch_rows<T, U, true>(a, s) : launch_rows<T, U, false>(a, s);
  return a.d.on ? launch_rows<T, 1, true>(a, s) : launch_rows<T, 1, false>(a, s);
}

}  // namespace

int norm_forward(int32_t type, const NormFwd& a, cudaStream_t s) {
  if (type == ROT_TYPE_F32) return run<float>(a, s);
  if (type == ROT_TYPE_F16) return run<__half>(a, s);
  return run<__nv_bfloat16>(a, s);
}

}  // namespace ops
}  // namespace rot
