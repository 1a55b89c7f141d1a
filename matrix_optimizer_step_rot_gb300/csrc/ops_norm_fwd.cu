// Layer norm forward (include/rot_ops.h): y and the hidden stream from x and
// the residual.  Bound by HBM: one read of each input, one write of each
// output; with dropout the generator's arithmetic is nearly as long.
//
// 16384 x 4096 in bfloat16 with residual and dropout: 96 us, 5.6 TB/s.
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
__global__ void __launch_bounds__(block_of(TPR), TPR == 1024 ? 1 : (U > 1 ? 640 : 1024) / block_of(TPR))
    norm_fwd_kernel(const __grid_constant__ NormFwd a) {
  constexpr int kBlock = block_of(TPR), RPB = kBlock / TPR;
  using E = typename Vec<U>::E;
  constexpr int P = Vec<U>::P;
  __shared__ __align__(16) float red[2][kBlock / 32];
  const int t = threadIdx.x % TPR;
  const bool busy = has_columns<U, N>(t, a.cols);  // (the same for a warp)
  const float inv = 1.f / (float)a.cols;
  const int64_t wanted = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = wanted < a.rows;
  const int64_t row = live ? wanted : a.rows - 1;
  int c[N];
  bool in[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    c[n] = column_of<U, TPR, N>(n, t);
    in[n] = (U > 1 && n < N - 1) || c[n] < a.cols;
    if (U > 1 && !in[n]) c[n] = 0;
  }
  Vec<U> h[N];
  E sum = all_of<E>(0.f);
  if (busy) {
    Run<T, U> x[N], r[N];
    get_runs(x, a.x, row * a.ldx, c, in);
    if (a.res) get_runs(r, a.res, row * a.ldr, c, in);
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = unpack(x[n]);
    if (DROP) drop_runs<U, N>(a.d, (uint64_t)row * a.cols, c, t, a.cols, h);
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
        if (live && in[n])
          put_run(a.h, row * a.ldh + (U > 1 ? c[n] : c[0] + 32 * n), stored);
        h[n] = unpack(stored);  // the norm reads what is stored
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int k = 0; k < P; ++k) {
        if (!in[n]) h[n].p[k] = all_of<E>(0.f);
        sum = add2(sum, h[n].p[k]);
      }
  }
  const float mean = row_sum<TPR, kBlock>(total(sum), red[0]) * inv;
  E sq = all_of<E>(0.f);
  if (busy) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float less = in[n] ? -mean : 0.f;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        h[n].p[k] = add2(h[n].p[k], all_of<E>(less));
        sq = fma2(h[n].p[k], h[n].p[k], sq);
      }
    }
  }
  const float rstd = inverse_root(row_sum<TPR, kBlock>(total(sq), red[1]) * inv + a.eps);
  if (!live || !busy) return;
  if (t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  Vec<U> w[N];
  get_weights<T>(w, a.w, a.w32, c, in);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int k = 0; k < P; ++k) h[n].p[k] = mul2(mul2(h[n].p[k], all_of<E>(rstd)), w[n].p[k]);
  if (a.b) {
    get_weights<T>(w, a.b, a.w32, c, in);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int k = 0; k < P; ++k) h[n].p[k] = add2(h[n].p[k], w[n].p[k]);
  }
  put_runs<T>(a.y, row * a.ldy, c, in, h);
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
    // (128 consecutive elements per warp; a thread meets its own again below)
    for (int c0 = threadIdx.x / 32 * 128; c0 < a.cols; c0 += 32 * 128) {
      const int c = c0 + threadIdx.x % 32;
      T x[4], r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool in = c + 32 * k < a.cols;
        x[k] = in ? ((const T*)a.x)[row * a.ldx + c + 32 * k] : from_f32<T>(0.f);
        r[k] = in && a.res ? ((const T*)a.res)[row * a.ldr + c + 32 * k] : from_f32<T>(0.f);
      }
      const uint32_t bits = a.d.on ? keep_bits<4>(a.d, (uint64_t)row * a.cols + c0) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f = to_f32(x[k]);
        if (a.h) {
          if (a.d.on) f = kept(a.d, bits >> k & 1, f);
          const T v = from_f32<T>(a.res ? __fadd_rn(to_f32(r[k]), f) : f);
          if (c + 32 * k < a.cols) ((T*)a.h)[row * a.ldh + c + 32 * k] = v;
          f = c + 32 * k < a.cols ? to_f32(v) : 0.f;
        }
        sum += f;
      }
    }
    const float mean = row_sum<1024, 1024>(sum, red[0]) * inv;
    float sq = 0.f;
    for (int c0 = threadIdx.x / 32 * 128; c0 < a.cols; c0 += 32 * 128)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + threadIdx.x % 32 + 32 * k;
        const float f = c < a.cols ? to_f32(src[c]) - mean : 0.f;
        sq += f * f;
      }
    const float rstd = inverse_root(row_sum<1024, 1024>(sq, red[1]) * inv + a.eps);
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    for (int c0 = threadIdx.x / 32 * 128; c0 < a.cols; c0 += 32 * 128) {
      float f[4], w[4], b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = min(c0 + (int)threadIdx.x % 32 + 32 * k, a.cols - 1);
        // (the last element for those past the end, which store nothing)
        f[k] = to_f32(src[c]);
        w[k] = load_weight<T, 1>(a.w, a.w32, c).p[0];
        b[k] = a.b ? load_weight<T, 1>(a.b, a.w32, c).p[0] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + threadIdx.x % 32 + 32 * k;
        if (c < a.cols)
          ((T*)a.y)[row * a.ldy + c] = from_f32<T>((f[k] - mean) * rstd * w[k] + b[k]);
      }
    }
  }
}

// A thread's share of a row: up to four 16-byte runs (so that what a thread
// does once per row weighs little), or single elements where the rows are not
// 16-byte aligned.
constexpr int kMostRuns = 4;

template <class T, int U, int TPR, int N, bool DROP>
int launch_runs(const NormFwd& a, unsigned grid, cudaStream_t s) {
  // (at or below a quarter of TPR * 4 runs the next smaller TPR takes the row:
  // those counts need no kernel)
  constexpr int least = TPR == 32 ? 1 : TPR == 128 ? 2 : 3;
  if constexpr (N > least) {
    if (a.cols <= (N - 1) * TPR * U) return launch_runs<T, U, TPR, N - 1, DROP>(a, grid, s);
  }
  norm_fwd_kernel<T, U, TPR, N, DROP><<<grid, block_of(TPR), 0, s>>>(a);
  return launched();
}
template <class T, int TPR, int N, bool DROP>
int launch_single(const NormFwd& a, unsigned grid, cudaStream_t s) {
  norm_fwd_kernel<T, 1, TPR, N, DROP><<<grid, block_of(TPR), 0, s>>>(a);
  return launched();
}

template <class T, int U, bool DROP>
int launch_rows(const NormFwd& a, cudaStream_t s) {
  const int tpr = U > 1 ? row_threads(a.cols, U * kMostRuns) : row_threads_single(a.cols);
  const int64_t per = tpr == 0 ? 1 : block_of(tpr) / tpr, blocks = (a.rows + per - 1) / per;
  if (blocks > 0x7FFFFFFF) return ROT_EINVAL;
  const unsigned grid = (unsigned)blocks;
  if constexpr (U == 1) {
    constexpr int N = kSingles;
    switch (tpr) {
      case 32:
        if (a.cols <= 32 * kFewSingles) return launch_single<T, 32, kFewSingles, DROP>(a, grid, s);
        return launch_single<T, 32, N, DROP>(a, grid, s);
      case 64: return launch_single<T, 64, N, DROP>(a, grid, s);
      case 128: return launch_single<T, 128, N, DROP>(a, grid, s);
      // shares of 16 instead of twice the threads, more rows in flight: 12000 x
      // 6001 in 247 us instead of 327, 16384 x 3001 in 162 instead of 183
      case 256: return launch_single<T, 128, 2 * N, DROP>(a, grid, s);
      case 512: return launch_single<T, 256, 2 * N, DROP>(a, grid, s);
      case 1024: return launch_single<T, 512, 2 * N, DROP>(a, grid, s);
    }
  } else {
    constexpr int N = kMostRuns;
    switch (tpr) {
      case 32: return launch_runs<T, U, 32, N, DROP>(a, grid, s);
      case 128: return launch_runs<T, U, 128, N, DROP>(a, grid, s);
      case 256: return launch_runs<T, U, 256, N, DROP>(a, grid, s);
      case 512: return launch_runs<T, U, 512, N, DROP>(a, grid, s);
      case 1024: return launch_runs<T, U, 1024, N, DROP>(a, grid, s);
    }
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
