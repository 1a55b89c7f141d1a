// Dropout and layer norm (include/rot_ops.h).  Both are bound by HBM: one
// read of every input, one write of every output, the dropout mask computed
// where it is used.
#include <algorithm>
#include <cmath>

#include "ops_common.cuh"
#include "profile.h"

namespace rot {
namespace ops {

Drop make_drop(double p, uint64_t seed, uint64_t offset) {
  Drop d;
  const double bar = std::nearbyint(p * 4294967296.0);
  d.on = bar > 0.0;  // (p below 2^-33 drops nothing, and 1 / (1 - p) rounds to 1)
  d.bar = d.on ? (uint32_t)(bar - 1.0) : 0u;
  d.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  const uint64_t b = (uint64_t)(uint32_t)offset * kPhiloxM1;
  d.first[0] = (uint32_t)(b >> 32) ^ k0;
  d.first[1] = (uint32_t)b;
  d.first[2] = (uint32_t)(offset >> 32) ^ k1;
  for (int r = 0; r < 9; ++r) {
    d.key[r][0] = k0 += 0x9E3779B9u;
    d.key[r][1] = k1 += 0xBB67AE85u;
  }
  return d;
}

namespace {

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------

// Runs of U consecutive elements of the row-major order, each in one row and
// one 16-byte access (the host checked); what is left of a single row goes
// element by element.  Occupancy hides the loads: 6 blocks per SM.
template <class T, int U>
__global__ void __launch_bounds__(256, 6)
    dropout_kernel(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y, int64_t ldy,
                   int64_t rows, int64_t cols, const __grid_constant__ Drop d) {
  const int64_t total = rows * cols, runs = total / U;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < runs;
       u += (int64_t)gridDim.x * 256) {
    const int64_t i0 = u * U;
    int64_t row = 0, col = i0;
    if (rows > 1) {
      row = i0 / cols;
      col = i0 - row * cols;
    }
    const Run<T, U> rx = raw_run<T, U>(x, row * ldx + col);
    Run<T, U> rr;
    if (res) rr = raw_run<T, U>(res, row * ldr + col);
    Vec<U> f = unpack(rx);
    drop_run(d, (uint64_t)i0, f);
    if (res) {
      const Vec<U> r = unpack(rr);
#pragma unroll
      for (int k = 0; k < Vec<U>::P; ++k) f.p[k] = add2(r.p[k], f.p[k]);
    }
    put_run(y, row * ldy + col, pack<T>(f));
  }
  // (a single row: others are multiples of U)
  if (blockIdx.x == 0 && threadIdx.x < total - runs * U) {
    const int64_t i = runs * U + threadIdx.x;
    Vec<1> f = {{to_f32(x[i])}};
    drop_run(d, (uint64_t)i, f);
    y[i] = from_f32<T>(res ? __fadd_rn(to_f32(res[i]), f.p[0]) : f.p[0]);
  }
}

// Rows that are not 16-byte aligned: four elements of one generator call per
// step, each found in its row.
template <class T>
__global__ void __launch_bounds__(256, 4)
    dropout_any_kernel(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y, int64_t ldy,
                       int64_t rows, int64_t cols, const __grid_constant__ Drop d) {
  const int64_t total = rows * cols, runs = (total + 3) / 4;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < runs;
       u += (int64_t)gridDim.x * 256) {
    const int64_t i0 = u * 4;
    const int64_t row0 = i0 / cols, col0 = i0 - row0 * cols;
    Vec<4> f;
    float r[4];
    int64_t row = row0, col = col0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool ok = i0 + k < total;
      (k & 1 ? f.p[k / 2].y : f.p[k / 2].x) = ok ? to_f32(x[row * ldx + col]) : 0.f;
      r[k] = ok && res ? to_f32(res[row * ldr + col]) : 0.f;
      if (++col == cols) col = 0, ++row;
    }
    drop_run(d, (uint64_t)i0, f);
    row = row0, col = col0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float v = k & 1 ? f.p[k / 2].y : f.p[k / 2].x;
      if (i0 + k < total) y[row * ldy + col] = from_f32<T>(res ? __fadd_rn(r[k], v) : v);
      if (++col == cols) col = 0, ++row;
    }
  }
}

template <class T>
int launch_dropout(const void* x, int64_t ldx, const void* res, int64_t ldr, void* y, int64_t ldy,
                   int64_t rows, int64_t cols, const Drop& d, cudaStream_t s) {
  constexpr int U = 16 / sizeof(T);
  if ((ldx == cols || rows == 1) && (ldy == cols || rows == 1) && (!res || ldr == cols || rows == 1)) {
    cols *= rows;  // one long row
    rows = 1;
    ldx = ldy = ldr = cols;
  }
  const int64_t total = rows * cols, runs = (total + 3) / 4;
  const bool vec = aligned16(x) && aligned16(y) && (!res || aligned16(res)) &&
                   (rows == 1 || (cols % U == 0 && rows16(x, ldx, sizeof(T)) &&
                                  rows16(y, ldy, sizeof(T)) && rows16(res, ldr, sizeof(T))));
  const int grid = (int)std::min<int64_t>((runs + 255) / 256, 24ll * sm_count());
  ProfScope prof(ROT_PROF_ELEMENTWISE, (double)total * sizeof(T) * (res ? 3 : 2), s);
  auto k = vec ? dropout_kernel<T, U> : dropout_any_kernel<T>;
  k<<<grid, 256, 0, s>>>((const T*)x, ldx, (const T*)res, ldr, (T*)y, ldy, rows, cols, d);
  return launched();
}

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------

struct NormFwd {
  const void *x, *res, *w, *b;
  void *h, *y;
  float *mean, *rstd;
  int64_t ldx, ldr, ldh, ldy, rows;
  int cols;
  int w32;  // weight and bias are float32 (otherwise of the row's type)
  float eps;
  Drop d;
};

struct NormBwd {
  const void *dy, *h, *w, *dh;
  const float *mean, *rstd;
  void *dres, *dx;
  float* part;  // [parts][2][cols]: dweight, dbias
  int64_t lddy, ldh, lddh, lddres, lddx, rows;
  int cols;
  int w32;
  Drop d;
};

template <class T, int U>
__device__ __forceinline__ Vec<U> load_weight(const void* w, bool w32, int c) {
  if (!w32) return unpack(raw_run<T, U>(w, c));
  Vec<U> f;
  if constexpr (U > 1) {
#pragma unroll
    for (int k = 0; k < U / 2; k += 2) {
      const float4 v = *reinterpret_cast<const float4*>((const float*)w + c + 2 * k);
      f.p[k] = make_float2(v.x, v.y), f.p[k + 1] = make_float2(v.z, v.w);
    }
  } else {
    f.p[0] = ((const float*)w)[c];
  }
  return f;
}

// 1 / sqrt(v): the approximation and one Newton step (as exact as the two
// rounded operations, at a few instructions); the plain operations at the ends
// of the range.
__device__ __forceinline__ float inverse_root(float v) {
  const float r = rsqrtf(v);
  if (!(v > 1e-36f && v < 1e36f)) return 1.f / sqrtf(v);
  return r * fmaf(-0.5f * v * r, r, 1.5f);
}

// Waits for the TPR threads of this thread's row (a block may hold several).
template <int TPR, int BLOCK>
__device__ __forceinline__ void row_barrier() {
  if constexpr (TPR == BLOCK)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / TPR), "n"(TPR) : "memory");
}

// Sums of two values over the TPR threads of a row, in one exchange; `red`
// holds a pair per warp of the block.  Calls in a row need different `red`
// arrays (a thread may still read the last one).
template <int TPR, int BLOCK>
__device__ __forceinline__ float2 row_sum2(float x, float y, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float2 v = make_float2(__shfl_xor_sync(0xffffffffu, x, o),
                                 __shfl_xor_sync(0xffffffffu, y, o));
    const float2 w = add2(make_float2(x, y), v);
    x = w.x, y = w.y;
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(x, y);
    row_barrier<TPR, BLOCK>();
    const float4* p = reinterpret_cast<const float4*>(red + warp / W * W);
    float2 sum = both(0.f);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const float4 v = p[i];
      sum = add2(sum, add2(make_float2(v.x, v.y), make_float2(v.z, v.w)));
    }
    return sum;
  }
  return make_float2(x, y);
}
template <int TPR, int BLOCK>
__device__ __forceinline__ float row_sum(float x, float* red) {
  x = warp_sum(x);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = x;
    row_barrier<TPR, BLOCK>();
    const float4* p = reinterpret_cast<const float4*>(red + warp / W * W);
    float2 sum = both(0.f);
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const float4 v = p[i];
      sum = add2(sum, add2(make_float2(v.x, v.y), make_float2(v.z, v.w)));
    }
    return sum.x + sum.y;
  }
  return x;
}

constexpr int block_of(int tpr) { return tpr > 128 ? tpr : 128; }

// A row in the registers of TPR threads, N runs of U elements each.  Every
// load of a row is issued before anything is computed or stored (a store may
// alias a later load as far as the compiler knows).
template <class T, int U, int TPR, int N>
__global__ void __launch_bounds__(block_of(TPR), TPR == 1024 ? 1 : 640 / block_of(TPR))
    norm_fwd_kernel(const __grid_constant__ NormFwd a) {
  constexpr int kBlock = block_of(TPR), RPB = kBlock / TPR;
  __shared__ __align__(16) float red[2][kBlock / 32];
  const int t = threadIdx.x % TPR;
  const float inv = 1.f / (float)a.cols;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < a.rows;
  Run<T, U> x[N], r[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * TPR + t) * U;
    if (live && c < a.cols) {
      x[n] = raw_run<T, U>(a.x, row * a.ldx + c);
      if (a.res) r[n] = raw_run<T, U>(a.res, row * a.ldr + c);
    }
  }
  Vec<U> h[N];
  using E = typename Vec<U>::E;
  constexpr int P = Vec<U>::P;
  E sum = all_of<E>(0.f);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * TPR + t) * U;
#pragma unroll
    for (int k = 0; k < P; ++k) h[n].p[k] = all_of<E>(0.f);
    if (live && c < a.cols) {
      h[n] = unpack(x[n]);
      if (a.h) {
        drop_run(a.d, (uint64_t)row * a.cols + c, h[n]);
        if (a.res) {
          const Vec<U> v = unpack(r[n]);
#pragma unroll
          for (int k = 0; k < P; ++k) h[n].p[k] = add2(v.p[k], h[n].p[k]);
        }
        const Run<T, U> stored = pack<T>(h[n]);
        put_run(a.h, row * a.ldh + c, stored);
        h[n] = unpack(stored);  // the norm reads what is stored
      }
#pragma unroll
      for (int k = 0; k < P; ++k) sum = add2(sum, h[n].p[k]);
    }
  }
  const float mean = row_sum<TPR, kBlock>(total(sum), red[0]) * inv;
  E sq = all_of<E>(0.f);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if ((n * TPR + t) * U < a.cols) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        h[n].p[k] = add2(h[n].p[k], all_of<E>(-mean));
        sq = fma2(h[n].p[k], h[n].p[k], sq);
      }
    }
  const float rstd = inverse_root(row_sum<TPR, kBlock>(total(sq), red[1]) * inv + a.eps);
  if (live && t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * TPR + t) * U;
    if (live && c < a.cols) {
      const Vec<U> w = load_weight<T, U>(a.w, a.w32, c);
      Vec<U> b;
#pragma unroll
      for (int k = 0; k < P; ++k) b.p[k] = all_of<E>(0.f);
      if (a.b) b = load_weight<T, U>(a.b, a.w32, c);
#pragma unroll
      for (int k = 0; k < P; ++k) h[n].p[k] = fma2(mul2(h[n].p[k], all_of<E>(rstd)), w.p[k], b.p[k]);
      put_run(a.y, row * a.ldy + c, pack<T>(h[n]));
    }
  }
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

// The gradient of one run, g, written out; dropped into dx.  d: the run of
// dh, already loaded.
template <class T, int U>
__device__ __forceinline__ void write_grad(const NormBwd& a, int64_t row, int c, Vec<U>& g,
                                           const Run<T, U>& d) {
  if (a.dh) {
    const Vec<U> v = unpack(d);
#pragma unroll
    for (int k = 0; k < Vec<U>::P; ++k) g.p[k] = add2(g.p[k], v.p[k]);
  }
  if (a.dres) put_run(a.dres, row * a.lddres + c, pack<T>(g));
  drop_run(a.d, (uint64_t)row * a.cols + c, g);
  put_run(a.dx, row * a.lddx + c, pack<T>(g));
}

template <int U>
__device__ __forceinline__ float at(const Vec<U>& v, int k) {
  if constexpr (U == 1)
    return v.p[0];
  else
    return k & 1 ? v.p[k / 2].y : v.p[k / 2].x;
}

// A block walks the rows with a stride and sums its columns' weight gradients,
// in registers or (SMEM: rows of 1024 threads, which leave no registers) in
// shared memory at places of the thread's own; each block writes one part at
// its end.
//
// 16-byte runs (U > 1) come through shared memory by asynchronous copies of
// kDepth rows ahead; a thread copies and reads its own runs alone, so that no
// thread waits for another's, and the registers are left to the sums.
template <int U, bool SMEM>
constexpr int kDepth = U > 1 && !SMEM ? 2 : 0;

__device__ __forceinline__ void copy16(void* smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(smem)),
               "l"(global)
               : "memory");
}

template <class T, int U, int TPR, int N, bool SMEM>
__global__ void __launch_bounds__(block_of(TPR), TPR == 1024 ? 1 : 512 / block_of(TPR))
    norm_bwd_kernel(const __grid_constant__ NormBwd a) {
  constexpr int kBlock = block_of(TPR), RPB = kBlock / TPR, D = kDepth<U, SMEM>;
  extern __shared__ __align__(16) float dyn[];  // SMEM: dweight, dbias sums; else the rows ahead
  __shared__ __align__(16) float2 red[2][kBlock / 32];
  __shared__ float join[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * N * U : 1];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const float inv = 1.f / (float)a.cols;
  using E = typename Vec<U>::E;
  constexpr int P = Vec<U>::P;
  Vec<U> dw[SMEM ? 1 : N], db[SMEM ? 1 : N];
  // (SMEM: run n of thread t at element (n * TPR + t) * U of each half)
  E* sums = reinterpret_cast<E*>(dyn);
  constexpr int kHalf = N * TPR * P;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if constexpr (SMEM)
        sums[(n * TPR + t) * P + k] = sums[kHalf + (n * TPR + t) * P + k] = all_of<E>(0.f);
      else
        dw[n].p[k] = db[n].p[k] = all_of<E>(0.f);
    }
  // rows ahead: [slot][array][run][thread]
  Run<T, U>* ahead = reinterpret_cast<Run<T, U>*>(dyn) + threadIdx.x;
  auto slot_of = [&](int slot, int array, int n) {
    return ahead + ((slot * 3 + array) * N + n) * kBlock;
  };
  auto fetch = [&](int slot, int64_t row) {
    if (row < a.rows) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = (n * TPR + t) * U;
        if (c < a.cols) {
          copy16(slot_of(slot, 0, n), (const T*)a.dy + row * a.lddy + c);
          copy16(slot_of(slot, 1, n), (const T*)a.h + row * a.ldh + c);
          if (a.dh) copy16(slot_of(slot, 2, n), (const T*)a.dh + row * a.lddh + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  const int64_t first = (int64_t)blockIdx.x * RPB + group;
  if constexpr (D > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, first + d * step);
  }
  int turn = 0, slot = 0;
  float mean = first < a.rows ? a.mean[first] : 0.f, rstd = first < a.rows ? a.rstd[first] : 0.f;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += step) {
    const int64_t row = base + group;
    const bool live = row < a.rows;
    if constexpr (D > 0) asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    Run<T, U> dy[N], h[N], dh[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * TPR + t) * U;
      if (live && c < a.cols) {
        if constexpr (D > 0) {
          dy[n] = *slot_of(slot, 0, n);
          h[n] = *slot_of(slot, 1, n);
        } else {
          dy[n] = raw_run<T, U>(a.dy, row * a.lddy + c);
          h[n] = raw_run<T, U>(a.h, row * a.ldh + c);
          if (a.dh) dh[n] = raw_run<T, U>(a.dh, row * a.lddh + c);
        }
      }
    }
    E s1 = all_of<E>(0.f), s2 = all_of<E>(0.f);
    Vec<U> hat[N], wdy[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * TPR + t) * U;
      if (live && c < a.cols) {
        const Vec<U> w = load_weight<T, U>(a.w, a.w32, c), y = unpack(dy[n]), x = unpack(h[n]);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          hat[n].p[k] = mul2(add2(x.p[k], all_of<E>(-mean)), all_of<E>(rstd));
          wdy[n].p[k] = mul2(y.p[k], w.p[k]);
          s1 = add2(s1, wdy[n].p[k]);
          s2 = fma2(wdy[n].p[k], hat[n].p[k], s2);
          if constexpr (SMEM) {
            E* q = sums + (n * TPR + t) * P + k;
            q[0] = fma2(y.p[k], hat[n].p[k], q[0]);
            q[kHalf] = add2(q[kHalf], y.p[k]);
          } else {
            dw[n].p[k] = fma2(y.p[k], hat[n].p[k], dw[n].p[k]);
            db[n].p[k] = add2(db[n].p[k], y.p[k]);
          }
        }
      }
    }
    const float rstd0 = rstd;
    if (row + step < a.rows) mean = a.mean[row + step], rstd = a.rstd[row + step];
    const float2 s = row_sum2<TPR, kBlock>(total(s1), total(s2), red[turn]);
    const float m1 = s.x * inv, m2 = s.y * inv;
    turn ^= 1;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * TPR + t) * U;
      if (live && c < a.cols) {
        if constexpr (D > 0) {
          if (a.dh) dh[n] = *slot_of(slot, 2, n);
        }
        Vec<U> g;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          g.p[k] = add2(wdy[n].p[k], all_of<E>(-m1));
          g.p[k] = mul2(fma2(hat[n].p[k], all_of<E>(-m2), g.p[k]), all_of<E>(rstd0));
        }
        write_grad(a, row, c, g, dh[n]);
      }
    }
    if constexpr (D > 0) {
      fetch(slot, row + D * step);
      slot = slot + 1 == D ? 0 : slot + 1;
    }
  }
  // this block's part of the weight gradient: the groups' sums in order
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int k = 0; k < U; ++k)
          join[group][(n * TPR + t) * U + k] = at<U>(which ? db[n] : dw[n], k);
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += kBlock) {
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < RPB; ++g) sum += join[g][c];
        part[which * a.cols + c] = sum;
      }
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = (n * TPR + t) * U;
        if (c < a.cols) {
#pragma unroll
          for (int k = 0; k < U; ++k) {
            if constexpr (SMEM)
              part[which * a.cols + c + k] = dyn[which * N * TPR * U + c + k];
            else
              part[which * a.cols + c + k] = at<U>(which ? db[n] : dw[n], k);
          }
        }
      }
    }
  }
}

// Rows too wide for the registers: the rows' gradients (two passes over a
// row) and the columns' partial sums in kernels of their own.
template <class T>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const __grid_constant__ NormBwd a) {
  __shared__ __align__(16) float2 red[2][32];
  const float inv = 1.f / (float)a.cols;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    const T* dy = (const T*)a.dy + row * a.lddy;
    const T* h = (const T*)a.h + row * a.ldh;
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += 1024) {
      const float wdy = to_f32(dy[c]) * load_weight<T, 1>(a.w, a.w32, c).p[0];
      s1 += wdy;
      s2 += wdy * ((to_f32(h[c]) - mean) * rstd);
    }
    const float2 s = row_sum2<1024, 1024>(s1, s2, red[turn]);
    s1 = s.x * inv, s2 = s.y * inv;
    turn ^= 1;
    for (int c = threadIdx.x; c < a.cols; c += 1024) {
      const float w = load_weight<T, 1>(a.w, a.w32, c).p[0];
      const float hat = (to_f32(h[c]) - mean) * rstd;
      Vec<1> g = {{rstd * (to_f32(dy[c]) * w - s1 - hat * s2)}};
      Run<T, 1> d;
      if (a.dh) d = raw_run<T, 1>(a.dh, row * a.lddh + c);
      write_grad(a, row, c, g, d);
    }
  }
}

template <class T>
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(const __grid_constant__ NormBwd a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float dy = to_f32(((const T*)a.dy)[row * a.lddy + c]);
    dw += dy * ((to_f32(((const T*)a.h)[row * a.ldh + c]) - a.mean[row]) * a.rstd[row]);
    db += dy;
  }
  float* part = a.part + (int64_t)blockIdx.y * 2 * a.cols;
  part[c] = dw;
  part[a.cols + c] = db;
}

// dweight and dbias: the parts' sums.  32 columns by 32 strided shares of the
// parts per block, joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_join_kernel(const float* part, int parts, int cols,
                                                         float* dweight, float* dbias) {
  __shared__ float share[32][33];
  wait_for_prior();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + lane, width = 2ll * cols;
  float sum = 0.f;
  if (i < width)
    for (int p = warp; p < parts; p += 32) sum += part[(int64_t)p * width + i];
  share[warp][lane] = sum;
  __syncthreads();
  sum = warp_sum(share[lane][warp]);  // column `warp` of this block
  const int64_t j = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && j < width) {
    if (j < cols)
      dweight[j] = sum;
    else if (dbias)
      dbias[j - cols] = sum;
  }
}

// Partial sums kept at most (the workspace's size does not depend on the GPU).
constexpr int kMaxParts = 608;

// A thread's share of a row: `runs` 16-byte runs (four, so that what a thread
// does once per row weighs little; two in the backward pass, which keeps two
// sums for each element), or 8 elements one by one where the rows are not
// 16-byte aligned.
template <int U>
constexpr int kFwdRuns = U > 1 ? 4 : 8;
template <int U>
constexpr int kBwdRuns = U > 1 ? 2 : 8;

// Threads per row that hold `cols` in shares of `share` elements; 0: too wide.
inline int row_threads(int cols, int share) {
  for (int t : {32, 128, 256, 512, 1024})
    if (cols <= t * share) return t;
  return 0;
}

template <class T, int U>
int launch_fwd(const NormFwd& a, cudaStream_t s) {
  constexpr int N = kFwdRuns<U>;
  const int tpr = row_threads(a.cols, U * N);
  const int rpb = tpr == 32 ? 4 : 1;
  const int64_t blocks = (a.rows + rpb - 1) / rpb;
  if (blocks > 0x7FFFFFFF) return ROT_EINVAL;
  const unsigned grid = (unsigned)blocks;
  switch (tpr) {
    case 32: norm_fwd_kernel<T, U, 32, N><<<grid, 128, 0, s>>>(a); break;
    case 128: norm_fwd_kernel<T, U, 128, N><<<grid, 128, 0, s>>>(a); break;
    case 256: norm_fwd_kernel<T, U, 256, N><<<grid, 256, 0, s>>>(a); break;
    case 512: norm_fwd_kernel<T, U, 512, N><<<grid, 512, 0, s>>>(a); break;
    case 1024: norm_fwd_kernel<T, U, 1024, N><<<grid, 1024, 0, s>>>(a); break;
    default: norm_fwd_wide_kernel<T><<<grid, 1024, 0, s>>>(a); break;
  }
  return launched();
}

template <class T>
int run_fwd(const NormFwd& a, cudaStream_t s) {
  constexpr int U = 16 / sizeof(T);
  ProfScope prof(ROT_PROF_ELEMENTWISE,
                 (double)a.rows * a.cols * sizeof(T) * (2 + (a.res != nullptr) + (a.h != nullptr)), s);
  const bool vec = a.cols % U == 0 && rows16(a.x, a.ldx, sizeof(T)) &&
                   rows16(a.res, a.ldr, sizeof(T)) && rows16(a.h, a.ldh, sizeof(T)) &&
                   rows16(a.y, a.ldy, sizeof(T)) && aligned16(a.w) && (!a.b || aligned16(a.b));
  return vec ? launch_fwd<T, U>(a, s) : launch_fwd<T, 1>(a, s);
}

template <class T, int U, int TPR, bool SMEM>
int launch_bwd_rows(const NormBwd& a, int* parts, cudaStream_t s) {
  constexpr int N = kBwdRuns<U>, block = block_of(TPR), rpb = block / TPR;
  constexpr int smem = SMEM ? 2 * N * U * TPR * 4 : kDepth<U, SMEM> * 3 * N * block * 16;
  auto k = norm_bwd_kernel<T, U, TPR, N, SMEM>;
  if constexpr (smem > 0) {
    static const cudaError_t attr =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (attr != cudaSuccess) return ROT_ECUDA;
  }
  const int per_sm = TPR == 1024 ? 1 : 512 / block;
  *parts = (int)std::min<int64_t>((a.rows + rpb - 1) / rpb,
                                  std::min(kMaxParts, per_sm * sm_count()));
  k<<<*parts, block, smem, s>>>(a);
  return launched();
}

template <class T, int U>
int launch_bwd(const NormBwd& a, int* parts, cudaStream_t s) {
  switch (row_threads(a.cols, U * kBwdRuns<U>)) {
    case 32: return launch_bwd_rows<T, U, 32, false>(a, parts, s);
    case 128: return launch_bwd_rows<T, U, 128, false>(a, parts, s);
    case 256: return launch_bwd_rows<T, U, 256, false>(a, parts, s);
    case 512: return launch_bwd_rows<T, U, 512, false>(a, parts, s);
    case 1024: return launch_bwd_rows<T, U, 1024, true>(a, parts, s);
  }
  norm_bwd_wide_kernel<T><<<(unsigned)std::min<int64_t>(a.rows, 1 << 20), 1024, 0, s>>>(a);
  const int e = launched();
  if (e != ROT_OK) return e;
  *parts = (int)std::min<int64_t>(a.rows, 64);
  ProfScope prof(ROT_PROF_ELEMENTWISE, 0.0, s);
  norm_bwd_cols_kernel<T><<<dim3((a.cols + 255) / 256, *parts), 256, 0, s>>>(a);
  return launched();
}

template <class T>
int run_bwd(const NormBwd& a, float* dweight, float* dbias, cudaStream_t s) {
  constexpr int U = 16 / sizeof(T);
  int parts = 0, e = ROT_OK;
  {
    ProfScope prof(ROT_PROF_ELEMENTWISE,
                   (double)a.rows * a.cols * sizeof(T) *
                       (3 + (a.dh != nullptr) + (a.dres != nullptr)), s);
    const bool vec = a.cols % U == 0 && rows16(a.dy, a.lddy, sizeof(T)) &&
                     rows16(a.h, a.ldh, sizeof(T)) && rows16(a.dh, a.lddh, sizeof(T)) &&
                     rows16(a.dres, a.lddres, sizeof(T)) && rows16(a.dx, a.lddx, sizeof(T)) &&
                     aligned16(a.w);
    e = vec ? launch_bwd<T, U>(a, &parts, s) : launch_bwd<T, 1>(a, &parts, s);
  }
  if (e != ROT_OK) return e;
  ProfScope prof(ROT_PROF_ELEMENTWISE, 0.0, s);
  return launch_behind(norm_join_kernel, (2 * a.cols + 31) / 32, 1024, 0, s, a.part, parts, a.cols,
                       dweight, dbias);
}

template <template <class> class Fn, class... Args>
int by_type(int32_t type, Args&&... args) {
  if (type == ROT_TYPE_F32) return Fn<float>::run(args...);
  if (type == ROT_TYPE_F16) return Fn<__half>::run(args...);
  return Fn<__nv_bfloat16>::run(args...);
}
template <class T>
struct FwdFn {
  static int run(const NormFwd& a, cudaStream_t s) { return run_fwd<T>(a, s); }
};
template <class T>
struct BwdFn {
  static int run(const NormBwd& a, float* dw, float* db, cudaStream_t s) {
    return run_bwd<T>(a, dw, db, s);
  }
};
template <class T>
struct DropFn {
  static int run(const void* x, int64_t ldx, const void* res, int64_t ldr, void* y, int64_t ldy,
                 int64_t rows, int64_t cols, const Drop& d, cudaStream_t s) {
    return launch_dropout<T>(x, ldx, res, ldr, y, ldy, rows, cols, d, s);
  }
};

inline bool bad_p(double p) { return !(p >= 0.0 && p <= 1.0); }

// rows * cols elements must be countable in 63 bits with room for a pitch
inline bool bad_size(int64_t rows, int64_t cols) {
  return rows < 0 || cols < 0 || (cols > 0 && rows > (int64_t(1) << 60) / cols);
}

}  // namespace
}  // namespace ops
}  // namespace rot

using namespace rot;
using namespace rot::ops;

extern "C" {

int rot_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y,
                int64_t ldy, int64_t rows, int64_t cols, int32_t type, double p, uint64_t seed,
                uint64_t offset, void* stream) {
  if (bad_size(rows, cols) || !float_type(type) || bad_p(p)) return ROT_EINVAL;
  if (ldx < cols || ldy < cols || (residual && ldr < cols)) return ROT_EINVAL;
  if (rows == 0 || cols == 0) return ROT_OK;
  if (!x || !y) return ROT_EINVAL;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  return guarded([&] {
    return by_type<DropFn>(type, x, ldx, residual, ldr, y, ldy, rows, cols,
                           make_drop(p, seed, offset), static_cast<cudaStream_t>(stream));
  });
}

int rot_layer_norm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           const void* weight, const void* bias, int32_t wtype, void* h_out,
                           int64_t ldh, void* y, int64_t ldy, float* mean, float* rstd,
                           int64_t rows, int64_t cols, int32_t type, float eps, double p,
                           uint64_t seed, uint64_t offset, void* stream) {
  if (rows < 0 || cols < 1 || cols > ROT_MAX_DIM || bad_size(rows, cols)) return ROT_EINVAL;
  if (!float_type(type) || (wtype != ROT_TYPE_F32 && wtype != type)) return ROT_EINVAL;
  if (bad_p(p) || !(eps >= 0.f)) return ROT_EINVAL;
  const bool mixes = residual || p > 0.0;
  if (ldx < cols || ldy < cols || (residual && ldr < cols) || (mixes && ldh < cols))
    return ROT_EINVAL;
  if (rows == 0) return ROT_OK;
  if (!x || !weight || !y || !mean || !rstd || (mixes && !h_out)) return ROT_EINVAL;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  NormFwd a;
  a.x = x, a.res = residual, a.w = weight, a.b = bias;
  a.h = mixes ? h_out : nullptr, a.y = y, a.mean = mean, a.rstd = rstd;
  a.ldx = ldx, a.ldr = ldr, a.ldh = ldh, a.ldy = ldy, a.rows = rows, a.cols = (int)cols;
  a.w32 = wtype == ROT_TYPE_F32, a.eps = eps, a.d = make_drop(p, seed, offset);
  return guarded([&] { return by_type<FwdFn>(type, a, static_cast<cudaStream_t>(stream)); });
}

uint64_t rot_layer_norm_work_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || cols > ROT_MAX_DIM) return 0;
  return align256(8ull * (uint64_t)cols * (uint64_t)std::min<int64_t>(rows, kMaxParts));
}

int rot_layer_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh,
                            const float* mean, const float* rstd, const void* weight,
                            int32_t wtype, const void* dh, int64_t lddh, void* dres_out,
                            int64_t lddres, void* dx, int64_t lddx, float* dweight, float* dbias,
                            int64_t rows, int64_t cols, int32_t type, double p, uint64_t seed,
                            uint64_t offset, void* work, uint64_t work_bytes, void* stream) {
  if (rows < 0 || cols < 1 || cols > ROT_MAX_DIM || bad_size(rows, cols)) return ROT_EINVAL;
  if (!float_type(type) || (wtype != ROT_TYPE_F32 && wtype != type) || bad_p(p))
    return ROT_EINVAL;
  if (lddy < cols || ldh < cols || lddx < cols || (dh && lddh < cols) ||
      (dres_out && lddres < cols))
    return ROT_EINVAL;
  if (!dweight || (p > 0.0 && rows > 0 && !dres_out)) return ROT_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    const int dev = check_device();
    if (dev != ROT_OK) return dev;
    if (cudaMemsetAsync(dweight, 0, 4 * cols, s) != cudaSuccess ||
        (dbias && cudaMemsetAsync(dbias, 0, 4 * cols, s) != cudaSuccess))
      return ROT_ECUDA;
    return ROT_OK;
  }
  if (!dy || !h || !mean || !rstd || !weight || !dx || !work) return ROT_EINVAL;
  if ((reinterpret_cast<uintptr_t>(work) & 255) ||
      work_bytes < rot_layer_norm_work_bytes(rows, cols))
    return ROT_EINVAL;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  NormBwd a;
  a.dy = dy, a.h = h, a.w = weight, a.dh = dh, a.mean = mean, a.rstd = rstd;
  a.dres = dres_out, a.dx = dx, a.part = static_cast<float*>(work);
  a.lddy = lddy, a.ldh = ldh, a.lddh = lddh, a.lddres = lddres, a.lddx = lddx;
  a.rows = rows, a.cols = (int)cols, a.w32 = wtype == ROT_TYPE_F32;
  a.d = make_drop(p, seed, offset);
  return guarded([&] { return by_type<BwdFn>(type, a, dweight, dbias, s); });
}

}  // extern "C"
