// Layer norm backward (include/rot_ops.h): the rows' gradients, and the weight
// gradient as partial sums and their join.  Bound by HBM, with dropout nearly
// as long in the generator's arithmetic.
//
// 16383 x 2048 in bfloat16 with the stream's gradient and dropout: 75 us and 4
// for the join, 4.2 TB/s.  Five blocks per SM instead of four leave too few
// registers (80 us), as do the generator's keys in shared memory (79 us).
#include <algorithm>

#include "ops_norm.cuh"
#include "profile.h"

namespace rot {
namespace ops {
namespace {

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
//
// Single elements (U = 1) have the next row's and the weights in registers
// instead (not with dropout and the sums in shared memory, which spills):
// 32768 x 1325 in 249 us; loaded where they are used, 282 us, and 319 and 326
// us on twice and 1.5 times the threads per SM, which spill.
template <int U, bool SMEM>
constexpr int kDepth = U > 1 && !SMEM ? 2 : 0;

__device__ __forceinline__ void copy16(void* smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(smem)),
               "l"(global)
               : "memory");
}

// Blocks per SM.
constexpr int per_sm_of(int tpr) { return tpr == 1024 ? 1 : 512 / block_of(tpr); }

template <class T, int U, int TPR, int N, bool SMEM, bool DROP>
__global__ void __launch_bounds__(block_of(TPR), per_sm_of(TPR))
    norm_bwd_kernel(const __grid_constant__ NormBwd a) {
  constexpr int kBlock = block_of(TPR), RPB = kBlock / TPR, D = kDepth<U, SMEM>;
  // single elements: the next row's, and the weights, in registers
  constexpr bool kNext = U == 1 && !(SMEM && DROP);
  extern __shared__ __align__(16) float dyn[];  // SMEM: dweight, dbias sums; else the rows ahead
  __shared__ __align__(16) float2 red[2][kBlock / 32];
  __shared__ float join[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * N * U : 1];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const bool busy = has_columns<U, N>(t, a.cols);  // (the same for a warp)
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
  // (past the row's end a thread takes its first element again, with a
  // gradient of 0, and stores nothing)
  int c[N];
  bool in[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    c[n] = column_of<U, TPR, N>(n, t);
    in[n] = c[n] < a.cols;
    if (U > 1 && !in[n]) c[n] = 0;
  }
  Vec<U> weight[N];
  if constexpr (kNext) get_weights<T>(weight, a.w, a.w32, c, in);
  // rows ahead: [slot][array][run][thread]
  Run<T, U>* ahead = reinterpret_cast<Run<T, U>*>(dyn) + threadIdx.x;
  auto slot_of = [&](int slot, int array, int n) {
    return ahead + ((slot * 3 + array) * N + n) * kBlock;
  };
  auto fetch = [&](int slot, int64_t row) {
    if (row < a.rows) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        copy16(slot_of(slot, 0, n), (const T*)a.dy + row * a.lddy + c[n]);
        copy16(slot_of(slot, 1, n), (const T*)a.h + row * a.ldh + c[n]);
        if (a.dh) copy16(slot_of(slot, 2, n), (const T*)a.dh + row * a.lddh + c[n]);
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
  Run<T, U> dy[N], h[N], dh[N];
  auto load = [&](int64_t row) {
    if (row >= a.rows || !busy) return;
    get_runs(dy, a.dy, row * a.lddy, c, in);
    get_runs(h, a.h, row * a.ldh, c, in);
    if (a.dh) get_runs(dh, a.dh, row * a.lddh, c, in);
  };
  if constexpr (kNext) load(first);
  int turn = 0, slot = 0;
  float mean = first < a.rows ? a.mean[first] : 0.f, rstd = first < a.rows ? a.rstd[first] : 0.f;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += step) {
    const int64_t row = base + group;
    const bool live = row < a.rows && busy;
    if constexpr (D > 0) asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    Vec<U> hat[N], wdy[N];
    E s1 = all_of<E>(0.f), s2 = all_of<E>(0.f);
    if (live) {  // (the same for a warp)
      if constexpr (D > 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
          dy[n] = *slot_of(slot, 0, n);
          h[n] = *slot_of(slot, 1, n);
        }
      } else if constexpr (!kNext) {
        load(row);
        if constexpr (U == 1) get_weights<T>(weight, a.w, a.w32, c, in);
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        Vec<U> w;
        if constexpr (U > 1)
          w = load_weight<T, U>(a.w, a.w32, c[n]);
        else
          w = weight[n];
        const Vec<U> x = unpack(h[n]);
        Vec<U> y = unpack(dy[n]);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          if (!in[n]) y.p[k] = all_of<E>(0.f);
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
    Run<T, U> dh0[N];
    if constexpr (kNext) {
#pragma unroll
      for (int n = 0; n < N; ++n) dh0[n] = dh[n];
      load(row + step);
    }
    const float rstd0 = rstd;
    if (row + step < a.rows) mean = a.mean[row + step], rstd = a.rstd[row + step];
    const float2 s = row_sum2<TPR, kBlock>(total(s1), total(s2), red[turn]);
    const float m1 = s.x * inv, m2 = s.y * inv;
    turn ^= 1;
    if (live) {
      Vec<U> g[N];
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int k = 0; k < P; ++k) {
          g[n].p[k] = add2(wdy[n].p[k], all_of<E>(-m1));
          g[n].p[k] = mul2(fma2(hat[n].p[k], all_of<E>(-m2), g[n].p[k]), all_of<E>(rstd0));
        }
      if (a.dh) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
          if constexpr (D > 0) dh[n] = *slot_of(slot, 2, n);
          const Vec<U> v = unpack(kNext ? dh0[n] : dh[n]);
#pragma unroll
          for (int k = 0; k < P; ++k) g[n].p[k] = add2(g[n].p[k], v.p[k]);
        }
      }
      if (a.dres) put_runs<T>(a.dres, row * a.lddres, c, in, g);
      if (DROP) drop_runs<U, N>(a.d, (uint64_t)row * a.cols, c, t, a.cols, g);
      put_runs<T>(a.dx, row * a.lddx, c, in, g);
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
          join[group][column_of<U, TPR, N>(n, t) + k] = at<U>(which ? db[n] : dw[n], k);
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
        const int c = column_of<U, TPR, N>(n, t);
        if (c < a.cols) {
#pragma unroll
          for (int k = 0; k < U; ++k) {
            if constexpr (SMEM)
              part[which * a.cols + c + k] = dyn[(which * N * TPR + n * TPR + t) * U + k];
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
    // (128 consecutive elements per warp)
    for (int c0 = threadIdx.x / 32 * 128; c0 < a.cols; c0 += 32 * 128) {
      const uint32_t bits = a.d.on ? keep_bits<4>(a.d, (uint64_t)row * a.cols + c0) : 0;
      float g[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = min(c0 + (int)threadIdx.x % 32 + 32 * k, a.cols - 1);
        const float w = load_weight<T, 1>(a.w, a.w32, c).p[0];
        const float hat = (to_f32(h[c]) - mean) * rstd;
        g[k] = rstd * (to_f32(dy[c]) * w - s1 - hat * s2);
        if (a.dh) g[k] = __fadd_rn(g[k], to_f32(((const T*)a.dh)[row * a.lddh + c]));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + threadIdx.x % 32 + 32 * k;
        if (c >= a.cols) continue;
        if (a.dres) ((T*)a.dres)[row * a.lddres + c] = from_f32<T>(g[k]);
        ((T*)a.dx)[row * a.lddx + c] = from_f32<T>(a.d.on ? kept(a.d, bits >> k & 1, g[k]) : g[k]);
      }
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

// A thread's share of a row: two 16-byte runs (it keeps two sums for each
// element), or single elements where the rows are not 16-byte aligned.
template <int U>
constexpr int kRuns = U > 1 ? 2 : kSingles;

template <class T, int U, int TPR, bool SMEM, bool DROP, int N = kRuns<U>>
int launch_bwd_rows(const NormBwd& a, int* parts, cudaStream_t s) {
  constexpr int block = block_of(TPR), rpb = block / TPR;
  constexpr int smem = SMEM ? 2 * N * U * TPR * 4 : kDepth<U, SMEM> * 3 * N * block * 16;
  auto k = norm_bwd_kernel<T, U, TPR, N, SMEM, DROP>;
  if constexpr (smem > 0) {
    static const cudaError_t attr =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (attr != cudaSuccess) return ROT_ECUDA;
  }
  constexpr int per_sm = per_sm_of(TPR);
  *parts = (int)std::min<int64_t>((a.rows + rpb - 1) / rpb,
                                  std::min(kMaxParts, per_sm * sm_count()));
  k<<<*parts, block, smem, s>>>(a);
  return launched();
}

template <class T, int U, bool DROP>
int launch_bwd(const NormBwd& a, int* parts, cudaStream_t s) {
  switch (U > 1 ? row_threads(a.cols, U * kRuns<U>) : row_threads_single(a.cols)) {
    case 32:
      if constexpr (U == 1) {
        if (a.cols <= 32 * kFewSingles)
          return launch_bwd_rows<T, U, 32, false, DROP, kFewSingles>(a, parts, s);
      }
      return launch_bwd_rows<T, U, 32, false, DROP>(a, parts, s);
    case 64:
      if constexpr (U == 1) return launch_bwd_rows<T, U, 64, false, DROP>(a, parts, s);
      break;
    case 128: return launch_bwd_rows<T, U, 128, false, DROP>(a, parts, s);
    case 256: return launch_bwd_rows<T, U, 256, false, DROP>(a, parts, s);
    case 512: return launch_bwd_rows<T, U, 512, false, DROP>(a, parts, s);
    case 1024:
      // (17610 x 4751: 506 us, on 1024 threads 650; without dropout 250 and 341)
      if constexpr (U == 1)
        return launch_bwd_rows<T, U, 512, true, DROP, 2 * kSingles>(a, parts, s);
      else
        return launch_bwd_rows<T, U, 1024, true, DROP>(a, parts, s);
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
int run(const NormBwd& a, float* dweight, float* dbias, cudaStream_t s) {
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
    if (vec)
      e = a.d.on ? launch_bwd<T, U, true>(a, &parts, s) : launch_bwd<T, U, false>(a, &parts, s);
    else
      e = a.d.on ? launch_bwd<T, 1, true>(a, &parts, s) : launch_bwd<T, 1, false>(a, &parts, s);
  }
  if (e != ROT_OK) return e;
  ProfScope prof(ROT_PROF_ELEMENTWISE, 0.0, s);
  return launch_behind(norm_join_kernel, (2 * a.cols + 31) / 32, 1024, 0, s, a.part, parts, a.cols,
                       dweight, dbias);
}

}  // namespace

int norm_backward(int32_t type, const NormBwd& a, float* dweight, float* dbias, cudaStream_t s) {
  if (type == ROT_TYPE_F32) return run<float>(a, dweight, dbias, s);
  if (type == ROT_TYPE_F16) return run<__half>(a, dweight, dbias, s);
  return run<__nv_bfloat16>(a, dweight, dbias, s);
}

}  // namespace ops
}  // namespace rot
