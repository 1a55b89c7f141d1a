// Dropout (include/rot_ops.h), and the entry points of layer norm (its kernels:
// ops_norm_fwd.cu, ops_norm_bwd.cu).  Bound by HBM: one read of every input,
// one write of the output, the mask computed where it is used.
//
// 16384 x 6144 in bfloat16 with a residual: 96 us, 6.3 TB/s.
#include <algorithm>
#include <cmath>

#include "ops_norm.cuh"
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

// Rows that are not 16-byte aligned: a warp takes kAny * 32 consecutive
// elements of the row-major order, lane by lane, and shares their generator
// calls; each element is found in its row.  32768 x 1325 in 79 us, bound by
// instructions; a warp's share in one row alone, with one address for all of
// it, 103 us.
constexpr int kAny = 8;

template <class T>
__global__ void __launch_bounds__(256, 4)
    dropout_any_kernel(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y, int64_t ldy,
                       int64_t rows, int64_t cols, const __grid_constant__ Drop d) {
  const int64_t total = rows * cols;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 8;
  for (int64_t u = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; u * (kAny * 32) < total;
       u += warps) {
    const int64_t i0 = u * (kAny * 32);
    const int64_t i = i0 + lane;
    int64_t row, col;
    if (total <= 0xFFFFFFFFll) {  // (a division of 32 bits is a fraction of one of 64)
      row = (uint32_t)i / (uint32_t)cols;
      col = (uint32_t)i - (uint32_t)row * (uint32_t)cols;
    } else {
      row = i / cols;
      col = i - row * cols;
    }
    const int left = (int)min(total - i, (int64_t)kAny * 32);  // of this lane's, 32 apart
    T v[kAny], r[kAny];
    const T* px = x + row * ldx + col;
    const T* pr = res ? res + row * ldr + col : nullptr;
    T* py[kAny];
    py[0] = y + row * ldy + col;
#pragma unroll
    for (int k = 0; k < kAny; ++k) {
      v[k] = 32 * k < left ? *px : from_f32<T>(0.f);
      r[k] = res && 32 * k < left ? *pr : from_f32<T>(0.f);
      if (k == kAny - 1) break;
      // 32 further, over the ends of rows (one at most unless they are short)
      px += 32, py[k + 1] = py[k] + 32, pr += 32;
      col += 32;
      if (col >= cols) {
        do {
          col -= cols;
          px += ldx - cols, py[k + 1] += ldy - cols, pr += ldr - cols;
        } while (cols < 32 && col >= cols);
      }
    }
    const uint32_t bits = d.on ? keep_bits<kAny>(d, (uint64_t)i0) : 0;
#pragma unroll
    for (int k = 0; k < kAny; ++k) {
      if (32 * k >= left) break;
      float f = to_f32(v[k]);
      if (d.on) f = kept(d, bits >> k & 1, f);
      *py[k] = from_f32<T>(res ? __fadd_rn(to_f32(r[k]), f) : f);
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Drop d = make_drop(p, seed, offset);
    if (type == ROT_TYPE_F32)
      return launch_dropout<float>(x, ldx, residual, ldr, y, ldy, rows, cols, d, s);
    if (type == ROT_TYPE_F16)
      return launch_dropout<__half>(x, ldx, residual, ldr, y, ldy, rows, cols, d, s);
    return launch_dropout<__nv_bfloat16>(x, ldx, residual, ldr, y, ldy, rows, cols, d, s);
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
  return guarded([&] { return norm_forward(type, a, static_cast<cudaStream_t>(stream)); });
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
  return guarded([&] { return norm_backward(type, a, dweight, dbias, s); });
}

}  // extern "C"
