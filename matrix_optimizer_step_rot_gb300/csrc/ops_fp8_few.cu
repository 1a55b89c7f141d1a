// C = A B^T for at most eight rows of A (rot_fp8_gemm, and rot_fp8_linear on a
// few tokens): bound by reading B once.
//
// The large kernel's 128-row tiles would be almost empty.  Here the roles
// turn: 16 rows of B are the tile's rows and the rows of A its 8 columns, so
// that one warp-wide mma.sync (m16n8k32, 8-bit operands, float32 sums) uses
// every byte of B that a thread loads.  Bytes come straight from global memory
// into the operand registers: the sum over K may take its elements in any
// order, so thread t of a row's four takes the 16 consecutive bytes at 16 t of
// each 64 as the operands of two instructions, and A's bytes, kept in shared
// memory, go the same way.  Each block of 128 of K is summed on its own and
// joins the total under its scales' exponent.
//
// A CTA takes 16 rows of B, its warps a share of K each, joined in a fixed
// order at the end.  With one or two tokens in a float type the CTA also
// rounds them to 8 bits itself, as the quantisation kernel does, so that a
// layer is one launch; with more that work, repeated by every CTA, would cost
// more than a launch.
//
// One token through 2048 x 6144: 5.9 us (12.6 MB; the latency of a launch, of
// the token's rounding and of the two loads' way is most of it).
#include <cuda_fp8.h>

#include <algorithm>

#include "ops_common.cuh"
#include "ops_fp8.h"
#include "profile.h"

namespace rot {
namespace ops {
namespace {

constexpr int kFewRows = 8;
constexpr int kSelfRounded = 2;  // rows of a float type that every CTA rounds itself
constexpr int kTile = 16;        // rows of B per CTA
constexpr int kWarps = 8;
constexpr int kDepth = 2;        // blocks of 128 of K on their way per warp
constexpr int kMaxShared = 100 << 10;

struct Few {
  const uint8_t *w, *sw;  // B: N x K, and its scales
  const void* x;          // A: M x K, float type, or 8-bit with scales sx
  const uint8_t* sx;
  void* y;
  int64_t ldw, ldsw, ldx, ldsx, ldy;
  int M, N, K, xtype, ytype, wsh, xsh, accumulate;
};

// v 2^e for any e that two scale bytes give, NaN where one of them is 255.
__device__ __forceinline__ float scaled(float v, int ea, int eb) {
  const int e = ea + eb - 127;  // biased
  if (e >= 1 && e <= 254 && max(ea, eb) < 255) return v * __uint_as_float((uint32_t)e << 23);
  return max(ea, eb) == 255 ? NAN : ldexpf(v, e - 127);
}

template <int W5, int X5>
__device__ __forceinline__ void mma16832(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
#define ROT_MMA(ta, tb)                                                              \
  asm volatile("mma.sync.aligned.m16n8k32.row.col.f32." ta "." tb                    \
               ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};" \
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                      \
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (W5 && X5)
    ROT_MMA("e5m2", "e5m2");
  else if constexpr (W5)
    ROT_MMA("e5m2", "e4m3");
  else if constexpr (X5)
    ROT_MMA("e4m3", "e5m2");
  else
    ROT_MMA("e4m3", "e4m3");
#undef ROT_MMA
}

// 16 bytes of a row from column k; what lies past column K reads as 0.
__device__ __forceinline__ uint4 load16(const uint8_t* p, int k, int K) {
  if (k + 16 <= K) return *reinterpret_cast<const uint4*>(p);
  uint32_t b[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int i = 0; i < K - k; ++i) {
    const uint32_t byte = (uint32_t)p[i] << (8 * (i & 3));
    b[0] |= i / 4 == 0 ? byte : 0u;
    b[1] |= i / 4 == 1 ? byte : 0u;
    b[2] |= i / 4 == 2 ? byte : 0u;
    b[3] |= i / 4 == 3 ? byte : 0u;
  }
  return make_uint4(b[0], b[1], b[2], b[3]);
}

// Row m of A by the whole CTA, rounded to E4M3: 16 elements per thread and
// turn, eight threads to a block of 128.
template <class T>
__device__ __forceinline__ void round_row(const Few& a, int m, uint8_t* xs, uint8_t* sx, int kpad) {
  const T* x = (const T*)a.x + m * a.ldx;
  const bool run16 = aligned16(x);
  constexpr int U = 16 / sizeof(T);
  for (int k0 = 0; k0 < kpad; k0 += 32 * kWarps * 16) {
    const int k = k0 + threadIdx.x * 16;
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = 0.f;
    if (run16 && k + 16 <= a.K) {
#pragma unroll
      for (int i = 0; i < 16; i += U) {
        float v[U];
        load_run(x + k + i, v);
#pragma unroll
        for (int j = 0; j < U; ++j) f[i + j] = v[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k + i < a.K) f[i] = to_f32(x[k + i]);
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(f[i]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (k < kpad) {
      const int b = scale_byte(amax, false);
      const float inv = inverse_scale(b);
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i / 4] |= to_f8(f[i], inv, false) << (8 * (i & 3));
      *reinterpret_cast<uint4*>(xs + (size_t)m * kpad + k) = make_uint4(w[0], w[1], w[2], w[3]);
      if (threadIdx.x % 8 == 0) sx[m * (kpad / 128) + k / 128] = (uint8_t)b;
    }
  }
}

template <int W5, int X5>
__global__ void __launch_bounds__(32 * kWarps, 3) fp8_few_kernel(const __grid_constant__ Few a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  const int kpad = (a.K + 127) / 128 * 128, blocks = kpad / 128;
  uint8_t* xs = dyn;                          // [M][kpad]
  uint8_t* sx = dyn + (size_t)a.M * kpad;     // [M][blocks]
  __shared__ float join[kWarps][kTile][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kTile;
  // this warp's blocks of K
  const int per = (blocks + kWarps - 1) / kWarps;
  const int b0 = min(blocks, warp * per), b1 = min(blocks, b0 + per);
  // this thread's rows of B (past the last one: the last one again, not stored)
  const int r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);
  const uint8_t* w0 = a.w + r0 * a.ldw + 16 * t;
  const uint8_t* w1 = a.w + r1 * a.ldw + 16 * t;
  const uint8_t* s0 = a.sw + (r0 >> a.wsh);
  const uint8_t* s1 = a.sw + (r1 >> a.wsh);

  wait_for_prior();  // (A and B may both come from the kernel before)
  uint4 v[kDepth][4];  // rows r0, r1 at k, then at k + 64
  int e[kDepth][2];
  auto fetch = [&](int b, uint4 (&q)[4], int (&s)[2]) {
    if (b >= b1) return;
    s[0] = s0[b * a.ldsw];
    s[1] = s1[b * a.ldsw];
    const int k = b * 128;
    if (k + 128 <= a.K) {
      q[0] = *reinterpret_cast<const uint4*>(w0 + k);
      q[1] = *reinterpret_cast<const uint4*>(w1 + k);
      q[2] = *reinterpret_cast<const uint4*>(w0 + k + 64);
      q[3] = *reinterpret_cast<const uint4*>(w1 + k + 64);
    } else {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
        if (k + 64 * h + 16 * t < a.K) {
          lo = load16(w0 + k + 64 * h, k + 64 * h + 16 * t, a.K);
          hi = load16(w1 + k + 64 * h, k + 64 * h + 16 * t, a.K);
        }
        if (h == 0)
          q[0] = lo, q[1] = hi;
        else
          q[2] = lo, q[3] = hi;
      }
    }
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) fetch(b0 + d, v[d], e[d]);

  if (a.xtype >= ROT_TYPE_E4M3) {
    for (int i = threadIdx.x; i < a.M * (kpad / 16); i += 32 * kWarps) {
      const int m = i / (kpad / 16), k = i % (kpad / 16) * 16;
      reinterpret_cast<uint4*>(xs)[i] =
          k < a.K ? load16((const uint8_t*)a.x + m * a.ldx + k, k, a.K) : make_uint4(0u, 0u, 0u, 0u);
    }
    for (int i = threadIdx.x; i < a.M * blocks; i += 32 * kWarps) {
      const int m = i / blocks, b = i - m * blocks;
      sx[i] = a.sx[b * a.ldsx + (m >> a.xsh)];
    }
  } else {
    for (int m = 0; m < a.M; ++m) {
      if (a.xtype == ROT_TYPE_F32)
        round_row<float>(a, m, xs, sx, kpad);
      else if (a.xtype == ROT_TYPE_F16)
        round_row<__half>(a, m, xs, sx, kpad);
      else
        round_row<__nv_bfloat16>(a, m, xs, sx, kpad);
    }
  }
  __syncthreads();

  // results: rows g and g + 8 of the tile, rows 2 t and 2 t + 1 of A
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const uint8_t* x0 = sx + min(2 * t, a.M - 1) * blocks;
  const uint8_t* x1 = sx + min(2 * t + 1, a.M - 1) * blocks;
  for (int bd = b0; bd < b1; bd += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int b = bd + d;
      if (b >= b1) break;  // (the same for the whole warp)
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (g < a.M)
          x = *reinterpret_cast<const uint4*>(xs + (size_t)g * kpad + b * 128 + 64 * h + 16 * t);
        const uint4 p = v[d][2 * h], q = v[d][2 * h + 1];
        mma16832<W5, X5>(c, p.x, q.x, p.y, q.y, x.x, x.y);
        mma16832<W5, X5>(c, p.z, q.z, p.w, q.w, x.z, x.w);
      }
      const int e0 = e[d][0], e1 = e[d][1];
      fetch(b + kDepth, v[d], e[d]);
      acc[0] += scaled(c[0], e0, x0[b]);
      acc[1] += scaled(c[1], e0, x1[b]);
      acc[2] += scaled(c[2], e1, x0[b]);
      acc[3] += scaled(c[3], e1, x1[b]);
    }
  }
  join[warp][g][2 * t] = acc[0];
  join[warp][g][2 * t + 1] = acc[1];
  join[warp][g + 8][2 * t] = acc[2];
  join[warp][g + 8][2 * t + 1] = acc[3];
  __syncthreads();
  const int r = threadIdx.x % kTile, m = threadIdx.x / kTile;
  if (m >= a.M || n0 + r >= a.N) return;
  float sum = 0.f;
#pragma unroll
  for (int q = 0; q < kWarps; ++q) sum += join[q][r][m];
  const int64_t o = m * a.ldy + n0 + r;
  if (a.ytype == ROT_TYPE_F32)
    ((float*)a.y)[o] = a.accumulate ? ((float*)a.y)[o] + sum : sum;
  else if (a.ytype == ROT_TYPE_F16)
    ((__half*)a.y)[o] = __float2half_rn(sum);
  else
    ((__nv_bfloat16*)a.y)[o] = __float2bfloat16_rn(sum);
}

template <int W5, int X5>
int launch_few(const Few& a, cudaStream_t s) {
  static const cudaError_t attr = cudaFuncSetAttribute(
      fp8_few_kernel<W5, X5>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
  if (attr != cudaSuccess) return ROT_ECUDA;
  const int kpad = (a.K + 127) / 128 * 128;
  const size_t smem = ((size_t)a.M * (kpad + kpad / 128) + 15) / 16 * 16;
  ProfScope prof(ROT_PROF_GEMM_F8, 2.0 * a.M * (double)a.N * a.K, s);
  return launch_behind(fp8_few_kernel<W5, X5>, (unsigned)((a.N + kTile - 1) / kTile), 32 * kWarps,
                       smem, s, a);
}

}  // namespace

// Where the kernel above takes a product: few rows, whose bytes fit shared
// memory.  With three to eight rows it is the faster of the two while B is
// small (4 rows, 2048 x 6144: 10 us against 13; 8 rows, 4096 x 12288: 28
// against 20, the rows' quantisation included).
bool fp8_few(int64_t M, int64_t N, int64_t K) {
  const int64_t kpad = (K + 127) / 128 * 128;
  return M <= kFewRows && M * (kpad + kpad / 128) + 15 <= kMaxShared &&
         (M <= kSelfRounded || N * K <= (16 << 20));
}
bool fp8_self_rounded(int64_t M, int64_t N, int64_t K) {
  return M <= kSelfRounded && fp8_few(M, N, K);
}

int fp8_few_product(const Prod& p, const void* x, int64_t ldx, int32_t xtype, cudaStream_t s) {
  Few a;
  a.w = p.b, a.sw = p.sb, a.x = x, a.sx = p.sa, a.y = p.c;
  a.ldw = p.ldb, a.ldsw = p.ldsb, a.ldx = ldx, a.ldsx = p.ldsa, a.ldy = p.ldc;
  a.M = p.M, a.N = p.N, a.K = p.K, a.xtype = xtype, a.ytype = p.ctype;
  a.wsh = p.bsh, a.xsh = p.ash, a.accumulate = p.accumulate;
  if (xtype == ROT_TYPE_E5M2) return p.b5 ? launch_few<1, 1>(a, s) : launch_few<0, 1>(a, s);
  return p.b5 ? launch_few<1, 0>(a, s) : launch_few<0, 0>(a, s);
}

}  // namespace ops
}  // namespace rot
