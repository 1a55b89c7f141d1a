// C = A B^T of 8-bit matrices with power-of-two block scales (rot_fp8_gemm) on
// the tensor cores: tcgen05 kind::mxf8f6f4, which multiplies each row's 32
// elements of K by a scale of one byte (UE8M0) as it reads them, so the scales
// cost nothing in the sums.
//
// Bound: the 8-bit tensor rate for large products.  A persistent kernel, one
// CTA per SM, walks the (tile, share of K) units of C.  Per CTA:
//   warp 0      one thread issues TMA loads of A (128 x 128 bytes) and B
//               (192 x 128 bytes) blocks into a five-deep ring
//   warp 1      allocates TMEM; one thread issues four MMAs of 128 x 192 x 32
//               per block, and every four blocks the copies of their scales to
//               TMEM (a cell holds four scales; the MMA names the one it takes)
//   warp 2      reads the scales and lays them out for those copies
//   warps 4-11  epilogue: each takes 32 rows x 96 columns
// 128 x 192 is the widest tile whose accumulator fits TMEM twice next to the
// scales, so that the epilogue overlaps the next tile's MMAs.
//
// Accuracy: the tensor cores truncate each partial sum they add to an
// accumulator, an error that grows with K.  An accumulator therefore takes at
// most 512 elements of K (16 additions); the epilogue adds these stretches in
// float32 registers.
//
// Few tiles: K is split over units whose float32 parts go to the workspace and
// are joined in a fixed order by a second kernel.
//
// Two products that do not wait for one another (a layer's gradients) are the
// units of one launch, the first one's and then the second one's, so that the
// second starts on the SMs that the first's last round leaves.
//
// 8192 x 12288 x 4096: 272 us, 3030 TFLOP/s; 6144 x 2048 x 4099 into float32:
// 49 us; with 4099 x 2048 x 6144 into bfloat16 in the same launch 82 us, 101 in
// two.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "ops_common.cuh"
#include "ops_fp8.h"
#include "profile.h"
#include "tc_ptx.cuh"

namespace rot {
namespace ops {
namespace {

constexpr int BM = 128, BN = 192, BK = 128;
constexpr int kStages = 5;
constexpr int kABytes = BM * BK, kBBytes = BN * BK, kStageBytes = kABytes + kBBytes;
constexpr int kScaleBytes = 512 + 1024;  // a stretch's: A's 128 rows, B's 192 (of 256)
constexpr int kSlots = 3;                // stretches of scales on their way
// Two barriers of arrival per stage, taken in turn: an issuing warp passes over
// the other's stretches without waiting, and a barrier tells only the last
// phase from the one before.  With one per stage a warp could reach a stage
// whose last load, the other warp's, had not arrived yet, and take it for its
// own.  When it waits for block x, its last own block is x - 5 or later, whose
// load was issued after block x - 10, the barrier's last use, was consumed.
constexpr int kFulls = 2 * kStages;
static_assert(kStages >= 5, "a warp's blocks are at most a stretch and one apart");
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8, kEpiCols = BN / 2;
constexpr int kStagingBytes = 32 * 64;  // per epilogue warp
constexpr int kSmem =
    1024 + kStages * kStageBytes + kSlots * kScaleBytes + kEpiWarps * kStagingBytes + 256;
static_assert(kSmem <= 232448, "dynamic shared memory above 227 KB");
constexpr int kStretch = 4;     // K blocks an accumulator takes, and a cell of scales holds
constexpr int kScaleCols = 12;  // TMEM columns of a stretch's scales: 4 of A, 8 of B
constexpr int kTmemCols = 512;
static_assert(2 * BN + kSlots * kScaleCols <= kTmemCols, "TMEM");

struct Part {
  CUtensorMap a, b;
  Prod p;
  int tiles_m, tiles_n, kblocks, splits, per;  // per: K blocks of a unit
  int units;
  void* c;  // C, or with split K the parts (float32)
  int64_t ldc;
  int accumulate;
};
// The products of one launch: the first one's units come first.
template <int N>
struct Mx {
  Part part[N];
  int units;
  int* status;
  unsigned long long limit_ns;
};

// Units in order: shares of a tile next to each other, tiles in groups of
// kGroupM rows of tiles, down a group's columns, so that the CTAs at work at
// any time share blocks of A and B in L2.  (16 rows of tiles by 9 or 10
// columns at once are nearly square in bytes: 8192 cubed in 349 us, against 369
// and 371 with groups of 8 and 4.)
constexpr int kGroupM = 16;

struct Unit {
  int m0, n0, k0, k1, split, which;  // which: the product
};
template <int N>
__device__ __forceinline__ Unit unit_of(const Mx<N>& all, int u) {
  Unit t;
  t.which = N > 1 && u >= all.part[0].units;
  if (t.which) u -= all.part[0].units;
  const Part& g = all.part[t.which];
  const int tile = u / g.splits;
  const int per_group = kGroupM * g.tiles_n;
  const int grp = tile / per_group, r = tile - grp * per_group;
  const int h = min(kGroupM, g.tiles_m - grp * kGroupM);
  t.split = u - tile * g.splits;
  t.m0 = (grp * kGroupM + r % h) * BM;
  t.n0 = r / h * BN;
  t.k0 = t.split * g.per;
  t.k1 = min(g.kblocks, t.k0 + g.per);
  return t;
}

// Bounded wait (ptx::mbar_wait) that looks at the clock only after a while:
// the usual wait is short, and reading the timer is not.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                     uint64_t limit_ns) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (ptx::mbar_try_wait(bar, parity)) return true;
  return ptx::mbar_wait(bar, parity, abort, limit_ns);
}

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  limit_ns = limit_ns > 100000000ull ? limit_ns : 100000000ull;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 0;; ++it) {
    if (ptx::mbar_try_wait(bar, parity)) return;
    if ((it & 63u) == 0u && (ptx::globaltimer_ns() - t0 > limit_ns || it > (1u << 30))) return;
  }
}

// The scales that a lane lays out for a stretch: rows lane, 32 + lane, .. of
// A's four groups and B's six, in its four K blocks.  Rows past the last one
// and blocks past k1 take the last one's: nothing of theirs is used, and no
// load waits for another's condition.
struct Scales {
  uint32_t v[10][kStretch];
};
__device__ __forceinline__ void load_scales(const Prod& p, const Unit& t, int kb, int lane,
                                            Scales& s) {
#pragma unroll
  for (int c = 0; c < 10; ++c) {
    const bool a = c < 4;
    const int r = min((a ? t.m0 + 32 * c : t.n0 + 32 * (c - 4)) + lane, (a ? p.M : p.N) - 1);
    const uint8_t* q = a ? p.sa + (r >> p.ash) : p.sb + (r >> p.bsh);
    const int64_t ld = a ? p.ldsa : p.ldsb;
#pragma unroll
    for (int j = 0; j < kStretch; ++j) s.v[c][j] = q[min(kb + j, t.k1 - 1) * ld];
  }
}

// A warp's 32 rows of C, 64 bytes of each (64 / sizeof(T) columns), of which
// this thread holds row `lane`: staged in 2 KB of shared memory, so that the
// warp then stores eight whole 64-byte pieces of rows at a time (one row per
// thread would store 16 bytes of 32 rows).  16-byte piece c of row r is at
// place c ^ (r / 2 & 3) of the row: neither side has bank conflicts.
template <class T>
__device__ __forceinline__ void stage_rows(uint8_t* stage, const float* v) {
  constexpr int U = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[U];
#pragma unroll
    for (int k = 0; k < U; ++k) f[k] = v[i * U + k];
    store_run(reinterpret_cast<T*>(stage + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)), f);
  }
  __syncwarp();
}

// Rows that are cut, not 16-byte aligned or added to: element by element, a
// row's columns side by side, eight steps' loads before their stores (one by
// one, 9547 x 1285 x 3418 into float32 took 88 us; so it takes 71).
template <class T>
__device__ __noinline__ void store_any(const uint8_t* stage, T* c, int64_t ldc, int rows, int cols,
                                       bool accumulate) {
  constexpr int W = 64 / sizeof(T), U = 16 / sizeof(T), kRows = 32 / W, kBatch = 8;
  const int lane = threadIdx.x & 31, k = lane % W;
  if (k >= cols) rows = 0;  // (no early return: the warp stays together)
  c += lane / W * ldc + k;
#pragma unroll 1
  for (int b = 0; b < W; b += kBatch) {
    T x[kBatch];
    float old[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = (b + j) * kRows + lane / W;
      x[j] = *reinterpret_cast<const T*>(stage + r * 64 + (((k / U) ^ (r >> 1 & 3)) << 4) +
                                         k % U * sizeof(T));
      old[j] = accumulate && r < rows ? to_f32(c[(b + j) * kRows * ldc]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if ((b + j) * kRows + lane / W < rows)
        c[(b + j) * kRows * ldc] = accumulate ? from_f32<T>(old[j] + to_f32(x[j])) : x[j];
  }
}

// A warp's 32 rows and kEpiCols columns from c on, cut to rows x cols.
template <class T>
__device__ __forceinline__ void store_tile(uint8_t* stage, T* c, int64_t ldc, int rows, int cols,
                                           const float* sum, bool accumulate) {
  constexpr int W = 64 / sizeof(T);
  const int lane = threadIdx.x & 31, r = lane >> 2, i = lane & 3;
  const bool whole = rows >= 32 && rows16(c, ldc, sizeof(T)) && !accumulate;
  const uint4* from = reinterpret_cast<const uint4*>(stage + r * 64 + ((i ^ (r >> 1 & 3)) << 4));
  uint8_t* to = reinterpret_cast<uint8_t*>(c + r * ldc) + 16 * i;
#pragma unroll
  for (int n = 0; n < kEpiCols; n += W) {
    if (n >= cols) break;
    stage_rows<T>(stage, sum + n);
    if (whole && n + W <= cols) {
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = from[q * 32];  // rows 8 q + r
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(to + (8 * q * ldc + n) * (int64_t)sizeof(T)) = v[q];
    } else {
      store_any(stage, c + n, ldc, rows, cols - n, accumulate);
    }
  }
  // the warp's next TMEM load wants all its lanes at once
  __syncwarp();
}

// C of type T, a second product's of float32.
template <class T, int N>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Mx<N> g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* scales = smem + kStages * kStageBytes;
  uint8_t* staging = scales + kSlots * kScaleBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kStagingBytes);
  uint64_t* empty = full + kFulls;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* sfull = tempty + 2;
  uint64_t* sempty = sfull + kSlots;
  uint64_t* done = sempty + kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // (the same in every lane, and known to be)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint64_t limit = g.limit_ns;
  auto ready = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity, abort_flag, limit)) != 0;
  };
  // The waits of each block leave a timeout to `aborted`, once per stretch:
  // once the flag is up, every wait returns after its first tries.
  auto aborted = [&] { return __any_sync(0xffffffffu, *abort_flag) != 0; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFulls; ++s) ptx::mbar_init(&full[s], 1);
    for (int s = 0; s < kStages; ++s) ptx::mbar_init(&empty[s], 1);
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tfull[a], 1);
      ptx::mbar_init(&tempty[a], kEpiWarps);
    }
    for (int s = 0; s < kSlots; ++s) {
      ptx::mbar_init(&sfull[s], 1);
      ptx::mbar_init(&sempty[s], 1);
    }
    ptx::mbar_init(&done[0], 1);
    ptx::mbar_init(&done[1], 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  wait_for_prior();  // (the operands may come from the kernel before)

  // Warps 0 and 1 run their loops as a whole, with one lane's copies and MMAs
  // in between: operands and addresses stay in uniform registers.  From a
  // branch on the lane number the issue of a block's four MMAs took 570 cycles,
  // half as long again as the MMAs.
  if (warp == 0) {
    // ------------------------------------------------------------ loads
    const bool one = ptx::elect_one();
    if (one) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ptx::tma_prefetch_desc(&g.part[i].a);
        ptx::tma_prefetch_desc(&g.part[i].b);
      }
    }
    int turn = 0;  // block mod kFulls
    uint32_t phase = 0, armed = 0, armed_parity = 0;  // phase: of full[turn]
    for (int u = blockIdx.x; u < g.units; u += gridDim.x) {
      const Unit t = unit_of(g, u);
      const Part& q = g.part[t.which];
      int kb = t.k0;
      while (kb < t.k1 && !aborted()) {
        const int k1 = min(t.k1, kb + kStretch);
        for (; kb < k1; ++kb) {
          // (a stage's uses alternate with the two halves of the turns)
          const int stage = turn < kStages ? turn : turn - kStages;
          wait(&empty[stage], turn < kStages ? 1u : 0u, abort_flag, limit);
          if (*abort_flag) break;  // (the stage may still be read)
          uint8_t* st = smem + stage * kStageBytes;
          if (one) {
            ptx::mbar_arrive_expect_tx(&full[turn], kStageBytes);
            ptx::tma_load_2d(st, &q.a, &full[turn], kb * BK, t.m0);
            ptx::tma_load_2d(st + kABytes, &q.b, &full[turn], kb * BK, t.n0);
          }
          armed |= 1u << turn;
          armed_parity = (armed_parity & ~(1u << turn)) | (phase << turn);
          if (++turn == kFulls) {
            turn = 0;
            phase ^= 1u;
          }
        }
      }
      if (kb < t.k1) break;
    }
    __syncwarp();
    for (int s = 0; s < kFulls; ++s)
      if (armed & (1u << s)) drain(&full[s], (armed_parity >> s) & 1u, limit);
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issue
    // Warp 1 takes the even stretches, warp 3 the odd ones, each with its own
    // accumulator: the issue of a block takes one warp longer than its MMAs.
    const int odd = warp >> 1;
    const bool one = ptx::elect_one();
    int block = 0, turn = 0, slot = 0;  // block: mod kFulls; phase: of full[block]
    uint32_t phase = 0, acc_phase = 0, slot_phase = 0;
    bool ok = true;
    const uint32_t d = tmem + (uint32_t)(odd * BN);
    for (int u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
      const Unit t = unit_of(g, u);
      const uint32_t idesc =
          ptx::idesc_mxf8(BM, BN, g.part[t.which].p.a5, g.part[t.which].p.b5);
      for (int kb = t.k0; kb < t.k1; kb += kStretch) {
        const int n = min(t.k1 - kb, kStretch);
        if (turn == odd) {
          wait(&sfull[slot], slot_phase, abort_flag, limit);
          wait(&tempty[odd], acc_phase ^ 1u, abort_flag, limit);
          ok = !aborted();
          if (!ok) break;
          ptx::tc_fence_after();
          // (copies and MMAs run in the order of issue)
          const uint32_t sc = ptx::smem_u32(scales + slot * kScaleBytes);
          const uint32_t sfa = tmem + (uint32_t)(2 * BN + slot * kScaleCols), sfb = sfa + 4;
          if (one) {
            ptx::tmem_cp_32x128b_x4(sfa, ptx::rows16_desc(sc));
            ptx::tmem_cp_32x128b_x4(sfb, ptx::rows16_desc(sc + 512));
            ptx::tmem_cp_32x128b_x4(sfb + 4, ptx::rows16_desc(sc + 1024));
          }
#pragma unroll
          for (int j = 0; j < kStretch; ++j) {
            if (j >= n) break;
            const int stage = block < kStages ? block : block - kStages;
            wait(&full[block], phase, abort_flag, limit);
            ptx::tc_fence_after();
            const uint32_t st = ptx::smem_u32(smem + stage * kStageBytes);
            const uint64_t da = ptx::sw128_kmajor_desc(st);
            const uint64_t db = ptx::sw128_kmajor_desc(st + kABytes);
            const uint32_t id = ptx::idesc_scales(idesc, j, j);
            if (one) {
#pragma unroll
              for (int i = 0; i < BK / 32; ++i)
                ptx::umma_mxf8(d, da + (uint64_t)(2 * i), db + (uint64_t)(2 * i), id, sfa, sfb,
                               (j > 0 || i > 0) ? 1u : 0u);
              ptx::umma_commit(&empty[stage]);
            }
            if (++block == kFulls) {
              block = 0;
              phase ^= 1u;
            }
          }
          if (one) {
            ptx::umma_commit(&tfull[odd]);
            ptx::umma_commit(&sempty[slot]);
          }
          acc_phase ^= 1u;
        } else {
          block += n;
          if (block >= kFulls) {
            block -= kFulls;
            phase ^= 1u;
          }
        }
        turn ^= 1;
        if (++slot == kSlots) {
          slot = 0;
          slot_phase ^= 1u;
        }
      }
    }
    if (one) ptx::umma_commit(&done[odd]);
    __syncwarp();
    drain(&done[odd], 0, limit);
  } else if (warp == 2) {
    // ------------------------------------------------------------ scales
    // A word per row, with the scales of the stretch's four K blocks, which
    // tcgen05.cp puts into lane l, column c for row 32 c + l.  The next
    // stretch's bytes are on their way while this one's are laid out.
    int slot = 0;
    uint32_t phase = 0;
    int u = blockIdx.x, kb;
    Unit t;
    Scales s;
    if (u < g.units) {
      t = unit_of(g, u);
      kb = t.k0;
      load_scales(g.part[t.which].p, t, kb, lane, s);
    }
    while (u < g.units) {
      uint32_t w[10];
#pragma unroll
      for (int c = 0; c < 10; ++c)
        w[c] = s.v[c][0] | s.v[c][1] << 8 | s.v[c][2] << 16 | s.v[c][3] << 24;
      kb += kStretch;
      if (kb >= t.k1) {
        u += gridDim.x;
        if (u < g.units) {
          t = unit_of(g, u);
          kb = t.k0;
        }
      }
      if (u < g.units) load_scales(g.part[t.which].p, t, kb, lane, s);
      if (!ready(&sempty[slot], phase ^ 1u)) break;
      uint4* q = reinterpret_cast<uint4*>(scales + slot * kScaleBytes);
      q[lane] = make_uint4(w[0], w[1], w[2], w[3]);
      q[32 + lane] = make_uint4(w[4], w[5], w[6], w[7]);
      q[64 + lane] = make_uint4(w[8], w[9], 0x7F7F7F7Fu, 0x7F7F7F7Fu);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sfull[slot]);
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * kEpiCols);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < g.units; u += gridDim.x) {
      const Unit t = unit_of(g, u);
      float sum[kEpiCols];
#pragma unroll
      for (int c = 0; c < kEpiCols; ++c) sum[c] = 0.f;
      for (int kb = t.k0; kb < t.k1; kb += kStretch) {
        if (!ready(&tfull[acc], acc_phase)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kEpiCols; c += 32) {
          uint32_t r[32];
          ptx::tmem_ld_32x32b_x32(lanes + (uint32_t)(acc * BN + c), r);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c + i] += __uint_as_float(r[i]);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&tempty[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      const Part& q = g.part[t.which];
      const int row = t.m0 + quarter * 32, n0 = t.n0 + half * kEpiCols;
      const int rows = q.p.M - row, cols = q.p.N - n0;
      if (!ok || rows <= 0 || cols <= 0) continue;
      uint8_t* stage = staging + (warp - 4) * kStagingBytes;
      const int64_t at = ((int64_t)t.split * q.p.M + row) * q.ldc + n0;
      if (N == 1 || std::is_same<T, float>::value || t.which == 0)
        store_tile(stage, static_cast<T*>(q.c) + at, q.ldc, rows, cols, sum, q.accumulate);
      else
        store_tile(stage, static_cast<float*>(q.c) + at, q.ldc, rows, cols, sum, q.accumulate);
    }
  }

  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag && g.status) atomicExch(g.status, ROT_ETIMEOUT);
}

// C from the parts, added in order of K.
__global__ void __launch_bounds__(256) fp8_join_kernel(const Prod p, int splits, int64_t ldp) {
  const int64_t total = (int64_t)p.M * p.N;
  wait_for_prior();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / p.N, n = i - m * p.N;
    float sum = 0.f;
    for (int s = 0; s < splits; ++s) sum += p.part[((int64_t)s * p.M + m) * ldp + n];
    const int64_t o = m * p.ldc + n;
    if (p.ctype == ROT_TYPE_F32)
      ((float*)p.c)[o] = p.accumulate ? ((float*)p.c)[o] + sum : sum;
    else if (p.ctype == ROT_TYPE_F16)
      ((__half*)p.c)[o] = __float2half_rn(sum);
    else
      ((__nv_bfloat16*)p.c)[o] = __float2bfloat16_rn(sum);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Shares of K for a product of `tiles` tiles: enough units for the 152 SMs
// while each keeps at least one stretch of K (the workspace's size must not
// depend on the GPU at hand).
constexpr int kSms = 152;

struct Shape {
  int64_t tiles_m, tiles_n, kblocks, splits, per, ldp;
};
Shape shape_of(int64_t M, int64_t N, int64_t K) {
  Shape s;
  s.tiles_m = (M + BM - 1) / BM;
  s.tiles_n = (N + BN - 1) / BN;
  s.kblocks = (K + BK - 1) / BK;
  const int64_t tiles = s.tiles_m * s.tiles_n;
  const int64_t most = (s.kblocks + kStretch - 1) / kStretch;
  const int64_t splits = std::max<int64_t>(1, std::min(most, kSms / std::max<int64_t>(tiles, 1)));
  // whole stretches per share
  s.per = (most + splits - 1) / splits * kStretch;
  s.splits = (s.kblocks + s.per - 1) / s.per;
  s.ldp = (N + 3) / 4 * 4;
  return s;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// rows x K bytes at a pitch of ld, boxes of box_rows x 128 with the 128-byte
// swizzle; bytes past K or past the last row read as 0.
int encode(CUtensorMap* map, const uint8_t* base, int64_t rows, int64_t K, int64_t ld,
           int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {(cuuint32_t)BK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base),
                               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ROT_OK : ROT_EINVAL;
}

template <class T, int N>
int launch_gemm(const Mx<N>& g, cudaStream_t stream) {
  static const cudaError_t attr = cudaFuncSetAttribute(
      fp8_gemm_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (attr != cudaSuccess) return ROT_ECUDA;
  double flops = 0.0;
  for (const Part& q : g.part) flops += 2.0 * q.p.M * (double)q.p.N * q.p.K;
  ProfScope prof(ROT_PROF_GEMM_F8, flops, stream);
  return launch_behind(fp8_gemm_kernel<T, N>, (unsigned)std::min(g.units, sm_count()), kThreads,
                       kSmem, stream, g);
}
// ctype: the first product's.
template <int N>
int launch_gemm(const Mx<N>& g, int ctype, cudaStream_t stream) {
  if (ctype == ROT_TYPE_F32) return launch_gemm<float, N>(g, stream);
  if (ctype == ROT_TYPE_F16) return launch_gemm<__half, N>(g, stream);
  return launch_gemm<__nv_bfloat16, N>(g, stream);
}

// A product's part of a launch.
int part_of(const Prod& p, const Shape& s, Part* g) {
  if (!encoder()) return ROT_ECUDA;
  if (s.tiles_m * s.tiles_n * s.splits > 0x7FFFFFFF) return ROT_EINVAL;  // (C beyond any memory)
  int e = encode(&g->a, p.a, p.M, p.K, p.lda, BM);
  if (e == ROT_OK) e = encode(&g->b, p.b, p.N, p.K, p.ldb, BN);
  if (e != ROT_OK) return e;
  g->p = p;
  g->tiles_m = (int)s.tiles_m, g->tiles_n = (int)s.tiles_n, g->kblocks = (int)s.kblocks;
  g->splits = (int)s.splits, g->per = (int)s.per;
  g->units = (int)(s.tiles_m * s.tiles_n * s.splits);
  const bool parts = s.splits > 1;
  g->c = parts ? p.part : p.c, g->ldc = parts ? s.ldp : p.ldc;
  g->accumulate = !parts && p.accumulate;
  return ROT_OK;
}

}  // namespace

uint64_t fp8_work_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  const Shape s = shape_of(M, N, K);
  return s.splits > 1 ? align256(4ull * s.splits * M * s.ldp) : 0;
}

int fp8_product(const Prod& p, int* status, cudaStream_t stream) {
  const Shape s = shape_of(p.M, p.N, p.K);
  Mx<1> g;
  int e = part_of(p, s, &g.part[0]);
  if (e != ROT_OK) return e;
  const bool parts = s.splits > 1;
  g.units = g.part[0].units, g.status = status, g.limit_ns = g_wait_limit_ns;
  e = launch_gemm(g, parts ? ROT_TYPE_F32 : p.ctype, stream);
  if (e != ROT_OK || !parts) return e;
  ProfScope prof(ROT_PROF_ELEMENTWISE, 4.0 * (s.splits + 1) * p.M * (double)p.N, stream);
  const int64_t blocks = ((int64_t)p.M * p.N + 255) / 256;
  return launch_behind(fp8_join_kernel, (unsigned)std::min<int64_t>(blocks, 8ll * sm_count()), 256, 0,
                       stream, p, (int)s.splits, s.ldp);
}

bool fp8_takes_two(int64_t M0, int64_t N0, int64_t K0, int64_t M1, int64_t N1, int64_t K1) {
  if (std::min({M0, N0, K0, M1, N1, K1}) <= 0 || fp8_few(M0, N0, K0) || fp8_few(M1, N1, K1))
    return false;
  const Shape s = shape_of(M0, N0, K0), t = shape_of(M1, N1, K1);
  return s.splits == 1 && t.splits == 1 &&
         s.tiles_m * s.tiles_n + t.tiles_m * t.tiles_n <= 0x7FFFFFFF;
}

int fp8_two_products(const Prod& p, const Prod& q, int* status, cudaStream_t stream) {
  Mx<2> g;
  int e = part_of(p, shape_of(p.M, p.N, p.K), &g.part[0]);
  if (e == ROT_OK) e = part_of(q, shape_of(q.M, q.N, q.K), &g.part[1]);
  if (e != ROT_OK) return e;
  g.units = g.part[0].units + g.part[1].units;
  g.status = status, g.limit_ns = g_wait_limit_ns;
  return launch_gemm(g, p.ctype, stream);
}

}  // namespace ops
}  // namespace rot
