// Entry points of the heads' operators (include/rot_ops.h), the rotation
// alone, and the join of the weights' gradients.
#include <cmath>

#include "ops_heads.cuh"

namespace rot {
namespace ops {

int heads_rotate(int32_t type, HeadArgs& q, int64_t tokens, bool il, cudaStream_t s) {
  return launch_heads_type<kRotate>(type, q, tokens, il, s);
}

namespace {

// The weights' gradients: the blocks' parts, 32 columns by 32 strided shares
// per block, joined in a fixed order.
__global__ void __launch_bounds__(1024) heads_join_kernel(const float* part, int parts, int dim,
                                                          float* dw0, float* dw1) {
  __shared__ float share[32][33];
  wait_for_prior();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = (dim + 31) / 32, second = blockIdx.x >= blocks;
  const int base = (blockIdx.x - second * blocks) * 32;
  float sum = 0.f;
  if (base + lane < dim)
    for (int p = warp; p < parts; p += 32)
      sum += part[((int64_t)p * 2 + second) * dim + base + lane];
  share[warp][lane] = sum;
  __syncthreads();
  sum = warp_sum(share[lane][warp]);  // column `warp` of this block
  if (lane == 0 && base + warp < dim) (second ? dw1 : dw0)[base + warp] = sum;
}

// An array of heads to write: its rows do not overlap.  (Strides in order of
// size: each one reaches past all that the smaller ones span.)
bool bad_out(const rot_heads* h, int64_t batch, int64_t tokens, int64_t dim) {
  std::pair<int64_t, int64_t> d[3] = {
      {h->batch_stride, batch}, {h->token_stride, tokens}, {h->head_stride, h->heads}};
  std::sort(d, d + 3);
  int64_t span = dim;
  for (const auto& [stride, size] : d) {
    if (size <= 1) continue;
    if (stride < span) return true;
    if (stride > (int64_t(1) << 48) / size) return true;
    span = stride * (size - 1) + span;
  }
  return false;
}
bool bad_in(const rot_heads* h, int64_t batch, int64_t tokens) {
  const int64_t most = int64_t(1) << 48;
  return !h || h->heads < 0 || h->heads > 65536 || h->batch_stride < 0 || h->token_stride < 0 ||
         h->head_stride < 0 || (batch > 1 && h->batch_stride > most / batch) ||
         (tokens > 1 && h->token_stride > most / tokens) ||
         (h->heads > 1 && h->head_stride > most / h->heads);
}
HeadStrides strides(const rot_heads* h) { return {h->batch_stride, h->token_stride, h->head_stride}; }

bool misaligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes; }

struct Given {
  const rot_heads *x, *dy, *out;
  const void* w;
};

// The checks that all entry points share; fills `a`.  grad: dy is there.
int set_up(HeadArgs& a, const Given (&g)[2], int64_t batch, int64_t tokens, int64_t dim,
           int32_t type, const rot_rotary* r, bool inverse, bool norm, bool grad) {
  if (batch < 0 || tokens < 0 || (batch > 0 && tokens > (1 << 30) / batch)) return ROT_EINVAL;
  if (dim < 1 || dim > ROT_MAX_HEAD_DIM || !float_type(type)) return ROT_EINVAL;
  a.dim = (int)dim, a.tokens = (uint32_t)std::max<int64_t>(tokens, 1);
  const int64_t es = type_bytes(type);
  for (int i = 0; i < 2; ++i) {
    const Given& v = g[i];
    if (i == 1 && !v.x && !v.out && !v.dy && !v.w) continue;
    if (bad_in(v.x, batch, tokens) || !v.out || bad_in(v.out, batch, tokens) ||
        v.out->heads != v.x->heads || bad_out(v.out, batch, tokens, dim))
      return ROT_EINVAL;
    if (grad && (bad_in(v.dy, batch, tokens) || v.dy->heads != v.x->heads)) return ROT_EINVAL;
    const bool some = batch * tokens > 0 && v.x->heads > 0;
    if (norm && !v.w && (some || grad)) return ROT_EINVAL;
    if (some) {
      const void* all[3] = {v.x->data, v.out->data, grad ? v.dy->data : v.x->data};
      for (const void* p : all)
        if (!p || misaligned(p, es)) return ROT_EINVAL;
    }
    HeadSide& sd = a.side[i];
    sd.x = v.x->data, sd.xs = strides(v.x);
    sd.out = v.out->data, sd.os = strides(v.out);
    if (grad) sd.dy = v.dy->data, sd.ds = strides(v.dy);
    sd.w = v.w;
    sd.heads = some ? (int32_t)v.x->heads : 0;
  }
  if (!r) return ROT_OK;
  if (r->rotated < 0 || r->rotated > dim || r->rotated % 2 || std::isnan(r->magnitude) ||
      (r->rotated > 0 && !r->turns) || misaligned(r->turns, 8))
    return ROT_EINVAL;
  if (r->positions && ((r->position_bytes != 4 && r->position_bytes != 8) ||
                       misaligned(r->positions, r->position_bytes) ||
                       r->position_batch_stride < 0 || r->position_token_stride < 0))
    return ROT_EINVAL;
  a.rotated = (int)r->rotated, a.turns = r->turns;
  a.positions = r->positions, a.position_bytes = r->position_bytes;
  a.pbs = r->position_batch_stride, a.pts = r->position_token_stride, a.start = r->start;
  a.cos_scale = r->magnitude, a.sin_scale = inverse ? -r->magnitude : r->magnitude;
  return ROT_OK;
}

// Bytes that a call moves.
double moved(const HeadArgs& a, int64_t tokens, int32_t type, int arrays) {
  return (double)tokens * (a.side[0].heads + a.side[1].heads) * a.dim * type_bytes(type) * arrays;
}

}  // namespace
}  // namespace ops
}  // namespace rot

using namespace rot;
using namespace rot::ops;

extern "C" {

int rot_rotate(const rot_heads* q, const rot_heads* q_out, const rot_heads* k,
               const rot_heads* k_out, int64_t batch, int64_t tokens, int64_t dim, int32_t type,
               const rot_rotary* rotary, int32_t inverse, void* stream) {
  HeadArgs a;
  if (!rotary) return ROT_EINVAL;
  const int e = set_up(a, {{q, nullptr, q_out, nullptr}, {k, nullptr, k_out, nullptr}}, batch,
                       tokens, dim, type, rotary, inverse != 0, false, false);
  if (e != ROT_OK) return e;
  if (!a.side[0].heads && !a.side[1].heads) return ROT_OK;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  return guarded([&] {
    ProfScope prof(ROT_PROF_ELEMENTWISE, moved(a, batch * tokens, type, 2),
                   static_cast<cudaStream_t>(stream));
    return heads_rotate(type, a, batch * tokens, rotary->interleaved != 0,
                        static_cast<cudaStream_t>(stream));
  });
}

int rot_head_norm_forward(const rot_heads* q, const void* q_weight, const rot_heads* q_out,
                          const rot_heads* k, const void* k_weight, const rot_heads* k_out,
                          int32_t wtype, int64_t batch, int64_t tokens, int64_t dim, int32_t type,
                          float eps, const rot_rotary* rotary, void* stream) {
  HeadArgs a;
  if ((wtype != ROT_TYPE_F32 && wtype != type) || !(eps >= 0.f) ||
      misaligned(q_weight, type_bytes(wtype)) || misaligned(k_weight, type_bytes(wtype)))
    return ROT_EINVAL;
  const int e = set_up(a, {{q, nullptr, q_out, q_weight}, {k, nullptr, k_out, k_weight}}, batch,
                       tokens, dim, type, rotary, false, true, false);
  if (e != ROT_OK) return e;
  if (!a.side[0].heads && !a.side[1].heads) return ROT_OK;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  a.w32 = wtype == ROT_TYPE_F32, a.eps = eps;
  return guarded([&] {
    ProfScope prof(ROT_PROF_ELEMENTWISE, moved(a, batch * tokens, type, 2),
                   static_cast<cudaStream_t>(stream));
    return heads_norm(type, a, batch * tokens, rotary && rotary->interleaved,
                      static_cast<cudaStream_t>(stream));
  });
}

uint64_t rot_head_norm_work_bytes(int64_t dim) {
  if (dim < 1 || dim > ROT_MAX_HEAD_DIM) return 0;
  return align256(8ull * (uint64_t)dim * kHeadParts);
}

int rot_head_norm_backward(const rot_heads* dq, const rot_heads* q, const void* q_weight,
                           const rot_heads* dq_out, float* dq_weight, const rot_heads* dk,
                           const rot_heads* k, const void* k_weight, const rot_heads* dk_out,
                           float* dk_weight, int32_t wtype, int64_t batch, int64_t tokens,
                           int64_t dim, int32_t type, float eps, const rot_rotary* rotary,
                           void* work, uint64_t work_bytes, void* stream) {
  HeadArgs a;
  if ((wtype != ROT_TYPE_F32 && wtype != type) || !(eps >= 0.f) ||
      misaligned(q_weight, type_bytes(wtype)) || misaligned(k_weight, type_bytes(wtype)) ||
      misaligned(dq_weight, 4) || misaligned(dk_weight, 4))
    return ROT_EINVAL;
  const int e = set_up(a, {{q, dq, dq_out, q_weight}, {k, dk, dk_out, k_weight}}, batch, tokens,
                       dim, type, rotary, true, true, true);
  if (e != ROT_OK) return e;
  if (!dq_weight || (k && !dk_weight) || (!k && dk_weight)) return ROT_EINVAL;
  if (!work || (reinterpret_cast<uintptr_t>(work) & 255) ||
      work_bytes < rot_head_norm_work_bytes(dim))
    return ROT_EINVAL;
  const int dev = check_device();
  if (dev != ROT_OK) return dev;
  a.w32 = wtype == ROT_TYPE_F32, a.eps = eps, a.part = static_cast<float*>(work);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return guarded([&] {
    a.blocks = 0;
    if (a.side[0].heads || a.side[1].heads) {
      ProfScope prof(ROT_PROF_ELEMENTWISE, moved(a, batch * tokens, type, 3), s);
      const int code = heads_norm_grad(type, a, batch * tokens, rotary && rotary->interleaved, s);
      if (code != ROT_OK) return code;
    }
    ProfScope prof(ROT_PROF_ELEMENTWISE, 0.0, s);
    return launch_behind(heads_join_kernel, ((int)dim + 31) / 32 * (k ? 2 : 1), 1024, 0, s,
                         (const float*)a.part, (int)a.blocks, (int)dim, dq_weight, dk_weight);
  });
}

}  // extern "C"
