// The operators on torch tensors (operators.py): checks of the tensors,
// outputs and workspaces from torch's allocator, and the call into librot on
// the current stream.  No arithmetic.
//
// A call of a small operator is host time alone: a layer norm of one token
// takes 8 us here, four allocations and a launch among them, and took 29 with
// the same checks in Python and the call through ctypes.
//
// The library's entry points come as addresses (bind), so that the one library
// the process has loaded is the one that runs.
#include <ATen/ATen.h>
#include <ATen/MemoryOverlap.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <tuple>

#include "rot_ops.h"

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

namespace {

#define ROT_ENTRIES(X)        \
  X(rot_dropout)              \
  X(rot_layer_norm_forward)   \
  X(rot_layer_norm_work_bytes) \
  X(rot_layer_norm_backward)  \
  X(rot_token_logprobs)       \
  X(rot_policy_loss)          \
  X(rot_fp8_quantize)         \
  X(rot_fp8_gemm_work_bytes)  \
  X(rot_fp8_gemm)             \
  X(rot_fp8_linear_work_bytes) \
  X(rot_fp8_linear)           \
  X(rot_fp8_linear_backward_work_bytes) \
  X(rot_fp8_linear_backward)  \
  X(rot_rotate)               \
  X(rot_head_norm_forward)    \
  X(rot_head_norm_work_bytes) \
  X(rot_head_norm_backward)   \
  X(rot_adamw_step)           \
  X(rot_adamw_step_counted)   \
  X(rot_gradient_norm_work_bytes) \
  X(rot_gradient_norm)

struct Entries {
#define X(name) decltype(&::name) name = nullptr;
  ROT_ENTRIES(X)
#undef X
} lib;
PyObject* rot_error = nullptr;  // binding.RotError

void check(int code, const char* where) {
  if (code == ROT_OK) return;
  PyErr_SetObject(rot_error, py::make_tuple(code, where).ptr());
  throw py::error_already_set();
}

[[noreturn]] void fail(const std::string& what) { throw py::value_error(what); }

int type_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return ROT_TYPE_F32;
    case at::kHalf: return ROT_TYPE_F16;
    case at::kBFloat16: return ROT_TYPE_BF16;
    default: return -1;
  }
}
int format_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat8_e4m3fn: return ROT_TYPE_E4M3;
    case at::kFloat8_e5m2: return ROT_TYPE_E5M2;
    default: return -1;
  }
}

// A tensor as rows of its last dimension: leading dimensions fold into the
// rows.
struct Rows {
  void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
};

Rows rows_of(const Tensor& t, const char* name, const Tensor* like = nullptr) {
  const std::string n = name;
  if (!t.defined() || !t.is_cuda()) fail(n + ": expected a CUDA tensor");
  if (like) {
    if (t.scalar_type() != like->scalar_type() || t.sizes() != like->sizes() ||
        t.device() != like->device())
      fail(n + ": expected the shape, type and device of the first tensor");
  } else {
    if (type_of(t) < 0) fail(n + ": expected float32, float16 or bfloat16");
    if (t.get_device() != c10::cuda::current_device())
      fail(n + ": not on the current device");
  }
  const int64_t dims = t.dim();
  if (dims == 0) fail(n + ": expected at least one dimension");
  Rows r;
  r.p = t.data_ptr();
  r.cols = t.size(dims - 1);
  r.rows = 1;  // (rows of no elements are rows, too)
  for (int64_t d = 0; d < dims - 1; ++d) r.rows *= t.size(d);
  r.ld = std::max<int64_t>(r.cols, 1);
  if (t.is_contiguous()) return r;
  if (r.cols > 1 && t.stride(dims - 1) != 1) fail(n + ": its last dimension is not contiguous");
  if (r.rows <= 1) return r;
  // the pitch, and each leading dimension a whole number of the next one's
  int64_t pitch = -1, span = 0;
  for (int64_t d = dims - 2; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (pitch < 0) {
      pitch = t.stride(d);
      span = pitch * t.size(d);
    } else {
      if (t.stride(d) != span)
        fail(n + ": its leading dimensions cannot be folded into rows without a copy");
      span *= t.size(d);
    }
  }
  if (pitch < r.cols) fail(n + ": its rows overlap");
  r.ld = pitch;
  return r;
}
Rows rows_of(const MaybeTensor& t, const char* name, const Tensor& like) {
  return t ? rows_of(*t, name, &like) : Rows();
}

// `size` contiguous elements of float32 or, with own, of like's type; null for
// none.
void* vector_of(const MaybeTensor& t, const char* name, int64_t size, const Tensor& like,
                at::ScalarType first, at::ScalarType second) {
  if (!t) return nullptr;
  if (!t->defined() || (t->scalar_type() != first && t->scalar_type() != second) ||
      t->device() != like.device() || t->dim() != 1 || t->numel() != size || !t->is_contiguous())
    fail(std::string(name) + ": expected " + std::to_string(size) +
         " contiguous elements of the right type on the first tensor's device");
  return t->data_ptr();
}

// Address of a contiguous tensor with an element for each row of `z`.
void* per_row(const MaybeTensor& t, const char* name, const Tensor& z, at::ScalarType type) {
  if (!t) return nullptr;
  if (!t->defined() || t->scalar_type() != type || t->device() != z.device() ||
      !t->is_contiguous() || t->sizes() != z.sizes().slice(0, z.dim() - 1))
    fail(std::string(name) + ": expected a contiguous " +
         (type == at::kLong ? "int64" : "float32") + " tensor with an element for each row");
  return t->data_ptr();
}

void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }
// A new tensor on like's device, without the way through the dispatcher (a
// layer norm of one token, of four: 6.0 us for 8.9).
Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}
Tensor floats(at::IntArrayRef sizes, const Tensor& like) { return fresh(sizes, at::kFloat, like); }
Tensor bytes(uint64_t n, const Tensor& like) { return fresh({(int64_t)n}, at::kByte, like); }

// A tensor that was there has been written: what autograd has saved of it no
// longer is what it holds.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(const MaybeTensor& t) {
  if (t) written(*t);
}

// ------------------------------------------------------------------ dropout
Tensor dropout(const Tensor& x, double p, uint64_t seed, uint64_t offset,
               const MaybeTensor& residual, const MaybeTensor& out) {
  const Rows a = rows_of(x, "x"), r = rows_of(residual, "residual", x);
  Tensor y = out ? *out : fresh(x.sizes(), x.scalar_type(), x);
  const Rows o = rows_of(y, "out", &x);
  check(lib.rot_dropout(a.p, a.ld, r.p, r.ld, o.p, o.ld, a.rows, a.cols, type_of(x), p, seed,
                        offset, stream()),
        "rot_dropout");
  written(out);
  return y;
}

// --------------------------------------------------------------- layer norm
std::tuple<Tensor, Tensor, Tensor, Tensor> layer_norm(const Tensor& x, const Tensor& weight,
                                                      const MaybeTensor& bias, double eps,
                                                      const MaybeTensor& residual, double p,
                                                      uint64_t seed, uint64_t offset) {
  const Rows a = rows_of(x, "x"), r = rows_of(residual, "residual", x);
  const void* w = vector_of(weight, "weight", a.cols, x, at::kFloat, x.scalar_type());
  const void* b = vector_of(bias, "bias", a.cols, x, weight.scalar_type(), weight.scalar_type());
  Tensor y = fresh(x.sizes(), x.scalar_type(), x);
  const bool mixes = residual.has_value() || p > 0;
  Tensor h = mixes ? fresh(x.sizes(), x.scalar_type(), x) : x;
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  Tensor mean = floats(lead, x), rstd = floats(lead, x);
  check(lib.rot_layer_norm_forward(a.p, a.ld, r.p, r.ld, w, b, type_of(weight),
                                   mixes ? h.data_ptr() : nullptr, a.cols, y.data_ptr(), a.cols,
                                   mean.data_ptr<float>(), rstd.data_ptr<float>(), a.rows, a.cols,
                                   type_of(x), (float)eps, p, seed, offset, stream()),
        "rot_layer_norm_forward");
  return {y, h, mean, rstd};
}

std::tuple<Tensor, Tensor, Tensor, MaybeTensor> layer_norm_backward(
    const Tensor& dy, const Tensor& h, const Tensor& mean, const Tensor& rstd,
    const Tensor& weight, const MaybeTensor& dh, double p, uint64_t seed, uint64_t offset,
    bool bias) {
  const Rows a = rows_of(dy, "dy"), b = rows_of(h, "h", &dy), c = rows_of(dh, "dh", dy);
  const void* w = vector_of(weight, "weight", a.cols, dy, at::kFloat, dy.scalar_type());
  for (const Tensor* t : {&mean, &rstd})
    if (!t->defined() || t->scalar_type() != at::kFloat || !t->is_contiguous() ||
        t->numel() != a.rows || t->device() != dy.device())
      fail("mean, rstd: expected contiguous float32 tensors with an element for each row");
  Tensor dx = fresh(dy.sizes(), dy.scalar_type(), dy);
  Tensor dres = p > 0 ? fresh(dy.sizes(), dy.scalar_type(), dy) : dx;
  Tensor dw = floats({a.cols}, dy);
  MaybeTensor db;
  if (bias) db = floats({a.cols}, dy);
  const uint64_t need = lib.rot_layer_norm_work_bytes(a.rows, a.cols);
  Tensor work = bytes(need, dy);
  check(lib.rot_layer_norm_backward(
            a.p, a.ld, b.p, b.ld, mean.data_ptr<float>(), rstd.data_ptr<float>(), w,
            type_of(weight), c.p, c.ld, p > 0 ? dres.data_ptr() : nullptr, a.cols, dx.data_ptr(),
            a.cols, dw.data_ptr<float>(), db ? db->data_ptr<float>() : nullptr, a.rows, a.cols,
            type_of(dy), p, seed, offset, work.data_ptr(), need, stream()),
        "rot_layer_norm_backward");
  return {dx, dres, dw, db};
}

// -------------------------------------------------------------- policy loss
Tensor token_logprobs(const Tensor& logits, const Tensor& targets, const MaybeTensor& weights) {
  const Rows z = rows_of(logits, "logits");
  const auto* t = static_cast<const int64_t*>(per_row(targets, "targets", logits, at::kLong));
  const auto* w = static_cast<const float*>(per_row(weights, "weights", logits, at::kFloat));
  Tensor logp = floats(targets.sizes(), logits);
  check(lib.rot_token_logprobs(z.p, z.ld, t, w, logp.data_ptr<float>(), z.rows, z.cols,
                               type_of(logits), stream()),
        "rot_token_logprobs");
  return logp;
}

std::tuple<Tensor, Tensor, MaybeTensor> policy_loss(
    const Tensor& logits, const Tensor& targets, const Tensor& old_logp, const Tensor& advantages,
    const Tensor& weights, const MaybeTensor& ref_logp, double clip_low, double clip_high,
    double kl_coef, bool grad, double grad_scale, const MaybeTensor& out) {
  const Rows z = rows_of(logits, "logits");
  const auto f = [&](const MaybeTensor& t, const char* name) {
    return static_cast<const float*>(per_row(t, name, logits, at::kFloat));
  };
  const auto* t = static_cast<const int64_t*>(per_row(targets, "targets", logits, at::kLong));
  const float *old = f(old_logp, "old_logp"), *adv = f(advantages, "advantages"),
              *w = f(weights, "weights"), *ref = f(ref_logp, "ref_logp");
  MaybeTensor d;
  Rows o;
  if (grad) {
    d = out ? *out : fresh(logits.sizes(), logits.scalar_type(), logits);
    o = rows_of(*d, "out", &logits);
  }
  Tensor loss = floats({}, logits), logp = floats(targets.sizes(), logits);
  Tensor terms = floats({z.rows}, logits);
  check(lib.rot_policy_loss(z.p, z.ld, t, old, ref, adv, w, loss.data_ptr<float>(),
                            logp.data_ptr<float>(), terms.data_ptr<float>(), o.p, o.ld, z.rows,
                            z.cols, type_of(logits), (float)clip_low, (float)clip_high,
                            (float)kl_coef, (float)grad_scale, stream()),
        "rot_policy_loss");
  if (grad) written(out);
  return {loss, logp, d};
}

// ------------------------------------------------------------ 8-bit matrices
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m; }

// Row pitch of an 8-bit matrix (of a single row, torch leaves the stride
// arbitrary).
int64_t pitch8(const Tensor& t) {
  return t.size(0) > 1 && t.size(1) > 0 ? t.stride(0) : up(t.size(1), 16) * 16;
}

struct Matrix8 {
  Tensor data, scale;
  Matrix8(int64_t rows, int64_t cols, int64_t block_rows, at::ScalarType type, const Tensor& like) {
    // rows of whole 128-byte lines, as the product's loads take them (6144 x
    // 2048 x 4099: 47 us, against 71 with rows 4112 bytes apart), where that
    // is not several times the matrix
    const int64_t to = cols > 64 ? 128 : 16;
    data = Tensor(at::detail::empty_strided_cuda({rows, cols}, {up(cols, to) * to, 1}, type,
                                                 like.device()));
    scale = fresh({up(cols, 128), up(rows, block_rows)}, at::kByte, like);
  }
};

using Pair = std::optional<std::tuple<Tensor, Tensor>>;

// (x in 8 bits, x transposed in 8 bits), each as (data, scale) where asked for.
std::tuple<Pair, Pair> fp8_quantize(const Tensor& x, int64_t block_rows, bool rows,
                                    bool transposed, bool e5m2) {
  const Rows a = rows_of(x, "x");
  if (block_rows != 1 && block_rows != 128) fail("block_rows: expected 1 or 128");
  if (!rows && !transposed) fail("nothing to write: rows and transposed are both false");
  const at::ScalarType type = e5m2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn;
  Pair q, t;
  void *qp = nullptr, *tp = nullptr;
  uint8_t *qs = nullptr, *ts = nullptr;
  int64_t qld = 0, tld = 0;
  if (rows) {
    Matrix8 m(a.rows, a.cols, block_rows, type, x);
    qp = m.data.data_ptr(), qs = m.scale.data_ptr<uint8_t>(), qld = pitch8(m.data);
    q = std::make_tuple(m.data, m.scale);
  }
  if (transposed) {
    Matrix8 m(a.cols, a.rows, block_rows, type, x);
    tp = m.data.data_ptr(), ts = m.scale.data_ptr<uint8_t>(), tld = pitch8(m.data);
    t = std::make_tuple(m.data, m.scale);
  }
  if (a.rows > 0 && a.cols > 0)
    check(lib.rot_fp8_quantize(a.p, a.ld, a.rows, a.cols, type_of(x),
                               e5m2 ? ROT_TYPE_E5M2 : ROT_TYPE_E4M3, (int32_t)block_rows, qp, qld,
                               qs, up(a.rows, block_rows), tp, tld, ts, up(a.cols, block_rows),
                               stream()),
          "rot_fp8_quantize");
  return {q, t};
}

// A product's operand from an Fp8Matrix's parts.
struct Operand {
  const void* p;
  const uint8_t* s;
  int64_t rows, cols, ld, lds;
  int format;
  int32_t block_rows;
};
Operand operand(const Tensor& d, const Tensor& s, int64_t block_rows, const char* name) {
  const std::string n = name;
  Operand o;
  if (!d.defined() || !d.is_cuda() || (o.format = format_of(d)) < 0 || d.dim() != 2 ||
      (d.size(1) > 1 && d.stride(1) != 1))
    fail(n + ": expected a 2-D float8_e4m3fn or float8_e5m2 CUDA tensor of unit column stride");
  if (d.get_device() != c10::cuda::current_device()) fail(n + ": not on the current device");
  o.p = d.data_ptr();
  o.rows = d.size(0), o.cols = d.size(1), o.ld = pitch8(d);
  if (reinterpret_cast<uintptr_t>(o.p) % 16 || o.ld % 16 || o.ld < o.cols)
    fail(n + ": its rows must start on multiples of 16 bytes");
  if (block_rows != 1 && block_rows != 128) fail(n + ": block_rows must be 1 or 128");
  o.block_rows = (int32_t)block_rows;
  o.lds = up(o.rows, block_rows);
  if (!s.defined() || s.scalar_type() != at::kByte || s.device() != d.device() || s.dim() != 2 ||
      s.size(0) != up(o.cols, 128) || s.size(1) != o.lds || !s.is_contiguous())
    fail(n + ": expected a contiguous uint8 scale of [ceil(columns / 128), ceil(rows / block_rows)]");
  o.s = s.data_ptr<uint8_t>();
  return o;
}

Tensor product_out(const MaybeTensor& out, int64_t M, int64_t N, at::ScalarType type,
                   bool accumulate, const Tensor& like) {
  if (accumulate && (!out || out->scalar_type() != at::kFloat))
    fail("accumulate: expected a float32 out");
  if (!out) return fresh({M, N}, type, like);
  if (out->dim() != 2 || out->size(0) != M || out->size(1) != N || out->device() != like.device())
    fail("out: expected " + std::to_string(M) + " x " + std::to_string(N) +
         " elements on the operands' device");
  return *out;
}

Tensor fp8_matmul(const Tensor& ad, const Tensor& as, int64_t ar, const Tensor& bd,
                  const Tensor& bs, int64_t br, at::ScalarType type, const MaybeTensor& out,
                  bool accumulate, uintptr_t status) {
  const Operand a = operand(ad, as, ar, "a"), b = operand(bd, bs, br, "b");
  if (a.cols != b.cols) fail("b: expected " + std::to_string(a.cols) + " columns");
  Tensor c = product_out(out, a.rows, b.rows, type, accumulate, ad);
  const Rows o = rows_of(c, "out");
  const uint64_t need = lib.rot_fp8_gemm_work_bytes(a.rows, b.rows, a.cols);
  Tensor work;
  if (need) work = bytes(need, ad);
  check(lib.rot_fp8_gemm(a.rows, b.rows, a.cols, a.p, a.ld, a.format, a.s, a.lds, a.block_rows,
                         b.p, b.ld, b.format, b.s, b.lds, b.block_rows, o.p,
                         std::max(o.ld, b.rows), type_of(c), accumulate,
                         need ? work.data_ptr() : nullptr, need,
                         reinterpret_cast<int32_t*>(status), stream()),
        "rot_fp8_gemm");
  written(out);
  return c;
}

std::vector<int64_t> with_last(const Tensor& t, int64_t last) {
  std::vector<int64_t> s = t.sizes().vec();
  s.back() = last;
  return s;
}

Tensor fp8_linear(const Tensor& x, const Tensor& wd, const Tensor& ws, int64_t wr,
                  uintptr_t status) {
  const Rows a = rows_of(x, "x");
  const Operand w = operand(wd, ws, wr, "weight");
  if (w.cols != a.cols) fail("weight: expected " + std::to_string(a.cols) + " columns");
  Tensor y = fresh(with_last(x, w.rows), x.scalar_type(), x);
  const uint64_t need = lib.rot_fp8_linear_work_bytes(a.rows, a.cols, w.rows);
  Tensor work;
  if (need) work = bytes(need, x);
  check(lib.rot_fp8_linear(a.rows, a.cols, w.rows, a.p, a.ld, type_of(x), w.p, w.ld, w.format, w.s,
                           w.lds, w.block_rows, y.data_ptr(), std::max<int64_t>(w.rows, 1),
                           need ? work.data_ptr() : nullptr, need,
                           reinterpret_cast<int32_t*>(status), stream()),
        "rot_fp8_linear");
  return y;
}

std::tuple<Tensor, Tensor> fp8_linear_backward(const Tensor& dy, const Tensor& x,
                                               const Tensor& wd, const Tensor& ws, int64_t wr,
                                               const MaybeTensor& dw, bool accumulate,
                                               uintptr_t status) {
  const Rows d = rows_of(dy, "dy"), a = rows_of(x, "x");
  if (x.scalar_type() != dy.scalar_type() || a.rows != d.rows)
    fail("x: expected " + std::to_string(d.rows) + " rows of dy's type");
  const Operand w = operand(wd, ws, wr, "weight_t");
  if (w.rows != a.cols || w.cols != d.cols)
    fail("weight_t: expected " + std::to_string(a.cols) + " x " + std::to_string(d.cols));
  if (dw && dw->scalar_type() != at::kFloat) fail("dw: expected float32");
  Tensor g = product_out(dw, d.cols, a.cols, at::kFloat, accumulate, x);
  const Rows o = rows_of(g, "dw");
  Tensor dx = fresh(with_last(dy, a.cols), dy.scalar_type(), dy);
  const uint64_t need = lib.rot_fp8_linear_backward_work_bytes(d.rows, a.cols, d.cols);
  Tensor work;
  if (need) work = bytes(need, x);
  check(lib.rot_fp8_linear_backward(d.rows, a.cols, d.cols, d.p, d.ld, a.p, a.ld, type_of(x), w.p,
                                    w.ld, w.format, w.s, w.lds, w.block_rows, dx.data_ptr(),
                                    std::max<int64_t>(a.cols, 1), g.data_ptr<float>(),
                                    std::max(o.ld, a.cols), accumulate,
                                    need ? work.data_ptr() : nullptr, need,
                                    reinterpret_cast<int32_t*>(status), stream()),
        "rot_fp8_linear_backward");
  written(dw);
  return {dx, g};
}

// -------------------------------------------------------------------- heads
// [batch, tokens, heads, dim] or [tokens, heads, dim], a head's elements next
// to one another.
struct Shape {
  int64_t batch, tokens, dim;
};
rot_heads heads_of(const Tensor& t, const char* name, const Tensor& first) {
  const std::string n = name;
  if (!t.defined() || !t.is_cuda()) fail(n + ": expected a CUDA tensor");
  const int64_t d = t.dim();
  if (&t == &first) {
    if (type_of(t) < 0) fail(n + ": expected float32, float16 or bfloat16");
    if (t.get_device() != c10::cuda::current_device()) fail(n + ": not on the current device");
    if (d != 3 && d != 4) fail(n + ": expected [tokens, heads, dim] or [batch, tokens, heads, dim]");
  } else if (t.scalar_type() != first.scalar_type() || t.device() != first.device() ||
             d != first.dim() || t.size(d - 1) != first.size(d - 1) ||
             t.sizes().slice(0, d - 2) != first.sizes().slice(0, d - 2)) {
    fail(n + ": expected the first tensor's type, device, tokens and head size");
  }
  if (t.size(d - 1) > 1 && t.stride(d - 1) != 1) fail(n + ": its last dimension is not contiguous");
  rot_heads h;
  h.data = t.data_ptr();
  h.heads = t.size(d - 2);
  h.head_stride = t.stride(d - 2), h.token_stride = t.stride(d - 3);
  h.batch_stride = d == 4 ? t.stride(0) : 0;
  return h;
}
rot_heads like_heads(const Tensor& t, const char* name, const Tensor& other, const Tensor& first) {
  if (t.defined() && t.sizes() != other.sizes()) fail(std::string(name) + ": expected the shape of its input");
  return heads_of(t, name, first);
}
Shape shape_of(const Tensor& t) {
  const int64_t d = t.dim();
  return {d == 4 ? t.size(0) : 1, t.size(d - 3), t.size(d - 1)};
}

struct Rotation {
  rot_rotary r = {};
  const rot_rotary* p = nullptr;
};
Rotation rotation_of(const MaybeTensor& turns, double magnitude, bool interleaved,
                     const MaybeTensor& positions, int64_t start, const Tensor& q) {
  Rotation o;
  if (!turns) return o;
  if (!turns->defined() || turns->scalar_type() != at::kLong || turns->dim() != 1 ||
      !turns->is_contiguous() || turns->device() != q.device())
    fail("rotary: expected contiguous int64 turns on the first tensor's device");
  o.p = &o.r;
  o.r.turns = reinterpret_cast<const uint64_t*>(turns->data_ptr());
  o.r.rotated = 2 * turns->numel();
  if (o.r.rotated > q.size(q.dim() - 1)) fail("rotary: more pairs than the heads have");
  o.r.magnitude = (float)magnitude, o.r.interleaved = interleaved, o.r.start = start;
  if (!positions) return o;
  const Tensor& p = *positions;
  if (!p.defined() || (p.scalar_type() != at::kLong && p.scalar_type() != at::kInt) ||
      p.device() != q.device())
    fail("positions: expected int64 or int32 on the first tensor's device");
  const Shape s = shape_of(q);
  const int64_t d = p.dim();
  if (d < 1 || d > q.dim() - 2 || p.size(d - 1) != s.tokens || (d == 2 && p.size(0) != s.batch))
    fail("positions: expected one for each token, or one for each token of a batch entry");
  o.r.positions = p.data_ptr();
  o.r.position_bytes = p.scalar_type() == at::kLong ? 8 : 4;
  o.r.position_token_stride = p.stride(d - 1);
  o.r.position_batch_stride = d == 2 ? p.stride(0) : 0;
  return o;
}

// An output must not lie in what other rows are read from or written to: the
// order of a call's rows is not fixed.  in_place: it may be that tensor itself.
// (Parts of one buffer that are not dense are held apart by the caller, but for
// their first elements.)
void apart(const MaybeTensor& out, const char* name, const MaybeTensor& other,
           const char* other_name, bool in_place) {
  if (!out || !other || !out->defined() || !other->defined()) return;
  const Tensor &a = *out, &b = *other;
  if (a.numel() == 0 || b.numel() == 0) return;
  bool over = a.data_ptr() == b.data_ptr();
  if (over && in_place && a.sizes() == b.sizes()) {
    over = false;
    for (int64_t d = 0; d < a.dim(); ++d) over |= a.size(d) > 1 && a.stride(d) != b.stride(d);
    if (!over) return;
  }
  if (over || at::get_overlap_status(a, b) == at::MemOverlapStatus::Partial)
    fail(std::string(name) + ": overlaps " + other_name);
}
void outputs_apart(const MaybeTensor& out, const MaybeTensor& k_out, const MaybeTensor& q,
                   const MaybeTensor& k) {
  if (!out && !k_out) return;
  apart(out, "out", q, "its input", true), apart(k_out, "k_out", k, "its input", true);
  apart(out, "out", k, "the other side's input", false);
  apart(k_out, "k_out", q, "the other side's input", false);
  apart(out, "out", k_out, "k_out", false);
}

std::tuple<Tensor, MaybeTensor> rotate(const Tensor& q, const MaybeTensor& k, const Tensor& turns,
                                       double magnitude, bool interleaved,
                                       const MaybeTensor& positions, int64_t start, bool inverse,
                                       const MaybeTensor& out, const MaybeTensor& k_out) {
  outputs_apart(out, k_out, q, k);
  const rot_heads a = heads_of(q, "q", q);
  if (!k && k_out) fail("k_out: there is no k");
  Tensor y = out ? *out : fresh(q.sizes(), q.scalar_type(), q);
  const rot_heads b = like_heads(y, "out", q, q);
  MaybeTensor z;
  rot_heads c, d;
  if (k) {
    c = heads_of(*k, "k", q);
    z = k_out ? *k_out : fresh(k->sizes(), k->scalar_type(), *k);
    d = like_heads(*z, "k_out", *k, q);
  }
  const Rotation r = rotation_of(turns, magnitude, interleaved, positions, start, q);
  const Shape s = shape_of(q);
  check(lib.rot_rotate(&a, &b, k ? &c : nullptr, k ? &d : nullptr, s.batch, s.tokens, s.dim,
                       type_of(q), r.p, inverse, stream()),
        "rot_rotate");
  written(out), written(k_out);
  return {y, z};
}

const void* head_weight(const Tensor& w, const char* name, const Tensor& q) {
  return vector_of(w, name, q.size(q.dim() - 1), q, at::kFloat, q.scalar_type());
}

std::tuple<Tensor, MaybeTensor> head_norm(const Tensor& q, const Tensor& q_weight,
                                          const MaybeTensor& k, const MaybeTensor& k_weight,
                                          double eps, const MaybeTensor& turns, double magnitude,
                                          bool interleaved, const MaybeTensor& positions,
                                          int64_t start, const MaybeTensor& out,
                                          const MaybeTensor& k_out) {
  outputs_apart(out, k_out, q, k);
  const rot_heads a = heads_of(q, "q", q);
  if (k.has_value() != k_weight.has_value()) fail("k, k_weight: expected both or neither");
  if (!k && k_out) fail("k_out: there is no k");
  const void *w = head_weight(q_weight, "q_weight", q), *v = nullptr;
  Tensor y = out ? *out : fresh(q.sizes(), q.scalar_type(), q);
  const rot_heads b = like_heads(y, "out", q, q);
  MaybeTensor z;
  rot_heads c, d;
  if (k) {
    c = heads_of(*k, "k", q);
    if (k_weight->scalar_type() != q_weight.scalar_type()) fail("k_weight: expected q_weight's type");
    v = head_weight(*k_weight, "k_weight", q);
    z = k_out ? *k_out : fresh(k->sizes(), k->scalar_type(), *k);
    d = like_heads(*z, "k_out", *k, q);
  }
  const Rotation r = rotation_of(turns, magnitude, interleaved, positions, start, q);
  const Shape s = shape_of(q);
  check(lib.rot_head_norm_forward(&a, w, &b, k ? &c : nullptr, v, k ? &d : nullptr,
                                  type_of(q_weight), s.batch, s.tokens, s.dim, type_of(q),
                                  (float)eps, r.p, stream()),
        "rot_head_norm_forward");
  written(out), written(k_out);
  return {y, z};
}

std::tuple<Tensor, MaybeTensor, Tensor, MaybeTensor> head_norm_backward(
    const Tensor& dq, const Tensor& q, const Tensor& q_weight, const MaybeTensor& dk,
    const MaybeTensor& k, const MaybeTensor& k_weight, double eps, const MaybeTensor& turns,
    double magnitude, bool interleaved, const MaybeTensor& positions, int64_t start,
    const MaybeTensor& out, const MaybeTensor& k_out) {
  outputs_apart(out, k_out, dq, dk);
  outputs_apart(out, k_out, q, k);
  const rot_heads a = heads_of(dq, "dq", dq), b = like_heads(q, "q", dq, dq);
  if (k.has_value() != k_weight.has_value() || k.has_value() != dk.has_value())
    fail("dk, k, k_weight: expected all or none");
  if (!k && k_out) fail("k_out: there is no k");
  const void *w = head_weight(q_weight, "q_weight", dq), *v = nullptr;
  Tensor y = out ? *out : fresh(dq.sizes(), dq.scalar_type(), dq);
  const rot_heads o = like_heads(y, "out", dq, dq);
  Tensor dw = floats({dq.size(dq.dim() - 1)}, dq);
  MaybeTensor z, dv;
  rot_heads c, d, p;
  if (k) {
    c = heads_of(*dk, "dk", dq), d = like_heads(*k, "k", *dk, dq);
    if (k_weight->scalar_type() != q_weight.scalar_type()) fail("k_weight: expected q_weight's type");
    v = head_weight(*k_weight, "k_weight", dq);
    z = k_out ? *k_out : fresh(dk->sizes(), dk->scalar_type(), *dk);
    p = like_heads(*z, "k_out", *dk, dq);
    dv = floats({dq.size(dq.dim() - 1)}, dq);
  }
  const Rotation r = rotation_of(turns, magnitude, interleaved, positions, start, dq);
  const Shape s = shape_of(dq);
  const uint64_t need = lib.rot_head_norm_work_bytes(s.dim);
  Tensor work = bytes(need, dq);
  check(lib.rot_head_norm_backward(&a, &b, w, &o, dw.data_ptr<float>(), k ? &c : nullptr,
                                   k ? &d : nullptr, v, k ? &p : nullptr,
                                   k ? dv->data_ptr<float>() : nullptr, type_of(q_weight), s.batch,
                                   s.tokens, s.dim, type_of(dq), (float)eps, r.p, work.data_ptr(),
                                   need, stream()),
        "rot_head_norm_backward");
  written(out), written(k_out);
  return {y, z, dw, dv};
}

// -------------------------------------------------------------------- AdamW
// Lists are read in place: a list of a hundred vectors is host time alone (113
// of them: 13 us a call here; as std::vector<Tensor> with the checks in Python
// 148).
PyObject* fp8_vector = nullptr;  // operators.Fp8Vector

// The current device, asked for once a tensor is a CUDA tensor.
struct Current {
  c10::DeviceIndex index = -1;
  bool has(const Tensor& t) {
    if (!t.defined() || !t.is_cuda()) return false;
    if (index < 0) index = c10::cuda::current_device();
    return t.get_device() == index;
  }
};

// A Python list or tuple.
struct List {
  py::object keep;
  Py_ssize_t size = 0;
  List(const py::object& o, const char* name) {
    PyObject* p = PySequence_Fast(o.ptr(), "");
    if (!p) {
      if (!PyErr_ExceptionMatches(PyExc_TypeError)) throw py::error_already_set();  // (its own)
      PyErr_Clear();
      fail(std::string(name) + ": expected a list");
    }
    keep = py::reinterpret_steal<py::object>(p);
    size = PySequence_Fast_GET_SIZE(p);
  }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(keep.ptr(), i); }
};
const Tensor& tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_CheckExact(o) && !THPVariable_Check(o))
    fail(std::string(name) + ": expected tensors, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// A flat tensor of a list.
void* flat(const Tensor& t, const char* name, int64_t n, Current& device) {
  if (!device.has(t)) fail(std::string(name) + ": expected CUDA tensors on the current device");
  if (!t.is_contiguous() || t.numel() != n)
    fail(std::string(name) + ": expected contiguous tensors with as many elements as the parameters");
  return t.data_ptr();
}
template <class T>
const T* word_of(const MaybeTensor& t, const char* name, at::ScalarType type, Current& device) {
  if (!t) return nullptr;
  if (!device.has(*t) || t->scalar_type() != type || t->numel() != 1)
    fail(std::string(name) + ": expected one element of the right type on the current device");
  return t->data_ptr<T>();
}

// A moment: a float32 tensor, or an Fp8Vector (scale is then set).
void* state_of(PyObject* o, const char* name, int64_t n, Current& device, uint8_t** scale) {
  *scale = nullptr;
  at::ScalarType type = at::kFloat;
  if (PyTuple_Check(o) && PyObject_TypeCheck(o, (PyTypeObject*)fp8_vector)) {
    const Tensor& s = tensor_of(PyTuple_GET_ITEM(o, 1), name);
    if (s.scalar_type() != at::kByte) fail(std::string(name) + ": expected uint8 scales");
    *scale = static_cast<uint8_t*>(flat(s, name, up(n, 128), device));
    o = PyTuple_GET_ITEM(o, 0);
    type = at::kFloat8_e4m3fn;
  }
  const Tensor& t = tensor_of(o, name);
  if (t.scalar_type() != type)
    fail(std::string(name) + ": expected float32 tensors, or Fp8Vectors of float8_e4m3fn");
  return flat(t, name, n, device);
}

void adamw(const py::object& params, const py::object& grads, const py::object& m,
           const py::object& v, const py::object& masters, int64_t step,
           const MaybeTensor& step_device, bool counts, double lr, const MaybeTensor& lr_device,
           double beta1, double beta2, double eps, double weight_decay, const MaybeTensor& norm,
           double max_norm, double scale, uint64_t seed) {
  const List ps(params, "params"), gs(grads, "grads"), m1(m, "m"), v1(v, "v");
  std::optional<List> ms;
  if (!masters.is_none()) ms.emplace(masters, "masters");
  const Py_ssize_t n = ps.size;
  if (gs.size != n || m1.size != n || v1.size != n || (ms && ms->size != n))
    fail("grads, m, v, masters: expected an entry for each parameter");
  Current device;
  std::vector<rot_adamw_tensor> list(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    rot_adamw_tensor& t = list[i];
    const Tensor &p = tensor_of(ps[i], "params"), &g = tensor_of(gs[i], "grads");
    t.n = p.numel();
    t.p = flat(p, "params", t.n, device);
    t.g = flat(g, "grads", t.n, device);
    t.p_type = type_of(p), t.g_type = type_of(g);
    if (t.p_type < 0 || t.g_type < 0)
      fail("params, grads: expected float32, float16 or bfloat16");
    if (g.sizes() != p.sizes()) fail("grads: expected the parameters' shapes");
    t.m = state_of(m1[i], "m", t.n, device, &t.m_scale);
    t.v = state_of(v1[i], "v", t.n, device, &t.v_scale);
    if (!t.m_scale != !t.v_scale && t.n > 0)
      fail("m, v: one in 8 bits, the other not");
    t.master = nullptr;
    if (ms && (*ms)[i] != Py_None) {
      const Tensor& w = tensor_of((*ms)[i], "masters");
      if (w.scalar_type() != at::kFloat) fail("masters: expected float32 tensors");
      t.master = static_cast<float*>(flat(w, "masters", t.n, device));
      if (t.p_type == ROT_TYPE_F32) fail("masters: a float32 parameter has none");
    } else if (t.p_type == ROT_TYPE_F16) {
      fail("masters: a float16 parameter needs one");
    }
  }
  rot_adamw_hyper h = {};
  h.lr = lr, h.beta1 = beta1, h.beta2 = beta2, h.eps = eps, h.weight_decay = weight_decay;
  h.scale = scale, h.max_norm = max_norm, h.step = step, h.seed = seed;
  h.lr_device = word_of<float>(lr_device, "lr", at::kFloat, device);
  h.step_device = word_of<int64_t>(step_device, "step", at::kLong, device);
  h.norm = word_of<float>(norm, "norm", at::kFloat, device);
  if (!counts) {
    check(lib.rot_adamw_step(list.data(), (int32_t)n, &h, stream()), "rot_adamw_step");
  } else {
    if (!step_device) fail("counts: expected a step on the device");
    Tensor work = bytes(ROT_ADAMW_COUNT_BYTES, *step_device);
    check(lib.rot_adamw_step_counted(list.data(), (int32_t)n, &h,
                                     step_device->data_ptr<int64_t>(), work.data_ptr(), stream()),
          "rot_adamw_step_counted");
    written(*step_device);
  }
  // (the moments are the optimizer's own: no graph has them; a counter takes
  // 12 ns, of a hundred vectors' 14 us a call)
  for (Py_ssize_t i = 0; i < n; ++i) {
    written(THPVariable_Unpack(ps[i]));
    if (list[i].master) written(THPVariable_Unpack((*ms)[i]));
  }
}

Tensor gradient_norm(const py::object& grads) {
  const List gs(grads, "grads");
  Current device;
  std::vector<rot_gradient> list(gs.size);
  for (Py_ssize_t i = 0; i < gs.size; ++i) {
    const Tensor& g = tensor_of(gs[i], "grads");
    list[i].g = flat(g, "grads", g.numel(), device);
    list[i].n = g.numel();
    list[i].type = type_of(g);
    if (list[i].type < 0) fail("grads: expected float32, float16 or bfloat16");
  }
  const at::Device on(at::kCUDA, c10::cuda::current_device());
  Tensor norm(at::detail::empty_cuda({}, at::kFloat, on, std::nullopt));
  const uint64_t need = lib.rot_gradient_norm_work_bytes((int32_t)list.size());
  Tensor work = bytes(need, norm);
  check(lib.rot_gradient_norm(list.data(), (int32_t)list.size(), norm.data_ptr<float>(),
                              work.data_ptr(), need, stream()),
        "rot_gradient_norm");
  return norm;
}

void bind(const py::dict& addresses, py::object error, py::object vector_class) {
#define X(name) \
  lib.name = reinterpret_cast<decltype(lib.name)>(addresses[#name].cast<uintptr_t>());
  ROT_ENTRIES(X)
#undef X
  rot_error = error.release().ptr();
  fp8_vector = vector_class.release().ptr();
}

}  // namespace

PYBIND11_MODULE(_rot_torch, m) {
  m.def("bind", &bind);
  m.def("dropout", &dropout);
  m.def("layer_norm", &layer_norm);
  m.def("layer_norm_backward", &layer_norm_backward);
  m.def("token_logprobs", &token_logprobs);
  m.def("policy_loss", &policy_loss);
  m.def("fp8_quantize", &fp8_quantize);
  m.def("fp8_matmul", &fp8_matmul);
  m.def("fp8_linear", &fp8_linear);
  m.def("fp8_linear_backward", &fp8_linear_backward);
  m.def("rotate", &rotate);
  m.def("head_norm", &head_norm);
  m.def("head_norm_backward", &head_norm_backward);
  m.def("adamw", &adamw);
  m.def("gradient_norm", &gradient_norm);
}
