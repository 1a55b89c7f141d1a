// The operators on torch tensors (operators.py): checks of the tensors,
// outputs and workspaces from torch's allocator, and the call into librot on
// the current stream.  No arithmetic.
//
// A call of a small operator is host time alone: a layer norm of one token
// takes 11 us here, four allocations and a launch among them, and took 21 with
// the same checks in Python and the call through ctypes.
//
// The library's entry points come as addresses (bind), so that the one library
// the process has loaded is the one that runs.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
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
  X(rot_fp8_linear_backward)

struct Entries {
#define X(name) decltype(&::name) name = nullptr;
  ROT_ENTRIES(X)
#undef X
} lib;
PyObject* rot_error = nullptr;  // binding.RotError

void bind(const py::dict& addresses, py::object error) {
#define X(name) \
  lib.name = reinterpret_cast<decltype(lib.name)>(addresses[#name].cast<uintptr_t>());
  ROT_ENTRIES(X)
#undef X
  rot_error = error.release().ptr();
}

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
Tensor floats(at::IntArrayRef sizes, const Tensor& like) {
  return at::empty(sizes, like.options().dtype(at::kFloat));
}
Tensor bytes(uint64_t n, const Tensor& like) {
  return at::empty({(int64_t)n}, like.options().dtype(at::kByte));
}

// ------------------------------------------------------------------ dropout
Tensor dropout(const Tensor& x, double p, uint64_t seed, uint64_t offset,
               const MaybeTensor& residual, const MaybeTensor& out) {
  const Rows a = rows_of(x, "x"), r = rows_of(residual, "residual", x);
  Tensor y = out ? *out : at::empty(x.sizes(), x.options());
  const Rows o = rows_of(y, "out", &x);
  check(lib.rot_dropout(a.p, a.ld, r.p, r.ld, o.p, o.ld, a.rows, a.cols, type_of(x), p, seed,
                        offset, stream()),
        "rot_dropout");
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
  Tensor y = at::empty(x.sizes(), x.options());
  const bool mixes = residual.has_value() || p > 0;
  Tensor h = mixes ? at::empty(x.sizes(), x.options()) : x;
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
  Tensor dx = at::empty(dy.sizes(), dy.options());
  Tensor dres = p > 0 ? at::empty(dy.sizes(), dy.options()) : dx;
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
    d = out ? *out : at::empty(logits.sizes(), logits.options());
    o = rows_of(*d, "out", &logits);
  }
  Tensor loss = floats({}, logits), logp = floats(targets.sizes(), logits);
  Tensor terms = floats({z.rows}, logits);
  check(lib.rot_policy_loss(z.p, z.ld, t, old, ref, adv, w, loss.data_ptr<float>(),
                            logp.data_ptr<float>(), terms.data_ptr<float>(), o.p, o.ld, z.rows,
                            z.cols, type_of(logits), (float)clip_low, (float)clip_high,
                            (float)kl_coef, (float)grad_scale, stream()),
        "rot_policy_loss");
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
    data = at::empty_strided({rows, cols}, {up(cols, to) * to, 1}, like.options().dtype(type));
    scale = at::empty({up(cols, 128), up(rows, block_rows)}, like.options().dtype(at::kByte));
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
  if (!out) return at::empty({M, N}, like.options().dtype(type));
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
  Tensor y = at::empty(with_last(x, w.rows), x.options());
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
  Tensor dx = at::empty(with_last(dy, a.cols), dy.options());
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
  return {dx, g};
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
}
