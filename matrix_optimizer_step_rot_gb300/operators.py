"""Training operators next to the optimizer step, on torch tensors.

Dropout from a counter-based generator, layer norm with the residual stream and
dropout in front of it, the clipped policy loss with its gradient, and linear
layers in 8-bit floating point with power-of-two block scales.  Between them
they carry a training step from hidden states to the float32 gradients that
`optimizer.RotatedAdam` reads.  include/rot_ops.h states the formulas, layouts
and errors; every function here checks its tensors, allocates its outputs and
workspace with torch and runs the library's kernels on the current stream, or
on `stream` (a torch.cuda.Stream: outputs and workspaces then belong to it, and
the inputs are marked as used on it; ordering it after their producers is the
caller's).  There is no other path than the library's.
"""

from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional, Tuple

import torch

from . import binding as B

_TYPES = {torch.float32: B.ROT_TYPE_F32, torch.float16: B.ROT_TYPE_F16,
          torch.bfloat16: B.ROT_TYPE_BF16}
_FORMATS = {torch.float8_e4m3fn: B.ROT_TYPE_E4M3, torch.float8_e5m2: B.ROT_TYPE_E5M2}


class Fp8Matrix(NamedTuple):
    """An R x C matrix in 8 bits: `data` (float8_e4m3fn or float8_e5m2; rows a
    multiple of 16 bytes apart) under one power-of-two scale for each block of
    `block_rows` x 128 elements.  scale: uint8, [ceil(C / 128), ceil(R /
    block_rows)], a byte e for 2^(e - 127), 255 for NaN."""
    data: torch.Tensor
    scale: torch.Tensor
    block_rows: int = 1

    def dequantize(self) -> torch.Tensor:
        """The float32 matrix it stands for (a diagnostic, in torch)."""
        rows, cols = self.data.shape
        e = self.scale.int().t()
        s = torch.where(e > 0, e << 23, 1 << 22).view(torch.float32)  # 2^(e - 127), e = 0 subnormal
        s = torch.where(e == 255, float("nan"), s)
        s = s.repeat_interleave(self.block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
        return self.data.float() * s


# ---------------------------------------------------------------------------
# argument checks
# ---------------------------------------------------------------------------


def _fail(what: str):
    raise ValueError(what)


def _matrix(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None) -> torch.Tensor:
    """t as a 2-D view with unit column stride: leading dimensions fold into
    the rows.  like: must have its shape, type and device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _fail(f"{name}: expected a CUDA tensor")
    if t.dtype not in _TYPES:
        _fail(f"{name}: expected float32, float16 or bfloat16, got {t.dtype}")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype
                             or t.device != like.device):
        _fail(f"{name}: expected shape {tuple(like.shape)}, {like.dtype} on {like.device}, got "
              f"{tuple(t.shape)}, {t.dtype} on {t.device}")
    if t.dim() == 0:
        _fail(f"{name}: expected at least one dimension")
    if t.dim() != 2:
        try:
            t = t.view(t.numel() // t.shape[-1] if t.shape[-1] else 0, t.shape[-1])
        except RuntimeError:
            _fail(f"{name}: its leading dimensions cannot be folded into rows without a copy")
    if t.shape[1] > 1 and t.stride(1) != 1:
        _fail(f"{name}: its last dimension is not contiguous")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        _fail(f"{name}: its rows overlap")
    return t


def _ld(t: Optional[torch.Tensor]) -> int:
    """Row pitch of a _matrix() view (torch leaves the stride of a single row,
    or of no row, arbitrary)."""
    if t is None:
        return 0
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _vector(t: Optional[torch.Tensor], name: str, size: int, device, dtypes) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype not in dtypes \
            or t.shape != (size,) or not t.is_contiguous():
        _fail(f"{name}: expected a contiguous tensor of {size} elements, "
              f"{' or '.join(str(d) for d in dtypes)}, on {device}")
    return t


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _word(x: int, name: str) -> int:
    x = int(x)
    if not 0 <= x < 1 << 64:
        _fail(f"{name}: expected a whole number from 0 to 2^64 - 1")
    return x


class _On:
    """The device and stream of one call: allocations and launches happen on
    `stream` if one is given."""

    def __init__(self, device: torch.device, stream, *inputs):
        if device.index is not None and device.index != torch.cuda.current_device():
            _fail(f"tensors on {device}, but the current device is "
                  f"cuda:{torch.cuda.current_device()}")
        self.given = stream
        if stream is not None:
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self) -> int:
        if self.given is None:
            self.scope = None
            return torch.cuda.current_stream().cuda_stream
        self.scope = contextlib.ExitStack()
        self.scope.enter_context(torch.cuda.stream(self.given))
        return self.given.cuda_stream

    def __exit__(self, *exc):
        if self.scope is not None:
            self.scope.close()


def _like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous output of t's shape."""
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, *,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """residual + dropout(x): element i (row-major) is kept, and scaled by
    1 / (1 - p), where the generator's word for (seed, offset, i) says so; the
    mask is never stored.  Give every call of a training run its own (seed,
    offset).  out: written instead of a new tensor (may be x or residual)."""
    x2 = _matrix(x, "x")
    r2 = None if residual is None else _matrix(residual, "residual", x)
    if out is not None:
        o2 = _matrix(out, "out", x)
    with _On(x.device, stream, x, residual, out) as s:
        if out is None:
            out = _like(x)
            o2 = out if x.dim() == 2 else out.view(x2.shape)
        B._check(B.lib().rot_dropout(x2.data_ptr(), _ld(x2), _ptr(r2), _ld(r2), o2.data_ptr(),
                                     _ld(o2), x2.shape[0], x2.shape[1], _TYPES[x.dtype], p,
                                     _word(seed, "seed"), _word(offset, "offset"), s),
                 "rot_dropout")
    return out


def dropout_backward(dy: torch.Tensor, p: float, seed: int, offset: int = 0, *,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of dropout()'s x from that of its result (the residual's
    gradient is dy itself): the same mask, computed again."""
    return dropout(dy, p, seed, offset, out=out, stream=stream)


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, *, residual: Optional[torch.Tensor] = None, p: float = 0.0,
               seed: int = 0, offset: int = 0, stream=None
               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, h, mean, rstd): the hidden stream h = residual + dropout(x) (x itself
    without either), and y = (h - mean) rstd weight + bias over its last
    dimension.  weight and bias: float32 or x's type.  mean and rstd: float32,
    one for each row; layer_norm_backward takes h, mean and rstd."""
    x2 = _matrix(x, "x")
    rows, cols = x2.shape
    r2 = None if residual is None else _matrix(residual, "residual", x)
    if weight is None:
        _fail("weight: expected a tensor")
    weight = _vector(weight, "weight", cols, x.device, (torch.float32, x.dtype))
    bias = _vector(bias, "bias", cols, x.device, (weight.dtype,))
    with _On(x.device, stream, x, residual, weight, bias) as s:
        y = _like(x)
        h = _like(x) if residual is not None or p > 0 else x
        h2 = None if h is x else (h if h.dim() == 2 else h.view(rows, cols))
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        B._check(B.lib().rot_layer_norm_forward(
            x2.data_ptr(), _ld(x2), _ptr(r2), _ld(r2), weight.data_ptr(), _ptr(bias),
            _TYPES[weight.dtype], _ptr(h2), cols, y.data_ptr(), cols, mean.data_ptr(),
            rstd.data_ptr(), rows, cols, _TYPES[x.dtype], eps, p, _word(seed, "seed"),
            _word(offset, "offset"), s), "rot_layer_norm_forward")
    return y, h, mean, rstd


def layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor, *, dh: Optional[torch.Tensor] = None, p: float = 0.0,
                        seed: int = 0, offset: int = 0, bias: bool = True, stream=None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(dx, dresidual, dweight, dbias) of layer_norm from dy and what the
    forward pass returned.  dh: the gradient that reaches h other than through
    the norm.  dresidual is h's whole gradient and dx that gradient through the
    dropout; without dropout they are one tensor.  dweight and dbias are
    float32 (bias=False: no dbias)."""
    dy2, h2 = _matrix(dy, "dy"), _matrix(h, "h", dy)
    rows, cols = dy2.shape
    d2 = None if dh is None else _matrix(dh, "dh", dy)
    if weight is None:
        _fail("weight: expected a tensor")
    weight = _vector(weight, "weight", cols, dy.device, (torch.float32, dy.dtype))
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if not isinstance(t, torch.Tensor) or not t.is_contiguous():
            _fail(f"{name}: expected a contiguous tensor")
        _vector(t.view(-1), name, rows, dy.device, (torch.float32,))
    with _On(dy.device, stream, dy, h, mean, rstd, weight, dh) as s:
        dx = _like(dy)
        dres = _like(dy) if p > 0 else dx
        dweight = torch.empty(cols, dtype=torch.float32, device=dy.device)
        dbias = torch.empty_like(dweight) if bias else None
        need = B.lib().rot_layer_norm_work_bytes(rows, cols)
        work = torch.empty(need, dtype=torch.uint8, device=dy.device)
        B._check(B.lib().rot_layer_norm_backward(
            dy2.data_ptr(), _ld(dy2), h2.data_ptr(), _ld(h2), mean.data_ptr(), rstd.data_ptr(),
            weight.data_ptr(), _TYPES[weight.dtype], _ptr(d2), _ld(d2),
            dres.data_ptr() if p > 0 else 0, cols, dx.data_ptr(), cols, dweight.data_ptr(),
            _ptr(dbias), rows, cols, _TYPES[dy.dtype], p, _word(seed, "seed"),
            _word(offset, "offset"), work.data_ptr(), need, s), "rot_layer_norm_backward")
    return dx, dres, dweight, dbias


# ---------------------------------------------------------------------------
# policy loss
# ---------------------------------------------------------------------------


def _tokens(logits, targets, **per_token):
    z = _matrix(logits, "logits")
    flat = {}
    for name, t in dict(targets=targets, **per_token).items():
        if t is None:
            flat[name] = None
            continue
        if not isinstance(t, torch.Tensor) or t.shape != logits.shape[:-1] or not t.is_contiguous() \
                or t.device != logits.device \
                or t.dtype != (torch.int64 if name == "targets" else torch.float32):
            _fail(f"{name}: expected a contiguous {'int64' if name == 'targets' else 'float32'} "
                  f"tensor of shape {tuple(logits.shape[:-1])} on {logits.device}")
        flat[name] = t
    return z, flat


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, *,
                   weights: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Log-probability (float32) of each target (int64) under the softmax of its
    row of logits.  Tokens with a weight of zero are not looked at and get 0;
    a target outside the vocabulary gives NaN."""
    z, f = _tokens(logits, targets, weights=weights)
    with _On(logits.device, stream, logits, targets, weights) as s:
        logp = torch.empty(targets.shape, dtype=torch.float32, device=logits.device)
        B._check(B.lib().rot_token_logprobs(z.data_ptr(), _ld(z), f["targets"].data_ptr(),
                                            _ptr(weights), logp.data_ptr(), z.shape[0], z.shape[1],
                                            _TYPES[logits.dtype], s), "rot_token_logprobs")
    return logp


def policy_loss(logits: torch.Tensor, targets: torch.Tensor, old_logp: torch.Tensor,
                advantages: torch.Tensor, weights: torch.Tensor, *,
                ref_logp: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, grad: bool = True,
                grad_scale: float = 1.0, out: Optional[torch.Tensor] = None, stream=None
                ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(loss, logp, dlogits): the sum over tokens of weight times the clipped
    policy term with its KL penalty, each token's log-probability, and
    grad_scale times the loss's gradient with respect to the logits, in their
    type (None with grad=False).  Tokens with a weight of zero are masked: none
    of their inputs is looked at, and their gradient row is 0.  out: written
    instead of a new dlogits; may be `logits` itself."""
    z, _ = _tokens(logits, targets, old_logp=old_logp, advantages=advantages, weights=weights,
                   ref_logp=ref_logp)
    if old_logp is None or advantages is None or weights is None:
        _fail("old_logp, advantages, weights: expected tensors")
    if out is not None:
        o2 = _matrix(out, "out", logits)
    with _On(logits.device, stream, logits, targets, old_logp, advantages, weights, ref_logp,
             out) as s:
        dev = logits.device
        loss = torch.empty((), dtype=torch.float32, device=dev)
        logp = torch.empty(targets.shape, dtype=torch.float32, device=dev)
        terms = torch.empty(max(z.shape[0], 1), dtype=torch.float32, device=dev)
        if not grad:
            out = o2 = None
        elif out is None:
            out = _like(logits)
            o2 = out if out.dim() == 2 else out.view(z.shape)
        B._check(B.lib().rot_policy_loss(
            z.data_ptr(), _ld(z), targets.data_ptr(), old_logp.data_ptr(), _ptr(ref_logp),
            advantages.data_ptr(), weights.data_ptr(), loss.data_ptr(), logp.data_ptr(),
            terms.data_ptr(), _ptr(o2), _ld(o2), z.shape[0], z.shape[1], _TYPES[logits.dtype],
            clip_low, clip_high, kl_coef, grad_scale, s), "rot_policy_loss")
    return loss, logp, out


# ---------------------------------------------------------------------------
# 8-bit matrices and linear layers
# ---------------------------------------------------------------------------

_status = {}  # device index -> the products' status word


def _status_word(device: torch.device) -> torch.Tensor:
    i = device.index if device.index is not None else torch.cuda.current_device()
    if i not in _status:
        _status[i] = torch.zeros(1, dtype=torch.int32, device=device)
    return _status[i]


def status(device="cuda") -> int:
    """Waits for the device, then reads and clears the products' status word:
    ROT_OK, or ROT_ETIMEOUT if a device-side wait gave up since the last
    call."""
    word = _status_word(torch.device(device))
    torch.cuda.synchronize(word.device)
    code = int(word.item())
    word.zero_()
    return code


def _fp8_empty(rows: int, cols: int, block_rows: int, dtype, device) -> Fp8Matrix:
    data = torch.empty(rows, (cols + 15) // 16 * 16, dtype=dtype, device=device)[:, :cols]
    scale = torch.empty((cols + 127) // 128, -(-rows // block_rows), dtype=torch.uint8,
                        device=device)
    return Fp8Matrix(data, scale, block_rows)


def _fp8_ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 and t.shape[1] > 0 else (t.shape[1] + 15) // 16 * 16


def fp8_quantize(x: torch.Tensor, *, block_rows: int = 1, rows: bool = True,
                 transposed: bool = False, dtype=torch.float8_e4m3fn, stream=None
                 ) -> Tuple[Optional[Fp8Matrix], Optional[Fp8Matrix]]:
    """(x in 8 bits, x transposed in 8 bits), each where asked for, from one
    read of x.  block_rows 1 (activations and gradients: a scale for each row
    and 128 columns) or 128 (weights: a scale for each 128 x 128)."""
    x2 = _matrix(x, "x")
    if block_rows not in (1, 128):
        _fail("block_rows: expected 1 or 128")
    if dtype not in _FORMATS:
        _fail("dtype: expected float8_e4m3fn or float8_e5m2")
    if not rows and not transposed:
        _fail("nothing to write: rows and transposed are both false")
    R, C = x2.shape
    with _On(x.device, stream, x) as s:
        q = _fp8_empty(R, C, block_rows, dtype, x.device) if rows else None
        t = _fp8_empty(C, R, block_rows, dtype, x.device) if transposed else None
        qa = (q.data.data_ptr(), _fp8_ld(q.data), q.scale.data_ptr(), q.scale.shape[1]) if rows \
            else (0, 0, 0, 0)
        ta = (t.data.data_ptr(), _fp8_ld(t.data), t.scale.data_ptr(), t.scale.shape[1]) \
            if transposed else (0, 0, 0, 0)
        B._check(B.lib().rot_fp8_quantize(x2.data_ptr(), _ld(x2), R, C, _TYPES[x.dtype],
                                          _FORMATS[dtype], block_rows, *qa, *ta, s),
                 "rot_fp8_quantize")
    return q, t


def _operand(m: Fp8Matrix, name: str, device=None):
    if not isinstance(m, Fp8Matrix):
        _fail(f"{name}: expected an Fp8Matrix")
    d, sc = m.data, m.scale
    if not d.is_cuda or d.dtype not in _FORMATS or d.dim() != 2 \
            or (d.shape[1] > 1 and d.stride(1) != 1):
        _fail(f"{name}: expected a 2-D float8_e4m3fn or float8_e5m2 CUDA tensor of unit column "
              "stride")
    if d.data_ptr() % 16 or _fp8_ld(d) % 16 or _fp8_ld(d) < d.shape[1]:
        _fail(f"{name}: its rows must start on multiples of 16 bytes")
    if m.block_rows not in (1, 128):
        _fail(f"{name}: block_rows must be 1 or 128")
    want = (-(-d.shape[1] // 128), -(-d.shape[0] // m.block_rows))
    if sc.dtype != torch.uint8 or sc.device != d.device or tuple(sc.shape) != want \
            or not sc.is_contiguous():
        _fail(f"{name}: expected a contiguous uint8 scale of shape {want} on {d.device}")
    if device is not None and d.device != device:
        _fail(f"{name}: expected a tensor on {device}")
    return d.data_ptr(), _fp8_ld(d), _FORMATS[d.dtype], sc.data_ptr(), sc.shape[1], m.block_rows


def fp8_matmul(a: Fp8Matrix, b: Fp8Matrix, *, dtype=torch.float32,
               out: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None
               ) -> torch.Tensor:
    """a b^T (M x N of `dtype`), or out += a b^T (accumulate, a float32 out):
    exact products, float32 sums."""
    pa = _operand(a, "a")
    pb = _operand(b, "b", a.data.device)
    (M, K), N = a.data.shape, b.data.shape[0]
    if b.data.shape[1] != K:
        _fail(f"b: expected {K} columns, got {b.data.shape[1]}")
    if out is not None:
        if out.shape != (M, N):
            _fail(f"out: expected shape {(M, N)}")
        _matrix(out, "out")
        if out.device != a.data.device:
            _fail(f"out: expected a tensor on {a.data.device}")
        dtype = out.dtype
    if accumulate and (out is None or out.dtype != torch.float32):
        _fail("accumulate: expected a float32 out")
    if dtype not in _TYPES:
        _fail("dtype: expected float32, float16 or bfloat16")
    with _On(a.data.device, stream, a.data, a.scale, b.data, b.scale, out) as s:
        if out is None:
            out = torch.empty(M, N, dtype=dtype, device=a.data.device)
        need = B.lib().rot_fp8_gemm_work_bytes(M, N, K)
        work = torch.empty(need, dtype=torch.uint8, device=a.data.device) if need else None
        B._check(B.lib().rot_fp8_gemm(M, N, K, *pa, *pb, out.data_ptr(), max(_ld(out), N),
                                      _TYPES[dtype], int(accumulate), _ptr(work), need,
                                      _status_word(a.data.device).data_ptr(), s), "rot_fp8_gemm")
    return out


def fp8_linear(x: torch.Tensor, weight: Fp8Matrix, *, stream=None) -> torch.Tensor:
    """x W^T in x's type: x (.., inner) is quantised by rows, W (outer x inner)
    is kept in 8 bits by the caller (fp8_quantize(w, block_rows=128))."""
    x2 = _matrix(x, "x")
    q, _ = fp8_quantize(x2, stream=stream)
    y = fp8_matmul(q, weight, dtype=x.dtype, stream=stream)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], y.shape[1])


def fp8_linear_backward(dy: torch.Tensor, x: torch.Tensor, weight_t: Fp8Matrix, *,
                        dw: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None
                        ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dw) of fp8_linear: dx = dy W in dy's type, from W's transpose in 8
    bits (the second result of fp8_quantize(w, block_rows=128,
    transposed=True)); dw = dy^T x in float32, what the optimizer step reads,
    both operands quantised along the tokens.  dw: written instead of a new
    tensor, or added to with accumulate."""
    dy2, x2 = _matrix(dy, "dy"), _matrix(x, "x")
    if dy2.shape[0] != x2.shape[0]:
        _fail(f"x: expected {dy2.shape[0]} rows, got {x2.shape[0]}")
    dq, dqt = fp8_quantize(dy2, transposed=True, stream=stream)
    _, xt = fp8_quantize(x2, rows=False, transposed=True, stream=stream)
    dx = fp8_matmul(dq, weight_t, dtype=dy.dtype, stream=stream)
    dw = fp8_matmul(dqt, xt, out=dw, accumulate=accumulate, stream=stream)
    return (dx if dy.dim() == 2 else dx.view(*dy.shape[:-1], dx.shape[1])), dw
