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
    if like is not None:
        if t.dtype != like.dtype or t.shape != like.shape or t.get_device() != like.get_device():
            _fail(f"{name}: expected shape {tuple(like.shape)}, {like.dtype} on {like.device}, got "
                  f"{tuple(t.shape)}, {t.dtype} on {t.device}")
    else:
        if t.dtype not in _TYPES:
            _fail(f"{name}: expected float32, float16 or bfloat16, got {t.dtype}")
        if t.get_device() != _current_device():
            _fail(f"{name}: on {t.device}, but the current device is cuda:{_current_device()}")
    if t.dim() != 2:
        if t.dim() == 0:
            _fail(f"{name}: expected at least one dimension")
        try:
            t = t.view(t.numel() // t.shape[-1] if t.shape[-1] else 0, t.shape[-1])
        except RuntimeError:
            _fail(f"{name}: its leading dimensions cannot be folded into rows without a copy")
    if not t.is_contiguous():
        rows, cols = t.shape
        if cols > 1 and t.stride(1) != 1:
            _fail(f"{name}: its last dimension is not contiguous")
        if rows > 1 and t.stride(0) < cols:
            _fail(f"{name}: its rows overlap")
    return t


def _ld(t: Optional[torch.Tensor]) -> int:
    """Row pitch of a _matrix() view (torch leaves the stride of a single row,
    or of no row, arbitrary)."""
    if t is None:
        return 0
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _vector(t: Optional[torch.Tensor], name: str, size: int, like: torch.Tensor,
            dtypes) -> Optional[torch.Tensor]:
    """t, `size` contiguous elements of one of `dtypes` on like's device (or None)."""
    if t is not None and (not isinstance(t, torch.Tensor) or t.dtype not in dtypes
                          or t.get_device() != like.get_device() or t.shape != (size,)
                          or not t.is_contiguous()):
        _fail(f"{name}: expected a contiguous tensor of {size} elements, "
              f"{' or '.join(str(d) for d in dtypes)}, on {like.device}")
    return t


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _word(x: int, name: str) -> int:
    if not 0 <= x < 1 << 64:
        _fail(f"{name}: expected a whole number from 0 to 2^64 - 1")
    return x


_current_device = torch.cuda.current_device


def _stream() -> int:
    return torch._C._cuda_getCurrentRawStream(_current_device())


def _on(stream, call, *inputs):
    """call() with `stream` current: its allocations and launches belong to it;
    the inputs are marked as used on it."""
    with torch.cuda.stream(stream):
        result = call()
    for t in inputs:
        for u in (t[:2] if isinstance(t, Fp8Matrix) else (t,)):
            if u is not None:
                u.record_stream(stream)
    return result


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
    if stream is not None:
        return _on(stream, lambda: dropout(x, p, seed, offset, residual=residual, out=out),
                   x, residual, out)
    x2 = _matrix(x, "x")
    rows, cols = x2.shape
    r2 = None if residual is None else _matrix(residual, "residual", x)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        ldo, po = cols, out.data_ptr()
    else:
        o2 = _matrix(out, "out", x)
        ldo, po = _ld(o2), o2.data_ptr()
    B._check(B.lib().rot_dropout(x2.data_ptr(), _ld(x2), _ptr(r2), _ld(r2), po, ldo, rows, cols,
                                 _TYPES[x.dtype], p, _word(seed, "seed"), _word(offset, "offset"),
                                 _stream()), "rot_dropout")
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
    if stream is not None:
        return _on(stream, lambda: layer_norm(x, weight, bias, eps, residual=residual, p=p,
                                              seed=seed, offset=offset),
                   x, weight, bias, residual)
    x2 = _matrix(x, "x")
    rows, cols = x2.shape
    r2 = None if residual is None else _matrix(residual, "residual", x)
    if weight is None:
        _fail("weight: expected a tensor")
    _vector(weight, "weight", cols, x, (torch.float32, x.dtype))
    _vector(bias, "bias", cols, x, (weight.dtype,))
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    h = x if residual is None and p == 0 else torch.empty_like(y)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    B._check(B.lib().rot_layer_norm_forward(
        x2.data_ptr(), _ld(x2), _ptr(r2), _ld(r2), weight.data_ptr(), _ptr(bias),
        _TYPES[weight.dtype], 0 if h is x else h.data_ptr(), cols, y.data_ptr(), cols,
        mean.data_ptr(), rstd.data_ptr(), rows, cols, _TYPES[x.dtype], eps, p,
        _word(seed, "seed"), _word(offset, "offset"), _stream()), "rot_layer_norm_forward")
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
    if stream is not None:
        return _on(stream, lambda: layer_norm_backward(dy, h, mean, rstd, weight, dh=dh, p=p,
                                                       seed=seed, offset=offset, bias=bias),
                   dy, h, mean, rstd, weight, dh)
    dy2, h2 = _matrix(dy, "dy"), _matrix(h, "h", dy)
    rows, cols = dy2.shape
    d2 = None if dh is None else _matrix(dh, "dh", dy)
    if weight is None:
        _fail("weight: expected a tensor")
    _vector(weight, "weight", cols, dy, (torch.float32, dy.dtype))
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if not isinstance(t, torch.Tensor) or not t.is_contiguous():
            _fail(f"{name}: expected a contiguous tensor")
        _vector(t if t.dim() == 1 else t.view(-1), name, rows, dy, (torch.float32,))
    L = B.lib()
    dx = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
    dres = torch.empty_like(dx) if p > 0 else dx
    dweight = torch.empty(cols, dtype=torch.float32, device=dy.device)
    dbias = torch.empty_like(dweight) if bias else None
    need = L.rot_layer_norm_work_bytes(rows, cols)
    work = torch.empty(need, dtype=torch.uint8, device=dy.device)
    B._check(L.rot_layer_norm_backward(
        dy2.data_ptr(), _ld(dy2), h2.data_ptr(), _ld(h2), mean.data_ptr(), rstd.data_ptr(),
        weight.data_ptr(), _TYPES[weight.dtype], _ptr(d2), _ld(d2),
        dres.data_ptr() if p > 0 else 0, cols, dx.data_ptr(), cols, dweight.data_ptr(),
        _ptr(dbias), rows, cols, _TYPES[dy.dtype], p, _word(seed, "seed"),
        _word(offset, "offset"), work.data_ptr(), need, _stream()), "rot_layer_norm_backward")
    return dx, dres, dweight, dbias


# ---------------------------------------------------------------------------
# policy loss
# ---------------------------------------------------------------------------


def _per_token(t: torch.Tensor, name: str, logits: torch.Tensor, dtype=torch.float32) -> int:
    """Address of a contiguous tensor with an element for each row of logits."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != logits.shape[:-1] \
            or not t.is_contiguous() or t.get_device() != logits.get_device():
        _fail(f"{name}: expected a contiguous {dtype} tensor of shape "
              f"{tuple(logits.shape[:-1])} on {logits.device}")
    return t.data_ptr()


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, *,
                   weights: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Log-probability (float32) of each target (int64) under the softmax of its
    row of logits.  Tokens with a weight of zero are not looked at and get 0;
    a target outside the vocabulary gives NaN."""
    if stream is not None:
        return _on(stream, lambda: token_logprobs(logits, targets, weights=weights),
                   logits, targets, weights)
    z = _matrix(logits, "logits")
    pt = _per_token(targets, "targets", logits, torch.int64)
    pw = 0 if weights is None else _per_token(weights, "weights", logits)
    logp = torch.empty(targets.shape, dtype=torch.float32, device=logits.device)
    B._check(B.lib().rot_token_logprobs(z.data_ptr(), _ld(z), pt, pw, logp.data_ptr(), z.shape[0],
                                        z.shape[1], _TYPES[logits.dtype], _stream()),
             "rot_token_logprobs")
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
    if stream is not None:
        return _on(stream, lambda: policy_loss(
            logits, targets, old_logp, advantages, weights, ref_logp=ref_logp, clip_low=clip_low,
            clip_high=clip_high, kl_coef=kl_coef, grad=grad, grad_scale=grad_scale, out=out),
            logits, targets, old_logp, advantages, weights, ref_logp, out)
    z = _matrix(logits, "logits")
    tokens, vocab = z.shape
    pt = _per_token(targets, "targets", logits, torch.int64)
    po = _per_token(old_logp, "old_logp", logits)
    pa = _per_token(advantages, "advantages", logits)
    pw = _per_token(weights, "weights", logits)
    pr = 0 if ref_logp is None else _per_token(ref_logp, "ref_logp", logits)
    logp = torch.empty(targets.shape, dtype=torch.float32, device=logits.device)
    loss = torch.empty((), dtype=torch.float32, device=logits.device)
    terms = torch.empty_like(logp)
    if not grad:
        out, pd, ldd = None, 0, 0
    elif out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        pd, ldd = out.data_ptr(), vocab
    else:
        o2 = _matrix(out, "out", logits)
        pd, ldd = o2.data_ptr(), _ld(o2)
    B._check(B.lib().rot_policy_loss(
        z.data_ptr(), _ld(z), pt, po, pr, pa, pw, loss.data_ptr(), logp.data_ptr(),
        terms.data_ptr(), pd, ldd, tokens,
        vocab, _TYPES[logits.dtype], clip_low, clip_high, kl_coef, grad_scale, _stream()),
        "rot_policy_loss")
    return loss, logp, out


# ---------------------------------------------------------------------------
# 8-bit matrices and linear layers
# ---------------------------------------------------------------------------

_status = {}  # device index -> the products' status word


def _status_word(like: torch.Tensor) -> int:
    """Address of the status word of like's device."""
    i = like.get_device()
    word = _status.get(i)
    if word is None:
        word = _status[i] = torch.zeros(1, dtype=torch.int32, device=like.device)
        torch.cuda.synchronize(word.device)  # (later calls may be on any stream)
    return word.data_ptr()


def status(device="cuda") -> int:
    """Waits for the device, then reads and clears the products' status word:
    ROT_OK, or ROT_ETIMEOUT if a device-side wait gave up since the last
    call."""
    device = torch.device(device)
    word = _status.get(_current_device() if device.index is None else device.index)
    torch.cuda.synchronize(device)
    if word is None:
        return B.ROT_OK
    code = int(word.item())
    word.zero_()
    return code


def _fp8_empty(rows: int, cols: int, block_rows: int, dtype, device) -> Fp8Matrix:
    # rows of whole 128-byte lines, as the product's loads take them (6144 x 2048 x 4099: 47 us,
    # against 71 with rows 4112 bytes apart), where that is not several times the matrix
    to = 128 if cols > 64 else 16
    data = torch.empty_strided((rows, cols), ((cols + to - 1) // to * to, 1), dtype=dtype,
                               device=device)
    scale = torch.empty(((cols + 127) // 128, -(-rows // block_rows)), dtype=torch.uint8,
                        device=device)
    return Fp8Matrix(data, scale, block_rows)


def _fp8_ld(t: torch.Tensor) -> int:
    # (of a single row, torch leaves the stride arbitrary)
    return t.stride(0) if t.shape[0] > 1 and t.shape[1] > 0 else (t.shape[1] + 15) // 16 * 16


def fp8_quantize(x: torch.Tensor, *, block_rows: int = 1, rows: bool = True,
                 transposed: bool = False, dtype=torch.float8_e4m3fn, stream=None
                 ) -> Tuple[Optional[Fp8Matrix], Optional[Fp8Matrix]]:
    """(x in 8 bits, x transposed in 8 bits), each where asked for, from one
    read of x.  block_rows 1 (activations and gradients: a scale for each row
    and 128 columns) or 128 (weights: a scale for each 128 x 128)."""
    if stream is not None:
        return _on(stream, lambda: fp8_quantize(x, block_rows=block_rows, rows=rows,
                                                transposed=transposed, dtype=dtype), x)
    x2 = _matrix(x, "x")
    if block_rows not in (1, 128):
        _fail("block_rows: expected 1 or 128")
    if dtype not in _FORMATS:
        _fail("dtype: expected float8_e4m3fn or float8_e5m2")
    if not rows and not transposed:
        _fail("nothing to write: rows and transposed are both false")
    R, C = x2.shape
    q = _fp8_empty(R, C, block_rows, dtype, x.device) if rows else None
    t = _fp8_empty(C, R, block_rows, dtype, x.device) if transposed else None
    qa = (q.data.data_ptr(), _fp8_ld(q.data), q.scale.data_ptr(), q.scale.shape[1]) if rows \
        else (0, 0, 0, 0)
    ta = (t.data.data_ptr(), _fp8_ld(t.data), t.scale.data_ptr(), t.scale.shape[1]) \
        if transposed else (0, 0, 0, 0)
    B._check(B.lib().rot_fp8_quantize(x2.data_ptr(), _ld(x2), R, C, _TYPES[x.dtype],
                                      _FORMATS[dtype], block_rows, *qa, *ta, _stream()),
             "rot_fp8_quantize")
    return q, t


def _operand(m: Fp8Matrix, name: str, device: int = -1):
    """The entry points' arguments for m, on `device` (any: the current one)."""
    if not isinstance(m, Fp8Matrix):
        _fail(f"{name}: expected an Fp8Matrix")
    d, sc, block_rows = m
    if not isinstance(d, torch.Tensor) or not d.is_cuda or d.dtype not in _FORMATS \
            or d.dim() != 2 or (d.shape[1] > 1 and d.stride(1) != 1):
        _fail(f"{name}: expected a 2-D float8_e4m3fn or float8_e5m2 CUDA tensor of unit column "
              "stride")
    if d.get_device() != (_current_device() if device < 0 else device):
        _fail(f"{name}: on {d.device}, expected cuda:{_current_device() if device < 0 else device}")
    (rows, cols), ld, p = d.shape, _fp8_ld(d), d.data_ptr()
    if p % 16 or ld % 16 or ld < cols:
        _fail(f"{name}: its rows must start on multiples of 16 bytes")
    if block_rows not in (1, 128):
        _fail(f"{name}: block_rows must be 1 or 128")
    blocks = -(-rows // block_rows)
    if not isinstance(sc, torch.Tensor) or sc.dtype != torch.uint8 \
            or sc.get_device() != d.get_device() or sc.shape != (-(-cols // 128), blocks) \
            or not sc.is_contiguous():
        _fail(f"{name}: expected a contiguous uint8 scale of shape {(-(-cols // 128), blocks)} "
              f"on {d.device}")
    return p, ld, _FORMATS[d.dtype], sc.data_ptr(), blocks, block_rows


def fp8_matmul(a: Fp8Matrix, b: Fp8Matrix, *, dtype=torch.float32,
               out: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None
               ) -> torch.Tensor:
    """a b^T (M x N of `dtype`), or out += a b^T (accumulate, a float32 out):
    exact products, float32 sums."""
    if stream is not None:
        return _on(stream, lambda: fp8_matmul(a, b, dtype=dtype, out=out, accumulate=accumulate),
                   a, b, out)
    pa = _operand(a, "a")
    pb = _operand(b, "b", a.data.get_device())
    (M, K), N = a.data.shape, b.data.shape[0]
    if b.data.shape[1] != K:
        _fail(f"b: expected {K} columns, got {b.data.shape[1]}")
    out, ldo = _product_out(out, M, N, dtype, accumulate, a.data)
    L = B.lib()
    need = L.rot_fp8_gemm_work_bytes(M, N, K)
    work = torch.empty(need, dtype=torch.uint8, device=out.device) if need else None
    B._check(L.rot_fp8_gemm(M, N, K, *pa, *pb, out.data_ptr(), ldo, _TYPES[out.dtype],
                            int(accumulate), _ptr(work), need, _status_word(out), _stream()),
             "rot_fp8_gemm")
    return out


def _product_out(out, M: int, N: int, dtype, accumulate: bool, like: torch.Tensor):
    """(out, its row pitch): the tensor given, checked, or a new one."""
    if accumulate and (out is None or out.dtype != torch.float32):
        _fail("accumulate: expected a float32 out")
    if out is None:
        if dtype not in _TYPES:
            _fail("dtype: expected float32, float16 or bfloat16")
        return torch.empty((M, N), dtype=dtype, device=like.device), N
    if out.shape != (M, N):
        _fail(f"out: expected shape {(M, N)}")
    _matrix(out, "out")
    return out, max(_ld(out), N)


def fp8_linear(x: torch.Tensor, weight: Fp8Matrix, *, stream=None) -> torch.Tensor:
    """x W^T in x's type: x (.., inner) is quantised by rows, W (outer x inner)
    is kept in 8 bits by the caller (fp8_quantize(w, block_rows=128))."""
    if stream is not None:
        return _on(stream, lambda: fp8_linear(x, weight), x, weight)
    x2 = _matrix(x, "x")
    pw = _operand(weight, "weight")
    (tokens, inner), outer = x2.shape, weight.data.shape[0]
    if weight.data.shape[1] != inner:
        _fail(f"weight: expected {inner} columns, got {weight.data.shape[1]}")
    L = B.lib()
    y = torch.empty((*x.shape[:-1], outer), dtype=x.dtype, device=x.device)
    need = L.rot_fp8_linear_work_bytes(tokens, inner, outer)
    work = torch.empty(need, dtype=torch.uint8, device=x.device)
    B._check(L.rot_fp8_linear(tokens, inner, outer, x2.data_ptr(), _ld(x2), _TYPES[x.dtype], *pw,
                              y.data_ptr(), outer, work.data_ptr(), need, _status_word(x),
                              _stream()), "rot_fp8_linear")
    return y


def fp8_linear_backward(dy: torch.Tensor, x: torch.Tensor, weight_t: Fp8Matrix, *,
                        dw: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None
                        ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dw) of fp8_linear: dx = dy W in dy's type, from W's transpose in 8
    bits (the second result of fp8_quantize(w, block_rows=128,
    transposed=True)); dw = dy^T x in float32, what the optimizer step reads,
    both operands quantised along the tokens.  dw: written instead of a new
    tensor, or added to with accumulate."""
    if stream is not None:
        return _on(stream, lambda: fp8_linear_backward(dy, x, weight_t, dw=dw,
                                                       accumulate=accumulate),
                   dy, x, weight_t, dw)
    dy2, x2 = _matrix(dy, "dy"), _matrix(x, "x")
    if x.dtype != dy.dtype or x2.shape[0] != dy2.shape[0]:
        _fail(f"x: expected {dy2.shape[0]} rows of {dy.dtype}, got {x2.shape[0]} of {x.dtype}")
    pw = _operand(weight_t, "weight_t")
    (tokens, outer), inner = dy2.shape, x2.shape[1]
    if weight_t.data.shape != (inner, outer):
        _fail(f"weight_t: expected shape {(inner, outer)}, got {tuple(weight_t.data.shape)}")
    if dw is not None and dw.dtype != torch.float32:
        _fail("dw: expected float32")
    dw, ldw = _product_out(dw, outer, inner, torch.float32, accumulate, x)
    L = B.lib()
    dx = torch.empty((*dy.shape[:-1], inner), dtype=dy.dtype, device=dy.device)
    need = L.rot_fp8_linear_backward_work_bytes(tokens, inner, outer)
    work = torch.empty(need, dtype=torch.uint8, device=x.device)
    B._check(L.rot_fp8_linear_backward(
        tokens, inner, outer, dy2.data_ptr(), _ld(dy2), x2.data_ptr(), _ld(x2), _TYPES[x.dtype],
        *pw, dx.data_ptr(), inner, dw.data_ptr(), ldw, int(accumulate), work.data_ptr(), need,
        _status_word(x), _stream()), "rot_fp8_linear_backward")
    return dx, dw
