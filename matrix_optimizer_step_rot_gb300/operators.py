"""Training operators next to the optimizer step, on torch tensors.

Dropout from a counter-based generator, layer norm with the residual stream and
dropout in front of it, the clipped policy loss with its gradient, and linear
layers in 8-bit floating point with power-of-two block scales.  Between them
they carry a training step from hidden states to the float32 gradients that
`optimizer.RotatedAdam` reads.  include/rot_ops.h states the formulas, layouts
and errors.  Every function checks its tensors (ValueError), allocates its
outputs and workspace with torch and runs the library's kernels on the current
stream (csrc/torch/torch_ops.cpp), or on `stream` (a torch.cuda.Stream: outputs
and workspaces then belong to it, and the inputs are marked as used on it;
ordering it after their producers is the caller's).  Tensors are on the current
device; a tensor of more than two dimensions is rows of its last one.  There is
no other path than the library's, and no part in torch's autograd: results do
not require gradients, whatever the inputs do, and the backward functions are
calls of their own, as the optimizer step is (examples/policy_step.py has them
together).  The first 8-bit product on a device
allocates its status word: let it run before a stream capture.
"""

from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple, Optional, Tuple

import torch

from . import binding as B

_TYPES = (torch.float32, torch.float16, torch.bfloat16)
_FORMATS = (torch.float8_e4m3fn, torch.float8_e5m2)


class Fp8Matrix(NamedTuple):
    """An R x C matrix in 8 bits: `data` (float8_e4m3fn or float8_e5m2; rows a
    multiple of 16 bytes apart, best of 128) under one power-of-two scale for
    each block of `block_rows` x 128 elements.  scale: uint8, [ceil(C / 128),
    ceil(R / block_rows)], a byte e for 2^(e - 127), 255 for NaN."""
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


_native = None


def _load():
    """The extension module, bound to the loaded library's entry points (raises
    if either has not been built)."""
    global _native
    L = B.lib()
    try:
        from . import _rot_torch
    except ImportError as e:
        raise RuntimeError("_rot_torch.so is missing or does not load: build it with "
                           "matrix_optimizer_step_rot_gb300.build.build()") from e
    _rot_torch.bind({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value
                     for n in B.header_symbols()}, B.RotError)
    _native = _rot_torch
    return _native


def _word(x: int, name: str) -> int:
    if not 0 <= x < 1 << 64:
        raise ValueError(f"{name}: expected a whole number from 0 to 2^64 - 1")
    return x


def _tensors(**given) -> None:
    for name, t in given.items():
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")


def _fp8(m, name: str) -> Fp8Matrix:
    if not isinstance(m, Fp8Matrix):
        raise ValueError(f"{name}: expected an Fp8Matrix, got {type(m).__name__}")
    return m


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
    return (_native or _load()).dropout(x, p, _word(seed, "seed"), _word(offset, "offset"),
                                        residual, out)


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
    _tensors(weight=weight)
    return (_native or _load()).layer_norm(x, weight, bias, eps, residual, p, _word(seed, "seed"),
                                           _word(offset, "offset"))


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
    _tensors(h=h, mean=mean, rstd=rstd, weight=weight)
    return (_native or _load()).layer_norm_backward(dy, h, mean, rstd, weight, dh, p,
                                                    _word(seed, "seed"), _word(offset, "offset"),
                                                    bias)


# ---------------------------------------------------------------------------
# policy loss
# ---------------------------------------------------------------------------


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, *,
                   weights: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Log-probability (float32) of each target (int64) under the softmax of its
    row of logits.  Tokens with a weight of zero are not looked at and get 0;
    a target outside the vocabulary gives NaN."""
    if stream is not None:
        return _on(stream, lambda: token_logprobs(logits, targets, weights=weights),
                   logits, targets, weights)
    _tensors(targets=targets)
    return (_native or _load()).token_logprobs(logits, targets, weights)


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
    of their inputs is looked at, and their gradient row is 0.  With kl_coef 0
    ref_logp is not looked at.  out: written instead of a new dlogits; may be
    `logits` itself."""
    if stream is not None:
        return _on(stream, lambda: policy_loss(
            logits, targets, old_logp, advantages, weights, ref_logp=ref_logp, clip_low=clip_low,
            clip_high=clip_high, kl_coef=kl_coef, grad=grad, grad_scale=grad_scale, out=out),
            logits, targets, old_logp, advantages, weights, ref_logp, out)
    _tensors(targets=targets, old_logp=old_logp, advantages=advantages, weights=weights)
    return (_native or _load()).policy_loss(logits, targets, old_logp, advantages, weights,
                                            ref_logp, clip_low, clip_high, kl_coef, grad,
                                            grad_scale, out)


# ---------------------------------------------------------------------------
# 8-bit matrices and linear layers
# ---------------------------------------------------------------------------

_status = {}  # device index -> (the products' status word, its address)
_making = threading.Lock()


def _status_word(like: torch.Tensor) -> int:
    """Address of the status word of like's device (0 for a tensor that the
    call will refuse)."""
    i = like.get_device()
    if i < 0:
        return 0
    if i not in _status:
        with _making:  # (one word for all threads: launched kernels keep its address)
            if i not in _status:
                word = torch.zeros(1, dtype=torch.int32, device=like.device)
                torch.cuda.synchronize(word.device)  # (later calls may be on any stream)
                _status[i] = word, word.data_ptr()
    return _status[i][1]


def status(device="cuda") -> int:
    """Waits for the device, then reads and clears the products' status word:
    ROT_OK, or ROT_ETIMEOUT if a device-side wait gave up since the last
    call."""
    device = torch.device(device)
    i = torch.cuda.current_device() if device.index is None else device.index
    torch.cuda.synchronize(device)
    if i not in _status:
        return B.ROT_OK
    word = _status[i][0]
    code = int(word.item())
    if code != B.ROT_OK:  # (what another thread's product writes from here on is left for the next call)
        word.zero_()
    return code


def fp8_quantize(x: torch.Tensor, *, block_rows: int = 1, rows: bool = True,
                 transposed: bool = False, dtype=torch.float8_e4m3fn, stream=None
                 ) -> Tuple[Optional[Fp8Matrix], Optional[Fp8Matrix]]:
    """(x in 8 bits, x transposed in 8 bits), each where asked for, from one
    read of x.  block_rows 1 (activations and gradients: a scale for each row
    and 128 columns) or 128 (weights: a scale for each 128 x 128)."""
    if stream is not None:
        return _on(stream, lambda: fp8_quantize(x, block_rows=block_rows, rows=rows,
                                                transposed=transposed, dtype=dtype), x)
    if dtype not in _FORMATS:
        raise ValueError("dtype: expected float8_e4m3fn or float8_e5m2")
    q, t = (_native or _load()).fp8_quantize(x, block_rows, rows, transposed,
                                             dtype == torch.float8_e5m2)
    return (None if q is None else Fp8Matrix(q[0], q[1], block_rows),
            None if t is None else Fp8Matrix(t[0], t[1], block_rows))


def fp8_matmul(a: Fp8Matrix, b: Fp8Matrix, *, dtype=torch.float32,
               out: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None
               ) -> torch.Tensor:
    """a b^T (M x N of `dtype`), or out += a b^T (accumulate, a float32 out):
    exact products, float32 sums."""
    if stream is not None:
        return _on(stream, lambda: fp8_matmul(a, b, dtype=dtype, out=out, accumulate=accumulate),
                   a, b, out)
    if dtype not in _TYPES:
        raise ValueError("dtype: expected float32, float16 or bfloat16")
    return (_native or _load()).fp8_matmul(*_fp8(a, "a"), *_fp8(b, "b"), dtype, out, accumulate,
                                           _status_word(a.data))


def fp8_linear(x: torch.Tensor, weight: Fp8Matrix, *, stream=None) -> torch.Tensor:
    """x W^T in x's type: x (.., inner) is quantised by rows, W (outer x inner)
    is kept in 8 bits by the caller (fp8_quantize(w, block_rows=128))."""
    if stream is not None:
        return _on(stream, lambda: fp8_linear(x, weight), x, weight)
    return (_native or _load()).fp8_linear(x, *_fp8(weight, "weight"), _status_word(x))


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
    _tensors(x=x)
    return (_native or _load()).fp8_linear_backward(dy, x, *_fp8(weight_t, "weight_t"), dw,
                                                    accumulate, _status_word(x))
