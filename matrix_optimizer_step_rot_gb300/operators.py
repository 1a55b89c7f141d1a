"""Training operators next to the optimizer step, on torch tensors.

Dropout from a counter-based generator, layer norm with the residual stream and
dropout in front of it, rotary positions and the norm of queries and keys, the
clipped policy loss with its gradient, linear layers in 8-bit floating point
with power-of-two block scales, and AdamW over many tensors with the norm of
their gradients.  Between them they carry a training step from hidden states to
the float32 gradients that `optimizer.RotatedAdam` reads, and step the
parameters that it does not take.  include/rot_ops.h states the formulas, layouts
and errors.  Every function checks its tensors (ValueError), allocates its
outputs and workspace with torch and runs the library's kernels on the current
stream (csrc/torch/torch_ops.cpp), or on `stream` (a torch.cuda.Stream: outputs
and workspaces then belong to it, and the inputs are marked as used on it;
ordering it after their producers is the caller's).  Tensors are on the current
device; a tensor of more than two dimensions is rows of its last one.  There is
no other path than the library's, and no part in torch's autograd: results do
not require gradients, whatever the inputs do, and the backward functions are
calls of their own, as the optimizer step is (examples/policy_step.py has them
together); but what a call writes in place (moments aside) has its version
counter moved on, so that a backward pass of torch that saved it fails.  New
tensors come from torch's CUDA allocator without its dispatcher: dispatch modes
do not see them, and deterministic mode does not fill them before they are
written.  The first 8-bit product on a device allocates its status word: let it
run before a stream capture.
"""

from __future__ import annotations

import ctypes
import math
import threading
from typing import NamedTuple, Optional, Sequence, Tuple, Union

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
                     for n in B.header_symbols()}, B.RotError, Fp8Vector)
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
        for u in t if isinstance(t, (tuple, list)) else (t,):
            if isinstance(u, tuple):
                for w in u:
                    if isinstance(w, torch.Tensor):
                        w.record_stream(stream)
            elif isinstance(u, torch.Tensor):
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
# heads: rotary positions, norm of queries and keys
# ---------------------------------------------------------------------------


class Rotary(NamedTuple):
    """What the heads of a model are rotated by: `turns` (int64, one for each
    pair: the part of a turn that a position adds, in units of 2^-64), a factor
    on the rotated pairs, and whether the pairs are neighbours (2i, 2i + 1) or
    (i, i + pairs).  A head's elements past the pairs are not rotated."""
    turns: torch.Tensor
    magnitude: float = 1.0
    interleaved: bool = False


def rotary_frequencies(rotated: int, base: float = 10000.0, *, factor: float = 1.0,
                       original_length: Optional[float] = None, low: float = 1.0,
                       high: float = 4.0, by_index: bool = False) -> torch.Tensor:
    """Radians that a position adds, for each pair of `rotated` elements
    (float64): base^(-2i / rotated).  For contexts `factor` times as long: all
    of them divided by it; or, with the original length, those pairs alone that
    make at most `low` turns over it, while those of `high` and more keep
    theirs, with a straight line in between over the turns, or over the pairs'
    indices (by_index)."""
    if rotated < 0 or rotated % 2:
        raise ValueError("rotated: expected an even number of elements")
    if not (base > 0 and factor > 0):
        raise ValueError("base, factor: expected numbers above 0")
    f = base ** (-torch.arange(0, rotated, 2, dtype=torch.float64) / max(rotated, 1))
    if original_length is None:
        return f / factor
    if not (original_length > 0 and 0 < low < high):
        raise ValueError("original_length, low, high: expected a length above 0 and 0 < low < high")
    turns = f * original_length / (2 * math.pi)
    if by_index:  # (turns fall with the index as a power of the base)
        keep = torch.log(turns / low) / math.log(high / low)
    else:
        keep = (turns - low) / (high - low)
    keep = keep.clamp(0, 1)
    return f * (keep + (1 - keep) / factor)


def rotary_table(frequencies, *, magnitude: float = 1.0, interleaved: bool = False,
                 device="cuda") -> Rotary:
    """A Rotary from radians per position (numbers, or a tensor; float64).  The
    turns hold the 53 bits of a float64 quotient: an angle at position p is off
    by at most p 2^-52 of its frequency, and by nothing that grows with p beyond
    that."""
    if isinstance(frequencies, torch.Tensor):
        frequencies = frequencies.double().tolist()
    words = []
    for f in frequencies:
        x = f / (2 * math.pi)
        n = round((x - math.floor(x)) * 2.0 ** 64) % (1 << 64)
        words.append(n - (1 << 64) if n >= 1 << 63 else n)
    return Rotary(torch.tensor(words, dtype=torch.int64, device=device), magnitude, interleaved)


def _rotary(r, required: bool):
    if r is None and not required:
        return None, 1.0, False
    if not isinstance(r, Rotary) or not isinstance(r.turns, torch.Tensor):
        raise ValueError(f"rotary: expected a Rotary, got {type(r).__name__}")
    return r


def rotate(q: torch.Tensor, rotary: Rotary, k: Optional[torch.Tensor] = None, *,
           positions: Optional[torch.Tensor] = None, start: int = 0,
           out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None
           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(q, k) turned by their tokens' positions.  [tokens, heads, dim] or
    [batch, tokens, heads, dim] of any strides (heads before tokens: pass the
    transposed view), a head's elements next to one another.  positions (int64
    or int32): one for each token, or [tokens] for all batch entries; without,
    token t is at start + t.  out, k_out: written instead of new tensors; may be
    q and k themselves, each its own, and nothing else that the call reads or
    writes."""
    if stream is not None:
        return _on(stream, lambda: rotate(q, rotary, k, positions=positions, start=start, out=out,
                                          k_out=k_out), q, rotary, k, positions, out, k_out)
    _tensors(q=q)
    return (_native or _load()).rotate(q, k, *_rotary(rotary, True), positions, start, False, out,
                                       k_out)


def rotate_backward(dq: torch.Tensor, rotary: Rotary, dk: Optional[torch.Tensor] = None, *,
                    positions: Optional[torch.Tensor] = None, start: int = 0,
                    out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gradients of rotate()'s q and k from those of its results: turned
    back, with the same magnitude."""
    if stream is not None:
        return _on(stream, lambda: rotate_backward(dq, rotary, dk, positions=positions,
                                                   start=start, out=out, k_out=k_out),
                   dq, rotary, dk, positions, out, k_out)
    _tensors(dq=dq)
    return (_native or _load()).rotate(dq, dk, *_rotary(rotary, True), positions, start, True, out,
                                       k_out)


def head_norm(q: torch.Tensor, q_weight: torch.Tensor, k: Optional[torch.Tensor] = None,
              k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
              rotary: Optional[Rotary] = None, positions: Optional[torch.Tensor] = None,
              start: int = 0, out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None, stream=None
              ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(q, k), each head x as x / sqrt(mean(x^2) + eps) weight, rotated behind
    that where `rotary` is given, in one pass.  Layouts, positions and outputs
    as rotate().  Weights: dim elements, float32 or q's type."""
    if stream is not None:
        return _on(stream, lambda: head_norm(q, q_weight, k, k_weight, eps, rotary=rotary,
                                             positions=positions, start=start, out=out,
                                             k_out=k_out),
                   q, q_weight, k, k_weight, rotary, positions, out, k_out)
    _tensors(q=q, q_weight=q_weight)
    return (_native or _load()).head_norm(q, q_weight, k, k_weight, eps, *_rotary(rotary, False),
                                          positions, start, out, k_out)


def head_norm_backward(dq: torch.Tensor, q: torch.Tensor, q_weight: torch.Tensor,
                       dk: Optional[torch.Tensor] = None, k: Optional[torch.Tensor] = None,
                       k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                       rotary: Optional[Rotary] = None, positions: Optional[torch.Tensor] = None,
                       start: int = 0, out: Optional[torch.Tensor] = None,
                       k_out: Optional[torch.Tensor] = None, stream=None
                       ) -> Tuple[torch.Tensor, Optional[torch.Tensor], torch.Tensor,
                                  Optional[torch.Tensor]]:
    """(dq, dk, dq_weight, dk_weight) of head_norm from the gradients of its
    results and its inputs.  The weights' gradients are float32: sums over all
    tokens and heads.  out, k_out: written instead of new dq and dk; may be the
    given gradients."""
    if stream is not None:
        return _on(stream, lambda: head_norm_backward(dq, q, q_weight, dk, k, k_weight, eps,
                                                      rotary=rotary, positions=positions,
                                                      start=start, out=out, k_out=k_out),
                   dq, q, q_weight, dk, k, k_weight, rotary, positions, out, k_out)
    _tensors(dq=dq, q=q, q_weight=q_weight)
    return (_native or _load()).head_norm_backward(dq, q, q_weight, dk, k, k_weight, eps,
                                                   *_rotary(rotary, False), positions, start, out,
                                                   k_out)


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


# ---------------------------------------------------------------------------
# AdamW over many tensors
# ---------------------------------------------------------------------------


class Fp8Vector(NamedTuple):
    """Elements in 8 bits: `data` (float8_e4m3fn, any shape) under one
    power-of-two scale (uint8, a byte e for 2^(e - 127), 255 for NaN) for every
    128 consecutive elements."""
    data: torch.Tensor
    scale: torch.Tensor

    def dequantize(self) -> torch.Tensor:
        """The float32 tensor it stands for (a diagnostic, in torch)."""
        e = self.scale.int()
        s = torch.where(e > 0, e << 23, 1 << 22).view(torch.float32)
        s = torch.where(e == 255, float("nan"), s).repeat_interleave(128)
        return (self.data.float().flatten() * s[:self.data.numel()]).view(self.data.shape)


State = Union[torch.Tensor, Fp8Vector]


def adamw_state(param: torch.Tensor, *, bits: int = 32) -> Tuple[State, State]:
    """(m, v) of a parameter before its first step: zeros, in float32 or (bits
    8) as Fp8Vectors, v's of its root."""
    if bits == 32:
        return (torch.zeros(param.shape, dtype=torch.float32, device=param.device),
                torch.zeros(param.shape, dtype=torch.float32, device=param.device))
    if bits != 8:
        raise ValueError("bits: expected 32 or 8")
    blocks = -(-param.numel() // 128)
    return tuple(Fp8Vector(torch.zeros(param.shape, dtype=torch.uint8, device=param.device)
                           .view(torch.float8_e4m3fn),
                           torch.zeros(blocks, dtype=torch.uint8, device=param.device))
                 for _ in range(2))


def gradient_norm(grads: Sequence[torch.Tensor], *, stream=None) -> torch.Tensor:
    """The root of the sum of all elements' squares (float32, on the device):
    contiguous tensors of any types and shapes, in two launches for up to a
    thousand of them."""
    if stream is not None:
        grads = list(grads)  # (read twice)
        return _on(stream, lambda: gradient_norm(grads), grads)
    return (_native or _load()).gradient_norm(grads)


def adamw(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], m: Sequence[State],
          v: Sequence[State], step, *, lr, beta1: float = 0.9, beta2: float = 0.999,
          eps: float = 1e-8, weight_decay: float = 0.0,
          masters: Optional[Sequence[Optional[torch.Tensor]]] = None,
          norm: Optional[torch.Tensor] = None, max_norm: float = 1.0, scale: float = 1.0,
          seed: int = 0, counts: bool = False, stream=None) -> None:
    """One AdamW step of all `params`, in place, with their states and masters:
    contiguous tensors of any shapes; float32 (and bfloat16, rounded at random)
    parameters, or 16-bit ones with a float32 master; gradients of any type;
    states as adamw_state() makes them.  Gradients are multiplied by `scale`,
    and clipped to max_norm where `norm` (gradient_norm()'s of them before
    `scale`) is given; where |scale| norm is not finite everything stays as it
    was.  step counts from 1; it and lr may be tensors of one element on the
    device (int64, float32), which a captured call reads when it is replayed.
    counts: step, a tensor, holds the steps taken so far, this call is the one
    after them, and it moves step on unless the norm has it not taken.  seed:
    the random rounding's, whose other half is the step: calls of the same step
    need different ones.  What is written must not overlap (one tensor twice is
    refused, views a part on are not noticed)."""
    if stream is not None:
        params, grads, m, v = list(params), list(grads), list(m), list(v)  # (read twice)
        masters = None if masters is None else list(masters)
        return _on(stream, lambda: adamw(params, grads, m, v, step, lr=lr, beta1=beta1,
                                         beta2=beta2, eps=eps, weight_decay=weight_decay,
                                         masters=masters, norm=norm, max_norm=max_norm,
                                         scale=scale, seed=seed, counts=counts),
                   params, grads, m, v, masters, norm, step, lr)
    on = isinstance(step, torch.Tensor), isinstance(lr, torch.Tensor)
    (_native or _load()).adamw(params, grads, m, v, masters, 1 if on[0] else step,
                               step if on[0] else None, counts, 0.0 if on[1] else lr,
                               lr if on[1] else None, beta1, beta2, eps, weight_decay, norm,
                               max_norm, scale, _word(seed, "seed"))
