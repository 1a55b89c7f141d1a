"""PyTorch-side plumbing around the C ABI: device buffers for the state and
workspace blobs, stream handles, and exports.  No optimizer arithmetic here."""

from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch

from . import binding as B
from . import operators as ops


class RotatedAdam:
    """Rotated-Adam step over a fixed list of float32 matrices.

    shapes: (m, n) per matrix; c_max: micro-group byte cap; state_format:
    ROT_STATE_FULL or ROT_STATE_COMPACT (bf16 moments, fp16 bases).  The state blob
    (M, v, U, V per matrix) and the workspace blob are torch uint8 tensors on
    `device`; the library writes them through raw pointers.
    """

    def __init__(self, shapes: Sequence[Tuple[int, int]], c_max: int, device="cuda",
                 beta1=0.9, beta2=0.999, eps=1e-8, lr=1e-3, rank_rtol=1e-3,
                 precision=B.ROT_PREC_3XTF32, state_format=B.ROT_STATE_FULL):
        self.plan = B.Plan(shapes, c_max, state_format=state_format)
        self.device = torch.device(device)
        sb, wb = self.plan.state_bytes()
        self.state = torch.empty(sb, dtype=torch.uint8, device=self.device)
        self.work = torch.empty(wb, dtype=torch.uint8, device=self.device)
        self.hyper = (float(beta1), float(beta2), float(eps), float(lr))
        self.rank_rtol = float(rank_rtol)
        self.precision = int(precision)
        B.rot_state_init(self.plan, self.state.data_ptr(), self._stream())

    def _stream(self, stream=None) -> int:
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        return int(s.cuda_stream)

    def step(self, W: Sequence[torch.Tensor], G: Sequence[torch.Tensor], refresh: bool,
             stream=None, precision=None) -> None:
        for w, g, (m, n) in zip(W, G, self.plan.shapes):
            assert w.dtype == torch.float32 and g.dtype == torch.float32
            assert w.is_contiguous() and g.is_contiguous() and tuple(w.shape) == (m, n)
        b1, b2, eps, lr = self.hyper
        B.rot_step(self.plan, [w.data_ptr() for w in W], [g.data_ptr() for g in G],
                   self.state.data_ptr(), self.work.data_ptr(), b1, b2, eps, lr, refresh,
                   self.precision if precision is None else int(precision), self.rank_rtol,
                   self._stream(stream))
        # (what autograd has saved of them no longer is what they hold)
        torch.autograd.graph.increment_version([w for w in W if not w.is_inference()])

    def export(self, item: int, which: int) -> torch.Tensor:
        m, n = self.plan.shapes[item]
        shape = {B.ROT_WHICH_M: (m, n), B.ROT_WHICH_V2: (m, n), B.ROT_WHICH_U: (m, m),
                 B.ROT_WHICH_V: (n, n)}[which]
        out = torch.empty(shape, dtype=torch.float32, device=self.device)
        B.rot_state_export(self.plan, self.state.data_ptr(), item, which, out.data_ptr(),
                           self._stream())
        return out

    def ranks(self, item: int) -> Tuple[int, int]:
        return B.rot_state_ranks(self.plan, self.state.data_ptr(), item, self._stream())

    def status(self) -> int:
        return B.rot_status(self.plan, self.state.data_ptr(), self._stream())


class AdamW:
    """AdamW over the parameters that RotatedAdam does not take (vectors,
    embeddings; operators.adamw): keeps their moments and counts the steps taken
    (`count`).  Only the device knows whether a norm lets a step be taken, so
    from the first step with one the count is a tensor there.

    bits: 32 or 8, of the moments.  masters: float32 masters of 16-bit
    parameters (float16 always has one; bfloat16 without is rounded at random).
    seed: the random rounding's; instances that step in the same run need
    different ones (0 unless told otherwise).  captured: the count is on the
    device from the start, so that a captured step() counts on when it is
    replayed."""

    def __init__(self, params: Sequence[torch.Tensor], lr=1e-3, beta1: float = 0.9,
                 beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0, *,
                 bits: int = 32, masters: bool = False, seed: int = 0, captured: bool = False):
        self.params = list(params)
        states = [ops.adamw_state(p, bits=bits) for p in self.params]
        self.m, self.v = [s[0] for s in states], [s[1] for s in states]
        keep = {torch.float16: True, torch.bfloat16: masters}
        self.masters = [p.detach().float() if keep.get(p.dtype, False) else None
                        for p in self.params]
        self.lr, self.hyper = lr, dict(beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay)
        self.seed = seed
        self.count = self._on_device(0) if captured else 0

    def _on_device(self, count: int) -> torch.Tensor:
        device = self.params[0].device if self.params else "cuda"
        return torch.full((1,), count, dtype=torch.int64, device=device)

    def step(self, grads: Sequence[torch.Tensor], *, norm: Optional[torch.Tensor] = None,
             max_norm: float = 1.0, scale: float = 1.0, stream=None) -> None:
        """One step; norm, max_norm, scale as operators.adamw."""
        count = self.count
        if norm is not None and not isinstance(count, torch.Tensor):
            with torch.cuda.stream(stream):
                # (captured like this, a step has its number for good)
                if torch.cuda.is_available() and not torch.cuda.is_current_stream_capturing():
                    count = self._on_device(count)
        counts = isinstance(count, torch.Tensor)
        ops.adamw(self.params, grads, self.m, self.v, count if counts else count + 1, lr=self.lr,
                  masters=self.masters, norm=norm, max_norm=max_norm, scale=scale, seed=self.seed,
                  counts=counts, stream=stream, **self.hyper)
        self.count = count if counts else count + 1  # (of a call that was not refused)

    def moments(self, item: int) -> Tuple[torch.Tensor, torch.Tensor]:
        """(m, v) of a parameter in float32."""
        m, v = self.m[item], self.v[item]
        if isinstance(m, ops.Fp8Vector):
            return m.dequantize(), v.dequantize().square()
        return m.clone(), v.clone()
