"""Fine-tuning the feed-forward of a DiT block: what a training step keeps on the GPU, and the step itself.

    y   = (silu(x Wg^T) * (x Wu^T)) Wd^T, u kept              forward        (sol_ffn)
    dx, dW_up (+)=, dW_down (+)=                               backward       (sol_ffn_backward)
    norm of both gradients and its clip factor, then AdamW     update         (sol_adamw_grad_norm, sol_adamw_step)

The parameters are f32; the products read bf16 copies that each update writes.  The two moments of every
parameter take 8 bytes (f32) or 2 (8 bits a value).  All buffers are made once, for up to ``max_tokens``
tokens; no call allocates, and the learning rate and the number of the step are read on the device, so that a
step can be captured in a CUDA graph and replayed (``capture``).
"""
from __future__ import annotations

import torch

from . import train

BF16 = torch.bfloat16


class StepGraph(torch.cuda.CUDAGraph):
    """A captured training step, and what its replays read."""

    reads: tuple

    def replay(self) -> None:
        super().replay()
        self.reads[0]._x = None  # its u is no longer that of an eager forward


class FeedForward:
    """A gated feed-forward block in training: w_up [2 * inner, d] (gated half first), w_down [d, inner]."""

    def __init__(self, w_up: torch.Tensor, w_down: torch.Tensor, max_tokens: int, *, state_bits: int = 32,
                 grad_dtype: torch.dtype = torch.float32, weight_decay: float = 0.0, betas=(0.9, 0.999),
                 eps: float = 1e-8, seed: int = 0):
        d, inner = w_down.shape
        if tuple(w_up.shape) != (2 * inner, d):
            raise ValueError(f"w_up must be [{2 * inner}, {d}], got {list(w_up.shape)}")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        dev = w_up.device
        self.d, self.inner, self.max_tokens = d, inner, max_tokens
        self.betas, self.eps, self.seed, self.state_bits = betas, eps, seed, state_bits
        self.params = [w.detach().to(torch.float32, copy=True).contiguous() for w in (w_up, w_down)]
        self.weights = [p.to(BF16) for p in self.params]
        self.grads = [torch.zeros(p.shape, dtype=grad_dtype, device=dev) for p in self.params]
        first, second = (torch.int8, torch.uint8) if state_bits == 8 else (torch.float32, torch.float32)
        self.m = [torch.zeros(p.shape, dtype=first, device=dev) for p in self.params]
        self.v = [torch.zeros(p.shape, dtype=second, device=dev) for p in self.params]
        scales = lambda: None if state_bits == 32 else [  # noqa: E731
            torch.zeros(-(-p.numel() // train.BLOCK), dtype=torch.float32, device=dev) for p in self.params]
        self.m_scales, self.v_scales = scales(), scales()
        self.optimizer = train.AdamW(self.params, self.grads, self.m, self.v, m_scales=self.m_scales,
                                     v_scales=self.v_scales, copies=self.weights, weight_decay=weight_decay)
        self.workspace = train.ffn_workspace(max_tokens, d, inner, device=dev)
        self.norm_workspace = self.optimizer.norm_workspace()
        empty = lambda cols: torch.empty((max_tokens, cols), dtype=BF16, device=dev)  # noqa: E731
        self.y, self.u, self.dx = empty(d), empty(2 * inner), empty(d)
        self.norm = torch.zeros(2, dtype=torch.float32, device=dev)  # of the last update's gradients, and its clip factor
        self.lr = torch.zeros(1, dtype=torch.float32, device=dev)
        self.step = torch.zeros(1, dtype=torch.int64, device=dev)
        self._x = None

    def infer(self, x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """y for x [n, d], nothing kept."""
        y = self.y[:x.shape[0]] if out is None else out
        return train.ffn(y, x, *self.weights, workspace=self.workspace)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """y for x [n, d], n <= max_tokens; keeps the pre-activation, and x itself (no copy, so it must stay as it is),
        for backward.  y lies in this object's buffer, which the next forward or infer writes."""
        n = x.shape[0]
        if n > self.max_tokens:
            raise ValueError(f"{n} tokens are more than max_tokens ({self.max_tokens})")
        y = train.ffn(self.y[:n], x, *self.weights, u=self.u[:n], workspace=self.workspace)
        self._x = x  # a call that was refused has not touched u
        return y

    def backward(self, dy: torch.Tensor, accumulate: bool = False) -> torch.Tensor:
        """dx (in this object's buffer) of the last forward's tokens; the weight gradients are set, or with accumulate added to."""
        if self._x is None:
            raise RuntimeError("backward needs a forward before it")
        n = self._x.shape[0]
        train.ffn_backward(dy, self._x, self.u[:n], *self.weights, dx=self.dx[:n], dw_up=self.grads[0],
                           dw_down=self.grads[1], accumulate=accumulate, workspace=self.workspace)
        return self.dx[:n]

    def update(self, max_norm: float = float("inf")) -> None:
        """One AdamW step at the learning rate ``self.lr`` holds, this block's gradients clipped to a norm of max_norm
        (infinite: not clipped; ``self.norm`` is measured all the same)."""
        self.optimizer.grad_norm(self.norm, max_norm, workspace=self.norm_workspace)
        self.step.add_(1)
        try:
            self.optimizer.step(lr=0.0, betas=self.betas, eps=self.eps, step=1, seed=self.seed, lr_device=self.lr,
                                step_device=self.step, grad_factor=self.norm[1:])
        except Exception:
            self.step.sub_(1)  # a refused step does not count
            raise

    def capture(self, x: torch.Tensor, dy: torch.Tensor, max_norm: float = float("inf")) -> torch.cuda.CUDAGraph:
        """A CUDA graph of forward, backward and update over the buffers x and dy, whose contents and ``self.lr``
        may change between replays.  Nothing runs now, and the last forward stays the one that ``backward`` belongs to;
        after a replay ``backward`` needs a forward of its own.
        The graph uses this object's buffers: replays must not overlap its other calls, and it must not outlive
        ``close``.  It keeps this object, x and dy alive."""
        g = StepGraph()
        g.reads = (self, x, dy)
        last = self._x
        try:
            with torch.cuda.device(self.lr.device), torch.cuda.graph(g):
                self.forward(x)
                self.backward(dy)
                self.update(max_norm)
        finally:
            self._x = last
        return g

    def moments(self, dtype: torch.dtype = torch.float32):
        """Copies of the moments as values: [(m, v), ...] of w_up and w_down."""
        if self.state_bits == 32:
            return [(m.to(dtype, copy=True), v.to(dtype, copy=True)) for m, v in zip(self.m, self.v)]
        out = []
        for q, r, s, t in zip(self.m, self.v, self.m_scales, self.v_scales):
            m, v = (torch.empty(q.shape, dtype=dtype, device=q.device) for _ in range(2))
            train.adamw_state_decode(m, v, q, r, s, t)
            out.append((m, v))
        return out

    def close(self) -> None:
        self.optimizer.close()
