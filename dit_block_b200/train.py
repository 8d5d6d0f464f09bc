"""ctypes binding of libsol's training operators (include/sol_train.h), same names without the
``sol_`` prefix: the gated feed-forward block, its backward pass, and AdamW.

As in :mod:`dit_block_b200.sol`: argument marshalling only, no fallback, a non-OK status raises
:class:`~dit_block_b200.sol.SolError`.  Calls run on torch's current stream of the tensors'
device unless ``stream`` is given; every tensor of a call lies on one CUDA device.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from . import sol

HEADER = os.path.join(os.path.dirname(sol.HEADER), "sol_train.h")
BLOCK = 256                  # SOL_ADAMW_BLOCK
NORM_WORKSPACE = 16384       # SOL_ADAMW_NORM_WORKSPACE

_P, _I64, _I32, _F, _D, _SZ, _E = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                                   ctypes.c_double, ctypes.c_size_t, ctypes.c_int)


class AdamwTensor(ctypes.Structure):
    """sol_adamw_tensor."""
    _fields_ = [("param", _P), ("copy", _P), ("grad", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P),
                ("n", _I64), ("weight_decay", _F)]


class AdamwScalars(ctypes.Structure):
    """sol_adamw_scalars."""
    _fields_ = [("lr", _D), ("beta1", _D), ("beta2", _D), ("eps", _D), ("step", _I64), ("seed", ctypes.c_uint64),
                ("lr_device", _P), ("step_device", _P), ("grad_factor", _P)]


SIGNATURES = {
    "sol_ffn_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "sol_ffn": ([_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _SZ, _I64, _I64, _I64, _E, _P], _E),
    "sol_ffn_backward": ([_P, _I64, _P, _I64, _P, _I64, _E, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                          _P, _SZ, _I64, _I64, _I64, _E, _P], _E),
    "sol_adamw_plan_create": ([ctypes.POINTER(_P), ctypes.POINTER(AdamwTensor), _I32, _E, _I32], _E),
    "sol_adamw_plan_destroy": ([_P], _E),
    "sol_adamw_step": ([_P, ctypes.POINTER(AdamwScalars), _P], _E),
    "sol_adamw_grad_norm": ([_P, _P, _F, _P, _SZ, _P], _E),
    "sol_adamw_state_decode": ([_P, _P, _E, _P, _P, _P, _P, _I64, _P], _E),
}

_lib = None


def lib() -> ctypes.CDLL:
    """libsol.so with the argument types of these functions set too."""
    global _lib
    if _lib is None:
        L = sol.lib()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _device(*tensors) -> torch.device:
    """The one CUDA device that all given tensors lie on."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("libsol takes CUDA tensors")
        if dev is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}: all of a call's tensors lie on one device")
        dev = t.device
    return dev


def _on(dev: torch.device):
    """Makes `dev` the current device for a call."""
    return contextlib.nullcontext() if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _matrix(name: str, t, rows: int, cols: int, *dtypes):
    if t is None:
        return
    if t.dim() != 2 or tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {list(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")


def _ld(t) -> int:
    """Row stride; a single row may have any."""
    if t is None:
        return 0
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("tensors must have unit column stride")
    return t.shape[1] if t.shape[0] <= 1 else t.stride(0)


# ---------------------------------------------------------------- gated feed-forward block

def ffn_workspace_bytes(n_tokens: int, d: int, inner: int) -> int:
    """Bytes of workspace that ffn and ffn_backward need (0: sizes they do not take)."""
    return int(lib().sol_ffn_workspace_bytes(int(n_tokens), int(d), int(inner)))


def ffn_workspace(n_tokens: int, d: int, inner: int, device=None) -> torch.Tensor:
    """A workspace for ffn and ffn_backward (uint8; torch allocations are 256-byte aligned)."""
    nb = ffn_workspace_bytes(n_tokens, d, inner)
    if nb == 0:
        raise ValueError("d and inner must be multiples of 8, n_tokens >= 0")
    return torch.empty((nb,), dtype=torch.uint8, device=device or "cuda")


def ffn(y, x, w_up, w_down, *, u=None, workspace, stream=None):
    """y = (silu(a) * b) . W_down^T with [a | b] = x . W_up^T  (sol_ffn); u, if given, receives
    [a | b] for ffn_backward.  x, y [n, d], w_up [2 * inner, d], w_down [d, inner], u [n, 2 * inner], bf16."""
    bf = torch.bfloat16
    n, d = x.shape
    inner = w_down.shape[1]
    for name, t, r, c in (("x", x, n, d), ("y", y, n, d), ("w_up", w_up, 2 * inner, d), ("w_down", w_down, d, inner),
                          ("u", u, n, 2 * inner)):
        _matrix(name, t, r, c, bf)
    dev = _device(x, y, w_up, w_down, u, workspace)
    with _on(dev):
        sol._check(lib().sol_ffn(sol._ptr(y), _ld(y), sol._ptr(u), _ld(u), sol._ptr(x), _ld(x), sol._ptr(w_up), _ld(w_up),
                                 sol._ptr(w_down), _ld(w_down), sol._ptr(workspace),
                                 workspace.numel() * workspace.element_size(), n, d, inner, sol.BF16,
                                 sol._stream(stream)), "sol_ffn")
    return y


def ffn_backward(dy, x, u, w_up, w_down, *, dx=None, dw_up=None, dw_down=None, accumulate=False, workspace,
                 stream=None):
    """Gradients of ffn from dy and the u that it kept (sol_ffn_backward): dx [n, d] bf16, dw_up and
    dw_down in bf16 or f32 (both of one type), each only where given; accumulate adds to the
    weight gradients' contents."""
    bf, f32 = torch.bfloat16, torch.float32
    n, d = x.shape
    inner = w_down.shape[1]
    for name, t, r, c in (("dy", dy, n, d), ("x", x, n, d), ("u", u, n, 2 * inner), ("w_up", w_up, 2 * inner, d),
                          ("w_down", w_down, d, inner), ("dx", dx, n, d)):
        _matrix(name, t, r, c, bf)
    _matrix("dw_up", dw_up, 2 * inner, d, bf, f32)
    _matrix("dw_down", dw_down, d, inner, bf, f32)
    types = {t.dtype for t in (dw_up, dw_down) if t is not None}
    if len(types) > 1:
        raise TypeError("dw_up and dw_down must have one type")
    grad_dt = sol.F32 if types == {f32} else sol.BF16
    dev = _device(dy, x, u, w_up, w_down, dx, dw_up, dw_down, workspace)
    with _on(dev):
        sol._check(lib().sol_ffn_backward(
            sol._ptr(dx), _ld(dx), sol._ptr(dw_up), _ld(dw_up), sol._ptr(dw_down), _ld(dw_down), grad_dt,
            int(bool(accumulate)), sol._ptr(dy), _ld(dy), sol._ptr(x), _ld(x), sol._ptr(u), _ld(u), sol._ptr(w_up),
            _ld(w_up), sol._ptr(w_down), _ld(w_down), sol._ptr(workspace), workspace.numel() * workspace.element_size(),
            n, d, inner, sol.BF16, sol._stream(stream)), "sol_ffn_backward")


# ---------------------------------------------------------------------------------- AdamW

def _flat(name, t, n, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} values")


class AdamW:
    """A plan of AdamW steps over many tensors (sol_adamw_plan_create), which holds the tensors.

    params f32, grads all f32 or all bf16, m and v f32, or int8 and uint8 with one f32 scale a block of
    256 values in m_scales / v_scales (zeros to begin with); copies: bf16 tensors (or None for
    some) that receive the updated parameters.  weight_decay: one number, or one a tensor.
    All contiguous, on one device, 16-byte aligned."""

    def __init__(self, params, grads, m, v, *, m_scales=None, v_scales=None, copies=None, weight_decay=0.0):
        self._handle = None
        n = len(params)
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(w) for w in weight_decay]
        copies = [None] * n if copies is None else list(copies)
        bits = 8 if m_scales is not None else 32
        scales = [(None, None)] * n if bits == 32 else list(zip(m_scales, v_scales or []))
        if not len(grads) == len(m) == len(v) == len(copies) == len(decay) == len(scales) == n:
            raise ValueError("params, grads, m, v, their scales, copies and weight_decay must have one entry a tensor")
        grad_type = grads[0].dtype if n else torch.float32
        if grad_type not in (torch.float32, torch.bfloat16):
            raise TypeError(f"gradients must be float32 or bfloat16, got {grad_type}")
        rows = (AdamwTensor * max(n, 1))()
        kept = []
        for i in range(n):
            k = params[i].numel()
            _flat("param", params[i], k, torch.float32)
            _flat("grad", grads[i], k, grad_type)
            _flat("m", m[i], k, torch.int8 if bits == 8 else torch.float32)
            _flat("v", v[i], k, torch.uint8 if bits == 8 else torch.float32)
            if copies[i] is not None:
                _flat("copy", copies[i], k, torch.bfloat16)
            for s in scales[i]:
                if bits == 8:
                    _flat("scale", s, -(-k // BLOCK), torch.float32)
            one = (params[i], copies[i], grads[i], m[i], v[i], *scales[i])
            kept.append(one)
            rows[i] = AdamwTensor(*(sol._ptr(t) for t in one), k, decay[i])
        self._kept = kept
        self.device = _device(*(t for one in kept for t in one)) or torch.device("cuda", torch.cuda.current_device())
        h = _P()
        with _on(self.device):
            sol._check(lib().sol_adamw_plan_create(ctypes.byref(h), rows, n,
                                                   sol.BF16 if grad_type == torch.bfloat16 else sol.F32, bits),
                       "sol_adamw_plan_create")
        self._handle = h.value

    def step(self, *, lr, betas=(0.9, 0.999), eps=1e-8, step, seed=0, lr_device=None, step_device=None,
             grad_factor=None, stream=None):
        """One step (sol_adamw_step).  lr_device (f32) and step_device (int64) are device scalars read in place
        of lr and step when the step runs; grad_factor (f32) multiplies the gradients."""
        for name, t, dtype in (("lr_device", lr_device, torch.float32), ("step_device", step_device, torch.int64),
                               ("grad_factor", grad_factor, torch.float32)):
            if t is not None:
                _flat(name, t, 1, dtype)
                if t.device != self.device:
                    raise ValueError(f"{name} must lie on {self.device}")
        h = AdamwScalars(float(lr), float(betas[0]), float(betas[1]), float(eps), int(step), int(seed) & (2 ** 64 - 1),
                         sol._ptr(lr_device), sol._ptr(step_device), sol._ptr(grad_factor))
        with _on(self.device):
            sol._check(lib().sol_adamw_step(self._handle, ctypes.byref(h), sol._stream(stream)), "sol_adamw_step")

    def norm_workspace(self) -> torch.Tensor:
        """A workspace for grad_norm (one for each of the calls that may overlap)."""
        return torch.empty(NORM_WORKSPACE, dtype=torch.uint8, device=self.device)

    def grad_norm(self, out, max_norm, *, workspace, stream=None):
        """out[0] = norm of all gradients, out[1] = min(1, max_norm / (out[0] + 1e-6))  (sol_adamw_grad_norm)."""
        _flat("out", out, 2, torch.float32)
        if _device(out, workspace) != self.device:
            raise ValueError(f"out and workspace must lie on {self.device}")
        with _on(self.device):
            sol._check(lib().sol_adamw_grad_norm(sol._ptr(out), self._handle, float(max_norm), sol._ptr(workspace),
                                                 workspace.numel() * workspace.element_size(), sol._stream(stream)),
                       "sol_adamw_grad_norm")
        return out

    def close(self):
        """Frees the plan: its steps have ended, and no captured graph that uses it is replayed any more."""
        if self._handle:
            h, self._handle = self._handle, None
            with _on(self.device):
                sol._check(lib().sol_adamw_plan_destroy(h), "sol_adamw_plan_destroy")
            self._kept = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def adamw_state_decode(m_out, v_out, m, v, m_scale, v_scale, *, stream=None):
    """The values that 8-bit moments stand for (sol_adamw_state_decode); m_out and v_out (either may be
    None) share one type, f32 or bf16."""
    outs = [t for t in (m_out, v_out) if t is not None]
    if not outs:
        return
    n = outs[0].numel()
    for name, out, q, s, dtype in (("m", m_out, m, m_scale, torch.int8), ("v", v_out, v, v_scale, torch.uint8)):
        if out is not None:
            _flat(name + "_out", out, n, outs[0].dtype)
            _flat(name, q, n, dtype)
            _flat(name + "_scale", s, -(-n // BLOCK), torch.float32)
    dev = _device(*outs, *(t for o, q, s in ((m_out, m, m_scale), (v_out, v, v_scale)) if o is not None for t in (q, s)))
    with _on(dev):
        sol._check(lib().sol_adamw_state_decode(sol._ptr(m_out), sol._ptr(v_out), sol._dtype(outs[0]), sol._ptr(m),
                                                sol._ptr(v), sol._ptr(m_scale), sol._ptr(v_scale), n, sol._stream(stream)),
                   "sol_adamw_state_decode")
