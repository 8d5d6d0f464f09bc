"""ctypes binding of libsol's training operators (include/sol_train.h), same names without the
``sol_`` prefix: the gated feed-forward block, its backward pass, and AdamW.

As in :mod:`dit_block_b200.sol`: argument marshalling only, no fallback, a non-OK status raises
:class:`~dit_block_b200.sol.SolError`.  Calls run on torch's current stream of the tensors'
device unless ``stream`` is given; every tensor of a call lies on one CUDA device.
"""
from __future__ import annotations

import ctypes
import os
import struct

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


def _rows(*names):
    return [f for n, ld in names for f in ((n, _P), (ld, _I64))]


class FfnDesc(ctypes.Structure):
    """sol_ffn_desc."""
    _fields_ = [*_rows(("y", "ld_y"), ("u", "ld_u"), ("x", "ld_x"), ("w_up", "ld_wu"), ("w_down", "ld_wd")),
                ("workspace", _P), ("workspace_bytes", _SZ), ("n_tokens", _I64), ("d", _I64), ("inner", _I64), ("dt", _E)]


class FfnBackwardDesc(ctypes.Structure):
    """sol_ffn_backward_desc."""
    _fields_ = [*_rows(("dx", "ld_dx"), ("dw_up", "ld_dwu"), ("dw_down", "ld_dwd"), ("dy", "ld_dy"), ("x", "ld_x"),
                       ("u", "ld_u"), ("w_up", "ld_wu"), ("w_down", "ld_wd")),
                ("workspace", _P), ("workspace_bytes", _SZ), ("n_tokens", _I64), ("d", _I64), ("inner", _I64), ("dt", _E),
                ("grad_dt", _E), ("accumulate", _I32)]


def _packer(form: str, of) -> struct.Struct:
    """The bytes of a ctypes structure from its fields, in a third of the time."""
    s = struct.Struct(form + "0q")  # with the structure's alignment at its end
    assert s.size == ctypes.sizeof(of)
    return s.pack


_pack_scalars = _packer("4dqQ3P", AdamwScalars)
_pack_ffn = _packer("PqPqPqPqPqPN3qi", FfnDesc)
_pack_ffn_backward = _packer("PqPqPqPqPqPqPqPqPN3q3i", FfnBackwardDesc)


SIGNATURES = {
    "sol_ffn_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "sol_ffn": ([_P, _P], _E),           # sol_ffn_desc, stream
    "sol_ffn_backward": ([_P, _P], _E),  # sol_ffn_backward_desc, stream
    "sol_adamw_plan_create": ([ctypes.POINTER(_P), ctypes.POINTER(AdamwTensor), _I32, _E, _I32], _E),
    "sol_adamw_plan_destroy": ([_P], _E),
    "sol_adamw_step": ([_P, _P, _P], _E),  # plan, sol_adamw_scalars, stream
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


def _call(name: str, device: int, stream, *args):
    """Calls a function whose last argument is the stream, with `device` the current one."""
    fn = getattr(_lib or lib(), name)
    stream = torch._C._cuda_getCurrentRawStream(device) if stream is None else sol._stream(stream)
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status:
        sol._check(status, name)


def _device(t) -> int:
    """The index of the CUDA device that a call's first tensor lies on; the others must lie there too."""
    device = t.get_device()
    if device < 0 or not t.is_cuda:
        raise ValueError("libsol takes CUDA tensors")
    return device


def _matrix(name: str, t, rows: int, cols: int, dtype, device: int):
    """(address, row stride) of a [rows, cols] argument; a single row may have any stride."""
    if t.dtype is dtype and t.shape == (rows, cols) and t.get_device() == device and t.is_contiguous():
        return t.data_ptr(), cols
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {list(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on device {device}, as the call's other tensors")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), s0 if rows > 1 else cols


def _space(workspace, device: int):
    if workspace.get_device() != device:
        raise ValueError(f"workspace must be a CUDA tensor on device {device}, as the call's other tensors")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.nbytes


_NONE = (0, 0)


# ---------------------------------------------------------------- gated feed-forward block

def ffn_workspace_bytes(n_tokens: int, d: int, inner: int) -> int:
    """Bytes of workspace that ffn and ffn_backward need (0: sizes they do not take)."""
    return int(lib().sol_ffn_workspace_bytes(int(n_tokens), int(d), int(inner)))


def ffn_workspace(n_tokens: int, d: int, inner: int, device=None) -> torch.Tensor:
    """A workspace for ffn and ffn_backward (uint8; torch allocations are 256-byte aligned)."""
    nb = ffn_workspace_bytes(n_tokens, d, inner)
    if nb == 0:
        raise ValueError("d and inner must be multiples of 8, n_tokens >= 0")
    return torch.empty((nb,), dtype=torch.uint8, device="cuda" if device is None else device)


def ffn(y, x, w_up, w_down, *, u=None, workspace, stream=None):
    """y = (silu(a) * b) . W_down^T with [a | b] = x . W_up^T  (sol_ffn); u, if given, receives
    [a | b] for ffn_backward.  x, y [n, d], w_up [2 * inner, d], w_down [d, inner], u [n, 2 * inner], bf16."""
    bf = torch.bfloat16
    n, d = x.shape
    inner = w_down.shape[1]
    dev = _device(x)
    desc = _pack_ffn(*_matrix("y", y, n, d, bf, dev), *(_NONE if u is None else _matrix("u", u, n, 2 * inner, bf, dev)),
                     *_matrix("x", x, n, d, bf, dev), *_matrix("w_up", w_up, 2 * inner, d, bf, dev),
                     *_matrix("w_down", w_down, d, inner, bf, dev), *_space(workspace, dev), n, d, inner, sol.BF16)
    _call("sol_ffn", dev, stream, desc)
    return y


def ffn_backward(dy, x, u, w_up, w_down, *, dx=None, dw_up=None, dw_down=None, accumulate=False, workspace,
                 stream=None):
    """Gradients of ffn from dy and the u that it kept (sol_ffn_backward): dx [n, d] bf16, dw_up and
    dw_down in bf16 or f32 (both of one type), each only where given; accumulate adds to the
    weight gradients' contents."""
    bf = torch.bfloat16
    n, d = x.shape
    inner = w_down.shape[1]
    grad = bf if dw_up is None and dw_down is None else (dw_down if dw_up is None else dw_up).dtype
    if grad is not bf and grad is not torch.float32:
        raise TypeError(f"dw_up and dw_down must be torch.bfloat16 or torch.float32, got {grad}")
    dev = _device(x)
    desc = _pack_ffn_backward(
        *(_NONE if dx is None else _matrix("dx", dx, n, d, bf, dev)),
        *(_NONE if dw_up is None else _matrix("dw_up", dw_up, 2 * inner, d, grad, dev)),
        *(_NONE if dw_down is None else _matrix("dw_down", dw_down, d, inner, grad, dev)),
        *_matrix("dy", dy, n, d, bf, dev), *_matrix("x", x, n, d, bf, dev), *_matrix("u", u, n, 2 * inner, bf, dev),
        *_matrix("w_up", w_up, 2 * inner, d, bf, dev), *_matrix("w_down", w_down, d, inner, bf, dev),
        *_space(workspace, dev), n, d, inner, sol.BF16, sol.BF16 if grad is bf else sol.F32, 1 if accumulate else 0)
    _call("sol_ffn_backward", dev, stream, desc)


# ---------------------------------------------------------------------------------- AdamW

def _flat(name, t, n, dtype, device: int):
    """Address of a contiguous argument of n values."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} values")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on device {device}, as the call's other tensors")
    return t.data_ptr()


class AdamW:
    """A plan of AdamW steps over many tensors (sol_adamw_plan_create), which holds the tensors: each step reads
    these gradients, written anew.

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
        dev = _device(params[0]) if n else torch.cuda.current_device()
        first, second = (torch.int8, torch.uint8) if bits == 8 else (torch.float32, torch.float32)
        for i in range(n):
            k = params[i].numel()
            blocks = -(-k // BLOCK)
            rows[i] = AdamwTensor(
                _flat("param", params[i], k, torch.float32, dev),
                None if copies[i] is None else _flat("copy", copies[i], k, torch.bfloat16, dev),
                _flat("grad", grads[i], k, grad_type, dev), _flat("m", m[i], k, first, dev), _flat("v", v[i], k, second, dev),
                *(None if s is None else _flat("scale", s, blocks, torch.float32, dev) for s in scales[i]), k, decay[i])
        self._kept = (list(params), list(grads), list(m), list(v), copies, scales)
        self.device = torch.device("cuda", dev)
        self._index = dev
        h = _P()
        with torch.cuda.device(dev):
            sol._check(lib().sol_adamw_plan_create(ctypes.byref(h), rows, n,
                                                   sol.BF16 if grad_type == torch.bfloat16 else sol.F32, bits),
                       "sol_adamw_plan_create")
        self._handle = h.value

    def step(self, *, lr, betas=(0.9, 0.999), eps=1e-8, step, seed=0, lr_device=None, step_device=None,
             grad_factor=None, stream=None):
        """One step (sol_adamw_step).  lr_device (f32) and step_device (int64) are device scalars read in place
        of lr and step when the step runs; grad_factor (f32) multiplies the gradients."""
        dev = self._index
        h = _pack_scalars(lr, betas[0], betas[1], eps, step, seed & 0xFFFFFFFFFFFFFFFF,
                          0 if lr_device is None else _flat("lr_device", lr_device, 1, torch.float32, dev),
                          0 if step_device is None else _flat("step_device", step_device, 1, torch.int64, dev),
                          0 if grad_factor is None else _flat("grad_factor", grad_factor, 1, torch.float32, dev))
        _call("sol_adamw_step", dev, stream, self._handle, h)

    def norm_workspace(self) -> torch.Tensor:
        """A workspace for grad_norm (one for each of the calls that may overlap)."""
        return torch.empty(NORM_WORKSPACE, dtype=torch.uint8, device=self.device)

    def grad_norm(self, out, max_norm, *, workspace, stream=None):
        """out[0] = norm of all gradients, out[1] = min(1, max_norm / (out[0] + 1e-6)), 1 for any norm but NaN where
        max_norm is infinite  (sol_adamw_grad_norm)."""
        dev = self._index
        _call("sol_adamw_grad_norm", dev, stream, _flat("out", out, 2, torch.float32, dev), self._handle, max_norm,
              *_space(workspace, dev))
        return out

    def close(self):
        """Frees the plan: its steps have ended, and no captured graph that uses it is replayed any more."""
        if self._handle:
            h, self._handle = self._handle, None
            with torch.cuda.device(self._index):
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
    out = v_out if m_out is None else m_out
    if out is None:
        return
    n, dtype, dev = out.numel(), out.dtype, _device(out)
    blocks = -(-n // BLOCK)

    def part(name, o, q, s, codes):
        if o is None:
            return None, None, None
        return (_flat(name + "_out", o, n, dtype, dev), _flat(name, q, n, codes, dev),
                _flat(name + "_scale", s, blocks, torch.float32, dev))

    mo, mq, ms = part("m", m_out, m, m_scale, torch.int8)
    vo, vq, vs = part("v", v_out, v, v_scale, torch.uint8)
    _call("sol_adamw_state_decode", dev, stream, mo, vo, sol._dtype(out), mq, vq, ms, vs, n)
