"""Host-side checks of the training operators' C ABI that need no GPU: exports, refusals and
workspace sizes.  The pointers are fake addresses; every call fails validation on the host or has
nothing to do, so none reaches the device."""
from __future__ import annotations

import ctypes
import re

import pytest
import torch

from dit_block_b200 import build, sol, train

FAKE = 1 << 30          # a 256-byte aligned address, never read
STEP = 1 << 26          # distance between fake tensors
INV, MIS, UNS = sol.ERR_INVALID_ARGUMENT, sol.ERR_MISALIGNED, sol.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build()
    return train.lib()


def last(L):
    return L.sol_last_error().decode()


def test_every_declared_function_is_exported_and_bound(L):
    with open(train.HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(sol_[a-z0-9_]+)\s*\(", text))
    assert names == set(train.SIGNATURES)
    for n in names:
        assert hasattr(L, n)
    for name, value in (("SOL_ADAMW_BLOCK", train.BLOCK), ("SOL_ADAMW_NORM_WORKSPACE", train.NORM_WORKSPACE)):
        assert int(re.search(rf"#define {name} (\d+)", text)[1]) == value


def test_workspace_bytes(L):
    ws = train.ffn_workspace_bytes
    assert ws(0, 64, 64) > 0
    for t, d, inner in ((1, 8, 8), (7, 64, 128), (1252, 5120, 13824), (31248, 5120, 13824)):
        n = ws(t, d, inner)
        assert n % 256 == 0 and n >= 6 * t * inner  # act and du
    for bad in ((-1, 64, 64), (4, 60, 64), (4, 64, 4), (4, 0, 64), (1 << 30, 64, 64), (4, 1 << 28, 64)):
        assert ws(*bad) == 0


FFN = dict(y=FAKE, ld_y=64, u=FAKE + STEP, ld_u=256, x=FAKE + 2 * STEP, ld_x=64, w_up=FAKE + 3 * STEP, ld_wu=64,
           w_down=FAKE + 4 * STEP, ld_wd=128, ws=FAKE + 5 * STEP, bytes=STEP, n=16, d=64, inner=128, dt=sol.BF16)


def ffn(L, **kw):
    a = {**FFN, **kw}
    return L.sol_ffn(ctypes.byref(train.FfnDesc(*a.values())), None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(dt=sol.F32), UNS, "bf16 only"),
    (dict(n=-1), INV, "negative"),
    (dict(n=1 << 30), UNS, "2^30"),
    (dict(d=60, ld_x=64), UNS, "multiples of 8"),
    (dict(inner=4), INV, "at least 8"),
    (dict(w_up=None), INV, "w_up is NULL"),
    (dict(w_down=FAKE + 8), MIS, "w_down is not 16-byte"),
    (dict(x=None), INV, "x is NULL"),
    (dict(y=None), INV, "y is NULL"),
    (dict(ld_x=56), INV, "below the row width"),
    (dict(ld_wd=132), MIS, "multiple of 8"),
    (dict(ld_u=248), INV, "ld of u"),
    (dict(ws=None), INV, "workspace is NULL"),
    (dict(ws=FAKE + 5 * STEP + 16), MIS, "256-byte"),
    (dict(bytes=1000), INV, "below the"),
    (dict(y=FAKE + 2 * STEP + 128), INV, "overlaps"),
    (dict(u=FAKE + 3 * STEP), INV, "overlaps w_up"),
    (dict(u=FAKE), INV, "y overlaps u"),
    (dict(ws=FAKE + 2 * STEP), INV, "workspace overlaps x"),
])
def test_ffn_refusals(L, kw, status, word):
    assert ffn(L, **kw) == status
    assert word in last(L), last(L)


def test_descriptors_are_packed_as_they_are_declared(L):
    """The bytes that the calls send against the structures' own, field by field."""
    for of, pack in ((train.FfnDesc, train._pack_ffn), (train.FfnBackwardDesc, train._pack_ffn_backward)):
        values = [i + 1 for i in range(len(of._fields_))]
        assert pack(*values) == bytes(of(*values))
    values = [.1, .2, .3, .4, 5, 6, 7, 8, 9]
    assert train._pack_scalars(*values) == bytes(train.AdamwScalars(*values))
    assert L.sol_ffn(None, None) == INV and "desc is NULL" in last(L)
    assert L.sol_ffn_backward(None, None) == INV and "desc is NULL" in last(L)


def test_ffn_of_no_tokens(L):
    assert ffn(L, n=0, x=None, y=None, u=None, ws=None, bytes=0) == sol.OK


BWD = dict(dx=FAKE, ld_dx=64, dw_up=FAKE + STEP, ld_dwu=64, dw_down=FAKE + 2 * STEP, ld_dwd=128,
           dy=FAKE + 3 * STEP, ld_dy=64, x=FAKE + 4 * STEP, ld_x=64, u=FAKE + 5 * STEP, ld_u=256, w_up=FAKE + 6 * STEP,
           ld_wu=64, w_down=FAKE + 7 * STEP, ld_wd=128, ws=FAKE + 8 * STEP, bytes=STEP, n=16, d=64, inner=128,
           dt=sol.BF16, gdt=sol.BF16, acc=0)


def bwd(L, **kw):
    a = {**BWD, **kw}
    return L.sol_ffn_backward(ctypes.byref(train.FfnBackwardDesc(*a.values())), None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(dt=sol.F32), UNS, "bf16 only"),
    (dict(gdt=2), UNS, "grad_dt"),
    (dict(dy=None), INV, "dy is NULL"),
    (dict(u=None), INV, "u is NULL"),
    (dict(x=None), INV, "x is NULL"),
    (dict(w_up=None), INV, "w_up is NULL"),
    (dict(dw_up=FAKE + STEP + 2), MIS, "dw_up"),
    (dict(ld_dwd=120), INV, "dw_down"),
    (dict(gdt=sol.F32, ld_dwu=66), MIS, "multiple of 4"),
    (dict(bytes=1), INV, "below the"),
    (dict(dx=FAKE + 3 * STEP), INV, "dx overlaps dy"),
    (dict(dw_up=FAKE + 6 * STEP), INV, "dw_up overlaps w_up"),
    (dict(dw_down=FAKE + STEP), INV, "dw_up overlaps dw_down"),
    (dict(ws=FAKE + 5 * STEP), INV, "workspace overlaps u"),
])
def test_ffn_backward_refusals(L, kw, status, word):
    assert bwd(L, **kw) == status
    assert word in last(L), last(L)


def test_ffn_backward_with_nothing_to_do(L):
    assert bwd(L, dx=None, dw_up=None, dw_down=None) == sol.OK
    assert bwd(L, n=0, acc=1, dy=None, x=None, u=None, dx=None, ws=None, bytes=0) == sol.OK


def tensor(i, n=1000, **kw):
    at = FAKE + i * 8 * STEP
    t = dict(param=at, copy=None, grad=at + STEP, m=at + 2 * STEP, v=at + 3 * STEP, m_scale=None, v_scale=None, n=n,
             weight_decay=0.0)
    t.update(kw)
    return train.AdamwTensor(*t.values())


def create(L, tensors, grad_dt=sol.F32, bits=32):
    h = ctypes.c_void_p()
    rows = (train.AdamwTensor * max(len(tensors), 1))(*tensors)
    return L.sol_adamw_plan_create(ctypes.byref(h), rows, len(tensors), grad_dt, bits)


EIGHT = dict(m_scale=FAKE + 4 * STEP, v_scale=FAKE + 5 * STEP)


@pytest.mark.parametrize("tensors,kw,status,word", [
    ([tensor(0)], dict(grad_dt=3), UNS, "grad_dt"),
    ([tensor(0)], dict(bits=16), UNS, "state_bits"),
    ([tensor(0, n=-1)], {}, INV, "must be in"),
    ([tensor(0, weight_decay=-0.1)], {}, INV, "weight_decay"),
    ([tensor(0, weight_decay=float("nan"))], {}, INV, "weight_decay"),
    ([tensor(0, param=None)], {}, INV, "param is NULL"),
    ([tensor(0), tensor(1, grad=None)], {}, INV, "tensor 1: grad is NULL"),
    ([tensor(0, m=FAKE + 8)], {}, MIS, "m is not 16-byte"),
    ([tensor(0)], dict(bits=8), INV, "m_scale is NULL"),
    ([tensor(0, **EIGHT)], {}, INV, "given for 32-bit"),
    ([tensor(0), tensor(0)], {}, INV, "overlaps"),                       # the same tensor twice
    ([tensor(0, m=FAKE + 3 * STEP)], {}, INV, "overlaps"),               # m and v in one buffer
    ([tensor(0), tensor(1, param=FAKE + 2000)], {}, INV, "overlaps"),
    ([tensor(0), tensor(1, copy=FAKE + STEP)], {}, INV, "overlaps"),     # a copy over a gradient
    ([tensor(0, n=1 << 24), tensor(1, param=FAKE + STEP - 16)], {}, INV, "overlaps"),
])
def test_adamw_plan_refusals(L, tensors, kw, status, word):
    assert create(L, tensors, **kw) == status
    assert word in last(L), last(L)


def scalars(**kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0, lr_device=None, step_device=None,
             grad_factor=None)
    a.update(kw)
    return train.AdamwScalars(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(lr=float("inf")), INV), (dict(eps=-1e-8), INV), (dict(beta1=1.0), INV), (dict(beta2=-0.1), INV),
    (dict(beta2=float("nan")), INV), (dict(step=0), INV), (dict(step_device=FAKE + 4), MIS),
    (dict(grad_factor=FAKE + 2), MIS), ({}, INV),  # the last: no plan
])
def test_adamw_step_refusals(L, kw, status):
    assert L.sol_adamw_step(None, ctypes.byref(scalars(**kw)), None) == status
    assert L.sol_adamw_step(None, None, None) == INV


def test_grad_norm_and_decode_refusals(L):
    n = train.NORM_WORKSPACE
    assert L.sol_adamw_grad_norm(None, None, 1.0, FAKE, n, None) == INV
    assert L.sol_adamw_grad_norm(FAKE + 4, None, 1.0, FAKE, n, None) == MIS
    for bad in (0.0, -1.0, float("nan")):
        assert L.sol_adamw_grad_norm(FAKE, None, bad, FAKE, n, None) == INV
        assert "max_norm" in last(L)
    assert L.sol_adamw_grad_norm(FAKE, None, 1.0, FAKE, n - 1, None) == INV
    assert L.sol_adamw_grad_norm(FAKE + STEP, None, 1.0, FAKE, n, None) == INV and "plan is NULL" in last(L)
    assert L.sol_adamw_grad_norm(FAKE + n - 8, None, 1.0, FAKE, n, None) == INV and "out overlaps" in last(L)
    d = L.sol_adamw_state_decode
    q, s = FAKE + STEP, FAKE + 2 * STEP
    assert d(FAKE, None, 2, q, None, s, None, 100, None) == UNS
    assert d(FAKE, None, sol.F32, None, None, s, None, 100, None) == INV
    assert d(FAKE + 4, None, sol.F32, q, None, s, None, 100, None) == MIS
    assert d(FAKE, FAKE + 16, sol.F32, q, q, s, s, 100, None) == INV and "overlaps" in last(L)
    assert d(FAKE, None, sol.F32, q, None, s, None, -1, None) == INV
    assert d(None, None, sol.F32, None, None, None, None, 0, None) == sol.OK
    assert d(None, None, sol.F32, None, None, None, None, 100, None) == sol.OK


def test_destroying_no_plan(L):
    assert L.sol_adamw_plan_destroy(None) == sol.OK


def test_binding_refuses_cpu_tensors_shapes_and_types():
    bf = torch.bfloat16
    x, wu, wd = torch.zeros(4, 64, dtype=bf), torch.zeros(256, 64, dtype=bf), torch.zeros(64, 128, dtype=bf)
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        train.ffn(torch.zeros_like(x), x, wu, wd, workspace=ws)
    with pytest.raises(TypeError, match="dw_up and dw_down must be"):
        train.ffn_backward(x, x, torch.zeros(4, 256, dtype=bf), wu, wd, dw_up=wu.double(), workspace=ws)
    check = train._matrix
    with pytest.raises(ValueError, match=r"w_up must be \[256, 64\]"):
        check("w_up", wu[:128], 256, 64, bf, -1)
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        check("x", x.float(), 4, 64, bf, -1)
    with pytest.raises(ValueError, match="unit column stride"):
        check("x", x.repeat(1, 2)[:, ::2], 4, 64, bf, -1)
    with pytest.raises(ValueError, match="on device 0"):
        check("x", x, 4, 64, bf, 0)
    assert check("x", x, 4, 64, bf, -1) == (x.data_ptr(), 64)
    assert check("x", x[:1], 1, 64, bf, -1)[1] == 64
    p = [torch.zeros(8)]
    with pytest.raises(ValueError, match="CUDA"):
        train.AdamW(p, p, p, p)
    with pytest.raises(ValueError, match="one entry"):
        train.AdamW(p, p, p, p, weight_decay=[0.0, 0.0])
    with pytest.raises(TypeError, match="gradients must be"):
        train.AdamW(p, [p[0].double()], p, p)
    with pytest.raises(ValueError, match="contiguous"):
        train._flat("grad", torch.zeros(16)[::2], 8, torch.float32, -1)
    with pytest.raises(TypeError, match="m must be"):
        train._flat("m", torch.zeros(8), 8, torch.int8, -1)


def test_a_workspace_is_taken_by_its_bytes():
    """One value expanded to many is no workspace, whatever its shape says."""
    one = torch.empty(1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="contiguous"):
        train._space(one.expand(1 << 20), -1)
    assert train._space(torch.empty(5, dtype=torch.float32), -1)[1] == 20
