"""GPU tests of the 8-bit moments where test_train_adamw_gpu leaves room: large scales, what a positive second moment
may be stored as, the rounding of a tensor's last block, and steps counted on the device over many values.

A stored value is one of the table's two around the moment.  Its decoding is off by at most four roundings of
2^-24 of itself, and the moment itself by what test_train_adamw_gpu.formula gives."""
from __future__ import annotations

import pytest
import torch

from dit_block_b200 import train
from test_train_adamw_gpu import BF, F64, HYPER, U, blocks_of, decode, formula, gen, neighbours, tables, tensors

pytestmark = pytest.mark.gpu

TOP = torch.finfo(torch.float32).max


def stored(t, k=0):
    """Values and scales of tensor k, in blocks and in 64 bits."""
    n = t["params"][k].numel()
    m, v = (blocks_of(x.to(F64), n) for x in decode(t, k))
    return m, v, t["m_scales"][k].to(F64)[:, None], t["v_scales"][k].to(F64)[:, None]


@pytest.mark.parametrize("n", [512, 700])
@pytest.mark.parametrize("top", [1.5e38, 2.9e38, TOP])
def test_second_moments_with_a_scale_near_the_end_of_fp32(n, top):
    """beta2 = 0, so that v is the square of the gradient, up to the largest number there is."""
    t = tensors([n], bits=8)
    g = torch.rand(n, device="cuda", generator=gen(3)) * top ** 0.5 * 0.999
    g[::256] = top ** 0.5 * (1 - 2.0 ** -23)
    t["grads"][0].copy_(g)
    with train.AdamW(**t) as opt:
        opt.step(step=1, lr=1e-3, betas=(0.9, 0.0), eps=1e-8)
    v = blocks_of(t["grads"][0].to(F64) ** 2, n)
    _, got, _, s = stored(t)
    assert (s - v.amax(1, keepdim=True)).abs().max() <= 8 * U * top
    assert (neighbours(v, s, tables()[1], got, 32 * U * s) | (v == 0)).all()
    assert ((got.amax(1, keepdim=True) - s).abs() <= 8 * U * s).all(), "the largest of a block"
    assert torch.isfinite(t["params"][0]).all()


@pytest.mark.parametrize("n", [512, 700])
@pytest.mark.parametrize("top", [1.5e38, TOP])
def test_first_moments_with_a_scale_near_the_end_of_fp32(n, top):
    """beta1 = 0, so that m is the gradient; its square is beyond fp32, which makes v's blocks NaN."""
    t = tensors([n], bits=8)
    g = (torch.rand(n, device="cuda", generator=gen(4)) * 2 - 1) * top
    g[::256] = top
    t["grads"][0].copy_(g)
    with train.AdamW(**t) as opt:
        opt.step(step=1, lr=1e-3, betas=(0.0, 0.999), eps=1e-8)
    m = blocks_of(t["grads"][0].to(F64), n)
    got, v, s, _ = stored(t)
    assert (s == m.abs().amax(1, keepdim=True)).all()
    assert (got * m >= 0).all()
    assert neighbours(m.abs(), s, tables()[0], got.abs(), 32 * U * s).all()
    assert ((got.abs().amax(1, keepdim=True) - s).abs() <= 8 * U * s).all(), "the largest of a block"
    assert blocks_of(torch.ones(n, device="cuda"), n)[v.isnan()].sum() == n


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 1e-13])
def test_small_eps(bits, eps):
    """Values that never had a gradient stay as they are, the others move as the formula says, whatever eps."""
    n = 600
    t = tensors([n], bits=bits)
    for k in ("m", "v"):
        t[k][0].zero_()
    t["grads"][0][::3] = 0
    p, g = t["params"][0].clone(), t["grads"][0].clone()
    zero = torch.zeros(n, device="cuda")
    want, _, _ = formula(p, g, zero, zero, 0.0, 1, eps=eps)
    with train.AdamW(**t) as opt:
        opt.step(step=1, lr=1e-3, eps=eps)
    got = t["params"][0]
    assert torch.equal(got[::3], p[::3])
    assert ((got.to(F64) - want[0]).abs() <= want[1])[g != 0].all()
