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


@pytest.mark.parametrize("grad_type", [torch.float32, BF])
def test_only_small_second_moments_are_stored_as_one(grad_type):
    """A value above the table's first step is stored as one of its two neighbours, no lower; one below it as
    that step, not as zero."""
    sizes = [3, 255, 257, 1000, 4097]
    t = tensors(sizes, grad_type, seed=2, bits=8)
    with train.AdamW(**t) as opt:
        opt.step(step=1, seed=11, **HYPER)
        for k, n in enumerate(sizes):
            g = t["grads"][k].to(F64)
            v = blocks_of(g * g * 1e-3, n)
            _, got, _, s = stored(t, k)
            second = tables()[1]
            low = second[1] * s
            small = v <= low * (1 + 2.0 ** -20)
            assert small.any() or n < 10
            near = neighbours(v, s, second, got, 32 * U * s * (v / s).clamp(min=float(second[1])))
            assert (near | small).all()
            assert (((got - low).abs() <= 32 * U * low) | ~small | (v == 0)).all()


@pytest.mark.parametrize("n", [100, 300, 511])
def test_rounding_of_a_last_block_is_unbiased(n):
    """As for whole blocks: the mean over R draws is off by at most 5 h / (2 sqrt(R)) and 2^-16 h, h the table's step."""
    draws = 400
    g = torch.randn(n, device="cuda", generator=gen(n))
    sums = torch.zeros(2, n, device="cuda", dtype=F64)
    for seed in range(draws):
        t = tensors([n], bits=8)
        t["grads"][0].copy_(g)
        with train.AdamW(**t) as opt:
            opt.step(step=1, seed=seed, **HYPER)
            sums += torch.stack(decode(t, 0)).to(F64)
    mean = sums / draws
    for value, table, got, floor in ((g.to(F64) * 0.1, tables()[0], mean[0], 0.0), (g.to(F64) ** 2 * 0.001, tables()[1], mean[1], 1.0)):
        x = blocks_of(value.abs(), n)
        s = x.amax(1, keepdim=True)
        k = (torch.searchsorted(table, x / s, right=True) - 1).clamp(0, len(table) - 2)
        h = (table[k + 1] - table[k]) * s
        bound = 5 * h / (2 * draws ** 0.5) + h * 2.0 ** -16 + 64 * U * s + floor * table[1] * s
        assert ((blocks_of(got.abs(), n) - x).abs() <= bound).all()


@pytest.mark.parametrize("sizes", [[1000, 5000], [70, 2_000_000]])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_counted_on_the_device_are_the_host_counted_ones(sizes, bits):
    """Few chunks count the step in each CTA, many in a kernel ahead: parameters, moments or their codes and
    scales, and copies, bit for bit those of calls with the host's step."""
    t, ref = tensors(sizes, BF, bits=bits), tensors(sizes, BF, bits=bits)
    copies, ref_copies = ([torch.zeros(n, device="cuda", dtype=BF) for n in sizes] for _ in range(2))
    lr, step, factor = torch.tensor([1e-3], device="cuda"), torch.tensor([1], device="cuda"), torch.tensor([0.5], device="cuda")
    opt = train.AdamW(**t, copies=copies, weight_decay=0.01)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(lr=0.5, step=77, seed=3, lr_device=lr, step_device=step, grad_factor=factor)
        step.add_(1)
    with train.AdamW(**ref, copies=ref_copies, weight_decay=0.01) as other:
        for n in range(1, 6):
            for x, y in zip(t["grads"], ref["grads"]):
                x.copy_(torch.randn(x.numel(), device="cuda", generator=gen(n)))
                y.copy_(x)
            graph.replay()
            other.step(lr=float(lr), step=n, seed=3, grad_factor=factor)
    torch.cuda.synchronize()
    for k in t:
        for a, b in zip(t[k], ref[k]):
            assert torch.equal(a, b), k
    assert all(torch.equal(a, b) for a, b in zip(copies, ref_copies))
    assert all((p != q).any() for p, q in zip(t["params"], tensors(sizes, BF, bits=bits)["params"]))
    del graph
    opt.close()


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
