"""GPU tests of AdamW over many tensors, the gradient norm and the 8-bit moments against the formulas in
64 bits.

Tolerances.  One step is some ten fp32 operations on a value; each is off by at most 2^-24 of its result
(2^-23 for the sums that a fused multiply-add forms without its inner rounding).  So m and v, sums of two
terms, are within 4 * 2^-24 of the terms' magnitudes; the update u = m^ / (sqrt(v^) + eps) is within 16 * 2^-24
of itself beyond m's own error, and p within lr times that plus 2 * 2^-24 of the magnitudes it is formed from.
"""
from __future__ import annotations

import pytest
import torch

from dit_block_b200 import sol, train

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
HYPER = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8)
MIXED = [1, 3, 4, 255, 256, 257, 1000, 4095, 4096, 4097, 0, 70001]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tensors(sizes, grad_type=F32, seed=0, bits=32):
    g = gen(seed)
    rnd = lambda n, std: torch.randn(n, device="cuda", generator=g) * std  # noqa: E731
    t = dict(params=[rnd(n, 0.02) for n in sizes], grads=[rnd(n, 1e-3).to(grad_type) for n in sizes])
    if bits == 32:
        t["m"] = [rnd(n, 3e-4) for n in sizes]
        t["v"] = [rnd(n, 1e-3).square() for n in sizes]
    else:
        blocks = [-(-n // train.BLOCK) for n in sizes]
        t["m"] = [torch.zeros(n, device="cuda", dtype=torch.int8) for n in sizes]
        t["v"] = [torch.zeros(n, device="cuda", dtype=torch.uint8) for n in sizes]
        t["m_scales"] = [torch.zeros(n, device="cuda") for n in blocks]
        t["v_scales"] = [torch.zeros(n, device="cuda") for n in blocks]
    return t


def formula(p, g, m, v, wd, step, factor=1.0, lr=1e-3, betas=(0.9, 0.999), eps=1e-8):
    """(p, m, v) after a step and their bounds, in 64 bits."""
    p, g, m, v = (t.to(F64) for t in (p, g, m, v))
    b1, b2 = betas
    g = g * factor
    em = 4 * U * (b1 * m.abs() + (1 - b1) * g.abs())
    ev = 4 * U * (b2 * v + (1 - b2) * g * g)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    root = (v / c2).sqrt() + eps
    up = m / c1 / root
    eup = (em / c1) / root + 16 * U * up.abs()
    move = lr * (wd * p + up)
    q = p - move
    ep = lr * eup + 4 * U * (p.abs() + lr * (wd * p).abs() + lr * up.abs())
    # values below fp32's normal range are off by its smallest step
    return (q, ep), (m, em + 1e-44), (v, ev + 1e-44)


def check(got, want, what):
    v, e = want
    off = (got.to(F64) - v).abs() - e
    assert got.numel() == 0 or off.max() <= 0, f"{what}: worst by {off.max():.3g}"


@pytest.mark.parametrize("grad_type", [F32, BF])
@pytest.mark.parametrize("copied", [False, True])
@pytest.mark.parametrize("step", [1, 2, 1000])
def test_step_f32(grad_type, copied, step):
    t = tensors(MIXED, grad_type)
    decay = [0.1 * (k % 3) for k in range(len(MIXED))]
    copies = [torch.zeros(n, device="cuda", dtype=BF) if k % 2 else None for k, n in enumerate(MIXED)] if copied else None
    want = [formula(p, g, m, v, w, step, **HYPER)
            for p, g, m, v, w in zip(t["params"], t["grads"], t["m"], t["v"], decay)]
    with train.AdamW(**t, copies=copies, weight_decay=decay) as opt:
        opt.step(step=step, **HYPER)
        torch.cuda.synchronize()
    for k, (p, m, v) in enumerate(want):
        check(t["params"][k], p, f"p of {MIXED[k]}")
        check(t["m"][k], m, f"m of {MIXED[k]}")
        check(t["v"][k], v, f"v of {MIXED[k]}")
        if copied and copies[k] is not None:
            assert torch.equal(copies[k], t["params"][k].to(BF))


def test_rows_around_a_tensor_are_left_alone():
    flat = {k: torch.full((64 + 1003 + 64,), 9.0, device="cuda") for k in ("params", "grads", "m", "v")}
    with train.AdamW(*([flat[k][64:64 + 1003]] for k in ("params", "grads", "m", "v"))) as opt:
        opt.step(step=1, **HYPER)
        torch.cuda.synchronize()
    for t in flat.values():
        assert (t[:64] == 9).all() and (t[64 + 1003:] == 9).all()
    assert (flat["params"][64:-64] != 9).all()


def test_many_tensors_are_each_their_own():
    sizes = [(37 * k) % 997 + 1 for k in range(700)]
    t = tensors(sizes)
    want = [formula(p, g, m, v, 0.01, 3, **HYPER) for p, g, m, v in zip(*(t[k] for k in ("params", "grads", "m", "v")))]
    with train.AdamW(**t, weight_decay=0.01) as opt:
        opt.step(step=3, **HYPER)
        torch.cuda.synchronize()
    for k, (p, m, v) in enumerate(want):
        check(t["params"][k], p, f"tensor {k}")
        check(t["m"][k], m, f"tensor {k}")


def test_nothing_to_step():
    for t in (tensors([]), tensors([0, 0])):
        with train.AdamW(**t) as opt:
            opt.step(step=1, **HYPER)
            out = torch.full((2,), 7.0, device="cuda")
            opt.grad_norm(out, 1.0, workspace=opt.norm_workspace())
            assert out.tolist() == [0.0, 1.0]


def test_a_zero_gradient_and_zero_moments():
    p = torch.randn(1000, device="cuda")
    z = lambda: torch.zeros(1000, device="cuda")  # noqa: E731
    before = p.clone()
    with train.AdamW([p], [z()], [z()], [z()]) as opt:
        opt.step(step=1, **HYPER)
    assert torch.equal(p, before)


@pytest.mark.parametrize("sizes", [[1000, 5000], [70, 2_000_000]])
def test_scalars_from_the_device_in_a_captured_step(sizes):
    """lr, step and the clip factor are read when the graph runs; the host's lr and step are not used."""
    t, ref = tensors(sizes), tensors(sizes)
    lr = torch.tensor([5e-4], device="cuda")
    step = torch.tensor([1], device="cuda")
    factor = torch.tensor([1.0], device="cuda")
    opt = train.AdamW(**t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(lr=0.5, step=77, lr_device=lr, step_device=step, grad_factor=factor)
        step.add_(1)
    with train.AdamW(**ref) as other:
        for n, (rate, f) in enumerate(((5e-4, 1.0), (1e-3, 0.5), (2e-3, 0.25)), 1):
            lr.fill_(rate)
            factor.fill_(f)
            graph.replay()
            other.step(lr=float(torch.tensor(rate, dtype=F32)), step=n, grad_factor=factor)
    torch.cuda.synchronize()
    assert step.item() == 4
    for k in ("params", "m", "v"):
        for a, b in zip(t[k], ref[k]):
            assert torch.equal(a, b)
    del graph
    opt.close()


# ------------------------------------------------------------------------------ norm

def norm_of(grads, max_norm=1.0):
    z = [torch.zeros(g.numel(), device="cuda") for g in grads]
    with train.AdamW([t.clone() for t in z], grads, [t.clone() for t in z], [t.clone() for t in z]) as opt:
        out = torch.zeros(2, device="cuda")
        opt.grad_norm(out, max_norm, workspace=opt.norm_workspace())
        return out.tolist()


@pytest.mark.parametrize("grad_type", [F32, BF])
@pytest.mark.parametrize("sizes", [[1], [3, 5], MIXED, [3_000_017]])
@pytest.mark.parametrize("scale", [1.0, 1e-25, 1e30])
def test_grad_norm(grad_type, sizes, scale):
    """Sixteen squares are added in fp32 (16 * 2^-24), the rest in 64 bits; the result is rounded once."""
    g = [torch.randn(n, device="cuda", generator=gen(n)).mul(scale).to(grad_type) for n in sizes]
    want = float(torch.cat([t.to(F64) for t in g]).norm())
    norm, factor = norm_of(g, max_norm=0.5)
    assert abs(norm - want) <= 20 * U * want
    assert abs(factor - min(1.0, 0.5 / (want + 1e-6))) <= 24 * U * factor + 1e-45


def test_grad_norm_extremes():
    top = torch.finfo(F32).max
    one = lambda *v: [torch.tensor(v, device="cuda")]  # noqa: E731
    assert norm_of(one(top / 2, 0.0))[0] == top / 2
    assert norm_of(one(1e-44))[0] == torch.tensor(1e-44).item()
    assert norm_of(one(0.0, 0.0)) == [0.0, 1.0]
    assert norm_of(one(float("inf"), 1.0)) == [float("inf"), 0.0]
    n, f = norm_of(one(float("nan"), float("inf")))
    assert n != n and f != f
    assert norm_of(one(3.0, 4.0), max_norm=float("inf")) == [5.0, 1.0]


def test_grad_norm_has_the_same_bits_every_time():
    g = [torch.randn(n, device="cuda", generator=gen(n)) for n in (1_000_003, 77, 4096)]
    assert len({tuple(norm_of(g)) for _ in range(5)}) == 1


# ------------------------------------------------------------------------------ 8-bit moments

def tables():
    first = (torch.arange(128, device="cuda", dtype=F64) / 127) ** 2
    second = (torch.arange(256, device="cuda", dtype=F64) / 255) ** 4
    return first, second


def blocks_of(x, n):
    """[blocks, 256] with zeros behind the last value."""
    out = torch.zeros(-(-n // train.BLOCK) * train.BLOCK, device=x.device, dtype=x.dtype)
    out[:n] = x
    return out.view(-1, train.BLOCK)


def decode(t, k):
    n = t["params"][k].numel()
    m, v = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    train.adamw_state_decode(m, v, t["m"][k], t["v"][k], t["m_scales"][k], t["v_scales"][k])
    return m, v


def neighbours(value, scale, table, got, bound):
    """got is one of the table's two values around `value` (both in blocks), up to `bound`."""
    unit = (value / torch.where(scale > 0, scale, 1)).clamp(0, 1)
    k = (torch.searchsorted(table, unit, right=True) - 1).clamp(0, len(table) - 2)
    lo, hi = table[k] * scale, table[k + 1] * scale
    return ((got - lo).abs() <= bound) | ((got - hi).abs() <= bound) | ((got - value).abs() <= bound)


@pytest.mark.parametrize("grad_type", [F32, BF])
def test_step_8bit(grad_type):
    t = tensors(MIXED, grad_type, bits=8)
    first, second = tables()
    state = [tuple(torch.zeros(n, device="cuda", dtype=F64) for _ in range(2)) for n in MIXED]
    copies = [torch.zeros(n, device="cuda", dtype=BF) if n % 2 else None for n in MIXED]
    with train.AdamW(**t, copies=copies, weight_decay=0.01) as opt:
        for step in (1, 2, 3):
            want = [formula(p, g, m, v, 0.01, step, **HYPER)
                    for p, g, (m, v) in zip(t["params"], t["grads"], state)]
            opt.step(step=step, seed=5, **HYPER)
            for k, n in enumerate(MIXED):
                if n == 0:
                    continue
                (p, ep), (m, em), (v, ev) = want[k]
                check(t["params"][k], (p, ep), f"p of {n}, step {step}")
                if copies[k] is not None:
                    assert torch.equal(copies[k], t["params"][k].to(BF))
                got_m, got_v = (x.to(F64) for x in decode(t, k))
                # scales: the block's largest magnitude
                bm, bv = blocks_of(m, n), blocks_of(v, n)
                s1, s2 = t["m_scales"][k].to(F64)[:, None], t["v_scales"][k].to(F64)[:, None]
                assert ((s1 - bm.abs().amax(1, keepdim=True)).abs() <= 8 * U * s1 + 1e-44).all()
                assert ((s2 - bv.amax(1, keepdim=True)).abs() <= 8 * U * s2 + 1e-44).all()
                # values: a neighbour in the table, of the sign of the moment
                gm, gv = blocks_of(got_m, n), blocks_of(got_v, n)
                assert (gm * bm >= 0).all()
                assert neighbours(bm.abs(), s1, first, gm.abs(), 32 * U * s1).all()
                low = second[1] * s2  # a positive second moment is never stored as zero
                assert (neighbours(bv, s2, second, gv, 32 * U * s2) | ((gv - low).abs() <= 32 * U * low)).all()
                assert (blocks_of(got_v, n)[bv > 0] > 0).all()
                state[k] = (got_m, got_v)


def test_8bit_rounding_is_unbiased_and_follows_the_seed():
    """The mean over many seeds of a stored moment is the moment: each is one of two values a step h apart, so the
    mean over R draws is off by a standard deviation of at most h / (2 sqrt(R)); five of them, and 2^-16 for the
    fractions' 16 bits."""
    n, draws = 2048, 400
    g = torch.randn(n, device="cuda", generator=gen(1))
    sums = torch.zeros(2, n, device="cuda", dtype=F64)
    seen = set()
    for seed in range(draws):
        t = tensors([n], bits=8)
        t["grads"][0].copy_(g)
        with train.AdamW(**t) as opt:
            opt.step(step=1, seed=seed, **HYPER)
            m, v = decode(t, 0)
        seen.add(tuple(t["m"][0][:64].tolist()))
        sums += torch.stack([m, v]).to(F64)
    assert len(seen) == draws
    mean = sums / draws
    first, second = tables()
    for value, table, got, floor in ((g.to(F64) * 0.1, first, mean[0], 0.0), (g.to(F64) ** 2 * 0.001, second, mean[1], 1.0)):
        x = value.abs().view(-1, train.BLOCK)
        s = x.amax(1, keepdim=True)
        k = (torch.searchsorted(table, x / s, right=True) - 1).clamp(0, len(table) - 2)
        h = (table[k + 1] - table[k]) * s
        bound = 5 * h / (2 * draws ** 0.5) + h * 2.0 ** -16 + 64 * U * s + floor * table[1] * s
        assert ((got.view(-1, train.BLOCK).abs() - x).abs() <= bound).all()


def test_8bit_moments_follow_f32_moments():
    """Over 200 steps of noisy gradients the 8-bit second moment neither stalls nor drifts: its mean over the
    tensor stays within 2 % of the f32 one's (each of 16384 values carries independent roundings of at most 1.6 %
    of the largest)."""
    n = 16384
    a, b = tensors([n], bits=32), tensors([n], bits=8)
    for k in ("m", "v"):
        a[k][0].zero_()
    with train.AdamW(**a) as x, train.AdamW(**b) as y:
        for step in range(1, 201):
            g = torch.randn(n, device="cuda", generator=gen(step)) * (1.0 if step < 100 else 0.3)
            a["grads"][0].copy_(g)
            b["grads"][0].copy_(g)
            x.step(step=step, **HYPER)
            y.step(step=step, seed=1, **HYPER)
        m, v = decode(b, 0)
    assert abs(v.double().mean() / a["v"][0].double().mean() - 1) < 0.02
    assert (m.double() - a["m"][0].double()).norm() / a["m"][0].double().norm() < 0.05


def test_8bit_nonfinite_gradients_show():
    t = tensors([1000], bits=8)
    t["grads"][0][300] = float("nan")
    t["grads"][0][700] = float("inf")
    with train.AdamW(**t) as opt:
        opt.step(step=1, **HYPER)
        m, v = decode(t, 0)
    for x in (m, v):
        bad = x.isnan().tolist()
        assert not any(bad[:256]) and all(bad[256:768]) and not any(bad[768:])


def test_8bit_tiny_and_huge_moments():
    """Blocks of fp32's smallest and largest magnitudes keep their scale and their largest value."""
    for size in (1e-18, 1e18):
        t = tensors([512], bits=8)
        t["grads"][0].copy_(torch.randn(512, device="cuda", generator=gen(2)) * size)
        with train.AdamW(**t) as opt:
            opt.step(step=1, **HYPER)
            m, v = decode(t, 0)
        want = (t["grads"][0].double() * 0.1)
        assert torch.isfinite(m).all() and torch.isfinite(v).all() and torch.isfinite(t["params"][0]).all()
        assert abs(m.double().abs().max() / want.abs().max() - 1) < 1e-5


def test_decode_types_and_ends():
    for n in (1, 7, 8, 256, 1003):
        q = torch.randint(-127, 128, (n,), device="cuda", dtype=torch.int8)
        r = torch.randint(0, 256, (n,), device="cuda", dtype=torch.uint8)
        s = torch.rand(-(-n // train.BLOCK), device="cuda") + 0.1
        per = s.double().repeat_interleave(train.BLOCK)[:n]
        want_m = torch.sign(q.double()) * (q.double() / 127) ** 2 * per
        want_v = (r.double() / 255) ** 4 * per
        for dtype, rounding in ((F32, 8 * U), (BF, 2.0 ** -8 + 8 * U)):
            flat = torch.full((2, n + 64), 3.0, device="cuda", dtype=dtype)
            ends = (n + 7) // 8 * 8
            m, v = flat[0, :n], torch.full((ends + 8,), 3.0, device="cuda", dtype=dtype)
            train.adamw_state_decode(m, v[:n], q, r, s, s)
            assert ((m.double() - want_m).abs() <= rounding * want_m.abs()).all()
            assert ((v[:n].double() - want_v).abs() <= rounding * want_v.abs()).all()
            assert (flat[0, n:] == 3).all() and (v[n:] == 3).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(bits):
    """A tensor of more than 2^32 values, zero but for its two ends, which step as tensors of their own do."""
    ends, gap = 5000, 1 << 32
    n = gap + ends
    g = torch.randn(ends, device="cuda", generator=gen(1)).to(BF)
    t = dict(params=[torch.zeros(n, device="cuda")], grads=[torch.zeros(n, device="cuda", dtype=BF)])
    if bits == 32:
        t["m"], t["v"] = [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")]
    else:
        t["m"], t["v"] = [torch.zeros(n, device="cuda", dtype=torch.int8)], [torch.zeros(n, device="cuda", dtype=torch.uint8)]
        blocks = -(-n // train.BLOCK)
        t["m_scales"], t["v_scales"] = [torch.zeros(blocks, device="cuda")], [torch.zeros(blocks, device="cuda")]
    t["grads"][0][:ends] = g
    t["grads"][0][gap:] = g
    out = torch.zeros(2, device="cuda")
    with train.AdamW(**t) as opt:
        opt.grad_norm(out, float("inf"), workspace=opt.norm_workspace())
        opt.step(step=1, **HYPER)
    assert abs(out[0].item() / (2 ** 0.5 * g.to(F64).norm().item()) - 1) < 1e-6
    zero = torch.zeros(ends, device="cuda")
    want = formula(zero, g, zero, zero, 0.0, 1, **HYPER)
    p = t["params"][0]
    check(p[:ends], want[0], "first values")
    assert torch.equal(p[gap:], p[:ends])
    assert p[ends:gap].abs().max() == 0
    if bits == 32:
        for k, w in (("m", want[1]), ("v", want[2])):
            check(t[k][0][gap:], w, k)
            assert t[k][0][ends:gap].abs().max() == 0
    else:
        m, v = torch.empty(n, device="cuda", dtype=BF), torch.empty(n, device="cuda", dtype=BF)
        train.adamw_state_decode(m, v, t["m"][0], t["v"][0], t["m_scales"][0], t["v_scales"][0])
        assert m[ends:gap].abs().max() == 0 and v[ends:gap].abs().max() == 0
        # the ends' own blocks, read by themselves
        at = gap // train.BLOCK
        mt, vt = torch.empty(ends, device="cuda", dtype=BF), torch.empty(ends, device="cuda", dtype=BF)
        train.adamw_state_decode(mt, vt, t["m"][0][gap:], t["v"][0][gap:], t["m_scales"][0][at:], t["v_scales"][0][at:])
        assert torch.equal(m[gap:], mt) and torch.equal(v[gap:], vt)
        # one of the table's two neighbours is within a step of it: 2 / 127 and 4 / 255 of the block's largest
        (bm, _), (bv, _) = want[1], want[2]
        assert ((mt.to(F64) - bm).abs() <= (2 / 127 + 2 ** -8) * bm.abs().max()).all()
        assert ((vt.to(F64) - bv).abs() <= (4 / 255 + 2 ** -8) * bv.max()).all()
    del t, p
    torch.cuda.empty_cache()


def test_refusals_on_the_device():
    t = tensors([100, 200])
    with pytest.raises(sol.SolError, match="overlaps"):
        train.AdamW(t["params"][:1] * 2, t["grads"][:1] * 2, t["m"][:1] * 2, t["v"][:1] * 2)
    with pytest.raises(sol.SolError, match="16-byte"):
        big = tensors([101])
        train.AdamW([big["params"][0][1:]], [big["grads"][0][1:]], [big["m"][0][1:]], [big["v"][0][1:]])
    with train.AdamW(**t) as opt:
        with pytest.raises(sol.SolError, match="step"):
            opt.step(step=0, **HYPER)
        with pytest.raises(TypeError, match="grad_factor"):
            opt.step(step=1, grad_factor=torch.ones(1, device="cuda", dtype=F64), **HYPER)
