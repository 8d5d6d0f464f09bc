"""GPU tests of the gated feed-forward block and its backward pass against the formulas in 64 bits.

Tolerances, per element, from first principles.  A product over K terms accumulates in fp32, each
addition off by at most one unit in the last place of what it holds (truncation included), so its
error is at most K * 2^-23 * S with S the sum of the terms' magnitudes.  A value rounded to bf16
(an operand of the next product, or an output) is off by at most 2^-8 of itself.  The activation
and its gradient are evaluated with an error of a few 2^-22, taken as 2^-20, relative to the sum of
the magnitudes they are formed from.  Errors are carried through the formulas to first order with
their second-order terms covered by a factor 1.1.
"""
from __future__ import annotations

import pytest
import torch

from dit_block_b200 import sol, train

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF, ACC, FN = 2.0 ** -8, 2.0 ** -23, 2.0 ** -20

SIZES = [  # n_tokens, d, inner
    (1, 8, 8), (1, 256, 512), (2, 64, 128), (7, 72, 1032), (31, 264, 136), (8, 136, 72), (9, 520, 264), (16, 64, 8200), (16, 1000, 336), (17, 72, 80), (57, 64, 72),
    (63, 128, 64), (64, 128, 64), (65, 72, 64), (120, 64, 128), (128, 256, 512),
    (129, 64, 200), (257, 1000, 328), (1000, 200, 2504), (4099, 64, 64), (300, 2560, 1024), (20, 2000, 6008),
    (600, 1536, 4104),
    # on both sides of where a few tokens end, in both directions
    (32, 640, 8200), (33, 64, 72), (40, 3000, 8000), (57, 2048, 2048), (57, 3000, 5000), (63, 1000, 4000), (64, 2504, 5120),
    (65, 1000, 3200), (96, 264, 520), (120, 1304, 1304), (128, 904, 1096), (200, 128, 256), (225, 64, 72),
    (300, 64, 72), (513, 64, 72), (20, 5120, 8200), (1, 64, 13000), (13, 200, 13000), (30, 3448, 200), (5, 5120, 64), (40, 184, 12000),
]


@pytest.fixture(scope="module", autouse=True)
def _flags():
    sol.device_errors(clear=True)
    yield
    assert sol.device_errors() == 0


def drawn(seed, rows, cols, std=1.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.full((rows, cols + pad), 7.0, device="cuda", dtype=BF)
    v = t[:, pad:]
    v.copy_(torch.randn(rows, cols, device="cuda", generator=g) * std)
    return v


def inputs(n, d, inner, pad=0, seed=0):
    return dict(x=drawn(seed + 1, n, d, 1.0, pad), w_up=drawn(seed + 2, 2 * inner, d, d ** -0.5, pad),
                w_down=drawn(seed + 3, d, inner, inner ** -0.5, pad))


def close(got, want, bound, what):
    g = got.to(F64)
    assert torch.isfinite(g).all(), what
    over = (g - want).abs() - bound
    assert over.max() <= 0, f"{what}: {int((over > 0).sum())} of {g.numel()} out of bounds, worst by {over.max():.3g}"
    # roundings are independent of each other: in norm, one of an operand and one of the output
    norm = want.norm()
    if want.numel() >= 1000 and norm > 0:
        assert (g - want).norm() / norm < 2 * HALF, what


def forward64(x, w_up, w_down):
    """(u, y) and their bounds."""
    x, w_up, w_down = (t.to(F64) for t in (x, w_up, w_down))
    d, inner = x.shape[1], w_down.shape[1]
    u = x @ w_up.T
    eu = d * ACC * (x.abs() @ w_up.abs().T)
    a, b = u[:, :inner], u[:, inner:]
    ea, eb = eu[:, :inner], eu[:, inner:]
    silu = a * torch.sigmoid(a)
    act = silu * b
    eact = 1.1 * (1.1 * ea * (b.abs() + eb) + silu.abs() * eb) + (FN + HALF) * act.abs()
    y = act @ w_down.T
    ey = eact @ w_down.abs().T + inner * ACC * (act.abs() @ w_down.abs().T) + HALF * y.abs() + 1e-30
    return u, 1.01 * (eu + HALF * u.abs()) + 1e-30, y, 1.01 * ey


def backward64(dy, x, u, w_up, w_down):
    """{name: (gradient, bound before its last rounding)}."""
    dy, x, u, w_up, w_down = (t.to(F64) for t in (dy, x, u, w_up, w_down))
    n, d, inner = x.shape[0], x.shape[1], w_down.shape[1]
    a, b = u[:, :inner], u[:, inner:]
    s = torch.sigmoid(a)
    act = a * s * b
    eact = (FN + HALF) * act.abs()
    d_act = dy @ w_down
    e = d * ACC * (dy.abs() @ w_down.abs())
    fa, fb = b * s * (1 + a * (1 - s)), a * s
    ma = b.abs() * s * (1 + a.abs() * (1 - s))  # magnitudes that fa is formed from
    du = torch.cat([d_act * fa, d_act * fb], 1)
    edu = torch.cat([fa.abs() * e + FN * ma * (d_act.abs() + e), fb.abs() * e + FN * du[:, inner:].abs()], 1)
    edu = 1.01 * (edu + HALF * (du.abs() + edu))
    out = {"dx": (du @ w_up, edu @ w_up.abs() + 2 * inner * ACC * (du.abs() @ w_up.abs())),
           "dw_up": (du.T @ x, edu.T @ x.abs() + n * ACC * (du.abs().T @ x.abs())),
           "dw_down": (dy.T @ act, dy.abs().T @ eact + n * ACC * (dy.abs().T @ act.abs()))}
    return out


def run_forward(i, keep=True, ws=None, **kw):
    n, d = i["x"].shape
    inner = i["w_down"].shape[1]
    y = torch.full((n, d), float("nan"), device="cuda", dtype=BF)
    u = torch.full((n, 2 * inner), float("nan"), device="cuda", dtype=BF) if keep else None
    ws = train.ffn_workspace(n, d, inner) if ws is None else ws
    train.ffn(y, i["x"], i["w_up"], i["w_down"], u=u, workspace=ws, **kw)
    return y, u


@pytest.mark.parametrize("n,d,inner", SIZES)
@pytest.mark.parametrize("pad", [0, 24])
def test_forward(n, d, inner, pad):
    i = inputs(n, d, inner, pad)
    u64, eu, y64, ey = forward64(**i)
    y, u = run_forward(i)
    close(u, u64, eu, "u")
    close(y, y64, ey, "y")
    alone, _ = run_forward(i, keep=False)
    assert torch.equal(alone, y), "y depends on whether u is kept"


def grads(n, d, inner, grad_type, pad=0, fill=float("nan")):
    def one(rows, cols, dtype):
        t = torch.full((rows, cols + pad), 5.0, device="cuda", dtype=dtype)
        t[:, :cols] = fill
        return t[:, :cols]
    return dict(dx=one(n, d, BF), dw_up=one(2 * inner, d, grad_type), dw_down=one(d, inner, grad_type))


@pytest.mark.parametrize("n,d,inner", SIZES)
@pytest.mark.parametrize("pad,grad_type", [(0, BF), (8, F32)])
def test_backward(n, d, inner, pad, grad_type):
    i = inputs(n, d, inner, pad)
    dy, u = drawn(4, n, d, 0.1, pad), drawn(5, n, 2 * inner, 2.0, pad)
    want = backward64(dy, u=u, **i)
    out = grads(n, d, inner, grad_type, pad)
    ws = train.ffn_workspace(n, d, inner)
    train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=ws, **out)
    def right(k, got):
        g, e = want[k]
        rounding = HALF if got.dtype == BF else 2.0 ** -24
        close(got, g, 1.01 * (e + rounding * (g.abs() + e)) + 1e-30, k)

    for k in out:
        right(k, out[k])
    if pad:  # what lies between the rows is left alone
        for t in out.values():
            assert (t._base[:, t.shape[1]:] == 5).all()
    # each alone, and each pair (the work is then shared out in another way)
    for some in (["dx"], ["dw_up"], ["dw_down"], ["dx", "dw_down"], ["dw_up", "dw_down"]):
        part = {k: torch.full_like(out[k], float("nan")) for k in some}
        train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=ws, **part)
        for k in part:
            right(k, part[k])


@pytest.mark.parametrize("n,d,inner", [(1, 64, 64), (130, 264, 136), (4099, 64, 64)])
@pytest.mark.parametrize("grad_type", [BF, F32])
def test_accumulate(n, d, inner, grad_type):
    i = inputs(n, d, inner)
    dy, u = drawn(4, n, d, 0.1), drawn(5, n, 2 * inner)
    want = backward64(dy, u=u, **i)
    out = grads(n, d, inner, grad_type)
    before = {}
    for k in ("dw_up", "dw_down"):
        out[k].normal_(generator=torch.Generator(device="cuda").manual_seed(9))
        before[k] = out[k].to(F64)
    train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=train.ffn_workspace(n, d, inner), accumulate=True,
                       **out)
    close(out["dx"], want["dx"][0], 1.01 * (want["dx"][1] + HALF * (want["dx"][0].abs() + want["dx"][1])) + 1e-30, "dx")
    for k in before:
        g, e = want[k]
        g = g + before[k]
        rounding = HALF if grad_type == BF else 2.0 ** -23  # the sum, and for bf16 its rounding
        close(out[k], g, 1.01 * (e + rounding * (g.abs() + e) + 2.0 ** -24 * g.abs()) + 1e-30, k)


def test_gradient_against_differences():
    """The directional derivative of sum(dy * y) along a random direction, from central differences of the
    block in 64 bits, against the kernels' gradients.  The kernels' u is the rounded one, so they are compared
    where u is exactly representable: differences are taken of the block as a function of u and of x, W given u
    linear; here through the whole chain with the tolerance of one rounding of u, du, act and each output."""
    n, d, inner = 40, 64, 96
    i = inputs(n, d, inner, seed=50)
    dy = drawn(54, n, d, 0.1)
    _, u = run_forward(i)
    out = grads(n, d, inner, F32)
    train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=train.ffn_workspace(n, d, inner), **out)

    def loss(x, w_up, w_down):
        v = x @ w_up.T
        a, b = v[:, :inner], v[:, inner:]
        return (dy.to(F64) * ((a * torch.sigmoid(a) * b) @ w_down.T)).sum()

    at = {k: t.to(F64) for k, t in i.items()}
    g = torch.Generator(device="cuda").manual_seed(3)
    for k, out_k in (("x", "dx"), ("w_up", "dw_up"), ("w_down", "dw_down")):
        direction = torch.randn(at[k].shape, device="cuda", generator=g, dtype=F64)
        h = 1e-5
        up, down = ({**at, k: at[k] + s * h * direction} for s in (1, -1))
        slope = (loss(**up) - loss(**down)) / (2 * h)
        terms = (out[out_k].to(F64) * direction)
        # each gradient element is off by up to four roundings (u, du or act, the product, the output) of 2^-8 of its
        # size, independent in sign between elements: in the sum over elements, in norm
        assert (terms.sum() - slope).abs() <= 4 * HALF * 4 * terms.norm(), (k, float(terms.sum()), float(slope))


def test_no_tokens():
    d, inner = 64, 128
    i = inputs(1, d, inner)
    e = torch.empty((0, d), device="cuda", dtype=BF)
    ws = train.ffn_workspace(0, d, inner)
    train.ffn(e.clone(), e, i["w_up"], i["w_down"], u=torch.empty((0, 2 * inner), device="cuda", dtype=BF), workspace=ws)
    out = grads(0, d, inner, F32, pad=8)
    args = (e, e, torch.empty((0, 2 * inner), device="cuda", dtype=BF), i["w_up"], i["w_down"])
    train.ffn_backward(*args, workspace=ws, **out)
    assert (out["dw_up"] == 0).all() and (out["dw_down"] == 0).all()
    assert (out["dw_up"]._base[:, d:] == 5).all()
    out["dw_up"].fill_(3.0)
    train.ffn_backward(*args, workspace=ws, accumulate=True, **out)
    assert (out["dw_up"] == 3).all()


@pytest.mark.parametrize("big", [30.0, 300.0, 3e4])
def test_far_activations(big):
    """Where the sigmoid is 0 or 1 to the last bit the gradient is finite and follows the formula."""
    n, d, inner = 64, 64, 128
    i = inputs(n, d, inner)
    dy, u = drawn(4, n, d, 0.1), drawn(5, n, 2 * inner, big)
    want = backward64(dy, u=u, **i)
    out = grads(n, d, inner, F32)
    train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=train.ffn_workspace(n, d, inner), **out)
    for k, (g, e) in want.items():
        close(out[k], g, 1.01 * e + HALF * (g.abs() + e) + 1e-30, k)


def test_a_nan_stays_in_its_token():
    n, d, inner = 200, 256, 512
    i = inputs(n, d, inner)
    clean, _ = run_forward(i)
    i["x"][77, 3] = float("nan")
    y, u = run_forward(i)
    other = torch.arange(n, device="cuda") != 77
    assert torch.equal(y[other], clean[other])
    assert y[77].isnan().all() and u[77].isnan().all()


@pytest.mark.parametrize("n,d,inner", [(1, 256, 512), (200, 264, 520), (5000, 64, 64), (9, 4096, 8192), (700, 2048, 4096)])
def test_the_same_bits_every_time_and_on_another_stream(n, d, inner):
    i = inputs(n, d, inner)
    dy = drawn(4, n, d, 0.1)
    y, u = run_forward(i)
    first = grads(n, d, inner, BF)
    ws = train.ffn_workspace(n, d, inner)
    train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=ws, **first)
    torch.cuda.synchronize()
    for _ in range(3):
        ws.fill_(255)  # nothing is kept in a workspace
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = grads(n, d, inner, BF)
        torch.cuda.synchronize()
        y2, u2 = torch.empty_like(y), torch.empty_like(u)
        train.ffn(y2, i["x"], i["w_up"], i["w_down"], u=u2, workspace=ws, stream=side)
        train.ffn_backward(dy, i["x"], u2, i["w_up"], i["w_down"], workspace=ws, stream=side, **out)
        side.synchronize()
        assert torch.equal(y2, y) and torch.equal(u2, u)
        for k in out:
            assert torch.equal(out[k], first[k]), k


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    shapes = [(1000, 200, 504), (64, 256, 512)]
    ins = [inputs(*s, seed=10 * k) for k, s in enumerate(shapes)]
    want = [run_forward(i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    spaces = [train.ffn_workspace(*s) for s in shapes]
    outs = [(torch.empty_like(y), torch.empty_like(u)) for y, u in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (y, u), ws, s in zip(ins, outs, spaces, streams):
            train.ffn(y, i["x"], i["w_up"], i["w_down"], u=u, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (y, u), (y0, u0) in zip(outs, want):
        assert torch.equal(y, y0) and torch.equal(u, u0)


def test_captured_and_replayed():
    n, d, inner = 96, 256, 512
    i = inputs(n, d, inner)
    dy = drawn(4, n, d, 0.1)
    ws = train.ffn_workspace(n, d, inner)
    y, u = torch.empty((n, d), device="cuda", dtype=BF), torch.empty((n, 2 * inner), device="cuda", dtype=BF)
    out = grads(n, d, inner, BF)

    def step():
        train.ffn(y, i["x"], i["w_up"], i["w_down"], u=u, workspace=ws)
        train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=ws, **out)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):  # new contents between replays
        i["x"].copy_(drawn(seed + 70, n, d))
        graph.replay()
        got = [t.clone() for t in (y, u, *out.values())]
        step()
        for a, b in zip(got, (y, u, *out.values())):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n,ld", [(16, (1 << 28) + (1 << 26)), (300, 1 << 24), (600, 1 << 23)])
def test_offsets_past_32_bits(n, ld):
    """Rows so far apart that elements lie more than 2^32 from the first: the bits of the same call on packed
    tensors."""
    d, inner = 72, 136

    def far(t, rows_apart=ld):
        out = torch.empty((t.shape[0], rows_apart), device="cuda", dtype=t.dtype)[:, :t.shape[1]]
        assert (out.shape[0] - 1) * rows_apart > 1 << 32
        return out.copy_(t)

    i = inputs(n, d, inner)
    dy = drawn(4, n, d, 0.1)
    ws = train.ffn_workspace(n, d, inner)
    y, u = torch.empty((n, d), device="cuda", dtype=BF), torch.empty((n, 2 * inner), device="cuda", dtype=BF)
    want = grads(n, d, inner, F32)
    train.ffn(y, i["x"], i["w_up"], i["w_down"], u=u, workspace=ws)
    train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=ws, **want)
    x, w_up, fy, fu = far(i["x"]), far(i["w_up"], 1 << 24), far(torch.zeros_like(y)), far(torch.zeros_like(u))
    train.ffn(fy, x, w_up, i["w_down"], u=fu, workspace=ws)
    assert torch.equal(fy, y) and torch.equal(fu, u)
    del fy
    got = {**grads(n, d, inner, F32), "dx": far(torch.zeros_like(y)), "dw_up": far(torch.zeros_like(want["dw_up"]), 1 << 24)}
    train.ffn_backward(far(dy), x, fu, w_up, i["w_down"], workspace=ws, **got)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    del x, w_up, fu, got
    torch.cuda.empty_cache()


def test_refused_sizes():
    i = inputs(4, 64, 128)
    with pytest.raises(sol.SolError, match="below the"):
        run_forward(i, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sol.SolError, match="overlaps"):
        train.ffn(i["x"], i["x"], i["w_up"], i["w_down"], workspace=train.ffn_workspace(4, 64, 128))
