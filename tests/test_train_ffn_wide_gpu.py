"""GPU tests of the feed-forward's largest tiles: a CTA pair on 512 x 256, which long calls take, at sizes whose
tokens and widths end inside a tile and a k-block.  Bounds as in test_train_ffn_gpu."""
from __future__ import annotations

import pytest
import torch

from dit_block_b200 import sol, train
from test_train_ffn_gpu import BF, F32, F64, HALF, backward64, close, drawn, forward64, grads, inputs, run_forward

pytestmark = pytest.mark.gpu

# n_tokens, d, inner.  On 512 x 256: the up projection of all, with last tiles that are shared out between workers in the
# first; the down projection of the first and third; dx and both weight gradients in one launch of all but the second, the
# last tiles shared out but in the last.
SIZES = [(2349, 3472, 3728), (1841, 2328, 3752), (2465, 3592, 5328), (2803, 3120, 528)]


@pytest.fixture(scope="module", autouse=True)
def _flags():
    sol.device_errors(clear=True)
    yield
    assert sol.device_errors() == 0


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


@pytest.mark.parametrize("n,d,inner", SIZES)
@pytest.mark.parametrize("grad_type", [BF, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("pad", [0, 8])
def test_backward(n, d, inner, grad_type, accumulate, pad):
    """Weight gradients of both types, set and added to; alone they are shared out in another way than beside dx."""
    i = inputs(n, d, inner, pad)
    dy, u = drawn(4, n, d, 0.1, pad), drawn(5, n, 2 * inner, 2.0, pad)
    want = backward64(dy, u=u, **i)
    ws = train.ffn_workspace(n, d, inner)
    for names in (("dx", "dw_up", "dw_down"), ("dw_up",), ("dw_down",)):
        out = {k: t for k, t in grads(n, d, inner, grad_type, pad).items() if k in names}
        before = {}
        for k in names:
            if accumulate and k != "dx":
                out[k].normal_(generator=torch.Generator(device="cuda").manual_seed(9))
                before[k] = out[k].to(F64)
        train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=ws, accumulate=accumulate, **out)
        for k, got in out.items():
            g, e = want[k]
            # the sum with what was there is one fp32 rounding more, then the output's own
            more = 0.0
            if k in before:
                g = g + before[k]
                more = 2.0 ** -24 * (g.abs() + e)
            rounding = HALF if got.dtype == BF else 2.0 ** -24
            close(got, g, 1.01 * (e + more + rounding * (g.abs() + e + more)) + 1e-30, k)
            if pad:
                assert (got._base[:, got.shape[1]:] == 5).all(), f"{k}: written between its rows"
    if grad_type == BF and not accumulate:
        # dx is the same whatever the weight gradients' type
        alone, again = (torch.empty((n, d), device="cuda", dtype=BF) for _ in range(2))
        f32 = {k: torch.empty(s, device="cuda") for k, s in (("dw_up", (2 * inner, d)), ("dw_down", (d, inner)))}
        bf = {k: t.to(BF) for k, t in f32.items()}
        train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=ws, dx=alone, **f32)
        train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=ws, dx=again, **bf)
        assert torch.equal(alone, again)
        for k in bf:  # and a bf16 gradient is the f32 one, rounded once
            assert torch.equal(bf[k], f32[k].to(BF)), k


def test_pre_activations_past_32_bits():
    """80,000 tokens of width 13,824: u and du hold more than 2^31 values.  dy is zero but for the first and the last
    tokens, so that the weight gradients are those tokens' alone; zero terms of a sum add no error."""
    n, d, inner, ends = 80_000, 64, 13_824, 150
    assert 2 * n * inner > 1 << 31
    i = inputs(n, d, inner)
    some = torch.cat([torch.arange(ends), torch.arange(n - ends, n)]).cuda()
    y, u = run_forward(i)
    u64, eu, y64, ey = forward64(i["x"][some], i["w_up"], i["w_down"])
    close(u[some], u64, eu, "u")
    close(y[some], y64, ey, "y")
    dy = torch.zeros((n, d), device="cuda", dtype=BF)
    dy[some] = drawn(4, 2 * ends, d, 0.1)
    out = grads(n, d, inner, F32)
    train.ffn_backward(dy, i["x"], u, i["w_up"], i["w_down"], workspace=train.ffn_workspace(n, d, inner), **out)
    want = backward64(dy[some], i["x"][some], u[some], i["w_up"], i["w_down"])
    assert (out["dx"][ends:-ends] == 0).all()
    out["dx"] = out["dx"][some]
    for k, got in out.items():
        g, e = want[k]
        rounding = HALF if got.dtype == BF else 2.0 ** -24
        close(got, g, 1.01 * (e + rounding * (g.abs() + e)) + 1e-30, k)
    del u, y, out, want
    torch.cuda.empty_cache()
