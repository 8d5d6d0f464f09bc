"""GPU tests of the fine-tuning path (dit_block_b200.finetune): forward, backward, clipped AdamW step together,
against the same formulas in 64 bits and against itself captured in a CUDA graph."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from dit_block_b200 import finetune, sol, workloads as wl
from test_train_adamw_gpu import F64, check, formula
from test_train_ffn_gpu import HALF, backward64, close, forward64

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
TINY = wl.WORKLOADS["tiny"]


def weights(d=TINY.d, inner=TINY.inner):
    w_up = wl.linear_weight(TINY, "w_up", 2 * inner, d, "cuda")
    return w_up.to(BF), wl.linear_weight(TINY, "w_down", d, inner, "cuda").to(BF)


def tokens(n, seed, d=TINY.d, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, d, device="cuda", generator=g) * std).to(BF)


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("n", [1, 32, 300])
def test_steps_follow_the_formulas(n, state_bits):
    ff = finetune.FeedForward(*weights(), 300, state_bits=state_bits, weight_decay=0.01, seed=3)
    ff.lr.fill_(1e-3)
    lr = float(ff.lr)
    for step in range(1, 4):
        x, dy = tokens(n, step), tokens(n, 10 + step, std=0.1)
        copies = [w.clone() for w in ff.weights]
        before = [p.clone() for p in ff.params]
        moments = ff.moments()
        y = ff.forward(x)
        u64, eu, y64, ey = forward64(x, *copies)
        close(y, y64, ey, "y")
        assert torch.equal(ff.infer(x, torch.empty_like(x)), y)
        u = ff.u[:n].clone()
        dx = ff.backward(dy)
        want = backward64(dy, x, u, *copies)
        for k, got in (("dx", dx), ("dw_up", ff.grads[0]), ("dw_down", ff.grads[1])):
            g, e = want[k]
            rounding = HALF if got.dtype == BF else 2.0 ** -24
            close(got, g, 1.01 * (e + rounding * (g.abs() + e)) + 1e-30, k)
        ff.update(max_norm=0.5)
        norm = torch.cat([g.to(F64).flatten() for g in ff.grads]).norm()
        assert abs(ff.norm[0].double() - norm) <= 20 * 2.0 ** -24 * norm
        factor = float(ff.norm[1])
        assert factor <= min(1.0, 0.5 / float(norm)) * (1 + 1e-6)
        for k in range(2):
            p, m, v = formula(before[k], ff.grads[k], *moments[k], 0.01, step, factor, lr=lr)
            # the factor times the gradient is one rounding more than formula() counts
            more = 2.0 ** -22 * lr * ((p[0] - before[k].to(F64)).abs() / lr)
            check(ff.params[k], (p[0], p[1] + more), "parameters")
            assert torch.equal(ff.weights[k], ff.params[k].to(BF))
            if state_bits == 32:
                check(ff.m[k], (m[0], 2 * m[1]), "first moment")
                check(ff.v[k], (v[0], 2 * v[1]), "second moment")
    assert int(ff.step) == 3
    assert sol.device_errors() == 0
    ff.close()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_captured_steps_are_the_eager_ones(state_bits):
    n = 48
    eager, captured = (finetune.FeedForward(*weights(), n, state_bits=state_bits, seed=7) for _ in range(2))
    x, dy = tokens(n, 1), tokens(n, 2, std=0.1)
    graph = captured.capture(x, dy, max_norm=1.0)
    for step in range(3):
        x.copy_(tokens(n, 20 + step))
        dy.copy_(tokens(n, 30 + step, std=0.1))
        for ff in (eager, captured):
            ff.lr.fill_(1e-3 / (step + 1))
        eager.forward(x)
        eager.backward(dy)
        eager.update(1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((eager.params, captured.params), (eager.m, captured.m), (eager.v, captured.v),
                     (eager.grads, captured.grads), ([eager.dx, eager.norm], [captured.dx, captured.norm])):
            for s, t in zip(a, b):
                assert torch.equal(s, t)
    assert int(captured.step) == 3
    del graph
    eager.close()
    captured.close()


def test_gradients_of_two_batches_add_up():
    ff = finetune.FeedForward(*weights(), 64)
    parts = [(tokens(40, 1), tokens(40, 2, std=0.1)), (tokens(24, 3), tokens(24, 4, std=0.1))]
    want = {"dw_up": 0, "dw_down": 0}
    bound = {"dw_up": 0, "dw_down": 0}
    for k, (x, dy) in enumerate(parts):
        ff.forward(x)
        g = backward64(dy, x, ff.u[:x.shape[0]], *ff.weights)
        ff.backward(dy, accumulate=k > 0)
        for name in want:
            want[name] = want[name] + g[name][0]
            bound[name] = bound[name] + g[name][1] + 2.0 ** -22 * want[name].abs()
    close(ff.grads[0], want["dw_up"], bound["dw_up"] + 1e-30, "dw_up")
    close(ff.grads[1], want["dw_down"], bound["dw_down"] + 1e-30, "dw_down")
    ff.close()


def test_misuse():
    w = weights()
    with pytest.raises(ValueError, match="w_up must be"):
        finetune.FeedForward(w[0][:-8], w[1], 8)
    with pytest.raises(ValueError, match="state_bits"):
        finetune.FeedForward(*w, 8, state_bits=16)
    ff = finetune.FeedForward(*w, 8)
    with pytest.raises(RuntimeError, match="forward before"):
        ff.backward(tokens(8, 1))
    with pytest.raises(ValueError, match="max_tokens"):
        ff.forward(tokens(9, 1))
    with pytest.raises(ValueError, match="dy must be"):
        ff.forward(tokens(8, 1))
        ff.backward(tokens(7, 1))
    ff.close()


def test_workspace_and_sizes_of_the_full_block():
    """The full-size block at one token and at a few hundred (d 5120, width 13,824)."""
    w = wl.WORKLOADS["lowres"]
    ff = finetune.FeedForward(wl.linear_weight(w, "w_up", 2 * w.inner, w.d, "cuda"),
                              wl.linear_weight(w, "w_down", w.d, w.inner, "cuda"), 260, state_bits=8, grad_dtype=BF)
    ff.lr.fill_(1e-4)
    for n in (1, 260):
        x, dy = tokens(n, n, w.d), tokens(n, n + 1, w.d, std=0.1)
        copies = [t.clone() for t in ff.weights]
        y = ff.forward(x)
        _, _, y64, ey = forward64(x, *copies)
        close(y, y64, ey, "y")
        u = ff.u[:n].clone()
        dx = ff.backward(dy)
        want = backward64(dy, x, u, *copies)
        for k, got in (("dx", dx), ("dw_up", ff.grads[0]), ("dw_down", ff.grads[1])):
            g, e = want[k]
            close(got, g, 1.01 * (e + HALF * (g.abs() + e)) + 1e-30, k)
        ff.update(1.0)
        assert all(torch.isfinite(p).all() for p in ff.params)
    ff.close()


def test_capture_as_the_first_use_of_a_process():
    """Nothing is set up on the side by an eager call that a capture could not do by itself."""
    code = """
import torch
from dit_block_b200 import finetune, sol
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
for n in (8, 300):
    x, dy = r(n, 256), r(n, 256)
    up, down = r(1024, 256) / 16, r(256, 512) / 16
    a, b = (finetune.FeedForward(up, down, n, state_bits=8) for _ in range(2))
    a.lr.fill_(1e-3); b.lr.fill_(1e-3)
    graph = a.capture(x, dy, 1.0)
    graph.replay()
    b.forward(x); b.backward(dy); b.update(1.0)
    torch.cuda.synchronize()
    for s, t in zip([a.y, a.dx, *a.grads, *a.params], [b.y, b.dx, *b.grads, *b.params]):
        assert torch.equal(s, t)
    del graph
    a.close(); b.close()
assert sol.device_errors() == 0
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
