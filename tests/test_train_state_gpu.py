"""GPU tests of what calls leave behind: the fine-tuning object after captures and refused calls, and the clip factor
where nothing is clipped."""
from __future__ import annotations

import gc
import weakref

import pytest
import torch

from dit_block_b200 import finetune, sol, train
from test_finetune_gpu import BF, tokens, weights
from test_train_adamw_gpu import norm_of, tensors

pytestmark = pytest.mark.gpu

INF = float("inf")


def test_nothing_is_clipped_without_a_limit():
    """max_norm infinite: the factor is 1 for an infinite norm too, so that the gradient that made it so stays
    with its own value; a NaN norm still shows."""
    one = lambda *v: [torch.tensor(v, device="cuda")]  # noqa: E731
    assert norm_of(one(INF, 1.0), max_norm=INF) == [INF, 1.0]
    assert norm_of(one(-INF, 0.0), max_norm=INF) == [INF, 1.0]
    assert norm_of(one(torch.finfo(torch.float32).max, 0.0), max_norm=INF)[1] == 1.0
    n, f = norm_of(one(float("nan"), 1.0), max_norm=INF)
    assert n != n and f != f
    assert norm_of(one(INF, 1.0), max_norm=1e38) == [INF, 0.0]


@pytest.mark.parametrize("bits", [32, 8])
def test_an_infinite_gradient_stays_with_its_value(bits):
    t = tensors([1000, 300], bits=bits)
    t["grads"][0][700] = INF
    with train.AdamW(**t) as opt:
        out = torch.zeros(2, device="cuda")
        opt.grad_norm(out, INF, workspace=opt.norm_workspace())
        opt.step(step=1, lr=1e-3, grad_factor=out[1:])
    bad = t["params"][0].isnan()
    assert bad[700] and bad.sum() == 1 and torch.isfinite(t["params"][1]).all()


def parts(ff, dy):
    return [t.clone() for t in (ff.backward(dy), *ff.grads)]


def test_a_capture_leaves_the_last_forward_as_it_was():
    ff = finetune.FeedForward(*weights(), 64)
    x, dy = tokens(64, 1), tokens(64, 2, std=0.1)
    ff.forward(x)
    want = parts(ff, dy)
    ff.forward(x)
    other = ff.capture(tokens(40, 3), tokens(40, 4))
    for a, b in zip(parts(ff, dy), want):
        assert torch.equal(a, b)
    del other
    ff.close()


def test_a_capture_is_no_forward():
    ff = finetune.FeedForward(*weights(), 8)
    graph = ff.capture(tokens(8, 1), tokens(8, 2))
    with pytest.raises(RuntimeError, match="forward before"):
        ff.backward(tokens(8, 2))
    del graph
    ff.close()


def test_a_refused_forward_leaves_the_last_one_as_it_was():
    ff = finetune.FeedForward(*weights(), 64)
    x, dy = tokens(64, 1), tokens(64, 2, std=0.1)
    y = ff.forward(x)
    want = parts(ff, dy)
    ff.forward(x)
    with pytest.raises(sol.SolError, match="overlaps"):
        ff.forward(y)
    with pytest.raises(TypeError, match="x must be"):
        ff.forward(x.float())
    for a, b in zip(parts(ff, dy), want):
        assert torch.equal(a, b)
    ff.close()


def test_a_refused_update_is_no_step():
    a, b = (finetune.FeedForward(*weights(), 8) for _ in range(2))
    x, dy = tokens(8, 1), tokens(8, 2)
    for ff in (a, b):
        ff.lr.fill_(1e-3)
        ff.forward(x)
        ff.backward(dy)
    with pytest.raises(sol.SolError, match="max_norm"):
        a.update(-1.0)
    a.betas = (0.9, 1.0)
    with pytest.raises(sol.SolError, match="beta1 and beta2"):
        a.update(1.0)
    a.betas = b.betas
    assert int(a.step) == 0
    for ff in (a, b):
        ff.update(1.0)
    for p, q in zip(a.params, b.params):
        assert torch.equal(p, q)
    a.close()
    b.close()


def test_a_graph_keeps_what_it_reads():
    """The buffers that a captured step reads live as long as the graph, whoever else holds them."""
    ff = finetune.FeedForward(*weights(), 8)
    x, dy = tokens(8, 1), tokens(8, 2)
    seen = [weakref.ref(t) for t in (x, dy, ff)]
    graph = ff.capture(x, dy)
    del x, dy, ff
    gc.collect()
    assert all(r() is not None for r in seen)
    graph.replay()
    torch.cuda.synchronize()
    del graph
    gc.collect()
    assert all(r() is None for r in seen)


@pytest.mark.parametrize("default", [BF, torch.float64])
def test_buffers_do_not_follow_the_default_type(default):
    w = weights()
    torch.set_default_dtype(default)
    try:
        ff = finetune.FeedForward(*w, 8, state_bits=8)
        ff.lr.fill_(1e-3)
        ff.forward(tokens(8, 1))
        ff.backward(tokens(8, 2).to(BF))
        ff.update(1.0)
        assert int(ff.step) == 1 and ff.moments()[0][0].dtype is torch.float32
    finally:
        torch.set_default_dtype(torch.float32)
    ff.close()


def test_a_replay_ends_the_last_forward():
    """A replay writes the pre-activation that an eager backward would read, and new weights."""
    ff = finetune.FeedForward(*weights(), 8)
    x, dy = tokens(8, 1), tokens(8, 2)
    graph = ff.capture(x, dy)
    ff.forward(tokens(8, 3))
    graph.replay()
    with pytest.raises(RuntimeError, match="forward before"):
        ff.backward(dy)
    ff.forward(x)
    ff.backward(dy)
    torch.cuda.synchronize()
    del graph
    ff.close()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_plan_let_go_of_during_a_capture(bits):
    """Freeing a plan that the captured stream does not use, as the garbage collector may at any time."""
    t, ref = tensors([1000], bits=bits), tensors([1000], bits=bits)
    opt, other = train.AdamW(**t), train.AdamW(**tensors([500], bits=bits))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(step=1, lr=1e-3)
        other.close()
        opt.step(step=2, lr=1e-3)
    graph.replay()
    with train.AdamW(**ref) as eager:
        for step in (1, 2):
            eager.step(step=step, lr=1e-3)
    torch.cuda.synchronize()
    for k in t:
        assert torch.equal(t[k][0], ref[k][0]), k
    del graph
    opt.close()
