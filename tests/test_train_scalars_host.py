"""Host-side checks of an AdamW step's scalars (no GPU: each call is refused, at last for want of a plan), and of
where workspaces lie."""
from __future__ import annotations

import ctypes

import pytest

from dit_block_b200 import build, sol
from test_train_host import last, scalars

from dit_block_b200 import train


@pytest.fixture(scope="module")
def L():
    build.build()
    return train.lib()


@pytest.mark.parametrize("eps,word", [
    (5e-324, "eps"), (1e-50, "eps"), (1e-45, "eps"), (1e-39, "eps"), (1.17e-38, "eps"),  # zero or subnormal in fp32
    (0.0, "plan is NULL"), (2.0 ** -126, "plan is NULL"), (1e-30, "plan is NULL"), (1e-8, "plan is NULL"),
])
def test_eps_is_zero_or_a_normal_number_of_fp32(L, eps, word):
    assert L.sol_adamw_step(None, ctypes.byref(scalars(eps=eps)), None) == sol.ERR_INVALID_ARGUMENT
    assert word in last(L), last(L)


@pytest.mark.parametrize("device,want", [(None, "cuda"), (0, 0), ("cuda:0", "cuda:0"), (1, 1)])
def test_a_workspace_lies_on_the_device_asked_for(L, monkeypatch, device, want):
    """Device 0 is a device, not "the current one"."""
    asked = []
    monkeypatch.setattr(train.torch, "empty", lambda *a, device, **kw: asked.append(device))
    train.ffn_workspace(4, 64, 64, device=device)
    sol.adaln_workspace(4, 256, 256, device=device)
    assert asked == [want] * 2 and all(type(a) is type(want) for a in asked)
