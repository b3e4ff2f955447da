"""What the linear layer's autograd form keeps for its backward, without a GPU: the
kernels are replaced, the call that would run them is looked at."""
import pytest
import torch

from gated_delta_rule_42_gb300 import dense


@pytest.fixture
def kept(monkeypatch):
    """The keep_preact of every forward."""
    seen = []

    def forward(x, weight, bias, activation, residual, keep_preact=False):
        seen.append(keep_preact)
        y = x @ weight.t()
        return y, y.clone() if keep_preact and activation is not None else None
    monkeypatch.setattr(dense, "linear_fwd", forward)
    return seen


def layer():
    return torch.randn(3, 4), torch.nn.Parameter(torch.randn(5, 4)), torch.nn.Parameter(torch.randn(5))


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_without_gradients(kept, mode):
    x, w, b = layer()
    with mode():
        y = dense.linear(x, w, b, activation="silu")
    assert kept == [False] and not y.requires_grad


def test_frozen_layers_keep_nothing(kept):
    x, w, b = layer()
    dense.linear(x, w.detach(), b.detach(), activation="silu")
    assert kept == [False]


def test_the_preactivation_is_kept_for_a_backward(kept, monkeypatch):
    x, w, b = layer()
    calls = []

    def backward(dy, x, weight, bias, activation, preact, need_dx, need_dweight):
        calls.append((preact is not None, need_dx, need_dweight))
        return None, torch.ones_like(weight), torch.ones_like(bias)
    monkeypatch.setattr(dense, "linear_bwd", backward)
    with torch.no_grad():
        with torch.enable_grad():
            y = dense.linear(x, w, b, activation="silu")
    y.sum().backward()
    assert kept == [True] and calls == [(True, False, True)]
    assert (w.grad == 1).all() and (b.grad == 1).all()


def test_a_problem_too_large_says_so(monkeypatch):
    """The library's refusal reaches the caller, not the allocator's error on a workspace of SIZE_MAX bytes."""
    from gated_delta_rule_42_gb300 import _lib, build
    build.build()
    monkeypatch.setattr(dense, "_check_input", lambda name, t: None)
    monkeypatch.setattr(dense, "_stream", lambda device: None)
    x = torch.empty(1, (1 << 24) + 8, dtype=torch.bfloat16)
    with pytest.raises(_lib.KdaError, match="linear: problem too large"):
        dense.linear_fwd(x, x)
    with pytest.raises(_lib.KdaError, match="linear: problem too large"):
        dense.linear_bwd(torch.empty(1, 1, dtype=torch.bfloat16), x, x)
