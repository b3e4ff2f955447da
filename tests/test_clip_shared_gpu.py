"""A tensor listed twice: it counts twice in the norm, and cannot be written twice in one call."""
import math

import pytest
import torch

import gated_delta_rule_42_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_42_gb300 import build
    build.build()


def test_a_tensor_is_written_once():
    a, b = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises(ValueError, match=r"tensors\[2\] shares its memory with tensors\[0\]"):
        kda.clip_grad_norm([a, b, a], 1.0)
    with pytest.raises(ValueError, match=r"out\[1\] shares its memory with out\[0\]"):
        kda.clip_grad_norm([a, b], 1.0, out=[b, b])
    assert (a == 1).all() and (b == 1).all()


def test_a_tensor_is_read_twice():
    a = torch.ones(8, device="cuda")
    out = [torch.empty_like(a), torch.empty_like(a)]
    assert float(kda.clip_grad_norm([a, a], 2.0, out=out)) == 4.0
    assert all(torch.allclose(o, torch.full_like(o, 0.5)) for o in out)


def test_empty_tensors_may_share_an_address():
    e = torch.empty(0, device="cuda")
    t = torch.ones(4, device="cuda")
    assert float(kda.clip_grad_norm([e, t, e, torch.empty(0, 3, device="cuda")], 1.0)) == 2.0
    assert math.isclose(float(t.square().sum()), 1.0, rel_tol=1e-5)
