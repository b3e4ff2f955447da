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
    with pytest.raises(RuntimeError, match="outputs 0 and 2 overlap"):
        kda.clip_grad_norm([a, b, a], 1.0)
    with pytest.raises(RuntimeError, match="outputs 0 and 1 overlap"):
        kda.clip_grad_norm([a, b], 1.0, out=[b, b])
    with pytest.raises(RuntimeError, match="outputs 1 and 0 overlap"):
        kda.clip_grad_norm([a[4:], a[:5]], 1.0)
    assert (a == 1).all() and (b == 1).all()


def test_views_of_one_buffer_in_any_order():
    for cuts in ([(0, 4), (4, 8), (8, 16)], [(8, 16), (0, 4), (4, 8)], [(4, 8), (4, 4), (8, 16), (0, 4), (8, 8)]):
        a = torch.ones(16, device="cuda")
        assert float(kda.clip_grad_norm([a[i:j] for i, j in cuts], 2.0)) == 4.0
        assert torch.allclose(a, torch.full_like(a, 0.5))


def test_a_tensor_is_read_twice():
    a = torch.ones(8, device="cuda")
    out = [torch.empty_like(a), torch.empty_like(a)]
    assert float(kda.clip_grad_norm([a, a], 2.0, out=out)) == 4.0
    assert all(torch.allclose(o, torch.full_like(o, 0.5)) for o in out)


def test_the_norm_alone_of_a_tensor_listed_twice():
    a = torch.ones(8, device="cuda")
    assert float(kda.clip_grad_norm([a, a], math.inf)) == 4.0 and (a == 1).all()
    with pytest.raises(RuntimeError, match="overlap"):  # here the outputs are written
        kda.clip_grad_norm([a, a], math.inf, out=[torch.empty_like(a)] * 2)


def test_empty_tensors_may_share_an_address():
    e = torch.empty(0, device="cuda")
    t = torch.ones(4, device="cuda")
    assert float(kda.clip_grad_norm([e, t, e, torch.empty(0, 3, device="cuda")], 1.0)) == 2.0
    assert math.isclose(float(t.square().sum()), 1.0, rel_tol=1e-5)
