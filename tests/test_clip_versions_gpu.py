"""Clipping counts as a modification of what it writes: autograd refuses a backward whose
saved tensor it changed."""
import math

import pytest
import torch

import gated_delta_rule_42_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_42_gb300 import build
    build.build()


def test_version_counters():
    a, b = torch.ones(40, device="cuda"), torch.ones(3, device="cuda", dtype=torch.bfloat16)
    kda.clip_grad_norm([a, b], 0.5)
    assert (a._version, b._version) == (1, 1)
    out = [torch.empty_like(a), torch.empty_like(b)]
    was = a._version, out[0]._version, out[1]._version
    kda.clip_grad_norm([a, b], 0.5, out=out)
    assert (a._version, out[0]._version, out[1]._version) == (was[0], was[1] + 1, was[2] + 1)
    kda.clip_grad_norm([a, b], math.inf)  # the norm alone: nothing is written
    assert (a._version, b._version) == (1, 1)


def test_autograd_sees_the_modification():
    x = torch.ones(8, device="cuda", requires_grad=True)
    saved = torch.full((8,), 2.0, device="cuda")
    loss = (x * saved).sum()
    kda.clip_grad_norm([saved], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_clipped():
    with torch.inference_mode():
        t = torch.full((16,), 3.0, device="cuda")
        assert float(kda.clip_grad_norm([t], 1.0)) == 12.0
    assert torch.allclose(t.clone(), torch.full((16,), 0.25, device="cuda"))
