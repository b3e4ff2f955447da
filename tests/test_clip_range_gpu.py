"""The gradients' norm over the whole range of fp32: squares of large elements pass
fp32, squares of small ones fall below it, and the norm of either is ordinary."""
import math

import pytest
import torch

import gated_delta_rule_42_gb300 as kda
from tests.test_dense_gpu import BF16, E32, F32, check_clip, gen, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_42_gb300 import build
    build.build()


# whole chunks, ragged ones, and elements off the 16-byte grid
@pytest.mark.parametrize("size,by", [(8192, 0), (3 * 8192 + 5, 0), (1000, 0), (20001, 1), (1, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-36, 1e-28, 1e-23, 1e-20, 1e-17, 1.0, 4e18, 2e19, 1e28, 1e33])
def test_norm_over_the_range(size, by, dtype, scale):
    g = rnd(gen(size), size + by)
    # sizes between half and twice `scale`, so that no element hides behind a larger one
    t = (torch.sign(g) * (0.5 + g.abs().clamp(max=1.5)) * scale).to(dtype)[by:]
    check_clip([t], 1.0, [torch.empty_like(t)])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_and_small_together(dtype):
    """One chunk and one thread with both: the large ones are the norm, and nothing overflows."""
    t = torch.full((8192 * 2 + 77,), 1e-25, device="cuda").to(dtype)
    t[5], t[8192 + 64] = 3e30, -4e30
    check_clip([t, torch.zeros(9000, device="cuda"), torch.full((50,), 1e-30, device="cuda")], 1e29,
               [torch.empty_like(t), torch.empty(9000, device="cuda"), torch.empty(50, device="cuda")])


def test_largest_values():
    big = torch.finfo(F32).max
    t = torch.tensor([big, 0.0, 0.0], device="cuda")
    assert abs(float(kda.clip_grad_norm([t], math.inf)) / big - 1) <= 40 * E32
    small = torch.tensor([2.0 ** -149, 0.0], device="cuda")
    assert float(kda.clip_grad_norm([small], 1.0)) == 2.0 ** -149


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("size", [8192, 300])
def test_not_finite_beside_large_and_small(bad, size):
    for other in (1e-30, 1e25):
        t = torch.full((size,), other, device="cuda")
        t[size // 2] = bad
        norm = float(kda.clip_grad_norm([t], math.inf))
        assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
