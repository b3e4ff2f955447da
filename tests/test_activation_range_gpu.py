"""The linear layer's activations and their slopes over z in [-20, 20], relative to
their own size: the tails are small, and a term that cancels there loses them whole.

A layer of one input with weight 1 is its activation: y = act(z), and with dy = 1 its
dx is the slope at the pre-activation.  Bounds count steps of fp32 (E32): expf is off
by 2, erfcf by 4, an addition, product or quotient by half of one."""
import math

import pytest
import torch

import gated_delta_rule_42_gb300 as kda
from tests.test_dense_gpu import BF16, E32, F32, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_42_gb300 import build
    build.build()


def points(dtype):
    z = torch.linspace(-20, 20, 40001, device="cuda", dtype=torch.float64).to(dtype)
    return torch.unique(z)


def exact(z, act):
    """(value, slope, size of the slope's terms) in 64 bits, without cancellation."""
    e = torch.exp(-z.abs())
    p = torch.where(z < 0, e, torch.ones_like(e)) / (1 + e)
    dp = e / (1 + e) ** 2
    if act == "sigmoid":
        return p, dp, dp
    if act == "silu":
        return z * p, p + z * dp, p + (z * dp).abs()
    c = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    d = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z * c, c + z * d, c + (z * d).abs()


def steps(z, act, dtype):
    """Relative error of the value's and the slope's terms, in steps of fp32."""
    if dtype == BF16:
        return 32 + z.abs()  # the exponential's argument is rounded once: |z| / 2 of a step and the instruction's two
    if act == "gelu":  # z / sqrt 2 is rounded twice, and the tail's exponent is z^2 / 2 of it
        return 16 + 2 * z * z
    return 8 + z.abs() * (act == "silu")  # silu's 1 - p is a difference, times z


def close(name, got, ref, bound):
    d = (got.double() - ref).abs() - bound
    i = int(d.argmax())
    assert float(d[i]) <= 0, (name, i, float(got[i]), float(ref[i]), float(bound[i]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
def test_value_and_slope(act, dtype):
    z = points(dtype)
    one = torch.ones(1, 1, device="cuda", dtype=dtype)
    value, slope, size = exact(z.double(), act)
    n = steps(z.double(), act, dtype) * E32
    # erfc's approximation in bf16 is 1.5e-7 off and 1 - erfc / 2 rounds once: absolute terms
    lost = 0.75e-7 + E32 if act == "gelu" and dtype == BF16 else 0.0
    tiny = 2.0 ** -120  # values below fp32's normal numbers are lost
    u = U[dtype]
    b_value = u * value.abs() + (1 + u) * (n * value.abs() + lost * z.double().abs()) + tiny
    b_slope = u * slope.abs() + (1 + u) * (n * size + lost) + tiny
    rows = z.view(-1, 1).contiguous()
    close("value", kda.linear_fwd(rows, one, activation=act)[0].view(-1), value, b_value)
    close("value of one row", kda.linear_fwd(one, rows, activation=act)[0].view(-1), value, b_value)
    dx, _, _ = kda.linear_bwd(torch.ones_like(rows), rows, one, activation=act, preact=rows, need_dweight=False)
    close("slope", dx.view(-1), slope, b_slope)


def test_sigmoid_slope_is_symmetric():
    z = points(F32)
    rows, one = z.view(-1, 1).contiguous(), torch.ones(1, 1, device="cuda")
    d = [kda.linear_bwd(torch.ones_like(rows), rows, one, activation="sigmoid", preact=s * rows, need_dweight=False)[0]
         for s in (1, -1)]
    assert torch.equal(d[0], d[1]) and bool((d[0] > 0).all())
