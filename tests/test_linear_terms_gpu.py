"""The linear layer's products with bounds tight enough that no term can be missing.

With an activation the worst case of dz's own roundings grows with the number of
terms until it covers a lost row.  So the products are checked apart from them: without
an activation; against products of the bf16 dz itself, made from the kept
pre-activation; and with operands that hold nothing but their last row or column."""
import pytest
import torch

import gated_delta_rule_42_gb300 as kda
from tests.test_dense_gpu import (BF16, E32, F32, LINEAR_SHAPES, U, act64, check_linear, dirty, gen, make_linear, rnd,
                                  within)

pytestmark = pytest.mark.gpu
IDS = ["x".join(map(str, s)) for s in LINEAR_SHAPES]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_42_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("i", range(len(LINEAR_SHAPES)), ids=IDS)
def test_without_activation(i, dtype):
    x, w, b, r, dy = make_linear(gen(100 + i), *LINEAR_SHAPES[i], dtype)
    check_linear(x, w, b, None, r, dy)


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("i", range(len(LINEAR_SHAPES)), ids=IDS)
def test_products_of_the_rounded_dz(i, act):
    """dx and dweight of bf16 against 64-bit products of dz rounded to bf16; a dz that lies so near a rounding
    border that fp32 may put it on either side is allowed both."""
    rows, outs, ins = LINEAR_SHAPES[i]
    x, w, b, _, dy = make_linear(gen(200 + i), rows, outs, ins, BF16)
    _, z = kda.linear_fwd(x, w, b, activation=act, keep_preact=True)
    dirty()
    dx, dw, _ = kda.linear_bwd(dy, x, w, b, activation=act, preact=z)
    zd, dyd, xd, wd = z.double(), dy.double(), x.double(), w.double()
    dz = dyd * act64(zd, act)[1]
    e = 16 * E32 * (1 + zd.abs()) * dyd.abs()
    dzb, either = dz.to(BF16).double(), (dz + e).to(BF16).double() - (dz - e).to(BF16).double()
    for name, got, ref, size, border, terms in (
            ("dx", dx, dzb @ wd, dzb.abs() @ wd.abs(), either @ wd.abs(), outs),
            ("dweight", dw, dzb.t() @ xd, dzb.abs().t() @ xd.abs(), either.t() @ xd.abs(), rows)):
        u = U[BF16]
        within(name, got, ref, u * ref.abs() + (1 + u) * (1.01 * border + (terms + 8) * E32 * size))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("i", range(len(LINEAR_SHAPES)), ids=IDS)
def test_the_last_terms_alone(i, dtype):
    """Each product with one term only, the last: a row of dz^T x, a column of dz W, a k of x W^T."""
    rows, outs, ins = LINEAR_SHAPES[i]
    g = gen(300 + i)
    x, w, dy = rnd(g, rows, ins, dtype=dtype), rnd(g, outs, ins, dtype=dtype), rnd(g, rows, outs, dtype=dtype)
    xk = torch.zeros_like(x)
    xk[:, -1] = x[:, -1]
    y, _ = kda.linear_fwd(xk, w)
    assert torch.equal(y, (x[:, -1:].float() * w[:, -1].float()).to(dtype))
    last = torch.zeros_like(dy)
    last[-1] = dy[-1]
    _, dw, _ = kda.linear_bwd(last, x, w, need_dx=False)
    assert torch.equal(dw, (dy[-1].float().unsqueeze(1) * x[-1].float()).to(dtype))
    column = torch.zeros_like(dy)
    column[:, -1] = dy[:, -1]
    dx, _, _ = kda.linear_bwd(column, x, w, need_dweight=False)
    assert torch.equal(dx, (dy[:, -1:].float() * w[-1].float()).to(dtype))
