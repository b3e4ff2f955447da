"""The tensor-core product when a wait of its pipeline gives up: the limit is made so
short that waits run out, and the kernel has to end what it has in flight, say so in
its word and leave the GPU as it was for the next call.  Nothing here faults or hangs:
every wait stays bounded."""
import ctypes

import pytest
import torch

import gated_delta_rule_42_gb300 as kda
from gated_delta_rule_42_gb300 import _lib, build, dense

A = 0x100000  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_refusals(lib):
    def call(rows=300, dtype=_lib.KDA_BF16, y=A, ws=A, wb=1 << 40, err=A, polls=0):
        s = _lib.KdaLinear(rows, 64, 32, dtype, 0, A, A, None, None)
        return lib.kda_debug_linear_waits(s, y, ws, wb, err, polls, None)
    assert call(rows=-1) == _lib.KDA_ERR_INVALID_ARG
    assert call(rows=8) == _lib.KDA_ERR_UNSUPPORTED and call(dtype=_lib.KDA_F32) == _lib.KDA_ERR_UNSUPPORTED
    assert call(rows=0) == _lib.KDA_ERR_UNSUPPORTED
    for kw in (dict(y=None), dict(err=None), dict(err=A + 2), dict(y=A + 1), dict(polls=-1), dict(polls=(1 << 24) + 1)):
        assert call(**kw) == _lib.KDA_ERR_INVALID_ARG
    s = _lib.KdaLinear(300, 64, 4096, _lib.KDA_BF16, 0, A, A, None, None)
    assert lib.kda_linear_fwd_workspace_size(s) > 0  # its k axis is split
    assert lib.kda_debug_linear_waits(s, A, None, 0, A, 0, None) == _lib.KDA_ERR_WORKSPACE


# one stage; more stages than the ring holds; split k axes; a band of tiles a pair works through in turn; odd sizes
SHAPES = [(64, 64, 64), (256, 256, 320), (256, 256, 448), (40, 4096, 4096), (300, 520, 1003), (4096, 2048, 64),
          (20000, 1024, 256), (5000, 4096, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("polls", [0, 1, 2, 5, 20, 100, 1000])
def test_waits_that_give_up(lib, polls):
    torch.manual_seed(polls)
    for rows, outs, ins in SHAPES:
        x = torch.randn(rows, ins, device="cuda", dtype=torch.bfloat16)
        w = torch.randn(outs, ins, device="cuda", dtype=torch.bfloat16)
        want, _ = kda.linear_fwd(x, w)
        s = dense._linear_struct(x, w, None, None, None)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        for _ in range(5):
            y = torch.empty_like(want)
            ws, wp, wb = dense._workspace(lib.kda_linear_fwd_workspace_size(s), x.device)
            _lib.check(lib, lib.kda_debug_linear_waits(s, y.data_ptr(), wp, wb, err.data_ptr(), polls,
                                                       dense._stream(x.device)))
            again, _ = kda.linear_fwd(x, w)  # right behind it: tensor memory is free and nothing is written late
            assert torch.equal(again, want)
            if int(err) == 0:  # every wait was long enough
                assert torch.equal(y, want)
        assert polls > 0 or int(err) == 1  # a wait of no polls always gives up
    assert int(kda.linear_status()) == 0  # its own word


@pytest.mark.gpu
def test_the_usual_limit(lib):
    x, w = (torch.randn(500, 500, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    want, _ = kda.linear_fwd(x, w)
    s = dense._linear_struct(x, w, None, None, None)
    y, err = torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws, wp, wb = dense._workspace(lib.kda_linear_fwd_workspace_size(s), x.device)
    _lib.check(lib, lib.kda_debug_linear_waits(ctypes.byref(s), y.data_ptr(), wp, wb, err.data_ptr(), 1 << 24,
                                               dense._stream(x.device)))
    assert torch.equal(y, want) and int(err) == 0
