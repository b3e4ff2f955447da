"""The linear layer's status word through the Python layer."""
import ctypes

import pytest
import torch

import gated_delta_rule_42_gb300 as kda
from gated_delta_rule_42_gb300 import _lib, dense

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_42_gb300 import build
    build.build()


def test_status_is_read_in_stream_order():
    x, w = torch.ones(300, 64, device="cuda", dtype=torch.bfloat16), torch.ones(64, 64, device="cuda", dtype=torch.bfloat16)
    kda.linear_fwd(x, w)
    before = kda.linear_status()
    assert before.dtype == torch.int32 and before.shape == () and before.is_cuda and int(before) == 0
    lib, p = _lib.load(), ctypes.c_void_p()
    _lib.check(lib, lib.kda_linear_status(ctypes.byref(p)))
    word = torch.as_tensor(dense._DeviceWord(p.value), device="cuda")
    try:
        word.fill_(1)
        during = kda.linear_status("cuda:0")
    finally:
        word.fill_(0)
    after = kda.linear_status("cuda")
    assert (int(before), int(during), int(after)) == (0, 1, 0)


def test_status_in_a_graph():
    kda.linear_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        status = kda.linear_status()
    status.fill_(7)
    graph.replay()
    assert int(status) == 0
