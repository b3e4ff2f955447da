"""Tensors of a device that is not the current one are refused before any launch: their
addresses and their stream's handle mean nothing on the device that would run the kernels."""
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_42_gb300 as kda
from gated_delta_rule_42_gb300 import cp, dense, inputs, ops


def current(monkeypatch, index):
    for module in (ops, dense):
        monkeypatch.setattr(module, "_current_device", lambda: index)


@pytest.mark.parametrize("stream", [ops._stream, dense._stream])
def test_another_device_is_refused(stream, monkeypatch):
    current(monkeypatch, 0)
    with pytest.raises(ValueError, match="on cuda:1, but the current device is cuda:0"):
        stream(torch.device("cuda", 1))


@pytest.mark.gpu
def test_every_call_refuses(monkeypatch):
    from gated_delta_rule_42_gb300 import build
    build.build()
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(6, 8, device="cuda")
    y, mean, rstd = kda.layer_norm_fwd(x)
    d = inputs.make_inputs(B=1, T=64, H=1, HV=1, K=64, V=64, dtype=torch.float32, seed=1, name="device").to("cuda")
    o, h, kctx = kda.chunk_kda_fwd_ctx(d.q, d.k, d.v, d.g, d.beta, output_final_state=True)
    m = torch.ones(1, 1, 64, 64, device="cuda")
    calls = [lambda: kda.layer_norm_fwd(x), lambda: kda.layer_norm_bwd(x, x, mean, rstd), lambda: kda.layer_norm(x),
             lambda: kda.linear_fwd(x, w), lambda: kda.linear_bwd(torch.ones(4, 6, device="cuda"), x, w),
             lambda: kda.linear(x, w), lambda: kda.clip_grad_norm([x], 1.0),
             lambda: kda.chunk_kda_fwd(d.q, d.k, d.v, d.g, d.beta), lambda: kda.chunk_kda(d.q, d.k, d.v, d.g, d.beta),
             lambda: kda.chunk_kda_fwd_ctx(d.q, d.k, d.v, d.g, d.beta),
             lambda: kda.chunk_kda_bwd(d.q, d.k, d.v, d.g, d.beta, None, None, o, None),
             lambda: kda.chunk_kda_bwd_ctx(d.q, d.k, d.v, d.g, d.beta, None, None, kctx, o, None),
             lambda: kda.chunk_kda_bwd_state(d.q, d.k, d.v, d.g, d.beta, None, None, o, None),
             lambda: kda.recurrent_kda(d.q, d.k, d.v, d.g, d.beta), lambda: cp.compose(m, m, None)]
    torch.cuda.synchronize()
    current(monkeypatch, 1)  # as if another GPU were the current one
    for call in calls:
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()
    monkeypatch.undo()
    assert (x == 1).all() and all(c() is not None for c in calls[:7])


def test_the_package_loads_with_a_torch_without_cuda():
    code = ("import torch; del torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream; "
            "import gated_delta_rule_42_gb300.cp")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
