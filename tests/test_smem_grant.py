"""Two host threads whose calls need different sizes of shared memory of one kernel: a
size once granted stays granted."""
import os
import subprocess
import sys

import pytest

from gated_delta_rule_42_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def run_host(source, tmp_path):
    """Compiles a host program of this folder against the library's sources and runs it."""
    exe = str(tmp_path / "host")
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-Xcicc", "-O0", "-Xptxas",
                    "-O0", "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(HERE, source), "-o", exe], check=True, capture_output=True, text=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=60)


def test_a_smaller_size_does_not_take_a_larger_one_back(tmp_path):
    r = run_host("host_smem_grant.cu", tmp_path)
    assert r.returncode == 0, r.stdout + r.stderr


THREADS = """
import threading, torch
import gated_delta_rule_42_gb300 as kda
errors, gate = [], threading.Barrier(2)
def work(width):
    x = torch.randn(40, width, device="cuda", dtype=torch.bfloat16)
    w, b = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
    _, mean, rstd = kda.layer_norm_fwd(x, w, b)
    gate.wait()
    try:
        for _ in range(50):
            kda.layer_norm_bwd(x, x, mean, rstd, w, b)
    except Exception as e:
        errors.append(f"{width}: {e}")
threads = [threading.Thread(target=work, args=(n,)) for n in (4096, 8192)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not errors, errors
"""


@pytest.mark.gpu
def test_two_threads_in_a_fresh_process():
    build.build()
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", THREADS], capture_output=True, text=True, timeout=300,
                           cwd=os.path.dirname(HERE))
        assert r.returncode == 0, r.stdout + r.stderr
