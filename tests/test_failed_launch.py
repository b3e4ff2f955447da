"""A launch that fails ends its call: what would have read its results is not launched."""
from tests.test_smem_grant import run_host


def test_nothing_follows_a_failed_launch(tmp_path):
    r = run_host("host_failed_launch.cu", tmp_path)
    assert r.returncode == 0, r.stdout + r.stderr
