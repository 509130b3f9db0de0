"""Barrier ordering of the attention kernels over keys in two pieces in their generated code (CPU only), by
the walk of test_barrier_order_block: every barrier is reached with the wave's own LDS reads complete."""
import os
import shutil
import subprocess

import pytest

from tests.test_barrier_order_block import barriers, bodies, build


def test_every_barrier_follows_the_waves_lds_reads(tmp_path):
    if not os.path.exists(build.HIPCC) and not shutil.which("hipcc"):
        pytest.skip("hipcc not available")
    assert "attention_spans.hip" in build.HIP_SOURCES
    out = tmp_path / "spans.s"
    cmd = [build.HIPCC] + build.HIP_FLAGS + ["-S", "--cuda-device-only", os.path.join(build.CSRC, "attention_spans.hip"), "-o",
                                             str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    least = {"attention_rows": 6, "attention_keys": 2}
    seen = set()
    for name, body in bodies(out.read_text()):
        total, bad = barriers(body)
        assert bad == 0, f"{name}: {bad} of {total} barriers reached with LDS reads in flight"
        for kernel, n in least.items():
            if kernel in name:
                seen.add(kernel)
                assert total >= n, f"{name}: only {total} barriers found"
    assert seen == set(least)
