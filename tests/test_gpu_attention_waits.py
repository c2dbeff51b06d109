"""The attention kernels' bounded waits, in a program of their own: a wait that nobody ends is given up with
KVX_ERR_TIMEOUT, in seconds at most, and copies in flight are waited for."""
import os
import subprocess

import pytest

from disaggregated_paged_kv_gb300 import build as kbuild

pytestmark = pytest.mark.gpu


def test_given_up_waits_and_copies_in_flight(tmp_path):
    src = os.path.join(kbuild.ROOT, "tests", "c", "attn_waits.cu")
    exe = str(tmp_path / "attn_waits")
    subprocess.run([kbuild.nvcc(), *kbuild.ARCH, "-O2", "-std=c++17", "-I", kbuild.INCLUDE, "-I", kbuild.CSRC, src,
                    "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert got.returncode == 0, got.stdout
    seconds, verdict = got.stdout.split()
    assert verdict == "ok"
    assert 0.05 < float(seconds) < 20
