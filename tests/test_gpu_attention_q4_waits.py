"""A wait that is given up while the 4-bit kernel's copies of parts of head vectors are on their way: they are waited for."""
import os
import subprocess

import pytest

from disaggregated_paged_kv_gb300 import build as kbuild

pytestmark = pytest.mark.gpu


def test_copies_in_flight_are_waited_for(tmp_path):
    src = os.path.join(kbuild.ROOT, "tests", "c", "attn_q4_waits.cu")
    exe = str(tmp_path / "attn_q4_waits")
    subprocess.run([kbuild.nvcc(), *kbuild.ARCH, "-O2", "-std=c++17", "-I", kbuild.INCLUDE, "-I", kbuild.CSRC, src,
                    "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert got.returncode == 0 and got.stdout == "ok\n", got.stdout
