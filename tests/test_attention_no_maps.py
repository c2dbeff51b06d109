"""Shared attention over 4-bit pools where the driver makes no tensor maps: the call takes copies that need none.  (On the
host alone: launches are stand-ins.)"""
import glob
import os
import subprocess

import pytest

from disaggregated_paged_kv_gb300 import build as kbuild
from disaggregated_paged_kv_gb300 import kvx

BOXES, TOKENS, PARTS = 0, 1, 2


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    if not os.path.exists(kvx.LIB_PATH) or len(glob.glob(os.path.join(kbuild.OUT_DIR, "*.o"))) < len(kbuild.SOURCES):
        kbuild.build()
    objs = [os.path.join(kbuild.OUT_DIR, os.path.splitext(s)[0] + ".o") for s in kbuild.SOURCES]
    out = str(tmp_path_factory.mktemp("maps") / "attn_no_maps")
    lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(kbuild.nvcc()))), "lib64")
    subprocess.run([kbuild.nvcc(), *kbuild.ARCH, "-std=c++17", "-cudart", "shared", "-I", kbuild.INCLUDE, "-I", kbuild.CSRC,
                    os.path.join(kbuild.ROOT, "tests", "c", "attn_no_maps.cu"), *objs, "-o", out, "-Xlinker", "-rpath=" + lib],
                   check=True)
    return out


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_copies_without_maps(exe, mode):
    got = subprocess.run([exe, str(mode)], capture_output=True, text=True, timeout=60)
    assert got.returncode == 0, got.stdout + got.stderr
    lines = got.stdout.splitlines()
    assert len(lines) == 20
    for line in lines:
        what, result = line.split(": ")
        kind, D, H = what.split()[0], int(what.split()[1]), int(what.split()[2])
        status, launches, copies = (int(x) for x in result.split())
        # (rows of 40 bytes a head are no whole pieces of 16 where the heads are odd in number)
        odd = D == 64 and H % 2 == 1
        without = PARTS if kind == "hnd" or odd else TOKENS
        want = without if mode < 2 or (odd and H > 1 and kind == "nhd") else BOXES
        assert (status, launches, copies) == (0, 2, want), line
