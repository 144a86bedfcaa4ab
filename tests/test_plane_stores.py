"""Scales of MX planes leave a 128x128 tile in stores that lie on their own size (on the host)."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT


@pytest.fixture(scope="module")
def width(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("probe") / "plane_stores_probe.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "fp8_fp4_tensor_amd", "csrc"), os.path.join(ROOT, "tests", "plane_stores_probe.cpp"),
                    "-o", out], check=True)
    f = ctypes.CDLL(out).scale_store_bytes
    return lambda per, first, codes: f(ctypes.c_int64(per), ctypes.c_int64(first), codes)


@pytest.mark.parametrize("halves", [1, 2])
def test_stores_lie_on_their_size(width, halves):
    """Every tile of a row of scales, of one tensor or of two halves side by side (the gradient of the gated activation,
    whose second half starts at code 2 of a word for 192 or 4160 columns)."""
    for blocks in list(range(1, 70)) + [129, 130, 258, 448]:
        per = halves * blocks
        for half in range(halves):
            for tile in range(0, blocks, 4):
                first, codes = half * blocks + tile, min(4, blocks - tile)
                w = width(per, first, codes)
                assert w in (1, 2, 4) and codes % w == 0
                for row in range(4):
                    assert (row * per + first) % w == 0, (blocks, half, tile, row)
                if codes == 4 and per % 4 == 0 and first % 4 == 0:
                    assert w == 4
