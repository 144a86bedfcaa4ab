"""Shapes that take each kernel of the operators on 8-bit data, and the launch
rules themselves, compiled for the host from csrc/plan.hpp."""
import ctypes
import functools
import os
import subprocess
import tempfile

from conftest import ROOT

# Products: tile, shares of k, rows of a scale of B, bf16, (m, n, k). Between them every kernel of k_gemm.hip.
GEMM = [
    ("few", False, 128, False, (9, 384, 640)), ("few", False, 128, True, (16, 4096, 256)),
    ("few", False, 1, False, (7, 131, 384)), ("few", False, 1, True, (12, 517, 1152)),
    ((256, 256), False, 128, False, (515, 19968, 128)), ((256, 256), False, 128, True, (386, 16512, 256)),
    ((256, 256), False, 1, False, (516, 19599, 256)), ((256, 256), False, 1, True, (16412, 385, 128)),
    ((256, 256), True, 128, False, (130, 8320, 5248)), ((256, 256), True, 128, True, (131, 5632, 3712)),
    ((256, 256), True, 1, False, (16493, 129, 1920)), ((256, 256), True, 1, True, (129, 2689, 7552)),
    ((128, 128), False, 128, False, (193, 12416, 128)), ((128, 128), False, 128, True, (65, 16512, 384)),
    ((128, 128), False, 1, False, (193, 12291, 256)), ((128, 128), False, 1, True, (16390, 65, 128)),
    ((128, 128), True, 128, False, (65, 3200, 2816)), ((128, 128), True, 128, True, (65, 1408, 4224)),
    ((128, 128), True, 1, False, (65, 2052, 4096)), ((128, 128), True, 1, True, (8196, 1, 1536)),
    ((64, 128), False, 128, False, (33, 16512, 128)), ((64, 128), False, 128, True, (33, 16512, 256)),
    ((64, 128), False, 1, False, (8234, 65, 128)), ((64, 128), False, 1, True, (8199, 65, 256)),
    ((64, 128), True, 128, False, (33, 2816, 1536)), ((64, 128), True, 128, True, (33, 1408, 3200)),
    ((64, 128), True, 1, False, (1373, 65, 1536)), ((64, 128), True, 1, True, (520, 65, 4096)),
    ((64, 64), False, 128, False, (33, 8320, 128)), ((64, 64), False, 128, True, (33, 8320, 256)),
    ((64, 64), False, 1, False, (8193, 1, 128)), ((64, 64), False, 1, True, (8193, 3, 256)),
    ((64, 64), True, 128, False, (33, 1408, 1536)), ((64, 64), True, 128, True, (33, 1408, 2048)),
    ((64, 64), True, 1, False, (1345, 1, 1536)), ((64, 64), True, 1, True, (1345, 5, 1536)),
    ((32, 64), False, 128, False, (17, 256, 128)), ((32, 64), False, 128, True, (31, 128, 640)),
    ((32, 64), False, 1, False, (17, 3, 128)), ((32, 64), False, 1, True, (30, 61, 384)),
    ((32, 64), True, 128, False, (1, 128, 7296)), ((32, 64), True, 128, True, (5, 256, 9216)),
    ((32, 64), True, 1, False, (1, 1, 7296)), ((32, 64), True, 1, True, (11, 67, 8192)),
]
# Whole rounds of 256x256 tiles, and the rows behind them: their tile, shares, rows of a scale of B, bf16, (m, n, k).
GEMM_REST = [
    ((256, 256), True, 128, False, (3742, 9856, 2688)), ((256, 256), True, 1, False, (3730, 9821, 2560)),
    ((256, 256), True, 128, True, (900, 16512, 2304)), ((256, 256), True, 1, True, (898, 16859, 2560)),
    ((128, 128), False, 1, False, (19602, 1793, 512)), ((128, 128), True, 128, True, (2637, 6272, 2048)),
    ((64, 128), True, 1, False, (5410, 9164, 1408)), ((64, 128), False, 128, True, (2210, 7296, 384)),
    ((64, 64), True, 1, True, (5945, 2730, 1920)), ((64, 64), False, 128, False, (3621, 13568, 384)),
    ((32, 64), True, 128, False, (13084, 3840, 1408)), ((32, 64), False, 1, True, (1025, 14469, 384)),
]


@functools.lru_cache(None)
def _lib():
    out = os.path.join(tempfile.mkdtemp(prefix="plan_probe"), "plan_probe.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "fp8_fp4_tensor_amd", "csrc"), os.path.join(ROOT, "tests", "plan_probe.cpp"),
                    "-o", out], check=True)
    return ctypes.CDLL(out)


def _call(name, count, *args):
    out = (ctypes.c_int64 * count)()
    getattr(_lib(), name)(*[ctypes.c_int64(a) for a in args], out)
    return list(out)


def gemm_plan(m, n, k, bf16):
    """(tile or "few", shares of k, leading rows on 256x256 tiles)."""
    kind, splits, main = _call("gemm_plan", 3, m, n, k, int(bf16))
    sizes = _call("tile_sizes", 10)
    return ("few" if kind < 0 else (sizes[2 * kind], sizes[2 * kind + 1])), splits, main


def attention_plan(heads, q_heads, dim, lens, counts, window=0, max_len=0, page=64):
    """(kernel, splits) as fq_attention plans the call of these sequences."""
    longest = max_len or -(-max(max(lens), 1) // page) * page
    window = 0 if window >= longest else window
    max_q = min(max(counts), sum(counts))
    rows, waves, splits, _, _ = _call("attention_plan", 5, len(lens), heads, q_heads, dim, max_q, longest, window)
    return ("many" if rows > 16 else f"few-{waves}"), splits
