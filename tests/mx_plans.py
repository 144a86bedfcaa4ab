"""Shapes that take each kernel of the products of microscaled operands, and
the launch rule itself, compiled for the host from csrc/plan.hpp."""
import ctypes
import functools
import os
import subprocess
import tempfile

from conftest import ROOT

E4M3, E5M2, E2M1 = 0, 1, 2
# What the launch rule tells apart: formats of A and of B, and whether results are bf16.
EIGHT = [(a, b) for a in (E4M3, E5M2) for b in (E4M3, E5M2)]
MIXED = [(E4M3, E2M1), (E2M1, E4M3), (E5M2, E2M1), (E2M1, E5M2)]
KINDS = {"8": (EIGHT, True), "4": ([(E2M1, E2M1)], True), "4-f32": ([(E2M1, E2M1)], False), "mixed": (MIXED, True),
         "widened": (EIGHT + MIXED, False)}

# kind, tile (None: the kernel for few rows), shares of k, rows on whole rounds of 256x256 tiles first, scales laid
# out first, (m, n, k). Between them every kernel of the product, with scales as planes have them and laid out.
T256, T128, T64, T6464 = (256, 256), (128, 256), (64, 128), (64, 64)
PLANS = []
for _k in KINDS:
    PLANS += [(_k, None, False, False, False, (5, 131, 416)), (_k, None, False, False, False, (16, 384, 4128)),
              (_k, T128, False, False, False, (16726, 130, 256)), (_k, T128, False, False, True, (16420, 130, 96)),
              (_k, T6464, False, False, False, (17, 1, 128)), (_k, T6464, False, False, True, (33, 66, 32))]
for _k in ("8", "4", "4-f32", "mixed"):
    PLANS += [(_k, T256, False, False, False, (16428, 267, 128)), (_k, T256, False, False, True, (16533, 257, 64))]
for _k in ("4", "4-f32"):
    PLANS += [(_k, T256, True, False, False, (8631, 67, 8704)), (_k, T256, True, False, True, (8223, 75, 8544)),
              (_k, T128, True, False, False, (73, 2782, 12032)), (_k, T128, True, False, True, (69, 2782, 11680)),
              (_k, T64, False, False, False, (8519, 66, 128)), (_k, T64, False, False, True, (8196, 65, 64)),
              (_k, T64, True, False, False, (65, 696, 9216)), (_k, T64, True, False, True, (687, 68, 8416)),
              (_k, T6464, True, False, False, (17, 1, 2432)), (_k, T6464, True, False, True, (17, 1, 2336)),
              (_k, T64, True, True, False, (1540, 10364, 3456)),
              (_k, T6464, True, True, False, (8256, 1918, 2688)), (_k, T6464, True, True, True, (8254, 1826, 3520))]
for _k in ("8", "mixed"):
    PLANS += [(_k, T128, True, False, False, (71, 2802, 7808)), (_k, T128, True, False, True, (65, 2769, 7456)),
              (_k, T64, True, False, False, (19, 1043, 4096)), (_k, T64, True, False, True, (19, 1096, 4064)),
              (_k, T6464, True, False, False, (18, 1, 1536)), (_k, T6464, True, False, True, (17, 1, 1440))]
PLANS += [
    ("4", T128, False, True, False, (1013, 18104, 1152)), ("4", T128, False, True, True, (991, 16478, 1248)),
    ("4", T64, False, True, False, (11704, 1308, 640)), ("4", T64, False, True, True, (18108, 796, 544)),
    ("4", T6464, False, True, False, (17238, 775, 384)), ("4", T6464, False, True, True, (16762, 775, 352)),
    ("4-f32", T128, False, True, False, (967, 16433, 1792)), ("4-f32", T128, False, True, True, (966, 16769, 1376)),
    ("4-f32", T64, False, True, False, (17556, 860, 896)), ("4-f32", T64, False, True, True, (17817, 797, 928)),
    ("4-f32", T6464, False, True, False, (17302, 775, 1152)), ("4-f32", T6464, False, True, True, (16607, 801, 832)),
    ("8", T256, True, False, False, (131, 2723, 12288)), ("8", T256, True, False, True, (8489, 68, 5568)),
    ("8", T256, True, True, True, (1424, 12025, 3360)), ("8", T128, False, True, False, (1312, 13099, 768)),
    ("8", T128, False, True, True, (1290, 13101, 672)), ("8", T128, True, True, False, (837, 19709, 2304)),
    ("8", T128, True, True, True, (2000, 8397, 2528)), ("8", T64, False, False, False, (1, 17600, 512)),
    ("8", T64, False, False, True, (1, 16675, 544)), ("8", T64, False, True, False, (17601, 827, 384)),
    ("8", T64, False, True, True, (17760, 780, 448)), ("8", T64, True, True, False, (5430, 3000, 2816)),
    ("8", T64, True, True, True, (770, 19638, 1984)), ("8", T6464, False, True, False, (17238, 775, 384)),
    ("8", T6464, False, True, True, (16762, 775, 352)), ("8", T6464, True, True, False, (13092, 1043, 1920)),
    ("8", T6464, True, True, True, (16465, 792, 2208)),
    ("mixed", T256, True, False, False, (9215, 66, 6528)), ("mixed", T256, True, False, True, (8193, 70, 6432)),
    ("mixed", T128, False, True, False, (18633, 1804, 512)), ("mixed", T128, False, True, True, (19168, 1825, 416)),
    ("mixed", T64, False, False, False, (1, 17596, 1024)), ("mixed", T64, False, False, True, (17, 16590, 32)),
    ("mixed", T64, False, True, False, (15072, 2065, 384)), ("mixed", T64, False, True, True, (11152, 2861, 288)),
    ("mixed", T6464, False, True, False, (18761, 1547, 512)), ("mixed", T6464, False, True, True, (18893, 1609, 288)),
    ("mixed", T6464, True, True, True, (13079, 2557, 1632)),
    ("widened", T256, False, False, False, (16440, 387, 128)), ("widened", T256, False, False, True, (16776, 387, 32)),
    ("widened", T256, True, False, False, (5448, 131, 10880)), ("widened", T256, True, False, True, (5478, 131, 11200)),
    ("widened", T128, True, False, False, (67, 2818, 5760)), ("widened", T128, True, False, True, (66, 2730, 5600)),
    ("widened", T64, False, False, False, (8519, 66, 128)), ("widened", T64, False, False, True, (8196, 65, 64)),
    ("widened", T64, False, True, False, (19822, 1054, 1152)), ("widened", T64, False, True, True, (19671, 1069, 864)),
    ("widened", T64, True, False, False, (72, 563, 4096)), ("widened", T64, True, False, True, (563, 65, 4032)),
    ("widened", T6464, True, False, False, (17, 1, 1024)), ("widened", T6464, True, False, True, (17, 1, 928)),
]
# Several 256x256 tiles for each CU, which a workgroup takes in turn (but where a tile is one step): whole steps, a last
# step that is short, rows and columns of tiles that are mostly past the end; kind, scales laid out first, (m, n, k).
WALKS = [("8", True, (5000, 12600, 1568)), ("8", False, (8192, 8192, 256)), ("4", True, (9000, 9000, 1056)),
         ("4", False, (8192, 8192, 256)), ("4-f32", True, (7169, 16400, 544)), ("mixed", True, (8193, 8161, 1056)),
         ("mixed", False, (8192, 8192, 128))]


@functools.lru_cache(None)
def _lib():
    out = os.path.join(tempfile.mkdtemp(prefix="mx_plan_probe"), "mx_plan_probe.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "fp8_fp4_tensor_amd", "csrc"), os.path.join(ROOT, "tests", "mx_plan_probe.cpp"),
                    "-o", out], check=True)
    return ctypes.CDLL(out)


def plan(m, n, k, fa, fb, bf16):
    """(tile or None, shares of k, leading rows on 256x256 tiles, whether scales are laid out first)."""
    out, sizes = (ctypes.c_int64 * 4)(), (ctypes.c_int64 * 8)()
    _lib().mx_plan(*[ctypes.c_int64(int(x)) for x in (m, n, k, fa == E2M1, fb == E2M1, bf16)], out)
    _lib().mx_tile_sizes(sizes)
    kind, splits, main, arranged = out
    return None if kind < 0 else (sizes[2 * kind], sizes[2 * kind + 1]), splits, main, bool(arranged)
