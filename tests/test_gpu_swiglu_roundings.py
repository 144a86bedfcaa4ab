"""fq_swiglu and its gradient against bounds that count each of their roundings, far
out on both tails of the gate."""
import numpy as np
import pytest
import torch

import block_util as B
from fp8_fp4_tensor_amd import fq
from test_gpu_norm import F32, d64, planes_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
# e = exp(-gate): one unit of the hardware's exponential and half of the fma that takes the exponent's error back, 1.5.
# What that leaves: the second order of the exponent's rounding, (87 log2(e) 2^-24)^2 / 2, and its constant's error in two
# fp32 terms, 87 * 2^-49: below 0.01 units each.
# s = 1 / (1 + e): e's share of 1 + e at most, half a unit of the sum and half of the refined reciprocal: 2.5.
# 1 - s: e s for positive gates, 1.5 + 2.5 + 0.5 = 4.5; less for the others, see the test of the cancelling slope. Each product
# adds half. Products of these errors stay below 0.1 units in all.
S, REST = 2.5, 4.5


def tiny(*factors):
    """Values below 2^-126 in magnitude may count as zero on the way."""
    return 2.0 ** -125 * (1 + sum(np.abs(f) for f in factors))


def gates(n, seed):
    """(gate, up, dy): gates spread evenly over both tails, and normal ones."""
    rng = np.random.default_rng(seed)
    g = np.concatenate((rng.uniform(-87, 87, n // 2), 2 * rng.standard_normal(n - n // 2)))
    return [v.astype(np.float32) for v in (g, rng.standard_normal(n), rng.standard_normal(n))]


def run(gate, up, dy, rows, planes):
    """(y, dgate, dup) in fp32, by the kernel for rows or the one for tiles (with colwise planes)."""
    cols = gate.size // rows
    x = torch.from_numpy(np.concatenate((gate.reshape(rows, cols), up.reshape(rows, cols)), 1)).cuda()
    y, dx = torch.empty((rows, cols), device="cuda"), torch.empty((rows, 2 * cols), device="cuda")
    d = fq.swiglu_desc(rows, cols, F32, F32)
    p, q = (planes_of("mx-e4m3", rows, c) if planes else None for c in (cols, 2 * cols))
    fq.fq_swiglu(d, x, y, p)
    fq.fq_swiglu_backward(d, x, torch.from_numpy(dy.reshape(rows, cols)).cuda(), dx, q)
    torch.cuda.synchronize()
    return [d64(t).reshape(-1) for t in (y, dx[:, :cols], dx[:, cols:])]


@pytest.mark.parametrize("planes", [False, True], ids=["rows", "tiles"])
def test_activation_counts_its_roundings(planes):
    gate, up, dy = gates(1 << 20, 11)
    y, dgate, dup = run(gate, up, dy, 256, planes)
    g, u, d = (v.astype(np.float64) for v in (gate, up, dy))
    s, rest = B.sigmoid(g), B.sigmoid(-g)
    slope, t = 1 + g * rest, tiny(g * u, d * u, d * u * g, d * g)
    for name, got, want, units in (("y", y, g * s * u, (S + 1.0 + 0.1) * np.abs(g * s * u)),
                                   ("dup", dup, d * s * g, (S + 1.0 + 0.1) * np.abs(d * s * g)),
                                   ("dgate", dgate, d * u * s * slope, np.abs(d * u * s) * (
                                       (S + 1.5 + 0.1) * np.abs(slope) + REST * np.abs(g * rest) + 0.5 * np.abs(slope)))):
        err, bound = np.abs(got - want), U * units + t
        assert np.all(err <= bound), (name, (err / bound).max(), g[(err / bound).argmax()])


@pytest.mark.parametrize("planes", [False, True], ids=["rows", "tiles"])
def test_slope_where_it_cancels(planes):
    """1 + gate (1 - s) is zero at a gate of -1.2785. There 1 - s is a difference: it is off by s's own error, of e's 1.5
    units the share 1 - s and the sum's and the reciprocal's halves, and by half a unit of [1/2, 1)."""
    rng = np.random.default_rng(5)
    n = 1 << 20
    gate = rng.uniform(-1.4, -1.15, n).astype(np.float32)
    one = np.ones(n, np.float32)
    _, dgate, _ = run(gate, one, one, 256, planes)
    g = gate.astype(np.float64)
    s, rest = B.sigmoid(g), B.sigmoid(-g)
    slope = 1 + g * rest
    off = s * (1.5 * rest + 1.0) + 0.25
    bound = U * s * (np.abs(g) * off + (S + 1.5 + 0.1) * np.abs(slope)) * 1.01
    err = np.abs(dgate - s * slope)
    assert np.all(err <= bound), ((err / bound).max(), g[(err / bound).argmax()])


def test_sigmoid_in_the_mean_square():
    """s is off by 5e-8: y = gate s (up = 1) has one rounding more, uniform within half a unit in the last place, which is
    2^-24 / sqrt(3) of the value at most."""
    for scale in (1.0, 4.0, 16.0):
        g = (scale * np.random.default_rng(3).standard_normal(1 << 20)).astype(np.float32)
        g = g[np.abs(g) < 80]
        g = g[:g.size // 2048 * 2048]
        one = np.ones_like(g)
        y, _, dup = run(g, one, one, 256, False)
        want = g.astype(np.float64) * B.sigmoid(g.astype(np.float64))
        for got in (y, dup):
            rms = np.sqrt(np.mean(((got - want) / np.where(want == 0, 1, want)) ** 2))
            assert rms <= np.hypot(5e-8, 2.0 ** -24 / np.sqrt(3)), (scale, rms)
