"""The weight's gradient of fq_rmsnorm_backward against a bound that counts its
additions."""
import numpy as np
import pytest
import torch

from fp8_fp4_tensor_amd import fq
from test_gpu_norm import F32, d64

pytestmark = pytest.mark.gpu


def weight_gradient(h, rstd, dy):
    rows, cols = h.shape
    d = fq.rmsnorm_desc(rows, cols, h_dtype=F32, y_dtype=F32)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    fq.fq_rmsnorm_backward(d, h, rstd, torch.ones(cols, device="cuda"), dy, dx, dw, None, fq.alloc_rmsnorm_workspace(d))
    torch.cuda.synchronize()
    return d64(dw)


@pytest.mark.parametrize("cols", [512, 1032, 4104])
def test_rows_of_partial_sums_meet_as_a_tree(cols):
    """32 rows of partial sums, one of them 1 and the others just below half of its last place: one after the other they
    would all be lost, 29 halves. A term takes a rounding of its own and five additions."""
    for lead in (0, 1, 13, 31):
        terms = np.full((32, cols), 0.95 * 2.0 ** -24)
        terms[lead] = 1.0
        terms = terms.astype(np.float32)
        dw = weight_gradient(torch.ones((32, cols), device="cuda"), torch.ones(32, device="cuda"), torch.from_numpy(terms).cuda())
        want = terms.astype(np.float64).sum(0)
        assert np.all(np.abs(dw - want) <= (1 + 5 + 0.1) * 2.0 ** -24 * want), (lead, np.abs(dw - want).max() * 2 ** 24)


@pytest.mark.parametrize("rows,cols", [(1003, 7168), (100003, 1032), (131072, 520), (70000, 2056), (20000, 8200)])
def test_weight_gradient_of_many_rows(rows, cols):
    """A workgroup (512 at most, 256 at least where there are as many rows) adds its rows one after the other, a thread
    of the second kernel every 32nd row of partial sums (2048 of them at most), then five additions; the value z and its product
    with dy take one each."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    h, dy, rstd = rn(rows, cols) + 0.3, rn(rows, cols) + 0.5, torch.rand(rows, generator=g, device="cuda") + 0.5
    dw = weight_gradient(h, rstd, dy)
    want, mag = np.zeros(cols), np.zeros(cols)
    for r in range(0, rows, 8192):
        part = dy[r:r + 8192].double() * h[r:r + 8192].double() * rstd[r:r + 8192, None].double()
        want += d64(part.sum(0))
        mag += d64(part.abs().sum(0))
    groups = 512 if rows >= 2048 else 256
    chain = rows / groups + 1 + 2048 / 32 + 5 + 2
    assert np.all(np.abs(dw - want) <= chain * 2.0 ** -24 * mag), (np.abs(dw - want) / mag).max() * 2.0 ** 24
