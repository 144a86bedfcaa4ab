"""Planes of the gated activation's gradient whose halves meet inside a word of
scales."""
import pytest
import torch

from fp8_fp4_tensor_amd import fq
from test_gpu_norm import BF16, BOTH, F32, planes_of, same_planes
from test_gpu_swiglu import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["mx-e4m3", "mx-e5m2", "mx-e2m1"])
def test_gradient_whose_second_half_starts_inside_a_word_of_scales(orc, kind):
    """cols / 32 = 2, 6, 10, 130 and odd: the scales of dup's tiles start at any byte of a word."""
    for rows, cols in ((128, 64), (160, 192), (256, 320), (128, 4160), (96, 1056), (128, 224)):
        for x_dt in (BF16, F32):
            x, dy = inputs(rows, cols, x_dt, BF16, rows + cols)
            dx, p = torch.empty((rows, 2 * cols), device="cuda"), planes_of(kind, rows, 2 * cols, BOTH, 0x5A)
            fq.fq_swiglu_backward(fq.swiglu_desc(rows, cols, F32), x.float(), dy, dx)
            fq.fq_swiglu_backward(fq.swiglu_desc(rows, cols, x_dt), x, dy, None, p)
            torch.cuda.synchronize()
            same_planes(orc, dx, p, kind, BOTH, f"{kind} {rows}x{cols}")
