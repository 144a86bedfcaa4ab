"""fq_gemm where its ranges end."""
import pytest
import torch

from fp8_fp4_tensor_amd import fq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,bf16", [(1 << 20, (1 << 14) + 256, True), (3, (1 << 32) + 128, False)])
def test_empty_depth_of_a_large_output(m, n, bf16):
    """k = 0 and m * n beyond 2^34 (2^32 threads of four values): zeros everywhere, or C kept with accumulate."""
    out = torch.full((m * n + 1024,), 3.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    view = out[:m * n].view(m, n)
    none, s = torch.empty((0,), dtype=torch.uint8, device="cuda"), torch.empty((0,), device="cuda")
    p = fq.Plane(none, s)
    if not bf16:
        fq.fq_gemm(fq.gemm_desc(m, n, 0, out_dtype=fq.FQ_IN_F32, accumulate=True), p, p, view)
        torch.cuda.synchronize()
        assert bool((out == 3.0).all())
    fq.fq_gemm(fq.gemm_desc(m, n, 0, out_dtype=fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32), p, p, view)
    torch.cuda.synchronize()
    assert not bool(view.any()) and bool((out[m * n:] == 3.0).all())
