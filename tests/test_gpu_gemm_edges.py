"""fq_gemm where its ranges end, and every kernel that it can take."""
import numpy as np
import pytest
import torch

import operator_plans as P
import operator_util as U
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


# ---------------------------------------------------------------- every kernel
def operands(m, n, k, b_rows, seed):
    """Finite codes of every magnitude and scales over 15 binades, on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def codes(r):
        c = torch.randint(0, 256, (r, k), generator=g, device="cuda", dtype=torch.uint8)
        return c.masked_fill_((c & 127) == 127, 0)

    rng = np.random.default_rng(seed)
    scales = [torch.from_numpy(U.random_scales(rng, (r, k // 128))).cuda() for r in (m, n if b_rows == 1 else n // 128)]
    return codes(m), scales[0], codes(n), scales[1]


def reference(a, sa, b, sb, b_rows):
    """operator_util.product on the GPU, in 64 bits."""
    table = torch.from_numpy(U.value_table(U.E4M3)).cuda()
    (m, k), n, nb = a.shape, b.shape[0], a.shape[1] // 128
    s = sb.double() if b_rows == 1 else sb.double().repeat_interleave(128, 0)
    va = (table[a.long()].view(m, nb, 128) * sa.double()[:, :, None]).view(m, k)
    vb = (table[b.long()].view(n, nb, 128) * s[:, :, None]).view(n, k)
    want = va @ vb.t()
    ma, mb = va.abs_(), vb.abs_()
    top = ma.view(m, nb, 128).amax(2) @ mb.view(n, nb, 128).amax(2).t().contiguous()
    return want, ma @ mb.t(), top


def check(got, want, s, top, k, bf16, what):
    err = (got.double() - want).abs_()
    norm = U.HALF_BF16 if bf16 else U.HALF_F32  # as product_norm_bound and product_bound, on the GPU
    sums = (128 + 2 + 2 * (k // 128 + 32)) * U.ULP32
    assert err.norm() <= norm * want.norm() + ((2.0 ** -12 if bf16 else 0.0) + sums) * s.norm() + 1e-37, what
    bound = sums * s
    if bf16:
        bound = bound + 128 * 2.0 ** -13 * top
    bound = bound + norm * (want.abs() + bound) + 1e-37
    assert bool((err <= bound).all()), f"{what}: {(err > bound).sum()} of {err.numel()}, worst {(err / bound).max():.3g}"


@pytest.mark.parametrize("tile,split,b_rows,bf16,shape", P.GEMM + P.GEMM_REST)
def test_every_kernel(tile, split, b_rows, bf16, shape):
    """Whole results, with guards around them; fp32 results once more, added to what is there."""
    m, n, k = shape
    a, sa, b, sb = operands(m, n, k, b_rows, m + n + k)
    want, s, top = reference(a, sa, b, sb, b_rows)
    pa, pb, pad = fq.Plane(a, sa), fq.Plane(b, sb), 1024
    buf = torch.full((m * n + 2 * pad,), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    out = buf[pad:-pad].view(m, n).fill_(float("nan"))
    d = fq.gemm_desc(m, n, k, b_rows, fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32)
    size = fq.fq_gemm_workspace(d)
    assert (size > 0) == split
    ws = torch.full((size + 2 * pad,), 0xFF, dtype=torch.uint8, device="cuda")
    fq.fq_gemm(d, pa, pb, out, ws[pad:pad + size])
    torch.cuda.synchronize()
    check(out, want, s, top, k, bf16, f"{tile} {shape}")
    if not bf16:
        start = torch.randn((m, n), device="cuda")
        out.copy_(start)
        fq.fq_gemm(fq.gemm_desc(m, n, k, b_rows, fq.FQ_IN_F32, accumulate=True), pa, pb, out, ws[pad:pad + size])
        torch.cuda.synchronize()
        total = want + start.double()
        err = (out.double() - total).abs_()
        sums = (128 + 2 + 2 * (k // 128 + 32)) * U.ULP32 * s
        bound = sums + U.HALF_F32 * (want.abs() + sums) + 2 * U.HALF_F32 * (total.abs() + s) + 1e-37
        assert bool((err <= bound).all()), f"{tile} {shape} accumulated: worst {(err / bound).max():.3g}"
    assert bool((buf[:pad] == 7.0).all()) and bool((buf[-pad:] == 7.0).all())
    assert bool((ws[:pad] == 0xFF).all()) and bool((ws[pad + size:] == 0xFF).all())
