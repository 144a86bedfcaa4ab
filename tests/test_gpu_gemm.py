"""fq_gemm on the GPU against the 64-bit product of the same codes and scales."""
import numpy as np
import pytest
import torch

import operator_util as U
from fp8_fp4_tensor_amd import fq
from fp8_fp4_tensor_amd import workloads as W
from gpu_util import dev

pytestmark = pytest.mark.gpu


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def operands(rng, m, n, k, b_rows, pow2=False):
    nb = k // 128
    return (U.random_codes(rng, (m, k)), U.random_scales(rng, (m, nb), pow2),
            U.random_codes(rng, (n, k)), U.random_scales(rng, (n if b_rows == 1 else n // 128, nb), pow2))


def run(a, sa, b, sb, b_rows, bf16, out=None, accumulate=False, stream=None):
    (m, k), n = a.shape, b.shape[0]
    d = fq.gemm_desc(m, n, k, b_rows, fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32, accumulate)
    if out is None:
        out = torch.full((m, n), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    fq.fq_gemm(d, fq.Plane(cuda(a), cuda(sa)), fq.Plane(cuda(b), cuda(sb)), out, fq.alloc_gemm_workspace(d), stream)
    torch.cuda.synchronize()
    return out


def check(got, ref, k, bf16, what):
    want, s, top = ref
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.linalg.norm(err) <= U.product_norm_bound(want, s, k, bf16), what
    bound = U.product_bound(want, s, top, k, bf16)
    assert np.all(err <= bound), (f"{what}: {(err > bound).sum()} of {err.size} out of bound, worst "
                                  f"{np.nanmax(err / bound):.3g}, nan {np.isnan(err).sum()}")


SHAPES = [  # m, n, k, rows of a scale of B
    (1, 128, 128, 128), (1, 128, 2048, 128), (3, 256, 1152, 128), (16, 384, 640, 128), (17, 128, 256, 128),
    (33, 512, 384, 128), (64, 256, 4096, 128), (65, 256, 512, 128), (127, 640, 256, 128), (128, 256, 1024, 128),
    (129, 384, 128, 128), (200, 1280, 640, 128), (255, 512, 768, 128), (300, 2048, 384, 128), (513, 768, 896, 128),
    (1, 1, 128, 1), (2, 3, 256, 1), (16, 17, 384, 1), (31, 129, 128, 1), (64, 130, 1024, 1), (100, 255, 512, 1),
    (129, 257, 256, 1), (260, 511, 640, 1), (384, 516, 1280, 1), (1024, 1030, 256, 1),
]


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("pow2", [False, True], ids=["fp32-scales", "pow2-scales"])
@pytest.mark.parametrize("m,n,k,b_rows", SHAPES)
def test_product(m, n, k, b_rows, pow2, bf16):
    rng = np.random.default_rng(m * 1000003 + n * 1009 + k + b_rows)
    a, sa, b, sb = operands(rng, m, n, k, b_rows, pow2)
    ref = U.product(a, sa, b, sb, b_rows)
    check(run(a, sa, b, sb, b_rows, bf16), ref, k, bf16, f"{m}x{n}x{k}")


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,b_rows", [
    (4000, 4096, 256, 128), (4100, 4001, 384, 1),            # the largest tiles, ragged, even and odd block counts
    (1500, 4096, 384, 128), (2000, 2050, 256, 1),
    (5000, 4096, 512, 128), (4500, 4097, 384, 1),            # more than a round of them: the rest on smaller tiles
    (16, 128, 7296, 128), (3, 515, 8192, 1), (30, 256, 9216, 128), (64, 384, 4224, 128), (100, 129, 6400, 1),
    (200, 512, 8192, 128), (300, 640, 4096, 128), (1, 8192, 384, 128), (16, 8191, 256, 1), (2, 4224, 1152, 128),
])
def test_every_tile_and_split(m, n, k, b_rows, bf16):
    """Shapes that take each tile size, whole and in shares of k."""
    rng = np.random.default_rng(m + n + k)
    a, sa, b, sb = operands(rng, m, n, k, b_rows)
    check(run(a, sa, b, sb, b_rows, bf16), U.product(a, sa, b, sb, b_rows), k, bf16, f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k,b_rows", [(5, 128, 256, 128), (70, 130, 384, 1), (300, 513, 256, 1), (9, 256, 4096, 128)])
def test_accumulate(m, n, k, b_rows):
    rng = np.random.default_rng(m)
    a, sa, b, sb = operands(rng, m, n, k, b_rows)
    want, s, top = U.product(a, sa, b, sb, b_rows)
    start = rng.standard_normal((m, n)).astype(np.float32)
    got = run(a, sa, b, sb, b_rows, False, out=cuda(start), accumulate=True)
    total = want + start
    bound = U.product_bound(want, s, top, k, False) + 2 * U.HALF_F32 * (np.abs(total) + s)
    assert np.all(np.abs(got.double().cpu().numpy() - total) <= bound)


def test_empty_products():
    a, sa = np.zeros((4, 0), np.uint8), np.zeros((4, 0), np.float32)
    b, sb = np.zeros((128, 0), np.uint8), np.zeros((1, 0), np.float32)
    assert torch.all(run(a, sa, b, sb, 128, True) == 0)
    keep = torch.full((4, 128), 3.0, device="cuda")
    assert torch.all(run(a, sa, b, sb, 128, False, out=keep, accumulate=True) == 3.0)
    rng = np.random.default_rng(1)
    a, sa, b, sb = operands(rng, 0, 128, 128, 128)
    assert run(a, sa, b, sb, 128, True).numel() == 0


def test_zero_and_extreme_codes():
    """All-zero blocks (the scales their recipes give), the largest codes, and zero codes of either sign."""
    m, n, k = 40, 256, 512
    a = np.full((m, k), 0x7E, np.uint8)
    b = np.full((n, k), 0xFE, np.uint8)
    a[:, 128:256] = 0x80
    b[128:, 256:384] = 0
    for pow2, zero in ((False, 1.0), (True, 2.0 ** -127)):
        sa, sb = np.full((m, 4), 0.5, np.float32), np.full((2, 4), 2.0, np.float32)
        sa[:, 1] = zero
        sb[1, 2] = zero
        check(run(a, sa, b, sb, 128, False), U.product(a, sa, b, sb, 128), k, False, f"pow2={pow2}")


@pytest.mark.parametrize("scale_mode", [fq.FQ_SCALE_DEFAULT, fq.FQ_SCALE_POW2], ids=["fp32", "pow2"])
def test_linear_layer_three_products(scale_mode):
    """Forward, input gradient and weight gradient from the library's own planes."""
    T, O, I = 256, 384, 512
    both = fq.FQ_ROWWISE | fq.FQ_COLWISE

    def quant(x, block):
        d = fq.desc(fq.FQ_BLOCK_FP32, fq.FQ_IN_BF16, fq.FQ_E4M3, *x.shape, block, both, scale_mode=scale_mode)
        q = fq.alloc_quantized(d)
        fq.fq_quantize(d, dev(x), q)
        torch.cuda.synchronize()
        return q

    X, Wt, G = W.normal((T, I), 1.0, 1), W.normal((O, I), 0.02, 2), W.normal((T, O), 1e-3, 3)
    qx, qw, qg = quant(X, (1, 128)), quant(Wt, (128, 128)), quant(G, (1, 128))

    def one(pa, pb, b_rows, bf16, what):
        m, n, k = pa.data.shape[0], pb.data.shape[0], pa.data.shape[1]
        d = fq.gemm_desc(m, n, k, b_rows, fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32)
        out = torch.empty((m, n), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        fq.fq_gemm(d, pa, pb, out, fq.alloc_gemm_workspace(d))
        torch.cuda.synchronize()
        h = lambda t, *shape: t.cpu().numpy().reshape(shape)
        ref = U.product(h(pa.data, m, k), h(pa.scale, m, k // 128), h(pb.data, n, k),
                            h(pb.scale, n if b_rows == 1 else n // 128, k // 128), b_rows)
        check(out, ref, k, bf16, what)
        return out

    row, col = fq.Plane.rowwise, fq.Plane.colwise
    y = one(row(qx), row(qw), 128, True, "forward")
    dx = one(row(qg), col(qw), 128, True, "input gradient")
    dw = one(col(qg), col(qx), 1, False, "weight gradient")
    # against the unquantized formula: a quantized value is within half a step of the block's amax range
    f = lambda x: W.bf16_bits_to_f32(x).astype(np.float64)
    for got, full in ((y, f(X) @ f(Wt).T), (dx, f(G) @ f(Wt)), (dw, f(G).T @ f(X))):
        # each factor is off by at most 2^-4 of itself or half a subnormal step (2^-10 of its scale): mean-square well under 2^-3
        assert np.linalg.norm(got.double().cpu().numpy() - full) <= 2.0 ** -3 * np.linalg.norm(full)


def test_gradients_against_differences():
    """L = <G, X W^T> is linear in X and in W: L(X') - L(X) = <dX, X' - X>, and the same for W."""
    rng = np.random.default_rng(5)
    T, O, I = 128, 256, 384
    x0, x1 = U.random_codes(rng, (T, I)), U.random_codes(rng, (T, I))
    w0, w1 = U.random_codes(rng, (O, I)), U.random_codes(rng, (O, I))
    g = U.random_codes(rng, (T, O))
    one = lambda r, c: np.ones((r, c // 128), np.float32)
    tile = lambda r, c: np.ones((r // 128, c // 128), np.float32)
    val = U.decode
    y = lambda x, w: run(x, one(T, I), w, tile(O, I), 128, False).double().cpu().numpy()
    dx = run(g, one(T, O), np.ascontiguousarray(w0.T), tile(I, O), 128, False).double().cpu().numpy()
    dw = run(np.ascontiguousarray(g.T), one(O, T), np.ascontiguousarray(x0.T), one(I, T), 1, False).double().cpu().numpy()
    mag = (np.abs(val(g)) * (np.abs(val(x0)) + np.abs(val(x1))) .dot(np.abs(val(w0)).T + np.abs(val(w1)).T)).sum()
    tol = 4 * 512 * U.ULP32 * mag
    base = (val(g) * y(x0, w0)).sum()
    assert abs((val(g) * y(x1, w0)).sum() - base - (dx * (val(x1) - val(x0))).sum()) <= tol
    assert abs((val(g) * y(x0, w1)).sum() - base - (dw * (val(w1) - val(w0))).sum()) <= tol


def test_same_bits_every_run_and_on_a_side_stream():
    rng = np.random.default_rng(7)
    for m, n, k, b_rows in ((7, 256, 4096, 128), (200, 512, 2048, 128), (300, 515, 1024, 1)):
        a, sa, b, sb = operands(rng, m, n, k, b_rows)
        first = run(a, sa, b, sb, b_rows, False)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        again = run(a, sa, b, sb, b_rows, False, stream=s)
        assert torch.equal(first, again)


def test_writes_only_its_output():
    """Guard rows before and behind the output stay as they were (ragged m and n)."""
    rng = np.random.default_rng(8)
    for m, n, k, b_rows, bf16 in ((5, 128, 256, 128, True), (67, 131, 256, 1, False), (300, 259, 384, 1, True), (130, 256, 256, 128, True)):
        a, sa, b, sb = operands(rng, m, n, k, b_rows)
        dt = torch.bfloat16 if bf16 else torch.float32
        pad = 1024
        buf = torch.full((m * n + 2 * pad,), 77.0, dtype=dt, device="cuda")
        run(a, sa, b, sb, b_rows, bf16, out=buf[pad:pad + m * n].view(m, n))
        assert torch.all(buf[:pad] == 77.0) and torch.all(buf[pad + m * n:] == 77.0)


def test_graph_replays():
    rng = np.random.default_rng(9)
    for m, n, k, b_rows in ((4, 256, 2048, 128), (150, 384, 1024, 128)):
        a, sa, b, sb = (cuda(t) for t in operands(rng, m, n, k, b_rows))
        d = fq.gemm_desc(m, n, k, b_rows)
        ws, out = fq.alloc_gemm_workspace(d), torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
        pa, pb = fq.Plane(a, sa), fq.Plane(b, sb)
        fq.fq_gemm(d, pa, pb, out, ws)
        torch.cuda.synchronize()
        want = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fq.fq_gemm(d, pa, pb, out, ws)
        for _ in range(4):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
