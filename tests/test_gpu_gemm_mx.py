"""fq_gemm_mx on the GPU against the 64-bit product of the same codes and scales."""
import numpy as np
import pytest
import torch

import block_util as B
from fp8_fp4_tensor_amd import fq
from fp8_fp4_tensor_amd import workloads as W
from gpu_util import dev

pytestmark = pytest.mark.gpu

E4, E5, E2 = fq.FQ_E4M3, fq.FQ_E5M2, fq.FQ_E2M1
PAIRS = [(a, b) for a in (E4, E5, E2) for b in (E4, E5, E2)]
NAMES = {E4: "e4m3", E5: "e5m2", E2: "e2m1"}
pair_ids = [f"{NAMES[a]}-{NAMES[b]}" for a, b in PAIRS]


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def operands(rng, m, n, k, fa, fb, spread=6):
    return (*B.random_operand(rng, m, k, fa, spread), *B.random_operand(rng, n, k, fb, spread))


def run(a, sa, fa, b, sb, fb, bf16, out=None, accumulate=False, stream=None):
    m, n, k = a.shape[0], b.shape[0], 32 * sa.shape[1]
    d = fq.gemm_mx_desc(m, n, k, fa, fb, fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32, accumulate)
    if out is None:
        out = torch.full((m, n), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    pa, pb = fq.MxPlane(cuda(a), cuda(sa), fa), fq.MxPlane(cuda(b), cuda(sb), fb)
    ws = fq.alloc_gemm_mx_workspace(d)
    torch.cuda.synchronize()  # the operands were copied on the current stream
    fq.fq_gemm_mx(d, pa, pb, out, ws, stream)
    torch.cuda.synchronize()
    return out


def check(got, ref, k, fa, fb, bf16, what):
    err = np.abs(got.double().cpu().numpy() - ref[0])
    assert np.linalg.norm(err) <= B.product_norm_bound(ref, k, fa, fb, bf16), what
    bound = B.product_bound(ref, k, fa, fb, bf16)
    assert np.all(err <= bound), (f"{what}: {(err > bound).sum()} of {err.size} out of bound, worst "
                                  f"{np.nanmax(err / bound):.3g}, nan {np.isnan(err).sum()}")


def one(m, n, k, fa, fb, bf16, spread=6):
    print(f"{m}x{n}x{k} {NAMES[fa]} {NAMES[fb]} bf16={bf16}", flush=True)
    rng = np.random.default_rng(m * 1000003 + n * 1009 + k + 10 * fa + fb)
    a, sa, b, sb = operands(rng, m, n, k, fa, fb, spread)
    check(run(a, sa, fa, b, sb, fb, bf16), B.product(a, sa, fa, b, sb, fb), k, fa, fb, bf16, f"{m}x{n}x{k}")


# rows, columns and depths around the tiles' and the instruction's, k short of 64, 128, 256 and 512 by every multiple of 32
SHAPES = [(1, 1, 32), (1, 128, 4096), (2, 3, 64), (15, 17, 96), (16, 384, 640), (17, 130, 160), (33, 515, 224),
          (64, 256, 1120), (65, 250, 256), (127, 640, 288), (130, 257, 1024), (200, 1281, 672), (300, 1000, 352),
          (513, 770, 928)]


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("fa,fb", PAIRS, ids=pair_ids)
def test_product(fa, fb, bf16):
    for m, n, k in SHAPES:
        one(m, n, k, fa, fb, bf16)


@pytest.mark.parametrize("fa,fb", [(E4, E4), (E2, E2), (E4, E2), (E5, E4)], ids=lambda f: NAMES[f])
def test_accumulate(fa, fb):
    for m, n, k in ((5, 128, 256), (70, 131, 384), (300, 513, 160), (9, 256, 4096)):
        rng = np.random.default_rng(m)
        a, sa, b, sb = operands(rng, m, n, k, fa, fb)
        ref = B.product(a, sa, fa, b, sb, fb)
        start = rng.standard_normal((m, n)).astype(np.float32)
        got = run(a, sa, fa, b, sb, fb, False, out=cuda(start), accumulate=True)
        total = ref[0] + start
        bound = B.product_bound(ref, k, fa, fb, False) + 2 * B.HALF_F32 * (np.abs(total) + ref[1])
        assert np.all(np.abs(got.double().cpu().numpy() - total) <= bound), (m, n, k)


def test_empty_products():
    z = lambda r, c: np.zeros((r, c), np.uint8)
    assert torch.all(run(z(4, 0), z(4, 0), E4, z(7, 0), z(7, 0), E2, True) == 0)
    keep = torch.full((4, 7), 3.0, device="cuda")
    assert torch.all(run(z(4, 0), z(4, 0), E4, z(7, 0), z(7, 0), E4, False, out=keep, accumulate=True) == 3.0)
    for m, n in ((0, 5), (5, 0), (0, 0)):
        assert run(z(m, 64), z(m, 2), E4, z(n, 64), z(n, 2), E4, True).numel() == 0


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_zero_blocks_largest_codes_and_far_scales(bf16):
    """The scale code 0 of an all-zero block, the largest codes, and scales 100 binades apart on either side."""
    for fa, fb, top_a, top_b in ((E4, E4, 0x7E, 0xFE), (E2, E2, 0x77, 0xFF), (E4, E2, 0x7E, 0xFF)):
        m, n, k = 40, 144, 512
        a = np.full((m, k * B.BITS[fa] // 8), top_a, np.uint8)
        b = np.full((n, k * B.BITS[fb] // 8), top_b, np.uint8)
        sa, sb = np.full((m, 16), 126, np.uint8), np.full((n, 16), 128, np.uint8)
        w = B.BITS[fa] * 32 // 8
        a[:, 3 * w:4 * w], sa[:, 3] = 0, 0
        sa[:, 5], sb[:, 5] = 227, 27      # 2^100 times 2^-100
        sa[:, 6], sb[:, 6] = 27, 227
        sa[3, 9] = 0                      # 2^-127 times finite codes: next to nothing
        check(run(a, sa, fa, b, sb, fb, bf16), B.product(a, sa, fa, b, sb, fb), k, fa, fb, bf16, f"{fa} {fb}")


def quantized(x, fmt, outputs=fq.FQ_ROWWISE | fq.FQ_COLWISE):
    d = fq.desc(fq.FQ_MX, fq.FQ_IN_BF16, fmt, *x.shape, (1, 32), outputs)
    q = fq.alloc_quantized(d)
    fq.fq_quantize(d, dev(x), q)
    torch.cuda.synchronize()
    return q


@pytest.mark.parametrize("fx,fw,fg", [(E4, E4, E4), (E4, E4, E5), (E2, E2, E2), (E4, E2, E5)],
                         ids=["e4m3", "e5m2-gradients", "e2m1", "mixed"])
def test_linear_layer_three_products(fx, fw, fg):
    """Forward, input gradient and weight gradient from the library's own planes; tokens no multiple of 128."""
    T, O, I = 224, 384, 544
    X, Wt, G = W.normal((T, I), 1.0, 1), W.normal((O, I), 0.02, 2), W.normal((T, O), 1e-3, 3)
    qx, qw, qg = quantized(X, fx), quantized(Wt, fw), quantized(G, fg)

    def product(pa, pb, m, n, k, bf16, what):
        d = fq.gemm_mx_desc(m, n, k, pa.fmt, pb.fmt, fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32)
        out = torch.empty((m, n), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        fq.fq_gemm_mx(d, pa, pb, out, fq.alloc_gemm_mx_workspace(d))
        torch.cuda.synchronize()
        h = lambda t, r: t.cpu().numpy().reshape(r, -1)
        ref = B.product(h(pa.data, m), h(pa.scale, m), pa.fmt, h(pb.data, n), h(pb.scale, n), pb.fmt)
        check(out, ref, k, pa.fmt, pb.fmt, bf16, what)
        return out

    row, col = fq.MxPlane.rowwise, fq.MxPlane.colwise
    y = product(row(qx, fx), row(qw, fw), T, O, I, True, "forward")
    dx = product(row(qg, fg), col(qw, fw), T, I, O, True, "input gradient")
    dw = product(col(qg, fg), col(qx, fx), O, I, T, False, "weight gradient")
    # against the unquantized formula: half a step of a value is 2^-4 (E4M3), 2^-3 (E5M2), 2^-2 (E2M1) of it, or for values next to
    # zero as much of a quarter of the block's largest; the mean square of both factors is below three quarters of the sum
    step = {E4: 2.0 ** -4, E5: 2.0 ** -3, E2: 2.0 ** -2}
    f = lambda x: W.bf16_bits_to_f32(x).astype(np.float64)
    for got, full, p, q in ((y, f(X) @ f(Wt).T, fx, fw), (dx, f(G) @ f(Wt), fg, fw), (dw, f(G).T @ f(X), fg, fx)):
        assert np.linalg.norm(got.double().cpu().numpy() - full) <= 0.75 * (step[p] + step[q]) * np.linalg.norm(full)


def test_gradients_against_differences():
    """L = <G, X W^T> is linear in X and in W: L(X') - L(X) = <dX, X' - X>, and the same for W."""
    rng = np.random.default_rng(5)
    T, O, I = 96, 160, 128
    one = lambda r, c: np.full((r, c // 32), 127, np.uint8)
    codes = lambda r, c: B.random_operand(rng, r, c, E4)[0]
    val = B.table(E4)
    x0, x1, w0, w1, g = codes(T, I), codes(T, I), codes(O, I), codes(O, I), codes(T, O)
    t = np.ascontiguousarray
    y = lambda x, w: run(x, one(T, I), E4, w, one(O, I), E4, False).double().cpu().numpy()
    dx = run(g, one(T, O), E4, t(w0.T), one(I, O), E4, False).double().cpu().numpy()
    dw = run(t(g.T), one(O, T), E4, t(x0.T), one(I, T), E4, False).double().cpu().numpy()
    mag = (np.abs(val[g]) * ((np.abs(val[x0]) + np.abs(val[x1])) @ (np.abs(val[w0]) + np.abs(val[w1])).T)).sum()
    tol = 4 * 512 * B.ULP32 * mag
    base = (val[g] * y(x0, w0)).sum()
    assert abs((val[g] * y(x1, w0)).sum() - base - (dx * (val[x1] - val[x0])).sum()) <= tol
    assert abs((val[g] * y(x0, w1)).sum() - base - (dw * (val[w1] - val[w0])).sum()) <= tol


def test_same_bits_every_run_and_on_a_side_stream():
    rng = np.random.default_rng(7)
    for m, n, k, fa, fb in ((7, 256, 4096, E4, E2), (200, 512, 2048, E4, E4), (300, 515, 1056, E2, E2)):
        a, sa, b, sb = operands(rng, m, n, k, fa, fb)
        for bf16 in (True, False):
            first = run(a, sa, fa, b, sb, fb, bf16)
            s = torch.cuda.Stream()
            assert torch.equal(first, run(a, sa, fa, b, sb, fb, bf16, stream=s))


def test_writes_only_its_output_and_workspace():
    """Guards before and behind the output and the workspace stay as they were (ragged m and n)."""
    rng = np.random.default_rng(8)
    pad = 1024
    for m, n, k, fa, fb, bf16 in ((5, 128, 256, E4, E4, True), (67, 131, 288, E2, E2, False), (300, 259, 416, E4, E2, True),
                                  (130, 1000, 4128, E5, E4, False), (40, 64, 8192, E2, E2, True)):
        a, sa, b, sb = operands(rng, m, n, k, fa, fb)
        dt = torch.bfloat16 if bf16 else torch.float32
        buf = torch.full((m * n + 2 * pad,), 77.0, dtype=dt, device="cuda")
        d = fq.gemm_mx_desc(m, n, k, fa, fb, fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32)
        z = fq.fq_gemm_mx_workspace(d)
        ws = torch.full((z + 2 * pad,), 77, dtype=torch.uint8, device="cuda")
        out = buf[pad:pad + m * n].view(m, n)
        fq.fq_gemm_mx(d, fq.MxPlane(cuda(a), cuda(sa), fa), fq.MxPlane(cuda(b), cuda(sb), fb), out, ws[pad:pad + z])
        torch.cuda.synchronize()
        check(out, B.product(a, sa, fa, b, sb, fb), k, fa, fb, bf16, f"{m}x{n}x{k}")
        for t, size in ((buf, m * n), (ws, z)):
            assert torch.all(t[:pad] == 77) and torch.all(t[pad + size:] == 77)


def test_neighbours_of_an_operand_do_not_matter():
    """What lies behind an operand in memory (NaN codes, scale codes 255) reaches no result."""
    rng = np.random.default_rng(11)
    for m, n, k, fa, fb in ((3, 20, 160, E4, E4), (70, 130, 96, E4, E2), (260, 300, 608, E2, E2), (33, 66, 4128, E5, E4)):
        a, sa, b, sb = operands(rng, m, n, k, fa, fb)

        def inside(x):
            flat = torch.full((x.size + 8192,), 255, dtype=torch.uint8, device="cuda")
            flat[4096:4096 + x.size] = cuda(x).view(-1)
            return flat[4096:4096 + x.size].view(x.shape)

        for bf16 in (True, False):
            d = fq.gemm_mx_desc(m, n, k, fa, fb, fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32)
            out = torch.empty((m, n), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
            fq.fq_gemm_mx(d, fq.MxPlane(inside(a), inside(sa), fa), fq.MxPlane(inside(b), inside(sb), fb), out,
                          fq.alloc_gemm_mx_workspace(d))
            torch.cuda.synchronize()
            check(out, B.product(a, sa, fa, b, sb, fb), k, fa, fb, bf16, f"{m}x{n}x{k}")


def test_graph_replays():
    rng = np.random.default_rng(9)
    for m, n, k, fa, fb in ((4, 256, 2048, E4, E2), (150, 384, 1056, E4, E4), (40, 64, 8192, E2, E2)):
        a, sa, b, sb = (cuda(t) for t in operands(rng, m, n, k, fa, fb))
        d = fq.gemm_mx_desc(m, n, k, fa, fb)
        ws, out = fq.alloc_gemm_mx_workspace(d), torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
        pa, pb = fq.MxPlane(a, sa, fa), fq.MxPlane(b, sb, fb)
        fq.fq_gemm_mx(d, pa, pb, out, ws)
        torch.cuda.synchronize()
        want = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fq.fq_gemm_mx(d, pa, pb, out, ws)
        for _ in range(4):
            out.zero_()
            if ws is not None:
                ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
