"""fq_rmsnorm and its gradients on the GPU: high-precision results against the
64-bit formula, planes against the oracle's recipe on the same fp32 values."""
import numpy as np
import pytest
import torch

import block_util as B
from fp8_fp4_tensor_amd import fq

pytestmark = pytest.mark.gpu

DT = {fq.FQ_IN_F32: torch.float32, fq.FQ_IN_BF16: torch.bfloat16}
F32, BF16 = fq.FQ_IN_F32, fq.FQ_IN_BF16
# recipe, format, block, scale mode
KINDS = {"mx-e4m3": (fq.FQ_MX, fq.FQ_E4M3, (1, 32), 0), "mx-e5m2": (fq.FQ_MX, fq.FQ_E5M2, (1, 32), 0),
         "mx-e2m1": (fq.FQ_MX, fq.FQ_E2M1, (1, 32), 0), "block": (fq.FQ_BLOCK_FP32, fq.FQ_E4M3, (1, 128), 0),
         "block-pow2": (fq.FQ_BLOCK_FP32, fq.FQ_E4M3, (1, 128), 1)}
BOTH = fq.FQ_ROWWISE | fq.FQ_COLWISE


def planes_of(kind, rows, cols, outputs=BOTH, fill=None):
    recipe, fmt, block, mode = KINDS[kind]
    d = fq.desc(recipe, F32, fmt, rows, cols, block, outputs, scale_mode=mode)
    q = fq.alloc_quantized(d)
    if fill is not None:
        for t in (q.row_data, q.row_scale, q.col_data, q.col_scale):
            if t is not None:
                t.fill_(fill)
    return fq.Planes(d, q)


def same_planes(orc, y, planes, kind, outputs, what):
    """The planes hold, byte for byte, what the recipe gives for the fp32 values y."""
    recipe, fmt, block, mode = KINDS[kind]
    y = y.cpu().numpy()
    want = orc.quantize_mx(y, outputs=outputs, fmt=fmt) if recipe == fq.FQ_MX else \
        orc.quantize_block(y, block, outputs=outputs, pow2=bool(mode))
    e = "e" if recipe == fq.FQ_MX else "s"
    q = planes.out
    for got, name in ((q.row_data, "q_row"), (q.row_scale, e + "_row"), (q.col_data, "q_col"), (q.col_scale, e + "_col")):
        if got is None:
            continue
        a, b = got.cpu().numpy().reshape(-1), want[name].reshape(-1)
        assert a.dtype == b.dtype and a.shape == b.shape and np.array_equal(a.view(np.uint8), b.view(np.uint8)), (
            f"{what} {name}: {(a != b).sum()} of {a.size} differ")


def inputs(rows, cols, x_dt, h_dt, w_dt, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = (rn(rows, cols) * 0.5 * scale).to(DT[x_dt])
    res = (rn(rows, cols) * (1 + 9 * (rn(cols) > 2)) * scale).to(DT[h_dt])
    return x, res, (1 + 0.3 * rn(cols)).to(DT[w_dt])


def d64(t):
    return t.double().cpu().numpy()


def check_norm(h, w, eps, rstd, y, what):
    """rstd and fp32 y of the stored h."""
    r, want = B.norm(d64(h), d64(w), eps)
    assert np.all(np.abs(d64(rstd) - r) <= B.RSTD_REL * r), what
    assert np.all(np.abs(d64(y) - want) <= B.Y_REL * np.abs(want) + 1e-37), what


# every row configuration (512, 1024, 2048, 4096, 8192, 16384, 32768 columns), just within and just past it
COLS = [32, 96, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 7168, 8192, 8224, 16384, 16416, 32768]


@pytest.mark.parametrize("cols", COLS)
def test_norm_and_planes(orc, cols):
    for n, (rows, kind, x_dt, h_dt, w_dt) in enumerate([(1, "mx-e4m3", BF16, BF16, F32), (5, "mx-e2m1", F32, BF16, BF16),
                                                        (96, "mx-e5m2", BF16, F32, F32), (160, "mx-e4m3", F32, F32, BF16),
                                                        (256, "mx-e2m1", BF16, BF16, F32)]):
        print(cols, rows, kind, flush=True)
        outputs = BOTH if rows % 32 == 0 else fq.FQ_ROWWISE
        x, res, w = inputs(rows, cols, x_dt, h_dt, w_dt, n)
        d = fq.rmsnorm_desc(rows, cols, x_dt, h_dt, w_dt, F32, eps=1e-5)
        h, rstd = torch.empty_like(res), torch.empty(rows, device="cuda")
        y, p = torch.empty((rows, cols), device="cuda"), planes_of(kind, rows, cols, outputs, 0x5A)
        fq.fq_rmsnorm(d, x, w, res, h, rstd, y, p)
        torch.cuda.synchronize()
        total = d64(x) + d64(res)
        assert np.all(np.abs(d64(h) - total) <= (B.half(h.dtype) + B.HALF_F32) * np.abs(total) * (1 + 2.0 ** -8))
        check_norm(h, w, d.eps, rstd, y, f"{rows}x{cols}")
        same_planes(orc, y, p, kind, outputs, f"{rows}x{cols}")


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("outputs", [fq.FQ_ROWWISE, fq.FQ_COLWISE, BOTH], ids=["row", "col", "both"])
def test_every_kind_without_residual(orc, kind, outputs):
    step = KINDS[kind][2][1]
    for rows, cols in ((step, step), (3 * step, 5 * step), (384, 1280), (640, 640 + step)):
        for x_dt in (BF16, F32):
            x, _, w = inputs(rows, cols, x_dt, x_dt, F32, rows)
            x[min(2, rows - 1)] = 0          # a row of zeros: its y is zeros, its blocks' amax too
            x[:, :step] *= 1e-30             # next to nothing beside the row's other blocks
            d = fq.rmsnorm_desc(rows, cols, x_dt, y_dtype=F32)
            y, rstd, p = torch.empty((rows, cols), device="cuda"), torch.empty(rows, device="cuda"), planes_of(kind, rows, cols, outputs, 0x5A)
            fq.fq_rmsnorm(d, x, w, rstd=rstd, y=y, planes=p)
            torch.cuda.synchronize()
            check_norm(x, w, d.eps, rstd, y, f"{rows}x{cols}")
            same_planes(orc, y, p, kind, outputs, f"{kind} {rows}x{cols}")
            # the same planes without the high-precision copy, and (rowwise alone) without rstd
            again = planes_of(kind, rows, cols, outputs, 0xA5)
            fq.fq_rmsnorm(d, x, w, rstd=None if outputs == fq.FQ_ROWWISE else rstd, planes=again)
            torch.cuda.synchronize()
            same_planes(orc, y, again, kind, outputs, f"{kind} {rows}x{cols} alone")


@pytest.mark.parametrize("cols", [8, 24, 504, 1000, 5000, 9000, 20008])
def test_result_alone_and_its_rounding(cols):
    """Columns that no block divides; bf16 results are the fp32 ones rounded."""
    rows = 37
    x, res, w = inputs(rows, cols, BF16, F32, F32, cols)
    out = []
    for y_dt in (F32, BF16):
        d = fq.rmsnorm_desc(rows, cols, BF16, F32, F32, y_dt)
        y, h = torch.empty((rows, cols), dtype=DT[y_dt], device="cuda"), torch.empty_like(res)
        rstd = torch.empty(rows, device="cuda")
        fq.fq_rmsnorm(d, x, w, res, h, rstd, y)
        torch.cuda.synchronize()
        out.append(y)
    check_norm(h, w, 1e-6, rstd, out[0], "f32")
    assert torch.equal(out[0].to(torch.bfloat16), out[1])


def test_strided_rows_and_in_place():
    """x as a slice of a wider tensor; h written over the residual, and over x."""
    rows, cols = 70, 1536
    wide = torch.randn((rows, 4096), device="cuda").to(torch.bfloat16)
    x = wide[:, 512:512 + cols]
    _, res, w = inputs(rows, cols, BF16, BF16, F32, 3)
    d = fq.rmsnorm_desc(rows, cols)
    y, h, y2 = (torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    fq.fq_rmsnorm(d, x.contiguous(), w, res, h, y=y)
    over = res.clone()
    fq.fq_rmsnorm(d, x, w, over, over, y=y2)
    xo = x.contiguous()
    y3 = torch.empty_like(y)
    fq.fq_rmsnorm(d, xo, w, res, xo, y=y3)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3) and torch.equal(over, h) and torch.equal(xo, h)
    assert d.x_stride == 0


def test_extreme_rows():
    """Rows near the ends of the range: eps alone, squares that vanish, squares near 2^127."""
    rows, cols = 4, 4096
    x = torch.zeros((rows, cols), device="cuda")
    x[1] = 1e-30
    x[2] = torch.randn(cols, device="cuda") * 1e17
    x[3, 7] = 1e-3
    w = torch.ones(cols, device="cuda")
    d = fq.rmsnorm_desc(rows, cols, F32, F32, F32, F32, eps=1e-12)
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    fq.fq_rmsnorm(d, x, w, rstd=rstd, y=y)
    torch.cuda.synchronize()
    check_norm(x, w, d.eps, rstd, y, "extremes")


# ---------------------------------------------------------------- gradients
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 96), (130, 512), (9, 520), (257, 1024), (1, 4096), (70, 2048),
                                       (67, 2056), (1030, 4104), (40, 8192), (33, 8200), (5, 16384), (3, 16392),
                                       (2, 32768), (2500, 264), (5000, 1032)])
def test_gradients(rows, cols):
    for h_dt, dy_dt, w_dt, past in ((BF16, BF16, F32, True), (F32, BF16, BF16, True), (BF16, F32, F32, False),
                                    (F32, F32, F32, True)):
        print(rows, cols, h_dt, dy_dt, flush=True)
        _, h, w = inputs(rows, cols, BF16, h_dt, w_dt, rows + cols)
        dy, dres, _ = inputs(rows, cols, dy_dt, h_dt, w_dt, rows + cols + 1, 1e-2)
        d = fq.rmsnorm_desc(rows, cols, h_dtype=h_dt, weight_dtype=w_dt, y_dtype=dy_dt)
        rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
        dx, dw = torch.empty_like(h), torch.full((cols,), float("nan"), device="cuda")
        fq.fq_rmsnorm_backward(d, h, rstd, w, dy, dx, dw, dres if past else None, fq.alloc_rmsnorm_workspace(d))
        torch.cuda.synchronize()
        want, wantw, bx, bw = B.norm_gradients(d64(h), d64(rstd), d64(w), d64(dy), d64(dres) if past else 0.0)
        bx = bx + B.half(dx.dtype) * (np.abs(want) + bx)
        assert np.all(np.abs(d64(dx) - want) <= bx), (np.abs(d64(dx) - want) / bx).max()
        assert np.all(np.abs(d64(dw) - wantw) <= bw + B.HALF_F32 * np.abs(wantw)), (np.abs(d64(dw) - wantw) / bw).max()


def test_gradients_against_differences():
    """<dx, e> and <dw, f> against the symmetric difference of <dy, y(x + t e, w + t f)>, the forward pass in 64 bits."""
    rng = np.random.default_rng(2)
    rows, cols, t = 12, 192, 1e-5
    h, w, dy = rng.standard_normal((rows, cols)), 1 + 0.3 * rng.standard_normal(cols), rng.standard_normal((rows, cols))
    e, f = rng.standard_normal((rows, cols)), rng.standard_normal(cols)
    h, w, dy = (x.astype(np.float32).astype(np.float64) for x in (h, w, dy))
    loss = lambda a, b: (dy * B.norm(a, b, 1e-5)[1]).sum()
    cuda = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()
    d = fq.rmsnorm_desc(rows, cols, F32, F32, F32, F32, eps=1e-5)
    rstd, y = torch.empty(rows, device="cuda"), torch.empty((rows, cols), device="cuda")
    fq.fq_rmsnorm(d, cuda(h), cuda(w), rstd=rstd, y=y)
    dx, dw = torch.empty((rows, cols), device="cuda"), torch.empty(cols, device="cuda")
    fq.fq_rmsnorm_backward(d, cuda(h), rstd, cuda(w), cuda(dy), dx, dw, ws=fq.alloc_rmsnorm_workspace(d))
    torch.cuda.synchronize()
    # the difference is off by t^2 times a third derivative of a few hundred at most, 1e-8, and 1e-16 / t of a sum of
    # magnitude 1e3, 1e-8; the gradients by the bounds above, with dx's dependence on rstd's own error (32 halves)
    gx, gw, bx, bw = B.norm_gradients(h, d64(rstd), w, dy, 0.0)
    tol = 1e-6 + (np.abs(e) * (bx + 3 * B.RSTD_REL * (np.abs(gx) + np.abs(dy * w) * d64(rstd)[:, None]))).sum()
    assert abs((d64(dx) * e).sum() - (loss(h + t * e, w) - loss(h - t * e, w)) / (2 * t)) <= tol
    tol = 1e-6 + (np.abs(f) * (bw + B.RSTD_REL * np.abs(dy * h * d64(rstd)[:, None]).sum(0))).sum()
    assert abs((d64(dw) * f).sum() - (loss(h, w + t * f) - loss(h, w - t * f)) / (2 * t)) <= tol


def test_weight_gradient_accumulates_and_may_be_left_out():
    rows, cols = 300, 768
    _, h, w = inputs(rows, cols, BF16, BF16, F32, 5)
    dy, dres, _ = inputs(rows, cols, BF16, BF16, F32, 6)
    rstd = (1 / torch.sqrt(h.float().square().mean(1) + 1e-6))
    d, a = fq.rmsnorm_desc(rows, cols), fq.rmsnorm_desc(rows, cols, accumulate=True)
    ws = fq.alloc_rmsnorm_workspace(d)
    dx, dw, two = torch.empty_like(h), torch.empty(cols, device="cuda"), torch.zeros(cols, device="cuda")
    fq.fq_rmsnorm_backward(d, h, rstd, w, dy, dx, dw, dres, ws)
    for _ in range(2):
        fq.fq_rmsnorm_backward(a, h, rstd, w, dy, dx, two, dres, ws)
    dx2, over = torch.empty_like(h), dres.clone()
    fq.fq_rmsnorm_backward(d, h, rstd, w, dy, dx2, None, dres)
    fq.fq_rmsnorm_backward(d, h, rstd, w, dy, over, None, over)  # dx over dres
    over_h = h.clone()
    fq.fq_rmsnorm_backward(d, over_h, rstd, w, dy, over_h, None, dres)  # and over h
    torch.cuda.synchronize()
    assert torch.equal(two, dw + dw) and torch.equal(dx, dx2) and torch.equal(dx, over) and torch.equal(dx, over_h)


def test_no_rows():
    d, a = fq.rmsnorm_desc(0, 256), fq.rmsnorm_desc(0, 256, accumulate=True)
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    r, w, dw = torch.empty(0, device="cuda"), torch.ones(256, device="cuda"), torch.full((256,), 3.0, device="cuda")
    fq.fq_rmsnorm(d, e, w, y=torch.empty_like(e))
    fq.fq_rmsnorm(d, e, w, rstd=r, planes=planes_of("mx-e4m3", 0, 256))
    fq.fq_rmsnorm_backward(a, e, r, w, e, e, dw)
    torch.cuda.synchronize()
    assert torch.all(dw == 3.0)
    fq.fq_rmsnorm_backward(d, e, r, w, e, e, dw)
    torch.cuda.synchronize()
    assert torch.all(dw == 0.0)


def test_writes_only_its_outputs():
    rows, cols, pad = 96, 672, 256
    x, res, w = inputs(rows, cols, BF16, BF16, F32, 8)

    def guarded(n, dt):
        b = torch.full((n + 2 * pad,), 77, dtype=dt, device="cuda")
        return b, b[pad:pad + n]

    hb, h = guarded(rows * cols, torch.bfloat16)
    yb, y = guarded(rows * cols, torch.bfloat16)
    rb, r = guarded(rows, torch.float32)
    qb, q = guarded(rows * cols, torch.uint8)
    tb, t = guarded(rows * cols, torch.uint8)
    sb, s = guarded(rows * cols // 32, torch.uint8)
    ub, u = guarded(rows * cols // 32, torch.uint8)
    v = lambda z: z.view(rows, cols)
    p = fq.Planes(fq.desc(fq.FQ_MX, F32, fq.FQ_E4M3, rows, cols, (1, 32), BOTH), fq.Quantized(q, s, t, u))
    d = fq.rmsnorm_desc(rows, cols)
    fq.fq_rmsnorm(d, x, w, res, v(h), r, v(y), p)
    wb, dw = guarded(cols, torch.float32)
    xb, dx = guarded(rows * cols, torch.bfloat16)
    z = fq.fq_rmsnorm_workspace(d)
    kb, ws = guarded(z, torch.uint8)
    fq.fq_rmsnorm_backward(d, v(h), r, w, v(y), v(dx), dw, res, ws)
    torch.cuda.synchronize()
    for b in (hb, yb, rb, qb, tb, sb, ub, wb, xb, kb):
        assert torch.all(b[:pad] == 77) and torch.all(b[-pad:] == 77)


def test_same_bits_on_a_side_stream_and_in_a_graph():
    for rows, cols in ((5, 4096), (608, 2080)):
        outputs = BOTH if rows % 32 == 0 else fq.FQ_ROWWISE
        x, res, w = inputs(rows, cols, BF16, BF16, F32, 8)
        dy, dres, _ = inputs(rows, cols, BF16, BF16, F32, 9)
        d = fq.rmsnorm_desc(rows, cols)
        h, rstd, dx, dw = torch.empty_like(res), torch.empty(rows, device="cuda"), torch.empty_like(res), torch.empty(cols, device="cuda")
        p, ws = planes_of("mx-e4m3", rows, cols, outputs), fq.alloc_rmsnorm_workspace(d)

        def step(stream=None):
            fq.fq_rmsnorm(d, x, w, res, h, rstd, None, p, stream)
            fq.fq_rmsnorm_backward(d, h, rstd, w, dy, dx, dw, dres, ws, stream)

        def state():
            torch.cuda.synchronize()
            q = p.out
            return [t.clone() for t in (h, rstd, dx, dw, q.row_data, q.row_scale, q.col_data, q.col_scale) if t is not None]

        step()
        want = state()
        step(torch.cuda.Stream())
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(3):
            for t in (h, rstd, dx, dw):
                t.zero_()
            ws.fill_(255)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(state(), want))
