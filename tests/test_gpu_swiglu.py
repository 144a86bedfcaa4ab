"""fq_swiglu and its gradient on the GPU: high-precision results against the
64-bit formula, planes against the oracle's recipe on the same fp32 values."""
import numpy as np
import pytest
import torch

import block_util as B
from fp8_fp4_tensor_amd import fq
from test_gpu_norm import BF16, BOTH, DT, F32, KINDS, d64, planes_of, same_planes

pytestmark = pytest.mark.gpu


def inputs(rows, cols, x_dt, dy_dt, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = rn(rows, 2 * cols) * 2
    x[:, :cols] *= 1 + 12 * (rn(rows, cols) > 2)  # gates far out on either side
    return x.to(DT[x_dt]), (rn(rows, cols) * 1e-2).to(DT[dy_dt])


SHAPES = [(1, 32), (3, 96), (48, 512), (32, 160), (96, 1056), (128, 128), (160, 4096), (257, 288), (384, 640)]


@pytest.mark.parametrize("x_dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", list(KINDS))
def test_forward(orc, kind, x_dt):
    step = KINDS[kind][2][1]
    for rows, cols in SHAPES:
        cols = -(-cols // step) * step
        outputs = BOTH if rows % step == 0 else fq.FQ_ROWWISE
        print(kind, rows, cols, flush=True)
        x, _ = inputs(rows, cols, x_dt, BF16, rows + cols)
        y, p = torch.empty((rows, cols), device="cuda"), planes_of(kind, rows, cols, outputs, 0x5A)
        fq.fq_swiglu(fq.swiglu_desc(rows, cols, x_dt, F32), x, y, p)
        half, alone = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"), planes_of(kind, rows, cols, outputs, 0xA5)
        fq.fq_swiglu(fq.swiglu_desc(rows, cols, x_dt, BF16), x, half)
        fq.fq_swiglu(fq.swiglu_desc(rows, cols, x_dt, BF16), x, None, alone)
        torch.cuda.synchronize()
        want, bound = B.swiglu(d64(x[:, :cols]), d64(x[:, cols:]))
        assert np.all(np.abs(d64(y) - want) <= bound), (np.abs(d64(y) - want) / bound).max()
        assert torch.equal(half, y.to(torch.bfloat16))
        for q in (p, alone):
            same_planes(orc, y, q, kind, outputs, f"{kind} {rows}x{cols}")


@pytest.mark.parametrize("x_dt,dy_dt", [(BF16, BF16), (F32, F32), (BF16, F32)], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("kind", list(KINDS))
def test_backward(orc, kind, x_dt, dy_dt):
    step = KINDS[kind][2][1]
    for rows, cols in SHAPES:
        cols = -(-cols // step) * step
        outputs = BOTH if rows % step == 0 else fq.FQ_ROWWISE
        print(kind, rows, cols, flush=True)
        x, dy = inputs(rows, cols, x_dt, dy_dt, rows + cols)
        # the fp32 gradient, from the same values as fp32
        dx = torch.empty((rows, 2 * cols), device="cuda")
        fq.fq_swiglu_backward(fq.swiglu_desc(rows, cols, F32, dy_dt), x.float(), dy, dx)
        p, alone, own = planes_of(kind, rows, 2 * cols, outputs, 0x5A), planes_of(kind, rows, 2 * cols, outputs, 0xA5), torch.empty_like(x)
        d = fq.swiglu_desc(rows, cols, x_dt, dy_dt)
        fq.fq_swiglu_backward(d, x, dy, own, p)
        fq.fq_swiglu_backward(d, x, dy, None, alone)
        torch.cuda.synchronize()
        dg, du, bg, bu = B.swiglu_gradients(d64(x[:, :cols]), d64(x[:, cols:]), d64(dy))
        for got, want, bound in ((dx[:, :cols], dg, bg), (dx[:, cols:], du, bu)):
            assert np.all(np.abs(d64(got) - want) <= bound), (np.abs(d64(got) - want) / bound).max()
        assert torch.equal(own, dx.to(DT[x_dt]))
        for q in (p, alone):
            same_planes(orc, dx, q, kind, outputs, f"{kind} {rows}x{cols}")


@pytest.mark.parametrize("outputs", [fq.FQ_ROWWISE, fq.FQ_COLWISE], ids=["row", "col"])
def test_one_plane(orc, outputs):
    rows, cols = 192, 352
    x, dy = inputs(rows, cols, BF16, BF16, 3)
    y, dx = torch.empty((rows, cols), device="cuda"), torch.empty((rows, 2 * cols), device="cuda")
    p, q = planes_of("mx-e4m3", rows, cols, outputs), planes_of("mx-e5m2", rows, 2 * cols, outputs)
    fq.fq_swiglu(fq.swiglu_desc(rows, cols, BF16, F32), x, y, p)
    fq.fq_swiglu_backward(fq.swiglu_desc(rows, cols, F32, BF16), x.float(), dy, dx)
    fq.fq_swiglu_backward(fq.swiglu_desc(rows, cols, BF16, BF16), x, dy, None, q)
    torch.cuda.synchronize()
    same_planes(orc, y, p, "mx-e4m3", outputs, "forward")
    same_planes(orc, dx, q, "mx-e5m2", outputs, "backward")


def test_columns_that_no_block_divides_and_strided_rows():
    for rows, cols in ((1, 8), (33, 24), (130, 1000), (200, 136)):
        x, dy = inputs(rows, cols, BF16, BF16, rows)
        wide = torch.full((rows, 2 * cols + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 32:32 + 2 * cols] = x
        s = wide[:, 32:32 + 2 * cols]
        d = fq.swiglu_desc(rows, cols)
        y, ys, dx, dxs = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(x), torch.empty_like(x)
        fq.fq_swiglu(d, x, y)
        fq.fq_swiglu(d, s, ys)
        fq.fq_swiglu_backward(d, x, dy, dx)
        fq.fq_swiglu_backward(d, s, dy, dxs)
        torch.cuda.synchronize()
        want, bound = B.swiglu(d64(x[:, :cols]), d64(x[:, cols:]))
        assert np.all(np.abs(d64(y) - want) <= bound + B.HALF_BF16 * (np.abs(want) + bound))
        assert torch.equal(y, ys) and torch.equal(dx, dxs) and d.x_stride == 0


def test_far_gates():
    """Gates where exp(-gate) is beyond fp32 or vanishes, and zeros of either sign."""
    cols = 64
    gate = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, 80, -80, 87, -87, 88.5, -88.5, 1000, -1000, 3e38, -3e38] * 4, device="cuda")
    x = torch.cat((gate, torch.full((cols,), 1.0, device="cuda")))[None].contiguous()
    dy = torch.ones((1, cols), device="cuda")
    y, dx = torch.empty((1, cols), device="cuda"), torch.empty((1, 2 * cols), device="cuda")
    fq.fq_swiglu(fq.swiglu_desc(1, cols, F32, F32), x, y)
    fq.fq_swiglu_backward(fq.swiglu_desc(1, cols, F32, F32), x, dy, dx)
    torch.cuda.synchronize()
    g = d64(x[:, :cols])
    want, bound = B.swiglu(g, 1.0)
    near = np.abs(g) < 100
    assert np.all(np.abs(d64(y) - want)[near] <= bound[near])
    # far out silu is the gate or zero, its slope one or zero, to the last bit
    far = ~near
    assert np.array_equal(d64(y)[far], np.where(g > 0, g, 0)[far])
    assert np.array_equal(d64(dx[:, :cols])[far], np.where(g > 0, 1.0, 0.0)[far])
    dg, du, bg, bu = B.swiglu_gradients(g[near], np.ones(near.sum()), np.ones(near.sum()))
    assert np.all(np.abs(d64(dx[:, :cols])[near] - dg) <= bg) and np.all(np.abs(d64(dx[:, cols:])[near] - du) <= bu)


def test_gradients_against_differences():
    rng = np.random.default_rng(4)
    rows, cols, t = 9, 96, 1e-5
    x = (2 * rng.standard_normal((rows, 2 * cols))).astype(np.float32).astype(np.float64)
    dy, e = rng.standard_normal((rows, cols)).astype(np.float32).astype(np.float64), rng.standard_normal(x.shape)
    loss = lambda a: (dy * B.swiglu(a[:, :cols], a[:, cols:])[0]).sum()
    cuda = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()
    dx = torch.empty((rows, 2 * cols), device="cuda")
    fq.fq_swiglu_backward(fq.swiglu_desc(rows, cols, F32, F32), cuda(x), cuda(dy), dx)
    torch.cuda.synchronize()
    _, _, bg, bu = B.swiglu_gradients(x[:, :cols], x[:, cols:], dy)
    # the difference: t^2 times a third derivative below a thousand, and 1e-16 / t times a sum below a thousand
    tol = 1e-6 + (np.abs(e) * np.concatenate((bg, bu), 1)).sum()
    assert abs((d64(dx) * e).sum() - (loss(x + t * e) - loss(x - t * e)) / (2 * t)) <= tol


def test_no_rows():
    e, w = (torch.empty((0, n), dtype=torch.bfloat16, device="cuda") for n in (64, 128))
    fq.fq_swiglu(fq.swiglu_desc(0, 64), w, e)
    fq.fq_swiglu(fq.swiglu_desc(0, 64), w, None, planes_of("mx-e4m3", 0, 64))
    fq.fq_swiglu_backward(fq.swiglu_desc(0, 64), w, e, w)
    torch.cuda.synchronize()


def test_writes_only_its_outputs():
    rows, cols, pad = 96, 672, 256
    x, dy = inputs(rows, cols, BF16, BF16, 8)

    def guarded(n, dt):
        b = torch.full((n + 2 * pad,), 77, dtype=dt, device="cuda")
        return b, b[pad:pad + n]

    for wide, call in ((cols, lambda d, y, p: fq.fq_swiglu(d, x, y, p)),
                       (2 * cols, lambda d, y, p: fq.fq_swiglu_backward(d, x, dy, y, p))):
        yb, y = guarded(rows * wide, torch.bfloat16)
        qb, q = guarded(rows * wide, torch.uint8)
        tb, t = guarded(rows * wide, torch.uint8)
        sb, s = guarded(rows * wide // 32, torch.uint8)
        ub, u = guarded(rows * wide // 32, torch.uint8)
        p = fq.Planes(fq.desc(fq.FQ_MX, F32, fq.FQ_E4M3, rows, wide, (1, 32), BOTH), fq.Quantized(q, s, t, u))
        call(fq.swiglu_desc(rows, cols), y.view(rows, wide), p)
        torch.cuda.synchronize()
        for b in (yb, qb, tb, sb, ub):
            assert torch.all(b[:pad] == 77) and torch.all(b[-pad:] == 77)


def test_same_bits_on_a_side_stream_and_in_a_graph():
    for rows, cols in ((5, 4096), (608, 2080)):
        outputs = BOTH if rows % 32 == 0 else fq.FQ_ROWWISE
        x, dy = inputs(rows, cols, BF16, BF16, 8)
        d = fq.swiglu_desc(rows, cols)
        y, dx = torch.empty_like(dy), torch.empty_like(x)
        p, q = planes_of("mx-e4m3", rows, cols, outputs), planes_of("mx-e5m2", rows, 2 * cols, outputs)

        def step(stream=None):
            fq.fq_swiglu(d, x, y, p, stream)
            fq.fq_swiglu_backward(d, x, dy, dx, q, stream)

        def state():
            torch.cuda.synchronize()
            return [t.clone() for o in (p.out, q.out) for t in (o.row_data, o.row_scale, o.col_data, o.col_scale)
                    if t is not None] + [y.clone(), dx.clone()]

        step()
        want = state()
        step(torch.cuda.Stream())
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(3):
            y.zero_(), dx.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(state(), want))
