"""fq_rmsnorm and fq_swiglu where their ranges end: results in place, strided
rows with colwise planes, tensors of several GiB, and grids that take turns."""
import pytest
import torch

from fp8_fp4_tensor_amd import fq
from test_gpu_norm import BF16, BOTH, F32, KINDS, inputs, planes_of, same_planes
from test_gpu_swiglu import inputs as gated_inputs

pytestmark = pytest.mark.gpu


def parts(p):
    return [t for t in (p.out.row_data, p.out.row_scale, p.out.col_data, p.out.col_scale) if t is not None]


@pytest.mark.parametrize("x_dt", [BF16, F32], ids=["bf16", "f32"])
def test_gradient_of_the_activation_in_place(x_dt):
    """dx over x, with columns that no thread's eight divide evenly and rows past a tile's end."""
    for rows, cols, outputs in ((3, 8, 0), (130, 1000, 0), (33, 4104, 0), (96, 1056, fq.FQ_ROWWISE), (96, 1056, BOTH),
                                (288, 160, fq.FQ_COLWISE)):
        x, dy = gated_inputs(rows, cols, x_dt, BF16, rows)
        d = fq.swiglu_desc(rows, cols, x_dt)
        p = q = None
        if outputs:
            p, q = (planes_of("mx-e5m2", rows, 2 * cols, outputs, 0x5A) for _ in range(2))
        dx = torch.empty_like(x)
        fq.fq_swiglu_backward(d, x, dy, dx, p)
        fq.fq_swiglu_backward(d, x, dy, x, q)
        torch.cuda.synchronize()
        assert torch.equal(x, dx) and (p is None or all(torch.equal(a, b) for a, b in zip(parts(p), parts(q))))


@pytest.mark.parametrize("kind", list(KINDS))
def test_strided_rows_with_planes(kind):
    """x a slice of a wider tensor with NaN around it."""
    rows, cols = 256, 384
    x, _, w = inputs(rows, cols, BF16, BF16, F32, 1)
    g, dy = gated_inputs(rows, cols, BF16, BF16, 2)

    def inside(t):
        wide = torch.full((rows, t.shape[1] + 48), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, 16:16 + t.shape[1]] = t
        return wide[:, 16:16 + t.shape[1]]

    got = []
    for a, b in ((x, g), (inside(x), inside(g))):
        rstd = torch.empty(rows, device="cuda")
        p, q, r = planes_of(kind, rows, cols), planes_of(kind, rows, cols), planes_of(kind, rows, 2 * cols)
        fq.fq_rmsnorm(fq.rmsnorm_desc(rows, cols), a, w, rstd=rstd, planes=p)
        fq.fq_swiglu(fq.swiglu_desc(rows, cols), b, planes=q)
        fq.fq_swiglu_backward(fq.swiglu_desc(rows, cols), b, dy, planes=r)
        got.append([rstd] + parts(p) + parts(q) + parts(r))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))


def same_rows(big, small, at, rows, cols_data, block):
    """Rows at .. at + rows - 1 of a large call's planes, and those rows as columns of the colwise one, are a small
    call's."""
    a, b = big.out, small.out
    view = lambda t, r: t.view(r, -1)
    R = big.rows
    assert torch.equal(view(a.row_data, R)[at:at + rows], view(b.row_data, rows))
    assert torch.equal(view(a.row_scale, R)[at:at + rows], view(b.row_scale, rows))
    if a.col_data is not None:
        per = a.col_data.numel() // cols_data * rows // R  # bytes of these rows
        lo = per * (at // rows)
        assert torch.equal(view(a.col_data, cols_data)[:, lo:lo + per], view(b.col_data, cols_data))
        lo, n = at // block, rows // block
        assert torch.equal(view(a.col_scale, cols_data)[:, lo:lo + n], view(b.col_scale, cols_data))


def fill(t, seed, scale=1.0):
    """Normal values, a chunk of rows at a time."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    step = max((1 << 29) // t.shape[1], 1)
    for r in range(0, t.shape[0], step):
        part = t[r:r + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return t


@pytest.mark.parametrize("kind,rows,cols", [("mx-e4m3", 1 << 19, 8256), ("mx-e2m1", (1 << 20) + 32, 4160),
                                            ("block", 1 << 21, 2176), ("mx-e5m2", (1 << 27) + 96, 32)])
def test_large_norm_and_its_gradient(kind, rows, cols):
    """Around 2^32 elements (the last case 2^27 rows, more tiles than a grid): slices equal small calls' results."""
    bf = torch.bfloat16
    x, res = (fill(torch.empty((rows, cols), dtype=bf, device="cuda"), s) for s in (1, 2))
    w = torch.rand(cols, device="cuda") + 0.5
    h, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    p = planes_of(kind, rows, cols)
    d = fq.rmsnorm_desc(rows, cols)
    fq.fq_rmsnorm(d, x, w, res, h, rstd, None, p)
    dx, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
    fq.fq_rmsnorm_backward(d, h, rstd, w, x, dx, dw, res, fq.alloc_rmsnorm_workspace(d))
    torch.cuda.synchronize()
    n = 128
    for at in (0, rows // 2 // n * n, (rows - n) // n * n):
        s = slice(at, at + n)
        small = fq.rmsnorm_desc(n, cols)
        h2, r2, dx2, q = torch.empty((n, cols), dtype=bf, device="cuda"), torch.empty(n, device="cuda"), torch.empty(
            (n, cols), dtype=bf, device="cuda"), planes_of(kind, n, cols)
        fq.fq_rmsnorm(small, x[s], w, res[s], h2, r2, None, q)
        fq.fq_rmsnorm_backward(small, h2, r2, w, x[s], dx2, None, res[s])
        torch.cuda.synchronize()
        assert torch.equal(h[s], h2) and torch.equal(rstd[s], r2) and torch.equal(dx[s], dx2)
        same_rows(p, q, at, n, cols, KINDS[kind][2][1])
    # rows behind the last whole 128
    tail = slice(rows - 32, rows)
    last = planes_of(kind, 32, cols, fq.FQ_ROWWISE)
    fq.fq_rmsnorm(fq.rmsnorm_desc(32, cols), x[tail], w, res[tail], torch.empty((32, cols), dtype=bf, device="cuda"),
                  planes=last)
    torch.cuda.synchronize()
    assert torch.equal(p.out.row_data.view(rows, -1)[tail], last.out.row_data.view(32, -1))
    assert torch.equal(p.out.row_scale.view(rows, -1)[tail], last.out.row_scale.view(32, -1))
    # the weight's gradient, summed in 64 bits by pieces; a sum of magnitudes bounds its error: a workgroup's chain of
    # rows / 512 additions at most, and 544 of partial sums, each half a unit
    want, mag = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    step = (1 << 28) // cols
    for r in range(0, rows, step):
        s = slice(r, r + step)
        z = x[s].double() * (h[s].double() * rstd[s, None])
        want += z.sum(0)
        mag += z.abs().sum(0)
    assert bool(((dw.double() - want).abs() <= (rows / 512 + 548) * 2.0 ** -24 * mag).all())


@pytest.mark.parametrize("kind,rows,cols", [("mx-e4m3", 1 << 18, 8256), ("mx-e2m1", (1 << 19) + 32, 4160),
                                            ("block-pow2", 1 << 20, 2176), ("mx-e5m2", (1 << 27) + 96, 32)])
def test_large_activation_and_its_gradient(kind, rows, cols):
    bf = torch.bfloat16
    x = fill(torch.empty((rows, 2 * cols), dtype=bf, device="cuda"), 1, 2.0)
    dy = fill(torch.empty((rows, cols), dtype=bf, device="cuda"), 2)
    p, q = planes_of(kind, rows, cols), planes_of(kind, rows, 2 * cols)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    d = fq.swiglu_desc(rows, cols)
    fq.fq_swiglu(d, x, y, p)
    fq.fq_swiglu_backward(d, x, dy, dx, q)
    alone = torch.empty_like(dx)
    fq.fq_swiglu_backward(d, x, dy, alone)  # by the kernel for rows
    torch.cuda.synchronize()
    assert torch.equal(dx, alone)
    n = 128
    for at in (0, rows // 2 // n * n, (rows - n) // n * n):
        s, small = slice(at, at + n), fq.swiglu_desc(n, cols)
        p2, q2 = planes_of(kind, n, cols), planes_of(kind, n, 2 * cols)
        y2, dx2 = torch.empty((n, cols), dtype=bf, device="cuda"), torch.empty((n, 2 * cols), dtype=bf, device="cuda")
        fq.fq_swiglu(small, x[s], y2, p2)
        fq.fq_swiglu_backward(small, x[s], dy[s], dx2, q2)
        torch.cuda.synchronize()
        assert torch.equal(y[s], y2) and torch.equal(dx[s], dx2)
        same_rows(p, p2, at, n, cols, KINDS[kind][2][1])
        same_rows(q, q2, at, n, 2 * cols, KINDS[kind][2][1])


def test_one_very_long_row():
    """cols = 2^28, the longest: 2^17 workgroups in a row."""
    cols = 1 << 28
    x = fill(torch.empty((256, 2 * cols // 256), dtype=torch.bfloat16, device="cuda"), 1).view(1, 2 * cols)
    y = torch.empty((1, cols), dtype=torch.bfloat16, device="cuda")
    p = planes_of("mx-e4m3", 1, cols, fq.FQ_ROWWISE)
    fq.fq_swiglu(fq.swiglu_desc(1, cols), x, y, p)
    for at in (0, cols - 4096):
        part = torch.cat((x[:, at:at + 4096], x[:, cols + at:cols + at + 4096]), 1)
        y2, q = torch.empty((1, 4096), dtype=torch.bfloat16, device="cuda"), planes_of("mx-e4m3", 1, 4096, fq.FQ_ROWWISE)
        fq.fq_swiglu(fq.swiglu_desc(1, 4096), part, y2, q)
        torch.cuda.synchronize()
        assert torch.equal(y[:, at:at + 4096], y2)
        assert torch.equal(p.out.row_data.view(-1)[at:at + 4096], q.out.row_data.view(-1))
        assert torch.equal(p.out.row_scale.view(-1)[at // 32:at // 32 + 128], q.out.row_scale.view(-1))


def test_last_rows_stay_as_they_were(orc):
    """Planes larger than a call's rows: what lies behind the last row is not written."""
    rows, cols = 37, 544
    x, res, w = inputs(rows, cols, BF16, BF16, F32, 4)
    g, _ = gated_inputs(rows, cols, BF16, BF16, 5)
    for call in ("norm", "activation"):
        data, scale = (torch.full((64 * n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (cols, cols // 32))
        d = fq.desc(fq.FQ_MX, F32, fq.FQ_E4M3, rows, cols, (1, 32))
        p = fq.Planes(d, fq.Quantized(data[:rows * cols], scale[:rows * cols // 32], None, None))
        y = torch.empty((rows, cols), device="cuda")
        if call == "norm":
            fq.fq_rmsnorm(fq.rmsnorm_desc(rows, cols, y_dtype=F32), x, w, res, torch.empty_like(res), y=y, planes=p)
        else:
            fq.fq_swiglu(fq.swiglu_desc(rows, cols, BF16, F32), g, y, p)
        torch.cuda.synchronize()
        same_planes(orc, y, p, "mx-e4m3", fq.FQ_ROWWISE, call)
        assert bool((data[rows * cols:] == 0x5A).all()) and bool((scale[rows * cols // 32:] == 0x5A).all())
