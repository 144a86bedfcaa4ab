"""fq_gemm_mx: every kernel that it can take, codes that are no numbers, several
calls at once, and operands and results of several GiB."""
import pytest
import torch

import block_util as B
import mx_plans as P
from fp8_fp4_tensor_amd import fq
from operator_util import HALF_BF16, HALF_F32, ULP32

pytestmark = pytest.mark.gpu

E4, E5, E2 = fq.FQ_E4M3, fq.FQ_E5M2, fq.FQ_E2M1


def operand(rows, k, fmt, seed):
    """(data, scale codes) on the GPU: finite codes of every magnitude, scales over 12 binades."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = torch.randint(0, 256, (rows, k * B.BITS[fmt] // 8), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == E4:
        c.masked_fill_((c & 127) == 127, 0)
    elif fmt == E5:
        c.masked_fill_((c & 127) >= 124, 0)
    return c, torch.randint(121, 134, (rows, k // 32), generator=g, device="cuda", dtype=torch.uint8)


def values(data, scale, fmt):
    """[rows, k] in 64 bits."""
    t = torch.from_numpy(B.table(fmt)).cuda()
    c = data if fmt != E2 else torch.stack((data & 15, data >> 4), 2).view(data.shape[0], -1)
    v = t[c.long()].view(*scale.shape, 32) * torch.exp2(scale.double() - 127)[:, :, None]
    return v.view(data.shape[0], -1)


def runs_top(v):
    """The largest magnitude of each run of 128."""
    pad = -v.shape[1] % 128
    return torch.nn.functional.pad(v.abs(), (0, pad)).view(v.shape[0], -1, 128).amax(2)


def reference(a, b):
    """block_util.product on the GPU, of 64-bit values."""
    return a @ b.t(), a.abs() @ b.abs().t(), runs_top(a) @ runs_top(b).t().contiguous()


def check(got, ref, k, fa, fb, bf16, what):
    """block_util.product_bound and product_norm_bound on the GPU."""
    c, s, top = ref
    err = (got.double() - c).abs_()
    half, sums = HALF_BF16 if bf16 else HALF_F32, (128 + 2 * (k // 128 + 32)) * ULP32
    narrow = bf16 and not (fa == E2 and fb == E2)
    assert err.norm() <= half * c.norm() + ((2.0 ** -12 if narrow else 0.0) + sums) * s.norm() + 1e-37, what
    bound = sums * s
    if narrow:
        bound = bound + 128 * 2.0 ** -13 * top
    bound = bound + half * (c.abs() + bound) + 1e-37
    assert bool((err <= bound).all()), f"{what}: {(err > bound).sum()} of {err.numel()}, worst {(err / bound).max():.3g}"


def call(a, b, fa, fb, out, accumulate=False, ws=None, stream=None):
    (m, n), k = out.shape, 32 * a[1].shape[1]
    d = fq.gemm_mx_desc(m, n, k, fa, fb, fq.FQ_IN_BF16 if out.dtype == torch.bfloat16 else fq.FQ_IN_F32, accumulate)
    fq.fq_gemm_mx(d, fq.MxPlane(*a, fa), fq.MxPlane(*b, fb), out, fq.alloc_gemm_mx_workspace(d) if ws is None else ws, stream)


def whole(kind, shape, pairs=None):
    m, n, k = shape
    every, bf16 = P.KINDS[kind]
    pad = 1024
    for fa, fb in pairs or every:
        print(kind, fa, fb, shape, flush=True)
        a, b = operand(m, k, fa, m + k), operand(n, k, fb, n + k + 1)
        va, vb = values(*a, fa), values(*b, fb)
        ref = reference(va, vb)
        buf = torch.full((m * n + 2 * pad,), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        out = buf[pad:-pad].view(m, n).fill_(float("nan"))
        call(a, b, fa, fb, out)
        torch.cuda.synchronize()
        check(out, ref, k, fa, fb, bf16, f"{kind} {fa} {fb} {shape}")
        if not bf16:
            once = out.clone()
            call(a, b, fa, fb, out, True)
            torch.cuda.synchronize()
            # C + product, rounded once: the product again (the same sums), added to itself
            assert torch.equal(out, once + once)
        assert bool((buf[:pad] == 7).all()) and bool((buf[-pad:] == 7).all())


@pytest.mark.parametrize("kind,tile,split,rest,arranged,shape", P.PLANS, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_every_kernel(kind, tile, split, rest, arranged, shape):
    """Whole results of every pair of formats, with guards around them."""
    whole(kind, shape)


@pytest.mark.parametrize("kind,arranged,shape", P.WALKS, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_several_tiles_a_workgroup(kind, arranged, shape):
    whole(kind, shape, P.KINDS[kind][0][:2])


def test_codes_that_are_no_numbers():
    """A NaN code or a scale code of 255 makes its row (of A) or column (of B) of C NaN, and nothing else."""
    for m, n, k, fa, fb in ((5, 64, 256, E4, E4), (5, 64, 256, E2, E4), (300, 520, 512, E4, E2), (200, 130, 384, E5, E4),
                            (16428, 267, 128, E4, E4), (70, 300, 1024, E2, E2)):
        for bf16 in (True, False):
            print(m, n, k, fa, fb, bf16, flush=True)
            a, b = operand(m, k, fa, 1), operand(n, k, fb, 2)
            clean = torch.empty((m, n), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
            call(a, b, fa, fb, clean)
            rows, cols = [m // 2], [n // 3]
            a[1][m // 2, k // 64], b[1][n // 3, 0] = 255, 255
            if fa != E2:
                a[0][m - 1, 5] = 0x7F
                rows.append(m - 1)
            if fb != E2:
                b[0][n - 1, k - 1] = 0xFF
                cols.append(n - 1)
            out = torch.empty_like(clean)
            call(a, b, fa, fb, out)
            torch.cuda.synchronize()
            mask = torch.zeros((m, n), dtype=torch.bool, device="cuda")
            mask[rows] = True
            mask[:, cols] = True
            assert torch.equal(out.isnan(), mask) and torch.equal(out[~mask], clean[~mask])


def test_infinities():
    """E5M2's infinity: infinite results of the sign of the code it meets, NaN where it meets a zero."""
    m, n, k = 40, 96, 256
    for bf16 in (True, False):
        a, b = operand(m, k, E5, 3), operand(n, k, E4, 4)
        b[0][:, 7] = torch.tensor([0x38, 0xB8, 0x00], dtype=torch.uint8, device="cuda").repeat(n // 3)  # 1, -1, 0
        a[0][3, 7] = 0x7C
        out = torch.empty((m, n), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        call(a, b, E5, E4, out)
        torch.cuda.synchronize()
        want = torch.tensor([float("inf"), -float("inf"), float("nan")], device="cuda").repeat(n // 3)
        assert torch.equal(out[3].float().nan_to_num(5.0, 1.0, -1.0), want.nan_to_num(5.0, 1.0, -1.0))
        rest = torch.cat((out[:3], out[4:]))
        assert bool(rest.isfinite().all())


def test_two_streams_at_once_and_one_operand_twice():
    """Calls in flight together, each with a workspace of its own; A and B the same memory."""
    n, k = 520, 4096
    planes = [(operand(n, k, f, 9), f) for f in (E4, E2)]
    alone = []
    for a, f in planes:
        out = torch.empty((n, n), device="cuda")
        call(a, a, f, f, out)
        alone.append(out)
    torch.cuda.synchronize()
    check(alone[0], reference(*[values(*planes[0][0], E4)] * 2), k, E4, E4, False, "A A^T")
    streams, outs = [torch.cuda.Stream() for _ in planes], [torch.empty((n, n), device="cuda") for _ in planes]
    works = [torch.empty(fq.fq_gemm_mx_workspace(fq.gemm_mx_desc(n, n, k, f, f, fq.FQ_IN_F32)) or 16, dtype=torch.uint8,
                         device="cuda") for _, f in planes]
    torch.cuda.synchronize()
    for _ in range(5):
        for (a, f), s, out, ws in zip(planes, streams, outs, works):
            call(a, a, f, f, out, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, alone))


# ---------------------------------------------------------------- far offsets
def test_long_rows():
    """k = 2^22, 4.4 GB of A and then of B; zeros but for the first and last blocks."""
    k, tail = 1 << 22, 256
    for m, n, fa, fb, bf16 in ((1056, 64, E4, E4, True), (64, 1056, E4, E4, False), (2100, 70, E2, E2, True), (3, 1040, E2, E4, True)):
        print(m, n, flush=True)

        def far(rows, fmt, seed):
            x, s = operand(rows, 2 * tail, fmt, seed)
            w = x.shape[1] // 2
            data = torch.zeros((rows, k * B.BITS[fmt] // 8), dtype=torch.uint8, device="cuda")
            scale = torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda")
            data[:, :w], data[:, -w:] = x[:, :w], x[:, w:]
            scale[:, :tail // 32], scale[:, -tail // 32:] = s[:, :tail // 32], s[:, tail // 32:]
            return (data, scale), values(x, s, fmt)

        (a, va), (b, vb) = far(m, fa, 1), far(n, fb, 2)
        out = torch.empty((m, n), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        call(a, b, fa, fb, out)
        torch.cuda.synchronize()
        check(out, reference(va, vb), 2 * tail, fa, fb, bf16, f"{m}x{n}x{k}")
        del a, b


@pytest.mark.parametrize("fa,fb,bf16", [(E4, E4, True), (E2, E2, False)])
def test_large_output(fa, fb, bf16):
    """67000 x 33000 (beyond 2^31 elements, 4.4 and 8.8 GB): every row and column at the ends, and one inside."""
    m, n, k = 67000, 33000, 160
    a, b = operand(m, k, fa, 1), operand(n, k, fb, 2)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    call(a, b, fa, fb, out)
    torch.cuda.synchronize()
    va, vb = values(*a, fa), values(*b, fb)
    for rows, cols in ((slice(0, 300), slice(0, n)), (slice(m - 300, m), slice(0, n)), (slice(0, m), slice(n - 300, n)),
                       (slice(65500, 65700), slice(0, n))):
        check(out[rows, cols], reference(va[rows], vb[cols]), k, fa, fb, bf16, f"{rows} {cols}")
    assert not bool(out.isnan().any())


def test_many_rows_of_few_columns():
    """2^25 rows, 2^30 elements of A: more workgroups than 2^16 in either direction."""
    m, n, k = (1 << 25) + 3, 24, 32
    a, b = operand(m, k, E4, 1), operand(n, k, E4, 2)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    call(a, b, E4, E4, out)
    vb = values(*b, E4)
    torch.cuda.synchronize()
    for at in (0, 1 << 24, m - 1000):
        check(out[at:at + 1000], reference(values(a[0][at:at + 1000], a[1][at:at + 1000], E4), vb), k, E4, E4, True, str(at))
    assert not bool(out.isnan().any())
