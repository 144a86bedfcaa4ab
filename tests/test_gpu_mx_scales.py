"""fq_gemm_mx over the whole range of E8M0 codes: a side whose values leave fp32's
range while the products do not, scales that are no numbers, the smallest scale,
and large terms that cancel."""
import pytest
import torch

import mx_plans as P
from fp8_fp4_tensor_amd import fq
from test_gpu_mx_edges import E2, E4, E5, call, check, operand, reference, values

pytestmark = pytest.mark.gpu

ONE = {E4: 0x38, E5: 0x3C, E2: 0x22}  # 1.0 (twice, packed)
WIDENED = [p for p in P.PLANS if p[0] == "widened"]
PAIRS = [(E4, E4), (E5, E4), (E5, E5), (E4, E2), (E2, E5)]
# shapes that take the kernel for few rows and each tile, with bf16 results of 8-bit and of 4-bit operands and with fp32
# results; between them scales as planes have them and laid out, whole and in shares of k
KERNELS = {kind: [next(p[5] for p in P.PLANS if p[0] == kind and p[1] == tile and p[5][2] >= 256)
                  for tile in (None, P.T6464, P.T64)] + [s for s in extra]
           for kind, extra in (("8", [(71, 2802, 7808), (131, 2723, 12288)]), ("4", [(73, 2782, 12032), (8223, 75, 8544)]),
                               ("mixed", [(71, 2802, 7808), (8193, 70, 6432)]),
                               ("widened", [(67, 2818, 5760), (66, 2730, 5600), (5448, 131, 10880)]))}
EVERY = [(kind, shape) for kind in KERNELS for shape in KERNELS[kind]]
name = lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v)


def result(m, n, bf16):
    return torch.full((m, n), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")


def test_shapes_take_their_kernels():
    for kind, shapes in KERNELS.items():
        pairs, bf16 = P.KINDS[kind]
        seen = {P.plan(*s, *pairs[0], bf16)[0] for s in shapes}
        assert seen == {None, P.T6464, P.T64, P.T128, P.T256}, (kind, seen)


@pytest.mark.parametrize("kind,tile,split,rest,arranged,shape", WIDENED, ids=name)
def test_values_beyond_fp32_on_one_side(kind, tile, split, rest, arranged, shape):
    """Rows of A (columns of B) with blocks at 2^123, beyond fp32 times the largest codes, against blocks at 2^-107: the
    products are moderate, and so is the result, also where fp32 results widen their operands."""
    m, n, k = shape
    for fa, fb in PAIRS:
        for accumulate in (False, True):
            a, b = operand(m, k, fa, 3 * m + k), operand(n, k, fb, 5 * n + k)
            a[1][::3, 0], b[1][:, 0] = 250, 20
            if k > 32:
                b[1][::2, -1], a[1][:, -1] = 250, 20
            out = result(m, n, False)
            if accumulate:
                out.zero_()
            print(shape, fa, fb, accumulate, flush=True)
            call(a, b, fa, fb, out, accumulate)
            torch.cuda.synchronize()
            check(out, reference(values(*a, fa), values(*b, fb)), k, fa, fb, False, f"{fa} {fb} {shape}")


@pytest.mark.parametrize("kind,shape", [e for e in EVERY if e[0] != "widened"], ids=name)
def test_far_scales_of_bf16_results(kind, shape):
    """The same with bf16 results, whose instruction takes the scales as they are."""
    m, n, k = shape
    for fa, fb in P.KINDS[kind][0]:
        a, b = operand(m, k, fa, 11), operand(n, k, fb, 12)
        a[1][::3, 0], b[1][:, 0] = 250, 20
        b[1][::2, -1], a[1][:, -1] = 250, 20
        out = result(m, n, True)
        call(a, b, fa, fb, out)
        torch.cuda.synchronize()
        check(out, reference(values(*a, fa), values(*b, fb)), k, fa, fb, True, f"{fa} {fb} {shape}")


@pytest.mark.parametrize("shape", [(5, 131, 416), (33, 66, 320), (563, 65, 4032), (67, 2818, 5760), (16440, 387, 128)], ids=name)
def test_other_rows_and_columns_stay_as_they_are(shape):
    """Rows of A and columns of B whose values are beyond fp32's range change no bit of the others, sums of which lie in the
    same instruction's tile; and each call gives the same."""
    m, n, k = shape
    for fa, fb in PAIRS:
        a, b = operand(m, k, fa, 7), operand(n, k, fb, 8)
        b[1][:, 0], a[1][:, 2] = 20, 20
        plain, out, again = (result(m, n, False) for _ in range(3))
        call(a, b, fa, fb, plain)
        a[1][1::4, 0], b[1][::3, 2] = 250, 250
        call(a, b, fa, fb, out)
        call(a, b, fa, fb, again)
        torch.cuda.synchronize()
        same = torch.ones((m, n), dtype=torch.bool, device="cuda")
        same[1::4], same[:, ::3] = False, False
        assert torch.equal(out[same], plain[same]) and torch.equal(out, again)
        check(out, reference(values(*a, fa), values(*b, fb)), k, fa, fb, False, f"{fa} {fb} {shape}")


def test_the_largest_scales():
    """Each code from 230 to 254, on either side, with bf16 and fp32 results."""
    m, n, k = 25, 40, 416
    for fa, fb in PAIRS + [(E2, E2)]:
        for bf16 in (True, False):
            a, b = operand(m, k, fa, 1), operand(n, k, fb, 2)
            a[1][:, 5], b[1][:, 5] = torch.arange(230, 255, dtype=torch.uint8, device="cuda"), 20
            b[1][:25, 9], a[1][:, 9] = torch.arange(230, 255, dtype=torch.uint8, device="cuda"), 20
            out = result(m, n, bf16)
            call(a, b, fa, fb, out)
            torch.cuda.synchronize()
            check(out, reference(values(*a, fa), values(*b, fb)), k, fa, fb, bf16, f"{fa} {fb} {bf16}")


def test_results_beyond_fp32_are_infinite():
    """Where the product itself is, the result is infinite, and only there."""
    k = 256
    for m, n in ((4, 32), (40, 64)):
        for fa, fb in PAIRS + [(E2, E2)]:
            for bf16 in (True, False):
                one = lambda r, f: (torch.full((r, k * (4 if f == E2 else 8) // 8), ONE[f], dtype=torch.uint8, device="cuda"),
                                    torch.full((r, k // 32), 127, dtype=torch.uint8, device="cuda"))
                a, b = one(m, fa), one(n, fb)
                a[1][1, 3], b[1][:, 3] = 250, 140  # 32 * 2^123 * 2^13 = 2^141
                b[1][2, 3] = 4                     # 32 * 2^123 * 2^-123 = 32
                out = result(m, n, bf16)
                call(a, b, fa, fb, out)
                torch.cuda.synchronize()
                want = torch.full((m, n), 224.0 + 32 * 2.0 ** 13, dtype=torch.float64, device="cuda")
                want[:, 2] = 224.0                 # and 2^-118
                want[1] = float("inf")
                want[1, 2] = 256.0
                assert torch.equal(out, want.to(out.dtype)), (m, n, fa, fb, bf16)


@pytest.mark.parametrize("kind,shape", EVERY, ids=name)
def test_scales_that_are_no_numbers(kind, shape):
    """Code 255 gives NaN whatever stands beside it: products of one sign, and a block of zeros."""
    m, n, k = shape
    pairs, bf16 = P.KINDS[kind]
    for fa, fb in pairs:
        one = lambda r, f: (torch.full((r, k * (4 if f == E2 else 8) // 8), ONE[f], dtype=torch.uint8, device="cuda"),
                            torch.full((r, k // 32), 127, dtype=torch.uint8, device="cuda"))
        a, b = one(m, fa), one(n, fb)
        wa, wb = a[0].shape[1] * 32 // k, b[0].shape[1] * 32 // k
        a[1][0, -1] = 255
        a[1][m - 1, 2], a[0][m - 1, 2 * wa:3 * wa] = 255, 0
        b[1][n - 1, 0] = 255
        rows, cols = {0, m - 1}, {n - 1}
        if n > 2:
            b[1][n // 2, 1], b[0][n // 2, wb:2 * wb] = 255, 0
            cols.add(n // 2)
        out = result(m, n, bf16)
        call(a, b, fa, fb, out)
        torch.cuda.synchronize()
        want = torch.full((m, n), float(k), device="cuda").to(out.dtype)
        want[sorted(rows)] = float("nan")
        want[:, sorted(cols)] = float("nan")
        assert torch.equal(out.isnan(), want.isnan()), (fa, fb, out.isnan().sum(), want.isnan().sum())
        assert torch.equal(out.nan_to_num(), want.nan_to_num()), (fa, fb)


@pytest.mark.parametrize("kind,shape", EVERY, ids=name)
def test_the_smallest_scale(kind, shape):
    """Code 0 is 2^-127: the only block that is not zero, against one at 2^100. Values below 2^-126 may count as zero
    in fp32 results with an 8-bit side."""
    m, n, k = shape
    pairs, bf16 = P.KINDS[kind]
    for fa, fb in pairs:
        a, b = operand(m, k, fa, m), operand(n, k, fb, n)
        at, w = k // 64, a[0].shape[1] * 32 // k
        a[0][:, :at * w], a[0][:, (at + 1) * w:] = 0, 0
        a[1][:, at], b[1][:, at] = 0, 227
        out = result(m, n, bf16)
        call(a, b, fa, fb, out)
        torch.cuda.synchronize()
        va, vb = values(*a, fa), values(*b, fb)
        c, s, top = reference(va, vb)
        # of 32 terms; what may count as zero is added to the bound
        err = (out.double() - c).abs()
        bound = 32 * 2.0 ** -23 * s
        if bf16 and not (fa == E2 and fb == E2):
            bound = bound + 32 * 2.0 ** -12 * top
        if kind == "widened":
            bound = bound + torch.where(va.abs() < 2.0 ** -126, va.abs(), 0.0) @ vb.abs().t()
        bound = bound + (2.0 ** -8 if bf16 else 2.0 ** -24) * (c.abs() + bound)
        assert bool((err <= bound).all()), (fa, fb, (err / bound).max())


@pytest.mark.parametrize("kind,shape", EVERY, ids=name)
def test_large_terms_that_cancel(kind, shape):
    """T = 448 (57344, 6) in one run of 128 and -T in the next, beside small terms: what is left is off by what the
    instruction keeps of a product beside the largest of its 128, 2^-12 of it (fp32 results, and 4 bits: by fp32's roundings)."""
    m, n, k = shape
    pairs, bf16 = P.KINDS[kind]
    for fa, fb in pairs:
        t = {E4: (0x7E, 0xFE, 448.0), E5: (0x7B, 0xFB, 57344.0), E2: (0x07, 0x0F, 6.0)}[fa]
        w = 4 if fa == E2 else 8
        for few in (True, False):
            a = (torch.zeros((m, k * w // 8), dtype=torch.uint8, device="cuda"),
                 torch.full((m, k // 32), 127, dtype=torch.uint8, device="cuda"))
            b = (torch.full((n, k * (4 if fb == E2 else 8) // 8), ONE[fb], dtype=torch.uint8, device="cuda"),
                 torch.full((n, k // 32), 127, dtype=torch.uint8, device="cuda"))
            a[0][:, 0], a[0][:, 128 * w // 8] = t[0], t[1]
            # in block 1 of the first run, one term or all 32, 2^0 to 2^-24 of T by rows
            small = slice(32 * w // 8, (33 if few else 64) * w // 8 + (few and w == 4))
            a[0][:, small] = ONE[fa] if not (few and fa == E2) else 2
            shift = torch.arange(m, device="cuda") % 25
            top = int(t[2]).bit_length() - 1
            a[1][:, 1] = (127 + top - shift).to(torch.uint8)
            terms = 1 if few else 32
            want = (terms * torch.exp2((top - shift).double()))[:, None].expand(m, n)
            out = result(m, n, bf16)
            call(a, b, fa, fb, out)
            torch.cuda.synchronize()
            narrow = bf16 and not (fa == E2 and fb == E2)
            # each of the terms is kept to 2^-12 of T; in fp32 the partial sums of at most 34 |T| take a rounding each
            bound = terms * 2.0 ** -12 * t[2] if narrow else 2 * (terms + 2) * 2.0 ** -24 * (2 * t[2] + want)
            bound = bound + (2.0 ** -8 if bf16 else 2.0 ** -24) * (want + bound)
            err = (out.double() - want).abs()
            assert bool((err <= bound).all()), (fa, fb, few, (err / bound).max())
