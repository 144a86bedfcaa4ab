"""Every kernel of the operators on 8-bit data is reached by the shapes that
the GPU tests run (on the host: the launch rules alone)."""
import pytest

import operator_plans as P
import test_gpu_kv as K
import test_gpu_kv_edges as E


@pytest.mark.parametrize("tile,split,b_rows,bf16,shape", P.GEMM)
def test_product_takes_its_kernel(tile, split, b_rows, bf16, shape):
    got, splits, main = P.gemm_plan(*shape, bf16)
    assert (got, splits > 1, main) == (tile, split, 0)
    assert b_rows == 1 or shape[1] % 128 == 0


@pytest.mark.parametrize("tile,split,b_rows,bf16,shape", P.GEMM_REST)
def test_product_with_a_rest_takes_its_kernels(tile, split, b_rows, bf16, shape):
    got, splits, main = P.gemm_plan(*shape, bf16)
    assert (got, splits > 1) == (tile, split) and main >= 256 and main % 256 == 0
    assert b_rows == 1 or shape[1] % 128 == 0


def test_products_reach_every_kernel():
    tiles = ["few", (256, 256), (128, 128), (64, 128), (64, 64), (32, 64)]
    want = {(t, s, b, f) for t in tiles for s in (False, True) for b in (1, 128) for f in (False, True)
            if not (t == "few" and s)}
    assert {x[:4] for x in P.GEMM} == want
    # the rows behind whole rounds: every tile, whole and (but for 256x256) in shares, both ways of scaling and both results
    assert {x[:2] for x in P.GEMM_REST} == {(t, s) for t in tiles[1:] for s in (False, True)} - {((256, 256), False)}
    assert {x[2:4] for x in P.GEMM_REST} == {(b, f) for b in (1, 128) for f in (False, True)}
    # the weight gradient's: fp32, 1x128 scales, the rest on the largest tiles in shares
    assert ((256, 256), True, 1, False) in {x[:4] for x in P.GEMM_REST}


def test_attention_takes_its_kernels():
    for name, (heads, q_heads, dim, lens, counts) in E.KERNELS.items():
        kernel, splits = P.attention_plan(heads, q_heads, dim, lens, counts)
        assert kernel.startswith(name[:3] if name.startswith("few") else "many"), name
        assert name.split("-")[1] == str(dim) and (splits > 1) == name.endswith("split"), name
    for name, (heads, q_heads, dim, lens, counts, window, cap, page, fmt) in E.MANY.items():
        assert P.attention_plan(heads, q_heads, dim, lens, counts, window, page=page) == ("many", 1), name
    for name, (heads, q_heads, dim, n, count, pages) in E.FAR.items():
        kernel, splits = P.attention_plan(heads, q_heads, dim, [n], [count])
        assert kernel.startswith(name.split("-")[0]) and (splits > 1) == name.endswith("split"), name


def test_attention_reaches_every_kernel():
    """Head dims, formats, waves of a workgroup and splits: all that the launcher has."""
    seen = set()
    for fmt, heads, q_heads, dim, page, block, lens, counts, window, cap in K.CASES:
        kernel, splits = P.attention_plan(heads, q_heads, dim, lens, counts, window, page=page)
        seen.add((dim, fmt, kernel, splits > 1))
    for heads, q_heads, dim, lens, counts, window, cap, page, fmt in E.MANY.values():
        kernel, splits = P.attention_plan(heads, q_heads, dim, lens, counts, window, page=page)
        seen.add((dim, fmt, kernel, splits > 1))
    for fmt, heads, q_heads, dim, lens, counts in E.FEW.values():
        kernel, splits = P.attention_plan(heads, q_heads, dim, lens, counts)
        seen.add((dim, fmt, kernel, splits > 1))
    want = set()
    for dim in (64, 128, 256):
        for fmt in (0, 1):
            want |= {(dim, fmt, "many", False), (dim, fmt, "few-4", False), (dim, fmt, "few-4", True)}
            if dim <= 128:
                want.add((dim, fmt, "few-8", False))
    assert seen == want, (want - seen, seen - want)
