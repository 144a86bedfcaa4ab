"""Every kernel of the products of microscaled operands is reached by the shapes
that the GPU tests run, and what the launch rule gives is sound (on the host)."""
import random

import pytest

import mx_plans as P
from fp8_fp4_tensor_amd import fq

name = lambda s: "x".join(map(str, s))


@pytest.mark.parametrize("kind,tile,split,rest,arranged,shape", P.PLANS, ids=lambda v: name(v) if isinstance(v, tuple) else str(v))
def test_product_takes_its_kernel(kind, tile, split, rest, arranged, shape):
    pairs, bf16 = P.KINDS[kind]
    for fa, fb in pairs:
        got, splits, main, laid = P.plan(*shape, fa, fb, bf16)
        assert (got, splits > 1, main > 0, laid) == (tile, split, rest, arranged), (fa, fb)


@pytest.mark.parametrize("kind,arranged,shape", P.WALKS)
def test_workgroups_take_several_tiles(kind, arranged, shape):
    m, n, k = shape
    pairs, bf16 = P.KINDS[kind]
    for fa, fb in pairs:
        got, splits, main, laid = P.plan(*shape, fa, fb, bf16)
        rows = main or m
        assert (main or got == (256, 256)) and (main or splits == 1) and laid == arranged, (got, splits, main, laid)
        assert -(-rows // 256) * -(-n // 256) > 512


def test_every_kernel_is_reached():
    for kind in P.KINDS:
        seen = {p[1:] for p in P.PLANS if p[0] == kind}
        assert any(s[0] is None for s in seen)
        for tile in (P.T256, P.T128, P.T64, P.T6464):
            for split in (False, True):
                for arranged in (False, True):
                    assert any(s[0] == tile and s[1] == split and s[3] == arranged for s in seen), (kind, tile, split, arranged)


def test_plans_are_sound():
    """Shares have a step each, the rows ahead of a rest are whole tiles, scales whose rows are no whole words are
    laid out, and the workspace is what the plan needs."""
    rng = random.Random(5)
    edge = [1, 2, 16, 17, 255, 256, 257, 4096, 65536]
    for i in range(6000):
        m, n = (rng.choice(edge) if rng.random() < 0.3 else int(2 ** rng.uniform(0, 18)) for _ in range(2))
        k = 32 * (rng.choice([1, 3, 4, 7, 8, 9, 16]) if rng.random() < 0.3 else int(2 ** rng.uniform(0, 13)))
        fa, fb, bf16 = rng.randrange(3), rng.randrange(3), rng.random() < 0.5
        tile, splits, main, arranged = P.plan(m, n, k, fa, fb, bf16)
        assert 1 <= splits <= 16 and main % 256 == 0 and 0 <= main < m
        if tile is None:
            assert m <= 16 and (splits, main, arranged) == (1, 0, False)
        else:
            steps = -(-k // (256 if fa == fb == P.E2M1 else 128))
            assert splits == 1 or steps // splits >= 2
            assert arranged or k % 128 == 0
        words = -(-k // 128)
        want = arranged * 256 * words * (-(-m // 64) + -(-n // 64)) + (splits > 1) * 4 * splits * (m - main) * n
        assert fq.fq_gemm_mx_workspace(fq.gemm_mx_desc(m, n, k, fa, fb, fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32)) == want
