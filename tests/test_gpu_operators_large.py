"""Offsets beyond 2^31 and 2^32: operands, outputs and caches of several GiB,
checked where they end."""
import numpy as np
import pytest
import torch

import operator_util as U
from fp8_fp4_tensor_amd import fq

pytestmark = pytest.mark.gpu


def codes(rng, shape):
    return torch.from_numpy(U.random_codes(rng, shape)).cuda()


def test_product_with_a_large_output():
    """70016 x 32768 fp32 (9.2 GB): the last rows and columns equal a small product's."""
    rng = np.random.default_rng(1)
    m, n, k, edge = 70016, 32768, 128, 256
    a, b = torch.zeros((m, k), dtype=torch.uint8, device="cuda"), torch.zeros((n, k), dtype=torch.uint8, device="cuda")
    sa, sb = torch.ones((m, 1), device="cuda"), torch.ones((n // 128, 1), device="cuda")
    a[-edge:], b[-edge:] = codes(rng, (edge, k)), codes(rng, (edge, k))
    out = torch.full((m, n), 7.0, device="cuda")
    d = fq.gemm_desc(m, n, k, out_dtype=fq.FQ_IN_F32)
    fq.fq_gemm(d, fq.Plane(a, sa), fq.Plane(b, sb), out, fq.alloc_gemm_workspace(d))
    torch.cuda.synchronize()
    want, s, top = U.product(a[-edge:].cpu().numpy(), sa[-edge:].cpu().numpy(), b[-edge:].cpu().numpy(),
                             sb[-2:].cpu().numpy(), 128)
    got = out[-edge:, -edge:].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= U.product_bound(want, s, top, k, False))
    assert torch.all(out[:-edge, -1024:] == 0) and torch.all(out[-1024:, :-edge] == 0)


@pytest.mark.parametrize("m,bf16", [(520, True), (520, False), (3, True)])
def test_product_with_long_rows(m, bf16):
    """k = 2^23: rows of 8 MiB, 4.4 GB of them; only the last blocks are not zero."""
    rng = np.random.default_rng(2)
    n, k, tail = 128, 1 << 23, 256
    a, b = torch.zeros((m, k), dtype=torch.uint8, device="cuda"), torch.zeros((n, k), dtype=torch.uint8, device="cuda")
    sa, sb = torch.ones((m, k // 128), device="cuda"), torch.ones((1, k // 128), device="cuda")
    a[:, -tail:], b[:, -tail:] = codes(rng, (m, tail)), codes(rng, (n, tail))
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    d = fq.gemm_desc(m, n, k, out_dtype=fq.FQ_IN_BF16 if bf16 else fq.FQ_IN_F32)
    fq.fq_gemm(d, fq.Plane(a, sa), fq.Plane(b, sb), out, fq.alloc_gemm_workspace(d))
    torch.cuda.synchronize()
    want, s, top = U.product(a[:, -tail:].cpu().numpy(), sa[:, -2:].cpu().numpy(), b[:, -tail:].cpu().numpy(),
                             sb[:, -2:].cpu().numpy(), 128)
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= U.product_bound(want, s, top, tail, bf16))


@pytest.mark.parametrize("q_len", [1, 700])
def test_cache_beyond_four_gib(q_len):
    """A sequence on the last pages of a 4.9 GB key cache equals the same one on a small cache's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    heads, q_heads, dim, page, pages, n = 8, 32, 128, 64, 75000, 900
    used = -(-n // page)

    def cache(count):
        c = fq.alloc_kv_cache(fq.FQ_E4M3, count, heads, dim, page, page)
        for t in (c.k, c.v):
            t[-used:] = 0x7F  # NaN codes wherever nothing is stored
        return c

    big, small = cache(pages), cache(used)
    assert big.k.numel() > 1 << 32
    rows = lambda m, h: torch.randn((m, h, dim), generator=g, device="cuda").to(torch.bfloat16)
    k, v, q = rows(n, heads), rows(n, heads), rows(q_len, q_heads)
    outs = []
    for c, last in ((big, pages), (small, used)):
        table = torch.arange(last - used, last, dtype=torch.int32, device="cuda")[None].contiguous()
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        fq.fq_kv_append(c, fq.KvBatch(table, lens, None, n, n), k, v)
        b, d = fq.KvBatch(table, lens, None, q_len, q_len), fq.attention_desc(q_heads)
        out, lse = torch.empty_like(q), torch.empty((q_len, q_heads), device="cuda")
        fq.fq_attention(c, b, d, q, out, lse, fq.alloc_attention_workspace(c, b, d))
        torch.cuda.synchronize()
        outs.append((out, lse))
    assert torch.equal(big.k[-used:], small.k) and torch.equal(big.v[-used:], small.v)
    assert torch.equal(big.k_scale[-used:], small.k_scale) and torch.equal(big.v_scale[-used:], small.v_scale)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.isfinite(outs[0][0].float()).all()
