"""The 8-bit cache's operators where their ranges end: batches of very unequal
sequences, bounds far above what they bound, extreme caps, scales and values."""
import numpy as np
import pytest
import torch

import operator_util as U
import test_gpu_kv as K
from fp8_fp4_tensor_amd import fq

pytestmark = pytest.mark.gpu


def empty_like(c: fq.KvCache) -> fq.KvCache:
    return fq.KvCache(c.fmt, c.block_tokens, *(torch.zeros_like(t) for t in (c.k, c.v, c.k_scale, c.v_scale)))


@pytest.mark.parametrize("batch,rows,heads,block", [(4096, 131072, 1, 16), (300, 5003, 3, 32), (65535, 70, 1, 128)])
def test_append_of_one_prompt_among_single_tokens(batch, rows, heads, block):
    """One call for all equals one call for the prompt and one for the single tokens. The first size has a block
    of the longest sequence for each of 4096 sequences: 4096 * 8193 workgroups of 256 threads, were all launched."""
    dim, page = 64, 256 if block < 128 else 128
    g = torch.Generator(device="cuda")
    g.manual_seed(batch)
    per = -(-rows // page)
    # the prompt's pages, then one page for each single token
    table = torch.full((batch, per), -1, dtype=torch.int32, device="cuda")
    at = batch // 3
    order = torch.randperm(per + batch - 1, generator=g, device="cuda").to(torch.int32)
    table[at] = order[:per]
    others = torch.tensor([i for i in range(batch) if i != at], device="cuda")
    table[others, 0] = order[per:]
    lens = torch.ones(batch, dtype=torch.int32, device="cuda")
    lens[at] = rows
    starts = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), lens.cumsum(0).to(torch.int32)])
    k, v = (torch.randn((rows + batch - 1, heads, dim), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    whole = empty_like(fq.alloc_kv_cache(fq.FQ_E4M3, per + batch - 1, heads, dim, page, block))
    apart = empty_like(whole)
    fq.fq_kv_append(whole, fq.KvBatch(table, lens, starts, rows + batch - 1, rows), k, v)
    torch.cuda.synchronize()
    one = fq.KvBatch(table[at:at + 1].contiguous(), lens[at:at + 1].clone(), None, rows, rows)
    fq.fq_kv_append(apart, one, k[at:at + rows], v[at:at + rows])
    rest = torch.cat([torch.arange(at, device="cuda"), torch.arange(at + rows, rows + batch - 1, device="cuda")])
    fq.fq_kv_append(apart, fq.KvBatch(table[others].contiguous(), lens[others].contiguous(), None, batch - 1, 1),
                    k[rest], v[rest])
    torch.cuda.synchronize()
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(whole, name), getattr(apart, name)), name


def test_a_loose_bound_of_rows():
    """max_q far above the rows: the same cache and the same attention."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    heads, q_heads, dim, page = 2, 4, 128, 64
    lens, counts = [70, 3, 40], [5, 3, 9]
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    sd = torch.tensor(K.starts(counts), dtype=torch.int32, device="cuda")
    k, v, q = (torch.randn((17, h, dim), generator=g, device="cuda").to(torch.bfloat16) for h in (heads, heads, q_heads))
    first, outs = empty_like(fq.alloc_kv_cache(fq.FQ_E4M3, 6, heads, dim, page)), []
    first.k_scale.fill_(2.0 ** -8)
    first.v_scale.fill_(2.0 ** -8)
    for max_q in (9, 1 << 24):
        c = empty_like(first)
        c.k_scale.copy_(first.k_scale)
        c.v_scale.copy_(first.v_scale)
        b, d = fq.KvBatch(table, ld, sd, 17, max_q), fq.attention_desc(q_heads)
        fq.fq_kv_append(c, b, k, v)
        out, lse = torch.empty_like(q), torch.empty((17, q_heads), device="cuda")
        fq.fq_attention(c, b, d, q, out, lse, fq.alloc_attention_workspace(c, b, d))
        torch.cuda.synchronize()
        outs.append((c.k, c.v, c.k_scale, c.v_scale, out, lse))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.isfinite(outs[0][4].float()).all()


# ---------------------------------------------------------------- the cap
# batch shapes that take each kernel: single tokens, whole and split; chunks of every head size
KERNELS = {
    "few-64": (1, 8, 64, [300, 41], [1, 1]), "few-128": (1, 4, 128, [300, 70], [1, 1]),
    "few-128-split": (1, 4, 128, [2100, 70], [1, 1]), "few-256-split": (2, 4, 256, [1100], [3]),
    "many-64": (32, 64, 64, [150, 128, 140, 200, 129, 300], [128] * 6), "many-128": (16, 64, 128, [520, 130], [515, 130]),
    "many-256": (16, 32, 256, [300, 20], [300, 20]),
}


def capped_row(q, k, v, see, scale, cap):
    """attention_row of operator_util with a cap's error relative to the score. tanh has a slope of at most 1, so
    a score's own error does not grow. Below half the cap the result is the score times a polynomial: four fused
    operations near 1, its fit (2^-26) and two products, under 4 units. Above it c2 (1 - 2 / (e + 1)): at most 2 c2
    times the reciprocal's unit, c2 each for the exponential's unit, the sum and the last rounding, and y's two
    roundings times y times tanh's slope, below c2 / 2 each: 6 units of c2, where c2 is at most 2.17 scores."""
    dim = q.shape[0]
    k, v = k[see], v[see]
    s = k @ q * scale
    eps = (dim + 4) * U.ULP32 * (np.abs(k) @ np.abs(q)).max() * abs(scale)
    s = cap * np.tanh(s / cap)
    eps += 14 * U.ULP32 * np.abs(s).max()
    eps += 2 * 1.5 * np.abs(s).max() * 2 * U.ULP32 + 4 * U.ULP32
    top = s.max()
    p = np.exp(s - top)
    z = p.sum()
    o, w, lse = p @ v / z, p @ np.abs(v) / z, top + np.log(z)
    sums = (int(see.sum()) / 16 + 64) * U.ULP32
    bound = (U.HALF_BF16 + 2 * eps + 2 * sums) * w
    return o, lse, bound + U.HALF_BF16 * (np.abs(o) + bound) + 1e-30, eps + sums + 4 * U.ULP32 * (abs(lse) + abs(top) + 1.0)


@pytest.mark.parametrize("cap", [1e-40, 1e-3, 2.0, 12.0, 1e3, 1e4, 1e6, 1e9, 1e20, 3e38])
@pytest.mark.parametrize("kernel", KERNELS)
def test_caps_of_any_size(kernel, cap):
    """From caps that leave nothing of the scores to caps that do nothing, with scores on both sides of half a cap."""
    heads, q_heads, dim, lens, counts = KERNELS[kernel]
    rng = np.random.default_rng(sorted(KERNELS).index(kernel))
    page, group = 64, q_heads // heads
    pages = sum(-(-n // page) for n in lens) + 2
    table = K.tables(rng, lens, page, pages)
    plain = K.filled(rng, 0, heads, dim, page, 64, lens, table, pages, spread=3.0)
    cap = float(np.float32(cap))
    q, out, lse = K.attend(plain, table, lens, counts, q_heads, softcap=cap, rng=rng)
    qs = K.starts(counts)
    qd, od, ld = q.double().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = [(i, j) for i in range(len(lens)) for j in range(0, counts[i], 97)]
    for i, j in rows:
        pos = lens[i] - counts[i] + j
        for h in range(0, heads, max(1, heads // 2)):
            k, v, there = plain.values(table[i], lens[i], h)
            see = there & (np.arange(lens[i]) <= pos)
            for u in (h * group, h * group + group - 1):
                o, z, eo, ez = capped_row(qd[qs[i] + j, u], k, v, see, 1.0 / np.sqrt(dim), cap)
                got, gz = od[qs[i] + j, u], ld[qs[i] + j, u]
                assert np.all(np.abs(got - o) <= eo), (i, j, u, (np.abs(got - o) / eo).max())
                assert abs(gz - z) <= ez, (i, j, u, gz, z, ez)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("zero_scales", [True, False], ids=["zero-scales", "tiny-scale"])
def test_large_queries_meet_tiny_factors(kernel, zero_scales):
    """Products near 1e33 times a factor that makes ordinary scores of them, or zeros: the factor is not held up."""
    heads, q_heads, dim, lens, counts = KERNELS[kernel]
    rng = np.random.default_rng(80)
    page, group = 64, q_heads // heads
    pages = sum(-(-n // page) for n in lens) + 2
    table = K.tables(rng, lens, page, pages)
    plain = K.filled(rng, 0, heads, dim, page, 32, lens, table, pages)
    q = K.bf16(rng, (sum(counts), q_heads, dim), 2.0 ** 100)
    scale = 2.0 ** -100 / np.sqrt(dim)
    if zero_scales:
        plain.ks[np.isfinite(plain.ks)] = 0.0
        scale = 1.0
    scale = float(np.float32(scale))
    q, out, lse = K.attend(plain, table, lens, counts, q_heads, scale=scale, q=q)
    K.check_attention(plain, table, lens, counts, q_heads, q, out, lse, scale=scale,
                      every=(61 if heads > 8 else 1))


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_query_that_is_no_number(kernel):
    """Its row says so, in out and in lse (-inf would mean a row that sees nothing); the other rows are as without it."""
    heads, q_heads, dim, lens, counts = KERNELS[kernel]
    rng = np.random.default_rng(81)
    page = 64
    pages = sum(-(-n // page) for n in lens) + 2
    table = K.tables(rng, lens, page, pages)
    plain = K.filled(rng, 0, heads, dim, page, 64, lens, table, pages)
    q, out, lse = K.attend(plain, table, lens, counts, q_heads, rng=rng)
    bad = q.clone()
    at = [(0, 0), (sum(counts) - 1, q_heads - 1), (sum(counts) // 2, q_heads // 2)]
    for (r, h), v in zip(at, (float("nan"), float("nan"), float("inf"))):
        bad[r, h, 5] = v
    _, got, gz = K.attend(plain, table, lens, counts, q_heads, q=bad)
    hit = torch.zeros((sum(counts), q_heads), dtype=torch.bool, device="cuda")
    for r, h in at:
        hit[r, h] = True
    assert torch.isnan(got[hit]).all() and torch.isnan(gz[hit]).all()
    assert torch.equal(got[~hit], out[~hit]) and torch.equal(gz[~hit], lse[~hit])


@pytest.mark.parametrize("dim,n,q_heads", [(128, 2700, 5), (64, 4700, 3), (256, 3100, 7)])
def test_odd_numbers_of_partial_results(dim, n, q_heads):
    """One row of an odd number of heads over an odd number of splits: accumulators are moved 16 bytes at a time,
    wherever the maxima and sums beside them end. Nothing is written outside the reported workspace."""
    rng = np.random.default_rng(82)
    page = 64
    pages = -(-n // page) + 2
    table = K.tables(rng, [n], page, pages)
    plain = K.filled(rng, 0, 1, dim, page, 64, [n], table, pages)
    dev, b, d = K.to_device(plain), K.batch_of(table, [n], [1]), fq.attention_desc(q_heads)
    size = fq.fq_attention_workspace(dev, b, d)
    splits = size // (q_heads * (dim + 2) * 4)
    assert size == splits * q_heads * (dim + 2) * 4 and (splits * q_heads) % 2 == 1 and splits > 1
    q = K.bf16(rng, (1, q_heads, dim)).cuda()
    pad = 4096
    ws = torch.full((size + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((1, q_heads), device="cuda")
    fq.fq_attention(dev, b, d, q, out, lse, ws[pad:pad + size])
    torch.cuda.synchronize()
    K.check_attention(plain, table, [n], [1], q_heads, q.cpu(), out, lse)
    assert bool((ws[:pad] == 0xA5).all()) and bool((ws[pad + size:] == 0xA5).all())
    # the accumulators are what the workspace begins with: finite 16-byte groups, then the pairs
    acc = ws[pad:pad + splits * q_heads * dim * 4].view(torch.float32)
    pairs = ws[pad + acc.numel() * 4:pad + size].view(torch.float32).view(q_heads, splits, 2)
    assert torch.isfinite(acc).all() and bool((pairs[..., 1] > 0).all())
    top = pairs[..., 0].amax(1, keepdim=True)
    z = (pairs[..., 1] * torch.exp2(pairs[..., 0] - top)).sum(1)
    assert torch.allclose(lse[0], (top[:, 0] + torch.log2(z)) * float(np.log(2.0)), rtol=0, atol=1e-4)


@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_writes_only_its_outputs(kernel):
    """Guards around out and lse stay as they were, with rows that do not fill a tile."""
    heads, q_heads, dim, lens, counts = KERNELS[kernel]
    rng = np.random.default_rng(83)
    page, n, pad = 64, sum(counts), 4096
    pages = sum(-(-x // page) for x in lens) + 2
    table = K.tables(rng, lens, page, pages)
    plain = K.filled(rng, 0, heads, dim, page, 64, lens, table, pages)
    dev, b, d = K.to_device(plain), K.batch_of(table, lens, counts), fq.attention_desc(q_heads)
    q = K.bf16(rng, (n, q_heads, dim)).cuda()
    out = torch.full((n * q_heads * dim + 2 * pad,), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n * q_heads + 2 * pad,), 7.0, device="cuda")
    o, z = out[pad:-pad].view(n, q_heads, dim), lse[pad:-pad].view(n, q_heads)
    o.fill_(float("nan"))
    z.fill_(float("nan"))
    fq.fq_attention(dev, b, d, q, o, z, fq.alloc_attention_workspace(dev, b, d))
    torch.cuda.synchronize()
    assert torch.isfinite(o.float()).all() and torch.isfinite(z).all()
    for t in (out, lse):
        assert bool((t[:pad] == 7.0).all()) and bool((t[-pad:] == 7.0).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_sequences_that_share_a_prefix(kernel):
    """The same pages in several rows of the table: the same results as of copies of them."""
    heads, q_heads, dim, lens, counts = KERNELS[kernel]
    rng = np.random.default_rng(84)
    page, batch = 64, max(2, len(lens))
    n = max(lens)
    lens, counts = [n - 3 * i for i in range(batch)], [min(max(counts), n - 3 * i) for i in range(batch)]
    need = -(-n // page)
    one = rng.permutation(need).astype(np.int32)
    plain = K.filled(rng, 0, heads, dim, page, 64, [need * page], one[None], need)
    q = K.bf16(rng, (sum(counts), q_heads, dim))
    shared = np.repeat(one[None], batch, 0)
    _, out, lse = K.attend(plain, shared, lens, counts, q_heads, q=q)
    apart = U.PlainCache(0, need * batch, heads, dim, page, 64, rng)
    for name in ("k", "v", "ks", "vs"):
        getattr(apart, name)[...] = np.concatenate([getattr(plain, name)] * batch)
    _, got, gz = K.attend(apart, shared + need * np.arange(batch, dtype=np.int32)[:, None], lens, counts, q_heads, q=q)
    assert torch.equal(got, out) and torch.equal(gz, lse) and torch.isfinite(out.float()).all()


# ---------------------------------------------------------------- every kernel
# heads, q_heads, dim, lens, counts, window, cap, page, format: calls that take the kernel for many rows
MANY = {
    "64-scales": (32, 64, 64, [150, 128, 140, 200, 129, 300], [128] * 6, 0, 0.0, 64, 0),
    "64-e5m2-window": (32, 96, 64, [700, 400, 333, 85, 120, 90], [85, 80, 85, 85, 0, 84], 90, 0.0, 16, 1),
    "64-cap": (32, 64, 64, [200] * 6, [128, 128, 127, 128, 1, 128], 0, 5.0, 256, 0),
    "128-e5m2": (16, 64, 128, [530, 300, 90], [511, 300, 0], 0, 0.0, 16, 1),
    "128-window-cap": (16, 64, 128, [700, 520, 130, 64], [600, 513, 130, 1], 130, 9.0, 128, 0),
    "256": (16, 32, 256, [300, 420, 20], [300, 257, 20], 77, 12.0, 32, 0),
    "256-e5m2": (16, 48, 256, [300, 211], [300, 200], 0, 0.0, 256, 1),
}
# format, heads, q_heads, dim, lens, counts: calls that take the kernel for few rows, whole on four and eight waves and split
FEW = {f"{name}-{dim}-{'e5m2' if fmt else 'e4m3'}": (fmt, heads, heads * group, dim, lens, counts)
       for dim in (64, 128, 256) for fmt in (0, 1)
       for name, heads, group, lens, counts in (
           ("whole", 16, 5, [70 + i for i in range(33)], [1] * 33), ("one", 2, 3, [900, 77], [2, 5]),
           ("split", 2, 4, [2500, 1030, 300], [1, 3, 0]))}


@pytest.mark.parametrize("name", MANY)
def test_many_rows(name):
    """Scales that are no powers of two, zeros among them, in every form of the kernel for many rows."""
    heads, q_heads, dim, lens, counts, window, cap, page, fmt = MANY[name]
    rng = np.random.default_rng(sorted(MANY).index(name))
    pages = sum(-(-n // page) for n in lens) + 2
    table = K.tables(rng, lens, page, pages)
    plain = K.filled(rng, fmt, heads, dim, page, min(page, 32), lens, table, pages, spread=2.0)
    for scales in (plain.ks, plain.vs):
        scales *= rng.uniform(0.4, 1.7, size=scales.shape).astype(np.float32)
        scales[rng.random(scales.shape) < 0.1] = 0.0
    q, out, lse = K.attend(plain, table, lens, counts, q_heads, window, cap, rng=rng)
    K.check_attention(plain, table, lens, counts, q_heads, q, out, lse, window, cap, every=67)


@pytest.mark.parametrize("name", FEW)
def test_few_rows(name):
    fmt, heads, q_heads, dim, lens, counts = FEW[name]
    rng = np.random.default_rng(100 + sorted(FEW).index(name))
    page = 64
    pages = sum(-(-n // page) for n in lens) + 2
    table = K.tables(rng, lens, page, pages)
    plain = K.filled(rng, fmt, heads, dim, page, 32, lens, table, pages, spread=2.0)
    q, out, lse = K.attend(plain, table, lens, counts, q_heads, rng=rng)
    K.check_attention(plain, table, lens, counts, q_heads, q, out, lse)


# heads, q_heads, dim, tokens, rows, pages of 64 tokens: caches whose keys pass 2^32 bytes
FAR = {"many-64": (8, 32, 64, 1600, 1500, 150000), "many-128": (8, 32, 128, 1200, 1000, 75000),
       "many-256": (8, 32, 256, 800, 700, 37500), "few-64-split": (8, 32, 64, 2000, 1, 150000),
       "few-256-split": (8, 32, 256, 2000, 1, 37500)}


@pytest.mark.parametrize("name", FAR)
def test_far_pages(name):
    """A sequence on the last pages of a cache of 4.9 GB of keys equals the same one on a small cache's."""
    heads, q_heads, dim, n, count, pages = FAR[name]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    page = 64
    used = -(-n // page)
    big, small = (fq.alloc_kv_cache(fq.FQ_E4M3, p, heads, dim, page, page) for p in (pages, used))
    assert big.k.numel() > 1 << 32
    for c in (big, small):
        c.k[-used:], c.v[-used:] = 0x7F, 0x7F  # NaN codes wherever nothing is stored
    k, v, q = (torch.randn((r, h, dim), generator=g, device="cuda").to(torch.bfloat16)
               for r, h in ((n, heads), (n, heads), (count, q_heads)))
    outs = []
    for c, last in ((big, pages), (small, used)):
        table = torch.arange(last - used, last, dtype=torch.int32, device="cuda")[None].contiguous()
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        fq.fq_kv_append(c, fq.KvBatch(table, lens, None, n, n), k, v)
        b, d = fq.KvBatch(table, lens, None, count, count), fq.attention_desc(q_heads)
        out, lse = torch.empty_like(q), torch.empty((count, q_heads), device="cuda")
        fq.fq_attention(c, b, d, q, out, lse, fq.alloc_attention_workspace(c, b, d))
        torch.cuda.synchronize()
        outs.append((out, lse))
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(big, name)[-used:], getattr(small, name)), name
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.isfinite(outs[0][0].float()).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("fmt", [fq.FQ_E4M3, fq.FQ_E5M2], ids=["e4m3", "e5m2"])
def test_append_beside_scales_that_are_no_powers_of_two(fmt, dtype):
    """A block that something else began keeps its larger scale: new codes are x / s, also where x / s lies half way
    between two codes (x times the rounded inverse then falls on either side)."""
    rng = np.random.default_rng(85)
    heads, dim, page, block = 2, 64, 16, 16
    odd = [3.0, 5.0, 3.0 * 2.0 ** -9, 7.0 * 2.0 ** -4, 5.0 * 2.0 ** 20, 3.0 * 2.0 ** -100]
    plain = U.PlainCache(fmt, len(odd), heads, dim, page, block, rng)
    man = 3 if fmt == fq.FQ_E4M3 else 2
    # half way between neighbours, over several binades and both signs
    ties = np.array([(1 + (2 * i + 1) / 2.0 ** (man + 1)) * 2.0 ** e for e in range(-5, 6) for i in range(2 ** man)])
    old, new = 5, 9
    x = np.zeros((len(odd), new, heads, dim))
    for i, s in enumerate(odd):
        plain.k[i, :, :old] = U.encode(rng.standard_normal((heads, old, dim)), fmt)
        plain.v[i, :, :, :old] = U.encode(rng.standard_normal((heads, dim, old)), fmt)
        plain.ks[i], plain.vs[i] = s, s
        x[i] = rng.choice(ties, size=(new, heads, dim)) * rng.choice([-1.0, 1.0], size=(new, heads, dim)) * s
    t = torch.from_numpy(x.reshape(-1, heads, dim)).to(dtype)
    assert np.array_equal(t.double().numpy(), x.reshape(-1, heads, dim))  # exact in either type
    dev = K.to_device(plain)
    table = np.arange(len(odd), dtype=np.int32)[:, None]
    K.append(dev, plain, table, [old + new] * len(odd), [new] * len(odd), t, -t)
    K.same(dev, plain, "beside older scales")
