"""The 8-bit cache on the GPU: fq_kv_append bit for bit and fq_attention within
its derived bounds, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import operator_util as U
from fp8_fp4_tensor_amd import fq

pytestmark = pytest.mark.gpu


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def to_device(c: U.PlainCache) -> fq.KvCache:
    return fq.KvCache(c.fmt, c.block, cuda(c.k), cuda(c.v), cuda(c.ks), cuda(c.vs))


def tables(rng, lens, page, pages):
    """A page table with random pages; unused entries are far out of range."""
    need = [-(-n // page) if n > 0 else 0 for n in lens]
    t = np.full((len(lens), max(max(need), 1)), 0x7fffff00, np.int32)
    order = rng.permutation(pages)[:sum(need)]
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def bf16(rng, shape, std=1.0):
    return (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * std).to(torch.bfloat16)


def batch_of(table, lens, counts, max_len=0):
    qs = starts(counts)
    return fq.KvBatch(cuda(table), cuda(np.asarray(lens, np.int32)), cuda(qs), int(qs[-1]), int(max(counts)), max_len)


def same(dev: fq.KvCache, want: U.PlainCache, what):
    for name, got, ref in (("k", dev.k, want.k), ("v", dev.v, want.v), ("k_scale", dev.k_scale, want.ks),
                           ("v_scale", dev.v_scale, want.vs)):
        g, r = got.cpu().numpy(), ref
        if r.dtype == np.float32:
            g, r = g.view(np.uint32), r.view(np.uint32)
        assert np.array_equal(g, r), f"{what}: {name}: {(g != r).sum()} of {g.size} differ"


def append(dev, plain, table, lens, counts, k, v, stream=None):
    b = batch_of(table, lens, counts)
    fq.fq_kv_append(dev, b, k.cuda(), v.cuda(), stream)
    torch.cuda.synchronize()
    qs = starts(counts)
    kd, vd = k.double().numpy(), v.double().numpy()
    for i, n in enumerate(lens):
        plain.append(table[i], n, kd[qs[i]:qs[i + 1]], vd[qs[i]:qs[i + 1]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [fq.FQ_E4M3, fq.FQ_E5M2], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("heads,dim,page,block", [(1, 64, 16, 16), (2, 128, 64, 64), (3, 128, 64, 16), (1, 256, 256, 128), (2, 64, 128, 32)])
def test_append_over_several_calls(heads, dim, page, block, fmt, dtype):
    """Prompts of odd lengths, then single tokens whose magnitudes make scales grow."""
    rng = np.random.default_rng(heads * 100 + dim + page + block + fmt)
    counts = [37, 1, 130, 0]
    steps = 6
    final = [c + steps for c in counts]
    pages = sum(-(-n // page) for n in final) + 2
    table = tables(rng, final, page, pages)
    plain = U.PlainCache(fmt, pages, heads, dim, page, block, rng)
    dev = to_device(plain)

    def rows(n, std):
        x = torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32)) * std
        return x.to(dtype)

    append(dev, plain, table, counts, counts, rows(sum(counts), 1.0), rows(sum(counts), 0.1))
    same(dev, plain, "prompt")
    lens = list(counts)
    for step in range(steps):
        lens = [n + 1 for n in lens]
        one = [1] * len(lens)
        append(dev, plain, table, lens, one, rows(len(lens), 4.0 ** (step % 3)), rows(len(lens), 3.0 ** (step % 4 - 2)))
        same(dev, plain, f"token {step}")


def test_append_zero_subnormal_and_largest_values():
    rng = np.random.default_rng(3)
    heads, dim, page, block = 1, 64, 16, 16
    plain = U.PlainCache(fq.FQ_E4M3, 6, heads, dim, page, block, rng)
    dev = to_device(plain)
    x = torch.zeros((96, heads, dim), dtype=torch.float32)
    x[16:32] = torch.from_numpy(rng.standard_normal((16, heads, dim)).astype(np.float32)) * 1e-38
    x[16, 0, :8] = 2.0 ** -149
    x[32:48, 0, 0] = 3.4028234663852886e38
    x[48:64] = 448.0
    x[64:80, 0, 3] = float(np.nextafter(np.float32(448.0), np.float32(1e9)))
    x[80:96] = -0.0
    table = tables(rng, [96], page, 6)
    append(dev, plain, table, [96], [96], x, x.clone())
    same(dev, plain, "values")


def test_append_takes_a_joint_projection_and_one_row_heads():
    """Keys and values as slices of one tensor, and q_start left out."""
    rng = np.random.default_rng(4)
    heads, dim, page, block, n = 2, 128, 32, 32, 5
    plain = U.PlainCache(fq.FQ_E4M3, 20, heads, dim, page, block, rng)
    dev = to_device(plain)
    lens = [1, 33, 64, 7, 90]
    table = tables(rng, lens, page, 20)
    for i, m in enumerate(lens):  # the older tokens
        if m > 1:
            old = bf16(rng, (m - 1, heads, dim))
            append(dev, plain, table[i:i + 1], [m - 1], [m - 1], old, old)
    qkv = bf16(rng, (n, 4 * heads * dim)).cuda()
    k = qkv[:, 2 * heads * dim:3 * heads * dim].view(n, heads, dim)
    v = qkv[:, 3 * heads * dim:].view(n, heads, dim)
    b = fq.KvBatch(cuda(table), cuda(np.asarray(lens, np.int32)), None, n, 1)
    fq.fq_kv_append(dev, b, k, v)
    torch.cuda.synchronize()
    for i, m in enumerate(lens):
        plain.append(table[i], m, k[i:i + 1].double().cpu().numpy(), v[i:i + 1].double().cpu().numpy())
    same(dev, plain, "slices")


def test_append_skips_what_does_not_fit():
    """Rows at negative positions, an absent page, lengths beyond the table: nothing outside is written."""
    rng = np.random.default_rng(5)
    heads, dim, page, block = 1, 64, 16, 16
    plain = U.PlainCache(fq.FQ_E4M3, 5, heads, dim, page, block, rng)
    dev = to_device(plain)
    x = bf16(rng, (60, heads, dim))
    table = np.array([[0, 1], [2, -1], [3, 5]], np.int32)
    lens, counts = [4, 20, 32], [10, 18, 32]
    append(dev, plain, table[1:2], [2], [2], x[:2] * 0.25, x[2:4] * 0.25)  # the second sequence's older tokens
    append(dev, plain, table, lens, counts, x, x.clone())
    same(dev, plain, "negative positions and absent pages")
    append(dev, plain, table[:1], [29], [25], x[:25] * 0.5, x[25:50] * 0.5)  # the first sequence up to the slots cut to below
    b = fq.KvBatch(cuda(table[:1]), cuda(np.array([1000], np.int32)), None, 3, 3)  # cut to the table's 32 slots
    fq.fq_kv_append(dev, b, x[:3].cuda(), x[:3].cuda())
    torch.cuda.synchronize()
    plain.append(table[0], 32, x[:3].double().numpy(), x[:3].double().numpy())
    same(dev, plain, "length beyond the table")


# ---------------------------------------------------------------- attention
def filled(rng, fmt, heads, dim, page, block, lens, table, pages, spread=1.0):
    """A cache whose used slots are finite and whose other slots hold anything."""
    plain = U.PlainCache(fmt, pages, heads, dim, page, block, rng)
    for i, n in enumerate(lens):
        for t0 in range(0, n, block):
            p = table[i][t0 // page]
            if not 0 <= p < pages:
                continue
            inner, m = t0 % page, min(block, n - t0)
            for h in range(heads):
                plain.k[p, h, inner:inner + m] = U.encode(rng.standard_normal((m, dim)) * 60, fmt)
                plain.v[p, h, :, inner:inner + m] = U.encode(rng.standard_normal((dim, m)) * 60, fmt)
                plain.ks[p, h, inner // block] = np.float32(spread * rng.uniform(0.5, 2.0) / 60)
                plain.vs[p, h, inner // block] = np.float32(rng.uniform(0.5, 2.0) / 60)
    return plain


def attend(plain, table, lens, counts, q_heads, window=0, softcap=0.0, scale=0.0, rng=None, q=None, max_len=0,
           with_lse=True, stream=None):
    n = int(sum(counts))
    if q is None:
        q = bf16(rng, (n, q_heads, plain.dim))
    dev = to_device(plain)
    b = batch_of(table, lens, counts, max_len)
    d = fq.attention_desc(q_heads, scale=scale, window=window, softcap=softcap)
    qd = q.cuda()
    out = torch.full((n, q_heads, plain.dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, q_heads), float("nan"), device="cuda") if with_lse else None
    ws = fq.alloc_attention_workspace(dev, b, d)
    if ws is not None:
        ws.fill_(255)
    fq.fq_attention(dev, b, d, qd, out, lse, ws, stream)
    torch.cuda.synchronize()
    return q, out, lse


def check_attention(plain, table, lens, counts, q_heads, q, out, lse, window=0, softcap=0.0, scale=0.0, every=1):
    group = q_heads // plain.heads
    scale = scale or 1.0 / np.sqrt(plain.dim)
    qs = starts(counts)
    q, out = q.double().numpy(), out.double().cpu().numpy()
    lse = lse.double().cpu().numpy()
    worst = 0.0
    for i, n in enumerate(lens):
        for h in range(plain.heads):
            k, v, there = plain.values(table[i], max(n, 0), h)
            at = np.arange(max(n, 0))
            for j in range(0, counts[i], every):
                pos = n - counts[i] + j
                see = there & (at <= pos)
                if window:
                    see &= at > pos - window
                for u in range(h * group, (h + 1) * group):
                    o, z, eo, ez = U.attention_row(q[qs[i] + j, u], k, v, see, scale, softcap)
                    got, gz = out[qs[i] + j, u], lse[qs[i] + j, u]
                    assert np.all(np.abs(got - o) <= eo), (i, j, u, np.abs(got - o).max(), (np.abs(got - o) / (eo + 1e-300)).max())
                    assert gz == z if np.isinf(z) else abs(gz - z) <= ez, (i, j, u, gz, z, ez)


CASES = [  # fmt, heads, q_heads, dim, page, block, lens, counts, window, softcap
    (0, 1, 1, 64, 16, 16, [1, 2, 15, 16, 17], [1, 1, 1, 1, 1], 0, 0.0),
    (0, 2, 8, 128, 64, 64, [1, 63, 64, 65, 300, 0], [1, 1, 1, 1, 1, 1], 0, 0.0),
    (1, 1, 5, 128, 32, 16, [257, 511], [1, 1], 0, 0.0),
    (0, 1, 16, 256, 128, 128, [129, 1000], [1, 1], 0, 0.0),
    (0, 2, 34, 64, 64, 32, [700, 30], [1, 1], 0, 0.0),
    (1, 2, 4, 256, 256, 128, [100, 333], [1, 1], 0, 0.0),
    (0, 1, 4, 128, 64, 64, [4000, 1, 2500], [1, 1, 1], 0, 0.0),
    (0, 1, 4, 128, 64, 64, [4000, 70, 2500], [1, 1, 1], 100, 0.0),
    (0, 1, 2, 128, 64, 64, [900, 70, 20], [1, 1, 1], 1, 0.0),
    (0, 2, 4, 128, 64, 64, [300, 70], [1, 1], 0, 20.0),
    (0, 1, 3, 128, 64, 64, [70, 5, 130], [70, 5, 33], 0, 0.0),
    (0, 2, 4, 64, 16, 16, [260, 200], [131, 17], 50, 0.0),
    (1, 1, 2, 256, 64, 64, [150, 3], [64, 3], 0, 15.0),
    (0, 1, 8, 128, 128, 64, [400, 90, 0, 6], [200, 1, 0, 10], 0, 0.0),
    (0, 8, 8, 128, 64, 64, [500], [300], 0, 0.0),
    (0, 1, 1, 128, 16, 16, [2000], [257], 300, 0.0),
    # many rows (a workgroup shares the keys): ragged, windows, caps, every head size and format
    (0, 16, 64, 128, 64, 64, [700, 520, 130, 64], [600, 513, 130, 1], 0, 0.0),
    (1, 16, 64, 128, 16, 16, [530, 300], [511, 300], 100, 0.0),
    (0, 32, 64, 64, 128, 32, [700, 40, 515], [450, 33, 515], 0, 25.0),
    (1, 32, 64, 64, 32, 32, [600, 900, 0], [600, 590, 0], 65, 0.0),
    (0, 16, 32, 256, 64, 64, [300, 420, 20], [300, 257, 20], 0, 0.0),
    (1, 32, 32, 256, 256, 128, [600, 140], [511, 130], 33, 30.0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(case):
    fmt, heads, q_heads, dim, page, block, lens, counts, window, softcap = case
    rng = np.random.default_rng(CASES.index(case))
    pages = sum(-(-n // page) for n in lens) + 3
    table = tables(rng, lens, page, pages)
    plain = filled(rng, fmt, heads, dim, page, block, lens, table, pages)
    q, out, lse = attend(plain, table, lens, counts, q_heads, window, softcap, rng=rng)
    check_attention(plain, table, lens, counts, q_heads, q, out, lse, window, softcap,
                    every=(67 if heads > 8 else 7) if max(counts) > 20 else 1)


def test_attention_many_rows_where_things_go_wrong():
    """The kernel for many rows: absent pages, rows before the start, NaN beyond the ends, a negative scale."""
    rng = np.random.default_rng(60)
    heads, q_heads, page = 16, 64, 64
    lens, counts = [500, 300, 0, 520], [520, 290, 300, 515]
    pages = sum(-(-n // page) for n in lens) + 3
    table = tables(rng, lens, page, pages)
    table[0, 2], table[1, 4], table[3, 0] = -7, pages, 0x7fffffff
    plain = filled(rng, 0, heads, 128, page, 64, lens, table, pages, spread=4.0)
    q, out, lse = attend(plain, table, lens, counts, q_heads, scale=-0.1, rng=rng)
    check_attention(plain, table, lens, counts, q_heads, q, out, lse, scale=-0.1, every=61)
    assert torch.all(out[:20] == 0) and torch.all(lse[810:1110] == -float("inf"))


def test_attention_large_scores_and_given_scale():
    """Scores of hundreds, where only the running maximum keeps the sums finite; a negative scale."""
    rng = np.random.default_rng(50)
    lens, counts, page = [500, 130], [1, 40], 64
    table = tables(rng, lens, page, 14)
    plain = filled(rng, 0, 1, 128, page, 64, lens, table, 14, spread=20.0)
    for scale in (0.5, -0.25):
        q, out, lse = attend(plain, table, lens, counts, 4, scale=scale, rng=rng)
        check_attention(plain, table, lens, counts, 4, q, out, lse, scale=scale, every=3)


@pytest.mark.parametrize("heads, q_heads, dim, lens, counts", [
    (1, 4, 128, [300, 70], [1, 1]), (16, 64, 128, [520, 130], [515, 130]), (32, 64, 64, [600, 40], [600, 33]),
    (16, 32, 256, [300, 20], [300, 20])])
def test_attention_scales_of_any_size(heads, q_heads, dim, lens, counts):
    """A cache that something else wrote: scales that are no powers of two, and zeros."""
    rng = np.random.default_rng(61)
    page = 64
    pages = sum(-(-n // page) for n in lens) + 2
    table = tables(rng, lens, page, pages)
    plain = filled(rng, 0, heads, dim, page, 32, lens, table, pages)
    for scales in (plain.ks, plain.vs):
        scales *= rng.uniform(0.4, 1.7, size=scales.shape).astype(np.float32)
        scales[rng.random(scales.shape) < 0.1] = 0.0
    q, out, lse = attend(plain, table, lens, counts, q_heads, rng=rng)
    check_attention(plain, table, lens, counts, q_heads, q, out, lse, every=67 if heads > 8 else 1)


def test_attention_absent_pages():
    """Tokens on pages outside the cache are not seen; a row with no page at all is empty."""
    rng = np.random.default_rng(51)
    lens, counts, page = [300, 128, 64], [2, 1, 1], 64
    table = tables(rng, lens, page, 12)
    table[0, 1], table[0, 3], table[2, 0] = -5, 12, -1
    table[1, 0] = 0x7fffffff
    plain = filled(rng, 0, 2, 128, page, 64, lens, table, 12)
    q, out, lse = attend(plain, table, lens, counts, 4, rng=rng)
    check_attention(plain, table, lens, counts, 4, q, out, lse)
    assert torch.all(out[3] == 0) and torch.all(lse[3] == -float("inf"))


def test_attention_rows_before_the_start():
    """More rows than tokens: the first ones see nothing."""
    rng = np.random.default_rng(52)
    lens, counts, page = [3, 0, 40], [7, 5, 60], 16
    table = tables(rng, lens, page, 8)
    plain = filled(rng, 0, 1, 64, page, 16, lens, table, 8)
    q, out, lse = attend(plain, table, lens, counts, 2, rng=rng)
    check_attention(plain, table, lens, counts, 2, q, out, lse)
    assert torch.all(out[:4] == 0) and torch.all(lse[7:12] == -float("inf"))


def test_attention_max_len_above_and_windows_over_freed_pages():
    """A loose max_len changes the split, not the result; pages that the window has left may be gone or reused."""
    rng = np.random.default_rng(53)
    lens, counts, page, window = [3000, 1100], [1, 1], 64, 200
    pages = 80
    table = tables(rng, lens, page, pages)
    plain = filled(rng, 0, 1, 128, page, 64, lens, table, pages)
    for i, n in enumerate(lens):
        first = (n - window) // page  # pages before this one are behind the window
        table[i, :first] = -1
    for max_len in (0, 3000):
        q, out, lse = attend(plain, table, lens, counts, 4, window, rng=rng, max_len=max_len)
        check_attention(plain, table, lens, counts, 4, q, out, lse, window)


def test_attention_strided_queries_no_lse_and_streams():
    rng = np.random.default_rng(54)
    lens, counts, page = [200, 90], [1, 1], 64
    table = tables(rng, lens, page, 8)
    plain = filled(rng, 0, 2, 128, page, 64, lens, table, 8)
    q, out, lse = attend(plain, table, lens, counts, 4, rng=rng)
    joint = torch.cat([q.view(2, -1), bf16(rng, (2, 512))], 1).cuda()
    view = joint[:, :512].view(2, 4, 128)
    dev, b, d = to_device(plain), batch_of(table, lens, counts), fq.attention_desc(4)
    ws = fq.alloc_attention_workspace(dev, b, d)
    again = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fq.fq_attention(dev, b, d, view, again, None, ws, s)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


def test_attention_of_an_empty_cache():
    rng = np.random.default_rng(55)
    plain = U.PlainCache(0, 0, 1, 64, 16, 16, rng)
    table = np.zeros((2, 3), np.int32)
    q, out, lse = attend(plain, table, [5, 0], [1, 1], 2, rng=rng)
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


def test_append_and_attention_in_a_graph():
    rng = np.random.default_rng(56)
    heads, q_heads, dim, page, block = 2, 8, 128, 64, 64
    lens = [600, 70, 1]
    table = tables(rng, lens, page, 16)
    plain = filled(rng, 0, heads, dim, page, block, lens, table, 16)
    dev, b, d = to_device(plain), batch_of(table, lens, [1, 1, 1]), fq.attention_desc(q_heads)
    k, v, q = (bf16(rng, (3, h, dim)).cuda() for h in (heads, heads, q_heads))
    out, lse = torch.empty_like(q), torch.empty((3, q_heads), device="cuda")
    ws = fq.alloc_attention_workspace(dev, b, d)

    def step():
        fq.fq_kv_append(dev, b, k, v)
        fq.fq_attention(dev, b, d, q, out, lse, ws)

    step()
    torch.cuda.synchronize()
    want, wz = out.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        out.zero_()
        lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wz)
