"""Refusals and sizes of the operators on 8-bit data, on the host (no GPU).

Every call here is refused, has nothing to do, or asks for sizes: no HIP call
is made. Pointers are fake and never read."""
import ctypes

import pytest
import torch

from fp8_fp4_tensor_amd import fq

B = 0x10000


@pytest.fixture(scope="module")
def L():
    return fq.lib()


def gemm(L, d, a=(B, B), b=(B, B), out=B, ws=None, n=0):
    pa, pb = (fq.FqPlane(*p) if p else None for p in (a, b))
    return L.fq_gemm(ctypes.byref(d) if d else None, ctypes.byref(pa) if pa else None,
                     ctypes.byref(pb) if pb else None, out, ws, n, None)


@pytest.mark.parametrize("m,n,k,rows,out,acc,want", [
    (-1, 128, 128, 128, 1, 0, fq.FQ_E_INVALID),
    (1, -128, 128, 128, 1, 0, fq.FQ_E_INVALID),
    (1, 128, -128, 128, 1, 0, fq.FQ_E_INVALID),
    (1, 128, 128, 128, 2, 0, fq.FQ_E_INVALID),
    (1, 128, 128, 128, -1, 0, fq.FQ_E_INVALID),
    (1, 128, 128, 128, 0, 2, fq.FQ_E_INVALID),
    (1, 128, 128, 64, 1, 0, fq.FQ_E_UNSUPPORTED),
    (1, 128, 128, 0, 1, 0, fq.FQ_E_UNSUPPORTED),
    (1, 128, 128, 128, 1, 1, fq.FQ_E_UNSUPPORTED),     # accumulating into bf16
    (1, 128, 100, 128, 1, 0, fq.FQ_E_SHAPE),
    (1, 100, 128, 128, 1, 0, fq.FQ_E_SHAPE),           # a 128-row tile cut short
    (1, 128, (1 << 23) + 128, 128, 1, 0, fq.FQ_E_SHAPE),
    (1 << 30, 128, 128, 128, 1, 0, fq.FQ_E_SHAPE),
    (1 << 20, 1 << 20, 128, 128, 1, 0, fq.FQ_E_SHAPE),
    (0, 128, 128, 128, 1, 0, fq.FQ_OK),
    (5, 0, 128, 1, 0, 1, fq.FQ_OK),
])
def test_gemm_shapes(L, m, n, k, rows, out, acc, want):
    d = fq.FqGemmDesc(m, n, k, rows, out, acc)
    z = ctypes.c_size_t()
    assert L.fq_gemm_workspace(ctypes.byref(d), ctypes.byref(z)) == want
    assert gemm(L, d) == want


def test_gemm_pointers(L):
    d = fq.gemm_desc(4, 128, 128)
    assert gemm(L, None) == fq.FQ_E_INVALID
    assert L.fq_gemm_workspace(None, None) == fq.FQ_E_INVALID
    assert L.fq_gemm_workspace(ctypes.byref(d), None) == fq.FQ_OK
    for kw in ({"a": None}, {"b": None}, {"out": None}, {"a": (None, B)}, {"a": (B, None)}, {"b": (None, B)},
               {"b": (B, None)}):
        assert gemm(L, d, **kw) == fq.FQ_E_INVALID, kw
    for kw in ({"out": B + 4}, {"a": (B + 8, B)}, {"a": (B, B + 4)}, {"b": (B + 1, B)}, {"b": (B, B + 8)}):
        assert gemm(L, d, **kw) == fq.FQ_E_ALIGN, kw


def test_gemm_workspace_is_required_where_reported(L):
    found = 0
    for m in (1, 33, 200, 300):
        for n, k in ((128, 18432), (512, 8192), (1024, 2048), (18432, 7168)):
            d = fq.gemm_desc(m, n, k)
            z = fq.fq_gemm_workspace(d)
            if z:
                found += 1
                assert gemm(L, d, ws=None, n=0) == fq.FQ_E_WORKSPACE
                assert gemm(L, d, ws=B, n=z - 1) == fq.FQ_E_WORKSPACE
                assert gemm(L, d, ws=B + 8, n=z) == fq.FQ_E_ALIGN
    assert found > 0


def cache(**kw):
    v = dict(format=0, kv_heads=2, head_dim=128, page_tokens=64, block_tokens=64, num_pages=8, k=B, v=B, k_scale=B,
             v_scale=B)
    v.update(kw)
    return fq.FqKvCache(**v)


def batch(**kw):
    v = dict(batch=2, max_pages=4, max_q=1, max_len=0, total_q=2, page_table=B, seq_lens=B, q_start=None)
    v.update(kw)
    return fq.FqKvBatch(**v)


def adesc(**kw):
    v = dict(q_heads=4, window=0, scale=0.0, softcap=0.0, q_stride=0)
    v.update(kw)
    return fq.FqAttentionDesc(**v)


def ref(x):
    return None if x is None else ctypes.byref(x)


def append(L, c, b, dt=1, k=B, ks=256, v=B, vs=256):
    return L.fq_kv_append(ref(c), ref(b), dt, k, ks, v, vs, None)


def attend(L, c, b, d, q=B, out=B, lse=None, ws=B, n=1 << 40):
    return L.fq_attention(ref(c), ref(b), ref(d), q, out, lse, ws, n, None)


BAD_CACHE = [
    ({"format": 3}, fq.FQ_E_INVALID), ({"format": -1}, fq.FQ_E_INVALID), ({"kv_heads": 0}, fq.FQ_E_INVALID),
    ({"num_pages": -1}, fq.FQ_E_INVALID), ({"format": fq.FQ_E2M1}, fq.FQ_E_UNSUPPORTED),
    ({"head_dim": 96}, fq.FQ_E_UNSUPPORTED), ({"head_dim": 0}, fq.FQ_E_UNSUPPORTED),
    ({"page_tokens": 8}, fq.FQ_E_UNSUPPORTED), ({"page_tokens": 48}, fq.FQ_E_UNSUPPORTED),
    ({"page_tokens": 512}, fq.FQ_E_UNSUPPORTED), ({"block_tokens": 8}, fq.FQ_E_UNSUPPORTED),
    ({"block_tokens": 128}, fq.FQ_E_UNSUPPORTED), ({"page_tokens": 256, "block_tokens": 256}, fq.FQ_E_UNSUPPORTED),
    ({"num_pages": 1 << 30}, fq.FQ_E_SHAPE), ({"kv_heads": 8192}, fq.FQ_E_SHAPE),
]
BAD_BATCH = [
    ({"batch": -1}, fq.FQ_E_INVALID), ({"max_pages": -1}, fq.FQ_E_INVALID), ({"max_q": -1}, fq.FQ_E_INVALID),
    ({"max_len": -1}, fq.FQ_E_INVALID), ({"total_q": -1}, fq.FQ_E_INVALID), ({"batch": 65536}, fq.FQ_E_SHAPE),
    ({"max_pages": 1 << 25}, fq.FQ_E_SHAPE), ({"max_q": 1 << 25}, fq.FQ_E_SHAPE), ({"total_q": 1 << 40}, fq.FQ_E_SHAPE),
    ({"page_table": None}, fq.FQ_E_INVALID), ({"seq_lens": None}, fq.FQ_E_INVALID), ({"page_table": B + 2}, fq.FQ_E_ALIGN),
    ({"seq_lens": B + 1}, fq.FQ_E_ALIGN), ({"q_start": B + 2}, fq.FQ_E_ALIGN),
]


@pytest.mark.parametrize("change,want", BAD_CACHE + [({"k": None}, fq.FQ_E_INVALID), ({"v": None}, fq.FQ_E_INVALID),
                                                     ({"k_scale": None}, fq.FQ_E_INVALID),
                                                     ({"v_scale": None}, fq.FQ_E_INVALID), ({"k": B + 8}, fq.FQ_E_ALIGN),
                                                     ({"v": B + 1}, fq.FQ_E_ALIGN), ({"k_scale": B + 4}, fq.FQ_E_ALIGN),
                                                     ({"v_scale": B + 4}, fq.FQ_E_ALIGN)])
def test_cache_is_checked(L, change, want):
    c = cache(**change)
    assert append(L, c, batch()) == want
    assert attend(L, c, batch(), adesc()) == want
    z = ctypes.c_size_t()
    if (change, want) in BAD_CACHE:
        assert L.fq_attention_workspace(ref(c), ref(batch()), ref(adesc()), ctypes.byref(z)) == want


@pytest.mark.parametrize("change,want", BAD_BATCH)
def test_batch_is_checked(L, change, want):
    assert append(L, cache(), batch(**change)) == want
    assert attend(L, cache(), batch(**change), adesc()) == want


def test_append_arguments(L):
    assert append(L, None, batch()) == fq.FQ_E_INVALID
    assert append(L, cache(), None) == fq.FQ_E_INVALID
    for kw, want in (({"dt": 2}, fq.FQ_E_INVALID), ({"k": None}, fq.FQ_E_INVALID), ({"v": None}, fq.FQ_E_INVALID),
                     ({"ks": 255}, fq.FQ_E_INVALID), ({"vs": 0}, fq.FQ_E_INVALID), ({"ks": 260}, fq.FQ_E_ALIGN),
                     ({"dt": 0, "vs": 258}, fq.FQ_E_ALIGN), ({"k": B + 8}, fq.FQ_E_ALIGN),
                     ({"ks": 1 << 40}, fq.FQ_E_SHAPE)):
        assert append(L, cache(), batch(), **kw) == want, kw
    for kw in ({"batch": 0}, {"max_q": 0}, {"total_q": 0}, {"max_pages": 0}):
        assert append(L, cache(), batch(**kw)) == fq.FQ_OK, kw
    assert append(L, cache(num_pages=0, k=None, v=None), batch()) == fq.FQ_OK


def test_attention_arguments(L):
    inf, nan = float("inf"), float("nan")
    assert attend(L, None, batch(), adesc()) == fq.FQ_E_INVALID
    assert attend(L, cache(), None, adesc()) == fq.FQ_E_INVALID
    assert attend(L, cache(), batch(), None) == fq.FQ_E_INVALID
    for kw, want in (({"q_heads": 0}, fq.FQ_E_INVALID), ({"q_heads": 3}, fq.FQ_E_UNSUPPORTED),
                     ({"window": -1}, fq.FQ_E_INVALID), ({"scale": nan}, fq.FQ_E_INVALID), ({"scale": inf}, fq.FQ_E_INVALID),
                     ({"softcap": -1.0}, fq.FQ_E_INVALID), ({"softcap": nan}, fq.FQ_E_INVALID),
                     ({"softcap": inf}, fq.FQ_E_INVALID), ({"q_stride": -8}, fq.FQ_E_INVALID),
                     ({"q_stride": 511}, fq.FQ_E_INVALID), ({"q_stride": 516}, fq.FQ_E_ALIGN),
                     ({"q_stride": 1 << 40}, fq.FQ_E_SHAPE), ({"q_heads": 1 << 20}, fq.FQ_E_SHAPE)):
        assert attend(L, cache(), batch(), adesc(**kw)) == want, kw
    for kw, want in (({"q": None}, fq.FQ_E_INVALID), ({"out": None}, fq.FQ_E_INVALID), ({"q": B + 8}, fq.FQ_E_ALIGN),
                     ({"out": B + 2}, fq.FQ_E_ALIGN), ({"lse": B + 2}, fq.FQ_E_ALIGN)):
        assert attend(L, cache(), batch(), adesc(), **kw) == want, kw
    for kw in ({"batch": 0}, {"max_q": 0}, {"total_q": 0}):
        assert attend(L, cache(), batch(**kw), adesc(), ws=None, n=0) == fq.FQ_OK, kw


def test_attention_workspace(L):
    c, d = cache(num_pages=1 << 16), adesc()
    z = ctypes.c_size_t()
    b = batch(max_pages=4096)
    assert L.fq_attention_workspace(ref(c), ref(b), ref(d), ctypes.byref(z)) == fq.FQ_OK and z.value > 0
    assert attend(L, c, b, d, ws=None, n=0) == fq.FQ_E_WORKSPACE
    assert attend(L, c, b, d, ws=B, n=z.value - 1) == fq.FQ_E_WORKSPACE
    assert attend(L, c, b, d, ws=B + 4, n=z.value) == fq.FQ_E_ALIGN
    assert L.fq_attention_workspace(ref(c), ref(batch(max_len=40)), ref(d), ctypes.byref(z)) == fq.FQ_OK and z.value == 0


# ---------------------------------------------------------------- the binding's own checks
def t8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def test_binding_refuses_tensors_that_do_not_fit():
    f = torch.zeros
    with pytest.raises(ValueError):
        fq.Plane(t8(4, 256).t(), f(4, 2))
    with pytest.raises(TypeError):
        fq.Plane(t8(4, 128), f(4, 1, dtype=torch.bfloat16))
    a, b = fq.Plane(t8(4, 128), f(4, 1)), fq.Plane(t8(128, 128), f(1, 1))
    d = fq.gemm_desc(4, 128, 128)
    with pytest.raises(TypeError):
        fq.fq_gemm(d, a, b, f(4, 128))
    with pytest.raises(ValueError):
        fq.fq_gemm(d, b, b, f(4, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fq.fq_gemm(fq.gemm_desc(4, 128, 128, 1), a, b, f(4, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fq.KvCache(0, 16, t8(2, 1, 32, 64), t8(2, 1, 32, 64), f(2, 1, 2), f(2, 1, 2))
    with pytest.raises(ValueError):
        fq.KvCache(0, 32, t8(2, 1, 32, 64), t8(2, 1, 64, 32), f(2, 1, 2), f(2, 1, 2))
    with pytest.raises(TypeError):
        fq.KvBatch(f(2, 3), f(2, dtype=torch.int32), None, 2, 1)
    with pytest.raises(ValueError):
        fq.KvBatch(f(2, 3, dtype=torch.int32), f(3, dtype=torch.int32), None, 2, 1)
    c = fq.KvCache(0, 16, t8(2, 2, 32, 64), t8(2, 2, 64, 32), f(2, 2, 2), f(2, 2, 2))
    bt = fq.KvBatch(f(2, 3, dtype=torch.int32), f(2, dtype=torch.int32), None, 2, 1)
    x = f(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fq.fq_kv_append(c, bt, x[:, :1], x)
    with pytest.raises(ValueError):
        fq.fq_kv_append(c, bt, f(2, 64, 2, dtype=torch.bfloat16).transpose(1, 2), x)
    with pytest.raises(TypeError):
        fq.fq_kv_append(c, bt, x, x.float())
    with pytest.raises(TypeError):
        fq.fq_attention(c, bt, fq.attention_desc(2), x, x.float())
    with pytest.raises(TypeError):
        fq.fq_attention(c, bt, fq.attention_desc(2), x, x.clone(), f(2, 3))
