"""What the binding of the operators on 8-bit data refuses before the library
sees it, on the host (no GPU): the tensors are on the CPU, so no call here may
reach a launch."""
import pytest
import torch

from fp8_fp4_tensor_amd import fq


class Stream:
    cuda_stream = 0


def z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


def cache(heads=2, dim=64, page=32, block=16, pages=2, fmt=fq.FQ_E4M3, dtype=torch.uint8):
    return fq.KvCache(fmt, block, z(pages, heads, page, dim, dtype=dtype), z(pages, heads, dim, page, dtype=dtype),
                      z(pages, heads, page // block), z(pages, heads, page // block))


def batch(rows, **kw):
    v = dict(page_table=z(rows, 2, dtype=torch.int32), seq_lens=z(rows, dtype=torch.int32), q_start=None,
             total_q=rows, max_q=1)
    v.update(kw)
    return fq.KvBatch(**v)


@pytest.mark.parametrize("rows", [2, 5])
def test_tokens_that_overlap_are_refused(rows):
    """A token stride below a token's own length, 0 among them: the library takes a stride of 0 for contiguous
    queries and would read rows behind the tensor's only one."""
    c, b, d = cache(), batch(rows), fq.attention_desc(4)
    out = z(rows, 4, 64, dtype=torch.bfloat16)
    one = z(1, 4, 64, dtype=torch.bfloat16)
    half = z(rows * 256, dtype=torch.bfloat16).as_strided((rows, 4, 64), (128, 64, 1))
    for q in (one.expand(rows, 4, 64), half):
        with pytest.raises(ValueError):
            fq.fq_attention(c, b, d, q, out, None, None, Stream)
        new = q[:, :2]
        with pytest.raises(ValueError):
            fq.fq_kv_append(c, b, new.expand(rows, 2, 64) if q.stride(0) == 0 else new.as_strided((rows, 2, 64), (64, 64, 1)),
                            z(rows, 2, 64, dtype=torch.bfloat16), Stream)


def test_attention_leaves_the_descriptor_alone(monkeypatch):
    """One descriptor serves caches of several head dims and queries of several strides, and never holds a
    call's own stride: another thread, or a workspace query, may be reading it."""
    seen = []
    real = fq.lib()

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

        def fq_attention(self, cache, batch, desc, *rest):
            got = desc._obj
            seen.append((got.q_heads, got.window, got.scale, got.softcap, got.q_stride))
            return fq.FQ_OK

    monkeypatch.setattr(fq, "lib", Lib)
    monkeypatch.setattr(fq, "_one_gpu", lambda *a: None, raising=False)
    d = fq.attention_desc(4, scale=0.5, window=7, softcap=2.0)
    for dim, joint in ((64, 4 * 64), (64, 4 * 64 + 128), (128, 4 * 128), (64, 1024), (256, 4 * 256 + 8)):
        c, b = cache(dim=dim), batch(3)
        q = z(3, joint, dtype=torch.bfloat16)[:, :4 * dim].view(3, 4, dim)
        fq.fq_attention(c, b, d, q, torch.empty((3, 4, dim), dtype=torch.bfloat16), None, None, Stream)
        assert seen[-1] == (4, 7, 0.5, 2.0, 0 if joint == 4 * dim else joint)
        assert (d.q_heads, d.window, d.scale, d.softcap, d.q_stride) == (4, 7, 0.5, 2.0, 0)
        for other in (64, 128, 256):
            fq.fq_attention_workspace(cache(dim=other), b, d)
    # a stride that the caller has set is not the call's: queries say theirs
    d.q_stride = 1 << 30
    fq.fq_attention(cache(), batch(3), d, z(3, 4, 64, dtype=torch.bfloat16), z(3, 4, 64, dtype=torch.bfloat16), None, None,
                    Stream)
    assert seen[-1][-1] == 0 and d.q_stride == 1 << 30


def test_handles_are_fixed():
    """The library's structs are filled once: an attribute that could be set afterwards would say one thing and
    the call do another, or leave the struct with a freed tensor's address."""
    p = fq.Plane(z(4, 128, dtype=torch.uint8), z(4, 1))
    c, b = cache(), batch(3, max_len=40)
    for h, names in ((p, ("data", "scale")),
                     (c, ("k", "v", "k_scale", "v_scale", "fmt", "block_tokens", "heads", "dim", "page_tokens", "pages")),
                     (b, ("page_table", "seq_lens", "q_start", "total_q", "max_q", "max_len"))):
        for name in names:
            was = getattr(h, name)
            for act in (lambda: setattr(h, name, 9), lambda: delattr(h, name)):
                with pytest.raises(AttributeError):
                    act()
            assert getattr(h, name) is was
    assert (b._c.max_len, b._c.total_q, b._c.max_q) == (b.max_len, b.total_q, b.max_q) == (40, 3, 1)


class Elsewhere(torch.Tensor):
    """A CPU tensor that says it is on a GPU: what the checks before the launch see."""

    @staticmethod
    def on(t, index):
        t = t.as_subclass(Elsewhere)
        t.index = index
        return t

    def get_device(self):
        return getattr(self, "index", -1)


def test_tensors_off_the_gpu_are_refused(monkeypatch):
    """A host address, or another GPU's, would fault the GPU inside the kernel. Every tensor of a call is asked."""
    monkeypatch.setattr(fq, "lib", lambda: pytest.fail("the library was called"))

    def refused(make, count):
        """make(on): `on` places each of the call's tensors in turn. Tensor `odd` alone is elsewhere."""
        for index in (-1, 1):
            for odd in range(count):
                at = iter(range(count))
                with pytest.raises(ValueError, match="GPU"):
                    make(lambda t: Elsewhere.on(t, index if next(at) == odd else 0))
        with pytest.raises(ValueError, match="GPU"):
            make(lambda t: t)

    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32

    def product(on):
        fq.fq_gemm(fq.gemm_desc(4, 128, 128), fq.Plane(on(z(4, 128, dtype=u8)), on(z(4, 1))),
                   fq.Plane(on(z(128, 128, dtype=u8)), on(z(1, 1))), on(z(4, 128, dtype=bf)), on(z(64, dtype=u8)), Stream)

    def handles(on):
        c = fq.KvCache(0, 16, on(z(2, 2, 32, 64, dtype=u8)), on(z(2, 2, 64, 32, dtype=u8)), on(z(2, 2, 2)), on(z(2, 2, 2)))
        return c, fq.KvBatch(on(z(3, 2, dtype=i32)), on(z(3, dtype=i32)), on(z(4, dtype=i32)), 3, 1)

    def append(on):
        fq.fq_kv_append(*handles(on), on(z(3, 2, 64)), on(z(3, 2, 64)), Stream)

    def attend(on):
        fq.fq_attention(*handles(on), fq.attention_desc(4), on(z(3, 4, 64, dtype=bf)), on(z(3, 4, 64, dtype=bf)),
                        on(z(3, 4)), on(z(64, dtype=u8)), Stream)

    refused(product, 6)
    refused(append, 9)
    refused(attend, 11)


def test_workspaces_are_whole():
    """A strided workspace's bytes are not where its size says."""
    ws = z(4, 64, dtype=torch.uint8)[:, :16]
    with pytest.raises(ValueError, match="workspace"):
        fq.fq_gemm(fq.gemm_desc(4, 128, 128), fq.Plane(z(4, 128, dtype=torch.uint8), z(4, 1)),
                   fq.Plane(z(128, 128, dtype=torch.uint8), z(1, 1)), z(4, 128, dtype=torch.bfloat16), ws, Stream)
    with pytest.raises(ValueError, match="workspace"):
        fq.fq_attention(cache(), batch(3), fq.attention_desc(4), z(3, 4, 64, dtype=torch.bfloat16),
                        z(3, 4, 64, dtype=torch.bfloat16), None, ws, Stream)


def test_codes_of_another_format_are_refused():
    """Bytes are taken as they are; a tensor that names its 8-bit format has to name the right one."""
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    for ok in (torch.uint8, torch.int8, e4):
        fq.Plane(z(4, 128, dtype=torch.uint8).view(ok), z(4, 1))
    with pytest.raises(TypeError):
        fq.Plane(z(4, 128, dtype=torch.uint8).view(e5), z(4, 1))
    for fmt, right, wrong in ((fq.FQ_E4M3, e4, e5), (fq.FQ_E5M2, e5, e4)):
        k, v, s = z(2, 2, 32, 64, dtype=torch.uint8), z(2, 2, 64, 32, dtype=torch.uint8), z(2, 2, 2)
        fq.KvCache(fmt, 16, k, v, s, s)
        fq.KvCache(fmt, 16, k.view(right), v.view(right), s, s)
        for a, b in ((wrong, right), (right, wrong), (torch.uint8, wrong)):
            with pytest.raises(TypeError):
                fq.KvCache(fmt, 16, k.view(a), v.view(b), s, s)
