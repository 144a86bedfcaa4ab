"""Refusals and sizes of the operators of a feed-forward block, on the host (no
GPU): every call here is refused, has nothing to do, or asks for sizes.
Pointers are fake and never read; tensors are on the CPU, so that no call of
the binding may reach a launch."""
import ctypes

import pytest
import torch

from fp8_fp4_tensor_amd import fq

P = 0x10000
BF, F32 = fq.FQ_IN_BF16, fq.FQ_IN_F32
BOTH = fq.FQ_ROWWISE | fq.FQ_COLWISE


@pytest.fixture(scope="module")
def L():
    return fq.lib()


def ref(x):
    return None if x is None else ctypes.byref(x)


# ---------------------------------------------------------------- product
def gemm(L, d, a=(P, P), b=(P, P), out=P, ws=None, n=0):
    pa, pb = (fq.FqPlane(*p) if p else None for p in (a, b))
    return L.fq_gemm_mx(ref(d), ref(pa), ref(pb), out, ws, n, None)


@pytest.mark.parametrize("m,n,k,fa,fb,out,acc,want", [
    (-1, 128, 128, 0, 0, 1, 0, fq.FQ_E_INVALID),
    (1, -128, 128, 0, 0, 1, 0, fq.FQ_E_INVALID),
    (1, 128, -32, 0, 0, 1, 0, fq.FQ_E_INVALID),
    (1, 128, 128, 3, 0, 1, 0, fq.FQ_E_INVALID),
    (1, 128, 128, 0, -1, 1, 0, fq.FQ_E_INVALID),
    (1, 128, 128, 0, 0, 2, 0, fq.FQ_E_INVALID),
    (1, 128, 128, 0, 0, 0, 2, fq.FQ_E_INVALID),
    (1, 128, 128, 2, 2, 1, 1, fq.FQ_E_UNSUPPORTED),   # accumulating into bf16
    (1, 128, 100, 0, 2, 1, 0, fq.FQ_E_SHAPE),
    (1, 128, 16, 2, 2, 1, 0, fq.FQ_E_SHAPE),
    (1, 128, (1 << 22) + 32, 0, 0, 1, 0, fq.FQ_E_SHAPE),
    (1 << 30, 128, 128, 0, 0, 1, 0, fq.FQ_E_SHAPE),
    (1, 1 << 30, 128, 0, 0, 1, 0, fq.FQ_E_SHAPE),
    (1 << 20, 1 << 20, 32, 0, 0, 1, 0, fq.FQ_E_SHAPE),
    (0, 128, 128, 0, 1, 1, 0, fq.FQ_OK),
    (5, 0, 128, 2, 1, 0, 1, fq.FQ_OK),
])
def test_gemm_mx_shapes(L, m, n, k, fa, fb, out, acc, want):
    d = fq.FqGemmMxDesc(m, n, k, fa, fb, out, acc)
    z = ctypes.c_size_t()
    assert L.fq_gemm_mx_workspace(ref(d), ref(z)) == want
    assert gemm(L, d) == want


def test_gemm_mx_pointers(L):
    d = fq.gemm_mx_desc(40, 128, 128)
    assert gemm(L, None) == fq.FQ_E_INVALID
    assert L.fq_gemm_mx_workspace(None, None) == fq.FQ_E_INVALID
    assert L.fq_gemm_mx_workspace(ref(d), None) == fq.FQ_OK
    for kw in ({"a": None}, {"b": None}, {"out": None}, {"a": (None, P)}, {"a": (P, None)}, {"b": (None, P)},
               {"b": (P, None)}):
        assert gemm(L, d, **kw) == fq.FQ_E_INVALID, kw
    for kw in ({"out": P + 4}, {"a": (P + 8, P)}, {"a": (P, P + 4)}, {"b": (P + 1, P)}, {"b": (P, P + 8)}):
        assert gemm(L, d, **kw) == fq.FQ_E_ALIGN, kw


# ---------------------------------------------------------------- norm
def planes(rows, cols, outputs=BOTH, recipe=fq.FQ_MX, fmt=fq.FQ_E4M3, block=(1, 32), **kw):
    return fq.desc(recipe, F32, fmt, rows, cols, block, outputs, **kw)


def quantized(row=(P, P), col=(P, P)):
    return fq.FqQuantized(fq.FqPlane(*row), fq.FqPlane(*col), None, None)


def norm(L, d, q=None, x=P, res=None, w=P, h=None, rstd=P, y=P, out=None):
    return L.fq_rmsnorm(ref(d), ref(q), x, res, w, h, rstd, y, ref(out), None)


def back(L, d, h=P, rstd=P, w=P, dy=P, dres=None, dx=P, dw=P, ws=P, n=1 << 40):
    return L.fq_rmsnorm_backward(ref(d), h, rstd, w, dy, dres, dx, dw, ws, n, None)


BAD_NORM = [
    (dict(rows=-1), fq.FQ_E_INVALID), (dict(cols=-8), fq.FQ_E_INVALID), (dict(x_dtype=2), fq.FQ_E_INVALID),
    (dict(h_dtype=-1), fq.FQ_E_INVALID), (dict(weight_dtype=2), fq.FQ_E_INVALID), (dict(y_dtype=7), fq.FQ_E_INVALID),
    (dict(accumulate=2), fq.FQ_E_INVALID), (dict(eps=0.0), fq.FQ_E_INVALID), (dict(eps=-1e-6), fq.FQ_E_INVALID),
    (dict(eps=float("nan")), fq.FQ_E_INVALID), (dict(eps=float("inf")), fq.FQ_E_INVALID),
    (dict(cols=100), fq.FQ_E_SHAPE), (dict(cols=32776), fq.FQ_E_SHAPE), (dict(rows=1 << 33), fq.FQ_E_SHAPE),
]


def ndesc(**kw):
    v = dict(rows=64, cols=256, x_dtype=BF, h_dtype=BF, weight_dtype=F32, y_dtype=BF, accumulate=0, eps=1e-6, x_stride=0)
    v.update(kw)
    return fq.FqRmsnormDesc(**v)


@pytest.mark.parametrize("bad,want", BAD_NORM)
def test_norm_fields(L, bad, want):
    d = ndesc(**bad)
    assert norm(L, d) == back(L, d) == L.fq_rmsnorm_workspace(ref(d), None) == want


def test_norm_arguments(L):
    d, q, o = ndesc(), planes(64, 256), quantized()
    assert norm(L, None) == back(L, None) == L.fq_rmsnorm_workspace(None, None) == fq.FQ_E_INVALID
    for kw in ({"x": None}, {"w": None}, {"y": None}, {"res": P}, {"h": P}, {"q": q}, {"q": q, "out": o, "rstd": None},
               {"q": q, "out": quantized(row=(None, P))}, {"q": q, "out": quantized(col=(P, None))}):
        assert norm(L, d, **kw) == fq.FQ_E_INVALID, kw
    for kw in ({"x": P + 8}, {"w": P + 4}, {"y": P + 2}, {"res": P + 8, "h": P}, {"res": P, "h": P + 8}, {"rstd": P + 2},
               {"q": q, "out": quantized(row=(P + 8, P))}, {"q": q, "out": quantized(col=(P, P + 4))}):
        assert norm(L, d, **kw) == fq.FQ_E_ALIGN, kw
    for stride, want in ((255, fq.FQ_E_INVALID), (-8, fq.FQ_E_INVALID), (260, fq.FQ_E_ALIGN), (1 << 34, fq.FQ_E_SHAPE)):
        assert norm(L, ndesc(x_stride=stride)) == want
    assert norm(L, ndesc(x_stride=258, x_dtype=F32)) == fq.FQ_E_ALIGN
    for kw in ({"h": None}, {"rstd": None}, {"w": None}, {"dy": None}, {"dx": None}):
        assert back(L, d, **kw) == fq.FQ_E_INVALID, kw
    for kw in ({"h": P + 8}, {"rstd": P + 1}, {"w": P + 8}, {"dy": P + 8}, {"dres": P + 4}, {"dx": P + 4}, {"dw": P + 4},
               {"ws": P + 8}):
        assert back(L, d, **kw) == fq.FQ_E_ALIGN, kw
    z = fq.fq_rmsnorm_workspace(d)
    assert z > 0 and back(L, d, ws=None) == back(L, d, n=z - 1) == fq.FQ_E_WORKSPACE


BAD_PLANES = [
    (dict(recipe=9), fq.FQ_E_INVALID), (dict(outputs=0), fq.FQ_E_INVALID), (dict(fmt=5), fq.FQ_E_INVALID),
    (dict(recipe=fq.FQ_NVFP4, fmt=fq.FQ_E2M1, block=(1, 16)), fq.FQ_E_UNSUPPORTED),
    (dict(recipe=fq.FQ_PER_TENSOR_CURRENT), fq.FQ_E_UNSUPPORTED), (dict(recipe=fq.FQ_PER_TENSOR_DELAYED), fq.FQ_E_UNSUPPORTED),
    (dict(recipe=fq.FQ_BLOCK_FP32, block=(128, 128)), fq.FQ_E_UNSUPPORTED), (dict(block=(1, 64)), fq.FQ_E_UNSUPPORTED),
    (dict(rounding=fq.FQ_ROUND_STOCHASTIC), fq.FQ_E_UNSUPPORTED), (dict(rows=32), fq.FQ_E_SHAPE), (dict(cols=512), fq.FQ_E_SHAPE),
]


@pytest.mark.parametrize("bad,want", BAD_PLANES)
def test_planes_of_an_operator(L, bad, want):
    v = dict(rows=128, cols=256)
    v.update(bad)
    q, o = planes(**v), quantized()
    assert norm(L, ndesc(rows=128), q, out=o) == want
    s = fq.FqSwigluDesc(128, 256, BF, BF, 0)
    assert L.fq_swiglu(ref(s), ref(q), P, None, ref(o), None) == want
    w = fq.FqSwigluDesc(128, 128, BF, BF, 0)
    assert L.fq_swiglu_backward(ref(w), ref(q), P, P, None, ref(o), None) == want


def test_rows_that_a_colwise_block_does_not_divide(L):
    o = quantized()
    for rows, recipe, block in ((33, fq.FQ_MX, (1, 32)), (96, fq.FQ_BLOCK_FP32, (1, 128))):
        assert norm(L, ndesc(rows=rows), planes(rows, 256, BOTH, recipe, block=block), out=o) == fq.FQ_E_SHAPE
    # a gradient's halves are whole blocks each
    s = fq.FqSwigluDesc(128, 64, BF, BF, 0)
    assert L.fq_swiglu_backward(ref(s), ref(planes(128, 128, BOTH, fq.FQ_BLOCK_FP32, block=(1, 128))), P, P, None, ref(o),
                                None) == fq.FQ_E_SHAPE


# ---------------------------------------------------------------- gated activation
def test_swiglu_arguments(L):
    def fwd(d, q=None, x=P, y=P, out=None):
        return L.fq_swiglu(ref(d), ref(q), x, y, ref(out), None)

    def bwd(d, q=None, x=P, dy=P, dx=P, out=None):
        return L.fq_swiglu_backward(ref(d), ref(q), x, dy, dx, ref(out), None)

    ok = dict(rows=64, cols=256, x_dtype=BF, y_dtype=BF, x_stride=0)
    for bad, want in ((dict(rows=-1), fq.FQ_E_INVALID), (dict(cols=-8), fq.FQ_E_INVALID), (dict(x_dtype=2), fq.FQ_E_INVALID),
                      (dict(y_dtype=-1), fq.FQ_E_INVALID), (dict(cols=4), fq.FQ_E_SHAPE), (dict(rows=1 << 28), fq.FQ_E_SHAPE),
                      (dict(x_stride=504), fq.FQ_E_INVALID), (dict(x_stride=516), fq.FQ_E_ALIGN),
                      (dict(x_stride=1 << 34), fq.FQ_E_SHAPE)):
        d = fq.FqSwigluDesc(**{**ok, **bad})
        assert fwd(d) == bwd(d) == want, bad
    d, q, o = fq.FqSwigluDesc(**ok), planes(64, 256), quantized()
    assert fwd(None) == bwd(None) == fwd(d, x=None) == fwd(d, y=None) == fwd(d, q) == fq.FQ_E_INVALID
    assert bwd(d, x=None) == bwd(d, dy=None) == bwd(d, dx=None) == fq.FQ_E_INVALID
    assert fwd(d, x=P + 8) == fwd(d, y=P + 8) == bwd(d, x=P + 4) == bwd(d, dy=P + 2) == bwd(d, dx=P + 8) == fq.FQ_E_ALIGN
    assert bwd(d, q, out=o) == fq.FQ_E_SHAPE  # the gradient has twice the columns
    empty = fq.FqSwigluDesc(0, 256, BF, BF, 0)
    assert fwd(empty, y=None) == bwd(empty, dx=None) == fq.FQ_OK


# ---------------------------------------------------------------- the binding, before the library sees a call
class Stream:
    cuda_stream = 0


def z(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype)


def plane(rows, k, fmt=fq.FQ_E4M3):
    return fq.MxPlane(z(rows, k // 2 if fmt == fq.FQ_E2M1 else k, dtype=torch.uint8), z(rows, k // 32, dtype=torch.uint8), fmt)


def test_mx_planes_are_checked():
    u8 = torch.uint8
    for data, scale, fmt, error in ((z(4, 64, dtype=u8).t(), z(64, 1, dtype=u8), 0, ValueError),
                                    (z(4, 64, dtype=u8), z(2, 4, dtype=u8).t(), 0, ValueError),
                                    (z(4, 64), z(4, 2, dtype=u8), 0, TypeError), (z(4, 64, dtype=u8), z(4, 2), 0, TypeError),
                                    (z(4, 64, dtype=torch.float8_e5m2), z(4, 2, dtype=u8), 0, TypeError),
                                    (z(4, 32, dtype=torch.int8), z(4, 2, dtype=u8), 2, TypeError)):
        with pytest.raises(error):
            fq.MxPlane(data, scale, fmt)
    p = plane(4, 64)
    with pytest.raises(AttributeError):
        p.fmt = 1
    fq.MxPlane(z(4, 64, dtype=torch.float8_e4m3fn), z(4, 2, dtype=u8).view(torch.float8_e8m0fnu), 0)


def test_gemm_mx_tensors_are_checked(monkeypatch):
    monkeypatch.setattr(fq, "lib", lambda: pytest.fail("the library was called"))
    d, bf = fq.gemm_mx_desc(4, 8, 64, fq.FQ_E4M3, fq.FQ_E2M1), torch.bfloat16
    a, b, out = plane(4, 64), plane(8, 64, fq.FQ_E2M1), z(4, 8, dtype=bf)
    for args, error in (((plane(4, 64, fq.FQ_E2M1), b, out), TypeError), ((a, plane(8, 64), out), TypeError),
                        ((plane(5, 64), b, out), ValueError), ((a, plane(8, 32, fq.FQ_E2M1), out), ValueError),
                        ((a, b, z(4, 9, dtype=bf)), ValueError), ((a, b, z(4, 8)), TypeError),
                        ((a, b, z(8, 4, dtype=bf).t()), TypeError), ((a, b, out), ValueError)):  # the last: on the CPU
        with pytest.raises(error):
            fq.fq_gemm_mx(d, *args, stream=Stream)
    with pytest.raises(ValueError):
        fq.fq_gemm_mx(d, a, b, out, z(16, 2, dtype=torch.uint8).t(), stream=Stream)


def target(rows, cols, outputs=fq.FQ_ROWWISE):
    d = planes(rows, cols, outputs)
    return fq.Planes(d, fq.alloc_quantized(d, "cpu"))


def test_targets_are_checked():
    d = planes(64, 64)
    for change, error in ((dict(row_data=z(63, 64, dtype=torch.uint8)), ValueError), (dict(col_scale=None), ValueError),
                          (dict(col_data=z(64, 128, dtype=torch.uint8)[:, ::2]), ValueError),
                          (dict(row_scale=z(32)), TypeError), (dict(row_data=z(64, 64, dtype=torch.int8)), TypeError)):
        q = fq.alloc_quantized(d, "cpu")
        for name, t in change.items():
            setattr(q, name, t)
        with pytest.raises(error):
            fq.Planes(d, q)
    t = fq.Planes(d, fq.alloc_quantized(d, "cpu"))
    d.rows = 32  # the caller's descriptor may change
    assert t._d.rows == 64
    with pytest.raises(AttributeError):
        t.rows = 3
    with pytest.raises(fq.FqError):
        fq.Planes(planes(33, 64), fq.Quantized())


def test_norm_tensors_are_checked(monkeypatch):
    bf = torch.bfloat16
    rows, cols = 4, 64
    t, wide = target(rows, cols), target(rows, 2 * cols)
    d, x, w, y, h = fq.rmsnorm_desc(rows, cols), z(rows, cols, dtype=bf), z(cols), z(rows, cols, dtype=bf), z(rows, cols, dtype=bf)
    r = z(rows)
    monkeypatch.setattr(fq, "lib", lambda: pytest.fail("the library was called"))
    for args, error in (((x, w), ValueError), ((x[:3], w, None, None, None, y), ValueError), ((x.float(), w, None, None, None, y), TypeError),
                        ((x, w.to(bf), None, None, None, y), TypeError), ((x, z(cols + 1), None, None, None, y), TypeError),
                        ((x, w, h, None, None, y), ValueError), ((x, w, None, h, None, y), ValueError),
                        ((x, w, h.float(), h, None, y), TypeError), ((x, w, h, h[:, :32], None, y), ValueError),
                        ((x, w, None, None, z(rows + 1), y), TypeError), ((x, w, None, None, r.double(), y), TypeError),
                        ((x, w, None, None, None, y.float()), TypeError), ((x, w, None, None, None, y.t()), ValueError),
                        ((x, w, None, None, None, None, wide), ValueError),
                        ((x[:1].expand(rows, cols), w, None, None, None, y), ValueError),
                        ((z(cols, rows, dtype=bf).t(), w, None, None, None, y), ValueError),
                        ((x, w, None, None, None, None, t), ValueError), ((x, w, None, None, r, y), ValueError)):  # on the CPU
        with pytest.raises(error):
            fq.fq_rmsnorm(d, *args, stream=Stream)
    good = (x, r, w, y, h, z(cols), h)
    for at, bad in ((0, x.float()), (0, x[:2]), (1, z(rows - 1)), (2, z(cols - 8)), (3, y.float()), (4, h.t()), (4, h.float()),
                    (5, z(cols, dtype=bf)), (5, z(2 * cols)[::2]), (6, h[:, :8]), (6, h)):
        args = list(good)
        args[at] = bad
        with pytest.raises((ValueError, TypeError)):
            fq.fq_rmsnorm_backward(d, *args, stream=Stream)


def test_swiglu_tensors_are_checked(monkeypatch):
    bf = torch.bfloat16
    t, wide = target(4, 64), target(4, 128)
    d, x, y, dx = fq.swiglu_desc(4, 64), z(4, 128, dtype=bf), z(4, 64, dtype=bf), z(4, 128, dtype=bf)
    monkeypatch.setattr(fq, "lib", lambda: pytest.fail("the library was called"))
    for args, error in (((x,), ValueError), ((x[:, :64], y), ValueError), ((x.float(), y), TypeError), ((x, y.float()), TypeError),
                        ((x, y.t()), ValueError), ((x, None, wide), ValueError), ((x[:1].expand(4, 128), y), ValueError),
                        ((x, y), ValueError), ((x, None, t), ValueError)):
        with pytest.raises(error):
            fq.fq_swiglu(d, *args, stream=Stream)
    for args, error in (((x, y), ValueError), ((x, y[:2], dx), ValueError), ((x, y.float(), dx), TypeError), ((x, y, y), ValueError),
                        ((x, y, dx.float()), TypeError), ((x, y, None, t), ValueError), ((x, y, dx), ValueError),
                        ((x, y, None, wide), ValueError)):
        with pytest.raises(error):
            fq.fq_swiglu_backward(d, *args, stream=Stream)


class Elsewhere(torch.Tensor):
    """A CPU tensor that says it is on a GPU: what the checks before the launch see."""

    @staticmethod
    def on(t, index):
        t = t.as_subclass(Elsewhere)
        t.index = index
        return t

    def get_device(self):
        return getattr(self, "index", -1)


@pytest.mark.parametrize("away", [-1, 1], ids=["host", "other-gpu"])
def test_tensors_elsewhere_are_refused(monkeypatch, away):
    """Every tensor of a call is asked where it is: a host address would fault the GPU inside the kernel."""
    bf = torch.bfloat16
    tp = {c: planes(4, c, fq.FQ_ROWWISE) for c in (64, 128)}
    sizes = {c: fq.fq_sizes(tp[c]) for c in tp}
    monkeypatch.setattr(fq, "fq_sizes", lambda d: sizes[d.cols])
    calls = {
        "gemm": (6, lambda t: fq.fq_gemm_mx(fq.gemm_mx_desc(4, 8, 64), fq.MxPlane(t(0, 4, 64, dtype=torch.uint8), t(1, 4, 2, dtype=torch.uint8), 0),
                                            fq.MxPlane(t(2, 8, 64, dtype=torch.uint8), t(3, 8, 2, dtype=torch.uint8), 0),
                                            t(4, 4, 8, dtype=bf), t(5, 16, dtype=torch.uint8), Stream)),
        "norm": (8, lambda t: fq.fq_rmsnorm(fq.rmsnorm_desc(4, 64), t(0, 4, 64, dtype=bf), t(1, 64), t(2, 4, 64, dtype=bf),
                                            t(3, 4, 64, dtype=bf), t(4, 4), t(5, 4, 64, dtype=bf),
                                            fq.Planes(tp[64], fq.Quantized(t(6, 4, 64, dtype=torch.uint8), t(7, 8, dtype=torch.uint8))), Stream)),
        "norm_backward": (8, lambda t: fq.fq_rmsnorm_backward(fq.rmsnorm_desc(4, 64), t(0, 4, 64, dtype=bf), t(1, 4), t(2, 64),
                                                              t(3, 4, 64, dtype=bf), t(4, 4, 64, dtype=bf), t(5, 64),
                                                              t(6, 4, 64, dtype=bf), t(7, 4096, dtype=torch.uint8), Stream)),
        "swiglu": (4, lambda t: fq.fq_swiglu(fq.swiglu_desc(4, 64), t(0, 4, 128, dtype=bf), t(1, 4, 64, dtype=bf),
                                             fq.Planes(tp[64], fq.Quantized(t(2, 4, 64, dtype=torch.uint8), t(3, 8, dtype=torch.uint8))), Stream)),
        "swiglu_backward": (5, lambda t: fq.fq_swiglu_backward(
            fq.swiglu_desc(4, 64), t(0, 4, 128, dtype=bf), t(1, 4, 64, dtype=bf), t(2, 4, 128, dtype=bf),
            fq.Planes(tp[128], fq.Quantized(t(3, 4, 128, dtype=torch.uint8), t(4, 16, dtype=torch.uint8))), Stream)),
    }
    monkeypatch.setattr(fq, "lib", lambda: pytest.fail("the library was called"))
    for name, (count, call) in calls.items():
        for odd in range(count):
            with pytest.raises(ValueError, match="one GPU"):
                call(lambda i, *s, dtype=torch.float32: Elsewhere.on(z(*s, dtype=dtype), away if i == odd else 0))


def test_tensors_of_a_gpu_that_is_not_current_are_refused(monkeypatch):
    monkeypatch.setattr(fq, "lib", lambda: pytest.fail("the library was called"))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = lambda *s, dtype=torch.bfloat16: Elsewhere.on(z(*s, dtype=dtype), 1)
    with pytest.raises(ValueError, match="current"):
        fq.fq_swiglu(fq.swiglu_desc(4, 64), t(4, 128), t(4, 64), stream=Stream)
    with pytest.raises(ValueError, match="current"):
        fq.fq_rmsnorm(fq.rmsnorm_desc(4, 64), t(4, 64), t(64, dtype=torch.float32), y=t(4, 64), stream=Stream)


def test_outputs_over_inputs(L):
    """What a kernel would read after it is written is refused; results over what is read first are not (they fail later
    or run, so only the refusals are seen here)."""
    Q, R, S = P + 4096, P + 8192, P + 12288
    for d, kw in ((ndesc(h_dtype=F32), dict(x=P, res=Q, h=P, y=R)), (ndesc(x_stride=512), dict(x=P, res=Q, h=P, y=R)),
                  (ndesc(), dict(x=P, y=P)), (ndesc(), dict(x=P, res=Q, h=R, y=R)), (ndesc(), dict(x=P, res=Q, h=R, y=Q))):
        assert norm(L, d, w=S, **kw) == fq.FQ_E_INVALID, kw
    assert back(L, ndesc(h_dtype=F32), h=P, dy=Q, dx=Q, dw=None) == fq.FQ_E_INVALID
    d, s = fq.FqSwigluDesc(64, 256, BF, BF, 0), fq.FqSwigluDesc(64, 256, BF, BF, 1024)
    assert L.fq_swiglu(ref(d), None, P, P, None, None) == fq.FQ_E_INVALID
    assert L.fq_swiglu_backward(ref(d), None, P, Q, Q, None, None) == fq.FQ_E_INVALID
    assert L.fq_swiglu_backward(ref(s), None, P, Q, P, None, None) == fq.FQ_E_INVALID


def test_largest_shapes(L):
    """Just past each limit, and sizes whose products would overflow 64 bits."""
    sw = lambda r, c: L.fq_swiglu(ref(fq.FqSwigluDesc(r, c, BF, BF, 0)), None, P, P + 4096, None, None)
    assert sw(1, (1 << 28) + 8) == sw(0, 1 << 62) == sw(1 << 62, 8) == sw((1 << 7) + 1, 1 << 28) == fq.FQ_E_SHAPE
    mx = lambda m, n, k: L.fq_gemm_mx_workspace(ref(fq.gemm_mx_desc(m, n, k)), None)
    assert mx((1 << 28) + 1, 1, 32) == mx(1, (1 << 28) + 1, 32) == mx(1, 1, (1 << 22) + 32) == fq.FQ_E_SHAPE
    assert mx(1 << 20, 1 << 17, 32) == mx(1 << 62, 1 << 62, 32) == fq.FQ_E_SHAPE
    assert mx(1 << 28, 1 << 8, 32) == mx(1, 1 << 28, 256) == mx(1 << 14, 1 << 14, 1 << 22) == fq.FQ_OK
    assert norm(L, ndesc(rows=1 << 62)) == norm(L, ndesc(rows=(1 << 28) + 1)) == fq.FQ_E_SHAPE
