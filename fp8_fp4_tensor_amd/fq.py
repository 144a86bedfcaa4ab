"""Thin ctypes binding of libfq.so (include/fq.h).

Argument marshalling only: the functions below pass torch device pointers,
shapes and the current HIP stream to the C entry points of the same names and
raise FqError on a non-OK status. Every step of the quantization runs in the
library's HIP kernels; torch supplies device memory and streams.

The library is loaded on first use from this package directory; if it is
missing the binding raises (build it with __graft_entry__.build()). There is
no fallback.
"""
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

# ---------------------------------------------------------------- enums (fq.h)
FQ_OK, FQ_E_INVALID, FQ_E_UNSUPPORTED, FQ_E_SHAPE, FQ_E_ALIGN, FQ_E_WORKSPACE, FQ_E_HIP = range(7)
FQ_IN_F32, FQ_IN_BF16 = 0, 1
FQ_E4M3, FQ_E5M2, FQ_E2M1 = 0, 1, 2
FQ_PER_TENSOR_CURRENT, FQ_PER_TENSOR_DELAYED, FQ_BLOCK_FP32, FQ_MX, FQ_NVFP4 = range(5)
FQ_ROWWISE, FQ_COLWISE = 1, 2
FQ_ROUND_NEAREST_EVEN, FQ_ROUND_STOCHASTIC = 0, 1
FQ_SCALE_DEFAULT, FQ_SCALE_POW2 = 0, 1
FQ_TRANSFORM_NONE, FQ_TRANSFORM_RHT16 = 0, 1

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfq.so")


class FqDesc(ctypes.Structure):
    _fields_ = [("recipe", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("format", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("block_rows", ctypes.c_int32),
                ("block_cols", ctypes.c_int32), ("outputs", ctypes.c_uint32), ("rounding", ctypes.c_int32),
                ("scale_mode", ctypes.c_int32), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("transform", ctypes.c_int32), ("rht_signs", ctypes.c_uint32)]


class FqPlane(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class FqQuantized(ctypes.Structure):
    _fields_ = [("rowwise", FqPlane), ("colwise", FqPlane), ("tensor_scale", ctypes.c_void_p),
                ("amax", ctypes.c_void_p)]


FQ_DELAYED_PENDING_BYTES = 8256


class FqDelayedState(ctypes.Structure):
    _fields_ = [("amax_history", ctypes.c_void_p), ("history_len", ctypes.c_int32), ("scale", ctypes.c_void_p),
                ("scale_inv", ctypes.c_void_p), ("pending", ctypes.c_void_p), ("step", ctypes.c_int64)]


class FqGemmDesc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("b_block_rows", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


class FqKvCache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("block_tokens", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class FqKvBatch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("total_q", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("q_start", ctypes.c_void_p)]


class FqAttentionDesc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float), ("q_stride", ctypes.c_int64)]


class FqGemmMxDesc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("a_format", ctypes.c_int32),
                ("b_format", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


class FqRmsnormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
                ("h_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64)]


class FqSwigluDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("x_stride", ctypes.c_int64)]


class FqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)}")


_lib = None
_P = ctypes.c_void_p
_SZ = ctypes.POINTER(ctypes.c_size_t)


def lib():
    """The loaded libfq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    dp = ctypes.POINTER(FqDesc)
    qp = ctypes.POINTER(FqQuantized)
    pp = ctypes.POINTER(FqPlane)
    gp = ctypes.POINTER(FqGemmDesc)
    cp = ctypes.POINTER(FqKvCache)
    bp = ctypes.POINTER(FqKvBatch)
    ap = ctypes.POINTER(FqAttentionDesc)
    mp = ctypes.POINTER(FqGemmMxDesc)
    np_ = ctypes.POINTER(FqRmsnormDesc)
    sp = ctypes.POINTER(FqSwigluDesc)
    sig = {
        "fq_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "fq_sizes": (ctypes.c_int, [dp, _SZ, _SZ, _SZ, _SZ, _SZ]),
        "fq_quantize": (ctypes.c_int, [dp, _P, qp, _P, ctypes.c_size_t, _P]),
        "fq_amax": (ctypes.c_int, [dp, _P, _P, _P, ctypes.c_size_t, _P]),
        "fq_quantize_with_amax": (ctypes.c_int, [dp, _P, _P, qp, _P, ctypes.c_size_t, _P]),
        "fq_quantize_delayed": (ctypes.c_int, [dp, _P, ctypes.POINTER(FqDelayedState), qp, _P, ctypes.c_size_t, _P]),
        "fq_delayed_flush": (ctypes.c_int, [dp, ctypes.POINTER(FqDelayedState), _P]),
        "fq_dequantize": (ctypes.c_int, [dp, qp, ctypes.c_int32, _P, ctypes.c_int32, _P]),
        "fq_requantize_transpose": (ctypes.c_int, [dp, qp, qp, _P]),
        "fq_quantize_noalloc": (ctypes.c_int, [dp, _P, qp, _P]),
        "fq_gemm_workspace": (ctypes.c_int, [gp, _SZ]),
        "fq_gemm": (ctypes.c_int, [gp, pp, pp, _P, _P, ctypes.c_size_t, _P]),
        "fq_kv_append": (ctypes.c_int, [cp, bp, ctypes.c_int32, _P, ctypes.c_int64, _P, ctypes.c_int64, _P]),
        "fq_attention_workspace": (ctypes.c_int, [cp, bp, ap, _SZ]),
        "fq_attention": (ctypes.c_int, [cp, bp, ap, _P, _P, _P, _P, ctypes.c_size_t, _P]),
        "fq_gemm_mx_workspace": (ctypes.c_int, [mp, _SZ]),
        "fq_gemm_mx": (ctypes.c_int, [mp, pp, pp, _P, _P, ctypes.c_size_t, _P]),
        "fq_rmsnorm": (ctypes.c_int, [np_, dp, _P, _P, _P, _P, _P, _P, qp, _P]),
        "fq_rmsnorm_workspace": (ctypes.c_int, [np_, _SZ]),
        "fq_rmsnorm_backward": (ctypes.c_int, [np_, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
        "fq_swiglu": (ctypes.c_int, [sp, dp, _P, _P, qp, _P]),
        "fq_swiglu_backward": (ctypes.c_int, [sp, dp, _P, _P, _P, qp, _P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def fq_status_str(status: int) -> str:
    return lib().fq_status_str(int(status)).decode()


status_str = fq_status_str


def _check(status: int, where: str):
    if status != FQ_OK:
        raise FqError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without a Stream object (a microsecond less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------- descriptors
def desc(recipe: int, in_dtype: int, fmt: int, rows: int, cols: int, block=(0, 0),
         outputs: int = FQ_ROWWISE, rounding: int = FQ_ROUND_NEAREST_EVEN, seed: int = 0, offset: int = 0,
         scale_mode: int = FQ_SCALE_DEFAULT, transform: int = FQ_TRANSFORM_NONE, rht_signs: int = 0) -> FqDesc:
    return FqDesc(recipe, in_dtype, fmt, rows, cols, block[0], block[1], outputs, rounding, scale_mode, seed,
                  offset, transform, rht_signs)


def in_dtype_of(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return FQ_IN_BF16
    if x.dtype == torch.float32:
        return FQ_IN_F32
    raise TypeError("inputs are float32 or bfloat16")


@dataclass
class Sizes:
    row_data: int
    row_scale: int
    col_data: int
    col_scale: int
    workspace: int


def fq_sizes(d: FqDesc) -> Sizes:
    v = [ctypes.c_size_t() for _ in range(5)]
    _check(lib().fq_sizes(ctypes.byref(d), *[ctypes.byref(x) for x in v]), "fq_sizes")
    return Sizes(*[x.value for x in v])


# ---------------------------------------------------------------- output buffers
@dataclass
class Quantized:
    """Device buffers of one quantized tensor (uint8 codes, fp32 or uint8 scales)."""
    row_data: Optional[torch.Tensor] = None
    row_scale: Optional[torch.Tensor] = None
    col_data: Optional[torch.Tensor] = None
    col_scale: Optional[torch.Tensor] = None
    tensor_scale: Optional[torch.Tensor] = None
    amax: Optional[torch.Tensor] = None

    def c(self) -> FqQuantized:
        return FqQuantized(FqPlane(_ptr(self.row_data), _ptr(self.row_scale)),
                           FqPlane(_ptr(self.col_data), _ptr(self.col_scale)),
                           _ptr(self.tensor_scale), _ptr(self.amax))


def _scale_dtype(d: FqDesc):
    return torch.float32 if d.recipe == FQ_BLOCK_FP32 else torch.uint8


def alloc_quantized(d: FqDesc, device="cuda") -> Quantized:
    """Allocate every plane fq_sizes reports for d (shaped, on `device`)."""
    z = fq_sizes(d)
    R, C = d.rows, d.cols
    q = Quantized()
    sd = _scale_dtype(d)
    es = 4 if sd == torch.float32 else 1
    packed = d.format == FQ_E2M1
    if z.row_data:
        q.row_data = torch.empty((R, C // 2) if packed else (R, C), dtype=torch.uint8, device=device)
    if z.col_data:
        q.col_data = torch.empty((C, R // 2) if packed else (C, R), dtype=torch.uint8, device=device)
    if z.row_scale:
        q.row_scale = torch.empty(z.row_scale // es, dtype=sd, device=device)
    if z.col_scale:
        q.col_scale = torch.empty(z.col_scale // es, dtype=sd, device=device)
    q.tensor_scale = torch.empty(1, dtype=torch.float32, device=device)
    q.amax = torch.empty(1, dtype=torch.float32, device=device)
    return q


def alloc_workspace(d: FqDesc, device="cuda") -> Optional[torch.Tensor]:
    n = fq_sizes(d).workspace
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device) if n else None


# ---------------------------------------------------------------- entry points
def fq_quantize(d: FqDesc, x: torch.Tensor, out: Quantized, ws: Optional[torch.Tensor] = None, stream=None):
    q = out.c()
    _check(lib().fq_quantize(ctypes.byref(d), _ptr(x), ctypes.byref(q), _ptr(ws),
                             0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)), "fq_quantize")


def fq_quantize_noalloc(d: FqDesc, x: torch.Tensor, out: Quantized, stream=None):
    """fq_quantize with the library's own per-GPU scratch array (no workspace)."""
    q = out.c()
    _check(lib().fq_quantize_noalloc(ctypes.byref(d), _ptr(x), ctypes.byref(q), _stream(stream)),
           "fq_quantize_noalloc")


def fq_amax(d: FqDesc, x: torch.Tensor, amax_out: torch.Tensor, ws: torch.Tensor, stream=None):
    _check(lib().fq_amax(ctypes.byref(d), _ptr(x), _ptr(amax_out), _ptr(ws), ws.numel() * ws.element_size(),
                         _stream(stream)), "fq_amax")


def fq_quantize_with_amax(d: FqDesc, x: torch.Tensor, amax_in: torch.Tensor, out: Quantized,
                          ws: Optional[torch.Tensor] = None, stream=None):
    q = out.c()
    _check(lib().fq_quantize_with_amax(ctypes.byref(d), _ptr(x), _ptr(amax_in), ctypes.byref(q), _ptr(ws),
                                       0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "fq_quantize_with_amax")


class DelayedState:
    """Delayed-scaling state in device memory plus the host step counter."""

    def __init__(self, history_len: int = 1024, device="cuda"):
        self.amax_history = torch.zeros(history_len, dtype=torch.float32, device=device)
        self.scale = torch.ones(1, dtype=torch.float32, device=device)
        self.scale_inv = torch.ones(1, dtype=torch.float32, device=device)
        self.pending = torch.zeros(FQ_DELAYED_PENDING_BYTES // 4, dtype=torch.float32, device=device)
        self.step = 0

    def c(self) -> FqDelayedState:
        return FqDelayedState(_ptr(self.amax_history), self.amax_history.numel(), _ptr(self.scale),
                              _ptr(self.scale_inv), _ptr(self.pending), self.step)

    def state_dict(self):
        """The state as it stands (call fq_delayed_flush first to make the
        window and scales current and the pending records unnecessary)."""
        return {"amax_history": self.amax_history.clone(), "scale": self.scale.clone(),
                "scale_inv": self.scale_inv.clone(), "pending": self.pending.clone(), "step": self.step}

    def load_state_dict(self, sd):
        self.amax_history.copy_(sd["amax_history"])
        self.scale.copy_(sd["scale"])
        self.scale_inv.copy_(sd["scale_inv"])
        if "pending" in sd:
            self.pending.copy_(sd["pending"])
        else:
            self.pending.zero_()
        self.step = int(sd["step"])


def fq_quantize_delayed(d: FqDesc, x: torch.Tensor, state: DelayedState, out: Quantized,
                        ws: Optional[torch.Tensor] = None, stream=None, advance: bool = True):
    q = out.c()
    st = state.c()
    _check(lib().fq_quantize_delayed(ctypes.byref(d), _ptr(x), ctypes.byref(st), ctypes.byref(q), _ptr(ws),
                                     0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "fq_quantize_delayed")
    if advance:
        state.step += 1


def fq_delayed_flush(d: FqDesc, state: DelayedState, stream=None):
    """Bring state's window and scales up to date after its last step."""
    st = state.c()
    _check(lib().fq_delayed_flush(ctypes.byref(d), ctypes.byref(st), _stream(stream)), "fq_delayed_flush")


def fq_dequantize(d: FqDesc, qt: Quantized, which: int, y: torch.Tensor, stream=None):
    """y (float32 or bfloat16) = the values of plane `which` of qt."""
    q = qt.c()
    _check(lib().fq_dequantize(ctypes.byref(d), ctypes.byref(q), which, _ptr(y), in_dtype_of(y), _stream(stream)),
           "fq_dequantize")


def fq_requantize_transpose(d: FqDesc, src: Quantized, dst: Quantized, stream=None):
    """MXFP8, or blockwise 1x128 with power-of-two scales: dst's colwise planes
    from src's rowwise planes (no high-precision source)."""
    a, b = src.c(), dst.c()
    _check(lib().fq_requantize_transpose(ctypes.byref(d), ctypes.byref(a), ctypes.byref(b), _stream(stream)),
           "fq_requantize_transpose")


# ---------------------------------------------------------------- operators on 8-bit data
_ELSEWHERE = "the tensors of a call are on one GPU"


def _one_gpu(on: int, *tensors: Optional[torch.Tensor]):
    """Tensors that are given are on GPU `on` (-1: none): a host address would fault the GPU inside the kernel."""
    if on < 0:
        raise ValueError(_ELSEWHERE)
    for t in tensors:
        if t is not None and t.get_device() != on:
            raise ValueError(_ELSEWHERE)


def _common_gpu(*tensors: Optional[torch.Tensor]) -> int:
    """The GPU that tensors share, -1 if there is none (the CPU: handles can be made there, calls cannot)."""
    given = [t.get_device() for t in tensors if t is not None]
    return given[0] if all(g == given[0] for g in given) else -1


_FLOAT8 = {FQ_E4M3: torch.float8_e4m3fn, FQ_E5M2: torch.float8_e5m2}


def _codes_of(fmt: int, *codes: torch.Tensor):
    """Codes are bytes; a float8 type says what they are, and has to be the format's."""
    for t in codes:
        if t.element_size() != 1 or (t.is_floating_point() and t.dtype != _FLOAT8.get(fmt)):
            raise TypeError("codes are 8-bit, and of the format where their type names one")


class _Handle:
    """A C struct with the tensors it points into. The struct is filled once, so
    the attributes are fixed: make another handle for other tensors or sizes."""

    def __setattr__(self, name, value):
        raise AttributeError(f"a {type(self).__name__} is fixed: make another one")

    def __delattr__(self, name):
        self.__setattr__(name, None)


class Plane(_Handle):
    """One quantized copy as an operand: codes and scales (kept alive here)."""

    def __init__(self, data: torch.Tensor, scale: torch.Tensor):
        if not (data.is_contiguous() and scale.is_contiguous()):
            raise ValueError("planes are contiguous")
        _codes_of(FQ_E4M3, data)
        if scale.dtype != torch.float32:
            raise TypeError("blockwise planes are 8-bit codes and float32 scales")
        c = FqPlane(data.data_ptr(), scale.data_ptr())
        self.__dict__.update(data=data, scale=scale, _sizes=(data.numel(), scale.numel()), _on=_common_gpu(data, scale),
                             _c=c, _ref=ctypes.byref(c))

    @classmethod
    def rowwise(cls, q: Quantized) -> "Plane":
        return cls(q.row_data, q.row_scale)

    @classmethod
    def colwise(cls, q: Quantized) -> "Plane":
        return cls(q.col_data, q.col_scale)


def gemm_desc(m: int, n: int, k: int, b_block_rows: int = 128, out_dtype: int = FQ_IN_BF16,
              accumulate: bool = False) -> FqGemmDesc:
    return FqGemmDesc(m, n, k, b_block_rows, out_dtype, int(accumulate))


def fq_gemm_workspace(d: FqGemmDesc) -> int:
    n = ctypes.c_size_t()
    _check(lib().fq_gemm_workspace(ctypes.byref(d), ctypes.byref(n)), "fq_gemm_workspace")
    return n.value


def alloc_gemm_workspace(d: FqGemmDesc, device="cuda") -> Optional[torch.Tensor]:
    n = fq_gemm_workspace(d)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _nbytes(ws: Optional[torch.Tensor]) -> int:
    if ws is None:
        return 0
    if not ws.is_contiguous():
        raise ValueError("a workspace is contiguous")
    return ws.numel() * ws.element_size()


def fq_gemm(d: FqGemmDesc, a: Plane, b: Plane, out: torch.Tensor, ws: Optional[torch.Tensor] = None, stream=None):
    """out [m, n] = A B^T of two blockwise planes (out += with d.accumulate)."""
    m, n, k = d.m, d.n, d.k
    nb = k // 128
    if a._sizes[0] != m * k or b._sizes[0] != n * k or out.numel() != m * n:
        raise ValueError("a is [m, k], b is [n, k] and out is [m, n]")
    if a._sizes[1] != m * nb or b._sizes[1] != (n if d.b_block_rows == 1 else n // 128) * nb:
        raise ValueError("a scale for each block of 128 (and for 128 rows of b with b_block_rows 128)")
    if in_dtype_of(out) != d.out_dtype or not out.is_contiguous():
        raise TypeError("out is contiguous and of the descriptor's out_dtype")
    size = _nbytes(ws)
    _one_gpu(a._on if a._on == b._on else -1, out, ws)
    _check(lib().fq_gemm(ctypes.byref(d), a._ref, b._ref, out.data_ptr(),
                         None if ws is None else ws.data_ptr(), size, _stream(stream)), "fq_gemm")


class KvCache(_Handle):
    """A paged 8-bit key/value cache (buffers and their shape)."""

    def __init__(self, fmt: int, block_tokens: int, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        pages, heads, page, dim = k.shape
        if tuple(v.shape) != (pages, heads, dim, page):
            raise ValueError("k is [pages, heads, page_tokens, dim] and v is [pages, heads, dim, page_tokens]")
        if block_tokens < 1 or any(tuple(s.shape) != (pages, heads, page // block_tokens) for s in (k_scale, v_scale)):
            raise ValueError("scales are [pages, heads, page_tokens / block_tokens]")
        _codes_of(fmt, k, v)
        if any(s.dtype != torch.float32 for s in (k_scale, v_scale)):
            raise TypeError("codes are 8-bit and scales float32")
        if not all(t.is_contiguous() for t in (k, v, k_scale, v_scale)):
            raise ValueError("cache buffers are contiguous")
        c = FqKvCache(fmt, heads, dim, page, block_tokens, pages, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                      v_scale.data_ptr())
        self.__dict__.update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, fmt=fmt, block_tokens=block_tokens, heads=heads,
                             dim=dim, page_tokens=page, pages=pages, _on=_common_gpu(k, v, k_scale, v_scale), _c=c,
                             _ref=ctypes.byref(c))


def alloc_kv_cache(fmt: int, pages: int, heads: int, dim: int, page_tokens: int = 64, block_tokens: int = 64,
                   device="cuda") -> KvCache:
    """An empty cache; its contents need no initialization."""
    if block_tokens < 1 or page_tokens % block_tokens:
        raise ValueError("a page holds whole blocks")
    s = (pages, heads, page_tokens // block_tokens)
    return KvCache(fmt, block_tokens,
                   torch.empty((pages, heads, page_tokens, dim), dtype=torch.uint8, device=device),
                   torch.empty((pages, heads, dim, page_tokens), dtype=torch.uint8, device=device),
                   torch.empty(s, dtype=torch.float32, device=device),
                   torch.empty(s, dtype=torch.float32, device=device))


class KvBatch(_Handle):
    """The sequences of a call: page_table [batch, max_pages], seq_lens [batch]
    and q_start [batch + 1] are int32 device tensors (q_start None: max_q rows
    of every sequence), whose contents may change between calls; max_len bounds
    seq_lens (0: what the table holds)."""

    def __init__(self, page_table: torch.Tensor, seq_lens: torch.Tensor, q_start: Optional[torch.Tensor],
                 total_q: int, max_q: int, max_len: int = 0):
        given = [t for t in (page_table, seq_lens, q_start) if t is not None]
        if any(t.dtype != torch.int32 or not t.is_contiguous() for t in given):
            raise TypeError("page_table, seq_lens and q_start are contiguous int32")
        batch, max_pages = page_table.shape
        if seq_lens.numel() != batch or (q_start is not None and q_start.numel() != batch + 1):
            raise ValueError("seq_lens has batch entries and q_start batch + 1")
        c = FqKvBatch(batch, max_pages, max_q, max_len, total_q, page_table.data_ptr(), seq_lens.data_ptr(),
                      None if q_start is None else q_start.data_ptr())
        self.__dict__.update(page_table=page_table, seq_lens=seq_lens, q_start=q_start, total_q=total_q, max_q=max_q,
                             max_len=max_len, _on=_common_gpu(*given), _c=c, _ref=ctypes.byref(c))


def _rows3(t: torch.Tensor, total: int, heads: int, dim: int, what: str) -> int:
    """The token stride of a [total, heads, dim] tensor whose tokens are each contiguous."""
    if t.shape != (total, heads, dim):
        raise ValueError(f"{what} is [total_q, heads, head_dim]")
    tokens, rows, dims = t.stride()
    if dims != 1 or (heads > 1 and rows != dim):
        raise ValueError(f"{what}: a token's heads are contiguous")
    if total <= 1:
        return heads * dim
    if tokens < heads * dim:  # an expanded row's 0 would mean contiguous to the library
        raise ValueError(f"{what}: tokens do not overlap")
    return tokens


def fq_kv_append(cache: KvCache, batch: KvBatch, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
    """Quantize k_new and v_new [total_q, heads, dim] into the last positions of their sequences."""
    ks = _rows3(k_new, batch.total_q, cache.heads, cache.dim, "k_new")
    vs = _rows3(v_new, batch.total_q, cache.heads, cache.dim, "v_new")
    dt = in_dtype_of(k_new)
    if v_new.dtype != k_new.dtype:
        raise TypeError("k_new and v_new have one dtype")
    _one_gpu(cache._on if cache._on == batch._on else -1, k_new, v_new)
    _check(lib().fq_kv_append(cache._ref, batch._ref, dt, k_new.data_ptr(), ks,
                              v_new.data_ptr(), vs, _stream(stream)), "fq_kv_append")


def attention_desc(q_heads: int, scale: float = 0.0, window: int = 0, softcap: float = 0.0) -> FqAttentionDesc:
    return FqAttentionDesc(q_heads, window, scale, softcap, 0)


def fq_attention_workspace(cache: KvCache, batch: KvBatch, d: FqAttentionDesc) -> int:
    n = ctypes.c_size_t()
    _check(lib().fq_attention_workspace(cache._ref, batch._ref, ctypes.byref(d),
                                        ctypes.byref(n)), "fq_attention_workspace")
    return n.value


def alloc_attention_workspace(cache: KvCache, batch: KvBatch, d: FqAttentionDesc,
                              device="cuda") -> Optional[torch.Tensor]:
    n = fq_attention_workspace(cache, batch, d)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def fq_attention(cache: KvCache, batch: KvBatch, d: FqAttentionDesc, q: torch.Tensor, out: torch.Tensor,
                 lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """out [total_q, q_heads, dim] bf16 (and lse [total_q, q_heads] fp32) = attention of q over the cache.
    The token stride is q's own, whatever d.q_stride holds."""
    stride = _rows3(q, batch.total_q, d.q_heads, cache.dim, "q")
    if stride == d.q_heads * cache.dim:
        stride = 0
    if stride != d.q_stride:  # a descriptor of this call: the caller's may be in use elsewhere
        d = FqAttentionDesc(d.q_heads, d.window, d.scale, d.softcap, stride)
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise TypeError("q and out are bfloat16")
    if out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out is contiguous and of q's shape")
    if lse is not None and (lse.dtype != torch.float32 or lse.numel() != batch.total_q * d.q_heads
                            or not lse.is_contiguous()):
        raise TypeError("lse is contiguous float32 [total_q, q_heads]")
    size = _nbytes(ws)
    _one_gpu(cache._on if cache._on == batch._on else -1, q, out, lse, ws)
    _check(lib().fq_attention(cache._ref, batch._ref, ctypes.byref(d), q.data_ptr(),
                              out.data_ptr(), None if lse is None else lse.data_ptr(),
                              None if ws is None else ws.data_ptr(), size, _stream(stream)), "fq_attention")


# ---------------------------------------------------------------- a feed-forward block on microscaled data
def _here(on: int, *tensors: Optional[torch.Tensor]):
    """Tensors that are given are on GPU `on`, and that is the current one: a launch goes there."""
    _one_gpu(on, *tensors)
    if on != torch.cuda.current_device():
        raise ValueError("the tensors of a call are on the current GPU")


class MxPlane(_Handle):
    """One MX copy as an operand: codes of `fmt` [rows, k] (or [rows, k / 2] packed) and E8M0 scales (kept alive here)."""

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, fmt: int):
        if not (data.is_contiguous() and scale.is_contiguous()):
            raise ValueError("planes are contiguous")
        if fmt == FQ_E2M1:
            if data.dtype != torch.uint8:
                raise TypeError("packed codes are bytes")
        else:
            _codes_of(fmt, data)
        if scale.dtype not in (torch.uint8, torch.float8_e8m0fnu):
            raise TypeError("MX scales are E8M0 bytes")
        c = FqPlane(data.data_ptr(), scale.data_ptr())
        self.__dict__.update(data=data, scale=scale, fmt=fmt, _sizes=(data.numel(), scale.numel()),
                             _on=_common_gpu(data, scale), _c=c, _ref=ctypes.byref(c))

    @classmethod
    def rowwise(cls, q: Quantized, fmt: int) -> "MxPlane":
        return cls(q.row_data, q.row_scale, fmt)

    @classmethod
    def colwise(cls, q: Quantized, fmt: int) -> "MxPlane":
        return cls(q.col_data, q.col_scale, fmt)


def gemm_mx_desc(m: int, n: int, k: int, a_format: int = FQ_E4M3, b_format: int = FQ_E4M3,
                 out_dtype: int = FQ_IN_BF16, accumulate: bool = False) -> FqGemmMxDesc:
    return FqGemmMxDesc(m, n, k, a_format, b_format, out_dtype, int(accumulate))


def fq_gemm_mx_workspace(d: FqGemmMxDesc) -> int:
    n = ctypes.c_size_t()
    _check(lib().fq_gemm_mx_workspace(ctypes.byref(d), ctypes.byref(n)), "fq_gemm_mx_workspace")
    return n.value


def alloc_gemm_mx_workspace(d: FqGemmMxDesc, device="cuda") -> Optional[torch.Tensor]:
    n = fq_gemm_mx_workspace(d)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def fq_gemm_mx(d: FqGemmMxDesc, a: MxPlane, b: MxPlane, out: torch.Tensor, ws: Optional[torch.Tensor] = None,
               stream=None):
    """out [m, n] = A B^T of two MX planes (out += with d.accumulate)."""
    m, n, k = d.m, d.n, d.k
    if a.fmt != d.a_format or b.fmt != d.b_format:
        raise TypeError("planes are of the descriptor's formats")
    if a._sizes != (m * k >> (a.fmt == FQ_E2M1), m * (k // 32)) or b._sizes != (n * k >> (b.fmt == FQ_E2M1), n * (k // 32)):
        raise ValueError("a is [m, k] and b is [n, k], with a scale for each 32 of a row")
    if out.numel() != m * n:
        raise ValueError("out is [m, n]")
    if in_dtype_of(out) != d.out_dtype or not out.is_contiguous():
        raise TypeError("out is contiguous and of the descriptor's out_dtype")
    size = _nbytes(ws)
    _here(a._on if a._on == b._on else -1, out, ws)
    _check(lib().fq_gemm_mx(ctypes.byref(d), a._ref, b._ref, out.data_ptr(), None if ws is None else ws.data_ptr(), size,
                            _stream(stream)), "fq_gemm_mx")


class Planes(_Handle):
    """What an operator quantizes its result to: a descriptor and the buffers alloc_quantized gives for it."""

    def __init__(self, d: FqDesc, out: Quantized):
        z = fq_sizes(d)
        sd = _scale_dtype(d)
        given = []
        for want, t, dtype in ((z.row_data, out.row_data, torch.uint8), (z.row_scale, out.row_scale, sd),
                               (z.col_data, out.col_data, torch.uint8), (z.col_scale, out.col_scale, sd)):
            if not want:
                continue
            if t is None or t.numel() * t.element_size() != want or not t.is_contiguous():
                raise ValueError("the planes have the sizes that fq_sizes reports, and are contiguous")
            if t.dtype != dtype:
                raise TypeError("codes are bytes, scales bytes (MX) or float32")
            given.append(t)
        copy = FqDesc.from_buffer_copy(d)  # the caller's may change
        q = FqQuantized(FqPlane(_ptr(out.row_data) if z.row_data else None, _ptr(out.row_scale) if z.row_scale else None),
                        FqPlane(_ptr(out.col_data) if z.col_data else None, _ptr(out.col_scale) if z.col_scale else None),
                        None, None)
        self.__dict__.update(out=out, rows=d.rows, cols=d.cols, _keep=given, _on=_common_gpu(*given) if given else -1,
                             _empty=not given, _d=copy, _q=q, _dref=ctypes.byref(copy), _qref=ctypes.byref(q))


_DTYPES = (torch.float32, torch.bfloat16)  # by fq_in_dtype


def _rows2(t: torch.Tensor, rows: int, cols: int, dtype: int, what: str):
    if t.dtype is not _DTYPES[dtype]:
        raise TypeError(f"{what} is of the descriptor's type")
    if t.shape != (rows, cols) or not t.is_contiguous():
        raise ValueError(f"{what} is contiguous [{rows}, {cols}]")


def _row_stride(t: torch.Tensor, rows: int, cols: int, dtype: int, what: str) -> int:
    """The row stride of a [rows, cols] tensor whose rows are each contiguous, 0 if the tensor is."""
    if t.dtype is not _DTYPES[dtype]:
        raise TypeError(f"{what} is of the descriptor's type")
    if t.shape != (rows, cols):
        raise ValueError(f"{what} is [{rows}, {cols}]")
    if t.is_contiguous():
        return 0
    step, one = t.stride()
    if one != 1 or step < cols:
        raise ValueError(f"{what}: rows are contiguous and do not overlap")
    return step


def _vector(t: Optional[torch.Tensor], n: int, dtype: int, what: str):
    if t is not None and (t.dtype is not _DTYPES[dtype] or t.numel() != n or not t.is_contiguous()):
        raise TypeError(f"{what} is contiguous, of {n} values and of its type")


def _target(planes: Optional[Planes], rows: int, cols: int, y: Optional[torch.Tensor], x: torch.Tensor) -> int:
    """The GPU of the results (x's own where there is nothing to write)."""
    if planes is None:
        if y is None:
            raise ValueError("nothing to write: neither planes nor a high-precision result")
        return y.get_device()
    if (planes.rows, planes.cols) != (rows, cols):
        raise ValueError(f"planes are of [{rows}, {cols}]")
    return x.get_device() if planes._empty else planes._on


def rmsnorm_desc(rows: int, cols: int, x_dtype: int = FQ_IN_BF16, h_dtype: int = FQ_IN_BF16,
                 weight_dtype: int = FQ_IN_F32, y_dtype: int = FQ_IN_BF16, eps: float = 1e-6,
                 accumulate: bool = False) -> FqRmsnormDesc:
    return FqRmsnormDesc(rows, cols, x_dtype, h_dtype, weight_dtype, y_dtype, int(accumulate), eps, 0)


def fq_rmsnorm(d: FqRmsnormDesc, x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
               h: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               planes: Optional[Planes] = None, stream=None):
    """h = x + residual, rstd = 1 / sqrt(mean h^2 + eps), y = h * rstd * weight, and planes of y. Without a residual
    h is x. The row stride is x's own, whatever d.x_stride holds."""
    rows, cols = d.rows, d.cols
    on = _target(planes, rows, cols, y, x)
    stride = _row_stride(x, rows, cols, d.x_dtype, "x")
    if (residual is None) != (h is None):
        raise ValueError("residual and h go together")
    if residual is not None:
        _rows2(residual, rows, cols, d.h_dtype, "residual")
        _rows2(h, rows, cols, d.h_dtype, "h")
    if y is not None:
        _rows2(y, rows, cols, d.y_dtype, "y")
    _vector(weight, cols, d.weight_dtype, "weight")
    _vector(rstd, rows, FQ_IN_F32, "rstd")
    _here(on, x, weight, residual, h, rstd, y)
    if stride != d.x_stride:  # a descriptor of this call: the caller's may be in use elsewhere
        d = FqRmsnormDesc.from_buffer_copy(d)
        d.x_stride = stride
    _check(lib().fq_rmsnorm(ctypes.byref(d), None if planes is None else planes._dref, x.data_ptr(),
                            None if residual is None else residual.data_ptr(), weight.data_ptr(),
                            None if h is None else h.data_ptr(), None if rstd is None else rstd.data_ptr(),
                            None if y is None else y.data_ptr(), None if planes is None else planes._qref,
                            _stream(stream)), "fq_rmsnorm")


def fq_rmsnorm_workspace(d: FqRmsnormDesc) -> int:
    n = ctypes.c_size_t()
    _check(lib().fq_rmsnorm_workspace(ctypes.byref(d), ctypes.byref(n)), "fq_rmsnorm_workspace")
    return n.value


def alloc_rmsnorm_workspace(d: FqRmsnormDesc, device="cuda") -> Optional[torch.Tensor]:
    n = fq_rmsnorm_workspace(d)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def fq_rmsnorm_backward(d: FqRmsnormDesc, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor,
                        dx: torch.Tensor, dweight: Optional[torch.Tensor] = None, dres: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None, stream=None):
    """dx (of x and of the residual) and dweight (fp32, += with d.accumulate) from dy and, past the norm, dres."""
    rows, cols = d.rows, d.cols
    _rows2(h, rows, cols, d.h_dtype, "h")
    _rows2(dy, rows, cols, d.y_dtype, "dy")
    _rows2(dx, rows, cols, d.h_dtype, "dx")
    if dres is not None:
        _rows2(dres, rows, cols, d.h_dtype, "dres")
    _vector(rstd, rows, FQ_IN_F32, "rstd")
    _vector(weight, cols, d.weight_dtype, "weight")
    _vector(dweight, cols, FQ_IN_F32, "dweight")
    size = _nbytes(ws)
    _here(h.get_device(), rstd, weight, dy, dx, dweight, dres, ws)
    _check(lib().fq_rmsnorm_backward(ctypes.byref(d), h.data_ptr(), rstd.data_ptr(), weight.data_ptr(), dy.data_ptr(),
                                     None if dres is None else dres.data_ptr(), dx.data_ptr(),
                                     None if dweight is None else dweight.data_ptr(),
                                     None if ws is None else ws.data_ptr(), size, _stream(stream)), "fq_rmsnorm_backward")


def swiglu_desc(rows: int, cols: int, x_dtype: int = FQ_IN_BF16, y_dtype: int = FQ_IN_BF16) -> FqSwigluDesc:
    return FqSwigluDesc(rows, cols, x_dtype, y_dtype, 0)


def _swiglu_x(d: FqSwigluDesc, x: torch.Tensor) -> FqSwigluDesc:
    stride = _row_stride(x, d.rows, 2 * d.cols, d.x_dtype, "x")
    return d if stride == d.x_stride else FqSwigluDesc(d.rows, d.cols, d.x_dtype, d.y_dtype, stride)


def fq_swiglu(d: FqSwigluDesc, x: torch.Tensor, y: Optional[torch.Tensor] = None, planes: Optional[Planes] = None,
              stream=None):
    """y = silu(gate) * up of x = [gate | up], and planes of y. The row stride is x's own."""
    on = _target(planes, d.rows, d.cols, y, x)
    if y is not None:
        _rows2(y, d.rows, d.cols, d.y_dtype, "y")
    d = _swiglu_x(d, x)
    _here(on, x, y)
    _check(lib().fq_swiglu(ctypes.byref(d), None if planes is None else planes._dref, x.data_ptr(),
                           None if y is None else y.data_ptr(), None if planes is None else planes._qref,
                           _stream(stream)), "fq_swiglu")


def fq_swiglu_backward(d: FqSwigluDesc, x: torch.Tensor, dy: torch.Tensor, dx: Optional[torch.Tensor] = None,
                       planes: Optional[Planes] = None, stream=None):
    """dx = [dgate | dup] from x = [gate | up] and dy, and planes of it. The row stride is x's own."""
    on = _target(planes, d.rows, 2 * d.cols, dx, x)
    _rows2(dy, d.rows, d.cols, d.y_dtype, "dy")
    if dx is not None:
        _rows2(dx, d.rows, 2 * d.cols, d.x_dtype, "dx")
    d = _swiglu_x(d, x)
    _here(on, x, dy, dx)
    _check(lib().fq_swiglu_backward(ctypes.byref(d), None if planes is None else planes._dref, x.data_ptr(),
                                    dy.data_ptr(), None if dx is None else dx.data_ptr(),
                                    None if planes is None else planes._qref, _stream(stream)), "fq_swiglu_backward")
