"""Plain 64-bit forms of the operators on 8-bit data, on the CPU, and their
error bounds. Nothing here uses the library."""
import numpy as np
import torch

E4M3, E5M2 = 0, 1
F8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
FMAX = {E4M3: 448.0, E5M2: 57344.0}
ULP32 = 2.0 ** -23          # one unit in the last place of an fp32 sum, relative
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_F32 = torch.finfo(torch.float32).eps / 2


def value_table(fmt: int) -> np.ndarray:
    """The 256 values of a format, from sign, exponent and mantissa fields (NaN codes as NaN)."""
    man, bias, top = (3, 7, 15) if fmt == E4M3 else (2, 15, 31)
    out = np.zeros(256)
    for c in range(256):
        e, m = (c & 127) >> man, c & ((1 << man) - 1)
        v = (m / (1 << man) + 1.0) * 2.0 ** (e - bias) if e else m / (1 << man) * 2.0 ** (1 - bias)
        if fmt == E4M3 and (c & 127) == 127:
            v = np.nan
        if fmt == E5M2 and e == top:
            v = np.inf if m == 0 else np.nan
        out[c] = -v if c & 128 else v
    return out


def decode(codes, fmt=E4M3) -> np.ndarray:
    return value_table(fmt)[np.asarray(codes, dtype=np.uint8)]


def encode(x: np.ndarray, fmt=E4M3) -> np.ndarray:
    """Codes of 64-bit values within the format's range: to nearest, ties to even."""
    man, low = (3, -6) if fmt == E4M3 else (2, -14)
    a = np.abs(x)
    e = np.maximum(np.where(a > 0, np.frexp(a)[1] - 1, low), low)
    steps = np.rint(np.ldexp(a, man - e)).astype(np.int64)
    code = steps + ((e - low) << man)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


# ---------------------------------------------------------------- matrix product
def random_codes(rng, shape, fmt=E4M3) -> np.ndarray:
    """Finite codes of every magnitude."""
    c = rng.integers(0, 256, size=shape, dtype=np.uint8)
    bad = ~np.isfinite(value_table(fmt))[c]
    c[bad] = 0
    return c


def random_scales(rng, shape, pow2=False) -> np.ndarray:
    e = rng.integers(-12, 3, size=shape)
    s = np.ldexp(1.0, e)
    if not pow2:
        s = s * rng.uniform(1.0, 2.0, size=shape)
    return s.astype(np.float32)


def product(a, sa, b, sb, b_rows):
    """(C, S, P): the product in 64 bits, the sum of its terms' magnitudes, and
    the sum over blocks of a block's largest term's magnitude."""
    m, k = a.shape
    n = b.shape[0]
    nb = k // 128
    va = (decode(a).reshape(m, nb, 128) * sa.astype(np.float64)[:, :, None]).reshape(m, k)
    s = sb.astype(np.float64) if b_rows == 1 else np.repeat(sb.astype(np.float64), 128, axis=0)
    vb = (decode(b).reshape(n, nb, 128) * s[:, :, None]).reshape(n, k)
    top = np.zeros((m, n))
    for i in range(nb):
        cut = slice(128 * i, 128 * i + 128)
        # an upper bound of the largest term: the row's largest value times the column's
        top += np.abs(va[:, cut]).max(1)[:, None] * np.abs(vb[:, cut]).max(1)[None, :]
    return va @ vb.T, np.abs(va) @ np.abs(vb).T, top


def product_bound(c, s, top, k, bf16):
    """Products of two 8-bit values are exact in fp32. A block's sum makes at
    most 128 additions, its scaling two products, the sum over blocks k/128
    fused steps and, where a workgroup's or a split's parts are joined, as
    many additions again: each off by at most one unit in the last place of a
    partial sum that is at most s. For bf16 outputs the 8-bit instruction
    aligns a block's products before adding: each is kept to 2^-13 of the
    largest, 128 of them. Then the output's own rounding."""
    out = (128 + 2 + 2 * (k // 128 + 32)) * ULP32 * s
    if bf16:
        out = out + 128 * 2.0 ** -13 * top
    return out + (HALF_BF16 if bf16 else HALF_F32) * (np.abs(c) + out) + 1e-37


def product_norm_bound(c, s, k, bf16):
    """The same over the whole matrix, where the products' own errors do not add
    up in one direction: the mean-square error of 128 values each off by up to
    2^-13 of the largest is below 2^-13 * sqrt(128) / 3 of it, below 2^-12 of
    the sum of the magnitudes."""
    out = (HALF_BF16 if bf16 else HALF_F32) * np.linalg.norm(c)
    return out + ((2.0 ** -12 if bf16 else 0.0) + (128 + 2 + 2 * (k // 128 + 32)) * ULP32) * np.linalg.norm(s) + 1e-37


# ---------------------------------------------------------------- cache
def scale_of(a, fmt):
    """The smallest power of two of at least 2^-126 with a <= Fmax * s."""
    p = -126
    while a > FMAX[fmt] * 2.0 ** p:
        p += 1
    return 2.0 ** p


class PlainCache:
    """The cache of one call in plain form: what the library's buffers should hold."""

    def __init__(self, fmt, pages, heads, dim, page, block, rng):
        self.fmt, self.pages, self.heads, self.dim, self.page, self.block = fmt, pages, heads, dim, page, block
        # whatever an earlier user left, NaN codes and scales among it
        self.k = rng.integers(0, 256, size=(pages, heads, page, dim), dtype=np.uint8)
        self.v = rng.integers(0, 256, size=(pages, heads, dim, page), dtype=np.uint8)
        self.ks = rng.choice(np.array([np.nan, np.inf, 1.0, 0.0, -3.0], np.float32), size=(pages, heads, page // block))
        self.vs = rng.choice(np.array([np.nan, np.inf, 1.0, 0.0, -3.0], np.float32), size=(pages, heads, page // block))

    def copy(self):
        c = object.__new__(PlainCache)
        c.__dict__ = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in self.__dict__.items()}
        return c

    def append(self, table, length, k_new, v_new):
        """k_new, v_new [rows, heads, dim] (64-bit values of the inputs) at positions length - rows .. length - 1."""
        n = k_new.shape[0]
        first = length - n
        start = max(first, 0)
        if length <= 0:
            return
        for b in range(start // self.block, (length - 1) // self.block + 1):
            lo, hi = max(b * self.block, start), min((b + 1) * self.block, length)
            if lo >= hi:
                continue
            page = table[b * self.block // self.page]
            if not 0 <= page < self.pages:
                continue
            inner = b * self.block % self.page
            for new, codes, scales in ((k_new, self.k[page], self.ks[page]),
                                       (v_new, self.v[page].transpose(0, 2, 1), self.vs[page])):
                for h in range(self.heads):
                    x = new[lo - first:hi - first, h]
                    s = scale_of(np.abs(x).max(), self.fmt)
                    old = codes[h, inner:inner + lo - b * self.block]
                    if lo > b * self.block:
                        was = float(scales[h, inner // self.block])
                        if s > was:
                            old[...] = encode(decode(old, self.fmt) * (was / s), self.fmt)
                        s = max(s, was)
                    codes[h, inner + lo - b * self.block:inner + hi - b * self.block] = encode(x / s, self.fmt)
                    scales[h, inner // self.block] = s

    def values(self, table, length, h):
        """(K, V) [length, dim] of one sequence and head, and which tokens are present."""
        k, v = np.zeros((length, self.dim)), np.zeros((length, self.dim))
        there = np.zeros(length, bool)
        for t0 in range(0, length, self.block):
            page = table[t0 // self.page]
            if not 0 <= page < self.pages:
                continue
            i, n = t0 % self.page, min(self.block, length - t0)
            k[t0:t0 + n] = decode(self.k[page, h, i:i + n], self.fmt) * float(self.ks[page, h, i // self.block])
            v[t0:t0 + n] = decode(self.v[page, h, :, i:i + n].T, self.fmt) * float(self.vs[page, h, i // self.block])
            there[t0:t0 + n] = True
        return k, v, there


def attention_row(q, k, v, see, scale, softcap):
    """One row in 64 bits: (out, lse, error bound of out, error bound of lse).

    Bounds. A score is a sum of dim exact products (bf16 x 8-bit) in fp32:
    off by at most dim + 4 units of the sum of their magnitudes; the base-2
    exponential adds two units of its argument's magnitude and two of its own;
    tanh by way of an exponential of 2 y adds at most 8 units of the cap. So a
    probability is off by a factor 1 + e, and after normalization by 2 e.
    Rounding p to bf16 is off by half a step of each term, the output by half
    a step of the result; fp32 sums of up to len terms by len units."""
    dim = q.shape[0]
    if not see.any():
        return np.zeros(dim), -np.inf, np.zeros(dim), 0.0
    k, v = k[see], v[see]
    s = k @ q * scale
    mag = (np.abs(k) @ np.abs(q)).max() * abs(scale)
    eps = (dim + 4) * ULP32 * mag
    if softcap:
        s = softcap * np.tanh(s / softcap)
        eps += 8 * ULP32 * softcap
    eps += 2 * 1.5 * np.abs(s).max() * 2 * ULP32 + 4 * ULP32
    top = s.max()
    p = np.exp(s - top)
    z = p.sum()
    lse = top + np.log(z)
    o = p @ v / z
    w = p @ np.abs(v) / z
    n = int(see.sum())
    sums = (n / 16 + 64) * ULP32     # additions a term goes through: its step's, its wave's, its split's
    bound = (HALF_BF16 + 2 * eps + 2 * sums) * w
    bound = bound + HALF_BF16 * (np.abs(o) + bound) + 1e-30
    return o, lse, bound, eps + sums + 4 * ULP32 * (abs(lse) + abs(top) + 1.0)
