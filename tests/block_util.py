"""Plain 64-bit forms of the operators of a feed-forward block on microscaled
data, and their error bounds. Nothing here uses the library."""
import numpy as np
import torch

from operator_util import E4M3, E5M2, HALF_BF16, HALF_F32, ULP32, value_table

E2M1 = 2
BITS = {E4M3: 8, E5M2: 8, E2M1: 4}


def table(fmt):
    if fmt != E2M1:
        return value_table(fmt)
    v = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return np.concatenate([v, -v])


def pack(codes, fmt):
    """Codes a byte each -> as the library holds them."""
    return codes if fmt != E2M1 else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(data, fmt):
    if fmt != E2M1:
        return data
    out = np.empty((data.shape[0], 2 * data.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = data & 15, data >> 4
    return out


def random_operand(rng, rows, k, fmt, spread=6):
    """(data, scale codes): finite codes of every magnitude, scales over 2 * spread binades."""
    t = table(fmt)
    codes = rng.integers(0, len(t), size=(rows, k)).astype(np.uint8)
    codes[~np.isfinite(t)[codes]] = 0
    return pack(codes, fmt), rng.integers(127 - spread, 127 + spread + 1, size=(rows, k // 32)).astype(np.uint8)


def values(data, scale, fmt):
    v = table(fmt)[unpack(data, fmt)]
    return v * np.repeat(np.ldexp(1.0, scale.astype(np.int64) - 127), 32, axis=1)


def product(a, sa, fa, b, sb, fb):
    """(C, S, P): the product in 64 bits, the sum of its terms' magnitudes, and the sum over runs of 128 elements
    of an upper bound of the run's largest term."""
    va, vb = values(a, sa, fa), values(b, sb, fb)
    k = va.shape[1]
    top = np.zeros((va.shape[0], vb.shape[0]))
    for i in range(0, k, 128):
        top += np.abs(va[:, i:i + 128]).max(1)[:, None] * np.abs(vb[:, i:i + 128]).max(1)[None, :]
    return va @ vb.T, np.abs(va) @ np.abs(vb).T, top


def product_bound(ref, k, fa, fb, bf16):
    """Products are exact in fp32. A run of 128 makes at most 128 additions, the sum over runs k/128, and where a
    workgroup's or a split's parts are joined as many additions again: each off by at most one unit in the last
    place of a partial sum that is at most S. For bf16 outputs with an 8-bit side the instruction aligns 128
    products before adding: each is kept to 2^-13 of the largest. Then the output's own rounding."""
    c, s, top = ref
    out = (128 + 2 * (k // 128 + 32)) * ULP32 * s
    if bf16 and not (fa == E2M1 and fb == E2M1):
        out = out + 128 * 2.0 ** -13 * top
    return out + (HALF_BF16 if bf16 else HALF_F32) * (np.abs(c) + out) + 1e-37


def product_norm_bound(ref, k, fa, fb, bf16):
    """Over the whole matrix, where the products' own errors do not add up in one direction (see operator_util)."""
    c, s, _ = ref
    wide = 2.0 ** -12 if bf16 and not (fa == E2M1 and fb == E2M1) else 0.0
    return ((HALF_BF16 if bf16 else HALF_F32) * np.linalg.norm(c)
            + (wide + (128 + 2 * (k // 128 + 32)) * ULP32) * np.linalg.norm(s) + 1e-37)


# ---------------------------------------------------------------- norm
def half(t):
    """Half a step of a result type, relative."""
    return {torch.bfloat16: HALF_BF16, torch.float32: HALF_F32}[t]


def norm(h, w, eps):
    """(rstd, y) in 64 bits of [rows, cols] h."""
    r = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return r, h * r[:, None] * w


# A row's squares are added in at most 32 steps of a thread, 6 of its wave and 16 of its waves, each off by half
# a unit relative to a sum of positive terms; mean, eps, root and quotient add four halves: the root halves all but
# the last two. Together below 32 halves; two products follow.
RSTD_REL = 32 * 2.0 ** -24
Y_REL = RSTD_REL + 2 * 2.0 ** -24


def norm_gradients(h, r, w, dy, dres):
    """(dx, dw, bound of dx, bound of dw) in 64 bits; r is the given rstd. Bounds without the output's rounding:
    z, g and their product carry three halves; the mean of g z is added in at most 54 steps (as above) and divided;
    dx takes three more operations on terms of these magnitudes. dw adds at most rows / 1024 + 1 terms a workgroup,
    then 128 and 32 of partial sums."""
    n = h.shape[1]
    z, g = h * r[:, None], dy * w
    mean = (g * z).sum(1, keepdims=True) / n
    mag = (np.abs(g * z)).sum(1, keepdims=True) / n
    dx = r[:, None] * (g - z * mean) + dres
    bx = (r[:, None] * (4 * np.abs(g) + 6 * np.abs(z * mean) + 60 * np.abs(z) * mag) + 2 * np.abs(dres)) * 2.0 ** -24
    dw = (dy * z).sum(0)
    bw = (h.shape[0] // 1024 + 170) * 2.0 ** -24 * np.abs(dy * z).sum(0)
    return dx, dw, bx + 1e-37, bw + 1e-37


# ---------------------------------------------------------------- gated activation
def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g < 0, e, 1.0) / (1.0 + e)


def swiglu(gate, up):
    """(y, bound). exp(-|g|) in base 2: the exponent's rounding 2^-24 |g| log2(e), worth 2^-24 |g| relative, a unit
    each for the exponential and the reciprocal, halves for 1 + e, e q and the two products: below 8 units.
    Magnitudes below 2^-126 may be zero on the way: exp(-|g|) below that is a zero."""
    y = gate * sigmoid(gate) * up
    return y, (np.abs(gate) * 2.0 ** -24 + 8 * ULP32) * np.abs(y) + 2.0 ** -125 * (1 + np.abs(gate * up))


def swiglu_gradients(gate, up, dy):
    """(dgate, dup, bound, bound)."""
    s, rest = sigmoid(gate), sigmoid(-gate)
    rel = np.abs(gate) * 2.0 ** -24 + 8 * ULP32
    dg = dy * up * s * (1 + gate * rest)
    # 1 + g (1 - s): the product is off by rel of itself, the sum by half a unit
    bg = np.abs(dy * up * s) * (rel * (1 + 2 * np.abs(gate * rest)) + 2 * ULP32)
    du = dy * gate * s
    tiny = 2.0 ** -125 * (1 + np.abs(dy * up) * (1 + np.abs(gate)) + np.abs(dy * gate))
    return dg, du, bg + tiny, rel * np.abs(du) + tiny
