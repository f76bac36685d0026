"""Layer norm and microscaled 4-bit values in float64.

Test infrastructure only: nothing in the package imports this, and it shares no code with the
library.  The definitions are include/ss.h's.
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def ln_fwd(x, w, b=None, res=None, eps=1e-5):
    r = x if res is None else x + res
    d = r - r.mean(-1, keepdims=True)
    y = d / np.sqrt(np.square(d).mean(-1, keepdims=True) + eps) * w
    return (y if b is None else y + b), r


def ln_bwd(dy, r, w, dr=None, eps=1e-5):
    d = r - r.mean(-1, keepdims=True)
    c = 1.0 / np.sqrt(np.square(d).mean(-1, keepdims=True) + eps)
    n, wdy = d * c, dy * w
    dx = c * (wdy - wdy.mean(-1, keepdims=True) - n * (wdy * n).mean(-1, keepdims=True))
    return (dx if dr is None else dx + dr), (dy * n).sum(0), dy.sum(0)


def mx4_quant(x):
    """codes [.., K] (one a place) and stored exponents [.., K / 32]."""
    v = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    top = np.abs(v).max(-1)
    bad = ~np.isfinite(v).all(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(top > 0, np.floor(np.log2(np.where(bad, 1.0, top))), -200.0)
    # log2 rounds: the power of two below or at the value, exactly
    e = np.where(np.where(bad, 1.0, top) < 2.0 ** e, e - 1, e)
    e = np.where(np.where(bad, 1.0, top) >= 2.0 ** (e + 1), e + 1, e)
    e = np.maximum(e - 2 + 127, 1).astype(np.int64)
    with np.errstate(invalid="ignore"):
        m = np.abs(np.where(bad[..., None], 0.0, v)) / 2.0 ** (e - 127.0)[..., None]
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.zeros(m.shape, np.int64)
    for n, x in enumerate(mid):     # a tie goes up where the code above is even
        code += (m >= x) if n % 2 else (m > x)
    code |= np.where(np.signbit(v), 8, 0)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x_shape(v)), np.where(bad, 255, e)


def x_shape(v):
    return (*v.shape[:-2], v.shape[-2] * 32)


def mx4_values(code, e):
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    scale = np.where(e == 255, np.nan, 2.0 ** (e - 127.0))
    return v * np.repeat(scale, 32, -1)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    c = np.empty((*b.shape[:-1], 2 * b.shape[-1]), np.int64)
    c[..., 0::2], c[..., 1::2] = b & 15, b >> 4
    return c
