"""Plain CPU definition of the norm and of the 4-bit weight format (test
infrastructure only, numpy float64)."""

from __future__ import annotations

import numpy as np

BLOCK = 32
#: magnitudes of the codes 0 .. 7; code 8 + c is the negative of code c
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rmsnorm(r, gamma, eps):
    """(y, rstd) of rows r [T, d]."""
    rstd = 1.0 / np.sqrt(np.mean(r * r, -1) + eps)
    return r * rstd[:, None] * gamma, rstd


def rmsnorm_bwd(dy, r, gamma, rstd, dres=None):
    """(dx, dgamma) for the gradient dy of y; rstd as the forward gave it."""
    xhat = r * rstd[:, None]
    dn = dy * gamma
    dx = rstd[:, None] * (dn - xhat * np.mean(dn * xhat, -1, keepdims=True))
    return dx if dres is None else dx + dres, (dy * xhat).sum(0)


def scale_byte4(amax):
    """127 + the least e with amax <= 7 * 2^e (0 at least); 127 where amax = 0, 255 where
    it is not finite."""
    amax = np.asarray(amax, np.float64)
    fine = np.isfinite(amax)
    f, ex = np.frexp(np.where(fine, amax, 1.0) / 7.0)
    e = np.maximum(np.where(f == 0.5, ex - 1, ex) + 127, 0)
    return np.where(fine, np.where(amax == 0, 127, e), 255).astype(np.int64)


def code4(y):
    """Codes of values |y| <= 7: the nearest, on a border the even one."""
    y = np.asarray(y, np.float64)
    m = np.abs(y)
    dist = np.abs(m[..., None] - E2M1)
    near = dist == dist.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return code + 8 * np.signbit(y)


def quant4(W):
    """[..., k] -> (codes [..., k], scale bytes [..., k / 32])."""
    W = np.asarray(W, np.float64)
    b = W.reshape(W.shape[:-1] + (W.shape[-1] // BLOCK, BLOCK))
    with np.errstate(invalid="ignore"):
        byte = scale_byte4(np.where(np.isfinite(b).all(-1), np.abs(b).max(-1), np.inf))
        y = np.where((byte == 255)[..., None], 0.0, b * np.ldexp(1.0, 127 - byte)[..., None])
    return code4(y).reshape(W.shape), byte


def unpack(packed):
    """Two codes a byte, the first in the low half."""
    p = np.asarray(packed, np.int64)
    return np.stack([p & 15, p >> 4], -1).reshape(p.shape[:-1] + (2 * p.shape[-1],))


def value4(code, byte):
    """The numbers codes stand for (NaN with scale byte 255)."""
    byte = np.asarray(byte, np.int64)
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, np.minimum(byte, 254) - 127))
    code = np.asarray(code, np.int64)
    return np.where(code > 7, -1.0, 1.0) * E2M1[code & 7] * np.repeat(s, BLOCK, -1)
