"""Plain CPU definition of the 8-bit expert path and of the AdamW step (test
infrastructure only, numpy float64).

A quantised matrix is e4m3 values with one power-of-two scale per 128 values;
functions here return both the values in the block's units and the biased scale
exponents ("bytes"), and ``value`` gives the numbers they stand for.
"""

from __future__ import annotations

import numpy as np

from .moe_oracle import store

BLOCK = 128


def round_e4m3(y) -> np.ndarray:
    """Nearest e4m3 value, ties to even: spacing 2^(e - 3) for |y| in
    [2^e, 2^(e+1)), the fixed 2^-9 below 2^-6.  |y| <= 448; not finite -> NaN."""
    y = np.asarray(y, np.float64)
    with np.errstate(invalid="ignore"):
        _, ex = np.frexp(np.where(np.isfinite(y), y, 0.0))
        step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
        r = np.rint(y / step) * step
    return np.where(np.isfinite(y), r, np.nan)


def scale_byte(amax) -> np.ndarray:
    """127 + the least e with amax <= 448 * 2^e (0 at least); 127 where amax = 0."""
    f, ex = np.frexp(np.asarray(amax, np.float64) / 448.0)
    e = np.where(f == 0.5, ex - 1, ex)
    return np.where(np.asarray(amax) == 0, 127, np.maximum(e + 127, 0)).astype(np.int64)


def _amax(b, axis):
    return np.where(np.isfinite(b), np.abs(b), 0.0).max(axis)


def quant_rows(x):
    """[..., k] -> (e4m3 values [..., k], scale bytes [..., k / 128])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // BLOCK, BLOCK))
    byte = scale_byte(_amax(b, -1))
    with np.errstate(invalid="ignore"):
        q = round_e4m3(b * np.ldexp(1.0, 127 - byte)[..., None])
    return q.reshape(x.shape), byte


def quant_weights(W):
    """[E, n, k] -> (e4m3 values [E, n, k], scale bytes [E, n / 128, k / 128])."""
    W = np.asarray(W, np.float64)
    E, n, k = W.shape
    b = W.reshape(E, n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    byte = scale_byte(_amax(b, (2, 4)))
    with np.errstate(invalid="ignore"):
        q = round_e4m3(b * np.ldexp(1.0, 127 - byte)[:, :, None, :, None])
    return q.reshape(E, n, k), byte


def value(q, byte, rows=1):
    """The numbers quantised values stand for; rows = 128 for weights."""
    s = np.ldexp(1.0, np.asarray(byte, np.int64) - 127)
    if rows > 1:
        s = np.repeat(s, rows, -2)
    return np.asarray(q, np.float64) * np.repeat(s, BLOCK, -1)


def requant(x):
    return value(*quant_rows(x))


def silu(g):
    return g / (1.0 + np.exp(-g))


def ffn_fwd_fp8(x, offsets, W_gu, W_down, quant=True):
    """Rows x [N, d] (the numbers the quantised rows stand for), weights likewise:
    {"g", "u", "a", "y"}, nothing rounded but the quantised a (quant=False: not
    even that)."""
    N, F = x.shape[0], W_down.shape[2]
    out = {"g": np.zeros((N, F)), "u": np.zeros((N, F)), "a": np.zeros((N, F)),
           "y": np.zeros((N, W_down.shape[1]))}
    for e in range(W_gu.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        h = x[r] @ W_gu[e].T
        g, u = h[:, :F], h[:, F:]
        a = silu(g) * u
        out["g"][r], out["u"][r], out["a"][r] = g, u, a
        out["y"][r] = (requant(a) if quant and a.size else a) @ W_down[e].T
    return out


def swiglu_bwd(da, g, u):
    s = 1.0 / (1.0 + np.exp(-g))
    return da * u * s * (1.0 + g * (1.0 - s)), da * g * s


def ffn_dgrad_fp8(d, gate, h, offsets, W_gu, W_down, quant=True):
    """Rows d [N, d] of the output gradient, gate [N] (or 1.0), stored h [N, 2F]:
    {"da", "dh", "dx", "ag"} with dh quantised before the second product."""
    N, F = d.shape[0], W_down.shape[2]
    gate = np.broadcast_to(np.asarray(gate, np.float64), (N,))[:, None]
    g, u = h[:, :F], h[:, F:]
    da, dx = np.zeros((N, F)), np.zeros((N, W_down.shape[1]))
    dh = np.zeros((N, 2 * F))
    for e in range(W_gu.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        da[r] = gate[r] * (d[r] @ W_down[e])
        dh[r] = np.concatenate(swiglu_bwd(da[r], g[r], u[r]), 1)
        dx[r] = (requant(dh[r]) if quant and dh[r].size else dh[r]) @ W_gu[e]
    return {"da": da, "dh": dh, "dx": dx, "ag": gate * silu(g) * u}


# ----------------------------------------------------------------------------
# AdamW
# ----------------------------------------------------------------------------
def _u32(x):
    return np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)


def _mul(a, c):
    return _u32(_u32(a) * np.uint64(c))


def random_bits(n, index, seed, step):
    """The two 20-bit numbers of every element of tensor `index`."""
    key = ((seed & 0xFFFFFFFF) ^ ((seed >> 32) * 0x85EBCA77 & 0xFFFFFFFF)
           ^ (step * 0x9E3779B1 & 0xFFFFFFFF) ^ (index * 0xC2B2AE3D & 0xFFFFFFFF))
    x = np.arange(n, dtype=np.uint64) ^ np.uint64(key)
    x = _mul(x ^ (x >> np.uint64(16)), 0x9E3779B1)
    x = _mul(x ^ (x >> np.uint64(15)), 0xC2B2AE3D)
    x = x ^ (x >> np.uint64(16))
    return ((x >> np.uint64(12)).astype(np.int64),
            (_mul(x, 0x9E3779B1) >> np.uint64(12)).astype(np.int64))


def quant_random(x, rnd, least=False):
    """[n] -> (values, bytes): blocks of 128, rounded up with probability rnd /
    2^20's share of the step: floor(|y| / step + rnd 2^-20) steps.  least: what is
    not zero is at least one step, as the second moment's root is stored."""
    n = x.size
    pad = np.concatenate([x, np.zeros(-n % BLOCK)]).reshape(-1, BLOCK)
    byte = scale_byte(_amax(pad, 1))
    with np.errstate(invalid="ignore"):
        y = (pad * np.ldexp(1.0, 127 - byte)[:, None]).reshape(-1)[:n]
        _, ex = np.frexp(np.where(np.isfinite(y), y, 0.0))
        step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
        q = np.floor(np.abs(y) / step + rnd * 2.0 ** -20) * step
        if least:
            q = np.where(np.abs(y) > 0, np.maximum(q, 2.0 ** -9), q)
        q = np.copysign(q, y)
    return np.where(np.isfinite(y), q, np.nan), byte


def adamw(p, grad, m, v, lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0):
    """(p, m, v) after one step."""
    g = grad_scale * grad
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = (1 - lr * weight_decay) * p - lr / (1 - beta1 ** step) * m / (
        np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p, m, v


__all__ = ["BLOCK", "round_e4m3", "scale_byte", "quant_rows", "quant_weights", "value", "requant",
           "silu", "ffn_fwd_fp8", "swiglu_bwd", "ffn_dgrad_fp8", "random_bits", "quant_random",
           "adamw", "store"]
