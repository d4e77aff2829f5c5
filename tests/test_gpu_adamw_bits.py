"""moe_adamw bit for bit against its formula evaluated in float32, one operation after
another (include/moe.h): every product, sum, root and quotient rounded to nearest, the
constants formed in float64 and rounded once, 8-bit states from the rounded results
with the stated random numbers.  No tolerance."""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from oracle import fp8_oracle as Q
from test_gpu_adamw import HP, make

pytestmark = pytest.mark.gpu

f32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def _np(t):
    return t.float().cpu().numpy()


def _state(t):
    n = t["param"].numel()
    if "m_s" not in t:
        return _np(t["m"]), _np(t["v"])
    m, r = [_np(t[k]) * np.repeat(np.ldexp(f32(1), t[k + "_s"].cpu().numpy().astype(int) - 127),
                                  128)[:n] for k in ("m", "v")]
    return m, r * r


def _codes(x, rnd, least):
    """(e4m3 codes, scale bytes) of float32 x."""
    n = x.size
    byte = Q.scale_byte(np.abs(np.concatenate([x, np.zeros(-n % 128, f32)])).reshape(-1, 128).max(1))
    y = x * np.repeat(np.ldexp(f32(1), 127 - byte), 128)[:n]
    mag = np.abs(y)
    normal = ((mag.view(np.int32).astype(np.int64) + rnd) >> 20) - 960
    small = np.floor(mag * f32(512) + rnd.astype(f32) * f32(2.0 ** -20)).astype(np.int64)
    code = np.where(mag >= f32(2.0 ** -6), normal, small)
    if least:
        code = np.where(mag > 0, np.maximum(code, 1), code)
    return (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8), byte.astype(np.uint8)


def _expected(t, index, step, scale, seed):
    b1, b2, lr = HP["beta1"], HP["beta2"], HP["lr"]
    m, v = _state(t)
    p = _np(t["param"] if t["master"] is None else t["master"])
    g = _np(t["grad"]) * f32(scale)
    m = m * f32(b1) + g * f32(1 - b1)
    v = v * f32(b2) + (g * g) * f32(1 - b2)
    r = np.sqrt(v)
    stp = m * f32(lr / (1 - b1 ** step)) / (r * f32(1 / np.sqrt(1 - b2 ** step)) + f32(HP["eps"]))
    p = p * f32(1 - lr * float(f32(t["weight_decay"]))) - stp
    out = {"param": torch.from_numpy(p).to(t["param"].dtype)}
    if t["master"] is not None:
        out["master"] = torch.from_numpy(p)
    if "m_s" not in t:
        return out | {"m": torch.from_numpy(m), "v": torch.from_numpy(v)}
    bits = Q.random_bits(p.size, index, seed, step)
    for k, x, rnd, least in (("m", m, bits[0], False), ("v", r, bits[1], True)):
        code, byte = _codes(x, rnd, least)
        out[k], out[k + "_s"] = torch.from_numpy(code), torch.from_numpy(byte)
    return out


def _same(got, want):
    got, want = got.cpu().contiguous(), want.contiguous()
    return torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_bit_for_bit(dtype, bits, master):
    ts = [make(n, dtype, bits, master, 40 + i, off=i % 5)
          for i, n in enumerate([1, 7, 8, 127, 129, 2047, 2048, 2049, 30001])]
    ta = M.AdamWTensors(ts)
    for step in (1, 2, 1000):
        want = [_expected(t, i, step, 0.5, 7) for i, t in enumerate(ts)]
        M.moe_adamw(ta, step=step, grad_scale=0.5, seed=7, **HP)
        for i, (t, w) in enumerate(zip(ts, want)):
            for k, x in w.items():
                assert _same(t[k], x), (step, i, k)
