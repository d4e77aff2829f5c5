"""The 8-bit expert path and the AdamW step without a GPU: pins of the oracle's
definitions, and every refusal of the entry points (no call here reaches a
launch)."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from oracle import fp8_oracle as Q

FAKE = C.c_void_p(0x1000)
ODD = C.c_void_p(0x1001)


# ---- the oracle -------------------------------------------------------------
def test_e4m3_rounding_against_torch():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(size=4000) * 2.0 ** -8,
                        [0.0, -0.0, 448, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0,
                         2.0 ** -6, 416.0, 432.0]]).astype(np.float32)
    t = torch.from_numpy(y).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(Q.round_e4m3(y), t)
    assert np.isnan(Q.round_e4m3([np.nan, np.inf, -np.inf])).all()
    # every e4m3 value is its own rounding
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    codes = codes[np.isfinite(codes)]
    assert np.array_equal(Q.round_e4m3(codes), codes)


@pytest.mark.parametrize("amax,byte", [
    (0.0, 127), (448.0, 127), (449.0, 128), (224.0, 126), (1.75, 119), (1.7500001, 120),
    (1.0, 119), (2.0 ** -130, 0), (float(np.finfo(np.float32).max), 247)])
def test_scale_closed_forms(amax, byte):
    assert Q.scale_byte(amax) == byte
    if byte:
        assert amax <= 448 * math.ldexp(1, byte - 127)


def test_quantisation_error_is_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(64, 384)) * np.exp(rng.normal(size=(64, 1)) * 3)
    q, b = Q.quant_rows(x)
    assert np.abs(q).max() <= 448 and (np.abs(q.reshape(64, 3, 128)).max(2) >= 224).all()
    err = np.abs(Q.value(q, b) - x)
    # half a step: 2^-4 of the value, or 2^-10 of the scale in the flat range
    floor = np.repeat(np.ldexp(1.0, b - 127), 128, -1) * 2.0 ** -10
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, floor) * (1 + 1e-12)).all()


def test_dgrad_definition_against_differences():
    """Without quantisation the dgrad is the derivative of <dout, y> by x."""
    rng = np.random.default_rng(2)
    off = np.array([0, 3, 3, 7])
    x = rng.normal(size=(7, 128))
    W_gu, W_down = rng.normal(size=(3, 256, 128)) * 0.1, rng.normal(size=(3, 128, 128)) * 0.1
    d, gate = rng.normal(size=(7, 128)), rng.uniform(0.2, 1, 7)
    f = Q.ffn_fwd_fp8(x, off, W_gu, W_down, quant=False)
    h = np.concatenate([f["g"], f["u"]], 1)
    got = Q.ffn_dgrad_fp8(d, gate, h, off, W_gu, W_down, quant=False)["dx"]
    loss = lambda z: (gate[:, None] * d * Q.ffn_fwd_fp8(z, off, W_gu, W_down, quant=False)["y"]).sum()
    for _ in range(6):
        v = rng.normal(size=x.shape)
        diff = (loss(x + 1e-5 * v) - loss(x - 1e-5 * v)) / 2e-5
        # second differences: O(1e-10) of the third derivative, 1e-16 / 1e-5 of rounding
        assert abs(diff - (got * v).sum()) <= 1e-7 * max(1.0, np.abs(got * v).sum())


def test_random_rounding_has_the_right_mean():
    n = 128 * 400
    bits, other = Q.random_bits(n, 3, (5 << 32) + 9, 17)
    assert bits.min() >= 0 and bits.max() < 1 << 20 and other.max() < 1 << 20
    # uniform: mean within 5 standard errors of the middle, and the two uncorrelated
    for b in (bits, other):
        assert abs(b.mean() / 2 ** 20 - 0.5) < 5 / math.sqrt(12 * n)
    assert abs(np.corrcoef(bits, other)[0, 1]) < 5 / math.sqrt(n)
    x = np.full(n, 17.3)
    x[::128] = 300.0  # the scale is 1: 17.3 lies between 16 and 18
    q, byte = Q.quant_random(x, bits)
    assert (byte == 127).all()
    inner = np.delete(q, np.s_[::128])
    assert set(np.unique(inner)) == {16.0, 18.0}
    assert abs(inner.mean() - 17.3) < 5 * 1.0 / math.sqrt(inner.size)


def test_adamw_definition_against_torch():
    rng = np.random.default_rng(3)
    p = torch.tensor(rng.normal(size=50), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    x, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.normal(size=50)
        p.grad = torch.tensor(g)
        opt.step()
        x, m, v = Q.adamw(x, g, m, v, 1e-2, 0.9, 0.95, 1e-8, 0.1, t)
        assert np.allclose(x, p.detach().numpy(), rtol=1e-12, atol=1e-14)


# ---- refusals ---------------------------------------------------------------
def _shape(**kw):
    base = dict(T=64, d=256, F=128, E=8, e_lo=0, E_l=8, K=2, dtype="bf16")
    base.update(kw)
    return M.make_shape(**base)


def _weights(**kw):
    f = {n: 0x1000 for n in M.FP8_WEIGHT_FIELDS}
    f.update(kw)
    return M.MoeFp8Weights(*[f[n] for n in M.FP8_WEIGHT_FIELDS])


def _fwd(s, xq=FAKE, xs=FAKE, pr=None, off=FAKE, to=FAKE, w=None, h=FAKE, a=FAKE, yp=FAKE, ws=FAKE,
         nb=1 << 40):
    w = _weights() if w is None else w
    return M.lib().moe_expert_ffn_fwd_fp8(C.byref(s), xq, xs, pr, off, to, C.byref(w), h, a, yp,
                                          ws, nb, None)


def _bwd(s, dq=FAKE, ds=FAKE, pr=None, gates=None, h=FAKE, off=FAKE, to=FAKE, w=None, dh=FAKE,
         dxp=FAKE, ag=None, ws=FAKE, nb=1 << 40):
    w = _weights() if w is None else w
    return M.lib().moe_ffn_dgrad_fp8(C.byref(s), dq, ds, pr, gates, h, off, to, C.byref(w), dh,
                                     dxp, ag, ws, nb, None)


def test_scale_ld_and_workspace():
    assert [M.moe_fp8_scale_ld(k) for k in (128, 512, 640, 2048, 16384)] == [4, 4, 8, 16, 128]
    s = _shape()
    assert M.moe_fp8_workspace_bytes(s) >= 128 * (2 * 128 + 4)
    assert M.moe_fp8_workspace_bytes(_shape(T=0)) > 0
    assert M.moe_fp8_workspace_bytes(_shape(d=192)) == 0
    assert _fwd(s, nb=M.moe_fp8_workspace_bytes(s) - 1) == M.MOE_ERR_WORKSPACE
    assert _bwd(s, nb=16) == M.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("kw", [dict(d=192), dict(F=64), dict(F=192), dict(d=64)])
def test_sizes_must_be_whole_blocks(kw):
    s = _shape(**kw)
    assert _fwd(s) == M.MOE_ERR_SHAPE and b"128" in M.lib().moe_last_error()
    assert _bwd(s) == M.MOE_ERR_SHAPE
    assert M.lib().moe_quant_rows_fp8(C.byref(s), FAKE, 4, None, FAKE, FAKE, None) == M.MOE_ERR_SHAPE
    w = _weights()
    assert M.lib().moe_quant_weights_fp8(C.byref(s), FAKE, FAKE, C.byref(w),
                                         None) == M.MOE_ERR_SHAPE


def test_products_need_16_bit_data():
    s = _shape(dtype="f32")
    assert _fwd(s) == M.MOE_ERR_UNSUPPORTED
    assert _bwd(s) == M.MOE_ERR_UNSUPPORTED
    # shape errors come first
    assert _fwd(_shape(dtype=9)) == M.MOE_ERR_DTYPE


def test_null_pointers():
    s = _shape()
    for n in ("xq", "xs", "off", "to", "yp", "ws"):
        assert _fwd(s, **{n: None}) == M.MOE_ERR_NULL, n
    for n in ("dq", "ds", "h", "off", "to", "dh", "dxp", "ws"):
        assert _bwd(s, **{n: None}) == M.MOE_ERR_NULL, n
    for n in ("gu", "gu_s", "down", "down_s"):
        assert _fwd(s, w=_weights(**{n: None})) == M.MOE_ERR_NULL, n
    for n in ("guT", "guT_s", "downT", "downT_s"):
        assert _bwd(s, w=_weights(**{n: None})) == M.MOE_ERR_NULL, n
    L = M.lib()
    assert L.moe_quant_rows_fp8(C.byref(s), None, 4, None, FAKE, FAKE, None) == M.MOE_ERR_NULL
    assert L.moe_quant_rows_fp8(C.byref(s), FAKE, -1, None, FAKE, FAKE, None) == M.MOE_ERR_SHAPE
    assert L.moe_quant_rows_fp8(C.byref(s), FAKE, 1 << 31, None, FAKE, FAKE,
                                None) == M.MOE_ERR_SHAPE
    # some of the transposed copies
    assert L.moe_quant_weights_fp8(C.byref(s), FAKE, FAKE, C.byref(_weights(downT=None)),
                                   None) == M.MOE_ERR_NULL
    assert L.moe_quant_weights_fp8(C.byref(s), FAKE, FAKE, None, None) == M.MOE_ERR_NULL


def test_gather_arguments():
    s = _shape()
    assert _bwd(s, pr=FAKE) == M.MOE_ERR_NULL             # gates missing
    assert _bwd(s, gates=FAKE) == M.MOE_ERR_ARG           # gates without the plan
    assert _bwd(s, ag=FAKE) == M.MOE_ERR_ARG
    big = _shape(T=1 << 23, d=256, K=2)                   # T * d = 2^31
    assert _fwd(big, pr=FAKE) == M.MOE_ERR_SHAPE
    assert _bwd(big, pr=FAKE, gates=FAKE) == M.MOE_ERR_SHAPE


def test_alignment():
    s = _shape()
    for n in ("xq", "xs", "h", "a", "yp", "ws"):
        assert _fwd(s, **{n: ODD}) == M.MOE_ERR_ARG, n
    for n in ("dq", "ds", "h", "dh", "dxp", "ws"):
        assert _bwd(s, **{n: ODD}) == M.MOE_ERR_ARG, n
    assert _bwd(s, pr=FAKE, gates=FAKE, ag=ODD) == M.MOE_ERR_ARG
    assert _fwd(s, w=_weights(gu=0x1004)) == M.MOE_ERR_ARG
    assert _fwd(s, w=_weights(gu_s=0x1002)) == M.MOE_ERR_ARG
    assert M.lib().moe_quant_rows_fp8(C.byref(s), ODD, 4, None, FAKE, FAKE, None) == M.MOE_ERR_ARG


def _adam(n=1, hp=None, **kw):
    t = dict(n=8, param=0x1000, master=None, grad=0x1000, m=0x1000, v=0x1000, m_s=None, v_s=None,
             dtype=M.MOE_BF16, state8=0, weight_decay=0.0, reserved=0)
    t.update(kw)
    h = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, seed=0, grad_scale_dev=None,
             grad_scale=1.0, reserved=0)
    h.update(hp or {})
    return M.lib().moe_adamw(C.byref(M.MoeAdamwTensor(**t)), n, C.byref(M.MoeAdamwHyper(**h)),
                             None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), M.MOE_ERR_SHAPE), (dict(hp=dict(beta1=1.0)), M.MOE_ERR_ARG),
    (dict(hp=dict(beta2=-0.1)), M.MOE_ERR_ARG), (dict(hp=dict(eps=0.0)), M.MOE_ERR_ARG),
    (dict(hp=dict(eps=1e-60)), M.MOE_ERR_ARG), (dict(hp=dict(lr=math.nan)), M.MOE_ERR_ARG),
    (dict(hp=dict(beta1=math.nan)), M.MOE_ERR_ARG), (dict(hp=dict(step=0)), M.MOE_ERR_ARG),
    (dict(hp=dict(grad_scale=math.inf)), M.MOE_ERR_ARG), (dict(hp=dict(reserved=1)), M.MOE_ERR_ARG),
    (dict(hp=dict(grad_scale_dev=0x1002)), M.MOE_ERR_ARG),
    (dict(dtype=5), M.MOE_ERR_DTYPE), (dict(state8=2), M.MOE_ERR_ARG),
    (dict(reserved=3), M.MOE_ERR_ARG), (dict(weight_decay=math.inf), M.MOE_ERR_ARG),
    (dict(param=None), M.MOE_ERR_NULL), (dict(grad=None), M.MOE_ERR_NULL),
    (dict(m=None), M.MOE_ERR_NULL), (dict(v=None), M.MOE_ERR_NULL),
    (dict(state8=1), M.MOE_ERR_NULL), (dict(m_s=0x1000), M.MOE_ERR_ARG),
    (dict(param=0x1001), M.MOE_ERR_ARG), (dict(master=0x1002), M.MOE_ERR_ARG),
    (dict(grad=0x1002), M.MOE_ERR_ARG), (dict(m=0x1002), M.MOE_ERR_ARG),
])
def test_adamw_refusals(kw, code):
    hp = kw.pop("hp", None) if "hp" in kw else None
    kw = dict(kw)
    if kw.get("n") == -1:
        assert _adam(n=-1) == code
        assert M.lib().moe_adamw(None, 1, None, None) == M.MOE_ERR_NULL
        return
    assert _adam(hp=hp, **kw) == code
    assert M.lib().moe_last_error()


def test_adamw_tensor_sizes():
    def call(size):
        h = M.MoeAdamwHyper(1e-3, 0.9, 0.95, 1e-8, 1, 0, None, 1.0, 0)
        t = M.MoeAdamwTensor(n=size, dtype=M.MOE_F32)
        return M.lib().moe_adamw(C.byref(t), 1, C.byref(h), None)

    assert call(-1) == M.MOE_ERR_SHAPE
    assert call(1 << 36) == M.MOE_ERR_SHAPE
    assert call((1 << 34) + 1) == M.MOE_ERR_SHAPE
    assert call(0) == M.MOE_OK          # nothing to do, nothing launched
    h = M.MoeAdamwHyper(1e-3, 0.9, 0.95, 1e-8, 1, 0, None, 1.0, 0)
    assert M.lib().moe_adamw(None, 0, C.byref(h), None) == M.MOE_OK


def test_binding_checks_tensors():
    s = _shape()
    cpu = torch.zeros(64, 256, dtype=torch.bfloat16)
    with pytest.raises(M.MoeError):
        M.moe_quant_rows_fp8(s, cpu, 64, None, cpu, cpu)
    with pytest.raises(ValueError):
        M.Fp8Weights(s, device="cpu", other=cpu)
    with pytest.raises(M.MoeError):
        M.AdamWTensors([dict(param=torch.zeros(4, dtype=torch.int32), grad=cpu, m=cpu, v=cpu)])
