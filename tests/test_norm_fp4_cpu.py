"""The norm and the calls on 4-bit weights without a GPU: pins of the oracle's
definitions, and every refusal of the entry points (no call here reaches a launch)."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from oracle import norm_fp4_oracle as N4

FAKE = C.c_void_p(0x1000)
ODD = C.c_void_p(0x1002)


# ---- the oracle -------------------------------------------------------------
@pytest.mark.parametrize("y,code", [
    (0.0, 0), (0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (2.50001, 5),
    (3.5, 6), (5.0, 6), (5.00001, 7), (6.0, 7), (7.0, 7), (-0.5, 9), (-0.1, 8), (-7.0, 15)])
def test_codes_closed_forms(y, code):
    assert N4.code4(y) == code


def test_codes_are_their_own_rounding():
    for c in range(16):
        v = (-1.0 if c > 7 else 1.0) * N4.E2M1[c & 7]
        assert N4.code4(v if c != 8 else -0.0) == c


@pytest.mark.parametrize("amax,byte", [
    (0.0, 127), (7.0, 127), (7.0001, 128), (3.5, 126), (1.0, 125), (0.875, 124), (0.8751, 125),
    (2.0 ** -140, 0), (float(np.finfo(np.float32).max), 253), (math.inf, 255), (math.nan, 255)])
def test_scales_closed_forms(amax, byte):
    assert N4.scale_byte4(amax) == byte


def test_quantisation_error():
    """Half a step: a quarter of a value between 2 and 6 units (5 becomes 4 or 6), never
    more than a unit, a quarter of a unit below 2."""
    rng = np.random.default_rng(0)
    W = rng.normal(size=(40, 256)) * np.exp(rng.normal(size=(40, 1)))
    code, byte = N4.quant4(W)
    unit = np.repeat(np.ldexp(1.0, byte - 127), 32, -1)
    err = np.abs(N4.value4(code, byte) - W) / unit
    m = np.abs(W) / unit
    assert m.max() <= 7
    assert (err <= np.where(m < 2, 0.25, np.where(m < 4, 0.5, 1.0)) + 1e-12).all()


def test_unpack():
    assert N4.unpack(np.array([[0x21, 0xF0]])).tolist() == [[1, 2, 0, 15]]


def test_a_block_with_nan_is_nan():
    W = np.ones((1, 96))
    W[0, 40] = np.inf
    code, byte = N4.quant4(W)
    v = N4.value4(code, byte)
    assert np.isnan(v[0, 32:64]).all() and (code[0, 32:64] == 0).all()
    assert (v[0, :32] == 1).all() and (v[0, 64:] == 1).all()


def test_norm_backward_against_differences():
    rng = np.random.default_rng(1)
    T, d, eps = 5, 48, 1e-3
    r, gamma, dy, dres = (rng.normal(size=sh) for sh in ((T, d), (d,), (T, d), (T, d)))
    _, rstd = N4.rmsnorm(r, gamma, eps)
    dx, dgamma = N4.rmsnorm_bwd(dy, r, gamma, rstd, dres)
    loss = lambda x, g: (dy * N4.rmsnorm(x, g, eps)[0]).sum() + (dres * x).sum()
    for _ in range(6):
        v, w = rng.normal(size=(T, d)), rng.normal(size=d)
        diff = (loss(r + 1e-5 * v, gamma + 1e-5 * w) - loss(r - 1e-5 * v, gamma - 1e-5 * w)) / 2e-5
        want = (dx * v).sum() + (dgamma * w).sum()
        # second differences: O(1e-10) of the third derivative, 1e-16 / 1e-5 of rounding
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want), np.abs(dx * v).sum())


# ---- refusals ---------------------------------------------------------------
def _shape(**kw):
    base = dict(T=64, d=256, F=128, E=8, e_lo=0, E_l=8, K=2, dtype="bf16")
    base.update(kw)
    return M.make_shape(**base)


def _norm(s, x=FAKE, res=None, gamma=FAKE, eps=1e-6, r=None, y=FAKE, q=None, qs=None, rstd=None):
    return M.lib().moe_rmsnorm(C.byref(s), x, res, gamma, eps, r, y, q, qs, rstd, None)


def _norm_bwd(s, dy=FAKE, r=FAKE, gamma=FAKE, rstd=FAKE, dres=None, dx=FAKE, dgamma=FAKE, acc=0,
              ws=FAKE, nb=1 << 40):
    return M.lib().moe_rmsnorm_bwd(C.byref(s), dy, r, gamma, rstd, dres, dx, dgamma, acc, ws, nb,
                                   None)


def _weights(**kw):
    f = {n: 0x1000 for n in M.FP4_WEIGHT_FIELDS}
    f.update(kw)
    return M.MoeFp4Weights(*[f[n] for n in M.FP4_WEIGHT_FIELDS])


def _quant(s, gu=FAKE, down=FAKE, w=None):
    return M.lib().moe_quant_weights_fp4(C.byref(s), gu, down, C.byref(w or _weights()), None)


def _dequant(s, gu=FAKE, down=FAKE, w=None):
    return M.lib().moe_dequant_weights_fp4(C.byref(s), C.byref(w or _weights()), gu, down, None)


def _fwd(s, xq=FAKE, xs=FAKE, pr=None, off=FAKE, to=FAKE, w=None, h=FAKE, a=FAKE, yp=FAKE, ws=FAKE,
         nb=1 << 40):
    return M.lib().moe_expert_ffn_fwd_fp4(C.byref(s), xq, xs, pr, off, to, C.byref(w or _weights()),
                                          h, a, yp, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), M.MOE_ERR_NULL), (dict(gamma=None), M.MOE_ERR_NULL),
    (dict(y=None), M.MOE_ERR_NULL), (dict(y=None, rstd=FAKE), M.MOE_ERR_NULL),
    (dict(q=FAKE), M.MOE_ERR_NULL), (dict(qs=FAKE), M.MOE_ERR_NULL),
    (dict(r=FAKE), M.MOE_ERR_ARG), (dict(eps=0.0), M.MOE_ERR_ARG),
    (dict(eps=-1e-6), M.MOE_ERR_ARG), (dict(eps=math.nan), M.MOE_ERR_ARG),
    (dict(eps=math.inf), M.MOE_ERR_ARG), (dict(eps=1e-60), M.MOE_ERR_ARG), (dict(eps=9e-31), M.MOE_ERR_ARG),
    (dict(x=ODD), M.MOE_ERR_ARG), (dict(res=ODD), M.MOE_ERR_ARG),
    (dict(gamma=ODD), M.MOE_ERR_ARG), (dict(res=FAKE, r=ODD), M.MOE_ERR_ARG),
    (dict(y=ODD), M.MOE_ERR_ARG), (dict(q=ODD, qs=FAKE), M.MOE_ERR_ARG),
    (dict(q=FAKE, qs=ODD), M.MOE_ERR_ARG), (dict(rstd=ODD), M.MOE_ERR_ARG)])
def test_norm_refusals(kw, code):
    assert _norm(_shape(), **kw) == code
    assert M.lib().moe_last_error()


def test_norm_shapes():
    s = _shape(d=192)
    assert _norm(s, q=FAKE, qs=FAKE) == M.MOE_ERR_SHAPE and b"128" in M.lib().moe_last_error()
    assert _norm(_shape(d=100)) == M.MOE_ERR_SHAPE
    assert _norm(_shape(dtype=7)) == M.MOE_ERR_DTYPE
    assert _norm(_shape(T=0)) == M.MOE_OK      # nothing to do, nothing launched
    assert _norm(_shape(T=0), x=None, y=None) == M.MOE_OK
    assert _norm_bwd(_shape(T=0), dy=None, r=None, rstd=None, dx=None, dgamma=None,
                     ws=None) == M.MOE_OK
    assert M.lib().moe_rmsnorm(None, FAKE, None, FAKE, 1e-6, None, FAKE, None, None, None,
                               None) == M.MOE_ERR_NULL


@pytest.mark.parametrize("kw,code", [
    *((dict([(n, None)]), M.MOE_ERR_NULL) for n in ("dy", "r", "gamma", "rstd", "dx", "ws")),
    *((dict([(n, ODD)]), M.MOE_ERR_ARG) for n in ("dy", "r", "gamma", "rstd", "dres", "dx",
                                                  "dgamma", "ws")),
    (dict(acc=M.MOE_ACCUM_DX), M.MOE_ERR_ARG), (dict(acc=4), M.MOE_ERR_ARG),
    (dict(nb=16), M.MOE_ERR_WORKSPACE)])
def test_norm_backward_refusals(kw, code):
    assert _norm_bwd(_shape(), **kw) == code
    assert M.lib().moe_last_error()


@pytest.mark.parametrize("d", [64, 512, 576, 2048, 2112, 16384])
def test_norm_workspace(d):
    last = 0
    for T in [*range(0, 70), *range(1000, 40000, 333)]:
        need = M.moe_rmsnorm_workspace_bytes(_shape(T=T, d=d))
        assert need >= last and 256 <= need <= max(256, 4 * d * min(max(T, 1), 1024) + 256), T
        last = need
    s = _shape(T=5000, d=d)
    assert _norm_bwd(s, nb=M.moe_rmsnorm_workspace_bytes(s) - 1) == M.MOE_ERR_WORKSPACE
    assert M.moe_rmsnorm_workspace_bytes(_shape(d=100)) == 0


@pytest.mark.parametrize("kw", [dict(d=192), dict(F=64), dict(F=192), dict(d=64)])
def test_sizes_must_be_whole_blocks(kw):
    s = _shape(**kw)
    for call in (_quant, _dequant, _fwd):
        assert call(s) == M.MOE_ERR_SHAPE and b"128" in M.lib().moe_last_error()
    assert M.moe_fp4_workspace_bytes(s) == 0


def test_fp4_null_pointers():
    s = _shape()
    for n in M.FP4_WEIGHT_FIELDS:
        for call in (_quant, _dequant, _fwd):
            assert call(s, w=_weights(**{n: None})) == M.MOE_ERR_NULL, n
    for call in (_quant, _dequant):
        assert call(s, gu=None) == M.MOE_ERR_NULL
        assert call(s, down=None) == M.MOE_ERR_NULL
    for n in ("xq", "xs", "off", "to", "yp", "ws"):
        assert _fwd(s, **{n: None}) == M.MOE_ERR_NULL, n
    assert M.lib().moe_quant_weights_fp4(C.byref(s), FAKE, FAKE, None, None) == M.MOE_ERR_NULL


def test_fp4_alignment_and_types():
    s = _shape()
    for call in (_quant, _dequant):
        assert call(s, gu=ODD) == M.MOE_ERR_ARG and call(s, down=ODD) == M.MOE_ERR_ARG
    for call in (_quant, _dequant, _fwd):
        assert call(s, w=_weights(gu=0x1008)) == M.MOE_ERR_ARG
        assert call(s, w=_weights(down_s=0x1002)) == M.MOE_ERR_ARG
    for n in ("xq", "xs", "h", "a", "yp", "ws"):
        assert _fwd(s, **{n: ODD}) == M.MOE_ERR_ARG, n
    assert _fwd(_shape(dtype="f32")) == M.MOE_ERR_UNSUPPORTED
    assert _fwd(_shape(T=1 << 23), pr=FAKE) == M.MOE_ERR_SHAPE   # T * d = 2^31
    assert _fwd(s, nb=M.moe_fp4_workspace_bytes(s) - 1) == M.MOE_ERR_WORKSPACE
    assert _fwd(_shape(T=0)) == M.MOE_OK
    assert _fwd(_shape(T=0), xq=None, xs=None, off=None, to=None, yp=None, ws=None) == M.MOE_OK


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,F,E,E_l,K", [(2048, 768, 128, 128, 8), (2048, 1408, 64, 8, 6),
                                         (128, 128, 1, 1, 1), (16384, 16384, 16, 2, 4)])
def test_fp4_workspace_never_falls(d, F, E, E_l, K, dtype):
    last = 0
    for T in [*range(0, 1400, 7), *range(1400, 20000, 97)]:
        need = M.moe_fp4_workspace_bytes(M.make_shape(T, d, F, E, 0, E_l, K, dtype))
        assert need >= last and 256 <= need <= T * K * 4 * F + 4096, T
        last = need


def test_binding_checks_tensors():
    s = _shape()
    cpu = torch.zeros(64, 256, dtype=torch.bfloat16)
    with pytest.raises(M.MoeError):
        M.moe_rmsnorm(s, cpu, None, cpu, 1e-6, None, cpu, None, None, None)
    with pytest.raises(M.MoeError):
        M.moe_rmsnorm_bwd(s, cpu, cpu, cpu, cpu, None, cpu, None, 0, None)
    with pytest.raises(M.MoeError):
        M.moe_quant_weights_fp4(s, cpu, cpu, None)
    with pytest.raises(M.MoeError):
        M.moe_dequant_weights_fp4(s, None, cpu, cpu)
    with pytest.raises(M.MoeError):
        M.moe_expert_ffn_fwd_fp4(s, cpu, cpu, None, cpu, cpu, None, None, None, cpu, None)
    with pytest.raises(ValueError):
        M.Fp4Weights(s, device="cpu", gu=cpu)
    with pytest.raises(M.MoeError):      # not on the GPU
        M.Fp4Weights(s, device="cpu")
