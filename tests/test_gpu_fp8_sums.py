"""What the sums of the 8-bit products keep, kernel by kernel.

fp16 data, and few rows of bf16 data, use exact products and round only their
float32 sums; bf16 tiles cut each of eight consecutive products at 2^-13 of the
largest of the eight (include/moe.h).

Tolerances, fixed before the first run.  Sums whose large products cancel and leave
a few small powers of two are exact in float32 and in both 16-bit types, so exact
kernels must give them bit for bit; a tile's six small products may each lose up to
2^-13 of the largest beside them.  On random operands a float32 sum of k exact
products rounds at most once per four products, toward zero at worst: k / 4 * 2^-23
of sum |terms|.
"""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
import test_gpu_fp8 as G
from moe_harness import host
from test_gpu_fp8 import DT, LAYERS, Layer

pytestmark = pytest.mark.gpu

BIG, SMALL = 256.0, 2.0 ** -6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def _layer(T, dtype):
    """One expert of 128 x 128 with T rows, everything zero: the operands are set by
    the test and quantised by ``_load``."""
    L = Layer(T, 128, 128, 1, 0, 1, 1, dtype, False)
    for t in (L.x, L.W_gu, L.W_down, L.h):
        t.zero_()
    return L


def _load(L):
    L.q, L.qs = L.quantise(L.x, L.T)
    M.moe_quant_weights_fp8(L.s, L.W_gu, L.W_down, L.w)


def _cancelling(t, w, c):
    """Rows t [n, 128] and weight columns w [128, m] (views) whose products are
    +-256 and six of SMALL * c[column]: sums of 6 SMALL c."""
    t[:, :2] = BIG
    t[:, 2:8] = SMALL
    w[0], w[1] = 1.0, -1.0
    w[2:8] = c


@pytest.mark.parametrize("product", ["gate_up", "dgrad_act", "dgrad_in"])
@pytest.mark.parametrize("T", [5, 600], ids=["few_rows", "tiles"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_cancelling_products(dtype, T, product):
    L = _layer(T, dtype)
    c = torch.tensor([1.0, 0.5, -1.0, 0.25] * 32, device="cuda", dtype=DT[dtype])
    if product == "gate_up":
        _cancelling(L.x, L.W_gu[0, :128].T, c)
        _load(L)
        got = L.forward()["h"][:, :128]
    elif product == "dgrad_act":
        # g = 0, u = 2: dg = da * 2 * (1 / 2), du = 0
        _cancelling(L.x, L.W_down[0], c)
        L.h[:, 128:] = 2.0
        _load(L)
        got = L.dgrad()["dh"][:, :128]
    else:
        # da = 1, g = 0: dg = u / 2 is the second product's operand
        L.x[:, 0] = 1.0
        L.W_down[0, 0] = 1.0
        _cancelling(L.h[:, 128:], L.W_gu[0, :128], c)
        L.h *= 2.0
        _load(L)
        got = L.dgrad()["dx"]
    want = 6 * SMALL * host(c)
    err = np.abs(host(got) - want)
    if dtype == "bf16" and T == 600:
        assert err.max() <= 6 * 2.0 ** -13 * BIG
    else:
        assert err.max() == 0.0, err.max()


@pytest.mark.parametrize("gather", [True, False], ids=["tokens", "dispatched"])
@pytest.mark.parametrize("name,dtype", [
    ("two_rows_each", "bf16"), ("ragged_tiles", "bf16"), ("half_tiles", "bf16"),
    ("many_experts", "bf16"), ("ragged_tiles", "f16"), ("over_a_tile", "f16"),
    ("tiles_odd_blocks", "f16"), ("tiles_window", "f16")])
def test_float32_sums(name, dtype, gather, monkeypatch):
    T, d, F = LAYERS[name][:3]
    monkeypatch.setattr(G, "EPS_SUM", max(d, 2 * F) / 4 * 2.0 ** -23)
    L = Layer(*LAYERS[name], dtype, gather, seed=len(name) + 7)
    L.check_forward(L.forward())
    L.check_dgrad(L.dgrad())
