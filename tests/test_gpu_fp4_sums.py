"""What the sums of the products on 4-bit weights keep, kernel by kernel, and what a row's
results depend on (include/moe.h).

fp16 data uses exact products and rounds only their float32 sums; bf16 data cuts each of
eight consecutive products at 2^-13 of the largest of the eight, for few rows too.

Tolerances, fixed before the first run, are those of the 8-bit products: sums whose large
products cancel and leave a few small powers of two are exact in float32 and in both 16-bit
types, so exact kernels must give them bit for bit, and where products are cut six small ones
may each lose up to 2^-13 of the largest beside them, or none where they are no smaller
than that.  On random operands a float32 sum of k exact products rounds at most once per four
products, toward zero at worst: k / 4 * 2^-23 of sum |terms|.  In another batch a float32 sum
is taken in another order at most, so it differs by twice that, and the 16-bit result by a
step where the sum crosses a border; the products are cut the same way, their groups being
fixed.
"""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
import test_gpu_fp8 as G
from moe_harness import host
from test_gpu_fp4 import Layer4
from test_gpu_fp8 import DT, LAYERS

pytestmark = pytest.mark.gpu

BIG = 256.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def _few(L):
    """The forward's results, and whether the kernels for few rows gave them."""
    M.moe_timing_enable()
    try:
        M.moe_timing_reset()
        out = L.forward()
        torch.cuda.synchronize()
        names = set(M.moe_timing_report())
    finally:
        M.moe_timing_disable()
    few = {n.endswith("_small") for n in names}
    assert len(few) == 1, names
    return out, few.pop()


@pytest.mark.parametrize("small", [2.0 ** -6, 2.0 ** -2])
@pytest.mark.parametrize("product", ["gate_up", "down"])
@pytest.mark.parametrize("T", [5, 600], ids=["few_rows", "tiles"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_cancelling_products(dtype, T, product, small):
    """Products of +-256 and six of small * c[column]: sums of 6 small c."""
    L = Layer4(T, 128, 128, 1, 0, 1, 1, dtype, False)
    for t in (L.x, L.W_gu, L.W_down):
        t.zero_()
    c = torch.tensor([1.0, 0.5, -1.0, 0.25] * 32, device="cuda", dtype=DT[dtype])
    row = torch.zeros(128, device="cuda", dtype=DT[dtype])
    row[:2], row[2:8] = BIG, small
    if product == "gate_up":
        L.x[:] = row
        W = L.W_gu[0, :128]
    else:
        # a = silu(32) u = 32 u, since exp(-32) adds nothing to 1 in float32
        L.x[:, 0] = 1.0
        L.W_gu[0, :128, 0] = 32.0
        L.W_gu[0, 128:, 0] = row / 32
        W = L.W_down[0]
    W[:, 0], W[:, 1] = 1.0, -1.0
    W[:, 2:8] = c[:, None]
    L.q, L.qs = L.quantise(L.x, L.T)
    M.moe_quant_weights_fp4(L.s, L.W_gu, L.W_down, L.w4)
    out, few = _few(L)
    assert few == (T == 5)
    if product == "down":
        assert torch.equal(out["a"], row.expand(T, -1))
    got = out["h"][:, :128] if product == "gate_up" else out["y"]
    err = np.abs(host(got) - 6 * small * host(c)).max()
    # the smallest product is small / 4
    if dtype == "bf16" and small / 4 < 2.0 ** -13 * BIG:
        assert err <= 6 * 2.0 ** -13 * BIG
    else:
        assert err == 0.0, err


@pytest.mark.parametrize("gather", [True, False], ids=["tokens", "dispatched"])
@pytest.mark.parametrize("name", ["two_rows_each", "ragged_tiles", "many_experts", "wide",
                                  "tiles_odd_blocks", "tiles_window", "tiles_past_the_grid"])
def test_float32_sums(name, gather, monkeypatch):
    d, F = LAYERS[name][1:3]
    monkeypatch.setattr(G, "EPS_SUM", max(d, F) / 4 * 2.0 ** -23)
    L = Layer4(*LAYERS[name], "f16", gather, seed=len(name) + 7)
    L.check_forward(L.forward())


def _moved(A, tokens):
    """The layer of A's tokens ``tokens``, in that order, with A's operands; and A's
    dispatched row of each of its dispatched rows."""
    B = Layer4(len(tokens), A.d, A.F, A.s.E, A.s.e_lo, A.E_l, A.K, A.dtype, True)
    t = torch.as_tensor(tokens, device="cuda")
    B.mb.idx.copy_(A.mb.idx[t])
    ws = torch.empty(M.moe_workspace_bytes(B.s), dtype=torch.uint8, device="cuda")
    M.moe_dispatch(B.s, None, B.mb.idx, B.mb.counts, B.mb.offsets, B.mb.row_of_pair,
                   B.mb.pair_of_row, B.mb.tile_offsets, None, ws)
    B.off = host(B.mb.offsets)
    B.N = int(B.off[-1])
    B.pair = host(B.mb.pair_of_row)[: B.N]
    B.q = A.q.view(torch.uint8)[t].view(torch.float8_e4m3fn)
    B.qs, B.w4 = A.qs[t], A.w4
    row_of = np.full(A.T * A.K, -1)
    row_of[A.pair] = np.arange(A.N)
    rows = row_of[np.asarray(tokens)[B.pair // B.K] * B.K + B.pair % B.K]
    assert (rows >= 0).all()
    return B, torch.as_tensor(rows, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape,few", [
    (LAYERS["seventeen_each"], True), (LAYERS["ragged_tiles"], True),
    ((40, 1152, 2176, 8, 0, 8, 3), True),      # several units of the reduction to a wave
    (LAYERS["tiles_window"], False), (LAYERS["tiles_halves"], False),
    (LAYERS["tiles_past_the_grid"], False)])
def test_rows_in_another_batch(shape, few, dtype):
    A = Layer4(*shape, dtype, True, seed=3)
    want, kind = _few(A)
    assert kind == few
    again = A.forward()
    assert all(torch.equal(again[n], want[n]) for n in want)
    rng = np.random.default_rng(5)
    for keep in (A.T, A.T - A.T // 16):
        B, rows = _moved(A, rng.permutation(A.T)[:keep])
        got, kind = _few(B)
        assert kind == few
        for n in want:
            x, y = got[n][: B.N], want[n][rows]
            if few or n != "y":
                assert torch.equal(x, y), (keep, n)
                continue
            # quantised values: at most half a step of e4m3 (2^-4) above the stored ones
            big = 1.07 * want["a"][: A.N].float().abs().max()
            col = np.abs(A.weights()[1]).sum(2).max()
            step = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]
            tol = 2 * A.F / 4 * 2.0 ** -23 * big * col + step * y.float().abs()
            assert ((x.float() - y.float()).abs() <= tol).all(), (keep, n)
