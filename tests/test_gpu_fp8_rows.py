"""What a row's results in the 8-bit products depend on (include/moe.h): the same
tokens in another order, and some of them left out, give the same bits where one
order of the sums is stated, and elsewhere differ by that order alone.

Tolerance, fixed before the first run: a float32 sum of k terms rounds at most k / 4
times (test_gpu_fp8_sums.py), 2^-23 of sum |terms| each, in either order; bf16 tiles cut
their products the same way in every order, the groups being fixed.  sum |terms| is at
most the largest |quantised value| times sum |weight| of the column.  The 16-bit result then
moves by one step at most where the sum crosses a border.
"""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from moe_harness import host
from test_gpu_fp8 import LAYERS, Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def _moved(A, tokens):
    """The layer of A's tokens ``tokens``, in that order, with A's operands."""
    shape = (len(tokens), A.d, A.F, A.s.E, A.s.e_lo, A.E_l, A.K)
    B = Layer(*shape, A.dtype, True)
    t = torch.as_tensor(tokens, device="cuda")
    B.mb.idx.copy_(A.mb.idx[t])
    ws = torch.empty(M.moe_workspace_bytes(B.s), dtype=torch.uint8, device="cuda")
    M.moe_dispatch(B.s, None, B.mb.idx, B.mb.counts, B.mb.offsets, B.mb.row_of_pair,
                   B.mb.pair_of_row, B.mb.tile_offsets, None, ws)
    B.off = host(B.mb.offsets)
    B.N = int(B.off[-1])
    B.pair = host(B.mb.pair_of_row)[: B.N]
    B.q = A.q.view(torch.uint8)[t].view(torch.float8_e4m3fn)
    B.qs, B.w = A.qs[t], A.w
    B.gates = A.gates.reshape(A.T, A.K)[tokens].reshape(-1)
    from_row = _row_of_moved(A, B, tokens)
    B.h[: B.N] = A.h[torch.as_tensor(from_row, device="cuda")]
    return B, from_row


def _row_of_moved(A, B, tokens):
    """A's dispatched row of each dispatched row of B."""
    row_of = np.full(A.T * A.K, -1)
    row_of[A.pair] = np.arange(A.N)
    rows = row_of[np.asarray(tokens)[B.pair // B.K] * B.K + B.pair % B.K]
    assert (rows >= 0).all()
    return rows


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["seventeen_each", "ragged_tiles", "tiles_window",
                                  "tiles_odd_blocks", "tiles_halves", "tiles_past_the_grid"])
def test_rows_in_another_batch(name, dtype):
    A = Layer(*LAYERS[name], dtype, True, seed=3)
    want = {**A.forward(), **A.dgrad()}
    again = {**A.forward(), **A.dgrad()}
    assert all(torch.equal(again[n], want[n]) for n in want)
    few = name in ("seventeen_each", "ragged_tiles")
    rng = np.random.default_rng(5)
    for keep in (A.T, A.T - A.T // 16):
        B, rows = _moved(A, rng.permutation(A.T)[:keep])
        got = {**B.forward(), **B.dgrad()}
        rows = torch.as_tensor(rows, device="cuda")
        for n in want:
            x, y = got[n][: B.N], want[n][rows]
            if few or n not in ("y", "dx"):
                assert torch.equal(x, y), (keep, n)
                continue
            k, W, v = (A.F, A.W_down, want["a"]) if n == "y" else (2 * A.F, A.W_gu, want["dh"])
            # quantised values: at most half a step of e4m3 (2^-4) above the stored ones
            big = 1.07 * v[: A.N].float().abs().max()
            col = W.float().abs().sum(2 if n == "y" else 1).max() * 1.07
            step = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]
            tol = 2 * k / 4 * 2.0 ** -23 * big * col + step * y.float().abs()
            assert ((x.float() - y.float()).abs() <= tol).all(), (keep, n)
