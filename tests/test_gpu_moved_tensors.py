"""Kept tensors whose memory moves between calls (test_moved_tensors_cpu.py): the
next call reads and writes where the tensors are now."""

import pytest
import torch

import combine_expert_ffn_amd as M
from test_gpu_adamw import HP, make
from test_gpu_fp8 import LAYERS, Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_window"])
def test_moved_weights(name):
    A, B = Layer(*LAYERS[name], "bf16", True, seed=1), Layer(*LAYERS[name], "bf16", True, seed=2)
    B.q, B.qs, B.mb, B.off, B.pair, B.N = A.q, A.qs, A.mb, A.off, A.pair, A.N
    B.h, B.gates = A.h, A.gates
    want = {**B.forward(), **B.dgrad()}
    for k, n in enumerate(M.FP8_WEIGHT_FIELDS):
        if k % 2:
            getattr(A.w, n).data = getattr(B.w, n).clone()
        else:
            setattr(A.w, n, getattr(B.w, n).clone())
    got = {**A.forward(), **A.dgrad()}
    assert all(torch.equal(got[n], want[n]) for n in want)
    A.w.gu_s.set_(torch.zeros(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(M.MoeError):
        A.forward()


@pytest.mark.parametrize("bits", [32, 8])
def test_moved_adamw_tensors(bits):
    a = [make(n, "bf16", bits, True, n) for n in (40, 3000)]
    b = [make(n, "bf16", bits, True, n) for n in (40, 3000)]
    ta, left = M.AdamWTensors(a), []
    for k in range(1, 4):
        for t in a:
            for n in ("param", "master", "grad", "m", "v"):
                left.append((t[n].detach(), t[n].detach().clone()))
                t[n].data = t[n].clone()
        M.moe_adamw(ta, step=k, seed=3, **HP)
        M.moe_adamw(b, step=k, seed=3, **HP)
        for x, y in zip(a, b):
            for n in ("param", "master", "m", "v"):
                assert torch.equal(x[n].view(torch.uint8), y[n].view(torch.uint8)), (k, n)
    for t, was in left:                       # the memory they left is as it was
        assert torch.equal(t.view(torch.uint8), was.view(torch.uint8))
