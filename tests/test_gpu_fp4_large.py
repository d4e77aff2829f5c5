"""Weights of 128 MB and more, which are quantised and read back past the caches: the same
codes, scales and values as expert by expert (those are held to the definition in
test_gpu_fp4.py), bit for bit.  And results of more than 2^31 elements.
"""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from moe_harness import host
from test_gpu_fp4 import Layer4
from test_gpu_norm import DT

pytestmark = pytest.mark.gpu

PAST = 128 << 20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def _past(call):
    """Which of the kernels that ``call`` launches go past the caches."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    names = [e.key for e in prof.key_averages() if "quant_weights_fp4" in e.key]
    assert names
    return {"true" in n or "Lb1E" in n for n in names}


def _bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,F,more", [(640, 1024, 0), (2048, 768, 1), (128, 128, 3)])
def test_quant_and_read_back(d, F, more, dtype):
    size = torch.finfo(DT[dtype]).bits // 8
    E = min(256, -(-PAST // (3 * d * F * size)) + more)
    g = torch.Generator(device="cuda").manual_seed(d + E)
    rnd = lambda *sh: (torch.randn(*sh, generator=g, device="cuda") * torch.exp(
        2 * torch.randn(*sh[:-1], 1, generator=g, device="cuda"))).to(DT[dtype])
    W = [rnd(E, 2 * F, d), rnd(E, d, F)]
    W[0][E - 1, 3, 7], W[1][E - 1, d - 1, F - 1], W[1][0, 0, 0] = float("nan"), float("inf"), 0.0
    W[0][1, 5, :64] = 0.0
    s, s1 = (M.make_shape(1, d, F, n, 0, n, 1, dtype) for n in (E, 1))
    w = M.Fp4Weights(s)
    past = E * 3 * d * F * size >= PAST
    assert _past(lambda: M.moe_quant_weights_fp4(s, *W, w)) == {past}
    back = [torch.full_like(x, 5.0) for x in W]
    assert _past(lambda: M.moe_dequant_weights_fp4(s, w, *back)) == {past}
    w1, b1 = M.Fp4Weights(s1), [torch.full_like(x[:1], 5.0) for x in W]
    for e in range(E):
        M.moe_quant_weights_fp4(s1, *(x[e:e + 1] for x in W), w1)
        for n in M.FP4_WEIGHT_FIELDS:
            assert torch.equal(getattr(w, n)[e], getattr(w1, n)[0]), (n, e)
        M.moe_dequant_weights_fp4(s1, w1, *b1)
        for x, y in zip(back, b1):
            assert torch.equal(_bits(x[e]), _bits(y[0])), e


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gather", [True, False], ids=["tokens", "dispatched"])
def test_rows_past_32_bits(gather, dtype):
    """140000 rows of 2 x 8192 values of h: the last expert's last rows."""
    T, d, F, E, K = 17500, 128, 8192, 10, 8
    s = M.make_shape(T, d, F, E, 0, E, K, dtype)
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *sh, std=1.0: (torch.randn(*sh, generator=g, device="cuda") * std).to(DT[dtype])
    w = M.Fp4Weights(s)
    M.moe_quant_weights_fp4(s, rnd(E, 2 * F, d, std=d ** -0.5), rnd(E, d, F, std=F ** -0.5), w)
    i32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device="cuda")
    counts, offsets, tiles, rop, por = i32(E), i32(E + 1), i32(E + 1), i32(T * K), i32(T * K)
    ws = torch.empty(max(M.moe_fp4_workspace_bytes(s), M.moe_workspace_bytes(
        M.make_shape(T, d, 64, E, 0, E, K, dtype))), dtype=torch.uint8, device="cuda")
    idx = (torch.arange(T)[:, None] + torch.arange(K)).remainder(E).to(torch.int32).cuda()
    M.moe_dispatch(s, None, idx, counts, offsets, rop, por, tiles, None, ws)
    rows = T if gather else T * K
    q = torch.zeros(rows, d, device="cuda").to(torch.float8_e4m3fn)
    qs = torch.zeros(rows, M.moe_fp8_scale_ld(d), dtype=torch.uint8, device="cuda")
    M.moe_quant_rows_fp8(s, rnd(rows, d), rows, None, q, qs)
    h = torch.empty(T * K, 2 * F, dtype=DT[dtype], device="cuda")
    a = torch.empty(T * K, F, dtype=DT[dtype], device="cuda")
    y = torch.empty(T * K, d, dtype=DT[dtype], device="cuda")
    assert h.numel() > 2 ** 31
    M.moe_expert_ffn_fwd_fp4(s, q, qs, por if gather else None, offsets, tiles, w, h, a, y, ws)
    hi = int(offsets[E])
    assert hi == T * K
    L = object.__new__(Layer4)
    L.dtype, L.gather, L.d, L.F, L.K, L.E_l = dtype, gather, d, F, K, 1
    L.N, L.off, L.pair = 40, np.array([0, 40]), host(por)[hi - 40:]
    L.q, L.qs = (q, qs) if gather else (q[-40:], qs[-40:])
    L.w4 = type("W", (), {n: getattr(w, n)[E - 1:] for n in M.FP4_WEIGHT_FIELDS})
    L.check_forward({"h": h[-40:], "a": a[-40:], "y": y[-40:]})
