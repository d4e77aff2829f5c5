"""Weights of 128 MB and more, which are quantised and read back past the caches: the same
codes, scales and values as expert by expert (those are held to the definition in
test_gpu_fp4.py), bit for bit.
"""

import pytest
import torch

import combine_expert_ffn_amd as M
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
