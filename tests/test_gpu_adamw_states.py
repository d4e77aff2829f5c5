"""The stored root of the second moment on the GPU: never zero by rounding, and steps
that stay bounded where half of a block's gradients are far below the other half
(bounds: test_adamw_states_cpu.py)."""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from moe_harness import host
from oracle import fp8_oracle as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def _zero(n):
    z = lambda: torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = lambda: torch.full((-(-n // 128),), 127, dtype=torch.uint8, device="cuda")
    return dict(param=torch.zeros(n, device="cuda"), grad=torch.zeros(n, device="cuda"), m=z(),
                v=z(), m_s=s(), v_s=s())


@pytest.mark.parametrize("n", [128, 1000, 4096])
def test_small_roots_are_kept(n):
    """One step from zero: sqrt(v) = sqrt(1 - beta2) |g|, over 22 orders of magnitude."""
    rng = np.random.default_rng(n)
    g = (rng.normal(size=n) * 10.0 ** rng.uniform(-16, 6, n)).astype(np.float32)
    g[rng.random(n) < 0.2] = 0.0
    t = _zero(n)
    t["grad"].copy_(torch.from_numpy(g))
    M.moe_adamw([t], lr=0.0, beta2=0.95, step=1, seed=5)
    q, byte = Q.quant_random(np.sqrt(0.05 * g.astype(np.float64) ** 2), Q.random_bits(n, 0, 5, 1)[1],
                             True)
    got = host(t["v"].float())
    assert np.array_equal(got == 0, g == 0)
    assert np.array_equal(host(t["v_s"]), byte)
    # one in a thousand may lie on a rounding border (test_gpu_adamw.py)
    assert (got != q).sum() <= max(1, n // 1000)
    # the first moment has no least value: some of the smallest are rounded to 0
    assert (host(t["m"].float())[g != 0] == 0).any()


@pytest.mark.parametrize("beta2,most", [(0.95, 23.6), (0.999, 149.2)])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-5, 1e-6])
def test_steps_stay_bounded(size, beta2, most):
    n = 128 * 64
    t = _zero(n)
    small = torch.arange(n, device="cuda") % 128 >= 64
    scale = torch.where(small, size, 1.0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ts = M.AdamWTensors([t])
    worst = 0.0
    for k in range(1, 201):
        t["grad"].copy_(torch.randn(n, generator=gen, device="cuda") * scale)
        t["param"].zero_()
        M.moe_adamw(ts, lr=1.0, beta1=0.9, beta2=beta2, step=k, seed=k)
        if k > 30:                 # the bias corrections' quotient is below 1 from here on
            worst = max(worst, t["param"].abs().max().item())
    assert worst <= most
