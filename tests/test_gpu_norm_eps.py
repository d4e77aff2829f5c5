"""moe_rmsnorm with eps of every size it accepts, beside rows whose squares pass float32's
range.  Tolerances are test_gpu_norm.py's: 2^-18 on a row's sum and root, half a step for
the rounding of what is stored."""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from moe_harness import host
from oracle import norm_fp4_oracle as N4
from test_gpu_norm import SUM, Norm, half_step, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [256, 1024, 4096])
@pytest.mark.parametrize("eps", [1e-30, 1e-3, 1e20, 1e30, 1e38, 3.4e38])
def test_eps_counts_beside_every_row(eps, d, dtype):
    """Ordinary rows, rows whose sum of squares passes float32's range, and one (row 5) whose
    mean, 3e35, does so up to d = 1024 with the largest eps only."""
    n = Norm(9, d, dtype, res=False)
    n.x[1] *= 2.0 ** 40
    n.x[2] *= 2.0 ** 66
    n.x[4] *= 2.0 ** 100
    n.x[5] = 3e35 ** 0.5
    n.x[7] = n.x[7].sign() * 2.0 ** 120
    n.x[8, 3] = 2.0 ** 80
    o = n.forward(eps=eps)
    r, gamma = host(n.x), host(n.gamma)
    y, rstd = N4.rmsnorm(r, gamma, float(np.float32(eps)))
    within("rstd", host(o["rstd"]), rstd, rstd * SUM)
    within("y", host(o["y"]), y, np.abs(y) * SUM * 2 + half_step(np.abs(y) * (1 + SUM), dtype))
