"""A short batch in the workspace of a longer one, whichever kernels run."""

import pytest
import torch

import combine_expert_ffn_amd as M
from test_gpu_fp8 import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_short_batches_in_a_long_ones_workspace(dtype):
    d, F, E, K = 640, 384, 4, 2
    size = M.moe_fp8_workspace_bytes(M.make_shape(2000, d, F, E, 0, E, K, dtype))
    ws = torch.empty(size + 4096, dtype=torch.uint8, device="cuda")
    for T in (2000, 1037, 512, 40, 1):
        L = Layer(T, d, F, E, 0, E, K, dtype, True, seed=T)
        L.ws = ws[:size]
        ws[size:] = 77
        L.check_forward(L.forward())
        L.check_dgrad(L.dgrad())
        assert (ws[size:] == 77).all(), T
