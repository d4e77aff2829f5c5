"""Skewed loads in the 8-bit products: the kernels for few rows only where no expert can
hold many, and right results where one expert has every token."""

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


def _kernels(L):
    M.moe_timing_enable()
    try:
        M.moe_timing_reset()
        out = {**L.forward(), **L.dgrad()}
        torch.cuda.synchronize()
        return out, set(M.moe_timing_report())
    finally:
        M.moe_timing_disable()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,d,F,E,E_l,K,small", [
    (16384, 512, 384, 64, 16, 1, False),    # 256 rows each on average, up to 16384
    (1024, 256, 128, 128, 128, 1, False),   # 8 rows each, up to 1024
    (64, 256, 128, 64, 8, 8, True),
    (257, 640, 384, 4, 4, 2, True),
    (1, 128, 128, 8, 8, 8, True),
])
def test_few_row_kernels_where_no_expert_can_hold_many(T, d, F, E, E_l, K, small, dtype):
    _, names = _kernels(Layer(T, d, F, E, 0, E_l, K, dtype, True))
    assert len(names) == 4
    assert all(n.endswith("_small") == small for n in names), names


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,K", [(100, 64, 1), (130, 64, 8), (257, 4, 1), (700, 128, 1)])
def test_all_tokens_on_the_same_experts(T, E, K, dtype):
    L = Layer(T, 256, 128, E, 0, min(E, 16), K, dtype, True, only=list(range(K)))
    assert L.off[1] == T
    L.check_forward(L.forward())
    L.check_dgrad(L.dgrad())
