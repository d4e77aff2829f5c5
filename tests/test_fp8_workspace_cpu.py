"""A workspace sized for the longest batch does for every shorter one."""

import pytest

import combine_expert_ffn_amd as M

SHAPES = {
    # d, F, E, E_l, K
    "128_experts": (2048, 768, 128, 128, 8),
    "a_window": (2048, 1408, 64, 8, 6),
    "four_small": (640, 384, 4, 4, 2),
    "one": (128, 128, 1, 1, 1),
    "256_experts": (256, 128, 256, 256, 8),
    "wide": (16384, 16384, 16, 2, 4),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", SHAPES)
def test_workspace_never_falls_as_the_batch_grows(name, dtype):
    d, F, E, E_l, K = SHAPES[name]
    last = 0
    for T in [*range(0, 1400), *range(1400, 20000, 97)]:
        need = M.moe_fp8_workspace_bytes(M.make_shape(T, d, F, E, 0, E_l, K, dtype))
        assert need >= last, T
        # a quantised row and its scales, or a few float32 rows: no more than the larger
        assert 256 <= need <= max(256, T * K * 8 * F + 512), T
        last = need
