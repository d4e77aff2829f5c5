"""The 8-bit calls' workspace: sized for the longest batch it does for every shorter
one, and it is on the device of the call."""

import pytest
import torch

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


def test_workspace_on_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(M, "_chk_all", lambda *a: 0)     # all tensors are on device 0
    monkeypatch.setattr(M, "_chk_ws", lambda *a: None)
    s = M.make_shape(4, 256, 128, 2, 0, 2, 1, "bf16")
    ws = torch.zeros(1 << 16, dtype=torch.uint8)         # on the host, device -1
    reached = pytest.raises(AttributeError)              # the weights, None here, come after
    for on, outcome in ((-1, pytest.raises(M.MoeError)), (0, reached)):
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: on)
        with outcome:
            M.moe_expert_ffn_fwd_fp8(s, ws, ws, None, ws, ws, None, None, None, ws, ws, 0)
        with pytest.raises(M.MoeError) if on else pytest.raises(AttributeError):
            M.moe_ffn_dgrad_fp8(s, ws, ws, None, None, ws, ws, ws, None, ws, ws, None, ws, 0)
