"""Every compiled kernel for few rows of the 4-bit experts against the float64 oracle: which
one runs follows from the shape, so the cases are one or more shapes for each, and a test asks
the profiler that they ran.  Where a kernel's blocks take further passes in a loop, one expert
has every token, which is more passes than the grid holds at once.  Tolerances are
test_gpu_fp8.py's.
"""

import re

import pytest
import torch

import combine_expert_ffn_amd as M
import combine_expert_ffn_amd._lib as L
from test_gpu_fp4 import Layer4

pytestmark = pytest.mark.gpu

# T, d, F, E, E_l, K, dtype, one expert has every token
CASES = [
    (10, 128, 128, 128, 1, 2, "f16", False),
    (1, 128, 128, 8, 1, 1, "bf16", False),
    (1, 640, 640, 64, 1, 2, "f16", False),
    (16, 640, 640, 64, 1, 1, "bf16", False),
    (274, 128, 1408, 2, 1, 1, "f16", False),
    (137, 1408, 128, 1, 1, 1, "f16", False),
    (137, 1408, 128, 1, 1, 1, "bf16", False),
    (108, 128, 1664, 2, 1, 2, "bf16", False),
    (79, 2432, 128, 2, 1, 2, "bf16", False),
    (99, 2176, 128, 1, 1, 1, "f16", False),
    (1, 128, 2176, 64, 1, 1, "f16", False),
    (2, 128, 2176, 8, 1, 1, "bf16", False),
    (690, 384, 384, 64, 1, 1, "bf16", True),
    (691, 384, 384, 16, 1, 1, "f16", True),
    (417, 640, 640, 4, 1, 1, "bf16", True),
    (420, 640, 640, 4, 1, 1, "f16", True),
    (170, 640, 640, 2, 2, 2, "bf16", False),
    (182, 128, 128, 64, 64, 8, "bf16", False),
    (739, 128, 128, 64, 64, 2, "f16", False),
    (256, 896, 1024, 1, 1, 1, "f16", False),
    (227, 1152, 1152, 1, 1, 1, "f16", False),
    (220, 1152, 1280, 1, 1, 1, "bf16", False),
    (198, 1024, 640, 4, 1, 4, "bf16", False),
    (206, 1024, 640, 1, 1, 1, "f16", False),
    (834, 1280, 384, 4, 1, 1, "bf16", True),
    (698, 1536, 384, 4, 1, 1, "f16", True),
    (1086, 1024, 2048, 16, 1, 3, "bf16", False),
    (225, 2176, 1024, 1, 1, 1, "bf16", False),
    (333, 2048, 128, 2, 2, 1, "bf16", False),
    (468, 2304, 640, 4, 1, 1, "bf16", True),
    (434, 2432, 640, 4, 1, 1, "f16", True),
    (349, 1280, 1024, 2, 2, 1, "f16", False),
    (203, 1024, 1152, 1, 1, 1, "f16", False),
    (419, 640, 1152, 4, 1, 1, "bf16", True),
    (422, 640, 1152, 16, 1, 1, "f16", True),
    (419, 640, 2176, 64, 1, 1, "f16", True),
    (427, 640, 2176, 8, 1, 1, "bf16", True),
    (253, 1024, 2176, 1, 1, 1, "f16", False),
    (229, 1024, 2304, 1, 1, 1, "bf16", False),
    (226, 1920, 1280, 1, 1, 1, "bf16", False),
    (200, 1024, 2560, 1, 1, 1, "bf16", False),
    (835, 1280, 1152, 4, 1, 1, "f16", True),
    (646, 1664, 1152, 4, 1, 1, "bf16", True),
    (754, 1408, 2176, 4, 1, 1, "f16", True),
    (695, 1536, 2176, 4, 1, 1, "bf16", True),
    (128, 2176, 1024, 16, 8, 3, "bf16", False),
]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


@pytest.mark.parametrize("T,d,F,E,E_l,K,dtype,one", CASES)
def test_forward(T, d, F, E, E_l, K, dtype, one):
    A = Layer4(T, d, F, E, 0, E_l, K, dtype, True, seed=d + F, only=[0] if one else None)
    assert not one or A.off[1] == T
    A.check_forward(A.forward())


@pytest.mark.parametrize("one", [False, True], ids=["even", "one_expert"])
@pytest.mark.parametrize("T,d,F,E,E_l,K,dtype", [
    (2437, 128, 384, 128, 128, 2, "f16"), (2964, 256, 128, 64, 64, 2, "f16"),
    (3045, 1536, 512, 32, 4, 2, "bf16")])
def test_long_batches_that_are_few_rows_to_an_expert(T, d, F, E, E_l, K, dtype, one):
    """Passes shorter than the launch shape's do not send a batch to the tiles; up to 191 of them
    over one expert that every token names."""
    A = Layer4(T, d, F, E, 0, E_l, K, dtype, True, only=[2] if one else None)
    assert not one or A.off[3] - A.off[2] == T
    M.moe_timing_enable()
    try:
        M.moe_timing_reset()
        out = A.forward()
        torch.cuda.synchronize()
        names = set(M.moe_timing_report())
    finally:
        M.moe_timing_disable()
    assert len(names) == 2 and all(n.endswith("_small") for n in names), names
    A.check_forward(out)


NUMBERS = r"fp4_small_kernelILi(\d)ELi(\d)ELi(\d)ELi(\d)ELb(\d)ENS0_\d(First|Second)I(t|DF16_)E"
NAMES = (r"fp4_small_kernel<(\d), (\d), (\d), (\d), (false|true), .*?(First|Second)"
         r"<(unsigned short|_Float16)>")
WORDS = {"false": "0", "true": "1", "unsigned short": "t", "_Float16": "DF16_"}


def _run(T, d, F, E, E_l, K, dtype):
    """A call on zeros with an even routing: which kernels run follows from the shape."""
    s = M.make_shape(T, d, F, E, 0, E_l, K, dtype)
    mb = M.MicroBatch(s)
    ws = torch.empty(max(M.moe_workspace_bytes(s), M.moe_fp4_workspace_bytes(s)),
                     dtype=torch.uint8, device="cuda")
    mb.idx.copy_((torch.arange(T)[:, None] + torch.arange(K)).remainder(E).to(torch.int32))
    M.moe_dispatch(s, None, mb.idx, mb.counts, mb.offsets, mb.row_of_pair, mb.pair_of_row,
                   mb.tile_offsets, None, ws)
    w = M.Fp4Weights(s)
    for n in M.FP4_WEIGHT_FIELDS:
        getattr(w, n).zero_()
    q = torch.zeros(T, d, device="cuda").to(torch.float8_e4m3fn)
    qs = torch.zeros(T, M.moe_fp8_scale_ld(d), dtype=torch.uint8, device="cuda")
    yp = torch.empty(T * K, d, dtype=mb.yp.dtype, device="cuda")
    M.moe_expert_ffn_fwd_fp4(s, q, qs, mb.pair_of_row, mb.offsets, mb.tile_offsets, w, None, None,
                             yp, ws)
    torch.cuda.synchronize()


def test_the_cases_run_every_compiled_kernel():
    text = open(L.LIB_PATH, "rb").read().decode("latin-1")
    compiled = set(re.findall(NUMBERS, text))
    assert len(compiled) > 50
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        for case in CASES:
            _run(*case[:-1])
    ran = set()
    for e in prof.key_averages():
        for pattern in (NUMBERS, NAMES):
            ran |= {tuple(WORDS.get(w, w) for w in m) for m in re.findall(pattern, e.key)}
    assert ran == compiled, (sorted(compiled - ran), sorted(ran - compiled))
