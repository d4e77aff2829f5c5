"""Every compiled kernel of the norm: all widths of a row's lanes, all types, short and long
batches and batches of 128 MB and more, which are read and written past the caches.

A row's results are those of the same row in a shorter batch, bit for bit (short batches are
held to float64 in test_gpu_norm.py and here), so the large batches are compared with their
halves.  dgamma, the only sum over rows, is held to float64 with a bound that counts the
roundings of the way it is summed, fixed before the first run: two for a term, one for every
addition that a term passes through, 2^-24 of the sum of magnitudes each.
  Up to 1024 rows (unless dx takes the place of dy or r): ceil(T / 64) rows of a thread, then
4 additions over lanes, 2 over waves, 1 with what is there.
  Else, with P rows of partial sums (the workspace's) and R rows at once to a block: ceil(T /
P R) rows of a thread, log2(R / 4) over lanes and 2 over waves (none with R = 1), and for P > 1
3 + ceil(P / 512) in a thread of the last sum, 2 + 16 over its lanes and waves; 1 with what is
there.
"""

import math
import re

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
import combine_expert_ffn_amd._lib as L
from moe_harness import host
from test_gpu_norm import DT, EPS, Norm

pytestmark = pytest.mark.gpu

# one for each number of lanes and of chunks to a lane
WIDTHS = [128, 256, 384, 640, 1152, 2176, 4224, 12416]
PAST = 128 << 20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def _rows(kind, d, dtype):
    size = torch.finfo(DT[dtype]).bits // 8
    T = {"few": 33, "long": 1500, "past": PAST // (d * size) + 7}[kind]
    assert (T * d * size >= PAST) == (kind == "past")
    return T


def _batch(T, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    rnd = lambda *sh: torch.randn(*sh, generator=g, device="cuda").to(DT[dtype])
    n = object.__new__(Norm)
    n.s, n.T, n.d, n.dtype, n.q = M.make_shape(T, d, 128, 1, 0, 1, 1, dtype), T, d, dtype, True
    n.x, n.res, n.dy, n.dres = (rnd(T, d) for _ in range(4))
    n.gamma = (1 + 0.3 * rnd(d).float()).to(DT[dtype])
    n.ws = torch.empty(M.moe_rmsnorm_workspace_bytes(n.s), dtype=torch.uint8, device="cuda")
    return n


def _part(n, lo, hi):
    p = object.__new__(Norm)
    p.T, p.d, p.dtype, p.q, p.gamma, p.ws = hi - lo, n.d, n.dtype, True, n.gamma, n.ws
    p.s = M.make_shape(p.T, n.d, 128, 1, 0, 1, 1, n.dtype)
    p.x, p.res, p.dy, p.dres = (t[lo:hi] for t in (n.x, n.res, n.dy, n.dres))
    return p


def _roundings(T, d, in_place):
    at_once = 256 // (16 if d <= 512 else (64 if d <= 2048 else 256))
    parts = M.moe_rmsnorm_workspace_bytes(M.make_shape(T, d, 128, 1, 0, 1, 1, "bf16")) // (4 * d)
    if T <= 1024 and not in_place and parts > 1:
        return 2 + -(-T // 64) + 4 + 2 + 1
    steps = 2 + -(-T // (parts * at_once)) + (math.log2(at_once / 4) + 2 if at_once > 1 else 0)
    return steps + (3 + -(-parts // 512) + 2 + 16 if parts > 1 else 0) + 1


def _check_dgamma(n, r, rstd, got, before=0.0, in_place=False):
    terms = n.dy.double() * (r.double() * rstd.double()[:, None])
    want, mag = terms.sum(0) + before, terms.abs().sum(0) + abs(before)
    # float64's own sums: T 2^-53 of the magnitudes, nothing beside this
    tol = _roundings(n.T, n.d, in_place) * 2.0 ** -24 * mag + 2.0 ** -149
    over = (got.double() - want).abs() - tol
    j = int(over.argmax())
    assert over[j] <= 0, (j, float(got[j]), float(want[j]), float(tol[j]))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("kind", ["few", "long", "past"])
def test_rows_and_sums(kind, d, dtype):
    n = _batch(_rows(kind, d, dtype), d, dtype)
    o = n.forward()
    dx, dg = n.backward(o["r"], o["rstd"], accumulate=M.MOE_ACCUM_DW)
    _check_dgamma(n, o["r"], o["rstd"], dg, before=3.0)
    at = n.dy.clone()
    dy, n.dy = n.dy, at
    again, dg = n.backward(o["r"], o["rstd"], dx=at)    # dx in dy's place
    n.dy = dy
    _check_dgamma(n, o["r"], o["rstd"], dg, in_place=True)
    assert torch.equal(again, dx)
    del again, at
    if kind == "few":
        n.check(o)
        n.check_backward(o["r"], o["rstd"], dx, None)
        return
    half = n.T // 2 + 1
    for lo, hi in ((0, half), (half, n.T)):
        p = _part(n, lo, hi)
        q = p.forward()
        for k in o:
            assert torch.equal(q[k].view(torch.uint8), o[k][lo:hi].view(torch.uint8)), (k, lo)
        e, _ = p.backward(q["r"], q["rstd"], dgamma=False)
        assert torch.equal(e, dx[lo:hi]), lo


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 64), (4, 2048), (5, 2048), (17, 512), (64, 16384),
                                 (1024, 64), (1024, 640), (1025, 640), (1024, 2112), (1025, 2112),
                                 (1300, 2176), (2048, 16384), (5000, 128), (20000, 64),
                                 (300000, 64)])
def test_dgamma_counts_its_roundings(T, d, dtype):
    n = _batch(T, d, dtype)
    r, rstd = n.x, torch.rsqrt(n.x.float().square().mean(1) + EPS)
    _, dg = n.backward(r, rstd)
    _check_dgamma(n, r, rstd, dg)
    at = r.clone()
    _, dg = n.backward(at, rstd, dx=at)
    _check_dgamma(n, r, rstd, dg, in_place=True)


NUMBERS = r"rmsnorm_(|bwd_)kernelI(t|DF16_|f)Li(\d+)ELi(\d)ELb(\d)E(?:Lb(\d)E)?E"
NAMES = (r"rmsnorm_(|bwd_)kernel<(unsigned short|_Float16|float), (\d+), (\d), (false|true)"
         r"(?:, (false|true))?>")
WORDS = {"false": "0", "true": "1", "unsigned short": "t", "_Float16": "DF16_", "float": "f"}


def test_the_cases_run_every_compiled_kernel():
    compiled = set(re.findall(NUMBERS, open(L.LIB_PATH, "rb").read().decode("latin-1")))
    assert len(compiled) > 100
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        for kind in ("few", "long", "past"):
            for d in WIDTHS:
                for dtype in DT:
                    n = _batch(_rows(kind, d, dtype), d, dtype)
                    o = n.forward()
                    n.backward(o["r"], o["rstd"])
                    torch.cuda.synchronize()
    ran = set()
    for e in prof.key_averages():
        for pattern in (NUMBERS, NAMES):
            ran |= {tuple(WORDS.get(w, w) for w in m) for m in re.findall(pattern, e.key)}
    assert ran == compiled, (sorted(compiled - ran), sorted(ran - compiled))
