"""moe_rmsnorm and moe_rmsnorm_bwd on the GPU against their float64 definitions.

Tolerances, fixed before the first run.  SUM = 2^-18 bounds a row's float32 sums: a lane
adds at most 64 products one after another and the lanes join in at most 10 more steps,
each step off by 2^-24 of the terms' magnitudes, 74 * 2^-24 < 2^-17; half of that in rstd
(a square root), the rest of it and of a dozen roundings more is below 2^-18 there.  For the
backward's mean, which enters in full, 2^-17.  Stored values round once more, by half a step.
"""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from oracle import fp8_oracle as Q
from oracle import norm_fp4_oracle as N4
from moe_harness import exact, host

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SUM = 2.0 ** -18
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def half_step(ref, dtype):
    """Half a step, with the flat range."""
    return np.abs(ref) * torch.finfo(DT[dtype]).eps / 2 + {
        "bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}[dtype]


def within(name, got, ref, tol):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.size:
        return
    assert np.isfinite(got).all(), f"{name}: not finite"
    over = np.abs(got - ref) - tol
    i = np.unravel_index(int(over.argmax()), over.shape)
    assert over[i] <= 0, f"{name}{i}: got {got[i]}, ref {ref[i]}, {int((over > 0).sum())} over"


class Norm:
    def __init__(self, T, d, dtype, res=True, q=True, seed=0):
        rng = np.random.default_rng(seed + T + d)
        g = lambda *sh: torch.from_numpy(rng.normal(size=sh).astype(np.float32)).to(
            DT[dtype]).cuda()
        self.s, self.T, self.d, self.dtype = M.make_shape(T, d, 128, 1, 0, 1, 1, dtype), T, d, dtype
        row = torch.from_numpy(np.exp(rng.normal(size=(T, 1))).astype(np.float32)).cuda()
        self.x = (g(T, d) * row).to(DT[dtype])
        self.res = (g(T, d) * row).to(DT[dtype]) if res else None
        self.gamma = (1 + 0.3 * g(d).float()).to(DT[dtype])
        self.dy, self.dres = g(T, d), g(T, d)
        self.q = q
        self.ws = torch.empty(M.moe_rmsnorm_workspace_bytes(self.s), dtype=torch.uint8,
                              device="cuda")

    def out(self, fill=5.0):
        e = lambda: torch.full((self.T, self.d), fill, dtype=DT[self.dtype], device="cuda")
        o = {"y": e(), "rstd": torch.full((self.T,), fill, device="cuda"),
             "r": e() if self.res is not None else None, "q": None, "qs": None}
        if self.q:
            o["q"] = e().to(torch.float8_e4m3fn)
            o["qs"] = torch.full((self.T, M.moe_fp8_scale_ld(self.d)), 77, dtype=torch.uint8,
                                 device="cuda")
        return o

    def forward(self, o=None, stream=None, eps=EPS):
        o = o or self.out()
        M.moe_rmsnorm(self.s, self.x, self.res, self.gamma, eps, o["r"], o["y"], o["q"], o["qs"],
                      o["rstd"], stream)
        return o

    def rows(self):
        if self.res is None:
            return self.x
        return (self.x.float() + self.res.float()).to(DT[self.dtype])

    def check(self, o, eps=EPS):
        r = self.rows()
        if o["r"] is not None:
            assert torch.equal(o["r"], r)
        y, rstd = N4.rmsnorm(host(r), host(self.gamma), eps)
        if o["rstd"] is not None:
            within("rstd", host(o["rstd"]), rstd, rstd * SUM)
        if o["y"] is not None:
            within("y", host(o["y"]), y, np.abs(y) * SUM * 2 + half_step(np.abs(y) * (1 + SUM),
                                                                         self.dtype))
        if o["q"] is not None and o["y"] is not None:
            q, qs = torch.zeros_like(o["q"]), torch.zeros_like(o["qs"])
            M.moe_quant_rows_fp8(self.s, o["y"], self.T, None, q, qs)
            assert torch.equal(q.view(torch.uint8), o["q"].view(torch.uint8))
            assert torch.equal(qs, o["qs"])
            rq, rb = Q.quant_rows(host(o["y"]))
            exact("q", host(o["q"].float()), rq)
            exact("scales", host(o["qs"])[:, : self.d // 128], rb)

    def backward(self, r, rstd, dres=True, dgamma=True, accumulate=0, stream=None, dx=None):
        dx = torch.full_like(self.x, 5.0) if dx is None else dx
        dg = torch.full((self.d,), 3.0, device="cuda") if dgamma else None
        M.moe_rmsnorm_bwd(self.s, self.dy, r, self.gamma, rstd, self.dres if dres else None, dx,
                          dg, accumulate, self.ws if dgamma else None, stream)
        return dx, dg

    def check_backward(self, r, rstd, dx, dg, dres=True, accumulate=0):
        dy, rr, g, s = host(self.dy), host(r), host(self.gamma), host(rstd)
        e = host(self.dres) if dres else None
        rx, rg = N4.rmsnorm_bwd(dy, rr, g, s, e)
        xhat, dn = rr * s[:, None], dy * g
        mean = np.mean(np.abs(dn * xhat), -1, keepdims=True)
        tol = s[:, None] * (np.abs(dn) * 8 * 2.0 ** -24 + np.abs(xhat) * mean * 2 * SUM)
        tol += 0 if e is None else 4 * 2.0 ** -24 * (np.abs(e) + np.abs(rx))
        within("dx", host(dx), rx, tol + half_step(np.abs(rx) + tol, self.dtype))
        if dg is None:
            return
        # a thread's rows, then the lanes, waves and blocks
        lanes = 16 if self.d <= 512 else (64 if self.d <= 2048 else 256)
        parts = min(1024, -(-self.T // (256 // lanes)))
        steps = -(-self.T // max(1, parts * (256 // lanes))) + parts / 16 + 32
        tol = (steps * 2.0 ** -24) * (np.abs(dy * xhat).sum(0) + 3.0)
        within("dgamma", host(dg), rg + (3.0 if accumulate else 0.0), tol + 2.0 ** -149)


SHAPES = [(1, 64), (1, 2048), (3, 128), (17, 192), (5, 512), (33, 576), (130, 640), (7, 1024),
          (65, 1088), (300, 2048), (9, 2112), (6, 4096), (40, 4224), (5, 8192), (3, 12352),
          (11, 16384), (5000, 128), (4300, 640), (1300, 2176)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm_and_backward(T, d, dtype):
    for res in (True, False):
        n = Norm(T, d, dtype, res, q=d % 128 == 0)
        o = n.forward()
        n.check(o)
        r = o["r"] if res else n.x
        for dres, acc in ((True, 0), (False, M.MOE_ACCUM_DW)):
            dx, dg = n.backward(r, o["rstd"], dres, True, acc)
            n.check_backward(r, o["rstd"], dx, dg, dres, acc)


@pytest.mark.parametrize("d", [256, 1024, 4096])
def test_optional_outputs(d):
    """Outputs left out change nothing in the others."""
    n = Norm(70, d, "bf16")
    full = n.forward()
    for left in (("r",), ("y",), ("q", "qs"), ("rstd",), ("r", "y", "rstd"), ("r", "q", "qs", "rstd")):
        o = n.out()
        o.update({k: None for k in left})
        n.forward(o)
        for k, t in o.items():
            assert t is None or torch.equal(t.view(torch.uint8), full[k].view(torch.uint8)), (left, k)
    dx, dg = n.backward(full["r"], full["rstd"])
    ex, none = n.backward(full["r"], full["rstd"], dgamma=False)
    assert none is None and torch.equal(dx, ex)


@pytest.mark.parametrize("d", [256, 1024, 4096])
def test_in_place(d):
    """r in the residual's place, y in the input's, dx in dy's, dres' or r's."""
    n = Norm(70, d, "bf16")
    full = n.forward()
    x, res = n.x.clone(), n.res.clone()
    M.moe_rmsnorm(n.s, x, res, n.gamma, EPS, res, x, None, None, None)
    assert torch.equal(res, full["r"]) and torch.equal(x, full["y"])
    x = n.x.clone()
    M.moe_rmsnorm(n.s, x, n.res, n.gamma, EPS, x, full["y"], None, None, None)
    assert torch.equal(x, full["r"])
    dx, _ = n.backward(full["r"], full["rstd"])
    for k in range(3):
        bufs = [n.dy.clone(), n.dres.clone(), full["r"].clone()]
        dg = torch.empty(d, device="cuda")
        M.moe_rmsnorm_bwd(n.s, bufs[0], bufs[2], n.gamma, full["rstd"], bufs[1], bufs[k], dg, 0,
                          n.ws)
        assert torch.equal(bufs[k], dx), k


@pytest.mark.parametrize("d", [128, 640, 4096])
def test_values_that_are_not_finite_stay_in_their_rows(d):
    n = Norm(40, d, "bf16", res=False)
    good = n.forward()
    n.x[3, 5], n.x[20, d - 1] = float("nan"), float("-inf")
    o = n.forward()
    keep = [i for i in range(40) if i not in (3, 20)]
    for k in ("y", "rstd", "qs"):
        assert torch.equal(o[k][keep], good[k][keep])
    assert torch.equal(o["q"].view(torch.uint8)[keep], good["q"].view(torch.uint8)[keep])
    assert o["y"][3].isnan().all() and o["q"][3].float().isnan().all()
    assert o["y"][20, d - 1].isnan() and (o["y"][20, : d - 1] == 0).all()
    assert (o["qs"][3, : d // 128] == 127).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_of_zeros_and_extremes(dtype):
    """A row of zeros gives zeros; small and large rows are normalised."""
    n = Norm(6, 256, dtype, res=False)
    n.x[0] = 0
    n.x[1] = n.x[1].sign() * 2.0 ** -14
    n.x[2] = n.x[2].sign() * (2.0 ** 15 if dtype == "f16" else 2.0 ** 60)
    n.x[3] = 0
    n.x[3, 7] = 1.0
    o = n.forward()
    n.check(o)
    assert (o["y"][0] == 0).all() and (o["qs"][0, :2] == 127).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [256, 1024, 4096])
def test_rows_past_the_range_of_their_squares(d, dtype):
    """Values up to the largest float32, beside ordinary rows of the same wave."""
    n = Norm(9, d, dtype, res=False)
    n.x[1] *= 2.0 ** 61
    n.x[4] *= 2.0 ** 100
    n.x[5] = n.x[5].sign() * 2.0 ** 127
    n.x[8, 3] = 2.0 ** 80
    o = n.forward()
    assert (o["rstd"][5] >= 2.0 ** -128).all()
    keep = [i for i in range(9) if i != 5]
    r, gamma = host(n.x), host(n.gamma)
    y, rstd = N4.rmsnorm(r, gamma, EPS)
    within("rstd", host(o["rstd"])[keep], rstd[keep], rstd[keep] * SUM)
    # row 5's rstd, 2^-127, is subnormal; y does not go through it
    within("y", host(o["y"]), y, np.abs(y) * SUM * 2 + half_step(np.abs(y) * (1 + SUM), dtype))


@pytest.mark.parametrize("d", [128, 640, 2112])
def test_no_tokens(d):
    n = Norm(0, d, "bf16", q=False)
    n.forward()
    _, dg = n.backward(n.x, torch.empty(0, device="cuda"))
    assert (dg == 0).all()
    _, dg = n.backward(n.x, torch.empty(0, device="cuda"), accumulate=M.MOE_ACCUM_DW)
    assert (dg == 3).all()


def test_rows_behind_the_last_are_left():
    n = Norm(30, 640, "bf16")
    o = n.out()
    s, n.s = n.s, M.make_shape(21, 640, 128, 1, 0, 1, 1, "bf16")
    n.forward(o)
    assert (o["y"][21:] == 5).all() and (o["r"][21:] == 5).all() and (o["rstd"][21:] == 5).all()
    assert (o["qs"][21:] == 77).all() and (o["q"][21:].float() == 5).all()
    r, rstd = o["r"].clone(), o["rstd"].clone()
    r[21:], rstd[21:] = float("nan"), float("nan")
    dx, dg = n.backward(r, rstd)
    assert (dx[21:] == 5).all() and dg.isfinite().all()
    n.s = s


@pytest.mark.parametrize("T,d", [(700, 640), (5000, 2048), (1500, 4096)])
def test_equal_calls_give_equal_bits(T, d):
    n = Norm(T, d, "bf16")
    o = n.forward()
    a = n.backward(o["r"], o["rstd"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = n.forward(stream=side)
    n.ws.fill_(255)
    torch.cuda.synchronize()
    b = n.backward(o["r"], o["rstd"], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(o[k].view(torch.uint8), p[k].view(torch.uint8)) for k in o)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # a row's result does not depend on the others
    few = Norm(9, d, "bf16")
    few.x, few.res, few.gamma = n.x[100:109].contiguous(), n.res[100:109].contiguous(), n.gamma
    q = few.forward()
    assert all(torch.equal(q[k].view(torch.uint8), o[k][100:109].view(torch.uint8)) for k in o)


def test_graph():
    """Captured forward and backward, replayed with eager work between."""
    n = Norm(333, 1024, "bf16")
    o = n.out()
    dx, dg = torch.empty_like(n.x), torch.empty(1024, device="cuda")
    run = lambda: (n.forward(o), M.moe_rmsnorm_bwd(n.s, n.dy, o["r"], n.gamma, o["rstd"], n.dres,
                                                   dx, dg, 0, n.ws))
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(3):
        n.x.copy_(torch.randn_like(n.x.float()))
        n.dy.copy_(torch.randn_like(n.x.float()))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o["r"], o["y"], o["rstd"], o["qs"], dx, dg)]
        n.check(o)
        run()
        assert all(torch.equal(x, y) for x, y in zip(got, (o["r"], o["y"], o["rstd"], o["qs"], dx,
                                                           dg)))


def test_long_batch():
    """Offsets past 2^31 elements: the last rows of 2.2e9 elements."""
    T, d = 136000, 16384
    s = M.make_shape(T, d, 128, 1, 0, 1, 1, "bf16")
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_()
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y, q = torch.empty_like(x), torch.empty(T, d, dtype=torch.float8_e4m3fn, device="cuda")
    qs = torch.empty(T, M.moe_fp8_scale_ld(d), dtype=torch.uint8, device="cuda")
    rstd, dg = torch.empty(T, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(M.moe_rmsnorm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm(s, x, None, gamma, EPS, None, y, q, qs, rstd)
    few = Norm(7, d, "bf16", res=False)
    few.x, few.gamma = x[-7:].contiguous(), gamma
    o = few.forward()
    few.check(o)
    for k, t in (("y", y), ("q", q), ("qs", qs), ("rstd", rstd)):
        assert torch.equal(o[k].view(torch.uint8), t[-7:].view(torch.uint8)), k
    M.moe_rmsnorm_bwd(s, y, x, gamma, rstd, None, y, dg, 0, ws)
    few.dy = o["y"]
    dx, _ = few.backward(few.x, o["rstd"], dres=False)
    assert torch.equal(dx, y[-7:]) and dg.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1024, 640), (1025, 640), (1024, 2112), (1025, 2112), (17, 512),
                                 (1024, 64), (4, 2048), (5, 2048), (2, 16384)])
def test_dgamma_whichever_way_it_is_summed(T, d, dtype):
    """Around the borders between the ways, and beside a dx that takes dy's or r's place,
    where dy and r can be read once only."""
    n = Norm(T, d, dtype, res=False, q=False)
    o = n.forward()
    dx, dg = n.backward(n.x, o["rstd"])
    n.check_backward(n.x, o["rstd"], dx, dg)
    dy, r = n.dy, n.x
    for k in ("dy", "r"):
        n.dy, at = dy.clone(), r.clone()
        got, dg = n.backward(at, o["rstd"], dx=n.dy if k == "dy" else at)
        n.dy = dy
        assert torch.equal(got, dx), k
        n.check_backward(r, o["rstd"], got, dg)
