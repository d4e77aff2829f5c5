"""The norm and the experts on 4-bit weights together with the calls around them: layers as a
serving loop runs them (norm -> route -> dispatch -> experts -> combine, and the next
layer's norm adds the residual), and a training step (4-bit forward, gradients through
the weights read back, norm backward).  All calls of a run share one workspace.

The forward is checked call by call against float64 of the call's own device inputs.  The
gradients are checked against float64 autograd at the stored h, a and yp, with a bound per
element that follows every 16-bit rounding (half a step u of each stored value)
through the absolute values of what comes after it; FLOAT bounds, relative to the sum
of magnitudes, float32 sums of at most 2^9 terms one after another (2^-15) and the
sigmoid's few 2^-22.  All fixed before the first run.
"""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
import oracle as O
from moe_harness import exact, host
from test_gpu_fp4 import Layer4
from test_gpu_norm import DT, EPS, Norm, half_step, within

pytestmark = pytest.mark.gpu

FLOAT = 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


class Stack:
    """Two layers' weights, the buffers of each, and one workspace for all calls."""

    def __init__(self, T, d, F, E, e_lo, E_l, K, dtype, seed=0):
        self.s = s = M.make_shape(T, d, F, E, e_lo, E_l, K, dtype)
        self.T, self.d, self.F, self.E, self.E_l, self.K = T, d, F, E, E_l, K
        self.dtype, dt = dtype, DT[dtype]
        rng = np.random.default_rng(seed + T)
        self.g = g = lambda *sh, std=1.0: torch.from_numpy(
            (rng.normal(size=sh) * std).astype(np.float32)).to(dt).cuda()
        e = lambda *sh: torch.full(sh, 5.0, dtype=dt, device="cuda")
        self.x0, self.res0 = g(T, d), g(T, d)
        self.layers = []
        for _ in range(2):
            L = type("L", (), {})()
            L.gamma, L.W_r = (1 + 0.3 * g(d).float()).to(dt), g(d, E, std=d ** -0.5)
            L.W = [g(E_l, 2 * F, d, std=d ** -0.5), g(E_l, d, F, std=F ** -0.5)]
            L.w4 = M.Fp4Weights(s)
            M.moe_quant_weights_fp4(s, *L.W, L.w4)
            L.mb = M.MicroBatch(s, fused=True)
            L.r, L.y, L.rstd = e(T, d), e(T, d), torch.full((T,), 5.0, device="cuda")
            L.q = torch.zeros(T, d, device="cuda").to(torch.float8_e4m3fn)
            L.qs = torch.zeros(T, M.moe_fp8_scale_ld(d), dtype=torch.uint8, device="cuda")
            L.mb.h.fill_(5.0), L.mb.a.fill_(5.0), L.mb.yp.fill_(5.0)
            self.layers.append(L)
        self.ws = torch.empty(max(M.moe_workspace_bytes(s), M.moe_fp4_workspace_bytes(s),
                                  M.moe_rmsnorm_workspace_bytes(s)), dtype=torch.uint8,
                              device="cuda")

    def layer(self, L, x, res, serving=True):
        s, mb = self.s, L.mb
        M.moe_rmsnorm(s, x, res, L.gamma, EPS, L.r, L.y, L.q, L.qs, L.rstd)
        M.moe_route(s, M.MOE_ROUTE_TOPK, L.y, L.W_r, None, mb.logits, mb.idx, mb.gates, self.ws)
        M.moe_dispatch(s, None, mb.idx, mb.counts, mb.offsets, mb.row_of_pair, mb.pair_of_row,
                       mb.tile_offsets, None, self.ws)
        M.moe_expert_ffn_fwd_fp4(s, L.q, L.qs, mb.pair_of_row, mb.offsets, mb.tile_offsets, L.w4,
                                 None if serving else mb.h, None if serving else mb.a, mb.yp,
                                 self.ws)
        M.moe_combine(s, mb.yp, mb.gates, mb.row_of_pair, mb.out)

    def forward(self):
        A, B = self.layers
        self.layer(A, self.x0, self.res0)
        self.layer(B, A.mb.out, A.r)

    def results(self):
        return [t for L in self.layers for t in (L.r, L.y, L.q.view(torch.uint8), L.qs, L.rstd,
                                                 L.mb.logits, L.mb.gates, L.mb.out)]

    def check(self, L, x, res, serving=True):
        n = object.__new__(Norm)
        n.s, n.T, n.d, n.dtype = self.s, self.T, self.d, self.dtype
        n.x, n.res, n.gamma, n.q = x, res, L.gamma, True
        n.check({"r": L.r, "y": L.y, "q": L.q, "qs": L.qs, "rstd": L.rstd})
        mb, y, W_r = L.mb, host(L.y), host(L.W_r)
        within("logits", host(mb.logits), y @ W_r, FLOAT * (np.abs(y) @ np.abs(W_r)))
        idx, gates = O.topk_route(host(mb.logits), self.K, "f64")
        exact("idx", host(mb.idx), idx)
        within("gates", host(mb.gates), gates, FLOAT * gates)
        f = object.__new__(Layer4)
        f.dtype, f.gather, f.d, f.F, f.K, f.E_l = self.dtype, True, self.d, self.F, self.K, self.E_l
        f.off, f.q, f.qs, f.w4 = host(mb.offsets), L.q, L.qs, L.w4
        f.N = int(f.off[-1])
        f.pair = host(mb.pair_of_row)[: f.N]
        f.check_forward({"h": None if serving else mb.h, "a": None if serving else mb.a,
                         "y": mb.yp})
        yp, rop = host(mb.yp), host(mb.row_of_pair)
        out = O.combine(yp, host(mb.gates), rop, "f64")
        mag = O.combine(np.abs(yp), host(mb.gates), rop, "f64")
        within("out", host(mb.out), out, FLOAT * mag + half_step(mag, self.dtype))


SHAPES = {
    "one_token": (1, 256, 128, 8, 0, 8, 2),
    "few_rows": (37, 384, 256, 8, 2, 4, 3),
    "ragged": (300, 640, 384, 16, 0, 16, 4),
    "tiles": (900, 256, 384, 3, 0, 3, 2),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", SHAPES)
def test_serving_layers(name, dtype):
    S = Stack(*SHAPES[name], dtype)
    S.forward()
    A, B = S.layers
    S.check(A, S.x0, S.res0)
    S.check(B, A.mb.out, A.r)


@pytest.mark.parametrize("name", ["one_token", "few_rows", "tiles"])
def test_serving_layers_in_graphs(name):
    """Two graphs, one per layer, that share the workspace; other inputs in each replay, and
    eager work with the same workspace in between."""
    S, E = Stack(*SHAPES[name], "bf16"), Stack(*SHAPES[name], "bf16")
    A, B = S.layers
    S.forward()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        S.layer(A, S.x0, S.res0)
    with torch.cuda.graph(graphs[1]):
        S.layer(B, A.mb.out, A.r)
    for k in range(4):
        x, res = S.g(S.T, S.d), S.g(S.T, S.d)
        for X in (S, E):
            X.x0.copy_(x), X.res0.copy_(res)
        E.forward()
        for t in S.results():
            t.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for got, want in zip(S.results(), E.results()):
            assert torch.equal(got, want), k
        S.ws.fill_(255)
        S.layer(A, S.x0, S.res0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", SHAPES)
def test_training_step(name, dtype):
    """loss = <dout, r + layer(norm(r))>, r = x + res."""
    S = Stack(*SHAPES[name], dtype, seed=1)
    s, L, dt = S.s, S.layers[0], DT[dtype]
    mb, T, d, F, K, E_l = L.mb, S.T, S.d, S.F, S.K, S.E_l
    S.layer(L, S.x0, S.res0, serving=False)
    S.check(L, S.x0, S.res0, serving=False)
    dout, cap = S.g(T, d), T * K
    xp = torch.empty(cap, d, dtype=dt, device="cuda")
    W = [torch.empty_like(w) for w in L.W]
    z = lambda *sh: torch.full(sh, 5.0, device="cuda")
    dW = [z(*w.shape) for w in W]
    dW_r, dgamma = z(d, S.E), z(d)
    dx = torch.empty(T, d, dtype=dt, device="cuda")
    M.moe_dequant_weights_fp4(s, L.w4, *W)
    M.moe_dispatch(s, L.y, mb.idx, mb.counts, mb.offsets, mb.row_of_pair, mb.pair_of_row,
                   mb.tile_offsets, xp, S.ws)
    M.moe_combine_bwd(s, dout, mb.yp, mb.gates, mb.row_of_pair, mb.dyp, mb.dgates)
    M.moe_route_bwd(s, M.MOE_ROUTE_TOPK, mb.dgates, mb.gates, mb.idx, L.y, mb.dlogits, dW_r, 0,
                    S.ws)
    M.moe_ffn_dgrad(s, mb.dyp, mb.h, mb.offsets, mb.tile_offsets, *W, mb.dh, mb.dxp, S.ws)
    M.moe_ffn_wgrad(s, xp, mb.a, mb.dh, mb.dyp, mb.offsets, *dW, 0)
    M.moe_dispatch_bwd(s, mb.dxp, mb.row_of_pair, mb.idx, mb.dlogits, L.W_r, mb.dx, 0, S.ws)
    M.moe_rmsnorm_bwd(s, mb.dx, L.r, L.gamma, L.rstd, dout, dx, dgamma, 0, S.ws)
    torch.cuda.synchronize()

    # float64 autograd at the stored values
    f64 = lambda t: torch.from_numpy(host(t))
    at = lambda value, node: value + (node - node.detach())
    N, off = int(mb.offsets[-1]), host(mb.offsets)
    pair = torch.from_numpy(host(mb.pair_of_row)[:N].astype(np.int64))
    idx = torch.from_numpy(host(mb.idx).astype(np.int64))
    r, gamma, W_r = f64(L.r), f64(L.gamma), f64(L.W_r)
    W4 = [torch.from_numpy(w) for w in Layer4.weights(L)]
    leaves = [r, gamma, W_r, *W4]
    for t in leaves:
        t.requires_grad_()
    xhat = r * (r.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
    y = at(f64(L.y), xhat * gamma)
    logits = y @ W_r
    gates = torch.softmax(logits.gather(1, idx), -1)
    each = lambda A, Ws: torch.cat([A[off[e]:off[e + 1]] @ Ws[e].T for e in range(E_l)])
    h = at(f64(mb.h[:N]), each(y[pair // K], W4[0]))
    a = at(f64(mb.a[:N]), torch.nn.functional.silu(h[:, :F]) * h[:, F:])
    yp = at(f64(mb.yp[:N]), each(a, W4[1]))
    yp.retain_grad(), h.retain_grad(), y.retain_grad(), logits.retain_grad()
    rows = yp * gates.reshape(-1)[pair][:, None]
    out = torch.zeros(T, d, dtype=torch.float64).index_add(0, pair // K, rows)
    (f64(dout) * (r + out)).sum().backward()

    # the bounds
    num = lambda t: np.abs(t.detach().numpy())
    half = lambda v: half_step(v, dtype) * (1 + 2.0 ** -6)
    per = lambda A, Ws: np.concatenate([A[off[e]:off[e + 1]] @ np.abs(Ws[e]) for e in range(E_l)])
    Wa, p = [num(w) for w in W4], pair.numpy()
    dyp, dh, dy, dlog = num(yp.grad), num(h.grad), num(y.grad), num(logits.grad)
    e_dyp = half(dyp) + FLOAT * dyp
    g_, u_ = h.detach().numpy()[:, :F], h.detach().numpy()[:, F:]
    sg = 1 / (1 + np.exp(-g_))
    k_h = np.concatenate([np.abs(u_ * sg * (1 + g_ * (1 - sg))), np.abs(g_ * sg)], 1)
    da, e_da = per(dyp, Wa[1]), per(e_dyp, Wa[1])
    e_dh = k_h * np.tile(e_da + FLOAT * da, 2) + half(dh) + FLOAT * np.tile(
        da * (np.abs(u_) + np.abs(g_)), 2)
    e_dxp = per(e_dh + FLOAT * dh, Wa[0])
    e_dxp += half(per(dh, Wa[0]))
    dg = np.zeros((T, K))
    dg.reshape(-1)[p] = (num(f64(dout))[p // K] * num(yp)).sum(-1)
    e_dlog = np.zeros((T, S.E))
    np.put_along_axis(e_dlog, idx.numpy(),
                      FLOAT * num(gates) * (dg + (num(gates) * dg).sum(-1, keepdims=True)) * 4, 1)
    e_dy = e_dlog @ num(W_r).T + FLOAT * (dlog @ num(W_r).T)
    np.add.at(e_dy, p // K, e_dxp)
    e_dy += half(dy + e_dy)
    xh, rstd = num(xhat), num(xhat).max(-1) / np.abs(host(L.r)).max(-1)
    e_dn, dn = (e_dy + FLOAT * dy) * num(gamma), dy * num(gamma)
    e_dx = rstd[:, None] * (e_dn + xh * (xh * (e_dn + FLOAT * dn)).mean(-1, keepdims=True))
    e_dx += half(num(r.grad) + e_dx)
    within("dx", host(dx), r.grad.numpy(), e_dx)
    within("dgamma", host(dgamma), gamma.grad.numpy(), ((e_dy + FLOAT * dy) * xh).sum(0))
    within("dW_r", host(dW_r), W_r.grad.numpy(), num(y).T @ (e_dlog + FLOAT * dlog))
    for n, got, w, left, e_left, right in (("dW_gu", dW[0], W4[0], dh, e_dh, num(y)[p // K]),
                                           ("dW_down", dW[1], W4[1], dyp, e_dyp, num(a))):
        tol = np.stack([(e_left + FLOAT * left)[off[e]:off[e + 1]].T @ right[off[e]:off[e + 1]]
                        for e in range(E_l)])
        within(n, host(got), w.grad.numpy(), tol + 2.0 ** -149)
