"""The norm and the 4-bit experts on another stream than the current one, and two calls at once on
two streams: inputs, outputs and workspaces are made on the current stream, which the others
wait for before the calls.  And long batches in captured graphs that share a workspace."""

import pytest
import torch

import combine_expert_ffn_amd as M
from test_gpu_fp4 import Layer4
from test_gpu_fp8 import LAYERS
from test_gpu_norm import Norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def _on(streams, calls):
    """Each call on its stream, behind the current stream's work; and their ends."""
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for st, call in zip(streams, calls):
        call(st)
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,d", [(1, 2048), (700, 640), (5000, 2048), (1500, 4096)])
def test_norm(T, d):
    n = Norm(T, d, "bf16")
    o = n.forward()
    dx, dg = n.backward(o["r"], o["rstd"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [n.out() for _ in streams]
    _on(streams, [lambda st, p=p: n.forward(p, stream=st) for p in outs])
    for p in outs:
        assert all(torch.equal(p[k].view(torch.uint8), o[k].view(torch.uint8)) for k in o)
    # a workspace each, full of what other calls left
    got = [(torch.full_like(dx, 5.0), torch.full_like(dg, 3.0), torch.full_like(n.ws, 255))
           for _ in streams]
    _on(streams, [lambda st, g=g: M.moe_rmsnorm_bwd(n.s, n.dy, o["r"], n.gamma, o["rstd"], n.dres,
                                                    g[0], g[1], 0, g[2], st) for g in got])
    for a, b, _ in got:
        assert torch.equal(a, dx) and torch.equal(b, dg)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["one_token", "sixteen_each", "ragged_tiles", "tiles_window",
                                  "tiles_halves"])
def test_experts(name, dtype):
    L = Layer4(*LAYERS[name], dtype, True)
    want = L.forward()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [{n: torch.full_like(t, 5.0) for n, t in want.items()} for _ in streams]
    spaces = [torch.full_like(L.ws, 255) for _ in streams]
    _on(streams, [lambda st, o=o, ws=ws: M.moe_expert_ffn_fwd_fp4(
        L.s, L.q, L.qs, L.mb.pair_of_row, L.mb.offsets, L.mb.tile_offsets, L.w4, o["h"], o["a"],
        o["y"], ws, st) for o, ws in zip(outs, spaces)])
    for o in outs:
        assert all(torch.equal(o[n], want[n]) for n in want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1500, 640), (5000, 2048), (1100, 8320)])
def test_norm_graphs_share_a_workspace(T, d, dtype):
    """dgamma's partial sums of two captured backward passes in one workspace, which eager work
    overwrites between the replays."""
    n, other = Norm(T, d, dtype, q=False), Norm(T, d, dtype, q=False, seed=1)
    calls, outs = [], []
    for m in (n, other):
        o = m.out()
        dx, dg = torch.empty_like(m.x), torch.empty(d, device="cuda")
        outs.append((o["r"], o["y"], o["rstd"], dx, dg))
        calls.append(lambda m=m, o=o, dx=dx, dg=dg: (m.forward(o), M.moe_rmsnorm_bwd(
            m.s, m.dy, o["r"], m.gamma, o["rstd"], m.dres, dx, dg, 0, n.ws)))
    for call in calls:
        call()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    for graph, call in zip(graphs, calls):
        with torch.cuda.graph(graph):
            call()
    for k in range(3):
        for m in (n, other):
            m.x.copy_(torch.randn_like(m.x.float()))
            m.dy.copy_(torch.randn_like(m.x.float()))
        for graph in graphs if k % 2 else graphs[::-1]:
            graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in out] for out in outs]
        n.ws.fill_(255)
        for call, out, was in zip(calls, outs, got):
            call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, was)), k
