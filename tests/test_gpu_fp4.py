"""The experts on 4-bit weights on the GPU against the float64 oracle.  Quantisation and
reading back are exact; the products' tolerances are those of the 8-bit ones (derived
there): the same row format, instruction and accumulation, other weights."""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from oracle import norm_fp4_oracle as N4
from moe_harness import exact, host
from test_gpu_fp8 import LAYERS, DT, Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


# ---- quantisation: exact ----------------------------------------------------
def _weights(rng, E_l, d, F, dtype):
    W = [(rng.normal(size=sh) * np.exp(3 * rng.normal(size=sh[:-1] + (1,)))).astype(np.float32)
         for sh in ((E_l, 2 * F, d), (E_l, d, F))]
    W[0][0, 0, :32] = 0.0                                    # an empty block
    W[0][0, 0, 32:64] = np.resize([7.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], 32)  # borders
    W[0][0, 1, 32:64] = -np.resize([6.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], 32)
    W[0][0, 1, 64:96] = np.resize([7.5, 0.5, 1.5, 2.5, 3.5, 5.0, 7.0, 10.0], 32)
    W[0][-1, 2, 5], W[0][-1, 3, d - 1], W[1][-1, 1, 40] = np.nan, np.inf, -np.inf
    big = {"bf16": 3.0e38, "f16": 65504.0, "f32": 3.4e38}[dtype]
    W[1][0, 0, 0] = big
    W[1][0, 1, :32] = 6e-8 if dtype == "f16" else 1e-39      # the smallest scales
    W[1][0, 2, :32] = 6e-8 if dtype == "f16" else 1e-41
    W[1][0, 3, :32] = -0.0
    return [torch.from_numpy(w).to(DT[dtype]) for w in W]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E_l,d,F", [(1, 128, 128), (3, 640, 256), (2, 256, 1408), (5, 384, 384)])
def test_quant_and_read_back(E_l, d, F, dtype):
    W = _weights(np.random.default_rng(d + F), E_l, d, F, dtype)
    s = M.make_shape(1, d, F, E_l, 0, E_l, 1, dtype)
    w = M.Fp4Weights(s)
    M.moe_quant_weights_fp4(s, W[0].cuda(), W[1].cuda(), w)
    back = [torch.zeros_like(x, device="cuda") for x in W]
    M.moe_dequant_weights_fp4(s, w, *back)
    for name, Wm, b in (("gu", W[0], back[0]), ("down", W[1], back[1])):
        code, byte = N4.quant4(Wm.double().numpy())
        exact(name + "_s", host(getattr(w, name + "_s")), byte)
        exact(name, N4.unpack(host(getattr(w, name))), code)
        v = torch.from_numpy(N4.value4(code, byte)).to(DT[dtype])
        assert torch.equal(b.cpu().isnan(), v.isnan())
        assert torch.equal(b.cpu().nan_to_num(7.0), v.nan_to_num(7.0))


def test_every_code_and_scale_reads_back():
    """All 256 scale bytes with all codes, in the three types."""
    d, F = 128, 128
    for dtype in ("bf16", "f16", "f32"):
        s = M.make_shape(1, d, F, 1, 0, 1, 1, dtype)
        w = M.Fp4Weights(s)
        code = torch.arange(16, dtype=torch.uint8)
        pair = (code[::2] | code[1::2] << 4).repeat(d // 16)          # 0 .. 15 again and again
        w.gu.copy_(pair.expand(1, 2 * F, d // 2))
        w.gu_s.copy_(torch.arange(256, dtype=torch.uint8).view(1, 2 * F, 1).expand(1, 2 * F, d // 32))
        w.down.copy_(pair.expand(1, d, F // 2))
        w.down_s.copy_((torch.arange(d * 4) % 256).to(torch.uint8).view(1, d, F // 32))
        out = [torch.zeros(1, 2 * F, d, dtype=DT[dtype], device="cuda"),
               torch.zeros(1, d, F, dtype=DT[dtype], device="cuda")]
        M.moe_dequant_weights_fp4(s, w, *out)
        for got, c, b in zip(out, (w.gu, w.down), (w.gu_s, w.down_s)):
            v = torch.from_numpy(N4.value4(N4.unpack(host(c)), host(b))).to(DT[dtype])
            assert torch.equal(got.cpu().isnan(), v.isnan()), dtype
            assert torch.equal(got.cpu().nan_to_num(7.0), v.nan_to_num(7.0)), dtype


# ---- the experts ------------------------------------------------------------
class Layer4(Layer):
    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.w4 = M.Fp4Weights(self.s)
        M.moe_quant_weights_fp4(self.s, self.W_gu, self.W_down, self.w4)
        self.ws = torch.empty(M.moe_fp4_workspace_bytes(self.s), dtype=torch.uint8, device="cuda")

    def weights(self):
        w = self.w4
        return (N4.value4(N4.unpack(host(w.gu)), host(w.gu_s)),
                N4.value4(N4.unpack(host(w.down)), host(w.down_s)))

    def forward(self, h=True, a=True, stream=None):
        out = {"h": self.buf(2 * self.F) if h else None, "a": self.buf(self.F) if a else None,
               "y": self.buf(self.d)}
        M.moe_expert_ffn_fwd_fp4(self.s, self.q, self.qs,
                                 self.mb.pair_of_row if self.gather else None, self.mb.offsets,
                                 self.mb.tile_offsets, self.w4, out["h"], out["a"], out["y"],
                                 self.ws, stream)
        return out


@pytest.mark.parametrize("gather", [True, False], ids=["tokens", "dispatched"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", LAYERS)
def test_forward(name, dtype, gather):
    L = Layer4(*LAYERS[name], dtype, gather, seed=len(name))
    L.check_forward(L.forward())


@pytest.mark.parametrize("T,E", [(40, 8), (700, 4)])
def test_no_local_rows(T, E):
    L = Layer4(T, 128, 128, E, 2, 2, 2, "bf16", True, only=[0, 1])
    assert L.N == 0
    L.untouched(**L.forward())


@pytest.mark.parametrize("T", [700, 2100])
def test_one_expert_has_every_row(T):
    L = Layer4(T, 128, 128, 8, 0, 8, 1, "bf16", True, only=[5])
    assert L.off[5] == 0 and L.off[6] == T
    L.check_forward(L.forward())


@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_window"])
def test_optional_outputs(name):
    """h and a left out (serving) change nothing in y."""
    L = Layer4(*LAYERS[name], "bf16", True)
    full = L.forward()
    for h, a in ((False, False), (True, False), (False, True)):
        part = L.forward(h, a)
        for n in ("h", "a", "y"):
            assert part[n] is None or torch.equal(part[n], full[n]), n


@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_window"])
def test_gathered_equals_dispatched(name):
    L = Layer4(*LAYERS[name], "bf16", True)
    f = L.forward()
    rows = torch.zeros(L.T * L.K, dtype=torch.int64)
    rows[: L.N] = torch.from_numpy(L.pair // L.K)
    P = Layer4(*LAYERS[name], "bf16", False)
    P.q = L.q.view(torch.uint8)[rows.cuda()].view(torch.float8_e4m3fn).contiguous()
    P.qs, P.w4 = L.qs[rows.cuda()].contiguous(), L.w4
    assert all(torch.equal(x, y) for x, y in zip(f.values(), P.forward().values()))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_odd_blocks"])
def test_nonfinite_token_stays_in_its_rows(name, dtype):
    L = Layer4(*LAYERS[name], dtype, True)
    good = L.forward()
    x = L.x.clone()
    x[7, 3], x[11, 64] = float("nan"), float("inf")
    L.q, L.qs = L.quantise(x, L.T)
    bad = L.forward()
    hit = np.isin(L.pair // L.K, [7, 11])
    assert hit.any()
    for n in ("h", "a", "y"):
        assert torch.equal(bad[n][: L.N][~hit], good[n][: L.N][~hit]), n
        assert not np.isfinite(host(bad[n], L.N)[hit]).any(), n


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_odd_blocks"])
def test_a_nan_block_reaches_its_outputs_only(name, dtype):
    """A weight that is not finite: its output column of its expert is NaN."""
    L = Layer4(*LAYERS[name], dtype, True)
    good = L.forward()
    j, e = L.F // 2 + 1, 0
    L.W_gu[e, L.F + j, 70] = float("inf")       # the up row of output j
    L.W_down[e, 33, 100] = float("nan")
    M.moe_quant_weights_fp4(L.s, L.W_gu, L.W_down, L.w4)
    bad = L.forward()
    lo, hi = L.off[e], L.off[e + 1]
    assert hi > lo
    h, g = host(bad["h"], L.N), host(good["h"], L.N)
    assert np.isnan(h[lo:hi, L.F + j]).all()
    h[lo:hi, L.F + j] = g[lo:hi, L.F + j]
    assert np.array_equal(h, g)
    a, g = host(bad["a"], L.N), host(good["a"], L.N)
    assert np.isnan(a[lo:hi, j]).all()
    a[lo:hi, j] = g[lo:hi, j]
    assert np.array_equal(a, g)
    y, g = host(bad["y"], L.N), host(good["y"], L.N)
    assert np.isnan(y[lo:hi]).all()             # through a's quantised row
    assert np.array_equal(y[hi:], g[hi:])


@pytest.mark.parametrize("T", [4, 8224])
def test_weights_past_32_bits(T):
    """256 experts of 8192 x 4096 (8.6 GB of gate and up in 4 bits): the rows of the last
    expert, for a few rows and for many."""
    d, F, E, K = 4096, 8192, 256, 8
    s = M.make_shape(T, d, F, E, 0, E, K, "bf16")
    gen = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda hi, *sh: torch.randint(hi[0], hi[1], sh, dtype=torch.uint8, device="cuda",
                                        generator=gen)
    w = M.Fp4Weights(s, gu=rnd((0, 256), E, 2 * F, d // 2), gu_s=rnd((118, 122), E, 2 * F, d // 32),
                     down=rnd((0, 256), E, d, F // 2), down_s=rnd((118, 122), E, d, F // 32))
    ws = torch.empty(max(M.moe_fp4_workspace_bytes(s), M.moe_workspace_bytes(
        M.make_shape(T, d, 64, E, 0, E, K, "bf16"))), dtype=torch.uint8, device="cuda")
    idx = torch.stack([(torch.arange(T) * 37 + 249 + k * 31) % E for k in range(K)], 1)
    idx[:4, 0] = 255
    idx[:4, 1:] = torch.arange(1, K) * 5
    i32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device="cuda")
    counts, offsets, tiles, rop, por = i32(E), i32(E + 1), i32(E + 1), i32(T * K), i32(T * K)
    M.moe_dispatch(s, None, idx.to(torch.int32).cuda(), counts, offsets, rop, por, tiles, None, ws)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=gen)
    q = torch.zeros(T, d, device="cuda").to(torch.float8_e4m3fn)
    qs = torch.zeros(T, M.moe_fp8_scale_ld(d), dtype=torch.uint8, device="cuda")
    M.moe_quant_rows_fp8(s, x, T, None, q, qs)
    h = torch.empty(T * K, 2 * F, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(T * K, d, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_ffn_fwd_fp4(s, q, qs, por, offsets, tiles, w, h, None, y, ws)
    # the last expert's rows as a layer of one expert
    lo, hi = int(offsets[E - 1]), int(offsets[E])
    lo = max(lo, hi - 40)
    assert hi - lo >= 4
    L = object.__new__(Layer4)
    L.dtype, L.gather, L.d, L.F, L.K, L.E_l = "bf16", True, d, F, K, 1
    L.N, L.off, L.pair = hi - lo, np.array([0, hi - lo]), host(por)[lo:hi]
    L.q, L.qs = q, qs
    L.w4 = type("W", (), {n: getattr(w, n)[E - 1:] for n in M.FP4_WEIGHT_FIELDS})
    L.check_forward({"h": h[lo:hi], "a": None, "y": y[lo:hi]})


@pytest.mark.parametrize("name", ["sixteen_each", "tiles_window"])
def test_equal_calls_give_equal_bits(name):
    """Again, on another stream, and with what the workspace held before."""
    L = Layer4(*LAYERS[name], "bf16", True)
    f = L.forward()
    L.ws.fill_(255)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = L.forward(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(f[n], g[n]) for n in f)


@pytest.mark.parametrize("name", ["sixteen_each", "tiles_window"])
def test_graph(name):
    L = Layer4(*LAYERS[name], "bf16", True)
    out = L.forward()
    run = lambda: M.moe_expert_ffn_fwd_fp4(L.s, L.q, L.qs, L.mb.pair_of_row, L.mb.offsets,
                                           L.mb.tile_offsets, L.w4, out["h"], out["a"], out["y"],
                                           L.ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(3):
        L.q, L.qs = (t.copy_(n) for t, n in zip((L.q, L.qs), L.quantise(
            torch.randn_like(L.x.float()).to(L.x.dtype), L.x.shape[0])))
        for t in out.values():
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in out.items()}
        L.check_forward(got)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n][: L.N], out[n][: L.N]) for n in out)


def test_weights_replaced_or_moved():
    """The struct follows a tensor that is replaced or whose memory is."""
    L = Layer4(*LAYERS["sixteen_each"], "bf16", True)
    a = L.forward()["y"]
    fresh = L.w4.gu.clone()
    L.w4.gu.zero_()
    L.w4.gu = fresh
    assert torch.equal(L.forward()["y"], a)
    moved = L.w4.down_s.clone()
    L.w4.down_s.zero_()
    L.w4.down_s.data = moved
    assert torch.equal(L.forward()["y"], a)
    L.w4.down = torch.zeros(3, dtype=torch.uint8, device="cuda")
    with pytest.raises(M.MoeError):
        L.forward()


def test_other_shape_is_refused():
    L = Layer4(*LAYERS["sixteen_each"], "bf16", True)
    s = M.make_shape(16, 256, 128, 8, 0, 8, 8, "bf16")
    with pytest.raises(M.MoeError):
        M.moe_quant_weights_fp4(s, L.W_gu, L.W_down, L.w4)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,d,F,E,E_l,K,on", [
    (100, 256, 128, 64, 16, 1, [0]), (257, 256, 128, 4, 4, 1, [2]),
    (700, 128, 128, 128, 16, 1, [9]),
    (1000, 1024, 256, 8, 8, 1, [5]), (150, 128, 256, 64, 16, 8, list(range(8))),
    (600, 256, 2048, 512, 1, 8, [0]),       # more passes than the grid holds at once
    (600, 128, 2048, 512, 3, 8, [1, 2, 7, 8, 9, 10, 11, 12]),
    (333, 640, 384, 256, 256, 8, [3, 64, 65, 127, 128, 191, 192, 255]),
])
def test_all_tokens_on_the_same_experts(T, d, F, E, E_l, K, on, dtype):
    L = Layer4(T, d, F, E, 0, E_l, K, dtype, True, only=on)
    assert max(L.off[1:] - L.off[:-1]) == T
    L.check_forward(L.forward())


@pytest.mark.parametrize("T,d,F,E,E_l,K,small", [
    (129, 512, 256, 128, 128, 7, True),      # 7 rows each on average, up to 129
    (4096, 256, 128, 64, 8, 1, False),       # 64 on average, in passes of 16, up to 4096
    (1100, 256, 128, 512, 1, 4, False),      # 9 rows on average, up to 1100
    (16384, 256, 128, 512, 1, 8, False),
])
def test_which_kernels_run(T, d, F, E, E_l, K, small):
    L = Layer4(T, d, F, E, 0, E_l, K, "bf16", True)
    M.moe_timing_enable()
    try:
        M.moe_timing_reset()
        out = L.forward()
        torch.cuda.synchronize()
        names = set(M.moe_timing_report())
    finally:
        M.moe_timing_disable()
    assert len(names) == 2 and all(n.endswith("_small") == small for n in names), names
    L.check_forward(out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,F", [(128, 128), (384, 256), (512, 512), (640, 384), (1024, 1152),
                                 (2176, 128), (256, 2432)])
def test_every_length_of_the_reduction(d, F, dtype):
    """One block to a wave, two, two units of two, and more; the last one half."""
    for T, E, K in ((3, 4, 2), (50, 4, 2), (150, 4, 1)):
        L = Layer4(T, d, F, E, 0, E, K, dtype, True, seed=d)
        L.check_forward(L.forward())


@pytest.mark.parametrize("T,d,F,E,K", [
    (1, 256, 128, 8, 8), (3, 128, 256, 64, 8), (16, 256, 128, 16, 4), (40, 640, 384, 8, 6),
    (150, 128, 128, 16, 8), (700, 128, 128, 4, 4)])
def test_tokens_that_name_an_expert_more_than_once(T, d, F, E, K):
    """An expert then has up to K T rows."""
    L = Layer4(T, d, F, E, 0, E, K, "bf16", True)
    L.mb.idx.copy_(torch.where(torch.arange(K) == K - 1, E - 1, 0).to(torch.int32).expand(T, K))
    ws = torch.empty(M.moe_workspace_bytes(L.s), dtype=torch.uint8, device="cuda")
    M.moe_dispatch(L.s, None, L.mb.idx, L.mb.counts, L.mb.offsets, L.mb.row_of_pair,
                   L.mb.pair_of_row, L.mb.tile_offsets, None, ws)
    L.off = host(L.mb.offsets)
    L.N, L.pair = int(L.off[-1]), host(L.mb.pair_of_row)[: int(L.off[-1])]
    assert L.N == T * K and L.off[1] == T * (K - 1)
    L.check_forward(L.forward())
