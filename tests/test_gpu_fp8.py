"""The 8-bit expert path on the GPU against the float64 oracle.

Tolerances, fixed before the first run.  EPS_SUM = 2^-12 of sum |terms| bounds a
product's sum: the 8-bit matrix instruction aligns each group of products to the
group's largest and drops what lies below its last bit (a separate measurement on
random operands: at most 9.1e-5 of sum |terms| = 2^-13.4); float32 accumulation
over at most 32768 terms adds far less.  Stored 16-bit values round once more, by
at most half a step.  A value quantised between the two products may fall on
either side of a rounding border within its own error, so the second product's
bound adds, per term, how far that quantisation can move (``_requant_slack``).
The sigmoid's exp2 and reciprocal cost a few 2^-23 relative.
"""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
import oracle as O
from oracle import fp8_oracle as Q
from moe_harness import exact, host

pytestmark = pytest.mark.gpu

EPS_SUM = 2.0 ** -12
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def half_step(ref, dtype):
    """Half a step at |ref|, doubled for a value that the error carries into the
    next binade, and the flat range."""
    return np.abs(ref) * {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype] + {
        "bf16": 2.0 ** -126, "f16": 2.0 ** -24}[dtype]


def within(name, got, ref, tol):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.size:
        return
    assert np.isfinite(got).all(), f"{name}: not finite"
    over = np.abs(got - ref) - tol
    i = np.unravel_index(int(over.argmax()), over.shape)
    assert over[i] <= 0, f"{name}{i}: got {got[i]}, ref {ref[i]}, tolerance {tol[i]}, " \
                         f"{int((over > 0).sum())} of {over.size} over"


def _requant_slack(x, err):
    """How far requant(x) can move when x moves by at most err."""
    base = Q.requant(x)
    b = np.abs(x).reshape(x.shape[:-1] + (x.shape[-1] // 128, 128))
    e = err.reshape(b.shape)
    slack = np.zeros_like(x)
    for lim in ((b + e).max(-1), (b - e).max(-1)):   # the scale with the largest magnitude moved
        s = np.repeat(np.ldexp(1.0, Q.scale_byte(np.maximum(lim, 0)) - 127), 128, -1)
        for z in (x - err, x + err):
            slack = np.maximum(slack, np.abs(Q.round_e4m3(np.clip(z / s, -448, 448)) * s - base))
    return slack


class Layer:
    """Random routing, quantised operands on the GPU, and their float64 values."""

    def __init__(self, T, d, F, E, e_lo, E_l, K, dtype, gather, seed=0, only=None):
        self.s = M.make_shape(T, d, F, E, e_lo, E_l, K, dtype)
        self.dtype, self.gather = dtype, gather
        self.T, self.d, self.F, self.K, self.E_l = T, d, F, K, E_l
        rng = np.random.default_rng(seed)
        score = rng.random((T, E))
        if only is not None:          # all tokens to these experts first
            score[:, only] += 1
        idx = np.argsort(-score, 1)[:, :K].astype(np.int32)
        self.mb = mb = M.MicroBatch(self.s)
        ws = torch.empty(M.moe_workspace_bytes(self.s), dtype=torch.uint8, device="cuda")
        mb.idx.copy_(torch.from_numpy(idx))
        M.moe_dispatch(self.s, None, mb.idx, mb.counts, mb.offsets,
                       mb.row_of_pair, mb.pair_of_row, mb.tile_offsets, None, ws)
        self.off = host(mb.offsets)
        self.N = int(self.off[-1])
        self.pair = host(mb.pair_of_row)[: self.N]
        self.gates = rng.uniform(0.05, 1, T * K).astype(np.float32)
        rows = T if gather else T * K
        g = lambda *sh, std=1.0: torch.from_numpy(
            (rng.normal(size=sh) * std).astype(np.float32)).cuda().to(DT[dtype])
        self.x = g(max(rows, 1), d)[:rows]
        self.q, self.qs = self.quantise(self.x, rows)
        self.W_gu, self.W_down = g(E_l, 2 * F, d, std=d ** -0.5), g(E_l, d, F, std=F ** -0.5)
        self.w = M.Fp8Weights(self.s)
        M.moe_quant_weights_fp8(self.s, self.W_gu, self.W_down, self.w)
        self.h = g(max(T * K, 1), 2 * F)[: T * K]
        self.ws = torch.empty(M.moe_fp8_workspace_bytes(self.s), dtype=torch.uint8, device="cuda")

    def quantise(self, x, rows):
        q = torch.zeros(max(rows, 1), self.d, device="cuda").to(torch.float8_e4m3fn)
        qs = torch.zeros(max(rows, 1), M.moe_fp8_scale_ld(self.d), dtype=torch.uint8,
                         device="cuda")
        M.moe_quant_rows_fp8(self.s, x, rows, None, q, qs)
        return q, qs

    def rows(self):
        """The dispatched rows' quantised values."""
        v = Q.value(host(self.q.float()), host(self.qs)[:, : self.d // 128])
        return v[self.pair // self.K] if self.gather else v[: self.N]

    def weights(self):
        kb = lambda t, k: host(t)[..., : k // 128]
        return (Q.value(host(self.w.gu.float()), kb(self.w.gu_s, self.d), 128),
                Q.value(host(self.w.down.float()), kb(self.w.down_s, self.F), 128))

    def buf(self, cols):
        """A [T*K, cols] buffer whose untouched rows keep the value 5."""
        n = self.T * self.K
        return torch.full((max(n, 1), cols), 5.0, device="cuda", dtype=DT[self.dtype])[:n]

    def forward(self, h=True, a=True, stream=None):
        out = {"h": self.buf(2 * self.F) if h else None, "a": self.buf(self.F) if a else None,
               "y": self.buf(self.d)}
        M.moe_expert_ffn_fwd_fp8(self.s, self.q, self.qs,
                                 self.mb.pair_of_row if self.gather else None, self.mb.offsets,
                                 self.mb.tile_offsets, self.w, out["h"], out["a"], out["y"],
                                 self.ws, stream)
        return out

    def dgrad(self, ag=True, stream=None):
        out = {"dh": self.buf(2 * self.F), "dx": self.buf(self.d),
               "ag": self.buf(self.F) if ag and self.gather else None}
        self.mb.gates.view(-1).copy_(torch.from_numpy(self.gates))
        gates = self.mb.gates if self.gather else None
        M.moe_ffn_dgrad_fp8(self.s, self.q, self.qs,
                            self.mb.pair_of_row if self.gather else None, gates, self.h,
                            self.mb.offsets, self.mb.tile_offsets, self.w, out["dh"], out["dx"],
                            out["ag"], self.ws, stream)
        return out

    def _each(self, A, W, transpose):
        out = np.zeros((self.N, W.shape[1] if transpose else W.shape[2]))
        for e in range(self.E_l):
            r = slice(self.off[e], self.off[e + 1])
            out[r] = A[r] @ (W[e].T if transpose else W[e])
        return out

    def untouched(self, **bufs):
        for n, t in bufs.items():
            if t is not None:
                assert (t[self.N:] == 5.0).all(), f"{n}: rows behind the last were written"

    def check_forward(self, out):
        x, (W_gu, W_down) = self.rows(), self.weights()
        ref = Q.ffn_fwd_fp8(x, self.off, W_gu, W_down)
        F = self.F
        eh = EPS_SUM * self._each(np.abs(x), np.abs(W_gu), True)
        g, u, eg, eu = ref["g"], ref["u"], eh[:, :F], eh[:, F:]
        # |silu'| <= 1.1, |silu(g)| <= |g|
        ea = 1.1 * eg * (np.abs(u) + eu) + np.abs(Q.silu(g)) * eu + np.abs(ref["a"]) * (
            np.abs(g) + 8) * 2.0 ** -22
        ey = self._each(_requant_slack(ref["a"], ea), np.abs(W_down), True)
        ey += EPS_SUM * 2 * self._each(np.abs(Q.requant(ref["a"])), np.abs(W_down), True)
        N = self.N
        if out["h"] is not None:
            h = np.concatenate([g, u], 1)
            within("h", host(out["h"], N), h, eh + half_step(np.abs(h) + eh, self.dtype))
        if out["a"] is not None:
            within("a", host(out["a"], N), ref["a"], ea + half_step(np.abs(ref["a"]) + ea,
                                                                    self.dtype))
        within("y", host(out["y"], N), ref["y"], ey + half_step(np.abs(ref["y"]) + ey, self.dtype))
        self.untouched(**out)

    def check_dgrad(self, out):
        d, (W_gu, W_down) = self.rows(), self.weights()
        gate = self.gates[self.pair].astype(np.float64) if self.gather else 1.0
        h, N, F = host(self.h, self.N), self.N, self.F
        ref = Q.ffn_dgrad_fp8(d, gate, h, self.off, W_gu, W_down)
        g, u = h[:, :F], h[:, F:]
        ed = EPS_SUM * np.reshape(gate, (-1, 1)) * self._each(np.abs(d), np.abs(W_down), False)
        da = np.abs(ref["da"]) + ed
        sg = 1 / (1 + np.exp(-g))
        rel = (np.abs(g) + 16) * 2.0 ** -21
        eh = np.concatenate([
            ed * np.abs(u) * 1.1 + da * np.abs(u) * sg * (1 + np.abs(g)) * rel,
            ed * np.abs(g) * sg + da * np.abs(g) * sg * rel], 1)
        within("dh", host(out["dh"], N), ref["dh"],
               eh + half_step(np.abs(ref["dh"]) + eh, self.dtype))
        ex = self._each(_requant_slack(ref["dh"], eh), np.abs(W_gu), False)
        ex += EPS_SUM * 2 * self._each(np.abs(Q.requant(ref["dh"])), np.abs(W_gu), False)
        within("dx", host(out["dx"], N), ref["dx"],
               ex + half_step(np.abs(ref["dx"]) + ex, self.dtype))
        if out["ag"] is not None:
            within("ag", host(out["ag"], N), ref["ag"],
                   half_step(ref["ag"], self.dtype) + np.abs(ref["ag"]) * rel)
        self.untouched(**out)


# ---- quantisation: exact ----------------------------------------------------
def _values(rng, rows, d, dtype):
    x = rng.normal(size=(rows, d)) * np.exp(rng.normal(size=(rows, 1)) * 4)
    x[rng.random(x.shape) < 0.1] = 0.0
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    return t


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 128), (3, 384), (17, 640), (130, 2048), (5, 16384)])
def test_quant_rows(rows, d, dtype):
    rng = np.random.default_rng(rows + d)
    t = _values(rng, rows, d, dtype)
    big = {"bf16": 3.0e38, "f16": 65504.0, "f32": 3.4e38}[dtype]
    t[0, :128] = 0.0                                     # an empty block
    t[-1, 5], t[-1, 9], t[-1, 11] = float("nan"), float("inf"), float("-inf")
    t[0, d - 1] = big                                    # the largest magnitude
    if rows > 1:
        t[1, :128] = torch.tensor([1.75 * 2.0 ** -3] + [2.0 ** -20] * 127).to(t.dtype)
        t[1, 128:256] = torch.tensor(1e-44 if dtype == "f32" else 6e-8).to(t.dtype)
    s = M.make_shape(rows, d, 128, 1, 0, 1, 1, dtype)
    ld = M.moe_fp8_scale_ld(d)
    q = torch.zeros(rows, d, device="cuda").to(torch.float8_e4m3fn)
    qs = torch.full((rows, ld), 77, dtype=torch.uint8, device="cuda")
    M.moe_quant_rows_fp8(s, t.cuda(), rows, None, q, qs)
    rq, rb = Q.quant_rows(t.double().numpy())
    got = host(q.float())
    assert np.array_equal(got, rq, equal_nan=True)
    exact("scales", host(qs)[:, : d // 128], rb)
    assert (host(qs)[:, d // 128:] == 0).all()


def test_quant_rows_stops_at_the_device_count():
    rng = np.random.default_rng(4)
    t = _values(rng, 50, 256, "bf16").cuda()
    s = M.make_shape(50, 256, 128, 1, 0, 1, 1, "bf16")
    for n in (0, 1, 33, 50, 70, -3):
        q = torch.full((50, 256), 3.0, device="cuda").to(torch.float8_e4m3fn)
        qs = torch.full((50, 4), 77, dtype=torch.uint8, device="cuda")
        M.moe_quant_rows_fp8(s, t, 50, torch.tensor([n], dtype=torch.int32, device="cuda"), q, qs)
        k = max(0, min(n, 50))
        rq, rb = Q.quant_rows(host(t))
        exact("q", host(q.float())[:k], rq[:k])
        exact("s", host(qs)[:k, :2], rb[:k])
        assert (host(q.float())[k:] == 3.0).all() and (host(qs)[k:] == 77).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E_l,d,F,transposed", [(1, 128, 128, True), (3, 640, 256, True),
                                                (2, 256, 1408, False), (5, 384, 384, True)])
def test_quant_weights(E_l, d, F, transposed, dtype):
    rng = np.random.default_rng(d + F)
    W = [torch.from_numpy((rng.normal(size=sh) * np.exp(rng.normal(size=(E_l, 1, 1)))
                           ).astype(np.float32)).to(DT[dtype])
         for sh in ((E_l, 2 * F, d), (E_l, d, F))]
    W[0][0, 3, 100] = float("nan")
    W[1][-1, :128, :128] = 0
    s = M.make_shape(1, d, F, E_l, 0, E_l, 1, dtype)
    w = M.Fp8Weights(s, transposed=transposed)
    M.moe_quant_weights_fp8(s, W[0].cuda(), W[1].cuda(), w)
    for name, Wm in (("gu", W[0]), ("down", W[1])):
        q, b = Q.quant_weights(Wm.double().numpy())
        n, k = Wm.shape[1:]
        assert np.array_equal(host(getattr(w, name).float()), q, equal_nan=True)
        sc = host(getattr(w, name + "_s"))
        exact(name + "_s", sc[..., : k // 128], b)
        assert (sc[..., k // 128:] == 0).all()
        if transposed:
            assert np.array_equal(host(getattr(w, name + "T").float()), q.transpose(0, 2, 1),
                                  equal_nan=True)
            sc = host(getattr(w, name + "T_s"))
            exact(name + "T_s", sc[..., : n // 128], b.transpose(0, 2, 1))
            assert (sc[..., n // 128:] == 0).all()
        else:
            assert getattr(w, name + "T") is None


# ---- the experts ------------------------------------------------------------
LAYERS = {
    # T, d, F, E, e_lo, E_l, K
    "one_token": (1, 256, 128, 8, 0, 8, 8),
    "one_token_one_expert": (1, 128, 128, 1, 0, 1, 1),
    "two_rows_each": (2, 384, 256, 4, 0, 4, 4),
    "no_tokens": (0, 128, 128, 4, 0, 4, 2),
    "ragged_tiles": (333, 128, 256, 4, 1, 3, 3),
    "over_a_tile": (600, 256, 128, 2, 0, 2, 2),
    "half_tiles": (65, 640, 384, 4, 0, 4, 2),
    "window": (150, 128, 128, 16, 5, 3, 4),
    "many_experts": (40, 256, 128, 256, 0, 256, 8),
    "sixteen_each": (16, 256, 256, 8, 0, 8, 8),
    "seventeen_each": (17, 256, 256, 8, 0, 8, 8),
    "sixty_four_each": (64, 128, 384, 4, 0, 4, 4),
    "wide": (9, 16384, 128, 2, 0, 2, 2),
    "wide_ffn": (9, 128, 16384, 2, 0, 2, 2),
    "wide_rows": (300, 2048, 256, 2, 0, 2, 1),
    # more than 256 rows to an expert, or much work in all: 256 x 256 tiles
    "tiles_one_block": (520, 128, 128, 2, 0, 2, 2),
    "tiles_odd_blocks": (300, 640, 384, 1, 0, 1, 1),
    "tiles_window": (900, 256, 640, 3, 1, 2, 1),
    "tiles_wide": (300, 16384, 128, 1, 0, 1, 1),
    "tiles_wide_ffn": (300, 128, 16384, 1, 0, 1, 1),
    "tiles_few_rows": (250, 2048, 2048, 2, 0, 2, 2),
    "tiles_forward_only": (120, 2048, 2048, 2, 0, 2, 2),
    "tiles_halves": (1100, 128, 1408, 8, 0, 8, 4),
    "tiles_past_the_grid": (8192, 128, 256, 64, 0, 64, 8),
}


@pytest.mark.parametrize("gather", [True, False], ids=["tokens", "dispatched"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", LAYERS)
def test_forward(name, dtype, gather):
    L = Layer(*LAYERS[name], dtype, gather, seed=len(name))
    L.check_forward(L.forward())


@pytest.mark.parametrize("gather", [True, False], ids=["tokens", "dispatched"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", LAYERS)
def test_dgrad(name, dtype, gather):
    L = Layer(*LAYERS[name], dtype, gather, seed=len(name) + 100)
    L.check_dgrad(L.dgrad())


@pytest.mark.parametrize("T", [4, 8224])
def test_weights_past_32_bits(T):
    """256 experts of 4096 x 4096 (8.6 GB of gate and up): the rows of the last expert,
    forward and gradient, for a few rows and for tiles."""
    d = F = 4096
    E, K = 256, 8
    s = M.make_shape(T, d, F, E, 0, E, K, "bf16")
    gen = torch.Generator(device="cuda").manual_seed(T)
    g = lambda *sh, std=1.0: torch.empty(sh, dtype=torch.bfloat16,
                                         device="cuda").normal_(0, std, generator=gen)
    W = [g(E, 2 * F, d, std=d ** -0.5), g(E, d, F, std=F ** -0.5)]
    w = M.Fp8Weights(s)
    M.moe_quant_weights_fp8(s, W[0], W[1], w)
    del W
    ws = torch.empty(max(M.moe_fp8_workspace_bytes(s), M.moe_workspace_bytes(s)),
                     dtype=torch.uint8, device="cuda")
    idx = torch.stack([(torch.arange(T) * 37 + 249 + k * 31) % E for k in range(K)], 1)
    idx[:4, 0] = 255
    idx[:4, 1:] = torch.arange(1, K) * 5
    i32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device="cuda")
    counts, offsets, tiles, rop, por = i32(E), i32(E + 1), i32(E + 1), i32(T * K), i32(T * K)
    M.moe_dispatch(s, None, idx.to(torch.int32).cuda(), counts, offsets, rop, por, tiles, None, ws)
    x, h = g(T, d), g(T * K, 2 * F)
    q = torch.zeros(T, d, device="cuda").to(torch.float8_e4m3fn)
    qs = torch.zeros(T, M.moe_fp8_scale_ld(d), dtype=torch.uint8, device="cuda")
    M.moe_quant_rows_fp8(s, x, T, None, q, qs)
    gates = torch.rand(T * K, device="cuda", generator=gen) + 0.05
    out = {n: g(T * K, c) for n, c in (("h", 2 * F), ("y", d), ("dh", 2 * F), ("dx", d))}
    M.moe_expert_ffn_fwd_fp8(s, q, qs, por, offsets, tiles, w, out["h"], None, out["y"], ws)
    M.moe_ffn_dgrad_fp8(s, q, qs, por, gates, h, offsets, tiles, w, out["dh"], out["dx"], None, ws)
    # the last expert's rows as a layer of one expert
    lo, hi = int(offsets[E - 1]), int(offsets[E])
    lo = max(lo, hi - 40)
    assert hi - lo >= 4
    L = object.__new__(Layer)
    L.dtype, L.gather, L.d, L.F, L.K, L.E_l = "bf16", True, d, F, K, 1
    L.N, L.off, L.pair = hi - lo, np.array([0, hi - lo]), host(por)[lo:hi]
    L.q, L.qs, L.gates, L.h = q, qs, host(gates).astype(np.float32), h[lo:hi]
    L.w = type("W", (), {n: getattr(w, n)[E - 1:] for n in ("gu", "gu_s", "down", "down_s")})
    part = {n: t[lo:hi] for n, t in out.items()}
    L.check_forward({"h": part["h"], "a": None, "y": part["y"]})
    L.check_dgrad({"dh": part["dh"], "dx": part["dx"], "ag": None})


@pytest.mark.parametrize("T,E", [(40, 8), (700, 4)])
def test_no_local_rows(T, E):
    """Every token is routed outside the window: nothing is written."""
    L = Layer(T, 128, 128, E, 2, 2, 2, "bf16", True, only=[0, 1])
    assert L.N == 0
    L.untouched(**L.forward())
    L.untouched(**L.dgrad())


@pytest.mark.parametrize("T", [700, 2100])
def test_one_expert_has_every_row(T):
    L = Layer(T, 128, 128, 8, 0, 8, 1, "bf16", True, only=[5])
    assert L.off[5] == 0 and L.off[6] == T
    L.check_forward(L.forward())
    L.check_dgrad(L.dgrad())


@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_window"])
def test_optional_outputs(name):
    """h and a left out (serving) change nothing in y; ag left out neither."""
    L = Layer(*LAYERS[name], "bf16", True)
    full = L.forward()
    for h, a in ((False, False), (True, False), (False, True)):
        part = L.forward(h, a)
        for n in ("h", "a", "y"):
            assert part[n] is None or torch.equal(part[n], full[n]), n
    d, e = L.dgrad(), L.dgrad(ag=False)
    assert torch.equal(d["dh"], e["dh"]) and torch.equal(d["dx"], e["dx"])


@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_window"])
def test_gathered_equals_dispatched(name):
    """Token rows read through the plan give what the permuted copy gives."""
    L = Layer(*LAYERS[name], "bf16", True)
    f, d = L.forward(), L.dgrad()
    rows = torch.zeros(L.T * L.K, dtype=torch.int64)
    rows[: L.N] = torch.from_numpy(L.pair // L.K)
    P = Layer(*LAYERS[name], "bf16", False)
    P.q = L.q.view(torch.uint8)[rows.cuda()].view(torch.float8_e4m3fn).contiguous()
    P.qs, P.w = L.qs[rows.cuda()].contiguous(), L.w
    assert all(torch.equal(x, y) for x, y in zip(f.values(), P.forward().values()))
    # a gate of one is no gate
    L.gates[:] = 1.0
    P.h = L.h
    d, e = L.dgrad(), P.dgrad()
    assert torch.equal(d["dh"], e["dh"]) and torch.equal(d["dx"], e["dx"])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_odd_blocks"])
def test_nonfinite_token_stays_in_its_rows(name, dtype):
    """A NaN or infinite activation poisons its own token's outputs only."""
    L = Layer(*LAYERS[name], dtype, True)
    clean = L.forward()
    L.x[7, 3], L.x[9, 100] = float("nan"), float("inf")
    L.q, L.qs = L.quantise(L.x, L.T)
    out = L.forward()
    bad = np.isin(L.pair // L.K, (7, 9))
    y, c = out["y"][: L.N].float().cpu(), clean["y"][: L.N].float().cpu()
    assert torch.isnan(y[torch.from_numpy(bad)]).all()
    assert torch.equal(y[torch.from_numpy(~bad)], c[torch.from_numpy(~bad)])


def test_refuses_another_shapes_weights():
    L = Layer(*LAYERS["one_token"], "bf16", True)
    w = M.Fp8Weights(M.make_shape(1, 256, 256, 8, 0, 8, 8, "bf16"))
    with pytest.raises(M.MoeError):
        M.moe_expert_ffn_fwd_fp8(L.s, L.q, L.qs, None, L.mb.offsets, L.mb.tile_offsets, w, None,
                                 None, L.buf(L.d), L.ws)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(M.MoeError) as e:
        M.moe_expert_ffn_fwd_fp8(L.s, L.q, L.qs, L.mb.pair_of_row, L.mb.offsets,
                                 L.mb.tile_offsets, L.w, None, None, L.buf(L.d), small)
    assert e.value.code == M.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["ragged_tiles", "tiles_odd_blocks"])
def test_infinite_products_stay_in_their_rows(name, dtype):
    """Activations whose products pass the type's range: the row's block scales come
    from its finite values, its infinities become NaN, and other rows keep theirs."""
    L = Layer(*LAYERS[name], dtype, True)
    clean = L.forward()
    L.qs[7, 0] = 254                       # the first block of token 7, times 2^127
    out = L.forward()
    bad = torch.from_numpy(np.isin(L.pair // L.K, (7,)))
    y, c = out["y"][: L.N].float().cpu(), clean["y"][: L.N].float().cpu()
    assert not torch.isfinite(y[bad]).any()
    assert torch.equal(y[~bad], c[~bad])


@pytest.mark.parametrize("name", ["one_token", "ragged_tiles", "tiles_window"])
def test_two_streams_and_graph_replays(name):
    """Calls on two streams with a workspace each, and a captured pair of calls
    replayed between eager work, give the eager results bit for bit."""
    A, B = Layer(*LAYERS[name], "bf16", True, seed=1), Layer(*LAYERS[name], "f16", True, seed=2)
    want = [(L.forward(), L.dgrad()) for L in (A, B)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    gates = [torch.from_numpy(L.gates).cuda() for L in (A, B)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for L, st in zip((A, B), streams):
            with torch.cuda.stream(st):
                got.append((L.forward(stream=st), L.dgrad(stream=st)))
    torch.cuda.synchronize()
    same = lambda x, y: all(torch.equal(p, q) for u, v in zip(x, y)
                            for p, q in zip(u.values(), v.values()) if p is not None)
    assert all(same(g, w) for g, w in zip(got, want))
    # capture
    out = {"h": A.buf(2 * A.F), "y": A.buf(A.d), "dh": A.buf(2 * A.F), "dx": A.buf(A.d)}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = torch.cuda.current_stream()
        M.moe_quant_rows_fp8(A.s, A.x, A.T, None, A.q, A.qs, st)
        M.moe_expert_ffn_fwd_fp8(A.s, A.q, A.qs, A.mb.pair_of_row, A.mb.offsets,
                                 A.mb.tile_offsets, A.w, out["h"], None, out["y"], A.ws, st)
        M.moe_ffn_dgrad_fp8(A.s, A.q, A.qs, A.mb.pair_of_row, gates[0], A.h, A.mb.offsets,
                            A.mb.tile_offsets, A.w, out["dh"], out["dx"], None, A.ws, st)
    for k in range(4):
        for t in out.values():
            t.fill_(5.0)
        if k == 2:
            A.x.mul_(0.5)          # half the activations: the same values, a scale lower
        g.replay()
        eager = (A.forward(), A.dgrad()) if k >= 2 else want[0]
        torch.cuda.synchronize()
        for n in ("h", "y"):
            assert torch.equal(out[n], eager[0][n]), (k, n)
        for n in ("dh", "dx"):
            assert torch.equal(out[n], eager[1][n]), (k, n)


def test_a_training_step_in_8_bits():
    """Route, dispatch, quantise, experts, combine and all of the backward as a
    layer would run them, then AdamW and the weights quantised again: every stage
    against the oracle on the inputs the GPU gave it, over two steps, the second
    with the updated weights."""
    T, d, F, E, K = 120, 256, 128, 8, 2
    s = M.make_shape(T, d, F, E, 0, E, K, "bf16")
    rng = np.random.default_rng(8)
    f32 = lambda *sh, std=1.0: torch.from_numpy((rng.normal(size=sh) * std).astype(np.float32)).cuda()
    masters = {"W_gu": f32(E, 2 * F, d, std=0.06), "W_down": f32(E, d, F, std=0.09),
               "W_r": f32(d, E, std=0.06)}
    W = {n: t.bfloat16() for n, t in masters.items()}
    grads = {n: torch.empty_like(t) for n, t in masters.items()}
    state = {n: [torch.zeros_like(t), torch.zeros_like(t)] for n, t in masters.items()}
    tensors = M.AdamWTensors([dict(param=W[n], master=masters[n], grad=grads[n], m=state[n][0],
                                   v=state[n][1], weight_decay=0.01) for n in W])
    w8 = M.Fp8Weights(s)
    ws = torch.empty(M.moe_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    w8s = torch.empty(M.moe_fp8_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    ld = M.moe_fp8_scale_ld(d)
    q8 = lambda: (torch.empty(T, d, device="cuda", dtype=torch.float8_e4m3fn),
                  torch.empty(T, ld, device="cuda", dtype=torch.uint8))
    (xq, xs), (dq, ds) = q8(), q8()
    for step in (1, 2):
        mb = M.MicroBatch(s, x=f32(T, d).bfloat16(), dout=f32(T, d).bfloat16(), fused_bwd=True)
        used = {n: host(t) for n, t in W.items()}
        M.moe_quant_weights_fp8(s, W["W_gu"], W["W_down"], w8)
        M.moe_route(s, M.MOE_ROUTE_TOPK, mb.x, W["W_r"], None, mb.logits, mb.idx, mb.gates, ws)
        M.moe_dispatch(s, None, mb.idx, mb.counts, mb.offsets, mb.row_of_pair, mb.pair_of_row,
                       mb.tile_offsets, None, ws)
        M.moe_quant_rows_fp8(s, mb.x, T, None, xq, xs)
        M.moe_expert_ffn_fwd_fp8(s, xq, xs, mb.pair_of_row, mb.offsets, mb.tile_offsets, w8, mb.h,
                                 None, mb.yp, w8s)
        M.moe_combine(s, mb.yp, mb.gates, mb.row_of_pair, mb.out)
        M.moe_combine_bwd(s, mb.dout, mb.yp, mb.gates, mb.row_of_pair, None, mb.dgates)
        M.moe_quant_rows_fp8(s, mb.dout, T, None, dq, ds)
        M.moe_ffn_dgrad_fp8(s, dq, ds, mb.pair_of_row, mb.gates, mb.h, mb.offsets,
                            mb.tile_offsets, w8, mb.dh, mb.dxp, mb.ag, w8s)
        M.moe_route_bwd(s, M.MOE_ROUTE_TOPK, mb.dgates, mb.gates, mb.idx, mb.x, mb.dlogits,
                        grads["W_r"], 0, ws)
        M.moe_dispatch_bwd(s, mb.dxp, mb.row_of_pair, mb.idx, mb.dlogits, W["W_r"], mb.dx, 0, ws)
        M.moe_ffn_wgrad_fused(s, None, mb.x, mb.pair_of_row, mb.ag, mb.dh, mb.dout, mb.offsets,
                              grads["W_gu"], grads["W_down"])
        before = {n: host(t) for n, t in masters.items()}
        mom = {n: [host(t) for t in state[n]] for n in state}
        M.moe_adamw(tensors, lr=1e-2, step=step, beta2=0.95)
        torch.cuda.synchronize()

        # the 8-bit stages, on the operands the GPU used
        L = Layer.__new__(Layer)
        L.__dict__.update(s=s, dtype="bf16", gather=True, T=T, d=d, F=F, K=K, E_l=E, mb=mb, w=w8,
                          off=host(mb.offsets), q=xq, qs=xs, h=mb.h,
                          gates=host(mb.gates).reshape(-1))
        L.N = int(L.off[-1])
        L.pair = host(mb.pair_of_row)[: L.N]
        assert L.N == T * K
        exact("W_gu", host(w8.gu.float()), Q.quant_weights(used["W_gu"])[0])
        xq_ref, xb_ref = Q.quant_rows(host(mb.x))
        exact("x", host(xq.float()), xq_ref)
        L.check_forward({"h": mb.h, "a": None, "y": mb.yp})
        L.q, L.qs = dq, ds
        L.check_dgrad({"dh": mb.dh, "dx": mb.dxp, "ag": mb.ag})
        # the weight gradients from the stored operands (float32 sums of at most
        # 240 products of bf16 values: 240 * 2^-24 of sum |terms|)
        tok = L.pair // K
        ag, dh, x, do = host(mb.ag), host(mb.dh), host(mb.x)[tok], host(mb.dout)[tok]
        for name, A_, B_ in (("W_gu", dh, x), ("W_down", do, ag)):
            for e in range(E):
                r = slice(L.off[e], L.off[e + 1])
                within("d" + name, host(grads[name])[e], A_[r].T @ B_[r],
                       np.abs(A_[r]).T @ np.abs(B_[r]) * 240 * 2.0 ** -24 + 1e-30)
        for n in masters:
            p, m, v = Q.adamw(before[n], host(grads[n]), *mom[n], 1e-2, 0.9, 0.95, 1e-8,
                              float(np.float32(0.01)), step)
            # eight float32 roundings on the way, each 2^-24 of a term
            within(n, host(masters[n]), p, (np.abs(p) + np.abs(before[n]) + 0.02) * 2.0 ** -21)
            assert torch.equal(W[n], masters[n].bfloat16())
