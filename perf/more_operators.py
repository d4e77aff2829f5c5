"""The layer's norm and the experts on 4-bit weights, as measured.

Five operators: the root-mean-square norm in front of the layer (the residual
added, the result in 16 bits and in the 8-bit row format) and its backward pass;
the quantisation of the expert weights to 4 bits (e2m1 values, one power-of-two
scale per 32 along the reduction) and their reading back; and the SwiGLU expert
FFN of 8-bit rows on 4-bit weights.

``run`` computes an operator in its plain form (elementary torch operations in
float32) or, with ``own`` set, through the package's entry points.
"""

import math

import torch

own = False

BLOCK = 128      # values per scale of an 8-bit row
BLOCK4 = 32      # values per scale of a 4-bit weight row
TILE_M = 256     # rows per tile of the dispatch plan (moe_tile_m)
EPS = 1e-6       # of the norm
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # decoding: one token enters the layer, for the router (16 bits) and the experts (8)
        {"name": "norm, one token", "op": "norm", "T": 1, "d": 2048, "dtype": "bf16",
         "res": True, "y": True, "q": True, "train": False},
        # a short prompt in full precision, no residual, an odd width
        {"name": "norm, 777 tokens, float32", "op": "norm", "T": 777, "d": 1088, "dtype": "f32",
         "res": False, "y": True, "q": False, "train": True},
        # a training micro-batch of the 128-expert layer, rstd kept for the backward
        {"name": "norm, 65536 tokens", "op": "norm", "T": 65536, "d": 2048, "dtype": "bf16",
         "res": True, "y": True, "q": True, "train": True},
        # the backward of a small micro-batch, no gradient beside the norm's
        {"name": "norm backward, 333 tokens", "op": "norm_bwd", "T": 333, "d": 640,
         "dtype": "f16", "res": False},
        # the backward of the large micro-batch, with the residual stream's gradient
        {"name": "norm backward, 65536 tokens", "op": "norm_bwd", "T": 65536, "d": 2048,
         "dtype": "bf16", "res": True},
        # one EP8 rank's eight experts, made ready for serving
        {"name": "quant 4-bit weights, 8 experts", "op": "quant", "E_l": 8, "d": 2048, "F": 1408,
         "dtype": "f16"},
        # the whole 128-expert layer
        {"name": "quant 4-bit weights, 128 experts", "op": "quant", "E_l": 128, "d": 2048,
         "F": 768, "dtype": "bf16"},
        # a small model's weights read back, to compare with the ones in full precision
        {"name": "read back, 4 experts", "op": "dequant", "E_l": 4, "d": 640, "F": 384,
         "dtype": "f32"},
        # the 128-expert layer's weights read back, for a backward pass in 16 bits
        {"name": "read back, 128 experts", "op": "dequant", "E_l": 128, "d": 2048, "F": 768,
         "dtype": "bf16"},
        # decoding: one token through its eight experts
        {"name": "ffn, one token", "op": "ffn", "T": 1, "d": 2048, "F": 768, "E": 128, "E_l": 128,
         "K": 8, "dtype": "bf16", "zipf": 0.0, "gather": True, "train": False},
        # a ragged prompt on an EP8 rank: skewed experts, most pairs elsewhere
        {"name": "ffn, ragged window", "op": "ffn", "T": 1333, "d": 2048, "F": 1408, "E": 64,
         "E_l": 8, "K": 6, "dtype": "f16", "zipf": 1.1, "gather": False, "train": False},
        # a large micro-batch of the 128-expert layer, h and a kept for the backward
        {"name": "ffn, 128 experts", "op": "ffn", "T": 16384, "d": 2048, "F": 768, "E": 128,
         "E_l": 128, "K": 8, "dtype": "bf16", "zipf": 0.0, "gather": True, "train": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "quant", "dequant", "ffn", "ffn",
                     "ffn"])
    if op in ("norm", "norm_bwd"):
        q = op == "norm" and rng.random() < 0.5
        d = 128 * log(1, 128) if q else 64 * log(1, 256)
        dtype = rng.choice(["bf16", "f16", "f32"])
        most = 65536 * 2048 // d // (2 if dtype == "f32" else 1)
        case = {"op": op, "T": min(log(1, 65536), most), "d": d, "dtype": dtype,
                "res": rng.random() < 0.5}
        if op == "norm":
            case |= {"y": not q or rng.random() < 0.5, "q": q, "train": rng.random() < 0.5}
        return case
    dtype = rng.choice(["bf16", "f16"])
    if op in ("quant", "dequant"):
        d, F = 128 * log(1, 32), 128 * log(1, 12)
        dtype = rng.choice(["bf16", "f16", "f32"])
        most = 128 * 2048 * 768 // (d * F) // (2 if dtype == "f32" else 1)
        return {"op": op, "E_l": max(1, min(log(1, 128), most)), "d": d, "F": F, "dtype": dtype}
    d, F = 128 * log(1, 24), 128 * log(1, 12)
    E = rng.choice([4, 8, 16, 64, 128])
    E_l = max(1, E // rng.choice([1, 1, 2, 8]))
    K = rng.randint(1, min(E, 8))
    # no more rows or products than the largest listed case
    T = min(log(1, 16384), max(1, 131072 * 2048 * 768 // (K * d * F)), 131072 // K)
    T = max(T, 8 * E // (E_l * K))  # some rows in the window
    return {"op": op, "T": T, "d": d, "F": F, "E": E, "E_l": E_l, "K": K, "dtype": dtype,
            "zipf": rng.choice([0.0, 1.1]), "gather": rng.random() < 0.5,
            "train": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# the formats: blocks of values with one power of two (a biased exponent) each
# ---------------------------------------------------------------------------
def _scale_ld(k):
    """Scale bytes per 8-bit row of k values: a multiple of four."""
    return (k // BLOCK + 3) // 4 * 4


def _pow2(e):
    return torch.exp2(e.to(torch.float64)).to(torch.float32)


def _scale_byte(amax, top):
    """Biased exponent of the smallest power of two s with amax / s <= 1.75 *
    2^top; 127 for a block of zeros.  amax: float32."""
    byte = (((amax.view(torch.int32) + 0x1FFFFF) >> 23) - top).clamp(0, 254)
    return torch.where(amax == 0, 127, byte)


def _quant8(x):
    """float32 [..., k] -> (e4m3 [..., k], scale bytes [..., k / 128]); e4m3's
    largest value is 448 = 1.75 * 2^8."""
    b = x.view(*x.shape[:-1], -1, BLOCK)
    byte = _scale_byte(torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1), 8)
    q = (b * _pow2(127 - byte)[..., None]).to(torch.float8_e4m3fn)
    return q.view(x.shape), byte.to(torch.uint8)


def _pad_scales(s, k):
    out = s.new_zeros(*s.shape[:-1], _scale_ld(k))
    out[..., :s.shape[-1]] = s
    return out


def _dequant8(q, s):
    """e4m3 [..., k] with scale bytes [..., >= k / 128] -> float32."""
    kb = q.shape[-1] // BLOCK
    b = q.float().view(*q.shape[:-1], kb, BLOCK)
    return (b * _pow2(s[..., :kb].int() - 127)[..., None]).view(q.shape)


def _quant4(x):
    """float32 [..., k] -> (codes, two a byte, the first in the low half
    [..., k / 2], scale bytes [..., k / 32]).  e2m1's magnitudes are 0, 0.5, 1,
    1.5, 2, 3, 4, 6; up to 7 = 1.75 * 2^2 is rounded to 6.  A block that holds
    a value that is not finite has scale byte 255 and codes 0: it is NaN."""
    b = x.view(*x.shape[:-1], -1, BLOCK4)
    fine = torch.isfinite(b).all(-1)
    byte = torch.where(fine, _scale_byte(b.abs().amax(-1), 2), 255)
    y = b * _pow2(127 - byte)[..., None]
    m = y.abs()
    code = torch.signbit(y).to(torch.uint8) * 8
    # borders halfway between neighbours; on one, the even code
    code += m > 0.25
    code += m >= 0.75
    code += m > 1.25
    code += m >= 1.75
    code += m > 2.5
    code += m >= 3.5
    code += m > 5
    code = (code * fine[..., None]).view(*x.shape[:-1], -1, 2)
    return code[..., 0] | code[..., 1] << 4, byte.to(torch.uint8)


def _dequant4(c, s):
    """Codes [..., k / 2] with scale bytes [..., k / 32] -> float32 [..., k]."""
    c = torch.stack((c & 15, c >> 4), -1).view(*s.shape, BLOCK4)
    m = (c & 7).float()
    m = torch.maximum(torch.maximum(m * 0.5, m - 2), m * 2 - 8)
    scale = torch.where(s == 255, math.nan, _pow2(s.int() - 127))[..., None]
    return torch.where(c > 7, -m, m).mul_(scale).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _stream(case, g):
    """Rows of a residual stream: each of its own size, some columns larger."""
    T, d = case["T"], case["d"]
    wide = torch.exp(0.7 * _randn(g, d))
    return (_randn(g, T, d) * wide * torch.exp(0.5 * _randn(g, T, 1))).to(DTYPES[case["dtype"]])


def _plan(case, g):
    """The dispatch plan of top-K routing, as moe_dispatch lays it out;
    "experts" and "R": the local experts with rows and the most rows that one
    has."""
    T, E, E_l, K = case["T"], case["E"], case["E_l"], case["K"]
    logits = _randn(g, T, E)
    if case["zipf"]:
        logits -= case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda"))
    flat = torch.topk(logits, K, dim=1)[1].reshape(-1)
    key = torch.where(flat < E_l, flat, E_l)  # the local window is [0, E_l)
    counts = torch.bincount(key, minlength=E_l + 1)[:E_l]
    N = int(counts.sum())
    pair_of_row = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    pair_of_row[:N] = torch.sort(key, stable=True)[1][:N].int()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return {"N": N, "R": int(counts.max()), "experts": torch.nonzero(counts).view(-1),
            "pair_of_row": pair_of_row, "offsets": torch.cat([zero, counts.cumsum(0)]).int(),
            "tile_offsets": torch.cat([zero, (-(-counts // TILE_M)).cumsum(0)]).int()}


def _weights4(case, g):
    E_l, d, F = case["E_l"], case["d"], case["F"]
    w = {}
    for name, n, k in (("gu", 2 * F, d), ("down", d, F)):
        w[name], w[name + "_s"] = _quant4(_randn(g, E_l, n, k, std=0.02))
    return w


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    dt = DTYPES[case["dtype"]]
    if op in ("norm", "norm_bwd"):
        T, d = case["T"], case["d"]
        st["gamma"] = (1 + 0.2 * _randn(g, d)).to(dt)
    if op == "norm":
        st["x"] = _stream(case, g)
        if case["res"]:
            st["res"], st["r"] = _stream(case, g), torch.zeros(T, d, dtype=dt, device="cuda")
        if case["y"]:
            st["y"] = torch.zeros(T, d, dtype=dt, device="cuda")
        if case["q"]:
            st["q"] = torch.zeros(T, d, dtype=torch.float8_e4m3fn, device="cuda")
            st["qs"] = torch.zeros(T, _scale_ld(d), dtype=torch.uint8, device="cuda")
        if case["train"]:
            st["rstd"] = torch.zeros(T, device="cuda")
    elif op == "norm_bwd":
        st["r"] = _stream(case, g)
        st["rstd"] = torch.rsqrt(st["r"].float().square().mean(1) + EPS)
        st["dy"] = (_randn(g, T, d) * torch.exp(0.5 * _randn(g, T, 1))).to(dt)
        if case["res"]:
            st["dres"] = _randn(g, T, d).to(dt)
        st["dx"] = torch.zeros(T, d, dtype=dt, device="cuda")
        st["dgamma"] = torch.zeros(d, device="cuda")
        # at least moe_rmsnorm_workspace_bytes: a row of float32 sums for every few tokens
        st["ws"] = torch.empty(4 * d * min(T, 2048) + 4096, dtype=torch.uint8, device="cuda")
    elif op in ("quant", "dequant"):
        E_l, d, F = case["E_l"], case["d"], case["F"]
        big = {"W_gu": (E_l, 2 * F, d), "W_down": (E_l, d, F)}
        if op == "quant":
            for name, shape in big.items():
                st[name] = _randn(g, *shape, std=0.02).to(dt)
            st["w"] = {}
            for name, (E, n, k) in (("gu", big["W_gu"]), ("down", big["W_down"])):
                st["w"][name] = torch.zeros(E, n, k // 2, dtype=torch.uint8, device="cuda")
                st["w"][name + "_s"] = torch.zeros(E, n, k // BLOCK4, dtype=torch.uint8,
                                                   device="cuda")
        else:
            st["w"] = _weights4(case, g)
            for name, shape in big.items():
                st[name] = torch.zeros(shape, dtype=dt, device="cuda")
    else:
        rows = case["T"] if case["gather"] else case["T"] * case["K"]
        q, s = _quant8(_randn(g, rows, case["d"]))
        st |= {"q": q, "s": _pad_scales(s, case["d"]), "w": _weights4(case, g)}
        st |= _plan(case, g)
        cap, F = case["T"] * case["K"], case["F"]
        for name, cols in (("h", 2 * F), ("a", F), ("yp", case["d"])):
            if case["train"] or name == "yp":
                st[name] = torch.zeros(cap, cols, dtype=dt, device="cuda")
        # at least moe_fp4_workspace_bytes: a [T*K, F] float32 matrix
        st["ws"] = torch.empty(cap * 4 * F + 4096, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _e8m0(s):
    """Scale bytes as the powers of two that they stand for."""
    return s.view(torch.float8_e8m0fnu)


def _plain_norm(st, case):
    dt, out = DTYPES[case["dtype"]], {}
    r = st["x"]
    if case["res"]:
        r = out["r"] = (r.float() + st["res"].float()).to(dt)
    r = r.float()
    rstd = 1 / torch.sqrt((r * r).mean(1) + EPS)
    y = (r * rstd[:, None] * st["gamma"].float()).to(dt)
    if case["y"]:
        out["y"] = y
    if case["q"]:
        q, s = _quant8(y.float())
        out["q"], out["qs"] = q, _e8m0(_pad_scales(s, case["d"]))
    if case["train"]:
        out["rstd"] = rstd
    return out


def _plain_norm_bwd(st, case):
    xhat = st["r"].float() * st["rstd"][:, None]
    dy = st["dy"].float()
    dn = dy * st["gamma"].float()
    dx = st["rstd"][:, None] * (dn - xhat * (dn * xhat).mean(1, keepdim=True))
    if case["res"]:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["dx"].dtype), "dgamma": (dy * xhat).sum(0)}


def _plain_ffn(st, case):
    F = case["F"]
    out = {n: torch.zeros_like(st[n]) for n in ("h", "a", "yp") if n in st}
    if not st["N"]:
        return out
    # [experts, R] row numbers of the experts that have rows, and which of them exist
    e = st["experts"]
    first, end = st["offsets"][e].long(), st["offsets"][e + 1].long()
    rows = first[:, None] + torch.arange(st["R"], device="cuda")
    rows, ok = torch.minimum(rows, end[:, None] - 1), rows < end[:, None]
    src = st["pair_of_row"][rows].long() // case["K"] if case["gather"] else rows
    W_gu = _dequant4(st["w"]["gu"][e], st["w"]["gu_s"][e])
    h = torch.bmm(_dequant8(st["q"], st["s"])[src], W_gu.transpose(1, 2))
    del W_gu
    g, u = h[..., :F], h[..., F:]
    a = g / (1 + torch.exp(-g)) * u
    W_down = _dequant4(st["w"]["down"][e], st["w"]["down_s"][e])
    y = torch.bmm(_dequant8(*_quant8(a)), W_down.transpose(1, 2))
    at = rows[ok]
    out["yp"][at] = y[ok].to(out["yp"].dtype)
    if case["train"]:
        out["h"][at] = h[ok].to(out["h"].dtype)
        out["a"][at] = a[ok].to(out["a"].dtype)
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state, case, op)
    if op == "norm":
        return _plain_norm(state, case)
    if op == "norm_bwd":
        return _plain_norm_bwd(state, case)
    if op == "quant":
        gu, down = _quant4(state["W_gu"].float()), _quant4(state["W_down"].float())
        return {"gu": gu[0], "gu_s": _e8m0(gu[1]), "down": down[0], "down_s": _e8m0(down[1])}
    if op == "dequant":
        w, dt = state["w"], DTYPES[case["dtype"]]
        return {"W_gu": _dequant4(w["gu"], w["gu_s"]).to(dt),
                "W_down": _dequant4(w["down"], w["down_s"]).to(dt)}
    return _plain_ffn(state, case)


def _run_own(st, case, op):
    import combine_expert_ffn_amd as M

    if "shape" not in st:
        st["shape"] = M.make_shape(case.get("T", 1), case["d"], case.get("F", 128),
                                   case.get("E", case.get("E_l", 1)), 0, case.get("E_l", 1),
                                   case.get("K", 1), case["dtype"])
        if "w" in st:
            st["fp4"] = M.Fp4Weights(st["shape"], **st["w"])
    s = st["shape"]
    if op == "norm":
        M.moe_rmsnorm(s, st["x"], st.get("res"), st["gamma"], EPS, st.get("r"), st.get("y"),
                      st.get("q"), st.get("qs"), st.get("rstd"))
        out = {n: st[n] for n in ("r", "y", "q", "rstd") if n in st}
        if "qs" in st:
            out["qs"] = _e8m0(st["qs"])
        return out
    if op == "norm_bwd":
        M.moe_rmsnorm_bwd(s, st["dy"], st["r"], st["gamma"], st["rstd"], st.get("dres"), st["dx"],
                          st["dgamma"], 0, st["ws"])
        return {"dx": st["dx"], "dgamma": st["dgamma"]}
    if op == "quant":
        M.moe_quant_weights_fp4(s, st["W_gu"], st["W_down"], st["fp4"])
        return {n: _e8m0(t) if n.endswith("_s") else t for n, t in st["w"].items()}
    if op == "dequant":
        M.moe_dequant_weights_fp4(s, st["fp4"], st["W_gu"], st["W_down"])
        return {"W_gu": st["W_gu"], "W_down": st["W_down"]}
    M.moe_expert_ffn_fwd_fp4(s, st["q"], st["s"], st["pair_of_row"] if case["gather"] else None,
                             st["offsets"], st["tile_offsets"], st["fp4"], st.get("h"),
                             st.get("a"), st["yp"], st["ws"])
    return {n: st[n] for n in ("h", "a", "yp") if n in st}


# ---------------------------------------------------------------------------
# the work of one pass
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    b = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if op == "norm":
        T, d = case["T"], case["d"]
        size = T * d * b * (1 + 2 * case["res"] + case["y"]) + d * b
        size += T * (d + d // BLOCK) if case["q"] else 0
        return {"bytes": size + (4 * T if case["train"] else 0), "flops": 7 * T * d}
    if op == "norm_bwd":
        T, d = case["T"], case["d"]
        return {"bytes": T * d * b * (3 + case["res"]) + 4 * T + d * (b + 4), "flops": 11 * T * d}
    if op in ("quant", "dequant"):
        n = case["E_l"] * 3 * case["F"] * case["d"]
        return {"bytes": n * b + n // 2 + n // BLOCK4, "flops": 2 * n}
    # rows of the local window, as expected of the routing
    T, d, F, E, E_l, K = (case[k] for k in ("T", "d", "F", "E", "E_l", "K"))
    p = [(e + 1.0) ** -case["zipf"] for e in range(E)]
    share = [1 - (1 - x / sum(p)) ** K for x in p[:E_l]]
    scale = K / sum(1 - (1 - x / sum(p)) ** K for x in p)
    N = T * min(K, sum(share) * scale)
    experts = sum(1 - (1 - x) ** T for x in share)
    src = min(T, N) if case["gather"] else N
    size = src * d + experts * 3 * d * F * (0.5 + 1 / BLOCK4) + N * d * b
    return {"bytes": size + (N * 3 * F * b if case["train"] else 0), "flops": 6 * N * d * F}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _grid_round(y, least, bits):
    """The nearest (ties to even) value with `bits` bits behind the leading one,
    spaced as at 2^least below it."""
    _, ex = torch.frexp(y)
    step = torch.exp2((ex - 1).clamp(min=least).double() - bits)
    return torch.round(y / step) * step


def _block_scale(amax, most):
    """Smallest power of two s with amax / s <= most, 1 where amax is 0."""
    f, ex = torch.frexp(amax / most)
    e = torch.where(f == 0.5, ex - 1, ex).clamp(-127, 127).double()
    return torch.where(amax == 0, 1.0, torch.exp2(e))


def _exact_rows8(x):
    """(e4m3 values, scales) of rows in blocks of 128."""
    b = x.unflatten(-1, (-1, BLOCK))
    s = _block_scale(b.abs().amax(-1, keepdim=True), 448.0)
    return _grid_round(b / s, -6, 3).flatten(-2), s.squeeze(-1)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_value4(c, s):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device="cuda")
    v = torch.empty(*c.shape, 2, dtype=torch.float64, device="cuda")
    v[..., 0], v[..., 1] = table[(c % 16).long()], table[(c // 16).long()]
    return v.flatten(-2) * torch.exp2(s.double() - 127).repeat_interleave(BLOCK4, -1)


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    dt = DTYPES[case["dtype"]]
    if op == "norm":
        out = {}
        r = st["x"].double()
        if case["res"]:
            r = r + st["res"].double()
            out["r"] = r
            r = r.to(dt).double()  # the norm is of the stored sum
        rstd = (r.square().sum(1) / case["d"] + EPS) ** -0.5
        y = st["gamma"].double() * r * rstd[:, None]
        if case["y"]:
            out["y"] = y
        if case["q"]:
            q, s = _exact_rows8(y.to(dt).double())  # of the 16-bit result
            qs = torch.full((case["T"], _scale_ld(case["d"])), 2.0 ** -127, dtype=torch.float64,
                            device="cuda")
            qs[:, :s.shape[1]] = s
            out["q"], out["qs"] = q, qs
        if case["train"]:
            out["rstd"] = rstd
        return out
    if op == "norm_bwd":
        r, dy, rstd = st["r"].double(), st["dy"].double(), st["rstd"].double()[:, None]
        dn = dy * st["gamma"].double()
        dx = rstd * dn - r * rstd ** 3 * (dn * r).sum(1, keepdim=True) / case["d"]
        if case["res"]:
            dx += st["dres"].double()
        return {"dx": dx, "dgamma": (dy * r * rstd).sum(0)}
    if op == "quant":
        out = {}
        for name in ("gu", "down"):
            b = st["W_" + name].double().unflatten(-1, (-1, BLOCK4))
            out[name] = None  # codes are whole numbers
            out[name + "_s"] = _block_scale(b.abs().amax(-1), 7.0)
        return out
    if op == "dequant":
        w = st["w"]
        return {"W_gu": _exact_value4(w["gu"], w["gu_s"]),
                "W_down": _exact_value4(w["down"], w["down_s"])}
    F = case["F"]
    names = [n for n in ("h", "a", "yp") if n in st]
    out = {n: torch.zeros(st[n].shape, dtype=torch.float64, device="cuda") for n in names}
    off = st["offsets"].tolist()
    for e in range(case["E_l"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        src = slice(lo, hi)
        if case["gather"]:
            src = torch.div(st["pair_of_row"][lo:hi].long(), case["K"], rounding_mode="floor")
        scale = torch.exp2(st["s"][src][:, :case["d"] // BLOCK].double() - 127)
        x = st["q"][src].double() * scale.repeat_interleave(BLOCK, 1)
        h = x @ _exact_value4(st["w"]["gu"][e], st["w"]["gu_s"][e]).T
        a = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
        q, s = _exact_rows8(a)
        y = (q * s.repeat_interleave(BLOCK, 1)) @ _exact_value4(st["w"]["down"][e],
                                                                st["w"]["down_s"][e]).T
        for n, v in (("h", h), ("a", a), ("yp", y)):
            if n in names:
                out[n][lo:hi] = v
    return out
