"""The 8-bit expert path and the optimizer step of the MoE layer, as measured.

Five operators: the block quantisation of activation rows and of the expert
weights (e4m3 values, one power-of-two scale per 128), the SwiGLU expert FFN on
the quantised operands (forward, and the activation gradient), and an AdamW
step over many tensors with its states in 32 or in 8 bits.

``run`` computes an operator in its plain form (elementary torch operations in
float32) or, with ``own`` set, through the package's entry points.
"""

import math

import torch

own = False

BLOCK = 128      # values per scale
TILE_M = 256     # rows per tile of the dispatch plan (moe_tile_m)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the tokens of one decoding batch, quantised before the expert products
        {"name": "quant rows, 33 tokens", "op": "quant_rows", "T": 33, "d": 2048, "dtype": "bf16"},
        # a training micro-batch of the 128-expert layer
        {"name": "quant rows, 65536 tokens", "op": "quant_rows", "T": 65536, "d": 2048,
         "dtype": "bf16"},
        # one EP8 rank's eight experts, held for serving (no transposed copies)
        {"name": "quant weights, 8 experts", "op": "quant_weights", "E_l": 8, "d": 2048, "F": 1408,
         "dtype": "f16", "transposed": False},
        # the whole 128-expert layer after an optimizer step, with the transposed
        # copies that the activation gradient reads
        {"name": "quant weights, 128 experts", "op": "quant_weights", "E_l": 128, "d": 2048,
         "F": 768, "dtype": "bf16", "transposed": True},
        # decoding: one token through its eight experts
        {"name": "ffn, one token", "op": "ffn", "T": 1, "d": 2048, "F": 768, "E": 128, "E_l": 128,
         "K": 8, "dtype": "bf16", "zipf": 0.0, "gather": True, "train": False},
        # a ragged prompt on an EP8 rank: skewed experts, most pairs elsewhere
        {"name": "ffn, ragged window", "op": "ffn", "T": 1333, "d": 2048, "F": 1408, "E": 64,
         "E_l": 8, "K": 6, "dtype": "f16", "zipf": 1.1, "gather": False, "train": False},
        # a training micro-batch of the 128-expert layer, h kept for the backward
        {"name": "ffn, 128 experts", "op": "ffn", "T": 16384, "d": 2048, "F": 768, "E": 128,
         "E_l": 128, "K": 8, "dtype": "bf16", "zipf": 0.0, "gather": True, "train": True},
        # a small micro-batch whose rows were dispatched before the call
        {"name": "dgrad, 4 experts", "op": "dgrad", "T": 257, "d": 640, "F": 384, "E": 4,
         "E_l": 4, "K": 2, "dtype": "f16", "zipf": 0.0, "gather": False},
        # the backward of the 128-expert micro-batch, output gradients by token
        {"name": "dgrad, 128 experts", "op": "dgrad", "T": 16384, "d": 2048, "F": 768, "E": 128,
         "E_l": 128, "K": 8, "dtype": "bf16", "zipf": 0.0, "gather": True},
        # the small tensors of a model: routers, biases, norms
        {"name": "adamw, 24 small, 32-bit", "op": "adamw", "tensors": 24, "n": 6001,
         "dtype": "f32", "bits": 32, "master": False},
        # one EP16 rank's experts, 32-bit states, bf16 weights with float32 masters
        {"name": "adamw, 8 experts, 32-bit", "op": "adamw", "tensors": 2, "n": 18874368,
         "dtype": "bf16", "bits": 32, "master": True},
        # the 128-expert layer's weights, 8-bit states
        {"name": "adamw, 128 experts, 8-bit", "op": "adamw", "tensors": 3, "n": 201326592,
         "dtype": "bf16", "bits": 8, "master": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quant_rows", "quant_weights", "ffn", "ffn", "dgrad", "dgrad", "adamw",
                     "adamw"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "quant_rows":
        d = 128 * log(1, 32)
        return {"op": op, "T": min(log(1, 65536), 65536 * 2048 // d), "d": d,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "quant_weights":
        d, F = 128 * log(1, 32), 128 * log(1, 12)
        return {"op": op, "E_l": max(1, min(log(1, 128), 128 * 2048 * 768 // (d * F))), "d": d,
                "F": F, "dtype": dtype, "transposed": rng.random() < 0.5}
    if op == "adamw":
        k = log(1, 64)
        bits = rng.choice([8, 32])
        return {"op": op, "tensors": k, "n": log(1, 60000000 // k),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "bits": bits,
                "master": rng.random() < 0.5}
    d, F = 128 * log(1, 24), 128 * log(1, 12)
    E = rng.choice([4, 8, 16, 64, 128])
    E_l = max(1, E // rng.choice([1, 1, 2, 8]))
    K = rng.randint(1, min(E, 8))
    # no more rows, weights or products than the largest listed case
    T = min(log(1, 16384), max(1, 131072 * 2048 * 768 // (K * d * F)), 131072 // K)
    T = max(T, 8 * E // (E_l * K))  # some rows in the window
    case = {"op": op, "T": T, "d": d, "F": F, "E": E, "E_l": E_l, "K": K, "dtype": dtype,
            "zipf": rng.choice([0.0, 1.1]), "gather": rng.random() < 0.5}
    if op == "ffn":
        case["train"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# the block format: e4m3 values, one E8M0 scale (a power of two) per block of 128
# ---------------------------------------------------------------------------
def _scale_ld(k):
    """Scale bytes per row of k values: a multiple of four."""
    return (k // BLOCK + 3) // 4 * 4


def _scale_byte(amax):
    """Biased exponent of the smallest power of two s with amax / s <= 448
    (= 1.75 * 2^8); 127 for a block of zeros.  amax: float32."""
    bits = amax.view(torch.int32)
    byte = (((bits + 0x1FFFFF) >> 23) - 8).clamp(0, 254)
    return torch.where(amax == 0, 127, byte)


def _pow2(e):
    return torch.exp2(e.to(torch.float64)).to(torch.float32)


def _quant(x):
    """float32 [..., k] -> (e4m3 [..., k], scale bytes [..., k / 128])."""
    b = x.view(*x.shape[:-1], -1, BLOCK)
    amax = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    byte = _scale_byte(amax)
    q = (b * _pow2(127 - byte)[..., None]).to(torch.float8_e4m3fn)
    return q.view(x.shape), byte.to(torch.uint8)


def _pad_scales(s, k):
    out = s.new_zeros(*s.shape[:-1], _scale_ld(k))
    out[..., :s.shape[-1]] = s
    return out


def _dequant(q, s):
    """e4m3 [..., k] with scale bytes [..., >= k / 128] -> float32."""
    kb = q.shape[-1] // BLOCK
    b = q.float().view(*q.shape[:-1], kb, BLOCK)
    return (b * _pow2(s[..., :kb].int() - 127)[..., None]).view(q.shape)


def _quant_w(W):
    """float32 [E, n, k] -> (e4m3 [E, n, k], scale bytes [E, n / 128, k / 128])."""
    E, n, k = W.shape
    b = W.view(E, n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    byte = _scale_byte(torch.where(torch.isfinite(b), b.abs(), 0.0).amax((2, 4)))
    q = (b * _pow2(127 - byte)[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(E, n, k), byte.to(torch.uint8)


def _dequant_w(q, s):
    E, n, k = q.shape
    b = q.float().view(E, n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    return (b * _pow2(s[:, :, :k // BLOCK].int() - 127)[:, :, None, :, None]).view(E, n, k)


def _t(q):
    """The transpose of the last two dimensions of an e4m3 tensor, laid out."""
    return q.view(torch.uint8).transpose(-1, -2).contiguous().view(torch.float8_e4m3fn)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _weights(case, g):
    """The experts' quantised weights, both ways round."""
    E_l, d, F = case["E_l"], case["d"], case["F"]
    w = {}
    for name, n, k in (("gu", 2 * F, d), ("down", d, F)):
        q, s = _quant_w(_randn(g, E_l, n, k, std=0.02))
        w[name], w[name + "_s"] = q, _pad_scales(s, k)
        w[name + "T"], w[name + "T_s"] = _t(q), _pad_scales(s.transpose(1, 2), n)
    return w


def _plan(case, g):
    """The dispatch plan of top-K routing, as moe_dispatch lays it out, and
    the gates; "experts" and "R": the local experts with rows and the most rows
    that one has."""
    T, E, E_l, K = case["T"], case["E"], case["E_l"], case["K"]
    logits = _randn(g, T, E)
    if case["zipf"]:
        logits -= case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda"))
    top, idx = torch.topk(logits, K, dim=1)
    flat = idx.reshape(-1)
    key = torch.where(flat < E_l, flat, E_l)  # the local window is [0, E_l)
    counts = torch.bincount(key, minlength=E_l + 1)[:E_l]
    N = int(counts.sum())
    pair = torch.sort(key, stable=True)[1][:N]
    pair_of_row = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    pair_of_row[:N] = pair.int()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    experts = torch.nonzero(counts).view(-1)
    return {
        "N": N, "R": int(counts.max()), "experts": experts, "pair_of_row": pair_of_row,
        "offsets": torch.cat([zero, counts.cumsum(0)]).int(),
        "tile_offsets": torch.cat([zero, (-(-counts // TILE_M)).cumsum(0)]).int(),
        "gates": torch.softmax(top, 1).reshape(-1).contiguous(),
    }


def _buffers(case, names):
    cap, d, F = case["T"] * case["K"], case["d"], case["F"]
    cols = {"h": 2 * F, "a": F, "yp": d, "dh": 2 * F, "dxp": d, "ag": F}
    return {n: torch.zeros(cap, cols[n], dtype=DTYPES[case["dtype"]], device="cuda")
            for n in names}


def _fp8_workspace(case):
    """At least moe_fp8_workspace_bytes: a [T*K, 2F] float32 matrix."""
    return torch.empty(case["T"] * case["K"] * 8 * case["F"] + 4096, dtype=torch.uint8,
                       device="cuda")


def _sizes(case):
    """Elements of each tensor of an optimizer step."""
    return [max(1, case["n"] >> min(i, 2)) + (i if i > 2 else 0) for i in range(case["tensors"])]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op == "quant_rows":
        x = _randn(g, case["T"], case["d"]) * torch.exp(_randn(g, case["T"], 1))
        st["x"] = x.to(DTYPES[case["dtype"]])
        st["q"] = torch.zeros(case["T"], case["d"], dtype=torch.float8_e4m3fn, device="cuda")
        st["s"] = torch.zeros(case["T"], _scale_ld(case["d"]), dtype=torch.uint8, device="cuda")
    elif op == "quant_weights":
        E_l, d, F = case["E_l"], case["d"], case["F"]
        st["W_gu"] = _randn(g, E_l, 2 * F, d, std=0.02).to(DTYPES[case["dtype"]])
        st["W_down"] = _randn(g, E_l, d, F, std=0.02).to(DTYPES[case["dtype"]])
        w = {}
        for name, n, k in (("gu", 2 * F, d), ("down", d, F)):
            w[name] = torch.zeros(E_l, n, k, dtype=torch.float8_e4m3fn, device="cuda")
            w[name + "_s"] = torch.zeros(E_l, n // BLOCK, _scale_ld(k), dtype=torch.uint8,
                                         device="cuda")
            if case["transposed"]:
                w[name + "T"] = torch.zeros(E_l, k, n, dtype=torch.float8_e4m3fn, device="cuda")
                w[name + "T_s"] = torch.zeros(E_l, k // BLOCK, _scale_ld(n), dtype=torch.uint8,
                                              device="cuda")
        st["w"] = w
    elif op in ("ffn", "dgrad"):
        rows = case["T"] if case["gather"] else case["T"] * case["K"]
        q, s = _quant(_randn(g, rows, case["d"]))
        st |= {"q": q, "s": _pad_scales(s, case["d"]), "w": _weights(case, g),
               "ws": _fp8_workspace(case)}
        st |= _plan(case, g)
        if op == "ffn":
            st |= _buffers(case, ["h", "a", "yp"] if case["train"] else ["yp"])
        else:
            st |= _buffers(case, ["h", "dh", "dxp"] + (["ag"] if case["gather"] else []))
            st["h"].copy_(_randn(g, *st["h"].shape, std=0.9))
    else:
        # the tensors lie in flat buffers, each from a multiple of 128 elements on
        dt, bits, sizes = DTYPES[case["dtype"]], case["bits"], _sizes(case)
        room = [-(-n // BLOCK) * BLOCK for n in sizes]
        real = torch.cat([(torch.arange(r, device="cuda") < n) for n, r in zip(sizes, room)])
        master, grad = _randn(g, sum(room), std=0.02) * real, _randn(g, sum(room), std=1e-3) * real
        m, r = _randn(g, sum(room), std=3e-4) * real, _randn(g, sum(room), std=1e-3).abs() * real
        flat = {"param": master.to(dt), "grad": grad}
        if case["master"]:
            flat["master"] = master
        if bits == 32:
            flat |= {"m": m, "v": r * r}
        else:
            flat["m"], flat["m_s"] = _quant(m)
            flat["v"], flat["v_s"] = _quant(r)
        st["flat"], st["tensors"], at = flat, [], 0
        for n, k in zip(sizes, room):
            st["tensors"].append({
                name: x[at // BLOCK:(at + k) // BLOCK] if name.endswith("_s") else x[at:at + n]
                for name, x in flat.items()})
            at += k
        st["hyper"] = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1,
                       "step": 1000 + seed % 1000, "grad_scale": 0.5, "seed": seed}
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _expert_rows(st):
    """[experts, R] row numbers of the experts that have rows, and which of
    them exist."""
    first, end = st["offsets"][st["experts"]].long(), st["offsets"][st["experts"] + 1].long()
    rows = first[:, None] + torch.arange(st["R"], device="cuda")
    return torch.minimum(rows, end[:, None] - 1), rows < end[:, None]


def _operand(st, rows):
    """The quantised rows that the dispatched rows read."""
    src = rows
    if st["case"]["gather"]:
        src = st["pair_of_row"][rows].long() // st["case"]["K"]
    return _dequant(st["q"], st["s"])[src]


def _requant(x):
    return _dequant(*_quant(x))


def _put(out, rows, ok, x):
    out[rows[ok]] = x[ok].to(out.dtype)


def _plain_ffn(st):
    case, F = st["case"], st["case"]["F"]
    out = {n: torch.zeros_like(st[n]) for n in ("h", "a", "yp") if n in st}
    if st["N"]:
        rows, ok = _expert_rows(st)
        W_gu = _dequant_w(st["w"]["gu"][st["experts"]], st["w"]["gu_s"][st["experts"]])
        W_down = _dequant_w(st["w"]["down"][st["experts"]], st["w"]["down_s"][st["experts"]])
        h = torch.bmm(_operand(st, rows), W_gu.transpose(1, 2))
        g, u = h[..., :F], h[..., F:]
        a = g / (1 + torch.exp(-g)) * u
        y = torch.bmm(_requant(a), W_down.transpose(1, 2))
        _put(out["yp"], rows, ok, y)
        if case["train"]:
            _put(out["h"], rows, ok, h)
            _put(out["a"], rows, ok, a)
    return out


def _plain_dgrad(st):
    case, F = st["case"], st["case"]["F"]
    names = ("dh", "dxp", "ag") if case["gather"] else ("dh", "dxp")
    out = {n: torch.zeros_like(st[n]) for n in names}
    if st["N"]:
        rows, ok = _expert_rows(st)
        W_gu = _dequant_w(st["w"]["gu"][st["experts"]], st["w"]["gu_s"][st["experts"]])
        W_down = _dequant_w(st["w"]["down"][st["experts"]], st["w"]["down_s"][st["experts"]])
        da = torch.bmm(_operand(st, rows), W_down)
        h = st["h"][rows].float()
        g, u = h[..., :F], h[..., F:]
        s = 1 / (1 + torch.exp(-g))
        if case["gather"]:
            gate = st["gates"][st["pair_of_row"][rows].long()][..., None]
            da = da * gate
            _put(out["ag"], rows, ok, gate * (g * s) * u)
        dh = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], -1)
        _put(out["dh"], rows, ok, dh)
        _put(out["dxp"], rows, ok, torch.bmm(_requant(dh), W_gu))
    return out


def _mul32(a, c):
    return (a * c) & 0xFFFFFFFF


def _random_bits(n, index, hyper):
    """Two 20-bit random numbers per element: a mix of the element's index
    with a key made of the seed, the step and the tensor's number."""
    key = ((hyper["seed"] & 0xFFFFFFFF) ^ (((hyper["seed"] >> 32) * 0x85EBCA77) & 0xFFFFFFFF)
           ^ ((hyper["step"] * 0x9E3779B1) & 0xFFFFFFFF) ^ ((index * 0xC2B2AE3D) & 0xFFFFFFFF))
    x = torch.arange(n, device="cuda") ^ key
    x = _mul32(x ^ (x >> 16), 0x9E3779B1)
    x = _mul32(x ^ (x >> 15), 0xC2B2AE3D)
    x = x ^ (x >> 16)
    return x >> 12, _mul32(x, 0x9E3779B1) >> 12


def _quant_random(x, rnd):
    """float32 [n] -> e4m3 [n], scale bytes: as _quant, but rounded up or down
    at random: a 20-bit number is added below the last kept bit, which is
    then cut off (below 2^-6 the values have the fixed spacing 2^-9)."""
    n = x.numel()
    b = torch.cat([x, x.new_zeros(-n % BLOCK)]).view(-1, BLOCK)
    byte = _scale_byte(torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1))
    y = (b * _pow2(127 - byte)[:, None]).view(-1)[:n]
    mag = y.abs()
    normal = ((mag.view(torch.int32).long() + rnd) >> 20) - 960
    small = torch.floor(mag * 512 + rnd.float() * 2.0 ** -20).nan_to_num(0, 0, 0).long()
    code = torch.where(mag >= 2.0 ** -6, normal, small)
    code = torch.where(torch.isfinite(y), code, 127)
    code = torch.where(torch.signbit(y), code + 128, code)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), byte.to(torch.uint8)


def _dequant_flat(q, s):
    return q.float() * _pow2(s.int() - 127).repeat_interleave(BLOCK)[:q.numel()]


def _f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def _plain_adamw(t, index, hyper):
    b1, b2, lr = hyper["beta1"], hyper["beta2"], hyper["lr"]
    wide = "m_s" not in t
    grad = t["grad"] * _f32(hyper["grad_scale"])
    m = t["m"] if wide else _dequant_flat(t["m"], t["m_s"])
    v = t["v"] if wide else _dequant_flat(t["v"], t["v_s"]).square()
    m = m * _f32(b1) + grad * _f32(1 - b1)
    v = v * _f32(b2) + grad * grad * _f32(1 - b2)
    p = t["master"] if "master" in t else t["param"].float()
    root = torch.sqrt(v)
    p = p * _f32(1 - lr * hyper["weight_decay"]) - m * _f32(lr / (1 - b1 ** hyper["step"])) / (
        root * _f32(1 / math.sqrt(1 - b2 ** hyper["step"])) + _f32(hyper["eps"]))
    t["param"].copy_(p)
    if "master" in t:
        t["master"].copy_(p)
    if wide:
        t["m"].copy_(m)
        t["v"].copy_(v)
    else:
        bits = _random_bits(p.numel(), index, hyper)
        for name, x, r in (("m", m, bits[0]), ("v", root, bits[1])):
            q, s = _quant_random(x, r)
            t[name].copy_(q)
            t[name + "_s"].copy_(s)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if own:
        return _run_own(st, case, op)
    if op == "quant_rows":
        q, s = _quant(st["x"].float())
        return {"q": q, "s": _pad_scales(s, case["d"])}
    if op == "quant_weights":
        out = {}
        for name, W in (("gu", st["W_gu"]), ("down", st["W_down"])):
            q, s = _quant_w(W.float())
            out[name], out[name + "_s"] = q, _pad_scales(s, W.shape[2])
            if case["transposed"]:
                out[name + "T"] = _t(q)
                out[name + "T_s"] = _pad_scales(s.transpose(1, 2), W.shape[1])
        return out
    if op == "ffn":
        return _plain_ffn(st)
    if op == "dgrad":
        return _plain_dgrad(st)
    [_plain_adamw(t, i, st["hyper"]) for i, t in enumerate(st["tensors"])]
    return {n: x for n, x in st["flat"].items() if n != "grad"}


def _run_own(st, case, op):
    import combine_expert_ffn_amd as M

    if op == "quant_rows":
        if "shape" not in st:
            st["shape"] = M.make_shape(case["T"], case["d"], 128, 1, 0, 1, 1, case["dtype"])
        M.moe_quant_rows_fp8(st["shape"], st["x"], case["T"], None, st["q"], st["s"])
        return {"q": st["q"], "s": st["s"]}
    if op == "adamw":
        if "list" not in st:
            st["list"] = M.AdamWTensors(
                [dict(t, weight_decay=st["hyper"]["weight_decay"]) for t in st["tensors"]])
        h = st["hyper"]
        M.moe_adamw(st["list"], lr=h["lr"], beta1=h["beta1"], beta2=h["beta2"], eps=h["eps"],
                    step=h["step"], grad_scale=h["grad_scale"], seed=h["seed"])
        return {n: x for n, x in st["flat"].items() if n != "grad"}
    if "shape" not in st:
        st["shape"] = M.make_shape(case.get("T", 1), case["d"], case["F"],
                                   case.get("E", case["E_l"]), 0, case["E_l"], case.get("K", 1),
                                   case["dtype"])
        st["fp8"] = M.Fp8Weights(st["shape"], **st["w"])
    s = st["shape"]
    if op == "quant_weights":
        M.moe_quant_weights_fp8(s, st["W_gu"], st["W_down"], st["fp8"])
        return st["w"]
    rows = st["pair_of_row"] if case["gather"] else None
    if op == "ffn":
        M.moe_expert_ffn_fwd_fp8(s, st["q"], st["s"], rows, st["offsets"], st["tile_offsets"],
                                 st["fp8"], st.get("h"), st.get("a"), st["yp"], st["ws"])
        return {n: st[n] for n in ("h", "a", "yp") if n in st}
    M.moe_ffn_dgrad_fp8(s, st["q"], st["s"], rows, st["gates"] if case["gather"] else None,
                        st["h"], st["offsets"], st["tile_offsets"], st["fp8"], st["dh"],
                        st["dxp"], st.get("ag"), st["ws"])
    return {n: st[n] for n in ("dh", "dxp", "ag") if n in st}


# ---------------------------------------------------------------------------
# the work of one pass
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    b = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if op == "quant_rows":
        n = case["T"] * case["d"]
        return {"bytes": n * (b + 1) + n // BLOCK, "flops": 3 * n}
    if op == "quant_weights":
        n = case["E_l"] * 3 * case["F"] * case["d"]
        return {"bytes": n * (b + (2 if case["transposed"] else 1)), "flops": 3 * n}
    if op == "adamw":
        n = sum(_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * (4 + state + (8 + b if case["master"] else 2 * b)), "flops": 16 * n}
    # rows of the local window, as expected of the routing
    T, d, F, E, E_l, K = (case[k] for k in ("T", "d", "F", "E", "E_l", "K"))
    p = [(e + 1.0) ** -case["zipf"] for e in range(E)]
    share = [1 - (1 - x / sum(p)) ** K for x in p[:E_l]]
    scale = K / sum(1 - (1 - x / sum(p)) ** K for x in p)
    N = T * min(K, sum(share) * scale)
    experts = sum(1 - (1 - x) ** T for x in share)
    flops = 6 * N * d * F
    src = min(T, N) if case["gather"] else N
    size = src * d + experts * 3 * d * F + N * d * b
    if op == "ffn":
        size += N * 3 * F * b if case["train"] else 0
    else:
        size += N * 4 * F * b + (N * F * b if case["gather"] else 0)
    return {"bytes": size, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_nearest(y):
    """The e4m3 value nearest to y (ties to even), float64."""
    _, ex = torch.frexp(y)
    step = torch.exp2((ex - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _block_scale(amax):
    """Smallest power of two s with amax / s <= 448, 1 where amax is 0."""
    f, ex = torch.frexp(amax / 448)
    e = torch.where(f == 0.5, ex - 1, ex).clamp(-127, 127).double()
    return torch.where(amax == 0, 1.0, torch.exp2(e))


def _exact_rounded(x):
    """What x stands for after quantisation in blocks of 128 of its last axis."""
    b = x.unflatten(-1, (-1, BLOCK))
    s = _block_scale(b.abs().amax(-1, keepdim=True))
    return (_e4m3_nearest(b / s) * s).flatten(-2)


def _value(q, s, down=1):
    k = q.shape[-1] // BLOCK
    e = s[..., :k].double() - 127
    if down > 1:
        e = e.repeat_interleave(down, -2)
    return q.double() * torch.exp2(e).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    op = case["op"]
    if op == "quant_rows" or op == "quant_weights":
        st = prepare(case, seed)
        if op == "quant_rows":
            b = st["x"].double().unflatten(-1, (-1, BLOCK))
            s = _block_scale(b.abs().amax(-1, keepdim=True))
            return {"q": _e4m3_nearest(b / s).flatten(-2), "s": None}
        out = {}
        for name in ("gu", "down"):
            W = st["W_" + name].double()
            b = W.unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK))
            s = _block_scale(b.abs().amax((2, 4), keepdim=True))
            q = _e4m3_nearest(b / s).flatten(3, 4).flatten(1, 2)
            out[name] = q
            if case["transposed"]:
                out[name + "T"] = q.transpose(1, 2).contiguous()
        return out
    if op == "adamw":
        return _exact_adamw(case, seed)
    st = prepare(case, seed)
    F, K = case["F"], case["K"]
    names = [n for n in ("h", "a", "yp") if n in st] if op == "ffn" else [
        n for n in ("dh", "dxp", "ag") if n in st]
    out = {n: torch.zeros(st[n].shape, dtype=torch.float64, device="cuda") for n in names}
    off = st["offsets"].tolist()
    for e in range(case["E_l"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        pair = st["pair_of_row"][lo:hi].long()
        src = torch.div(pair, K, rounding_mode="floor") if case["gather"] else slice(lo, hi)
        x = _value(st["q"][src], st["s"][src])
        W_gu = _value(st["w"]["gu"][e], st["w"]["gu_s"][e], BLOCK)
        W_down = _value(st["w"]["down"][e], st["w"]["down_s"][e], BLOCK)
        if op == "ffn":
            h = x @ W_gu.T
            a = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
            now = {"h": h, "a": a, "yp": _exact_rounded(a) @ W_down.T}
        else:
            h = st["h"][lo:hi].double()
            g, u, sg = h[:, :F], h[:, F:], torch.sigmoid(h[:, :F])
            gate = st["gates"][pair].double()[:, None] if case["gather"] else 1.0
            da = gate * (x @ W_down)
            dh = torch.cat([da * u * (sg + g * sg * (1 - sg)), da * g * sg], 1)
            now = {"dh": dh, "dxp": _exact_rounded(dh) @ W_gu, "ag": gate * g * sg * u}
        for n in names:
            out[n][lo:hi] = now[n]
    return out


def _exact_adamw(case, seed):
    st = prepare(case, seed)
    h = st["hyper"]
    out = {n: torch.zeros(x.shape, dtype=torch.float64, device="cuda")
           for n, x in st["flat"].items() if n != "grad" and not n.endswith("_s")}
    b1, b2, t_, at = h["beta1"], h["beta2"], h["step"], 0
    for index, t in enumerate(st["tensors"]):
        n = t["grad"].numel()
        g = t["grad"].double() * h["grad_scale"]
        m, v = t["m"].double(), t["v"].double()
        if case["bits"] == 8:
            m = m * torch.exp2(t["m_s"].double() - 127).repeat_interleave(BLOCK)[:n]
            v = (v * torch.exp2(t["v_s"].double() - 127).repeat_interleave(BLOCK)[:n]) ** 2
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        p = t.get("master", t["param"]).double()
        p = p - h["lr"] * (m / (1 - b1 ** t_) / (torch.sqrt(v / (1 - b2 ** t_)) + h["eps"])
                           + h["weight_decay"] * p)
        if case["bits"] == 8:
            rounded = []
            for x, r in zip((m, v.sqrt()), _random_bits(n, index, h)):
                pad = torch.cat([x, x.new_zeros(-n % BLOCK)]).view(-1, BLOCK)
                s = _block_scale(pad.abs().amax(1)).repeat_interleave(BLOCK)[:n]
                y = (x / s).abs()
                step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
                rounded.append(torch.copysign(
                    torch.floor(y / step + r.double() * 2.0 ** -20) * step, x))
            m, v = rounded
        for name, x in (("param", p), ("master", p), ("m", m), ("v", v)):
            if name in out:
                out[name][at:at + n] = x
        at += -(-n // BLOCK) * BLOCK
    return out
