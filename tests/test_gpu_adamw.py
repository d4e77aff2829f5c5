"""moe_adamw on the GPU against the float64 definition.

Tolerances, fixed before the first run: the step is a fixed sequence of float32
operations, each off by at most half a step (2^-24 relative).  m and v are three
roundings of sums of same-scale terms; the update's quotient adds the roundings
of its two factors, the root, the sum and the division, eight in all; so 2^-21 of
the magnitudes that enter (8 * 2^-24).  An 8-bit state is either of the two
values around the exact one: within one e4m3 step (2^-3 of the value at most), and
equal to the oracle's on all but the elements that the float32 error carries over
a rounding border (a share of about 2^-24 * 2^20 / 2^20 per unit of error: far below
1 in 1000).
"""

import numpy as np
import pytest
import torch

import combine_expert_ffn_amd as M
from oracle import fp8_oracle as Q
from moe_harness import host

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HP = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()


def make(n, dtype, bits, master, seed, off=0):
    """A tensor and its state; off: elements by which every buffer is shifted, so
    that pointers are aligned to their element type only."""
    rng = np.random.default_rng(seed)
    f = lambda std: torch.from_numpy((rng.normal(size=n) * std).astype(np.float32)).cuda()

    def place(x):
        big = torch.zeros(n + off + 8, dtype=x.dtype, device="cuda")
        big[off: off + n] = x
        return big[off: off + n]

    p = f(0.05)
    t = dict(param=place(p.to(DT[dtype])), grad=place(f(1e-2)), weight_decay=0.1,
             master=place(p) if master else None)
    m, r = f(3e-3), f(1e-2).abs()
    if bits == 32:
        return dict(t, m=place(m), v=place(r * r))
    out = dict(t)
    for name, x in (("m", m), ("v", r)):
        q, b = Q.quant_rows(np.concatenate([host(x), np.zeros(-n % 128)]))
        code = torch.from_numpy(q[:n].astype(np.float32)).cuda().to(torch.float8_e4m3fn)
        out[name] = place(code.view(torch.uint8)).view(torch.float8_e4m3fn)
        out[name + "_s"] = torch.from_numpy(b.astype(np.uint8)).cuda()
    return out


def state_of(t):
    n = t["param"].numel()
    if "m_s" not in t:
        return host(t["m"]), host(t["v"])
    val = lambda k: host(t[k].float()) * np.repeat(np.ldexp(1.0, host(t[k + "_s"]).astype(int)
                                                            - 127), 128)[:n]
    return val("m"), val("v") ** 2


def snapshot(tensors):
    return [dict(p=host(t["master"] if t.get("master") is not None else t["param"]),
                 g=host(t["grad"]), mv=state_of(t)) for t in tensors]


def check(tensors, before, step, scale=1.0, seed=0, **hp):
    hp = dict(HP, **hp)
    for i, (t, b) in enumerate(zip(tensors, before)):
        n = b["p"].size
        if n == 0:
            continue
        wd = float(np.float32(t.get("weight_decay", 0.0)))
        p, m, v = Q.adamw(b["p"], b["g"], *b["mv"], hp["lr"], hp["beta1"], hp["beta2"],
                          hp["eps"], wd, step, scale)
        upd = np.abs(hp["lr"] * m / (1 - hp["beta1"] ** step)) / (
            np.sqrt(v / (1 - hp["beta2"] ** step)) + hp["eps"])
        m_mag = hp["beta1"] * np.abs(b["mv"][0]) + (1 - hp["beta1"]) * np.abs(scale * b["g"])
        upd = upd * m_mag / np.maximum(np.abs(m), 1e-300)   # m's own rounding, before the quotient
        tol = (np.abs(b["p"]) + upd) * 2.0 ** -21 + 1e-37
        if t.get("master") is not None:
            assert (np.abs(host(t["master"]) - p) <= tol).all(), f"master {i}"
            assert torch.equal(t["param"], t["master"].to(t["param"].dtype)), f"param {i}"
        else:
            half = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8,
                    torch.float16: 2.0 ** -11}[t["param"].dtype]
            flat = 2.0 ** -24 if t["param"].dtype == torch.float16 else 0.0
            assert (np.abs(host(t["param"]) - p) <= tol + (np.abs(p) + tol) * half + flat).all(), \
                f"param {i}"
        if "m_s" not in t:
            assert (np.abs(host(t["m"]) - m) <= m_mag * 2.0 ** -21 + 1e-45).all(), f"m {i}"
            assert (np.abs(host(t["v"]) - v) <= v * 2.0 ** -21 + 1e-45).all(), f"v {i}"
            continue
        bits = Q.random_bits(n, i, seed, step)
        for name, x, r in (("m", m, bits[0]), ("v", np.sqrt(v), bits[1])):
            q, byte = Q.quant_random(x, r)
            got, gb = host(t[name].float()), host(t[name + "_s"])
            # a scale may differ only where the largest value lies on its border
            assert (gb != byte).sum() <= max(1, byte.size // 1000), f"{name}_s {i}"
            same = np.repeat(gb == byte, 128)[:n]
            # elements whose m is the small difference of two larger terms carry
            # their absolute error: counted with the rest
            assert (got != q)[same].sum() <= max(1, n // 1000), f"{name} {i}"
            step_ = np.maximum(np.abs(q) * 2.0 ** -3, 2.0 ** -9)
            assert (np.abs(got - q) <= step_ * 1.01)[same].all(), f"{name} {i}"


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_sizes(dtype, bits, master):
    sizes = [1, 7, 8, 127, 128, 129, 0, 1000, 2047, 2048, 2049, 70001]
    ts = [make(n, dtype, bits, master, 10 + i) for i, n in enumerate(sizes)]
    before = snapshot(ts)
    M.moe_adamw(ts, step=3, grad_scale=0.5, seed=77, **HP)
    check(ts, before, 3, 0.5, 77)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("off", [1, 2, 3, 4, 8])
def test_unaligned(bits, off):
    ts = [make(300, "bf16", bits, True, off, off), make(41, "f32", bits, False, off, off)]
    before = snapshot(ts)
    M.moe_adamw(ts, step=1, seed=(9 << 40) + 5, **HP)
    check(ts, before, 1, 1.0, (9 << 40) + 5)


def test_more_tensors_than_one_launch_takes():
    """Mixed types, sizes and state widths over several launches, and the
    elements beside each tensor left alone."""
    ts = []
    for i in range(97):
        ts.append(make(1 + 37 * i % 700, ["bf16", "f16", "f32"][i % 3], 8 if i % 2 else 32,
                       i % 5 == 0, i, off=i % 4))
    around = [t["param"].storage_offset() for t in ts]
    assert max(around) == 3
    before = snapshot(ts)
    M.moe_adamw(ts, step=11, seed=4, **HP)
    check(ts, before, 11, 1.0, 4)
    for t in ts:
        whole = torch.as_strided(t["param"], (t["param"].storage_offset() + t["param"].numel() + 4,),
                                 (1,), 0)
        k = t["param"].storage_offset()
        assert (whole[:k] == 0).all() and (whole[k + t["param"].numel():] == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_shared_memory_is_refused(bits):
    """The same tensor twice, or a buffer inside another, would be a race; one
    gradient for two tensors is fine."""
    a, b = make(300, "bf16", bits, True, 1), make(300, "bf16", bits, True, 2)
    M.AdamWTensors([a, dict(b, grad=a["grad"])])
    for bad in (dict(a), dict(b, param=a["param"]), dict(b, master=a["grad"]),
                dict(b, m=a["v"]), dict(b, grad=b["master"]), dict(b, v=b["m"])):
        with pytest.raises(M.MoeError) as e:
            M.AdamWTensors([a, bad])
        assert e.value.code == M.MOE_ERR_ARG
    flat = torch.zeros(700, dtype=torch.bfloat16, device="cuda")
    M.AdamWTensors([dict(a, param=flat[:300]), dict(b, param=flat[300:600])])
    with pytest.raises(M.MoeError):
        M.AdamWTensors([dict(a, param=flat[:300]), dict(b, param=flat[299:599])])


def test_device_gradient_scale():
    a, b = [make(500, "bf16", 8, True, 1)], [make(500, "bf16", 8, True, 1)]
    clip = torch.tensor([0.25], device="cuda")
    M.moe_adamw(a, step=2, grad_scale=2.0, grad_scale_dev=clip, seed=1, **HP)
    M.moe_adamw(b, step=2, grad_scale=0.5, seed=1, **HP)
    for k in ("param", "master", "m_s", "v_s"):
        assert torch.equal(a[0][k], b[0][k]), k
    assert torch.equal(a[0]["m"].view(torch.uint8), b[0]["m"].view(torch.uint8))


def test_zero_gradients_and_states():
    """An untouched tensor only decays; zero blocks keep scale 1."""
    t = make(260, "f32", 8, False, 2)
    for k in ("m", "v"):
        t[k].view(torch.uint8).zero_()
        t[k + "_s"].fill_(127)
    t["grad"].zero_()
    p = host(t["param"])
    M.moe_adamw([t], step=1, seed=3, **HP)
    keep = np.float32(1.0 - HP["lr"] * float(np.float32(0.1)))
    assert np.array_equal(host(t["param"]).astype(np.float32), p.astype(np.float32) * keep)
    assert (host(t["m"].float()) == 0).all() and (host(t["v"].float()) == 0).all()
    assert (host(t["m_s"]) == 127).all() and (host(t["v_s"]) == 127).all()


def test_nonfinite_gradient_stays_in_its_element():
    a, b = make(300, "f32", 8, False, 5), make(300, "f32", 8, False, 5)
    a["grad"][130] = float("nan")
    a["grad"][131] = float("inf")
    M.moe_adamw([a], step=4, seed=3, **HP)
    M.moe_adamw([b], step=4, seed=3, **HP)
    ok = torch.ones(300, dtype=torch.bool, device="cuda")
    ok[130:132] = False
    assert torch.equal(a["param"][ok], b["param"][ok])
    assert torch.isnan(a["param"][130]) and torch.isnan(a["m"].float()[130])
    # blocks without them are as without them
    assert torch.equal(a["m"].view(torch.uint8)[256:], b["m"].view(torch.uint8)[256:])
    assert torch.isfinite(a["m"].float()[ok]).all()


def test_same_arguments_same_results_other_seed_others():
    run = lambda seed, step=5: (lambda t: (M.moe_adamw([t], step=step, seed=seed, **HP),
                                           host(t["m"].float()))[1])(make(4000, "bf16", 8, True, 6))
    a = run(1)
    assert np.array_equal(a, run(1))
    assert (a != run(2)).any() and (a != run(1, 6)).any()


def test_many_steps_follow_the_moments():
    """8-bit states follow a constant gradient: sqrt(v) approaches |g| at the rate
    beta2 gives, which rounding to nearest could not do (1 - beta2 = 1/1000 is
    far below half a step).  After 600 steps v is g^2 (1 - 0.999^600) = 0.451 g^2; the mean
    over 4096 elements of a walk whose every step is right in the mean has a
    standard error of at most one e4m3 step (12.5%) / 64 times the root of the
    number of independent rounding errors kept, below 1%: 5% is allowed."""
    n = 4096
    g = torch.ones(n, device="cuda") * 0.01
    t = dict(param=torch.zeros(n, device="cuda"), grad=g,
             m=torch.zeros(n, device="cuda").to(torch.float8_e4m3fn),
             v=torch.zeros(n, device="cuda").to(torch.float8_e4m3fn),
             m_s=torch.full((n // 128,), 127, dtype=torch.uint8, device="cuda"),
             v_s=torch.full((n // 128,), 127, dtype=torch.uint8, device="cuda"))
    ts = M.AdamWTensors([t])
    for k in range(1, 601):
        M.moe_adamw(ts, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, step=k, seed=k)
    m, v = state_of(t)
    assert abs(m.mean() / 0.01 - 1) < 0.05
    assert abs(np.sqrt(v).mean() / (0.01 * np.sqrt(1 - 0.999 ** 600)) - 1) < 0.05


def test_captured_step_replays():
    """A captured step, replayed between eager work, equals as many eager steps."""
    a, b = [make(5000, "bf16", 8, True, 9)], [make(5000, "bf16", 8, True, 9)]
    ta, tb = M.AdamWTensors(a), M.AdamWTensors(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_adamw(ta, step=7, seed=2, stream=torch.cuda.current_stream(), **HP)
    for k in range(4):
        g.replay()
        M.moe_adamw(tb, step=7, seed=2, **HP)
        a[0]["grad"].mul_(0.9)
        b[0]["grad"].mul_(0.9)
        torch.cuda.synchronize()
        for n in ("param", "master", "m_s", "v_s"):
            assert torch.equal(a[0][n], b[0][n]), (k, n)
        assert torch.equal(a[0]["v"].view(torch.uint8), b[0]["v"].view(torch.uint8))
