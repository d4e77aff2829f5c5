"""Objects that keep tensors between calls follow a tensor whose memory moves: the
addresses they hand to the library are those of the tensors now, checked again."""

import pytest
import torch

import combine_expert_ffn_amd as M

E4M3 = torch.float8_e4m3fn


@pytest.fixture
def on_cpu(monkeypatch):
    """The tensor checks without the one for the device."""
    checks = []

    def chk(s, fn, name, t, kind, numel, optional=False):
        checks.append(name)
        if t is None and optional:
            return
        if t.numel() < numel:
            raise M.MoeError(M.MOE_ERR_ARG, f"{name} has {t.numel()} elements")

    monkeypatch.setattr(M, "_chk", chk)
    return checks


def _weights():
    return M.Fp8Weights(M.make_shape(4, 256, 128, 2, 0, 2, 1, "bf16"), device="cpu")


def _pointers(w):
    w._current()
    return [getattr(w.struct, n) for n in M.FP8_WEIGHT_FIELDS]


def _now(w):
    return [getattr(w, n).data_ptr() for n in M.FP8_WEIGHT_FIELDS]


def test_weights_follow_their_tensors(on_cpu):
    w = _weights()
    assert _pointers(w) == _now(w)
    n = len(on_cpu)
    assert _pointers(w) == _now(w) and len(on_cpu) == n      # nothing moved, nothing checked
    w.gu.data = torch.zeros_like(w.gu)
    assert _pointers(w) == _now(w)
    w.downT_s.set_(torch.zeros_like(w.downT_s))
    assert _pointers(w) == _now(w)
    w.down = torch.zeros(w.down.shape, dtype=torch.uint8).view(E4M3)
    assert _pointers(w) == _now(w) and len(on_cpu) > n


def test_weights_that_shrank_are_refused(on_cpu):
    w = _weights()
    whole = w.gu_s.clone()
    w.gu_s.set_(torch.zeros(1, dtype=torch.uint8))
    for _ in range(2):                                       # and not taken on the second try
        with pytest.raises(M.MoeError):
            w._current()
    w.gu_s.set_(whole)
    assert _pointers(w) == _now(w)


def _tensors():
    f = lambda n: torch.zeros(n)
    return [dict(param=f(n), grad=f(n), m=f(n), v=f(n), master=None) for n in (5, 300)]


def _adam_pointers(a):
    a._current()
    return [getattr(a.array[i], k) for i in range(len(a.tensors)) for k in ("param", "grad", "m", "v")]


def _adam_now(ts):
    return [t[k].data_ptr() for t in ts for k in ("param", "grad", "m", "v")]


def test_adamw_tensors_follow_their_memory(on_cpu):
    ts = _tensors()
    a = M.AdamWTensors(ts)
    assert _adam_pointers(a) == _adam_now(ts)
    n = len(on_cpu)
    assert _adam_pointers(a) == _adam_now(ts) and len(on_cpu) == n
    ts[0]["grad"].data = torch.ones(5)
    ts[1]["param"].set_(torch.ones(300))
    assert _adam_pointers(a) == _adam_now(ts) and len(on_cpu) > n


def test_adamw_tensors_of_another_size_or_sharing_memory_are_refused(on_cpu):
    ts = _tensors()
    a = M.AdamWTensors(ts)
    ts[1]["v"].resize_(100000)
    for _ in range(2):
        with pytest.raises(M.MoeError):
            a._current()
    ts[1]["v"].resize_(300)
    assert _adam_pointers(a) == _adam_now(ts)
    ts[1]["m"].data = ts[1]["v"].data
    with pytest.raises(M.MoeError):
        a._current()


def test_a_held_address_is_not_given_away(on_cpu):
    """The memory a tensor had stays allocated until the next call has seen the move."""
    ts = _tensors()
    a = M.AdamWTensors(ts)
    old = ts[0]["grad"].data_ptr()
    ts[0]["grad"].data = torch.ones(7)
    assert old in [t.data_ptr() for t in a._kept]
    with pytest.raises(M.MoeError):
        a._current()
