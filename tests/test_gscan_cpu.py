"""The gated linear recurrence without a GPU: the float64 implementation that the GPU tests compare with (against
differences and a closed form), and the refusals of the C ABI and of the binding (no HIP call is made)."""
import os

import pytest
import torch

from linear_rnn_amd import wkv
from tests import gscan_ref as ref

F32, BF16 = wkv.RWKV7_DTYPE_F32, wkv.RWKV7_DTYPE_BF16
OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_ALIAS, E_MODE = 0, -1, -2, -4, -5, -6, -11
BASE, GAP = 1 << 40, 1 << 36


@pytest.mark.parametrize("kind", ref.KINDS)
@pytest.mark.parametrize("lens", [None, [5, 0, 3]])
def test_reference_gradients_against_differences(kind, lens):
    x = ref.make(3, 6, 4, torch.float64, 1, resets=0)
    x["log_w"], x["state_in"], x["dstate_out"] = (x[n].double() for n in ("log_w", "state_in", "dstate_out"))

    def loss(**kw):
        z = dict(x, **kw)
        out = ref.forward(z["x"], z["log_w"], z["state_in"], lens, kind)
        return float((out["y"][0] * x["dy"]).sum() + (out["state"][0] * x["dstate_out"]).sum())

    got = ref.backward(x["x"], x["log_w"], x["state_in"], lens, x["dy"], x["dstate_out"], kind)
    g = torch.Generator().manual_seed(2)
    for name, grad in (("x", "dx"), ("log_w", "dlog_w"), ("state_in", "dstate_in")):
        way = torch.randn(x[name].shape, generator=g, dtype=torch.float64)
        step = 1e-6
        if name == "log_w":
            way = way * x[name].abs()  # stays below 0
        diff = (loss(**{name: x[name] + step * way}) - loss(**{name: x[name] - step * way})) / (2 * step)
        want = float((got[grad][0] * way).sum())
        # central differences: step^2 of the third derivative, and 2^-53 of the loss over the step
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), (name, diff, want)


def test_reference_of_a_constant_decay():
    w, T = 0.75, 9
    lw = torch.full((1, T, 1), w, dtype=torch.float64).log()
    one = torch.ones(1, T, 1, dtype=torch.float64)
    for kind, s in (("plain", 1.0), ("mix", 1 - w), ("norm", (1 - w * w) ** 0.5)):
        y = ref.forward(one, lw, None, None, kind)["y"][0][0, :, 0]
        want = s * (1 - w ** torch.arange(1, T + 1, dtype=torch.float64)) / (1 - w)
        assert torch.allclose(y, want, rtol=1e-14)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(wkv.LIB_PATH):
        pytest.skip("HIP library not built")
    return wkv.lib()


def ptrs(n):
    return [BASE + i * GAP for i in range(n)]


def prefill(L, p=None, B=2, T=3, D=64, dtype=BF16, mode=0):
    # x, log_w, state_in, lens, y, state_out
    return L.rwkv7_gscan_prefill(*(ptrs(6) if p is None else p), B, T, D, dtype, mode, None)


def step(L, p=None, B=2, T=1, D=64, dtype=BF16, mode=0):
    # x, log_w, state_in, y, state_out
    return L.rwkv7_gscan_step(*(ptrs(5) if p is None else p), B, T, D, dtype, mode, None)


def backward(L, p=None, B=2, T=3, D=64, dtype=BF16, mode=0):
    # x, log_w, state_in, lens, dy, dstate_out, dx, dlog_w, dstate_in
    return L.rwkv7_gscan_backward(*(ptrs(9) if p is None else p), B, T, D, dtype, mode, None)


CALLS = [(prefill, 6, (2, 3, 5), (4, 5)), (step, 5, (2, 4), (3, 4)), (backward, 9, (2, 3, 5, 8), (6, 7, 8))]


@pytest.mark.parametrize("call", [prefill, step, backward])
def test_bad_kinds_and_sizes(L, call):
    assert call(L, dtype=2) == E_DTYPE and call(L, dtype=-1) == E_DTYPE
    assert call(L, mode=3) == E_MODE and call(L, mode=-1) == E_MODE
    assert "input scale" in wkv.rwkv7_wkv_strerror(E_MODE)
    for bad in (dict(B=-1), dict(T=-1), dict(D=-1), dict(D=(1 << 20) + 1, B=1), dict(B=1 << 22, D=64), dict(B=1 << 62, D=64)):
        assert call(L, **bad) == E_SHAPE, bad
    if call is step:
        assert step(L, T=0) == E_SHAPE and step(L, T=2) == E_SHAPE
    else:
        for bad in (dict(T=1 << 36, B=1, D=1), dict(T=1 << 30, B=1, D=4096), dict(T=(1 << 63) - 1, D=2)):
            assert call(L, **bad) == E_SHAPE, bad


@pytest.mark.parametrize("call,n,optional,outs", CALLS)
def test_null_and_misaligned_pointers(L, call, n, optional, outs):
    for i in range(n):
        p = ptrs(n)
        p[i] += 8
        assert call(L, p) == E_ALIGN, i
        if i not in optional:
            p = ptrs(n)
            p[i] = None
            assert call(L, p) == E_NULL, i


@pytest.mark.parametrize("call,n,optional,outs", CALLS)
def test_overlaps(L, call, n, optional, outs):
    in_place = {prefill: (5, 2), step: (4, 2), backward: (8, 5)}[call]
    for out in outs:
        for i in range(n):
            if i != out and {i, out} != set(in_place):
                p = ptrs(n)
                p[out] = p[i]
                assert call(L, p) == E_ALIAS, (out, i)
    p = ptrs(n)  # in place is exactly the same address, not a shifted one
    p[in_place[0]] = p[in_place[1]] + 16
    assert call(L, p) == E_ALIAS


def test_empty_work_needs_no_device(L):
    assert prefill(L, B=0) == OK and prefill(L, D=0) == OK and prefill(L, [None] * 6, B=0) == OK
    assert step(L, B=0) == OK and step(L, [None] * 5, D=0) == OK
    assert backward(L, B=0) == OK and backward(L, [None] * 9, D=0) == OK
    assert prefill(L, [None] * 6, T=0) == OK and backward(L, [None] * 9, T=0) == OK


@pytest.fixture
def no_library(monkeypatch):
    def forbidden():
        raise AssertionError("the library was called before the arguments were checked")
    monkeypatch.setattr(wkv, "lib", forbidden)


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses(no_library):
    half = torch.bfloat16
    good = dict(x=z(2, 5, 64, dtype=half), log_w=z(2, 5, 64), state_in=z(2, 64), lens=z(2, dtype=torch.int32),
                y=z(2, 5, 64, dtype=half), state_out=None)
    for name, value, match in (("x", z(2, 5, 64, dtype=torch.float16), "x has dtype"), ("x", z(2, 64), "x must be"),
                               ("x", z(2, 5, 128)[..., ::2], "x must be"), ("log_w", z(2, 5), "log_w has shape"),
                               ("log_w", z(2, 5, 64, dtype=half), "log_w has dtype"), ("log_w", None, "log_w is required"),
                               ("state_in", z(2, 64, dtype=half), "state_in has dtype"), ("state_in", z(64), "state_in has shape"),
                               ("lens", z(2, dtype=torch.int64), "lens has dtype"), ("lens", z(3, dtype=torch.int32), "lens has shape"),
                               ("y", z(2, 5, 64), "y has dtype"), ("y", None, "y is required"),
                               ("state_out", z(2, 1, 64), "state_out has shape")):
        with pytest.raises(ValueError, match=match):
            wkv.rwkv7_gscan_prefill(**dict(good, **{name: value}))
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_gscan_prefill(**good)
    with pytest.raises(ValueError, match="must be a"):
        wkv.gscan(z(4, 64), z(4, 64))
    one = dict(x=z(2, 1, 64), log_w=z(2, 1, 64), state_in=z(2, 64), y=z(2, 1, 64), state_out=z(2, 64))
    for name, value, match in (("y", z(2, 64), "y has shape"), ("state_out", z(2, 63), "state_out has shape")):
        with pytest.raises(ValueError, match=match):
            wkv.rwkv7_gscan_step(**dict(one, **{name: value}))
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_gscan_step(**one)
    grad = dict(x=z(2, 5, 64), log_w=z(2, 5, 64), state_in=None, lens=None, dy=z(2, 5, 64), dstate_out=None, dx=z(2, 5, 64),
                dlog_w=z(2, 5, 64), dstate_in=z(2, 64))
    for name, value, match in (("dy", z(2, 5, 64, dtype=half), "dy has dtype"), ("dx", None, "dx is required"),
                               ("dlog_w", z(2, 5), "dlog_w has shape"), ("dstate_out", z(2, 63), "dstate_out has shape"),
                               ("dstate_in", z(64), "dstate_in has shape")):
        with pytest.raises(ValueError, match=match):
            wkv.rwkv7_gscan_backward(**dict(grad, **{name: value}))
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_gscan_backward(**grad)
