"""The gated linear unit without a GPU: the float64 implementation that the GPU tests compare with (against
differences), and the refusals of the C ABI and of the binding (no HIP call is made)."""
import os

import pytest
import torch

from linear_rnn_amd import wkv
from tests import glu_ref as ref

F32, BF16 = wkv.RWKV7_DTYPE_F32, wkv.RWKV7_DTYPE_BF16
OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_ALIAS, E_MODE = 0, -1, -2, -4, -5, -6, -11
BASE, GAP = 1 << 40, 1 << 36


@pytest.mark.parametrize("kind", ref.ACTS)
def test_reference_gradients_against_differences(kind):
    x = ref.make(5, 6, 4, torch.float64, 1)

    def loss(**kw):
        z = dict(x, **kw)
        return float((ref.forward(z["x"], z["w_gate"], z["w_up"], kind)["h"][0] * x["dh"]).sum())

    out = ref.forward(x["x"], x["w_gate"], x["w_up"], kind)
    got = ref.backward(x["x"], x["w_gate"], x["w_up"], out["gate"][0], out["up"][0], x["dh"], kind)
    g = torch.Generator().manual_seed(2)
    for name, grad in (("x", "dx"), ("w_gate", "dw_gate"), ("w_up", "dw_up")):
        way, h = torch.randn(x[name].shape, generator=g, dtype=torch.float64), 1e-6
        diff = (loss(**{name: x[name] + h * way}) - loss(**{name: x[name] - h * way})) / (2 * h)
        want = float((got[grad][0] * way).sum())
        # central differences: h^2 of the third derivative, and 2^-53 of the loss over h
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), (name, diff, want)


def test_reference_activations():
    g = torch.linspace(-9, 9, 101, dtype=torch.float64)
    for kind, f in (("sigmoid", torch.sigmoid), ("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
                    ("relu2", lambda t: torch.relu(t) ** 2)):
        t = g.clone().requires_grad_(True)
        y = f(t)
        (d,) = torch.autograd.grad(y.sum(), t)
        a, slope, _, _ = ref.act(g, kind)
        assert torch.allclose(a, y.detach(), rtol=1e-12, atol=1e-15) and torch.allclose(slope, d, rtol=1e-12, atol=1e-15), kind


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(wkv.LIB_PATH):
        pytest.skip("HIP library not built")
    return wkv.lib()


def ptrs(n):
    return [BASE + i * GAP for i in range(n)]


def forward(L, p=None, M=4, D=64, F=128, dtype=BF16, act=1):
    # x, w_gate, w_up, h, gate, up
    return L.rwkv7_glu_forward(*(ptrs(6) if p is None else p), M, D, F, dtype, act, None)


def backward(L, p=None, M=4, D=64, F=128, dtype=BF16, act=1):
    # x, w_gate, w_up, gate, up, dh, dx, dw_gate, dw_up
    return L.rwkv7_glu_backward(*(ptrs(9) if p is None else p), M, D, F, dtype, act, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_bad_kinds_and_sizes(L, call):
    assert call(L, dtype=2) == E_DTYPE and call(L, dtype=-1) == E_DTYPE
    assert call(L, act=4) == E_MODE and call(L, act=-1) == E_MODE
    assert "activation" in wkv.rwkv7_wkv_strerror(E_MODE)
    for bad in (dict(M=-1), dict(D=0), dict(D=-1), dict(F=-1), dict(M=(1 << 28) + 1), dict(D=(1 << 20) + 1),
                dict(F=(1 << 20) + 1), dict(M=1 << 28, F=1024), dict(M=1 << 28, D=1024), dict(D=1 << 20, F=1 << 20),
                dict(M=1 << 62),
                dict(M=1 << 27, D=129)):
        assert call(L, **bad) == E_SHAPE, bad


@pytest.mark.parametrize("call,n,pairs", [(forward, 6, [(4, 5)]), (backward, 9, [(7, 8)])])
def test_null_and_misaligned_pointers(L, call, n, pairs):
    for i in range(n):
        p = ptrs(n)
        p[i] += 2
        assert call(L, p) == E_ALIGN, i
        p = ptrs(n)
        p[i] = None
        if call is backward and i == 6:
            continue  # dx may be left out
        assert call(L, p) == E_NULL, i  # of a pair, both or neither
    p = [None] * 6 + [None] * 3
    assert backward(L, p, M=4) == E_NULL


@pytest.mark.parametrize("call,n,outs", [(forward, 6, (3, 4, 5)), (backward, 9, (6, 7, 8))])
def test_overlaps(L, call, n, outs):
    for out in outs:
        for i in range(n):
            if i != out:
                p = ptrs(n)
                p[out] = p[i]
                assert call(L, p) == E_ALIAS, (out, i)


def test_empty_work_needs_no_device(L):
    assert forward(L, M=0) == OK and forward(L, F=0) == OK and forward(L, [None] * 6, M=0) == OK
    assert backward(L, [None] * 9, M=0) == OK and backward(L, [None] * 9, F=0) == OK
    assert backward(L, ptrs(6) + [None] * 3) == OK  # nothing asked for


@pytest.fixture
def no_library(monkeypatch):
    def forbidden():
        raise AssertionError("the library was called before the arguments were checked")
    monkeypatch.setattr(wkv, "lib", forbidden)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses(no_library):
    good = dict(x=z(2, 5, 64), w_gate=z(64, 128), w_up=z(64, 128), h=z(2, 5, 128), gate=z(2, 5, 128), up=z(2, 5, 128))
    for name, value, match in (("x", z(2, 5, 64, dtype=torch.float16), "x has dtype"), ("x", z(), "x must be"),
                               ("x", z(2, 5, 128)[..., ::2], "x must be"), ("w_gate", z(64), "w_gate must be"),
                               ("w_gate", z(63, 128), "w_gate has shape"), ("w_gate", z(128, 64).t(), "w_gate must be contiguous"),
                               ("w_up", z(64, 127), "w_up has shape"), ("w_up", z(64, 128, dtype=torch.float32), "w_up has dtype"),
                               ("w_up", None, "w_up is required"), ("h", z(10, 128), "h has shape"), ("h", None, "h is required"),
                               ("gate", z(2, 5, 64), "gate has shape"), ("up", z(2, 5, 128, dtype=torch.float32), "up has dtype")):
        with pytest.raises((ValueError, TypeError), match=match):
            wkv.rwkv7_glu_forward(**dict(good, **{name: value}))
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_glu_forward(**good)
    with pytest.raises(ValueError, match="w_gate has shape"):
        wkv.glu(z(4, 64), z(32, 8), z(32, 8))
    good = dict(x=z(5, 64), w_gate=z(64, 128), w_up=z(64, 128), gate=z(5, 128), up=z(5, 128), dh=z(5, 128), dx=z(5, 64),
                dw_gate=z(64, 128), dw_up=z(64, 128))
    for name, value, match in (("gate", None, "gate is required"), ("dh", z(5, 64), "dh has shape"),
                               ("dx", z(5, 128), "dx has shape"), ("dw_gate", z(128, 64), "dw_gate has shape"),
                               ("dw_up", z(64, 128, dtype=torch.float32), "dw_up has dtype")):
        with pytest.raises(ValueError, match=match):
            wkv.rwkv7_glu_backward(**dict(good, **{name: value}))
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_glu_backward(**good)
