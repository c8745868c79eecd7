"""The layer norm without a GPU: the float64 implementation that the GPU tests compare with (against
differences), and the refusals of the C ABI and of the binding (no HIP call is made)."""
import os

import pytest
import torch

from linear_rnn_amd import wkv
from tests import layernorm_ref as ref

F32, BF16 = wkv.RWKV7_DTYPE_F32, wkv.RWKV7_DTYPE_BF16
OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_ALIAS = 0, -1, -2, -4, -5, -6
BASE, GAP = 1 << 40, 1 << 34


@pytest.mark.parametrize("G", [1, 3])
def test_reference_gradients_against_differences(G):
    x = ref.make(4, 12, G, torch.float64, torch.float64, 1)
    _, mean, rstd = ref.forward(x["x"], x["weight"], x["bias"], G, 1e-3)
    got = ref.backward(x["x"], x["weight"], mean, rstd, x["dy"], G)

    def loss(**kw):
        z = dict(x, **kw)
        return float((ref.forward(z["x"], z["weight"], z["bias"], G, 1e-3)[0] * x["dy"]).sum())

    g = torch.Generator().manual_seed(2)
    for name, grad in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias")):
        base = x[name].double()
        way, h = torch.randn(base.shape, generator=g, dtype=torch.float64), 1e-5
        diff = (loss(**{name: base + h * way}) - loss(**{name: base - h * way})) / (2 * h)
        want = float((got[grad] * way).sum())
        # central differences: h^2 of the third derivative, and 2^-53 of the loss over h
        assert abs(diff - want) <= 1e-6 * max(1.0, abs(want)), (name, diff, want)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(wkv.LIB_PATH):
        pytest.skip("HIP library not built")
    return wkv.lib()


def ptrs(n):
    return [BASE + i * GAP for i in range(n)]


def forward(L, p=None, M=4, D=128, G=2, eps=1e-5, xd=BF16, yd=BF16):
    # x, weight, bias, y, mean, rstd
    return L.rwkv7_layernorm_forward(*(ptrs(6) if p is None else p), M, D, G, eps, xd, yd, None)


def backward(L, p=None, M=4, D=128, G=2, xd=BF16, yd=BF16):
    # x, weight, mean, rstd, dy, dx, dweight, dbias
    return L.rwkv7_layernorm_backward(*(ptrs(8) if p is None else p), M, D, G, xd, yd, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_bad_kinds_and_sizes(L, call):
    assert call(L, xd=2) == E_DTYPE and call(L, yd=-1) == E_DTYPE
    for bad in (dict(M=-1), dict(D=-64), dict(G=0), dict(G=-1), dict(G=3), dict(D=(1 << 24) + 64, G=1), dict(M=1 << 50),
                dict(M=1 << 60, D=64, G=1)):
        assert call(L, **bad) == E_SHAPE, bad
    for eps in (-1e-5, float("nan"), float("inf")):
        assert forward(L, eps=eps) == E_SHAPE


@pytest.mark.parametrize("call,n,optional", [(forward, 6, (1, 2, 4, 5)), (backward, 8, (1, 6, 7))])
def test_null_and_misaligned_pointers(L, call, n, optional):
    for i in range(n):
        p = ptrs(n)
        p[i] += 4
        assert call(L, p) == E_ALIGN, i
        if i not in optional:
            p = ptrs(n)
            p[i] = None
            assert call(L, p) == E_NULL, i


@pytest.mark.parametrize("call,n,outs", [(forward, 6, (3, 4, 5)), (backward, 8, (5, 6, 7))])
def test_overlaps(L, call, n, outs):
    for out in outs:
        for i in range(n):
            if i == out:
                continue
            p = ptrs(n)
            p[out] = p[i]
            assert call(L, p) == E_ALIAS, (out, i)


def test_empty_work_needs_no_device(L):
    assert forward(L, M=0) == OK and forward(L, D=0, G=1) == OK and forward(L, [None] * 6, M=0) == OK
    assert backward(L, D=0, G=1) == OK
    p = ptrs(8)
    p[6] = p[7] = None  # no rows and no sums over them
    assert backward(L, p, M=0) == OK


@pytest.fixture
def no_library(monkeypatch):
    def forbidden():
        raise AssertionError("the library was called before the arguments were checked")
    monkeypatch.setattr(wkv, "lib", forbidden)


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses(no_library):
    good = dict(x=z(3, 5, 64), weight=z(64), bias=z(64), y=z(3, 5, 64, dtype=torch.bfloat16), mean=z(3, 5, 4),
                rstd=z(3, 5, 4), groups=4)
    for name, value, match in (("x", z(3, 5, 64, dtype=torch.float16), "x has dtype"), ("x", z(3, 5, 128)[..., ::2], "x must be"),
                               ("groups", 5, "divisor"), ("groups", 0, "divisor"), ("weight", z(63), "weight has shape"),
                               ("bias", z(64, dtype=torch.bfloat16), "bias has dtype"), ("y", z(15, 64), "y has shape"),
                               ("y", None, "y is required"), ("mean", z(3, 5), "mean has shape"),
                               ("rstd", z(3, 5, 1), "rstd has shape")):
        with pytest.raises(ValueError, match=match):
            wkv.rwkv7_layernorm_forward(**dict(good, **{name: value}))
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_layernorm_forward(**good)
    with pytest.raises(ValueError, match="x must be"):
        wkv.rwkv7_layernorm_forward(**dict(good, x=z()))

    good = dict(x=z(3, 64), weight=None, mean=z(3, 1), rstd=z(3, 1), dy=z(3, 64, dtype=torch.bfloat16), dx=z(3, 64),
                dweight=z(64), dbias=None)
    for name, value, match in (("mean", None, "mean is required"), ("rstd", z(3, 2), "rstd has shape"), ("dy", z(64), "dy has shape"),
                               ("dx", z(3, 64, dtype=torch.bfloat16), "dx has dtype"), ("dweight", z(65), "dweight has shape"),
                               ("dbias", z(128)[::2], "dbias must be contiguous")):
        with pytest.raises(ValueError, match=match):
            wkv.rwkv7_layernorm_backward(**dict(good, **{name: value}))
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_layernorm_backward(**good)
