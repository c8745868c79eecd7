"""The linear attention without a GPU: the float64 implementation that the GPU tests compare with
(against differences), and the refusals of the C ABI and of the binding (no HIP call is made)."""
import os

import pytest
import torch

from linear_rnn_amd import wkv
from tests import linattn_ref as ref

F32, BF16 = wkv.RWKV7_DTYPE_F32, wkv.RWKV7_DTYPE_BF16
HEAD, TOKEN = wkv.RWKV7_DECAY_HEAD, wkv.RWKV7_DECAY_TOKEN
OK, E_NULL, E_SHAPE, E_HEAD, E_DTYPE, E_ALIGN, E_ALIAS, E_DECAY = 0, -1, -2, -3, -4, -5, -6, -10
BASE, GAP = 1 << 40, 1 << 34


# ---- the float64 implementation

@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("lens", [None, [3, 6]])
def test_reference_gradients_against_differences(decay, lens):
    x = ref.make(2, 6, 2, torch.float64, decay, seed=1)
    x["log_w"] = x["log_w"].double()
    x["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    grads, _ = ref.backward(x)

    def loss(z):
        y, s, _, _ = ref.forward(z)
        live = torch.ones(2, 6, dtype=torch.bool) if lens is None else \
            torch.arange(6)[None, :] < x["lens"][:, None]
        return float((y * torch.where(live[:, :, None, None], x["dy"], 0.0)).sum() + (s * x["dstate_out"]).sum())

    g = torch.Generator().manual_seed(2)
    for name, grad in (("r", "dr"), ("k", "dk"), ("v", "dv"), ("log_w", "dlog_w"), ("state_in", "dstate_in")):
        x[name] = x[name].double()
        way = torch.randn(x[name].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        diff = (loss(dict(x, **{name: x[name] + h * way})) - loss(dict(x, **{name: x[name] - h * way}))) / (2 * h)
        want = float((grads[grad] * way).sum())
        # central differences: h^2 of the third derivative, and 2^-53 of the loss over h
        assert abs(diff - want) <= 1e-6 * max(1.0, abs(want)), (name, diff, want)


# ---- refusals of the C ABI

@pytest.fixture(scope="module")
def L():
    if not os.path.exists(wkv.LIB_PATH):
        pytest.skip("HIP library not built")
    return wkv.lib()


def ptrs(n):
    return [BASE + i * GAP for i in range(n)]


def prefill(L, p=None, B=2, T=3, H=4, N=64, dtype=BF16, decay=TOKEN):
    # r, log_w, k, v, state_in, lens, y, state_out
    return L.rwkv7_linattn_prefill(*(ptrs(8) if p is None else p), B, T, H, N, dtype, decay, None)


def step(L, p=None, B=2, T=1, H=4, N=64, dtype=BF16, decay=TOKEN):
    # r, log_w, k, v, state_in, y, state_out
    return L.rwkv7_linattn_step(*(ptrs(7) if p is None else p), B, T, H, N, dtype, decay, None)


@pytest.mark.parametrize("call", [prefill, step])
def test_bad_kinds_and_sizes(L, call):
    assert call(L, dtype=2) == E_DTYPE
    assert call(L, decay=2) == E_DECAY and call(L, decay=-1) == E_DECAY
    assert "decay" in wkv.rwkv7_wkv_strerror(E_DECAY)
    for N in (0, 32, 65, 128):
        assert call(L, N=N) == E_HEAD
    for bad in (dict(B=-1), dict(T=-1), dict(H=-4), dict(B=1 << 22, H=4), dict(H=(1 << 18) + 1, B=1),
                dict(B=1 << 62, H=4), dict(T=1 << 60)):
        assert call(L, **bad) == E_SHAPE, bad
    assert step(L, T=2) == E_SHAPE and step(L, T=0) == E_SHAPE


def test_most_heads(L):
    p = ptrs(8)
    p[4] = p[7] = None  # no state, so that a call without tokens has nothing to do
    assert prefill(L, p, B=1 << 21, T=0, H=1) == 0
    assert prefill(L, p, B=(1 << 21) + 1, T=0, H=1) == E_SHAPE


@pytest.mark.parametrize("call,n,optional", [(prefill, 8, (4, 5, 7)), (step, 7, (4, 6))])
def test_null_and_misaligned_pointers(L, call, n, optional):
    for i in range(n):
        p = ptrs(n)
        p[i] += 4
        assert call(L, p) == E_ALIGN, i
        if i not in optional:
            p = ptrs(n)
            p[i] = None
            assert call(L, p) == E_NULL, i


@pytest.mark.parametrize("call,n,y,s", [(prefill, 8, 6, 7), (step, 7, 5, 6)])
def test_overlaps(L, call, n, y, s):
    for out in (y, s):
        for i in range(n):
            if i == out:
                continue
            p = ptrs(n)
            p[out] = p[i] + (1024 if i == 4 and out == s else 0)  # state_out may be state_in, but not part of it
            if i in (1, 5) and n == 8:  # small inputs: an output that starts before and ends behind them
                p[out] = p[i] - 16
            assert call(L, p) == E_ALIAS, (out, i)


def backward(L, p=None, B=2, T=3, H=4, N=64, dtype=BF16, decay=TOKEN):
    # r, log_w, k, v, state_in, lens, dy, dstate_out, dr, dlog_w, dk, dv, dstate_in
    return L.rwkv7_linattn_backward(*(ptrs(13) if p is None else p), B, T, H, N, dtype, decay, None)


def test_backward_refusals(L):
    assert backward(L, dtype=2) == E_DTYPE and backward(L, decay=2) == E_DECAY and backward(L, N=128) == E_HEAD
    for bad in (dict(B=-1), dict(T=-1), dict(H=-4), dict(B=1 << 22, H=4), dict(H=(1 << 18) + 1, B=1), dict(T=1 << 60)):
        assert backward(L, **bad) == E_SHAPE, bad
    for i in range(13):
        p = ptrs(13)
        p[i] += 4
        assert backward(L, p) == E_ALIGN, i
        if i not in (4, 5, 7, 12):
            p = ptrs(13)
            p[i] = None
            assert backward(L, p) == E_NULL, i
    for out in (8, 9, 10, 11, 12):
        for i in range(13):
            if i == out:
                continue
            p = ptrs(13)
            p[out] = p[i] + (1024 if i == 7 and out == 12 else 0)  # dstate_in may be dstate_out, but not part of it
            assert backward(L, p) == E_ALIAS, (out, i)


def test_empty_work_needs_no_device(L):
    assert prefill(L, B=0) == OK and prefill(L, H=0) == OK and step(L, B=0) == OK
    p = ptrs(8)
    p[7] = None  # no tokens and no state_out
    assert prefill(L, p, T=0) == OK
    p[7] = p[4]  # no tokens, the state in place
    assert prefill(L, p, T=0) == OK
    assert prefill(L, [None] * 8, B=0) == OK
    assert backward(L, B=0) == OK and backward(L, H=0) == OK
    p = ptrs(13)
    p[12] = p[7]
    assert backward(L, p, T=0) == OK


# ---- refusals of the binding

B, T, H, N = 2, 5, 3, 64


@pytest.fixture
def no_library(monkeypatch):
    def forbidden():
        raise AssertionError("the library was called before the arguments were checked")
    monkeypatch.setattr(wkv, "lib", forbidden)


def good(T=T):
    x = [torch.zeros((B, T, H, N), dtype=torch.bfloat16) for _ in range(3)]
    return {"r": x[0], "log_w": torch.zeros((B, T, H)), "k": x[1], "v": x[2], "state_in": torch.zeros((B, H, N, N)),
            "lens": torch.zeros((B,), dtype=torch.int32), "y": torch.zeros((B, T, H, N), dtype=torch.bfloat16),
            "state_out": torch.zeros((B, H, N, N))}


BAD = [("r", torch.zeros((B, T, H * N), dtype=torch.bfloat16), "r must be"),
       ("r", torch.zeros((B, T, H, N), dtype=torch.float16), "r has dtype"),
       ("log_w", torch.zeros((B, H)), "log_w has shape"),
       ("log_w", torch.zeros((H + 1,)), "log_w has shape"),
       ("log_w", torch.zeros((B, T, H), dtype=torch.bfloat16), "log_w has dtype"),
       ("log_w", torch.zeros((B, T, 2 * H))[..., ::2], "log_w must be contiguous"),
       ("k", torch.zeros((B, T, H, N)), "k has dtype"),
       ("v", torch.zeros((B, T - 1, H, N), dtype=torch.bfloat16), "v has shape"),
       ("v", torch.zeros((B, T, H, 2 * N), dtype=torch.bfloat16)[..., ::2], "v must be contiguous"),
       ("state_in", torch.zeros((B, H, N, N), dtype=torch.bfloat16), "state_in has dtype"),
       ("lens", torch.zeros((B,), dtype=torch.int64), "lens has dtype"),
       ("lens", torch.zeros((B + 1,), dtype=torch.int32), "lens has shape"),
       ("y", torch.zeros((B, T, H, N)), "y has dtype"),
       ("y", None, "y is required"),
       ("state_out", torch.zeros((B, H, N)), "state_out has shape")]


@pytest.mark.parametrize("name,value,match", BAD)
def test_binding_refuses(no_library, name, value, match):
    a = dict(good(), **{name: value})
    with pytest.raises(ValueError, match=match):
        wkv.rwkv7_linattn_prefill(**a)
    if name != "lens":
        del a["lens"]
        with pytest.raises(ValueError, match=match):
            wkv.rwkv7_linattn_step(**a)


@pytest.mark.parametrize("name,value,match", [b for b in BAD if b[0] not in ("y", "state_out")] + [
    ("dy", None, "dy is required"), ("dy", torch.zeros((B, T, H, N)), "dy has dtype"),
    ("dr", torch.zeros((B, T, H, N)), "dr has dtype"), ("dk", torch.zeros((B, T, H), dtype=torch.bfloat16), "dk has shape"),
    ("dv", None, "dv is required"), ("dlog_w", torch.zeros((H,)), "dlog_w has shape"),
    ("dlog_w", torch.zeros((B, T, H), dtype=torch.bfloat16), "dlog_w has dtype"),
    ("dstate_out", torch.zeros((H, N, N)), "dstate_out has shape"), ("dstate_in", torch.zeros((H, N, N)), "dstate_in has")])
def test_binding_refuses_backward(no_library, name, value, match):
    a = good()
    a = {n: a[n] for n in ("r", "log_w", "k", "v", "state_in", "lens")}
    a.update({n: torch.zeros((B, T, H, N), dtype=torch.bfloat16) for n in ("dy", "dr", "dk", "dv")},
             dlog_w=torch.zeros((B, T, H)), dstate_out=None, dstate_in=None)
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_linattn_backward(**a)
    with pytest.raises(ValueError, match=match):
        wkv.rwkv7_linattn_backward(**dict(a, **{name: value}))


def test_binding_refuses_host_tensors(no_library):
    with pytest.raises(ValueError, match="must be on a HIP device"):
        wkv.rwkv7_linattn_prefill(**good())
    with pytest.raises(TypeError, match="log_w must be a torch.Tensor"):
        wkv.rwkv7_linattn_prefill(**dict(good(), log_w=0.5))
