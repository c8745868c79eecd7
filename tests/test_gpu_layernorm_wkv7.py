"""A time-mix layer's recurrence with ln_x in training: wkv7, the norm of its heads, and back through the norm's
gradients into the recurrence's. Each operator is held to its own float64 values on the inputs that it got."""
import numpy as np
import pytest

import oracle
from linear_rnn_amd import wkv
from linear_rnn_amd.inputs import CONFIGS, make_cotangents, make_inputs
from tests import layernorm_ref
from tests.gpu_util import TOL_BF16, TOL_F32, rel, say, to_dev

pytestmark = pytest.mark.gpu
GRADS = ("dr", "dw", "dk", "dv", "da", "db", "dstate_in")


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    oracle.build(force=False)
    return t


def chain(torch, d, w, b, do, ds, H, stream=None):
    y, s = wkv.wkv7(*(d[n] for n in "rwkvab"), state_in=d["state_in"], stream=stream)
    rows = y.view(*y.shape[:2], H * 64)
    o, mean, rstd = wkv.layernorm(rows, w, b, groups=H, eps=oracle.GROUP_NORM_EPS, stream=stream)
    n = wkv.layernorm_backward(rows, w, mean, rstd, do, groups=H, stream=stream)
    g = wkv.wkv7_backward(*(d[n] for n in "rwkvab"), n["dx"].view(y.shape), d["state_in"], ds, stream=stream)
    return dict(g, y=y, s=s, o=o, mean=mean, rstd=rstd, dx=n["dx"], dweight=n["dweight"], dbias=n["dbias"])


@pytest.mark.parametrize("name,tol", [("tiny-prefill-f32", TOL_F32), ("L12-D768-prefill", TOL_BF16)])
@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (2, 65, 3), (3, 200, 5)])
def test_recurrence_norm_and_both_gradients(torch, B, T, H, name, tol):
    say("wkv7 with ln_x and back", name, B, T, H)
    x = make_inputs(CONFIGS[name], B=B, T=T, H=H, seed=900 + T, with_state=True)
    ct = make_cotangents(B, T, H, seed=T + 3)
    d = to_dev(x)
    g = torch.Generator().manual_seed(T)
    w, b = 1 + 0.2 * torch.randn(H * 64, generator=g), 0.2 * torch.randn(H * 64, generator=g)
    do = torch.from_numpy(ct["dy"]).view(B, T, H * 64)
    ds = torch.from_numpy(ct["dstate_out"])
    args = (d, w.cuda(), b.cuda(), do.cuda(), ds.cuda(), H)
    got = chain(torch, *args)
    torch.cuda.synchronize()
    yr, sr = oracle.wkv7(*(x[n] for n in "rwkvab"), state_in=x["state_in"])
    assert rel(got["y"].cpu().numpy(), yr) <= tol and rel(got["s"].cpu().numpy(), sr) <= tol
    flat, flat_do = got["y"].cpu().view(B * T, H * 64), do.reshape(B * T, -1)
    eps = oracle.GROUP_NORM_EPS
    want, lim = layernorm_ref.forward(flat, w, b, H, eps), layernorm_ref.forward_limits(flat, w, b, H, eps, torch.float32)
    layernorm_ref.check("o", got["o"].reshape(B * T, -1), want[0], lim[0])
    assert rel(got["o"].cpu().numpy().reshape(B, T, H, 64),
               oracle.group_norm(got["y"].cpu().numpy(), w.numpy(), b.numpy())) <= TOL_F32
    m, r = got["mean"].cpu().view(B * T, H), got["rstd"].cpu().view(B * T, H)
    want, lim = layernorm_ref.backward(flat, w, m, r, flat_do, H), layernorm_ref.backward_limits(flat, w, m, r, flat_do, H)
    layernorm_ref.check("dx", got["dx"].reshape(B * T, -1), want["dx"], lim["dx"])
    for n in ("dweight", "dbias"):
        layernorm_ref.check(n, got[n], want[n], lim[n])
    dy = np.ascontiguousarray(got["dx"].cpu().numpy().reshape(B, T, H, 64))
    gr = oracle.wkv7_backward(*(x[n] for n in "rwkvab"), dy, state_in=x["state_in"], dstate_out=ct["dstate_out"])
    e = {n: rel(got[n].cpu().numpy(), gr[n]) for n in GRADS}
    assert max(e.values()) <= tol, e


def test_captured_with_eager_calls_between(torch):
    say("wkv7 with ln_x and back, in a graph")
    B, T, H = 2, 130, 3
    x = make_inputs(CONFIGS["L12-D768-prefill"], B=B, T=T, H=H, seed=950, with_state=True)
    ct = make_cotangents(B, T, H, seed=7)
    d = to_dev(x)
    w, b = (torch.rand(H * 64, device="cuda") + 0.5 for _ in range(2))
    args = (d, w, b, torch.from_numpy(ct["dy"]).cuda().view(B, T, H * 64), torch.from_numpy(ct["dstate_out"]).cuda(), H)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = chain(torch, *args, stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        held = chain(torch, *args, stream=st)
    for step in range(4):
        args[3].normal_()
        for t in held.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = chain(torch, *args, stream=st)
        st.synchronize()
        assert all(torch.equal(held[n], eager[n]) for n in held), step
        assert not torch.equal(held["dr"], first["dr"])
