"""A layer of a gated linear recurrent model, there and back: norm, gated linear recurrence, norm, gated linear unit, and
their gradients, with a generated token behind the prompt. Each operator is held to its own float64 values on the inputs
that it got, and the whole to float64 differentiation."""
import pytest

from linear_rnn_amd import wkv
from tests import glu_ref, gscan_ref, layernorm_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
KIND, ACT, EPS = wkv.RWKV7_INPUT_NORM, wkv.RWKV7_ACT_SILU, 1e-5


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def make(torch, B, T, D, F, dtype, seed, lens):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, scale=1.0):
        return torch.randn(shape, generator=g) * scale

    d = {"x": n(B, T, D), "w1": 1 + n(D, scale=0.2), "b1": n(D, scale=0.2), "w2": 1 + n(D, scale=0.2), "b2": n(D, scale=0.2),
         "log_w": -torch.exp(torch.rand(B, T, D, generator=g) * 5 - 5), "state": n(B, D), "da": n(B, T, F).to(dtype),
         "ds": n(B, D), "wg": n(D, F, scale=D ** -0.5).to(dtype), "wu": n(D, F, scale=D ** -0.5).to(dtype)}
    if lens is not None:
        d["lens"] = torch.tensor(lens, dtype=torch.int32)
    return d


def layer(d, dtype, stream=None):
    o = {}
    o["n1"], o["m1"], o["r1"] = wkv.layernorm(d["x"], d["w1"], d["b1"], eps=EPS, out_dtype=dtype, stream=stream)
    o["y"], o["s"] = wkv.gscan(o["n1"], d["log_w"], d["state"], lens=d.get("lens"), input=KIND, stream=stream)
    o["n2"], o["m2"], o["r2"] = wkv.layernorm(o["y"], d["w2"], d["b2"], eps=EPS, stream=stream)
    o["h"], o["gate"], o["up"] = wkv.glu(o["n2"], d["wg"], d["wu"], act=ACT, want_pre=True, stream=stream)
    g = wkv.glu_backward(o["n2"], d["wg"], d["wu"], o["gate"], o["up"], d["da"], act=ACT, stream=stream)
    o["dn2"], o["dwg"], o["dwu"] = g["dx"], g["dw_gate"], g["dw_up"]
    n = wkv.layernorm_backward(o["y"], d["w2"], o["m2"], o["r2"], o["dn2"], stream=stream)
    o["dy"], o["dw2"], o["db2"] = n["dx"], n["dweight"], n["dbias"]
    q = wkv.gscan_backward(o["n1"], d["log_w"], o["dy"], d["state"], lens=d.get("lens"), dstate_out=d["ds"], input=KIND,
                           stream=stream)
    o["dn1"], o["dlog_w"], o["dstate"] = q["dx"], q["dlog_w"], q["dstate_in"]
    n = wkv.layernorm_backward(d["x"], d["w1"], o["m1"], o["r1"], o["dn1"], stream=stream)
    o["dx"], o["dw1"], o["db1"] = n["dx"], n["dweight"], n["dbias"]
    return o


CASES = [(1, 1, 64, 128, None), (2, 200, 72, 96, None), (3, 300, 40, 56, [300, 0, 17]), (2, 1500, 64, 100, None)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,T,D,F,lens", CASES)
def test_each_operator_on_what_it_got(torch, B, T, D, F, lens, dtype):
    dt = getattr(torch, dtype)
    say("gated layer", B, T, D, F, dtype)
    c = make(torch, B, T, D, F, dt, T, lens)
    o = layer({n: t.cuda() for n, t in c.items()}, dt)
    o = {n: t.cpu() for n, t in o.items()}
    rows = B * T

    def norm(x, w, b, out, dy, mean, rstd, dx, dw, db, y_dtype):
        x, out, dy, dx = (t.reshape(rows, D) for t in (x, out, dy, dx))
        mean, rstd = mean.view(rows, 1), rstd.view(rows, 1)
        want, lim = layernorm_ref.forward(x, w, b, 1, EPS), layernorm_ref.forward_limits(x, w, b, 1, EPS, y_dtype)
        layernorm_ref.check("norm", out, want[0], lim[0])
        want, lim = layernorm_ref.backward(x, w, mean, rstd, dy, 1), layernorm_ref.backward_limits(x, w, mean, rstd, dy, 1)
        for name, got in (("dx", dx), ("dweight", dw), ("dbias", db)):
            layernorm_ref.check(name, got, want[name], lim[name])

    norm(c["x"], c["w1"], c["b1"], o["n1"], o["dn1"], o["m1"], o["r1"], o["dx"], o["dw1"], o["db1"], dt)
    norm(o["y"], c["w2"], c["b2"], o["n2"], o["dn2"], o["m2"], o["r2"], o["dy"], o["dw2"], o["db2"], dt)
    want = gscan_ref.forward(o["n1"], c["log_w"], c["state"], lens, "norm")
    gscan_ref.check("y", o["y"], want["y"])
    gscan_ref.check("s", o["s"], want["state"])
    want = gscan_ref.backward(o["n1"], c["log_w"], c["state"], lens, o["dy"], c["ds"], "norm")
    for name, got in (("dx", "dn1"), ("dlog_w", "dlog_w"), ("dstate_in", "dstate")):
        gscan_ref.check(name, o[got], want[name])
    flat = {n: o[n].reshape(rows, -1) for n in ("n2", "gate", "up", "h", "dn2")}
    want = glu_ref.forward(flat["n2"], c["wg"], c["wu"], "silu")
    for name in ("h", "gate", "up"):
        glu_ref.check(name, flat[name], want[name])
    want = glu_ref.backward(flat["n2"], c["wg"], c["wu"], flat["gate"], flat["up"], c["da"].reshape(rows, F), "silu")
    for name, got in (("dx", flat["dn2"]), ("dw_gate", o["dwg"]), ("dw_up", o["dwu"])):
        glu_ref.check(name, got, want[name])


@pytest.mark.parametrize("B,T,D,F,lens", CASES[1:])
def test_the_whole_against_differentiation(torch, B, T, D, F, lens):
    """float32. Eight operators one behind the other, each at most 64 half steps of float32 off in 2-norm, which the norms
    (weights and spreads within a factor of two) and the products may double: 8 * 64 * 2 * 2^-24 = 6e-5."""
    c = make(torch, B, T, D, F, torch.float32, T + 1, lens)
    o = layer({n: t.cuda() for n, t in c.items()}, torch.float32)
    v = {n: t.double().requires_grad_(t.dtype == torch.float32) for n, t in c.items() if n != "lens"}
    keep = torch.ones(B, T, dtype=torch.bool) if lens is None else torch.arange(T)[None] < torch.tensor(lens)[:, None]

    def norm(x, w, b):
        return torch.nn.functional.layer_norm(x, (D,), w, b, EPS)

    n1, h, ys = norm(v["x"], v["w1"], v["b1"]), v["state"], []
    scale = torch.sqrt(-torch.expm1(2 * v["log_w"]))
    for t in range(T):
        k = keep[:, t, None]
        h = torch.where(k, v["log_w"][:, t].exp() * h + scale[:, t] * n1[:, t], h)
        ys.append(torch.where(k, h, torch.zeros_like(h)))
    n2 = norm(torch.stack(ys, 1), v["w2"], v["b2"])
    a = torch.nn.functional.silu(n2 @ v["wg"]) * (n2 @ v["wu"])
    names = {"x": "dx", "w1": "dw1", "b1": "db1", "w2": "dw2", "b2": "db2", "log_w": "dlog_w", "state": "dstate", "wg": "dwg",
             "wu": "dwu"}
    grads = torch.autograd.grad((a * v["da"].detach()).sum() + (h * v["ds"].detach()).sum(), [v[n] for n in names])
    for got, want in [(o["h"], a), (o["s"], h)] + [(o[names[n]], g) for n, g in zip(names, grads)]:
        want = want.detach()
        far = float((got.cpu().double() - want).norm() / want.norm())
        assert far <= 6e-5, (far, tuple(want.shape))


def test_captured_and_replayed(torch):
    c = {n: t.cuda() for n, t in make(torch, 2, 1500, 72, 96, torch.bfloat16, 5, None).items()}
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = layer(c, torch.bfloat16, stream)
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = layer(c, torch.bfloat16, stream)
    for _ in range(3):
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want)
        layer(c, torch.bfloat16, stream)
        stream.synchronize()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_tokens_behind_a_prompt(torch, dtype):
    """A prompt and then token by token, in place, is the longer prompt: within the two's bounds."""
    B, T, D, more = 3, 260, 72, 5
    dt = getattr(torch, dtype)
    x = gscan_ref.make(B, T + more, D, dt, seed=8, resets=0)
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    part = lambda a, b: (d["x"][:, a:b].contiguous(), d["log_w"][:, a:b].contiguous())
    _, state = wkv.gscan(*part(0, T), d["state_in"], input=KIND)
    want = gscan_ref.forward(x["x"], x["log_w"], x["state_in"], None, "norm")
    y = torch.empty(B, 1, D, dtype=dt, device="cuda")
    for t in range(T, T + more):
        wkv.rwkv7_gscan_step(*part(t, t + 1), state, y, state, input=KIND)
        gscan_ref.check("y", y[:, 0], tuple(w[:, t] for w in want["y"]))
    gscan_ref.check("state", state, want["state"])
