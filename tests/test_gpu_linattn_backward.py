"""GPU parity of the linear attention's gradients against the float64 reverse pass, and of the linear
attention, the norm of its heads and both their gradients together."""
import pytest

from linear_rnn_amd import wkv
from tests import layernorm_ref
from tests import linattn_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f32": "float32"}


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def dev(x):
    return {n: (t.cuda() if t is not None else None) for n, t in x.items()}


def run(d, **kw):
    return wkv.linattn_backward(d["r"], d["log_w"], d["k"], d["v"], d["dy"], state_in=d["state_in"], lens=d["lens"],
                                dstate_out=d["dstate_out"], **kw)


def check_all(torch, x, got):
    want, mag = ref.backward(x)
    B, T, H, _ = x["r"].shape
    bf16 = x["r"].dtype == torch.bfloat16
    for n in ("dr", "dk", "dv"):
        assert got[n].dtype == x["r"].dtype
        ref.check(n, got[n], want[n], mag[n], T, bf16)
    # dlog_w: a state's sums and a gradient's (twice the roundings of one), 2 * 64 * 64 + 64 terms of the product
    # of the two; of one decay for all tokens, their sum besides
    more = 32 * 130 + (32 * (B + T) if x["log_w"].dim() == 1 else 0)
    ref.check("dlog_w", got["dlog_w"], want["dlog_w"], mag["dlog_w"], 2 * T + more, False)
    ref.check("dstate_in", got["dstate_in"], want["dstate_in"], mag["dstate_in"], T, False)


def compare(torch, x, what):
    say("linattn backward", what)
    got = run(dev(x))
    torch.cuda.synchronize()
    check_all(torch, x, got)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 97, 127, 128, 129, 300])
def test_lengths(torch, T, decay, dtype):
    x = ref.make(2, T, 3, getattr(torch, DT[dtype]), decay, seed=10 + T, state=T % 2 == 1)
    compare(torch, x, ("lengths", T, decay, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [256, 515, 1300, 2100])
def test_one_head(torch, T, dtype):
    """One head: segments, their pieces and the blocks inside a piece."""
    x = ref.make(1, T, 1, getattr(torch, DT[dtype]), "token", seed=40 + T, resets=0.01)
    compare(torch, x, ("one head", T, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [128, 515, 1300])
def test_float32_outputs_are_as_good_as_float32(torch, T, dtype):
    """dlog_w and dstate_in are float32 whatever the type of the others. Of inputs with random signs nothing cancels
    but by chance, so the 2-norm of the error is that of the roundings on the way to the value: about 1000 of at most
    2^-24 each (count in linattn_ref), on average 0.4 of that and of a sum that has half its size: 32 * 0.4 * 0.7 * 2^-24,
    under 2^-20 of the value's norm. Products with two bfloat16 pieces (2^-17) would leave more."""
    x = ref.make(2, T, 4, getattr(torch, DT[dtype]), "token", seed=60 + T, state=True)
    say("linattn backward float32 outputs", T, dtype)
    got = run(dev(x))
    want, _ = ref.backward(x)
    for n in ("dlog_w", "dstate_in"):
        err = float((got[n].cpu().to(ref.F64) - want[n]).norm() / want[n].norm())
        assert err <= 2.0 ** -20, (n, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H", [(20, 150, 40), (9, 700, 32), (1, 129, 300), (2, 900, 64)])
def test_many_heads(torch, B, T, H, dtype):
    x = ref.make(B, T, H, getattr(torch, DT[dtype]), "head", seed=50)
    compare(torch, x, ("many heads", B, T, H, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_at_their_ends(torch, dtype):
    base = ref.make(1, 200, 4, getattr(torch, DT[dtype]), "token", seed=60)
    for name, lw in (("none", 0.0), ("all reset", -float("inf")), ("underflow", -90.0), ("faint", -1e-7)):
        compare(torch, dict(base, log_w=torch.full_like(base["log_w"], lw)), ("decay", name, dtype))
    x = dict(base, log_w=base["log_w"].clone())
    for h in range(4):
        x["log_w"][0, h::7 + h, h] = -float("inf")
    got = compare(torch, x, ("decay", "some resets", dtype))
    assert not got["dlog_w"].cpu()[torch.isinf(x["log_w"])].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("T", [300, 1100])
def test_lens(torch, T, decay, dtype):
    lens = [0, 1, 31, 32, 100, 128, 129, T - 1, T, T + 1, -5, 2 ** 31 - 1, -2 ** 31]
    x = ref.make(len(lens), T, 2, getattr(torch, DT[dtype]), decay, seed=70)
    x["lens"] = torch.tensor(lens, dtype=torch.int32)
    for b, n in enumerate(lens):
        n = max(0, min(T, n))
        for name in ("r", "k", "v", "dy"):
            x[name][b, n:] = (float("nan"), float("inf"), -float("inf"))[b % 3]
        if decay == "token":
            x["log_w"][b, n:] = (float("nan"), float("inf"), -float("inf"))[b % 3]
    got = compare(torch, x, ("lens", T, decay, dtype))
    for b, n in enumerate(lens):
        n = max(0, min(T, n))
        for name in ("dr", "dk", "dv") + (("dlog_w",) if decay == "token" else ()):
            assert not got[name][b, n:].any()
        if n == 0:
            assert torch.equal(got["dstate_in"][b].cpu(), x["dstate_out"][b])


def test_without_states_in_place_and_empty(torch):
    x = ref.make(2, 140, 3, torch.bfloat16, "token", seed=80)
    d = dev(x)
    g = run(d)
    g0 = run(d, want_dstate=False)
    assert g0["dstate_in"] is None and all(torch.equal(g[n], g0[n]) for n in ("dr", "dk", "dv", "dlog_w"))
    ds = d["dstate_out"].clone()  # the gradient of the state in place
    out = {n: torch.empty_like(g[n]) for n in ("dr", "dlog_w", "dk", "dv")}
    wkv.rwkv7_linattn_backward(d["r"], d["log_w"], d["k"], d["v"], d["state_in"], None, d["dy"], ds, out["dr"],
                               out["dlog_w"], out["dk"], out["dv"], ds)
    assert torch.equal(ds, g["dstate_in"]) and all(torch.equal(out[n], g[n]) for n in out)
    for B, T in ((2, 0), (0, 140)):
        e = {n: (d[n][:B, :T].contiguous() if n in ("r", "k", "v", "dy") else d[n]) for n in d}
        e["log_w"] = torch.full((3,), -0.1, device="cuda")
        e["state_in"], e["dstate_out"] = d["state_in"][:B], d["dstate_out"][:B]
        g = run(e)
        assert g["dlog_w"].shape == (3,) and not g["dlog_w"].any() and torch.equal(g["dstate_in"], e["dstate_out"])


@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("B,T,H", [(2, 300, 3), (1, 3000, 2)])
def test_repeats_bit_for_bit_and_graph(torch, B, T, H, decay):
    x = ref.make(B, T, H, torch.bfloat16, decay, seed=91)
    d = dev(x)
    first = run(d)
    names = list(first)
    for _ in range(3):
        g = run(d)
        assert all(torch.equal(first[n], g[n]) for n in names)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = {n: torch.empty_like(first[n]) for n in names}

    def call():
        wkv.rwkv7_linattn_backward(d["r"], d["log_w"], d["k"], d["v"], d["state_in"], None, d["dy"], d["dstate_out"],
                                   out["dr"], out["dlog_w"], out["dk"], out["dv"], out["dstate_in"], stream=st)

    call()
    st.synchronize()
    assert all(torch.equal(first[n], out[n]) for n in names)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for seed in (92, 93):
        z = ref.make(B, T, H, torch.bfloat16, decay, seed=seed)
        for n in ("r", "k", "v", "log_w", "dy", "state_in", "dstate_out"):
            d[n].copy_(z[n])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        once = {n: out[n].clone() for n in names}
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(once[n], out[n]) for n in names)
        if seed == 93:
            check_all(torch, z, once)


@pytest.mark.parametrize("decay", ["head", "token"])
def test_against_differences(torch, decay):
    """The gradients against differences of the forward kernel's own outputs, in float32."""
    x = ref.make(2, 150, 2, torch.float32, decay, seed=95)
    d = dev(x)
    got = run(d)

    def loss(**kw):
        z = dict(d, **kw)
        y, s = wkv.linattn(z["r"], z["log_w"], z["k"], z["v"], state_in=z["state_in"])
        return float((y.double() * d["dy"].double()).sum() + (s.double() * d["dstate_out"].double()).sum())

    g = torch.Generator(device="cuda").manual_seed(3)
    for name, grad in (("r", "dr"), ("k", "dk"), ("v", "dv"), ("log_w", "dlog_w"), ("state_in", "dstate_in")):
        # along the gradient itself, so that the difference is large against the outputs' rounding: h |grad|^2
        way = got[grad] / got[grad].norm()
        h = 0.01 if name != "log_w" else 1e-4
        diff = (loss(**{name: d[name] + h * way}) - loss(**{name: d[name] - h * way})) / (2 * h)
        want = float(got[grad].norm())
        # loss is linear in r, k (with S_0 fixed), v, S_0 and smooth in log_w; its rounding: every output to about
        # 2^-20 of its size (see the forward's bound), of both signs, over 2h; log_w's third derivative besides
        y, s = wkv.linattn(d["r"], d["log_w"], d["k"], d["v"], state_in=d["state_in"])
        noise = 2.0 ** -20 * float(((y * d["dy"]).double().square().sum() + (s * d["dstate_out"]).double().square().sum()).sqrt())
        assert abs(diff - want) <= 4 * noise / h + (1e-3 * want if name == "log_w" else 1e-6 * want), (name, diff, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_and_norm_of_its_heads_together(torch, dtype):
    """A layer's use of both: y = linattn, o = norm over each head's 64 channels, and back, with the intermediate
    values as the kernels rounded them; each operator is held to its own float64 values on those inputs."""
    B, T, H = 2, 200, 5
    dt = getattr(torch, DT[dtype])
    x = ref.make(B, T, H, dt, "token", seed=99)
    d = dev(x)
    g = torch.Generator().manual_seed(4)
    w, b = 1 + 0.2 * torch.randn(H * 64, generator=g), 0.2 * torch.randn(H * 64, generator=g)
    do = torch.randn(B, T, H * 64, generator=g).to(dt)
    y, s = wkv.linattn(d["r"], d["log_w"], d["k"], d["v"], state_in=d["state_in"])
    rows = y.view(B, T, H * 64)
    o, mean, rstd = wkv.layernorm(rows, w.cuda(), b.cuda(), groups=H, eps=64e-5)
    n = wkv.layernorm_backward(rows, w.cuda(), mean, rstd, do.cuda(), groups=H)
    got = wkv.linattn_backward(d["r"], d["log_w"], d["k"], d["v"], n["dx"].view(B, T, H, 64), state_in=d["state_in"],
                               dstate_out=d["dstate_out"])
    torch.cuda.synchronize()
    yr, sr, ya, sa = ref.forward(x)
    ref.check("y", y, yr, ya, T, dtype == "bf16")
    flat = rows.cpu().reshape(B * T, H * 64)
    want = layernorm_ref.forward(flat, w, b, H, 64e-5)
    lim = layernorm_ref.forward_limits(flat, w, b, H, 64e-5, dt)
    layernorm_ref.check("o", o.reshape(B * T, -1), want[0], lim[0])
    m, r = mean.cpu().view(B * T, H), rstd.cpu().view(B * T, H)
    flat_do = do.reshape(B * T, -1)
    want = layernorm_ref.backward(flat, w, m, r, flat_do, H)
    lim = layernorm_ref.backward_limits(flat, w, m, r, flat_do, H)
    layernorm_ref.check("dx", n["dx"].reshape(B * T, -1), want["dx"], lim["dx"])
    for name in ("dweight", "dbias"):
        layernorm_ref.check(name, n[name], want[name], lim[name])
    check_all(torch, dict(x, dy=n["dx"].cpu().view(B, T, H, 64)), got)
