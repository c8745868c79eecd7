"""The linear attention and the layer norm at the ends of what their header allows: offsets past 32 bits, two
streams at once, graphs that share a stream's workspace, and a workspace that would have to grow during capture."""
import threading

import pytest

from linear_rnn_amd import wkv
from tests import linattn_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def near(torch, got, want, name):
    """Results of two runs that part a sequence differently: float32 sums in another order, rounded to bfloat16 once in
    each run (2^-8 twice)."""
    d, n = float((got.float() - want.float()).norm()), float(want.float().norm())
    assert n > 0 and d <= 2.0 ** -7 * n, (name, d, n)


def test_linattn_offsets_past_32_bits(torch):
    """4.8 GB a tensor, 2.4e9 elements: the last tokens against a call that starts there from the state, and the
    gradients in two parts that meet there."""
    B, T, H, cut = 1, 49152, 768, 48000
    say("linattn offsets past 32 bits", B, T, H)
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(scale=1.0):
        return torch.empty(B, T, H, 64, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=g)

    r, k, v, dy = normal(), normal(0.125), normal(), normal()
    log_w = -0.05 - torch.rand(B, T, H, device="cuda", generator=g)
    tail = [t[:, cut:] for t in (r, log_w, k, v)]
    head = [t[:, :cut] for t in (r, log_w, k, v)]
    y, s = wkv.linattn(r, log_w, k, v)
    _, mid = wkv.linattn(*head)
    y1, s1 = wkv.linattn(*tail, state_in=mid)
    near(torch, y[:, cut:], y1, "y")
    near(torch, s, s1, "state")
    del y, y1
    whole = wkv.linattn_backward(r, log_w, k, v, dy)
    last = wkv.linattn_backward(*tail, dy[:, cut:], state_in=mid)
    for n in ("dr", "dk", "dv", "dlog_w"):
        near(torch, whole[n][:, cut:], last[n], n)
    first = wkv.linattn_backward(*head, dy[:, :cut], dstate_out=last["dstate_in"])
    for n in ("dr", "dk", "dv", "dlog_w"):
        near(torch, whole[n][:, cut - 1000:cut], first[n][:, -1000:], n)
        near(torch, whole[n][:, :1000], first[n][:, :1000], n)
    near(torch, whole["dstate_in"], first["dstate_in"], "dstate_in")


def test_layernorm_offsets_past_32_bits(torch):
    M, D = 600_000, 4096
    say("layernorm offsets past 32 bits", M, D)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty(M, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w, b = (torch.empty(D, device="cuda").normal_(generator=g) for _ in range(2))
    dy = torch.zeros_like(x)
    dy[-100:].normal_(generator=g)
    y, mean, rstd = wkv.layernorm(x, w, b)
    y1, mean1, rstd1 = wkv.layernorm(x[-100:], w, b)
    assert torch.equal(y[-100:], y1) and torch.equal(mean[-100:], mean1) and torch.equal(rstd[-100:], rstd1)
    whole = wkv.layernorm_backward(x, w, mean, rstd, dy)
    last = wkv.layernorm_backward(x[-100:], w, mean1, rstd1, dy[-100:])
    assert torch.equal(whole["dx"][-100:], last["dx"]) and not whole["dx"][:-100].any()
    for n in ("dweight", "dbias"):  # 100 float32 terms in two orders: 2 * 100 roundings of 2^-24 of their magnitudes at most
        assert float((whole[n] - last[n]).norm() / last[n].norm()) <= 200 * 2.0 ** -24, n


def chain(torch, d, out, stream):
    """A prompt in segments, its heads' norm, and the gradients of both, into `out`."""
    H = d["r"].shape[2]
    flat = [t.view(*t.shape[:2], H * 64) for t in (out["y"], out["n"], d["dy"], out["dn"])]
    wkv.rwkv7_linattn_prefill(d["r"], d["log_w"], d["k"], d["v"], d["state_in"], None, out["y"], out["s"], stream=stream)
    wkv.rwkv7_layernorm_forward(flat[0], d["w"], None, flat[1], out["mean"], out["rstd"], groups=H, eps=64e-5, stream=stream)
    wkv.rwkv7_layernorm_backward(flat[0], d["w"], out["mean"], out["rstd"], flat[2], flat[3], out["dw"], None, groups=H,
                                 stream=stream)
    wkv.rwkv7_linattn_backward(d["r"], d["log_w"], d["k"], d["v"], d["state_in"], None, out["dn"], None, out["dr"],
                               out["dlog_w"], out["dk"], out["dv"], out["ds"], stream=stream)


def case(torch, B, T, H, seed):
    d = {n: t.cuda() for n, t in ref.make(B, T, H, torch.bfloat16, "token", seed=seed).items() if t is not None}
    d["w"] = torch.rand(H * 64, device="cuda") + 0.5
    out = {n: torch.empty_like(d["r"]) for n in ("y", "n", "dn", "dr", "dk", "dv")}
    out.update(s=torch.empty_like(d["state_in"]), ds=torch.empty_like(d["state_in"]), dlog_w=torch.empty_like(d["log_w"]),
               mean=torch.empty(B, T, H, device="cuda"), rstd=torch.empty(B, T, H, device="cuda"),
               dw=torch.empty_like(d["w"]))
    return d, out


def clones(out):
    return {n: t.clone() for n, t in out.items()}


def test_two_streams_at_once(torch):
    say("two streams at once")
    cases = [case(torch, 1, 3000, 2, 71), case(torch, 2, 2100, 3, 72)]
    want = []
    for d, out in cases:
        chain(torch, d, out, None)
        torch.cuda.synchronize()
        want.append(clones(out))
        for t in out.values():
            t.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(6):
        for (d, out), st in zip(cases, streams):
            chain(torch, d, out, st)
    torch.cuda.synchronize()
    for (d, out), w in zip(cases, want):
        assert all(torch.equal(out[n], w[n]) for n in w)


def test_two_threads_on_one_stream(torch):
    """Their calls' kernels use one workspace and do not fall between each other."""
    say("two threads on one stream")
    cases = [case(torch, 1, 3000, 2, 75), case(torch, 2, 2100, 3, 76)]
    st = torch.cuda.Stream()
    want = []
    for d, out in cases:
        chain(torch, d, out, st)
        st.synchronize()
        want.append(clones(out))
    torch.cuda.synchronize()
    bad = []

    def work(n):
        d, out = cases[n]
        for _ in range(20):
            chain(torch, d, out, st)
        st.synchronize()
        bad.extend((n, name) for name in want[n] if not torch.equal(out[name], want[n][name]))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_two_graphs_of_one_stream(torch):
    """Both use the stream's workspace; replayed one after the other, with eager calls and growth between them, each
    replay gives its call's results."""
    say("two graphs of one stream")
    st = torch.cuda.Stream()
    cases = [case(torch, 1, 2500, 2, 81), case(torch, 2, 1500, 3, 82)]
    want, graphs = [], []
    for d, out in cases:
        chain(torch, d, out, st)
        st.synchronize()
        want.append(clones(out))
    for d, out in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            chain(torch, d, out, st)
        graphs.append(g)
    big, big_out = case(torch, 2, 5000, 8, 83)
    for step in range(4):
        for (d, out), w, g in zip(cases, want, graphs):
            for t in out.values():
                t.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(out[n], w[n]) for n in w), step
            if step == 1:
                chain(torch, big, big_out, st)  # the workspace grows; the graphs keep theirs
                torch.cuda.synchronize()


def test_growth_during_capture_is_refused(torch):
    """A backward that needs 335 MB of workspace on a stream that has had no such call."""
    say("growth during capture")
    st = torch.cuda.Stream()
    d, out = case(torch, 4, 4096, 64, 91)
    torch.cuda.synchronize()

    def call():
        wkv.rwkv7_linattn_backward(d["r"], d["log_w"], d["k"], d["v"], None, None, d["dy"], None, out["dr"], out["dlog_w"],
                                   out["dk"], out["dv"], None, stream=st)

    with pytest.raises(wkv.Rwkv7Error):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=st):
            call()
    torch.cuda.synchronize()
    call()  # the refusal leaves the stream as it was
    torch.cuda.synchronize()
    first = clones(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for t in out.values():
        t.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], first[n]) for n in ("dr", "dk", "dv", "dlog_w"))
