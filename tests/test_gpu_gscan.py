"""The gated linear recurrence on the GPU against float64, at the sizes and masks where it can go wrong."""
import threading

import pytest

from linear_rnn_amd import wkv
from tests import gscan_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
KIND = {"plain": wkv.RWKV7_INPUT_PLAIN, "mix": wkv.RWKV7_INPUT_MIX, "norm": wkv.RWKV7_INPUT_NORM}


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


# one token and tile edges (128 tokens; 32 where D leaves one to three of 64 channels over), widths below, at and behind 64 channels, odd
# ones, few channels over many tokens (segments), many sequences (none)
SIZES = [(1, 1, 1), (2, 1, 64), (1, 2, 3), (2, 7, 5), (2, 31, 66), (1, 33, 65), (3, 127, 64), (2, 128, 68), (2, 129, 128),
         (1, 257, 130), (2, 300, 1000), (1, 3001, 64), (5, 1000, 4), (1, 700, 33), (300, 40, 20), (130, 70, 130), (1, 4500, 96), (1, 9000, 24), (1, 4500, 33),
         (4, 0, 16)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("kind", ref.KINDS)
@pytest.mark.parametrize("B,T,D", SIZES)
def test_prompt_and_gradients(torch, B, T, D, kind, dtype):
    say("gscan", B, T, D, kind, dtype)
    x = ref.make(B, T, D, getattr(torch, dtype), seed=B * 1000003 + T * 1009 + D)
    d = cuda(x)
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"], input=KIND[kind])
    got = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=KIND[kind])
    want = ref.forward(x["x"], x["log_w"], x["state_in"], None, kind)
    ref.check("y", y, want["y"])
    ref.check("state", s, want["state"])
    for n, v in ref.backward(x["x"], x["log_w"], x["state_in"], None, x["dy"], x["dstate_out"], kind).items():
        ref.check(n, got[n], v)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,T,D", [(6, 300, 72), (6, 150, 37), (6, 2000, 8)])
def test_padded_batch(torch, B, T, D, dtype):
    """Lengths of zero, one, a tile's edge, all, and values outside [0, T]; anything may stand behind the end."""
    lens = [0, 1, 128, T, -5, T + 9]
    say("gscan padded", B, T, D, dtype)
    x = ref.make(B, T, D, getattr(torch, dtype), seed=7)
    for n, v in (("x", float("nan")), ("log_w", float("nan")), ("dy", float("inf"))):
        for b, m in enumerate(lens):
            x[n][b, max(m, 0):] = v
    d = cuda(x)
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"], lens=dl, input=KIND["norm"])
    want = ref.forward(x["x"], x["log_w"], x["state_in"], lens, "norm")
    ref.check("y", y, want["y"])
    ref.check("state", s, want["state"])
    assert torch.equal(s[0], d["state_in"][0])
    got = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], lens=dl, dstate_out=d["dstate_out"], input=KIND["norm"])
    for n, v in ref.backward(x["x"], x["log_w"], x["state_in"], lens, x["dy"], x["dstate_out"], "norm").items():
        ref.check(n, got[n], v)
    for b, m in enumerate(lens):
        assert not y[b, max(m, 0):].any() and not got["dx"][b, max(m, 0):].any() and not got["dlog_w"][b, max(m, 0):].any()


@pytest.mark.parametrize("kind", ref.KINDS)
def test_decays_at_the_ends(torch, kind):
    """Decays of exactly one and zero, close to one, and too small for float32, each over a whole sequence."""
    values = [0.0, -1e-30, -1e-7, -1e-3, -0.17, -0.175, -0.35, -0.36, -80.0, -200.0, -float("inf"), -3e38]
    x = ref.make(1, 300, len(values), torch.float32, seed=3, resets=0)
    x["log_w"] = torch.tensor(values).expand(1, 300, -1).contiguous()
    d = cuda(x)
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"], input=KIND[kind])
    want = ref.forward(x["x"], x["log_w"], x["state_in"], None, kind)
    ref.check("y", y, want["y"])
    ref.check("state", s, want["state"])
    got = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=KIND[kind])
    for n, v in ref.backward(x["x"], x["log_w"], x["state_in"], None, x["dy"], x["dstate_out"], kind).items():
        ref.check(n, got[n], v)
    assert not got["dlog_w"][..., values.index(-float("inf"))].any()


def test_reset_parts_packed_sequences(torch):
    """A decay of zero keeps what is before it away: the tokens from it on are those of a sequence of their own."""
    x = cuda(ref.make(1, 400, 64, torch.float32, seed=4, state=False, resets=0))
    x["log_w"][:, 150] = -float("inf")
    y, s = wkv.gscan(x["x"], x["log_w"])
    y1, s1 = wkv.gscan(x["x"][:, 150:].contiguous(), x["log_w"][:, 150:].contiguous())
    far = (y[:, 150:] - y1).abs().max() / y1.abs().max()
    assert far <= 1e-5, far  # the two are cut into tiles differently
    x["x"][:, :150] = 1e30
    y2, s2 = wkv.gscan(x["x"], x["log_w"])
    assert torch.equal(y2[:, 150:], y[:, 150:]) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("kind", ref.KINDS)
@pytest.mark.parametrize("B,D", [(1, 1), (3, 7), (2, 6), (4, 768), (70, 1000)])
def test_step(torch, B, D, kind, dtype):
    """The step is the prompt of one token, bit for bit, also in place and from no state."""
    say("gscan step", B, D, kind, dtype)
    x = ref.make(B, 1, D, getattr(torch, dtype), seed=11, resets=0.1)
    d = cuda(x)
    for state in (d["state_in"], None):
        y, s = wkv.gscan_step(d["x"], d["log_w"], state, input=KIND[kind])
        y1, s1 = wkv.gscan(d["x"], d["log_w"], state, input=KIND[kind])
        assert torch.equal(y, y1) and torch.equal(s, s1)
        want = ref.forward(x["x"], x["log_w"], None if state is None else x["state_in"], None, kind)
        ref.check("y", y, want["y"])
        ref.check("state", s, want["state"])
    place, y2 = d["state_in"].clone(), torch.empty_like(d["x"])
    wkv.rwkv7_gscan_step(d["x"], d["log_w"], place, y2, place, input=KIND[kind])
    y, s = wkv.gscan_step(d["x"], d["log_w"], d["state_in"], input=KIND[kind])
    assert torch.equal(place, s) and torch.equal(y2, y)
    wkv.rwkv7_gscan_step(d["x"], d["log_w"], d["state_in"], y2, None, input=KIND[kind])
    assert torch.equal(y2, y)


@pytest.mark.parametrize("B,T,D", [(1, 2000, 64), (2, 100, 128), (1, 500, 7)])
def test_in_place_and_left_out_states(torch, B, T, D):
    """The final state over the initial one, their gradients likewise, and calls that want neither."""
    d = cuda(ref.make(B, T, D, torch.bfloat16, seed=5))
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"], input=KIND["mix"])
    g = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=KIND["mix"])
    place, ds, y1 = d["state_in"].clone(), d["dstate_out"].clone(), torch.empty_like(y)
    wkv.rwkv7_gscan_prefill(d["x"], d["log_w"], place, None, y1, place, input=KIND["mix"])
    assert torch.equal(place, s) and torch.equal(y1, y)
    dx, dw = torch.empty_like(g["dx"]), torch.empty_like(g["dlog_w"])
    wkv.rwkv7_gscan_backward(d["x"], d["log_w"], d["state_in"], None, d["dy"], ds, dx, dw, ds, input=KIND["mix"])
    assert torch.equal(dx, g["dx"]) and torch.equal(dw, g["dlog_w"]) and torch.equal(ds, g["dstate_in"])
    y2, none = wkv.gscan(d["x"], d["log_w"], d["state_in"], input=KIND["mix"], want_state=False)
    assert none is None and torch.equal(y2, y)
    g2 = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=KIND["mix"],
                            want_dstate=False)
    assert g2["dstate_in"] is None and torch.equal(g2["dx"], g["dx"])
    zero = torch.zeros_like(place)
    for a, b in ((None, zero), (zero, None)):
        ya, sa = wkv.gscan(d["x"], d["log_w"], a)
        yb, sb = wkv.gscan(d["x"], d["log_w"], b)
        assert torch.equal(ya, yb) and torch.equal(sa, sb)
        ga = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], a, dstate_out=a)
        gb = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], b, dstate_out=b)
        assert all(torch.equal(ga[n], gb[n]) for n in ga)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [1, 5, 300, 1500, 9000])
@pytest.mark.parametrize("D", [4, 5, 7, 37, 63, 67, 126, 129])
def test_odd_widths(torch, D, T, dtype):
    """Rows that begin anywhere, states in place, next to values that have to stay."""
    B, kind = (2, "norm") if T < 1000 else (1, "mix")
    say("gscan", B, T, D, kind, dtype)
    x = ref.make(B, T, D, getattr(torch, dtype), seed=T + D)
    outs, rooms = {}, []

    def place(like):
        room = torch.full((like.numel() + 512,), 7.0, dtype=like.dtype, device="cuda")
        rooms.append((room, like.numel()))
        out = room[256:256 + like.numel()].view(like.shape)
        out.copy_(like)
        return out

    d = {n: place(t) for n, t in x.items()}
    for n, like in (("y", "x"), ("dx", "x"), ("dlog_w", "log_w")):
        outs[n] = place(x[like])
    outs["state"], outs["dstate_in"] = place(x["state_in"]), place(x["dstate_out"])
    wkv.rwkv7_gscan_prefill(d["x"], d["log_w"], outs["state"], None, outs["y"], outs["state"], input=KIND[kind])
    wkv.rwkv7_gscan_backward(d["x"], d["log_w"], d["state_in"], None, d["dy"], outs["dstate_in"], outs["dx"], outs["dlog_w"],
                             outs["dstate_in"], input=KIND[kind])
    want = {**ref.forward(x["x"], x["log_w"], x["state_in"], None, kind),
            **ref.backward(x["x"], x["log_w"], x["state_in"], None, x["dy"], x["dstate_out"], kind)}
    for n, t in outs.items():
        ref.check(n, t, want[n])
    for room, n in rooms:
        assert (room[:256] == 7).all() and (room[256 + n:] == 7).all()


def test_no_tokens(torch):
    d = cuda(ref.make(3, 0, 40, torch.bfloat16, seed=6))
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"])
    assert y.shape == (3, 0, 40) and torch.equal(s, d["state_in"])
    assert not wkv.gscan(d["x"], d["log_w"])[1].any()
    g = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"])
    assert torch.equal(g["dstate_in"], d["dstate_out"])
    assert not wkv.gscan_backward(d["x"], d["log_w"], d["dy"])["dstate_in"].any()


@pytest.mark.parametrize("B,T", [(2, 130), (1, 600)])
def test_sequences_and_channels_are_their_own(torch, B, T):
    """The largest width, whose tiles reach past 2^29 bytes: a part of the channels, and one sequence, bit for bit."""
    D = 1 << 20
    say("gscan widest", B, T, D)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    lw = -torch.rand(B, T, D, device="cuda", generator=g)
    y, s = wkv.gscan(x, lw)
    grads = wkv.gscan_backward(x, lw, x)
    part = slice(D - 16384, D)
    x1, lw1 = x[-1:, :, part].contiguous(), lw[-1:, :, part].contiguous()
    y1, s1 = wkv.gscan(x1, lw1)
    assert torch.equal(y[-1:, :, part], y1) and torch.equal(s[-1:, part], s1)
    g1 = wkv.gscan_backward(x1, lw1, x1)
    assert torch.equal(grads["dx"][-1:, :, part], g1["dx"]) and torch.equal(grads["dlog_w"][-1:, :, part], g1["dlog_w"])


def test_offsets_past_32_bits(torch):
    """2.4e9 elements: the last tokens against a call that starts there, and the gradients in two parts that meet."""
    B, T, D, cut = 1, 73728, 32768, 73000
    say("gscan offsets past 32 bits", B, T, D)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    lw = torch.empty(B, T, D, device="cuda").uniform_(-0.5, -0.01, generator=g)
    y, s = wkv.gscan(x, lw)
    _, mid = wkv.gscan(x[:, :cut], lw[:, :cut])
    y1, s1 = wkv.gscan(x[:, cut:], lw[:, cut:], mid)

    def near(a, b):  # float32 sums cut differently (100 tokens count, 5 roundings each), then a rounding to bfloat16 in each
        a, b = a.float(), b.float()
        assert float((a - b).norm()) <= 2.0 ** -7 * float(b.norm()) and float(b.norm()) > 0

    near(y[:, cut:], y1)
    near(s, s1)
    del y, y1
    whole = wkv.gscan_backward(x, lw, x)
    last = wkv.gscan_backward(x[:, cut:], lw[:, cut:], x[:, cut:], state_in=mid)
    for n in ("dx", "dlog_w"):
        near(whole[n][:, cut:], last[n])
    first = wkv.gscan_backward(x[:, cut - 2000:cut].contiguous(), lw[:, cut - 2000:cut].contiguous(),
                               x[:, cut - 2000:cut].contiguous(), dstate_out=last["dstate_in"])
    near(whole["dx"][:, cut - 1000:cut], first["dx"][:, -1000:])


def chain(d, out, stream):
    """A prompt in segments, its gradients, and a token behind it, into `out`."""
    wkv.rwkv7_gscan_prefill(d["x"], d["log_w"], d["state_in"], None, out["y"], out["s"], input=KIND["mix"], stream=stream)
    wkv.rwkv7_gscan_backward(d["x"], d["log_w"], d["state_in"], None, out["y"], d["dstate_out"], out["dx"], out["dw"],
                             out["ds"], input=KIND["mix"], stream=stream)
    wkv.rwkv7_gscan_step(d["x1"], d["w1"], out["s"], out["y1"], out["s"], input=KIND["mix"], stream=stream)


def case(torch, B, T, D, seed):
    d = cuda(ref.make(B, T, D, torch.bfloat16, seed=seed))
    d["x1"], d["w1"] = d["x"][:, :1].contiguous(), d["log_w"][:, -1:].contiguous()
    return d, {"y": torch.empty_like(d["x"]), "dx": torch.empty_like(d["x"]), "dw": torch.empty_like(d["log_w"]),
               "s": torch.empty_like(d["state_in"]), "ds": torch.empty_like(d["state_in"]), "y1": torch.empty_like(d["x1"])}


def clones(out):
    return {n: t.clone() for n, t in out.items()}


def same(torch, a, b):
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_two_streams_and_two_threads(torch):
    cases = [case(torch, 2, 1500 + 200 * i, 64, i) for i in range(4)]
    want = []
    for d, out in cases:
        chain(d, out, None)
        torch.cuda.synchronize()
        want.append(clones(out))
        for t in out.values():
            t.zero_()
    shared, own = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def work(i, stream):
        for _ in range(10):
            chain(*cases[i], stream)

    threads = [threading.Thread(target=work, args=(i, s)) for i, s in enumerate((shared, shared, own, own))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (_, out), w in zip(cases, want):
        same(torch, out, w)


def test_graphs_that_share_a_workspace(torch):
    """Two graphs of one stream, replayed in turn with eager work between them."""
    stream = torch.cuda.Stream()
    cases = [case(torch, 2, 1500, 64, 1), case(torch, 1, 900, 128, 2)]
    want, graphs = [], []
    with torch.cuda.stream(stream):
        for d, out in cases:
            chain(d, out, stream)
            stream.synchronize()
            want.append(clones(out))
    for d, out in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            chain(d, out, stream)
        graphs.append(g)
    for turn in range(3):
        for _, out in cases:
            for t in out.values():
                t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graphs[0].replay()
            wkv.gscan(cases[0][0]["x"], cases[0][0]["log_w"], stream=stream)
            graphs[1].replay()
        stream.synchronize()
        for (_, out), w in zip(cases, want):
            same(torch, out, w)


def test_outputs_on_another_stream(torch):
    """The allocating calls on a stream of their own, many in a row with nothing kept: memory is that stream's."""
    d = cuda(ref.make(2, 600, 64, torch.bfloat16, seed=9))
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"])
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(20):
        y1, s1 = wkv.gscan(d["x"], d["log_w"], d["state_in"], stream=stream)
    stream.synchronize()
    assert torch.equal(y, y1) and torch.equal(s, s1)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,T,D", [(1, 900, 130), (2, 8192, 64), (1, 600, 7), (40, 4000, 132)])
def test_gradients_without_waiting(torch, B, T, D, dtype):
    """A workgroup that looks for the other tiles' maps only once leaves its tile to a second kernel: the same bits."""
    import ctypes
    polls = getattr(ctypes.CDLL(wkv.LIB_PATH), "_ZN5rwkv715set_gscan_pollsEi")
    say("gscan without waiting", B, T, D, dtype)
    d = cuda(ref.make(B, T, D, getattr(torch, dtype), seed=12))
    want = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=KIND["mix"])
    torch.cuda.synchronize()
    polls(0)
    try:
        for _ in range(3):
            got = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=KIND["mix"])
            torch.cuda.synchronize()
            assert all(torch.equal(got[n], want[n]) for n in want)
    finally:
        polls(64)


def test_the_same_call_gives_the_same_bits(torch):
    """Whatever order the workgroups come in: many calls, alone and beside other work on the device."""
    d = cuda(ref.make(3, 5000, 100, torch.bfloat16, seed=13))
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"], input=KIND["norm"])
    g = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=KIND["norm"])
    torch.cuda.synchronize()
    other, a = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    for i in range(20):
        if i % 2:
            with torch.cuda.stream(other):
                a @ a
        y1, s1 = wkv.gscan(d["x"], d["log_w"], d["state_in"], input=KIND["norm"])
        g1 = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=KIND["norm"])
        assert torch.equal(y1, y) and torch.equal(s1, s) and all(torch.equal(g1[n], g[n]) for n in g)
    torch.cuda.synchronize()


def test_growth_during_capture_is_refused(torch):
    """A stream whose workspace is too small: the call fails before any launch, and works after an eager one."""
    stream = torch.cuda.Stream()
    d, out = case(torch, 1, 3000, 192, 14)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        with pytest.raises(wkv.Rwkv7Error):
            wkv.rwkv7_gscan_prefill(d["x"], d["log_w"], None, None, out["y"], None, stream=stream)
        with pytest.raises(wkv.Rwkv7Error):
            wkv.rwkv7_gscan_backward(d["x"], d["log_w"], None, None, d["dy"], None, out["dx"], out["dw"], None, stream=stream)
    chain(d, out, stream)
    stream.synchronize()
    want = clones(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        chain(d, out, stream)
    g.replay()
    torch.cuda.synchronize()
    same(torch, out, want)
