"""The gated linear unit on the GPU against float64, at the sizes where it can go wrong."""
import threading

import pytest

from linear_rnn_amd import wkv
from tests import glu_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
ACT = {"sigmoid": wkv.RWKV7_ACT_SIGMOID, "silu": wkv.RWKV7_ACT_SILU, "gelu": wkv.RWKV7_ACT_GELU, "relu2": wkv.RWKV7_ACT_RELU2}


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def cuda(x):
    return {n: t.cuda() for n, t in x.items()}


def forward(d, act, **kw):
    return wkv.glu(d["x"], d["w_gate"], d["w_up"], act=ACT[act], **kw)


def backward(d, act, **kw):
    return wkv.glu_backward(d["x"], d["w_gate"], d["w_up"], d["gate"], d["up"], d["dh"], act=ACT[act], **kw)


# rows: one to a few, tile edges; channels: below, at and behind a step of 64, not a multiple of 8; hidden channels
# below, at and behind a tile, odd
SIZES = [(1, 8, 8), (1, 1, 1), (3, 7, 5), (1, 768, 2048), (5, 64, 136), (16, 40, 24), (17, 200, 264), (33, 64, 100), (64, 96, 130),
         (65, 72, 256), (128, 128, 128), (129, 1000, 136), (255, 200, 129), (256, 256, 512), (257, 264, 520), (300, 33, 1000),
         (1000, 512, 1365), (2000, 16, 72), (20, 72, 8200),
         (100, 768, 2048), (400, 768, 1000)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_forward_and_gradients(torch, M, D, F, dtype):
    act = ref.ACTS[(M + D + F) % 4]
    say("glu", M, D, F, dtype, act)
    x = ref.make(M, D, F, getattr(torch, dtype), seed=M * 10007 + D * 101 + F)
    d = cuda(x)
    got = dict(zip(("h", "gate", "up"), forward(d, act, want_pre=True)))
    for n, v in ref.forward(x["x"], x["w_gate"], x["w_up"], act).items():
        ref.check(n, got[n], v)
        if M * F >= 10000:
            ref.norm(n, got[n], v, D)
    h, none, none2 = forward(d, act)
    assert none is None and none2 is None and torch.equal(h, got["h"])
    grads = backward(d, act)
    for n, v in ref.backward(x["x"], x["w_gate"], x["w_up"], x["gate"], x["up"], x["dh"], act).items():
        ref.check(n, grads[n], v)
        if v[0].numel() >= 10000:
            ref.norm(n, grads[n], v, 2 * F if n == "dx" else M)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M", [4, 40, 200])
def test_activations(torch, M, act, dtype):
    """Small and large pre-activations, whose exponentials vanish or overflow."""
    for size in (0.01, 1.0, 40.0, 300.0):
        x = ref.make(M, 64, 96, getattr(torch, dtype), seed=3, size=size)
        d = cuda(x)
        got = dict(zip(("h", "gate", "up"), forward(d, act, want_pre=True)))
        for n, v in ref.forward(x["x"], x["w_gate"], x["w_up"], act).items():
            ref.check(n, got[n], v)
        grads = backward(d, act)
        for n, v in ref.backward(x["x"], x["w_gate"], x["w_up"], x["gate"], x["up"], x["dh"], act).items():
            ref.check(n, grads[n], v)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_what_stands_next_to_the_operands(torch, dtype):
    """Operands in the middle of larger buffers of NaN: nothing outside them is read into a result or written."""
    for M, D, F in ((3, 24, 40), (70, 40, 72), (300, 72, 136), (5, 7, 9), (130, 33, 21)):
        x = ref.make(M, D, F, getattr(torch, dtype), seed=8)
        d, room = {}, {}
        for n, t in x.items():
            big = torch.full((t.numel() + 4096,), float("nan"), dtype=t.dtype, device="cuda")
            big[2048:2048 + t.numel()] = t.flatten().cuda()
            room[n], d[n] = big, big[2048:2048 + t.numel()].view(t.shape)
        outs, whole = {}, {}
        for n, like in (("h", "gate"), ("g", "gate"), ("u", "gate"), ("dx", "x"), ("dw_gate", "w_gate"), ("dw_up", "w_up")):
            k = x[like].numel()
            whole[n] = torch.full((k + 4096,), 7.0, dtype=x[like].dtype, device="cuda")
            outs[n] = whole[n][2048:2048 + k].view(x[like].shape)
        wkv.rwkv7_glu_forward(d["x"], d["w_gate"], d["w_up"], outs["h"], outs["g"], outs["u"], act=ACT["silu"])
        wkv.rwkv7_glu_backward(d["x"], d["w_gate"], d["w_up"], d["gate"], d["up"], d["dh"], outs["dx"], outs["dw_gate"],
                               outs["dw_up"], act=ACT["silu"])
        want = ref.forward(x["x"], x["w_gate"], x["w_up"], "silu")
        ref.check("h", outs["h"], want["h"])
        ref.check("gate", outs["g"], want["gate"])
        ref.check("up", outs["u"], want["up"])
        for n, v in ref.backward(x["x"], x["w_gate"], x["w_up"], x["gate"], x["up"], x["dh"], "silu").items():
            ref.check(n, outs[n], v)
        for n, t in whole.items():
            assert (t[:2048] == 7).all() and (t[2048 + outs[n].numel():] == 7).all(), (n, M, D, F)


def test_rows_are_their_own(torch):
    """A row's result is the same bits beside any other rows; NaN and infinity in one row stay there."""
    for M, D, F, dtype in ((300, 136, 264, "bfloat16"), (50, 136, 264, "bfloat16"), (300, 72, 40, "float32"), (20, 72, 40, "float32")):
        d = cuda(ref.make(M, D, F, getattr(torch, dtype), seed=4))
        h, _, _ = forward(d, "gelu")
        d["x"][7, 3], d["x"][7, 9] = float("nan"), float("inf")
        bad, _, _ = forward(d, "gelu")
        assert torch.isnan(bad[7]).all()
        assert torch.equal(torch.cat([bad[:7], bad[8:]]), torch.cat([h[:7], h[8:]]))


def test_leading_dimensions_and_left_out_gradients(torch):
    d = cuda(ref.make(60, 64, 128, torch.bfloat16, seed=5))
    h, gate, up = forward(d, "silu", want_pre=True)
    x3 = d["x"].view(3, 20, 64)
    h3, g3, u3 = wkv.glu(x3, d["w_gate"], d["w_up"], act=ACT["silu"], want_pre=True)
    assert h3.shape == (3, 20, 128) and torch.equal(h3.view(60, 128), h) and torch.equal(u3.view(60, 128), up)
    g = wkv.glu_backward(x3, d["w_gate"], d["w_up"], g3, u3, h3, act=ACT["silu"])
    only_x = wkv.glu_backward(x3, d["w_gate"], d["w_up"], g3, u3, h3, act=ACT["silu"], want_dw=False)
    only_w = wkv.glu_backward(x3, d["w_gate"], d["w_up"], g3, u3, h3, act=ACT["silu"], want_dx=False)
    assert g["dx"].shape == x3.shape and torch.equal(only_x["dx"], g["dx"]) and only_x["dw_up"] is None
    assert only_w["dx"] is None and torch.equal(only_w["dw_gate"], g["dw_gate"]) and torch.equal(only_w["dw_up"], g["dw_up"])
    one = wkv.glu(d["x"][0], d["w_gate"], d["w_up"], act=ACT["silu"])[0]
    assert one.shape == (128,)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_no_rows_and_no_hidden_channels(torch, dtype):
    t = getattr(torch, dtype)
    for M, F in ((0, 40), (5, 0)):
        d = cuda(ref.make(M, 24, F, t, seed=6))
        assert forward(d, "silu", want_pre=True)[0].shape == (M, F)
        g = {"dx": torch.ones_like(d["x"]), "dw_gate": torch.ones_like(d["w_gate"]), "dw_up": torch.ones_like(d["w_up"])}
        wkv.rwkv7_glu_backward(d["x"], d["w_gate"], d["w_up"], d["gate"], d["up"], d["dh"], g["dx"], g["dw_gate"], g["dw_up"])
        assert not any(v.any() for v in g.values())


def test_offsets_past_32_bits(torch):
    """An output of 4.6e9 elements and an input of 2.3e9: the last rows against a call of their own, bit for bit."""
    M, D, F = 280_000, 8192, 16400
    say("glu offsets past 32 bits", M, D, F)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.empty(M, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    wg, wu = (torch.empty(D, F, dtype=torch.bfloat16, device="cuda").normal_(0, 0.01, generator=g) for _ in range(2))
    h, _, _ = wkv.glu(x, wg, wu)
    last, _, _ = wkv.glu(x[-1000:], wg, wu)
    assert torch.equal(h[-1000:], last)
    del h, last
    pre = torch.empty(M, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = wg[:, :128].contiguous()
    dh = torch.zeros_like(pre)
    dh[-700:] = pre[:700]
    grads = wkv.glu_backward(x, w, w, pre, pre, dh)
    part = wkv.glu_backward(x[-700:], w, w, pre[-700:], pre[-700:], dh[-700:])
    assert torch.equal(grads["dx"][-700:], part["dx"]) and not grads["dx"][:-700].any()
    for n in ("dw_gate", "dw_up"):  # the same products in sums cut differently, rounded to bfloat16 in each
        a, b = grads[n].float(), part[n].float()
        assert float((a - b).norm()) <= 2.0 ** -7 * float(b.norm()), n


def chain(d, out, stream):
    """Forward and backward in a row, into `out`."""
    wkv.rwkv7_glu_forward(d["x"], d["w_gate"], d["w_up"], out["h"], out["gate"], out["up"], act=ACT["silu"], stream=stream)
    wkv.rwkv7_glu_backward(d["x"], d["w_gate"], d["w_up"], out["gate"], out["up"], out["h"], out["dx"], out["dw_gate"],
                           out["dw_up"], act=ACT["silu"], stream=stream)


def case(torch, M, D, F, dtype, seed):
    d = cuda(ref.make(M, D, F, dtype, seed=seed))
    out = {n: torch.empty_like(d["gate"]) for n in ("h", "gate", "up")}
    out.update(dx=torch.empty_like(d["x"]), dw_gate=torch.empty_like(d["w_gate"]), dw_up=torch.empty_like(d["w_up"]))
    return d, out


def clones(out):
    return {n: t.clone() for n, t in out.items()}


def same(torch, a, b):
    assert all(torch.equal(a[n], b[n]) for n in a)


def cases_of(torch):
    return [case(torch, 1500, 72, 200, torch.bfloat16, 1), case(torch, 700, 60, 130, torch.float32, 2),
            case(torch, 900, 33, 90, torch.bfloat16, 3), case(torch, 20, 64, 256, torch.float32, 4)]


def test_two_streams_and_two_threads(torch):
    cases, want = cases_of(torch), []
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
    stream = torch.cuda.Stream()
    cases, want, graphs = cases_of(torch), [], []
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
            for g, (d, _) in zip(graphs, cases):
                g.replay()
                wkv.glu(d["x"], d["w_gate"], d["w_up"], stream=stream)
        stream.synchronize()
        for (_, out), w in zip(cases, want):
            same(torch, out, w)


def test_outputs_on_another_stream(torch):
    d = cuda(ref.make(200, 64, 128, torch.bfloat16, seed=9))
    h, gate, up = forward(d, "silu", want_pre=True)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(20):
        h1, g1, u1 = forward(d, "silu", want_pre=True, stream=stream)
    stream.synchronize()
    assert torch.equal(h, h1) and torch.equal(gate, g1) and torch.equal(up, u1)


def test_growth_during_capture_is_refused(torch):
    stream = torch.cuda.Stream()
    d, out = case(torch, 3000, 130, 1001, torch.bfloat16, 10)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        with pytest.raises(wkv.Rwkv7Error):
            wkv.rwkv7_glu_forward(d["x"], d["w_gate"], d["w_up"], out["h"], None, None, stream=stream)
        with pytest.raises(wkv.Rwkv7Error):
            wkv.rwkv7_glu_backward(d["x"], d["w_gate"], d["w_up"], d["gate"], d["up"], d["dh"], out["dx"], None, None,
                                   stream=stream)
    chain(d, out, stream)
    stream.synchronize()


def test_many_rows_of_few_channels(torch):
    """More rows than a grid's second dimension has, in products of one tile of columns."""
    for dtype in (torch.float32, torch.bfloat16):
        x = ref.make(2_200_000, 8, 8, dtype, seed=11)
        d = cuda(x)
        h = forward(d, "silu")[0]
        part = slice(2_199_000, 2_200_000)
        ref.check("h", h[part], ref.forward(x["x"][part], x["w_gate"], x["w_up"], "silu")["h"])
        g = backward(d, "silu", want_dw=False)
        want = ref.backward(x["x"][part], x["w_gate"], x["w_up"], x["gate"][part], x["up"][part], x["dh"][part], "silu")
        ref.check("dx", g["dx"][part], want["dx"])


# float32: few rows, each height of the float32 instructions' tiles (16 to 80 rows), pieces; bfloat16: few rows of even and
# odd widths, 32 rows at a time, tiles of each shape, whole and in parts
@pytest.mark.parametrize("act,M,D,F,dtype", [
    ("gelu", 7, 770, 2049, "float32"), ("gelu", 30, 769, 2050, "float32"), ("silu", 100, 770, 2049, "float32"), ("silu", 140, 770, 2049, "float32"),
    ("silu", 250, 770, 2049, "float32"), ("relu2", 515, 333, 1001, "float32"), ("sigmoid", 1000, 333, 1001, "float32"),
    ("gelu", 515, 770, 2049, "float32"), ("silu", 3000, 770, 2049, "float32"),
    ("gelu", 7, 770, 2050, "bfloat16"), ("silu", 31, 30, 2, "bfloat16"), ("silu", 20, 771, 130, "bfloat16"),
    ("relu2", 90, 770, 2046, "bfloat16"), ("silu", 700, 200, 2056, "bfloat16"), ("gelu", 300, 2048, 5000, "bfloat16"),
    ("sigmoid", 1030, 768, 1031, "bfloat16"), ("silu", 2600, 264, 1000, "bfloat16"), ("gelu", 4100, 1000, 2054, "bfloat16"),
    ("relu2", 8200, 72, 264, "bfloat16"), ("silu", 300, 4096, 100, "bfloat16"),
    ("silu", 2500, 200, 2056, "bfloat16"), ("gelu", 400, 1000, 2056, "bfloat16")])
def test_each_way(torch, act, M, D, F, dtype):
    """Operands in the middle of larger buffers of NaN, outputs next to what has to stay."""
    say("glu", M, D, F, act, dtype)
    dt = getattr(torch, dtype)
    x = ref.make(M, D, F, dt, seed=M + 1)
    d = {}
    for n in ("x", "w_gate", "w_up"):
        big = torch.full((x[n].numel() + 4096,), float("nan"), dtype=dt, device="cuda")
        d[n] = big[2048:2048 + x[n].numel()].view(x[n].shape)
        d[n].copy_(x[n])
    whole = [torch.full((M * F + 4096,), 7.0, dtype=dt, device="cuda") for _ in range(3)]
    got = [t[2048:2048 + M * F].view(M, F) for t in whole]
    wkv.rwkv7_glu_forward(d["x"], d["w_gate"], d["w_up"], *got, act=ACT[act])
    want = ref.forward(x["x"], x["w_gate"], x["w_up"], act)
    for n, t in zip(("h", "gate", "up"), got):
        ref.check(n, t, want[n])
        if M * F >= 10000:
            ref.norm(n, t, want[n], D)
    for t in whole:
        assert (t[:2048] == 7).all() and (t[2048 + M * F:] == 7).all()
