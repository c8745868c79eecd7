"""GPU parity of the linear attention with a decay for each head against the float64 recurrence."""
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


def dev(x):
    return {n: (t.cuda() if t is not None else None) for n, t in x.items()}


def run(x, **kw):
    d = dev(x)
    return wkv.linattn(d["r"], d["log_w"], d["k"], d["v"], state_in=d["state_in"], lens=d["lens"], **kw)


def compare(torch, x, what):
    say("linattn", what)
    y, s = run(x)
    torch.cuda.synchronize()
    yr, sr, ya, sa = ref.forward(x)
    T, bf16 = x["r"].shape[1], x["r"].dtype == torch.bfloat16
    assert y.dtype == x["r"].dtype and s.dtype == torch.float32
    ref.check("y", y, yr, ya, T, bf16)
    ref.check("state", s, sr, sa, T, False)
    return y, s


DT = {"bf16": "bfloat16", "f32": "float32"}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 97, 127, 128, 129, 300])
def test_prefill_lengths(torch, T, decay, dtype):
    """Every tail of a 16-token tile, of a wave's 32 tokens and of a workgroup's 128."""
    x = ref.make(2, T, 3, getattr(torch, DT[dtype]), decay, seed=10 + T, state=T % 2 == 1)
    compare(torch, x, ("lengths", T, decay, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 515, 2100])
def test_prefill_one_head(torch, T, dtype):
    """One head: the sequence is what there is to spread over the device."""
    x = ref.make(1, T, 1, getattr(torch, DT[dtype]), "token", seed=40 + T, resets=0.01)
    compare(torch, x, ("one head", T, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_many_heads(torch, dtype):
    x = ref.make(20, 150, 40, getattr(torch, DT[dtype]), "head", seed=50)
    compare(torch, x, ("many heads", dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_decays_at_their_ends(torch, dtype):
    """No decay at all, resets at every place of a tile, resets everywhere, and decays that underflow."""
    base = ref.make(1, 200, 4, getattr(torch, DT[dtype]), "token", seed=60)
    for name, lw in (("none", 0.0), ("all reset", -float("inf")), ("underflow", -90.0), ("faint", -1e-7)):
        x = dict(base, log_w=torch.full_like(base["log_w"], lw))
        compare(torch, x, ("decay", name, dtype))
    x = dict(base, log_w=base["log_w"].clone())
    for h in range(4):
        x["log_w"][0, h::7 + h, h] = -float("inf")
    compare(torch, x, ("decay", "some resets", dtype))
    x["log_w"] = x["log_w"].clamp_min(-1e30)
    compare(torch, x, ("decay", "large finite", dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_prefill_lens(torch, decay, dtype):
    """Sequences that end anywhere, lengths out of range, and padding that holds NaNs and infinities."""
    lens = [0, 1, 31, 32, 100, 128, 129, 299, 300, 301, -5, 2 ** 31 - 1, -2 ** 31]
    x = ref.make(len(lens), 300, 2, getattr(torch, DT[dtype]), decay, seed=70)
    x["lens"] = torch.tensor(lens, dtype=torch.int32)
    for b, n in enumerate(lens):
        n = max(0, min(300, n))
        for name in "rkv":
            x[name][b, n:] = (float("nan"), float("inf"), -float("inf"))[b % 3]
        if decay == "token":
            x["log_w"][b, n:] = (float("nan"), float("inf"), -float("inf"))[b % 3]
    y, s = compare(torch, x, ("lens", decay, dtype))
    for b, n in enumerate(lens):
        n = max(0, min(300, n))
        assert not y[b, n:].any()
        if n == 0:
            assert torch.equal(s[b].cpu(), x["state_in"][b])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_lens_in_segments(torch, dtype):
    """Few heads, so that a sequence is taken in segments, which begin before, at and behind its end."""
    T, lens = 2100, [0, 1, 511, 512, 513, 1024, 1500, 2099, 2100]
    x = ref.make(len(lens), T, 2, getattr(torch, DT[dtype]), "token", seed=72, resets=0.002)
    x["lens"] = torch.tensor(lens, dtype=torch.int32)
    for b, n in enumerate(lens):
        for name in ("r", "k", "v", "log_w"):
            x[name][b, n:] = (float("nan"), float("inf"), -float("inf"))[b % 3]
    y, s = compare(torch, x, ("lens in segments", dtype))
    for b, n in enumerate(lens):
        assert not y[b, n:].any()
    assert torch.equal(s[0].cpu(), x["state_in"][0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_resumes_in_place(torch, dtype):
    """Parts of a prompt one after the other, the state updated in place."""
    x = ref.make(2, 333, 3, getattr(torch, DT[dtype]), "token", seed=80)
    d = dev(x)
    s = d["state_in"].clone()
    ys = []
    for lo, hi in ((0, 1), (1, 130), (130, 162), (162, 333)):
        part = {n: d[n][:, lo:hi].contiguous() for n in ("r", "k", "v", "log_w")}
        y = torch.empty_like(part["r"])
        say("linattn resume", dtype, lo, hi)
        wkv.rwkv7_linattn_prefill(part["r"], part["log_w"], part["k"], part["v"], s, None, y, s)
        ys.append(y)
    yr, sr, ya, sa = ref.forward(x)
    bf16 = dtype == "bf16"
    # three more passes of a state through memory: exact (float32)
    ref.check("y", torch.cat(ys, 1), yr, ya, 333 + 4 * 32, bf16)
    ref.check("state", s, sr, sa, 333 + 4 * 32, False)


def test_prefill_without_state_out_and_empty(torch):
    x = ref.make(2, 50, 2, torch.bfloat16, "head", seed=90)
    y0, s0 = run(x)
    y1, s1 = run(x, want_state=False)
    assert s1 is None and torch.equal(y0, y1)
    d = dev(x)
    y, s = wkv.linattn(d["r"][:, :0].contiguous(), d["log_w"], d["k"][:, :0].contiguous(), d["v"][:, :0].contiguous(),
                       state_in=d["state_in"])
    assert y.shape == (2, 0, 2, 64) and torch.equal(s, d["state_in"])
    y, s = wkv.linattn(d["r"][:0], d["log_w"], d["k"][:0], d["v"][:0])
    assert y.shape == (0, 50, 2, 64) and s.shape == (0, 2, 64, 64)


@pytest.mark.parametrize("B,T,H", [(2, 300, 3), (1, 3000, 2)])
def test_prefill_repeats_bit_for_bit(torch, B, T, H):
    d = dev(ref.make(B, T, H, torch.bfloat16, "token", seed=91))
    args = (d["r"], d["log_w"], d["k"], d["v"])
    y0, s0 = wkv.linattn(*args, state_in=d["state_in"])
    for _ in range(5):
        y, s = wkv.linattn(*args, state_in=d["state_in"])
        assert torch.equal(y, y0) and torch.equal(s, s0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("B,H,state", [(1, 1, True), (3, 5, True), (7, 12, False), (300, 8, True)])
def test_step(torch, B, H, state, decay, dtype):
    x = ref.make(B, 1, H, getattr(torch, DT[dtype]), decay, seed=100 + B, state=state, resets=0.05)
    d = dev(x)
    say("linattn step", B, H, state, decay, dtype)
    y, s = wkv.linattn_step(d["r"], d["log_w"], d["k"], d["v"], d["state_in"])
    yr, sr, ya, sa = ref.forward(x)
    ref.check("y", y, yr, ya, 1, dtype == "bf16")
    ref.check("state", s, sr, sa, 1, False)
    if state:  # in place, the same bits
        s2, y2 = d["state_in"].clone(), torch.empty_like(y)
        wkv.rwkv7_linattn_step(d["r"], d["log_w"], d["k"], d["v"], s2, y2, s2)
        assert torch.equal(s, s2) and torch.equal(y, y2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_steps(torch, dtype):
    x = ref.make(2, 70, 3, getattr(torch, DT[dtype]), "token", seed=110)
    d = dev(x)
    cut = {n: d[n][:, :61].contiguous() for n in ("r", "log_w", "k", "v")}
    y0, s = wkv.linattn(cut["r"], cut["log_w"], cut["k"], cut["v"], state_in=d["state_in"])
    ys = [y0]
    for t in range(61, 70):
        one = {n: d[n][:, t:t + 1].contiguous() for n in ("r", "log_w", "k", "v")}
        y = torch.empty_like(one["r"])
        wkv.rwkv7_linattn_step(one["r"], one["log_w"], one["k"], one["v"], s, y, s)
        ys.append(y)
    yr, sr, ya, sa = ref.forward(x)
    ref.check("y", torch.cat(ys, 1), yr, ya, 70 + 9 * 32, dtype == "bf16")
    ref.check("state", s, sr, sa, 70 + 9 * 32, False)


def test_other_stream_and_graph(torch):
    """On a stream of the caller's, and captured in a graph whose replays read new inputs."""
    B, T, H = 2, 1100, 3
    x = ref.make(B, T, H, torch.bfloat16, "token", seed=120)
    d = dev(x)
    y, s = torch.empty_like(d["r"]), torch.empty_like(d["state_in"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def call():
        wkv.rwkv7_linattn_prefill(d["r"], d["log_w"], d["k"], d["v"], d["state_in"], None, y, s, stream=st)

    call()
    st.synchronize()
    yr, sr, ya, sa = ref.forward(x)
    ref.check("y", y, yr, ya, T, True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for seed in (121, 122, 123):
        z = ref.make(B, T, H, torch.bfloat16, "token", seed=seed)
        for n in ("r", "k", "v", "log_w", "state_in"):
            d[n].copy_(z[n])
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        y1, s1 = y.clone(), s.clone()
        call()  # the eager call between replays
        torch.cuda.synchronize()
        assert torch.equal(y, y1) and torch.equal(s, s1)
        yr, sr, ya, sa = ref.forward(z)
        ref.check("y", y1, yr, ya, T, True)
        ref.check("state", s1, sr, sa, T, False)
