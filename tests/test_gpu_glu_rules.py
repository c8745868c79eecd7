"""Few rows of many channels in the gated linear unit: those that go by tiles and sums in parts, and those beside them that
do not, with operands in the middle of larger buffers of NaN and outputs next to what has to stay."""
import pytest

from linear_rnn_amd import wkv
from tests import glu_ref as ref
from tests.gpu_util import new_stream, say

pytestmark = pytest.mark.gpu
ACT = {"sigmoid": wkv.RWKV7_ACT_SIGMOID, "silu": wkv.RWKV7_ACT_SILU, "gelu": wkv.RWKV7_ACT_GELU, "relu2": wkv.RWKV7_ACT_RELU2}


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,D,F", [(1, 16384, 256), (1, 4096, 256), (17, 16384, 100), (32, 8192, 512), (32, 4096, 2048), (32, 4096, 4096),
                                   (20, 8190, 1002), (16, 8192, 260), (32, 30002, 66), (3, 1 << 20, 8)])
def test_few_rows_of_many_channels(torch, M, D, F, dtype):
    say("glu few rows, many channels", M, D, F, dtype)
    act = ref.ACTS[(M + D // 2 + F // 2) % 4]
    dt = getattr(torch, dtype)
    x = ref.make(M, D, F, dt, seed=M + D + F)
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
    h = torch.empty_like(got[0])
    wkv.rwkv7_glu_forward(d["x"], d["w_gate"], d["w_up"], h, None, None, act=ACT[act])
    assert torch.equal(h, got[0])


# no workspace, as the header says, and with one
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,D,F,none", [(1, 1024, 8, True), (32, 1024, 2, True), (32, 1024, 5504, True), (17, 768, 16384, True), (32, 2, 100, True),
                                        (32, 16384, 256, False), (32, 8192, 512, False)])
def test_capture(torch, M, D, F, none, dtype):
    """On a stream without a workspace; a call that needs one is refused there and can be captured behind an eager one."""
    say("glu few rows, capture", M, D, F, dtype)
    x = ref.make(M, D, F, getattr(torch, dtype), seed=5)
    d = {n: x[n].cuda() for n in ("x", "w_gate", "w_up")}
    h = torch.empty(M, F, dtype=d["x"].dtype, device="cuda")
    want, stream = ref.forward(x["x"], x["w_gate"], x["w_up"], "silu")["h"], new_stream()
    torch.cuda.synchronize()

    def call():
        wkv.rwkv7_glu_forward(d["x"], d["w_gate"], d["w_up"], h, None, None, act=ACT["silu"], stream=stream)

    g, refused = torch.cuda.CUDAGraph(), False
    with torch.cuda.graph(g, stream=stream):
        try:
            call()
        except wkv.Rwkv7Error:
            refused = True
    assert refused == (not none)
    if refused:
        call()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            call()
    eager = wkv.glu(d["x"], d["w_gate"], d["w_up"], act=ACT["silu"])[0]
    for _ in range(3):
        h.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref.check("h", h, want)
        assert torch.equal(h, eager)
