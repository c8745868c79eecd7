"""The gated linear recurrence by single channels (1 to 3 of a row's channels behind a multiple of 64): many units walk
their tokens whatever their number, without the workspace, few pass maps on."""
import pytest

from linear_rnn_amd import wkv
from tests import gscan_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def cuda(x):
    return {n: t.cuda() for n, t in x.items()}


@pytest.mark.parametrize("B,T,D", [(160, 700, 1), (80, 700, 65), (82, 1300, 66), (54, 700, 131), (2, 220, 65)])
def test_many_units_need_no_workspace(torch, B, T, D):
    """On a stream without a workspace, under capture, where one cannot be had."""
    say("gscan single channels, capture", B, T, D)
    x = ref.make(B, T, D, torch.bfloat16, seed=T + D)
    d = cuda(x)
    y, s = torch.empty_like(d["x"]), torch.empty_like(d["state_in"])
    stream, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        wkv.rwkv7_gscan_prefill(d["x"], d["log_w"], d["state_in"], None, y, s, input=wkv.RWKV7_INPUT_MIX, stream=stream)
    want = ref.forward(x["x"], x["log_w"], x["state_in"], None, "mix")
    for _ in range(3):
        y.zero_(), s.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref.check("y", y, want["y"])
        ref.check("state", s, want["state"])
    y1, s1 = wkv.gscan(d["x"], d["log_w"], d["state_in"], input=wkv.RWKV7_INPUT_MIX)
    assert torch.equal(y1, y) and torch.equal(s1, s)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,T,D", [(159, 9000, 1), (160, 9000, 1), (1, 9000, 65), (3, 225, 65), (3, 257, 65), (64, 700, 65), (64, 1500, 65)])
def test_both_sides_of_the_rule(torch, B, T, D, dtype):
    say("gscan single channels", B, T, D, dtype)
    x = ref.make(B, T, D, getattr(torch, dtype), seed=B + T)
    d = cuda(x)
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"], input=wkv.RWKV7_INPUT_NORM)
    want = ref.forward(x["x"], x["log_w"], x["state_in"], None, "norm")
    ref.check("y", y, want["y"])
    ref.check("state", s, want["state"])
