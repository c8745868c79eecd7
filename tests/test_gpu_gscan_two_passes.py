"""Gradients of the gated linear recurrence over many tiles a sequence, in two passes above 160 (64 where D leaves one to
three of 64 channels over) and in one below, of padded batches: lengths that end before, at and behind a tile's edge, in the first tiles and in the last, anything behind them."""
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


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,D", [(20481, 20), (20600, 103), (9000, 64), (20480, 24), (2200, 65), (2081, 67), (4500, 130)])
def test_padded_batch(torch, T, D, dtype):
    tile = 32 if D % 64 in (1, 2, 3) else 128
    lens = [0, 1, tile - 1, tile, 64 * tile + 1, T - 1, T, -3, T + 7]
    B = len(lens)
    assert T > 64 * tile and D >= 16
    say("gscan two passes, padded", B, T, D, dtype)
    x = ref.make(B, T, D, getattr(torch, dtype), seed=T + D)
    for n, v in (("x", float("nan")), ("log_w", float("nan")), ("dy", float("inf"))):
        for b, m in enumerate(lens):
            x[n][b, max(m, 0):] = v
    d = {n: t.cuda() for n, t in x.items()}
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = ref.backward(x["x"], x["log_w"], x["state_in"], lens, x["dy"], x["dstate_out"], "norm")
    got = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], lens=dl, dstate_out=d["dstate_out"],
                             input=wkv.RWKV7_INPUT_NORM)
    for n, v in want.items():
        ref.check(n, got[n], v)
    for b, m in enumerate(lens):
        assert not got["dx"][b, max(m, 0):].any() and not got["dlog_w"][b, max(m, 0):].any()
    # the gradient of the state in place
    place, dx, dw = d["dstate_out"].clone(), torch.empty_like(got["dx"]), torch.empty_like(got["dlog_w"])
    wkv.rwkv7_gscan_backward(d["x"], d["log_w"], d["state_in"], dl, d["dy"], place, dx, dw, place, input=wkv.RWKV7_INPUT_NORM)
    assert torch.equal(place, got["dstate_in"]) and torch.equal(dx, got["dx"]) and torch.equal(dw, got["dlog_w"])


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,T,D", [(1, 20480, 64), (3, 20000, 100), (2, 12000, 1024)])
def test_one_pass_without_waiting(torch, B, T, D, dtype):
    """Up to 160 tiles whose workgroups leave them to the second kernel: the same bits."""
    import ctypes
    polls = getattr(ctypes.CDLL(wkv.LIB_PATH), "_ZN5rwkv715set_gscan_pollsEi")
    say("gscan one pass without waiting", B, T, D, dtype)
    d = {n: t.cuda() for n, t in ref.make(B, T, D, getattr(torch, dtype), seed=T).items()}

    def call():
        out = wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"], input=wkv.RWKV7_INPUT_MIX)
        torch.cuda.synchronize()
        return out

    want = call()
    polls(0)
    try:
        for _ in range(3):
            got = call()
            assert all(torch.equal(got[n], want[n]) for n in want)
    finally:
        polls(64)
