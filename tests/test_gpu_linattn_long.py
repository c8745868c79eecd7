"""The linear attention where a workgroup takes many blocks and a segment many pieces, against float64 (computed on the
device, elementwise and by sums, as the sequences are long)."""
import pytest

from linear_rnn_amd import wkv
from tests import linattn_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f32": "float32"}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def dev(x):
    return {n: (t.cuda() if t is not None else None) for n, t in x.items()}


def pad(torch, x, lens):
    """Lengths, and what nothing may read behind them."""
    x["lens"] = torch.tensor(lens, dtype=torch.int32)
    for b, n in enumerate(lens):
        for name in ("r", "k", "v", "dy") + (("log_w",) if x["log_w"].dim() == 3 else ()):
            x[name][b, n:] = (NAN, INF, -INF)[b % 3]


def forward(torch, d):
    with torch.device("cuda"):
        return [t.cpu() for t in ref.forward(d)]


def backward(torch, d):
    with torch.device("cuda"):
        out, mag = ref.backward(d)
    return {n: t.cpu() for n, t in out.items()}, {n: t.cpu() for n, t in mag.items()}


def prompt(torch, x, what):
    say("linattn long", what)
    T, bf16 = x["r"].shape[1], x["r"].dtype == torch.bfloat16
    d = dev(x)
    y, s = wkv.linattn(d["r"], d["log_w"], d["k"], d["v"], state_in=d["state_in"], lens=d["lens"])
    torch.cuda.synchronize()
    yr, sr, ya, sa = forward(torch, d)
    ref.check("y", y, yr, ya, T, bf16)
    ref.check("state", s, sr, sa, T, False)
    return y, s


# More pieces of 512 tokens than there are compute units (256): segments of two or three pieces, so the states that are
# kept lie closer together than the pieces' sums, and the last segment may be shorter than the others.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,lens", [(1, 8191, 32, None), (4, 4500, 10, [4500, 2047, 1, 3600]), (2, 5500, 13, [5121, 5120])])
def test_segments_of_several_pieces(torch, B, T, H, lens, dtype):
    x = ref.make(B, T, H, getattr(torch, DT[dtype]), "token", seed=200 + B, resets=5e-4)
    if lens:
        pad(torch, x, lens)
    prompt(torch, x, ("segments of several pieces", B, T, H, dtype))


# As many heads as compute units: a workgroup takes a whole sequence, and with 11 blocks comes round to each of the
# four places that log w of a block may have more than twice.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [None, [1300, 1299, 1153, 1152, 1025, 640, 33, 0]])
def test_many_blocks_in_a_row(torch, lens, dtype):
    x = ref.make(8, 1300, 32, getattr(torch, DT[dtype]), "token", seed=210, resets=2e-3)
    if lens:
        pad(torch, x, lens)
    y, s = prompt(torch, x, ("many blocks", dtype))
    if lens:
        assert torch.equal(s[7].cpu(), x["state_in"][7]) and not y[7].any()


# Gradients with four to eleven blocks of a sequence to a workgroup, each with the next one's rows on their way.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("B,T,H,lens", [(2, 900, 64, None), (2, 900, 64, [899, 385]), (8, 1300, 32, None)])
def test_gradients_of_many_blocks(torch, B, T, H, lens, decay, dtype):
    x = ref.make(B, T, H, getattr(torch, DT[dtype]), decay, seed=220 + T, resets=2e-3 if decay == "token" else 0.0)
    if lens:
        pad(torch, x, lens)
    say("linattn long", "gradients of many blocks", B, T, H, lens, decay, dtype)
    d = dev(x)
    got = wkv.linattn_backward(d["r"], d["log_w"], d["k"], d["v"], d["dy"], state_in=d["state_in"], lens=d["lens"],
                               dstate_out=d["dstate_out"])
    torch.cuda.synchronize()
    want, mag = backward(torch, d)
    for n in ("dr", "dk", "dv"):
        ref.check(n, got[n], want[n], mag[n], T, dtype == "bf16")
    # dlog_w: a state's sums and a gradient's, the 2 * 64 * 64 + 64 terms of the product of the two, of one decay for all
    # tokens also their sum (the count of linattn_ref in 32nds of a token)
    more = 32 * 130 + (32 * (B + T) if decay == "head" else 0)
    ref.check("dlog_w", got["dlog_w"], want["dlog_w"], mag["dlog_w"], 2 * T + more, False)
    ref.check("dstate_in", got["dstate_in"], want["dstate_in"], mag["dstate_in"], T, False)


def test_last_tokens_behind_32_bit_offsets(torch):
    """2.4e9 elements a tensor. log w is under -0.05 and about -0.55: what came more than 500 tokens before is forgotten
    (e^-25 at the most that can be, e^-240 in these draws), so float64 over the last 1,715 tokens of a few heads, from no state, holds
    for the last 1,215 of a call of 49,152; these begin 47,937 tokens in, not where a block does."""
    B, T, H, cut, run = 1, 49152, 768, 47937, 500
    heads = [0, 1, 383, 767]
    say("linattn last tokens behind 32-bit offsets")
    g = torch.Generator(device="cuda").manual_seed(9)

    def normal(scale=1.0):
        return torch.empty(B, T, H, 64, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=g)

    d = {"r": normal(), "k": normal(0.125), "v": normal(), "dy": normal(), "state_in": None, "dstate_out": None, "lens": None}
    d["log_w"] = -0.05 - torch.rand(B, T, H, device="cuda", generator=g)
    part = {n: (t[:, cut - run:, heads].contiguous() if t is not None else None) for n, t in d.items()}
    # the draws' sums over any run of 500 tokens
    assert float(part["log_w"].double().cumsum(1)[:, run - 1].max()) < -200
    n = T - cut + run
    y, s = wkv.linattn(d["r"], d["log_w"], d["k"], d["v"])
    torch.cuda.synchronize()
    yr, sr, ya, sa = forward(torch, part)
    ref.check("y", y[:, cut:, heads], yr[:, run:], ya[:, run:], n, True)
    ref.check("state", s[:, heads], sr, sa, n, False)
    del y, s
    got = wkv.linattn_backward(d["r"], d["log_w"], d["k"], d["v"], d["dy"])
    torch.cuda.synchronize()
    want, mag = backward(torch, part)
    for name in ("dr", "dk", "dv"):
        ref.check(name, got[name][:, cut:, heads], want[name][:, run:], mag[name][:, run:], n, True)
    ref.check("dlog_w", got["dlog_w"][:, cut:, heads], want["dlog_w"][:, run:], mag["dlog_w"][:, run:], 2 * n + 32 * 130, False)
