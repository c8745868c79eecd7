"""The gated linear recurrence with more workgroups than one launch holds: sequences on both sides of the launches' edges
against float64, and against a call of their own, bit for bit."""
import pytest

from linear_rnn_amd import wkv
from tests import gscan_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
B = (1 << 22) + 5
# both sides of the edges of launches of 2^20 (1024 threads) and 2^22 (256) workgroups, the first and the last
EDGES = [slice(0, 3), slice((1 << 20) - 3, (1 << 20) + 3), slice((1 << 21) - 3, (1 << 21) + 3), slice((1 << 22) - 3, B)]


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def make(torch, B, T, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, kind=torch.float32):
        return torch.empty(shape, dtype=kind, device="cuda").normal_(generator=g)

    return {"x": n(B, T, D, kind=dtype), "log_w": torch.empty(B, T, D, device="cuda").uniform_(-2.0, -0.01, generator=g),
            "dy": n(B, T, D, kind=dtype), "state_in": n(B, D), "dstate_out": n(B, D)}


def part(d, rows):
    return {n: t[rows].clone() for n, t in d.items()}


def backward(d):
    return wkv.gscan_backward(d["x"], d["log_w"], d["dy"], d["state_in"], dstate_out=d["dstate_out"])


def check_backward(torch, d, got):
    for rows in EDGES:
        some = part(d, rows)
        own = backward(some)
        h = {n: t.cpu() for n, t in some.items()}
        want = ref.backward(h["x"], h["log_w"], h["state_in"], None, h["dy"], h["dstate_out"], "plain")
        for n, v in want.items():
            ref.check(n, got[n][rows], v)
            assert torch.equal(got[n][rows], own[n]), n


@pytest.mark.parametrize("T,D", [(1, 1), (1, 4), (7, 1)])
def test_prompt(torch, T, D):
    say("gscan many sequences, prompt", B, T, D)
    d = make(torch, B, T, D, torch.float32, 1)
    y, s = wkv.gscan(d["x"], d["log_w"], d["state_in"])
    for rows in EDGES:
        some = part(d, rows)
        y1, s1 = wkv.gscan(some["x"], some["log_w"], some["state_in"])
        assert torch.equal(y[rows], y1) and torch.equal(s[rows], s1)
        want = ref.forward(some["x"].cpu(), some["log_w"].cpu(), some["state_in"].cpu(), None, "plain")
        ref.check("y", y[rows], want["y"])
        ref.check("state", s[rows], want["state"])


def test_gradients_without_tokens(torch):
    """Only the join runs: every sequence's gradient of the final state is that of the initial one."""
    say("gscan many sequences, gradients of no tokens", B)
    d = make(torch, B, 0, 1, torch.float32, 2)
    assert torch.equal(backward(d)["dstate_in"], d["dstate_out"])
    ds = d["dstate_out"].clone()
    wkv.rwkv7_gscan_backward(d["x"], d["log_w"], d["state_in"], None, d["dy"], ds, d["x"].clone(), d["log_w"].clone(), ds)
    assert torch.equal(ds, d["dstate_out"])


@pytest.mark.parametrize("T,D", [(33, 1), (1, 16)])
def test_gradients(torch, T, D):
    """Two passes with the join between them, and the one pass of a single tile."""
    say("gscan many sequences, gradients", B, T, D)
    d = make(torch, B, T, D, torch.float32, 3)
    check_backward(torch, d, backward(d))


def test_tiles_that_pass_maps_on(torch):
    """Workgroups take numbers over several launches."""
    B, T, D = 240_000, 2100, 4
    say("gscan many sequences, passing maps on", B, T, D)
    d = make(torch, B, 1, D, torch.bfloat16, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    lw = torch.empty(B, T, D, device="cuda").uniform_(-0.5, -0.01, generator=g)
    y, s = wkv.gscan(x, lw, d["state_in"])
    for rows in (slice(0, 200), slice(116_400, 116_600), slice(B - 200, B)):  # 2^21 workgroups end in the middle of the last tile
        y1, s1 = wkv.gscan(x[rows].clone(), lw[rows].clone(), d["state_in"][rows].clone())
        assert torch.equal(y[rows], y1) and torch.equal(s[rows], s1)
    rows = slice(B - 2, B)
    want = ref.forward(x[rows].cpu(), lw[rows].cpu(), d["state_in"][rows].cpu(), None, "plain")
    ref.check("y", y[rows], want["y"])
    ref.check("state", s[rows], want["state"])
