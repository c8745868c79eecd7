"""Gradients of the linear attention whose states between blocks pass the workspace's 1 GiB, so that the heads are taken in
slabs, against float64 (computed on the device)."""
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


def on_device(torch, x):
    with torch.device("cuda"):
        return ref.backward(x)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_border_inside_a_batch_entry(torch, decay, dtype):
    """9,009 heads of 300 tokens: 1.2 GB of states and gradients (float32: 2.1), parted between two heads of one sequence."""
    B, T, H = 91, 300, 99
    say("linattn slabs", decay, dtype)
    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(17)

    def normal(*shape, scale=1.0, t=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=t).normal_(0, scale, generator=g)

    x = {"r": normal(B, T, H, 64, t=dt), "k": normal(B, T, H, 64, scale=0.125, t=dt), "v": normal(B, T, H, 64, t=dt),
         "dy": normal(B, T, H, 64, t=dt), "state_in": normal(B, H, 64, 64, scale=0.1),
         "dstate_out": normal(B, H, 64, 64, scale=0.1)}
    shape = (H,) if decay == "head" else (B, T, H)
    x["log_w"] = -torch.exp(torch.rand(shape, device="cuda", generator=g) * 4.5 - 5.0)
    x["lens"] = torch.full((B,), T, dtype=torch.int32, device="cuda")
    x["lens"][::7] = torch.arange(0, 13, device="cuda", dtype=torch.int32) * 25
    keep = x["dstate_out"].clone()
    out = wkv.linattn_backward(x["r"], x["log_w"], x["k"], x["v"], x["dy"], state_in=x["state_in"], lens=x["lens"],
                               dstate_out=x["dstate_out"])
    # the gradient of the state in place, as the slabs share nothing of the caller's
    again = {n: torch.empty_like(out[n]) for n in ("dr", "dlog_w", "dk", "dv")}
    wkv.rwkv7_linattn_backward(x["r"], x["log_w"], x["k"], x["v"], x["state_in"], x["lens"], x["dy"], keep, again["dr"],
                               again["dlog_w"], again["dk"], again["dv"], keep)
    torch.cuda.synchronize()
    assert torch.equal(keep, out["dstate_in"]) and all(torch.equal(again[n], out[n]) for n in again)
    total = [torch.zeros(H, dtype=ref.F64, device="cuda") for _ in range(2)]
    for b in range(0, B, 13):
        part = {n: (t if n == "log_w" and decay == "head" else t[b:b + 13]) for n, t in x.items()}
        want, mag = on_device(torch, part)
        for n in ("dr", "dk", "dv", "dstate_in"):
            ref.check(n, out[n][b:b + 13], want[n].cpu(), mag[n].cpu(), T, dtype == "bfloat16" and n != "dstate_in")
        if decay == "token":  # twice the roundings of a state, and the product of two states (as for the other gradients)
            ref.check("dlog_w", out["dlog_w"][b:b + 13], want["dlog_w"].cpu(), mag["dlog_w"].cpu(), 2 * T + 32 * 130, False)
        else:
            total[0] += want["dlog_w"]
            total[1] += mag["dlog_w"]
        del want, mag
    if decay == "head":
        ref.check("dlog_w", out["dlog_w"], total[0].cpu(), total[1].cpu(), 2 * T + 32 * 130 + 32 * (B + T), False)


def test_one_head_larger_than_the_workspace(torch):
    """3.5 million tokens of two heads: 1.1 GB of states each. Their decays (log w under -0.05, about -0.55) forget what is
    500 tokens away, so float64 over the last and the first 1,700 tokens holds for 1,200 of them."""
    B, T, H, n, run = 1, 3_500_000, 2, 1700, 500
    say("linattn slabs", "one head", T)
    g = torch.Generator(device="cuda").manual_seed(18)

    def normal(scale=1.0):
        return torch.empty(B, T, H, 64, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=g)

    x = {"r": normal(), "k": normal(0.125), "v": normal(), "dy": normal(), "state_in": None, "dstate_out": None, "lens": None}
    x["log_w"] = -0.05 - torch.rand(B, T, H, device="cuda", generator=g)
    out = wkv.linattn_backward(x["r"], x["log_w"], x["k"], x["v"], x["dy"])
    torch.cuda.synchronize()
    for lo, keep in ((T - n, slice(run, n)), (0, slice(0, n - run))):
        part = {k: (t[:, lo:lo + n].contiguous() if t is not None else None) for k, t in x.items()}
        want, mag = on_device(torch, part)
        for name in ("dr", "dk", "dv", "dlog_w"):
            f32 = name == "dlog_w"
            ref.check(name, out[name][:, lo:lo + n][:, keep], want[name][:, keep].cpu(), mag[name][:, keep].cpu(),
                      2 * n + 32 * 130 if f32 else n, not f32)
    ref.check("dstate_in", out["dstate_in"], want["dstate_in"].cpu(), mag["dstate_in"].cpu(), n, False)


def test_workspace_is_bounded(torch):
    """A call whose states take 2.7 GB leaves at most the slabs' 1 GiB allocated (and what the runtime itself takes)."""
    B, T, H = 4, 16384, 64
    say("linattn slabs", "bounded")
    x = {n: torch.zeros(B, T, H, 64, device="cuda") for n in ("r", "k", "v", "dy", "dr", "dk", "dv")}
    log_w = torch.full((H,), -0.1, device="cuda")
    dlog_w = torch.empty_like(log_w)
    st = torch.cuda.Stream()

    def call(T):
        at = {n: t[:, :T].contiguous() if T < t.shape[1] else t for n, t in x.items()}
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        wkv.rwkv7_linattn_backward(at["r"], log_w, at["k"], at["v"], None, None, at["dy"], None, at["dr"], dlog_w, at["dk"],
                                   at["dv"], None, stream=st)
        torch.cuda.synchronize()
        return free - torch.cuda.mem_get_info()[0]

    call(1)  # code and kernel arguments
    assert call(T) <= (1 << 30) + (64 << 20)
    assert call(T) <= 0
    assert not dlog_w.any()
