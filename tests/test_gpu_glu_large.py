"""The gated linear unit where its operands are large for one launch or for the workspace."""
import pytest

from linear_rnn_amd import wkv
from tests import glu_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def test_weights_whose_copies_take_several_launches(torch):
    """Copies of two weights of 4.3e9 elements are 1.07e9 threads, more than one launch has; every channel of k counts in
    every column, some of which are looked at."""
    M, D, F = 2, 65536, 65537
    assert 2 * D * ((F + 63) // 64 * 64) // 8 > 1 << 30
    say("glu weights of several launches", M, D, F)
    g = torch.Generator(device="cuda").manual_seed(1)
    wg, wu = (torch.empty(D, F, dtype=torch.bfloat16, device="cuda").normal_(0, D ** -0.5, generator=g) for _ in range(2))
    x = torch.empty(M, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    h, gate, up = wkv.glu(x, wg, wu, act=wkv.RWKV7_ACT_SILU, want_pre=True)
    for cols in (slice(0, 5), slice(32768, 32773), slice(F - 5, F)):
        want = ref.forward(x.cpu(), wg[:, cols].cpu(), wu[:, cols].cpu(), "silu")
        for n, t in (("h", h), ("gate", gate), ("up", up)):
            ref.check(n, t[:, cols], want[n])



def make(torch, M, D, F, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, scale=1.0):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0, scale, generator=g)

    return {"x": n(M, D), "w_gate": n(D, F, scale=D ** -0.5), "w_up": n(D, F, scale=D ** -0.5), "gate": n(M, F), "up": n(M, F),
            "dh": n(M, F)}


# rows whose dg and du (and x's copies, where D is odd or float32) pass 4 GiB: two slabs, or three, the last one shorter;
# weights' gradients in one part and in several
@pytest.mark.parametrize("dtype,M,D,F", [("bfloat16", 1200, 8, 1 << 20), ("bfloat16", 1300, 9, (1 << 20) - 1), ("bfloat16", 300_000, 8, 4096),
                                         ("float32", 500, 5, 1 << 20), ("float32", 200_000, 24, 4100), ("bfloat16", 280_000, 512, 4096)])
def test_gradients_in_slabs_of_rows(torch, dtype, M, D, F):
    """Some rows of dx, on both sides of every slab's edge, and some columns of the weights' gradients, which every row
    counts in, against float64 on the device, also of calls that want only one of them; a graph's replays give the same bits."""
    say("glu slabs", dtype, M, D, F)
    x = make(torch, M, D, F, getattr(torch, dtype), 2)

    def call(out, stream=None):
        wkv.rwkv7_glu_backward(x["x"], x["w_gate"], x["w_up"], x["gate"], x["up"], x["dh"], out["dx"], out["dw_gate"], out["dw_up"],
                               act=wkv.RWKV7_ACT_SILU, stream=stream)

    def room():
        o = {"dx": torch.full_like(x["x"], 7.0), "dw_gate": torch.full_like(x["w_gate"], 7.0), "dw_up": torch.full_like(x["w_up"], 7.0)}
        torch.cuda.synchronize()
        return o

    copied = dtype == "float32" or D % 8 != 0
    row = (3 if dtype == "float32" else 1) * 2 * (2 * ((F + 63) // 64 * 64) + ((D + 7) // 8 * 8 if copied else 0))
    most = (1 << 32) // row // 128 * 128
    slabs = -(-M // most)
    assert slabs >= 2
    step = -(-(-(-M // slabs)) // 128) * 128
    edges = sorted({r for e in range(0, M + 1, step) for r in (e - 2, e - 1, e, e + 1) if 0 <= r < M} | {M - 2, M - 1})
    rows = torch.tensor(edges, device="cuda")
    names = ("x", "w_gate", "w_up", "gate", "up", "dh")
    want = {"dx": ref.backward(*(x[n] if n in ("w_gate", "w_up") else x[n][rows] for n in names), "silu")["dx"]}
    columns = (slice(0, 8), slice(F - 8, F))
    for cols in columns:
        some = ref.backward(*(x[n] if n == "x" else x[n][:, cols] for n in names), "silu")
        want.update({(n, cols.start): some[n] for n in ("dw_gate", "dw_up")})

    def verify(out):
        if out["dx"] is not None:
            ref.check("dx", out["dx"][rows], tuple(t.cpu() for t in want["dx"]))
        for n in ("dw_gate", "dw_up"):
            for cols in columns if out[n] is not None else ():
                v = tuple(t.cpu() for t in want[n, cols.start])
                ref.check(n, out[n][:, cols], v)
                ref.norm(n, out[n][:, cols], v, M)

    got = room()
    call(got)
    torch.cuda.synchronize()
    verify(got)
    for left_out in (("dx",), ("dw_gate", "dw_up")):
        out = {**room(), **dict.fromkeys(left_out)}
        call(out)
        torch.cuda.synchronize()
        verify(out)
    stream, g, out = torch.cuda.Stream(), torch.cuda.CUDAGraph(), room()
    call(out, stream)
    stream.synchronize()
    with torch.cuda.graph(g, stream=stream):
        call(out, stream)
    for _ in range(3):
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], got[n]) for n in got)


@pytest.mark.parametrize("dtype,M,D,F", [("bfloat16", 2_200_000, 1001, 24), ("float32", 115_000, 6400, 1024)])
def test_forward_in_slabs_of_rows(torch, dtype, M, D, F):
    """x whose copies pass 4 GiB: every row beside the same rows in a call of their own, bit for bit, and some against
    float64."""
    say("glu forward slabs", dtype, M, D, F)
    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(M, D, dtype=dt, device="cuda").normal_(generator=g)
    wg, wu = (torch.empty(D, F, dtype=dt, device="cuda").normal_(0, D ** -0.5, generator=g) for _ in range(2))
    assert M * ((D + 63) // 64 * 64) * 2 * (3 if dtype == "float32" else 1) > 1 << 32
    got = wkv.glu(x, wg, wu, want_pre=True)
    h, _, _ = wkv.glu(x, wg, wu)
    assert torch.equal(h, got[0])
    rows = torch.cat([torch.arange(max(0, e - 3), min(M, e + 3), device="cuda") for e in range(0, M + 1, 128)])
    rows = rows[torch.randperm(len(rows), device="cuda", generator=g)[:3000]]
    with torch.device("cuda"):
        want = ref.forward(x[rows], wg, wu, "silu")
    for n, t in zip(("h", "gate", "up"), got):
        ref.check(n, t[rows], tuple(v.cpu() for v in want[n]))
    half = M // 2 // 128 * 128
    for some in (slice(0, half), slice(half, M)):  # tiles of the same rows, in other slabs
        again = wkv.glu(x[some].clone(), wg, wu, want_pre=True)
        assert all(torch.equal(a, b[some]) for a, b in zip(again, got))


def test_workspace_is_bounded(torch):
    """Gradients whose dg and du take 8.6 GB leave the slabs' 4 GiB allocated, and the weights' sums and parts."""
    M, D, F = 262144, 64, 8192
    say("glu slabs bounded", M, D, F)
    x = make(torch, M, D, F, torch.bfloat16, 4)
    out = {"dx": torch.empty_like(x["x"]), "dw_gate": torch.empty_like(x["w_gate"]), "dw_up": torch.empty_like(x["w_up"])}
    stream = torch.cuda.Stream()

    def call(rows):
        at = {n: (t if "w_" in n else t[:rows]) for n, t in {**x, **out}.items()}
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        wkv.rwkv7_glu_backward(at["x"], at["w_gate"], at["w_up"], at["gate"], at["up"], at["dh"], at["dx"], at["dw_gate"], at["dw_up"],
                               stream=stream)
        torch.cuda.synchronize()
        return free - torch.cuda.mem_get_info()[0]

    call(1)  # code and kernel arguments
    # two sums of at most 256 MiB of parts each, and the weights' sum
    assert call(M) <= (1 << 32) + (1 << 29) + 8 * D * F + (64 << 20)
    assert call(M) <= 0
