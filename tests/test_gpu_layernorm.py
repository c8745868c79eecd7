"""GPU parity of the layer norm over groups of channels, forward and backward, against float64."""
import pytest

from linear_rnn_amd import wkv
from tests import layernorm_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16"]


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def cuda(t):
    return None if t is None else t.cuda()


def both(torch, M, D, G, xk, yk, seed, affine=True, eps=1e-5, offset=1.0):
    say("layernorm", M, D, G, xk, yk, affine)
    x = ref.make(M, D, G, dt(torch, xk), dt(torch, yk), seed, offset)
    w, b = (x["weight"], x["bias"]) if affine else (None, None)
    y, mean, rstd = wkv.layernorm(x["x"].cuda(), cuda(w), cuda(b), groups=G, eps=eps, out_dtype=dt(torch, yk))
    torch.cuda.synchronize()
    want, lim = ref.forward(x["x"], w, b, G, eps), ref.forward_limits(x["x"], w, b, G, eps, dt(torch, yk))
    assert y.dtype == dt(torch, yk)
    for name, got, r, l in zip(("y", "mean", "rstd"), (y, mean, rstd), want, lim):
        ref.check(name, got, r, l)
    g = wkv.layernorm_backward(x["x"].cuda(), cuda(w), mean, rstd, x["dy"].cuda(), groups=G)
    torch.cuda.synchronize()
    m, s = mean.cpu(), rstd.cpu()
    gr, gl = ref.backward(x["x"], w, m, s, x["dy"], G), ref.backward_limits(x["x"], w, m, s, x["dy"], G)
    assert g["dx"].dtype == dt(torch, xk)
    for name in ("dx", "dweight", "dbias"):
        ref.check(name, g[name], gr[name], gl[name])
    return x, y, mean, rstd, g


@pytest.mark.parametrize("yk", KINDS)
@pytest.mark.parametrize("xk", KINDS)
@pytest.mark.parametrize("D", [1, 2, 7, 8, 16, 17, 63, 64, 65, 100, 128, 200, 256, 257, 512, 768, 1023, 1024, 1025, 1096, 2048,
                               2049, 4096, 4099, 8192, 8193, 12288, 16384, 16385, 20001])
def test_one_group(torch, D, xk, yk):
    """Every size at which another number of threads, of vectors or another kernel takes over."""
    both(torch, 5, D, 1, xk, yk, seed=D)


@pytest.mark.parametrize("xk,yk", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("G,n", [(2, 64), (12, 64), (16, 64), (32, 64), (33, 64), (64, 64), (100, 64), (3, 1), (5, 9), (40, 16),
                                 (7, 130), (2, 1000), (3, 4104), (2, 16385), (300, 8)])
@pytest.mark.parametrize("M", [1, 7, 300])
def test_groups(torch, M, G, n, xk, yk):
    if M * G * n > 2_000_000:
        M = 9
    both(torch, M, G * n, G, xk, yk, seed=M + G + n, eps=64e-5)


@pytest.mark.parametrize("xk", KINDS)
@pytest.mark.parametrize("M,D,G", [(5000, 64, 1), (4099, 128, 2), (2500, 771, 1), (3001, 1024, 16), (1301, 4096, 1), (701, 8192, 2),
                                   (523, 8192, 1)])
def test_many_rows(torch, M, D, G, xk):
    """Every workgroup takes several rows, and the sums over rows meet from all of them."""
    both(torch, M, D, G, xk, xk, seed=M)


def test_without_weight_bias_or_statistics(torch):
    x, y, mean, rstd, g = both(torch, 33, 192, 3, "bf16", "bf16", seed=1, affine=False)
    d = x["x"].cuda()
    y2, m2, r2 = wkv.layernorm(d, groups=3, want_stats=False)
    assert m2 is None and r2 is None and torch.equal(y, y2)
    g2 = wkv.layernorm_backward(d, None, mean, rstd, x["dy"].cuda(), groups=3, want_dweight=False)
    assert g2["dweight"] is None and torch.equal(g2["dx"], g["dx"])
    one = torch.empty(192, device="cuda")
    for which in (0, 1):  # one of the two sums alone
        dx = torch.empty_like(d)
        wkv.rwkv7_layernorm_backward(d, None, mean, rstd, x["dy"].cuda(), dx, *((one, None) if which == 0 else (None, one)),
                                     groups=3)
        assert torch.equal(one, g["dbias" if which else "dweight"]) and torch.equal(dx, g["dx"])


def test_leading_dimensions_and_empty(torch):
    x = ref.make(24, 128, 2, torch.float32, torch.float32, 2)
    d = x["x"].cuda()
    y, m, r = wkv.layernorm(d, groups=2)
    y3, m3, r3 = wkv.layernorm(d.view(2, 3, 4, 128), groups=2)
    assert torch.equal(y3.view(24, 128), y) and m3.shape == (2, 3, 4, 2) and torch.equal(r3.view(24, 2), r)
    y1, m1, _ = wkv.layernorm(d[0].contiguous(), groups=2)
    assert torch.equal(y1, y[0]) and m1.shape == (2,)
    y0, m0, r0 = wkv.layernorm(d[:0])
    assert y0.shape == (0, 128) and m0.shape == (0, 1)
    g = wkv.layernorm_backward(d[:0], None, m0, r0, d[:0])
    assert g["dx"].shape == (0, 128) and not g["dweight"].any() and not g["dbias"].any()


@pytest.mark.parametrize("D", [64, 771, 4096, 20000])
def test_constant_rows_and_rows_that_are_not_finite(torch, D):
    """A constant row has variance 0; a row with a NaN or an infinity spoils itself and no other."""
    x = ref.make(6, D, 1, torch.float32, torch.float32, 3)["x"]
    x[1] = 3.0
    x[3, D // 2] = float("nan")
    x[4, 0] = float("inf")
    y, mean, rstd = wkv.layernorm(x.cuda())
    want, lim = ref.forward(x, None, None, 1, 1e-5), ref.forward_limits(x, None, None, 1, 1e-5, torch.float32)
    good = [0, 1, 2, 5]
    ref.check("y", y[good], want[0][good], lim[0][good])
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    # 3.0 is exact in every partial sum's mean up to its rounding: y is at most that rounding over sqrt(eps)
    assert y[1].abs().max() <= 64 * 2.0 ** -24 * 3.0 / 1e-5 ** 0.5


def test_large_offset(torch):
    """Rows whose mean is far larger than their spread: the variance is not a difference of squares."""
    both(torch, 64, 1024, 1, "f32", "f32", seed=4, offset=0.0)
    x = ref.make(16, 1024, 1, torch.float32, torch.float32, 5, offset=0.0)["x"] + 1000.0
    y, mean, rstd = wkv.layernorm(x.cuda())
    want, lim = ref.forward(x, None, None, 1, 1e-5), ref.forward_limits(x, None, None, 1, 1e-5, torch.float32)
    for name, got, r, l in zip(("y", "mean", "rstd"), (y, mean, rstd), want, lim):
        ref.check(name, got, r, l)


def test_repeats_streams_and_graph(torch):
    M, D, G = 900, 512, 8
    x = ref.make(M, D, G, torch.bfloat16, torch.bfloat16, 6)
    d, w, b, dy = x["x"].cuda(), x["weight"].cuda(), x["bias"].cuda(), x["dy"].cuda()
    st = torch.cuda.Stream()
    y, dx = torch.empty_like(d), torch.empty_like(d)
    mean, rstd = (torch.empty(M, G, device="cuda") for _ in range(2))
    dw, db = (torch.empty(D, device="cuda") for _ in range(2))
    st.wait_stream(torch.cuda.current_stream())

    def call():
        wkv.rwkv7_layernorm_forward(d, w, b, y, mean, rstd, groups=G, stream=st)
        wkv.rwkv7_layernorm_backward(d, w, mean, rstd, dy, dx, dw, db, groups=G, stream=st)

    call()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for seed in (7, 8, 9):
        z = ref.make(M, D, G, torch.bfloat16, torch.bfloat16, seed)
        d.copy_(z["x"])
        dy.copy_(z["dy"])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in (y, mean, rstd, dx, dw, db)]
        for _ in range(3):
            call()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(first, (y, mean, rstd, dx, dw, db)))
        m, s = mean.cpu(), rstd.cpu()
        gr = ref.backward(z["x"], x["weight"], m, s, z["dy"], G)
        gl = ref.backward_limits(z["x"], x["weight"], m, s, z["dy"], G)
        for name, got in (("dx", dx), ("dweight", dw), ("dbias", db)):
            ref.check(name, got, gr[name], gl[name])
