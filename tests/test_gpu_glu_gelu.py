"""GELU's lower tail: g Phi(g) and its slope keep their digits where Phi is small, in every way that the unit goes.

Bounds, relative, in float32's half steps U = 2^-24. Phi(g) = erfc(-g / sqrt 2) / 2: the argument carries its constant's and
its product's rounding, 2 U, which erfc passes on by |t erfc'(t) / erfc(t)| <= g^2 + 2 for t = -g / sqrt 2 above 0 (from
erfc(t) >= 2 / sqrt pi exp(-t^2) / (t + sqrt(t^2 + 2))) and by less than 2 below; erfc itself is taken as 8 U, the products
around it as 2 U. phi(g) = exp2(-g^2 log2(e) / 2) / sqrt(2 pi): its argument carries 3 U of g^2 / 2, the exponential 2 U, the
products and constants 4 U. Values below the smallest normal float32 may count as 0."""
import math

import pytest

from linear_rnn_amd import wkv
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -24, 2.0 ** -126


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def gelu(torch, g):
    """g Phi(g) and its slope in float64, and how far float32 evaluations may be off each."""
    g = g.double().cpu()
    c = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
    p = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    e_c = (2 * (g * g + 2) + 10) * U * c + TINY
    e_p = (1.5 * g * g + 6) * U * (g * p).abs() + g.abs() * TINY
    a, s = g * c, c + g * p
    return a, g.abs() * e_c + U * a.abs(), s, e_c + e_p + U * s.abs()


def test_bound_of_the_tail(torch):
    """The reference itself against the tail's continued fraction, and the inequality that its bound uses."""
    for g in (-2.0, -4.0, -5.5, -8.0, -10.0):
        t = -g / math.sqrt(2)
        f = 0.0
        for k in range(400, 0, -1):  # erfc(t) = exp(-t^2) / sqrt pi / (t + 1/2 / (t + 1 / (t + 3/2 / (t + ...))))
            f = k / 2 / (t + f)
        want = math.exp(-t * t) / math.sqrt(math.pi) / (t + f) / 2
        a, _, s, _ = gelu(torch, torch.tensor([g], dtype=torch.float64))
        assert abs(float(a) / (g * want) - 1) <= 1e-12
        assert abs(float(s) - (want + g * math.exp(-g * g / 2) / math.sqrt(2 * math.pi))) <= 1e-12 * abs(float(s))
        slope = 2 / math.sqrt(math.pi) * math.exp(-t * t)
        assert t * slope / (2 * want) <= g * g + 2


def near(name, got, want, e, steps):
    """`steps`: roundings to the outputs' type on the way."""
    half = steps * (float(2.0 ** -8) if got.element_size() == 2 else 0.0)
    over = ((got.double().cpu() - want).abs() - e - half * (want.abs() + e)).max()
    assert over <= 0, "%s: %g over its bound" % (name, float(over))


# rows, channels, hidden channels: few rows, the float32 instructions, pieces, tiles whole and in parts
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("M,D,F", [(4, 2, 1000), (300, 2, 64), (300, 1024, 64), (515, 770, 2049), (4096, 768, 2048)])
def test_forward(torch, M, D, F, dtype):
    say("glu gelu tail", M, D, F, dtype)
    dt = getattr(torch, dtype)
    # g = x_0 times a factor of the column near 1, u = 1: each pre-activation is one product, whatever the order of the sum
    x = torch.zeros(M, D, dtype=dt, device="cuda")
    x[:, 0] = torch.linspace(-10.0, -2.0, M, device="cuda").to(dt)
    x[:, 1] = 1
    wg, wu = (torch.zeros(D, F, dtype=dt, device="cuda") for _ in range(2))
    wg[0] = torch.linspace(0.75, 1.25, F, device="cuda").to(dt)
    wu[1] = 1
    h, gate, up = wkv.glu(x, wg, wu, act=wkv.RWKV7_ACT_GELU, want_pre=True)
    assert (up == 1).all()
    # float32: the pre-activation as it left; bfloat16: the exact product, which float32 holds
    g = gate if dt == torch.float32 else x[:, :1].double() * wg[0].double()
    a, e, _, _ = gelu(torch, g)
    near("h", h, a, e, 1)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_gradients(torch, dtype):
    """One row of one channel, 1: the weights' gradients are dg and du themselves."""
    dt = getattr(torch, dtype)
    F = 4001
    say("glu gelu tail gradients", F, dtype)
    g = torch.linspace(-12.0, 6.0, F, device="cuda").to(dt).view(1, F)
    one, w = torch.ones(1, 1, dtype=dt, device="cuda"), torch.ones(1, F, dtype=dt, device="cuda")
    got = wkv.glu_backward(one, w, w, g, torch.ones_like(g), torch.ones_like(g), act=wkv.RWKV7_ACT_GELU)
    a, e_a, s, e_s = gelu(torch, g)
    near("dw_gate", got["dw_gate"], s, e_s, 1)
    near("dw_up", got["dw_up"], a, e_a, 1)
