"""Plain float64 gated linear unit and its gradients, with bounds on what the kernels' arithmetic may be off.

Nothing here uses the package: torch on the CPU, float64 throughout.

A sum of n products in float32, in any order, has at most one rounding for each product, of at most the sum S of the
products' magnitudes: n U S. A float32 operand is three bfloat16 pieces (exactly: 8 + 8 + 8 bits), the second and
third at most 2^-8 and 2^-16 of it, and the products of orders 3 and 4 are left out: 2 * 2^-24 + 2^-32 of S. The
products of orders 1 and 2 are added first, while the sum is below 2^-6 S: 5 n U 2^-6 S, together at most
(1.1 n + 3) U S. Such a bound has to hold for every element; over all of them the roundings add up like independent
ones, which norm() holds the results to.
"""
import math

import torch

F64 = torch.float64
U = 2.0 ** -24  # float32: half a step, relative
TINY = 2.0 ** -126  # the reciprocal's and the matrix cores' results and operands below it may count as 0
ACTS = ("sigmoid", "silu", "gelu", "relu2")  # in the order of their codes


def make(M, D, F, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(dtype)

    return {"x": n(M, D), "w_gate": n(D, F, scale=size * D ** -0.5), "w_up": n(D, F, scale=D ** -0.5),
            "gate": n(M, F, scale=size), "up": n(M, F), "dh": n(M, F)}


def act(g, kind):
    """The activation, its derivative, and what float32 evaluations of the two may be off."""
    e, f = torch.sigmoid(g), torch.sigmoid(-g)  # 1 - e would lose its digits above 37 in float64 too
    if kind == "relu2":
        r = g.clamp_min(0)
        return r * r, 2 * r, 2 * U * r * r, U * r
    if kind == "gelu":
        c = torch.special.ndtr(g)
        p = g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        # 1 + erf is off by its magnitude's roundings (a few of 1), not by its value's
        return g * c, c + p, 6 * U * g.abs(), 6 * U + p.abs() * (2 * g * g + 8) * U
    # the exponential's argument has two roundings of its magnitude
    far = (2 * g.abs() + 8) * U
    if kind == "sigmoid":
        return e, e * f, e * far + TINY, 2 * e * f * far + TINY
    return g * e, e * (1 + g * f), (g * e).abs() * far + g.abs() * TINY, 3 * e * (1 + g.abs() * f) * far + (1 + g.abs()) * TINY


def _terms(n, f32):
    return (1.1 * n + 3) * U if f32 else (n + 1) * U


def forward(x, w_gate, w_up, kind):
    """{name: (value, bound before the output's rounding)} of h, gate and up."""
    f32 = x.dtype == torch.float32
    x, wg, wu = (t.to(F64) for t in (x, w_gate, w_up))
    g, u = x @ wg, x @ wu
    k = _terms(x.shape[1], f32)
    e_g, e_u = k * (x.abs() @ wg.abs()), k * (x.abs() @ wu.abs())
    a, slope, e_a, _ = act(g, kind)
    e_a = e_a + slope.abs() * e_g + 2 * e_g * e_g  # no activation's second derivative is above 2, half of it counts
    h = a * u
    return {"h": (h, e_a * (u.abs() + e_u) + a.abs() * e_u + U * h.abs() + 1e-37), "gate": (g, e_g), "up": (u, e_u)}


def backward(x, w_gate, w_up, gate, up, dh, kind):
    f32 = x.dtype == torch.float32
    x, wg, wu, g, u, d = (t.to(F64) for t in (x, w_gate, w_up, gate, up, dh))
    a, slope, e_a, e_s = act(g, kind)
    dg, du = d * u * slope, d * a
    half = 0.0 if f32 else 2.0 ** -8  # where they enter the products
    e_dg = (1 + half) * ((d * u).abs() * e_s + 2 * U * dg.abs()) + half * dg.abs() + TINY
    e_du = (1 + half) * (d.abs() * e_a + U * du.abs()) + half * du.abs() + TINY
    m, f, ax = _terms(x.shape[0], f32), _terms(2 * g.shape[1], f32), x.abs().t()
    dx = dg @ wg.t() + du @ wu.t()
    e_dx = (f * dg.abs() + (1 + f) * e_dg) @ wg.abs().t() + (f * du.abs() + (1 + f) * e_du) @ wu.abs().t()
    return {"dx": (dx, e_dx + 1e-37), "dw_gate": (x.t() @ dg, ax @ (m * dg.abs() + (1 + m) * e_dg) + 1e-37),
            "dw_up": (x.t() @ du, ax @ (m * du.abs() + (1 + m) * e_du) + 1e-37)}


def check(name, got, want):
    ref, e = want
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    half = torch.finfo(got.dtype).eps / 2
    got = got.detach().cpu().to(F64)
    assert torch.isfinite(got).all(), name
    if got.numel():
        over = ((got - ref).abs() - e - half * (ref.abs() + e)).max()
        assert over <= 0, "%s: %g over its bound" % (name, float(over))


def norm(name, got, want, n):
    """In 2-norm, over many elements. bfloat16: the output's rounding and that of dg and du, each at most 2^-8 of a
    value and independent, so 2^-8 / sqrt 3 of the norm each at most: 2^-8 together. float32: n roundings, each of a
    partial sum that in the mean square is no larger than the whole: U sqrt n, with 4 for the pieces, the activation
    and roundings that are not to nearest inside the matrix cores."""
    ref = want[0]
    limit = 2.0 ** -8 if got.dtype == torch.bfloat16 else 4 * U * math.sqrt(n + 16)
    far = float((got.detach().cpu().to(F64) - ref).norm() / ref.norm())
    assert far <= limit, "%s: %g in 2-norm, at most %g" % (name, far, limit)
