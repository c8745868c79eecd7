"""Plain float64 gated linear recurrence, token by token, with bounds on what float32 arithmetic may be off.

Nothing here uses the package: torch on the CPU, float64 throughout.
"""
import math

import torch

F64 = torch.float64
U = 2.0 ** -24  # float32: half a step, relative
KINDS = ("plain", "mix", "norm")  # in the order of their codes


def make(B, T, D, dtype, seed, state=True, resets=0.02):
    g = torch.Generator().manual_seed(seed)

    def n(*shape):
        return torch.randn(shape, generator=g)

    x = {"x": n(B, T, D).to(dtype), "log_w": -torch.exp(torch.rand(B, T, D, generator=g) * 9 - 8), "dy": n(B, T, D).to(dtype),
         "state_in": n(B, D) if state else None, "dstate_out": n(B, D) if state else None}
    if resets:
        x["log_w"][torch.rand(B, T, generator=g) < resets] = -math.inf
        x["log_w"][torch.rand(B, T, D, generator=g) < resets] = 0.0
    return x


def _scale(lw, kind):
    """s, its derivative to log w, and the relative errors of w, of s and of the derivative in float32."""
    w = lw.exp()
    # the argument of the exponential has two roundings, the exponential one of a whole step
    e_w = torch.where(torch.isinf(lw), 0.0, 2 * U * lw.abs() + 2 * U)
    if kind == "plain":
        return torch.ones_like(lw), torch.zeros_like(lw), e_w, torch.zeros_like(lw), torch.zeros_like(lw)
    z, p, e_p = (-lw, w, e_w) if kind == "mix" else (-2 * lw, w * w, 2 * e_w + U)
    q = -torch.expm1(-z)
    # the series' roundings (each later one counts by half or less), or 1 - p with p's error
    e_q = 8 * U + torch.where(z > 0.34, p * e_p / q.clamp_min(0.28), 0.0)
    if kind == "mix":
        return q, -w, e_w, e_q, e_w
    s = q.sqrt()
    return s, torch.where(s > 0, -p / s.clamp_min(1e-300), 0.0), e_w, e_q / 2 + 2 * U, e_p + e_q / 2 + 6 * U


def _keep(lens, B, T):
    t = torch.arange(T)[None, :]
    return torch.ones(B, T, dtype=torch.bool) if lens is None else t < torch.as_tensor(lens)[:, None].clamp(0, T)


def _walk(w, b, first, e_w, e_b, keep, order):
    """v <- w v + b over the tokens in `order`: the values after each, and how far any order of the sum may be off:
    each token's decay and input carry their own errors and five roundings (their product into a map, the sum, and
    the compositions, of which there are fewer than tokens), and the joins around it 64 more of the magnitudes."""
    v = first.clone()
    size, err = first.abs(), torch.zeros_like(first)
    values, bounds = torch.zeros_like(b), torch.zeros_like(b)
    for t in order:
        k = keep[:, t, None]
        err = torch.where(k, w[:, t] * (err + (e_w[:, t] + 5 * U) * size) + b[:, t].abs() * (e_b[:, t] + 5 * U), err)
        size = torch.where(k, w[:, t] * size + b[:, t].abs(), size)
        v = torch.where(k, w[:, t] * v + b[:, t], v)
        values[:, t], bounds[:, t] = v, err + 64 * U * size + 1e-37
    return values, bounds, v, err + 64 * U * size + 1e-37


def _clean(x, keep):
    """Widened, with zeros in place of whatever is behind a sequence's end."""
    return torch.where(keep[..., None], x.to(F64), 0.0)


def forward(x, log_w, state_in, lens, kind):
    """{name: (value, bound)} of y and state; y's bound without its rounding to the output type."""
    B, T, D = x.shape
    keep = _keep(lens, B, T)
    lw = _clean(log_w, keep)
    s, _, e_w, e_s, _ = _scale(lw, kind)
    first = torch.zeros(B, D, dtype=F64) if state_in is None else state_in.to(F64)
    y, e_y, state, e_state = _walk(lw.exp(), s * _clean(x, keep), first, e_w, e_s, keep, range(T))
    k = keep[..., None]
    return {"y": (torch.where(k, y, 0.0), torch.where(k, e_y, 0.0)), "state": (state, e_state)}


def backward(x, log_w, state_in, lens, dy, dstate_out, kind):
    B, T, D = x.shape
    keep = _keep(lens, B, T)
    lw, x, dy = _clean(log_w, keep), _clean(x, keep), _clean(dy, keep)
    w = lw.exp()
    s, slope, e_w, e_s, e_slope = _scale(lw, kind)
    first = torch.zeros(B, D, dtype=F64) if state_in is None else state_in.to(F64)
    h, e_h, _, _ = _walk(w, s * x, first, e_w, e_s, keep, range(T))
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    e_before = torch.cat([torch.zeros(B, 1, D, dtype=F64), e_h[:, :-1]], 1) + 64 * U * before.abs()
    last = torch.zeros(B, D, dtype=F64) if dstate_out is None else dstate_out.to(F64)
    # what comes back through token t is c = w (dy + c): a walk of the map's own kind with b = w dy
    c, e_c, d0, e_d0 = _walk(w, w * dy, last, e_w, e_w + U, keep, range(T - 1, -1, -1))
    come = torch.cat([c[:, 1:], last[:, None]], 1)
    # behind a sequence's end the walk stays at `last`, as it starts
    e_come = torch.cat([e_c[:, 1:], torch.zeros(B, 1, D, dtype=F64)], 1) + 64 * U * come.abs()
    g = dy + come
    e_g = e_come + U * g.abs()
    through = w * before + slope * x
    e_through = w * (e_before + (e_w + 2 * U) * before.abs()) + (slope * x).abs() * (e_slope + 3 * U)
    dx, dlw = s * g, through * g
    e_dx = s * (e_g + (e_s + 2 * U) * g.abs())
    e_dlw = through.abs() * (e_g + 2 * U * g.abs()) + e_through * (g.abs() + e_g) + 1e-37
    k = keep[..., None]
    zero = {"dx": (dx, e_dx), "dlog_w": (dlw, e_dlw)}
    out = {n: (torch.where(k, v, 0.0), torch.where(k, e, 0.0)) for n, (v, e) in zero.items()}
    out["dstate_in"] = (d0, e_d0)
    return out


def check(name, got, want):
    ref, e = want
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    got = got.detach().cpu().to(F64)
    assert torch.isfinite(got).all(), name
    if got.numel():
        over = ((got - ref).abs() - e - half * (ref.abs() + e)).max()
        assert over <= 0, "%s: %g over its bound" % (name, float(over))
