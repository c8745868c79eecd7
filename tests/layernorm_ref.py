"""Plain float64 layer norm over groups of channels, with bounds on what float32 sums may be off.

Nothing here uses the package: torch on the CPU, float64 throughout.
"""
import torch

F64 = torch.float64
U = 2.0 ** -24  # float32: half a step, relative


def make(M, D, G, x_dtype, y_dtype, seed, offset=1.0):
    g = torch.Generator().manual_seed(seed)

    def n(*shape):
        return torch.randn(shape, generator=g)

    return {"x": (n(M, D) * torch.exp(n(M, 1)) + offset * n(1, D)).to(x_dtype), "weight": 1 + 0.3 * n(D),
            "bias": 0.3 * n(D), "dy": n(M, D).to(y_dtype), "G": G}


def forward(x, weight, bias, G, eps):
    M, D = x.shape
    n = D // G
    x = x.to(F64).view(M, G, n)
    w = torch.ones(D, dtype=F64) if weight is None else weight.to(F64)
    b = torch.zeros(D, dtype=F64) if bias is None else bias.to(F64)
    mean = x.mean(-1)
    rstd = 1 / ((x - mean[..., None]).square().mean(-1) + eps).sqrt()
    xh = (x - mean[..., None]) * rstd[..., None]
    return xh.view(M, D) * w + b, mean, rstd


def backward(x, weight, mean, rstd, dy, G):
    """From the given mean and rstd (float32 inputs of the call, exact here)."""
    M, D = x.shape
    n = D // G
    w = torch.ones(D, dtype=F64) if weight is None else weight.to(F64)
    dy = dy.to(F64)
    xh = (x.to(F64).view(M, G, n) - mean.to(F64)[..., None]) * rstd.to(F64)[..., None]
    g = (dy * w).view(M, G, n)
    dx = rstd.to(F64)[..., None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return {"dx": dx.view(M, D), "dweight": (dy * xh.view(M, D)).sum(0), "dbias": dy.sum(0)}


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


# A sum over a group of n channels: a thread adds at most 16 (or n / 1024) values in turn, then at most 6
# doublings in a wave and 16 waves: 40 + n / 1024 roundings; with the products and scales around it, 64.
def _depth(n):
    return 64 + n // 1024


def forward_limits(x, weight, bias, G, eps, y_dtype):
    """Bounds for y, mean, rstd."""
    M, D = x.shape
    n = D // G
    c = _depth(n)
    y, mean, rstd = forward(x, weight, bias, G, eps)
    xg = x.to(F64).view(M, G, n)
    size = xg.abs().mean(-1)
    e_mean = c * U * size
    # the variance: its sum's roundings, and the mean's error squared (its first order cancels)
    e_rstd = rstd * (c * U + (e_mean * rstd).square())
    w = torch.ones(D, dtype=F64) if weight is None else weight.to(F64).abs()
    b = torch.zeros(D, dtype=F64) if bias is None else bias.to(F64).abs()
    xh = (xg - mean[..., None]).abs() * rstd[..., None]
    e_xh = (e_mean[..., None] + 2 * U * (xg.abs() + size[..., None])) * rstd[..., None] + xh * (e_rstd / rstd)[..., None]
    e_y = e_xh.view(M, D) * w + 4 * U * (xh.view(M, D) * w + b)
    return _half_step(y_dtype) * (y.abs() + e_y) + e_y, e_mean + U * mean.abs(), e_rstd + 2 * U * rstd


def backward_limits(x, weight, mean, rstd, dy, G):
    M, D = x.shape
    n = D // G
    c = _depth(n)
    ref = backward(x, weight, mean, rstd, dy, G)
    w = torch.ones(D, dtype=F64) if weight is None else weight.to(F64)
    dy = dy.to(F64).abs()
    m, s = mean.to(F64)[..., None], rstd.to(F64)[..., None]
    xg = x.to(F64).view(M, G, n)
    xh = ((xg - m) * s).abs()
    e_xh = 3 * U * xh + U * (xg.abs() + m.abs()) * s
    g = (dy * w.abs()).view(M, G, n)
    gx = (g * xh).mean(-1, keepdim=True)
    e = s * (c * U * (g + g.mean(-1, keepdim=True) + 2 * xh * gx) + e_xh * gx + xh * (g * e_xh).mean(-1, keepdim=True))
    e = e.view(M, D)
    # at most one rounding for each row and product, whatever the order of the sum over rows
    e_w = (2 + M) * U * (dy * xh.view(M, D)).sum(0) + (dy * e_xh.view(M, D)).sum(0)
    return {"dx": _half_step(x.dtype) * (ref["dx"].abs() + e) + e, "dweight": e_w, "dbias": M * U * dy.sum(0)}


def check(name, got, ref, limit):
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), name
    if got.numel():
        over = ((got - ref).abs() - limit).max()
        assert over <= 0, "%s: %g over its bound" % (name, float(over))
