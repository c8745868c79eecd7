"""Bounds on the layer norm's sums over rows (dweight, dbias) from the order they are taken in.

A thread adds the rows it takes one after the other, a workgroup its R rows, and 16 threads a channel the rows of partial
sums, which 15 additions join. `depth` counts the longest such chain; each addition is off by at most 2^-24 of the sum so
far, which the sum of the magnitudes bounds.
"""
import torch

from tests.layernorm_ref import F64, U


def threads(n):
    """(threads of a group, threads of a workgroup) of the gradients' kernels, or None where a group is read three times."""
    if n % 8 == 0:
        for most, lanes in ((64, 8), (128, 16), (256, 32), (1024, 64), (2048, 128), (4096, 512), (16384, 1024)):
            if n <= most:
                return lanes, (1024 if lanes > 256 else 256)
    else:
        for most, lanes in ((64, 16), (1024, 64), (2048, 128), (4096, 256), (8192, 512)):
            if n <= most:
                return lanes, (512 if lanes == 512 else 256)
    return None


def split(M, D, G):
    """(rows of partial sums, rows of a workgroup at a time)."""
    t = threads(D // G)
    if t is None:
        return min(M, max(1, min(64, 2 ** 23 // D))), 1
    slots = t[1] // t[0]
    S = min(G, slots)
    R = slots // S
    slabs = -(-G // S)
    return max(1, min((2 ** 18 if t[1] > 256 else 2 ** 17) // t[1] // slabs, -(-M // R))), R


def depth(M, D, G):
    nb, R = split(M, D, G)
    return -(-M // (nb * R)) + (R - 1) + -(-nb // 16) + 15


def sums(x, mean, rstd, dy, G):
    """dweight, dbias in float64; the sums of their terms' magnitudes; what the terms themselves may be off, summed and as
    the root of the squares."""
    M, D = x.shape
    m, s = mean.to(F64)[..., None], rstd.to(F64)[..., None]
    xg = x.to(F64).view(M, G, D // G)
    xh = ((xg - m) * s).view(M, D)
    # x - mean, its product with rstd and that with dy round once each (fused: not all of them do)
    off = ((3 * U * (xg - m).abs() + U * (xg.abs() + m.abs())) * s).view(M, D)
    dy = dy.to(F64)
    off = off * dy.abs()
    zero = torch.zeros(D, dtype=F64)
    return {"dweight": ((dy * xh).sum(0), (dy * xh).abs().sum(0), off.sum(0), off.square().sum(0).sqrt()),
            "dbias": (dy.sum(0), dy.abs().sum(0), zero, zero)}


def check(name, got, want, M, D, G):
    """Every channel within depth roundings of the magnitudes; and, as roundings of both signs add as the root of their
    squares, all of them within the root of that."""
    ref, mag, off, off2 = want
    got = got.detach().cpu().to(F64)
    c = depth(M, D, G)
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    over = (got - ref).abs() - (c * U * mag + off)
    assert over.max() <= 0, "%s: %g over its bound" % (name, float(over.max()))
    err, bound = float((got - ref).norm()), float(c ** 0.5 * U * mag.norm() + off2.norm())
    assert err <= bound, "%s: 2-norm of the error %g, bound %g" % (name, err, bound)
