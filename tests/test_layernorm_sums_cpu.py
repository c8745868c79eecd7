"""What the bounds on the layer norm's sums over rows let through: float32 sums in the kernels' order, and not the same
with the workgroups' partial sums, or the terms, rounded to bfloat16."""
import pytest
import torch

from tests import layernorm_ref as ref
from tests import layernorm_sums as sums

SIZES = [(5000, 64, 1), (4099, 128, 2), (3001, 1024, 16), (2500, 771, 1), (1301, 4096, 1)]


def in_order(M, D, G, terms, rows, each):
    """The kernels' sum of float32 terms [M, D]: `each` is what becomes of a term, `rows` of a partial row."""
    nb, R = sums.split(M, D, G)
    lanes = torch.zeros(nb * R, D)
    for m0 in range(0, M, nb * R):
        n = min(nb * R, M - m0)
        lanes[:n] += each(terms[m0:m0 + n])
    lanes = lanes.view(nb, R, D)
    part = lanes[:, 0]
    for r in range(1, R):
        part = part + lanes[:, r]
    part = rows(part)
    out = torch.zeros(16, D)
    for i in range(nb):
        out[i % 16] += part[i]
    total = out[0]
    for i in range(1, 16):
        total = total + out[i]
    return total


def keep(t):
    return t


def round16(t):
    return t.to(torch.bfloat16).float()


@pytest.mark.parametrize("M,D,G", SIZES)
def test_bounds_tell_float32_sums_from_rounded_ones(M, D, G):
    x = ref.make(M, D, G, torch.float32, torch.float32, seed=M)
    _, mean, rstd = ref.forward(x["x"], x["weight"], x["bias"], G, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    want = sums.sums(x["x"], mean, rstd, x["dy"], G)
    xh = ((x["x"].view(M, G, -1) - mean[..., None]) * rstd[..., None]).view(M, D)
    for name, terms in (("dweight", x["dy"] * xh), ("dbias", x["dy"])):
        sums.check(name, in_order(M, D, G, terms, keep, keep), want[name], M, D, G)
        for rows, each in ((round16, keep), (keep, round16)):
            with pytest.raises(AssertionError):
                sums.check(name, in_order(M, D, G, terms, rows, each), want[name], M, D, G)


def test_splits_cover_the_rows():
    for M in (1, 3, 64, 1000, 70001):
        for D, G in ((1, 1), (64, 1), (771, 1), (768, 12), (4096, 1), (8200, 1), (9999, 1), (16384, 1), (20000, 1), (6400, 100)):
            nb, R = sums.split(M, D, G)
            assert nb >= 1 and R >= 1 and (nb - 1) * R < M
            assert sums.depth(M, D, G) >= -(-M // (nb * R))
