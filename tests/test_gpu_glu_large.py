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
