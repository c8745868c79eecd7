"""The layer norm's sums over rows, held to the roundings of the order they are taken in."""
import pytest

from linear_rnn_amd import wkv
from tests import layernorm_ref as ref
from tests import layernorm_sums as sums
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


@pytest.mark.parametrize("yk", ["float32", "bfloat16"])
@pytest.mark.parametrize("xk", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,D,G", [(5000, 64, 1), (4099, 128, 2), (3001, 1024, 16), (2500, 771, 1), (1301, 4096, 1), (40000, 192, 3),
                                   (701, 8200, 1), (601, 9999, 1), (333, 16384, 1), (217, 20000, 1), (7, 768, 12)])
def test_sums_over_rows(torch, M, D, G, xk, yk):
    say("layernorm sums", M, D, G, xk, yk)
    x = ref.make(M, D, G, getattr(torch, xk), getattr(torch, yk), seed=M + D)
    _, mean, rstd = ref.forward(x["x"], None, None, G, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    g = wkv.layernorm_backward(x["x"].cuda(), x["weight"].cuda(), mean.cuda(), rstd.cuda(), x["dy"].cuda(), groups=G)
    torch.cuda.synchronize()
    want = sums.sums(x["x"], mean, rstd, x["dy"], G)
    for name in ("dweight", "dbias"):
        sums.check(name, g[name], want[name], M, D, G)
