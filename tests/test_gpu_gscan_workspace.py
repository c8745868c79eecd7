"""Which prompts of the gated linear recurrence need the workspace, as the header says: a call that needs none can be
captured on a stream that has none, one that needs it is refused there."""
import re

import pytest

from linear_rnn_amd import wkv
from tests.gpu_util import new_stream, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def stated(B, T, D):
    """True: none, False: needed, None: left open."""
    units, singles = B * -(-D // 64), D % 64 in (1, 2, 3)
    if singles:
        return True if T <= 224 or units >= 160 else None
    return T <= 384 or (units >= 192 and T <= 2048)


def test_the_header_states_this():
    with open(wkv.__file__.replace("linear_rnn_amd/wkv.py", "include/rwkv7_wkv.h")) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    assert "A prompt needs no workspace up to 384 tokens, and none up to 2048 where B*ceil(D/64) is 192 or more; " \
           "where D mod 64 is 1, 2 or 3 none up to 224 tokens, and none at any length where B*ceil(D/64) is 160 or more." in text


@pytest.mark.parametrize("B,T,D", [(1, 384, 64), (1, 385, 64), (191, 384, 64), (191, 385, 64), (191, 2048, 64), (192, 2048, 64),
                                   (192, 2049, 64), (8, 4096, 1536), (3, 2048, 4096), (2, 2048, 4096), (200, 2300, 4),
                                   (1, 224, 65), (1, 3000, 65), (80, 5000, 65), (79, 225, 1), (159, 224, 1), (160, 5000, 1)])
def test_workspace_of_a_prompt(torch, B, T, D):
    say("gscan workspace", B, T, D)
    x = torch.zeros(B, T, D, dtype=torch.bfloat16, device="cuda")
    lw, y = torch.zeros(B, T, D, device="cuda"), torch.empty_like(x)
    stream, g, refused = new_stream(), torch.cuda.CUDAGraph(), False
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        try:
            wkv.rwkv7_gscan_prefill(x, lw, None, None, y, None, stream=stream)
        except wkv.Rwkv7Error:
            refused = True
    none = stated(B, T, D)
    assert none is None or refused == (not none), (B, T, D)
