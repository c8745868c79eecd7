"""Streams that the other tests do not pass: each thread's own (hipStreamPerThread)."""
import threading

import pytest

from linear_rnn_amd import wkv
from tests.gpu_util import say
from tests.test_gpu_operator_limits import case, chain, clones

pytestmark = pytest.mark.gpu
PER_THREAD = 2  # hipStreamPerThread


@pytest.fixture(scope="module")
def torch():
    import torch as t
    wkv.lib()
    return t


def test_two_threads_on_their_own_streams(torch):
    """One handle, two streams that run side by side: each has a workspace of its own."""
    say("hipStreamPerThread in two threads")
    cases = [case(torch, 1, 3000, 2, 77), case(torch, 2, 2100, 3, 78)]
    want = []
    for d, out in cases:
        chain(torch, d, out, None)
        torch.cuda.synchronize()
        want.append(clones(out))
        for t in out.values():
            t.zero_()
    torch.cuda.synchronize()
    failed = []

    def work(n):
        try:
            d, out = cases[n]
            for _ in range(20):
                chain(torch, d, out, PER_THREAD)
            torch.cuda.synchronize()  # the thread's stream ends with it
        except Exception as e:  # shown by the assertion below
            failed.append((n, e))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for (d, out), w in zip(cases, want):
        assert all(torch.equal(out[n], w[n]) for n in w)
