"""Streams: each thread's own (hipStreamPerThread), and whose memory the allocating functions return."""
import threading

import pytest

from linear_rnn_amd import wkv
from linear_rnn_amd.inputs import CONFIGS, make_cotangents, make_inputs, make_stack_inputs
from tests.gpu_util import say, to_dev
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


def stream_of(torch, t):
    """The stream that torch's allocator holds a tensor's memory for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not memory of the allocator")


def calls(torch, d, stream):
    """The tensors that every allocating function returns."""
    r, k, v, y = d["r"], d["k"], d["v"], d["dy"]
    w = torch.full_like(r, 0.9)
    wf = torch.full(r.shape, -1.0, device="cuda")
    rows = y.view(y.shape[0], y.shape[1], -1)
    mean, rstd = (torch.ones(rows.shape[:-1] + (r.shape[2],), device="cuda") for _ in range(2))
    f = torch.zeros(r.shape, device="cuda")
    one = [t[:, :1].contiguous() for t in (r, d["log_w"], k, v)]
    torch.cuda.synchronize()
    out = [wkv.wkv7(r, w, k, v, k, v, stream=stream), wkv.tmix(r, wf, k, v, k, v, stream=stream),
           tuple(wkv.wkv7_backward(r, w, k, v, k, v, f, stream=stream).values()),
           wkv.linattn(r, d["log_w"], k, v, stream=stream), wkv.linattn_step(*one, stream=stream),
           tuple(wkv.linattn_backward(r, d["log_w"], k, v, y, stream=stream).values()),
           wkv.layernorm(rows, groups=r.shape[2], stream=stream),
           tuple(wkv.layernorm_backward(rows, None, mean, rstd, rows, groups=r.shape[2], stream=stream).values())]
    return [t for o in out for t in o]


def test_allocated_outputs_are_of_the_stream(torch):
    say("allocated outputs")
    d, _ = case(torch, 2, 40, 3, 79)
    st = torch.cuda.Stream()
    for stream, owner in ((None, torch.cuda.current_stream().cuda_stream), (st, st.cuda_stream), (st.cuda_stream, st.cuda_stream)):
        got = calls(torch, d, stream)
        assert len(got) == 2 + 2 + 7 + 2 + 2 + 5 + 3 + 3
        assert {stream_of(torch, t) for t in got} == {owner}
        torch.cuda.synchronize()
        del got
    with pytest.raises(ValueError, match="hipStreamPerThread"):
        wkv.linattn(d["r"], d["log_w"], d["k"], d["v"], stream=PER_THREAD)


def test_two_threads_of_the_recurrence_on_one_stream(torch):
    """The split prefill, the gradients and the stack pass records from kernel to kernel in the stream's workspace."""
    say("recurrence, two threads on one stream")
    st = torch.cuda.Stream()
    cases = []
    for n, (B, T, H) in enumerate(((1, 700, 3), (2, 450, 2))):
        x = make_inputs(CONFIGS["L12-D768-prefill"], B=B, T=T, H=H, seed=30 + n, with_state=True)
        d = to_dev(x)
        k = make_stack_inputs(2, B, 60, H, "bf16", seed=40 + n)
        d["w_in"], d["w_out"] = (torch.from_numpy(k[i].view("int16")).cuda().view(torch.bfloat16) for i in ("w_in", "w_out"))
        d["vecs"], d["x"], d["states"] = (torch.from_numpy(k[i]).cuda() for i in ("vecs", "x", "states"))
        d["dy"] = torch.from_numpy(make_cotangents(B, T, H, seed=n)["dy"]).cuda()
        cases.append(d)
    torch.cuda.synchronize()

    def call(d):
        a = [d[n] for n in "rwkvab"]
        with torch.cuda.stream(st):
            out = {"y": wkv.wkv7(*a, state_in=d["state_in"], algo=wkv.RWKV7_ALGO_CHUNKED_SPLIT)}
            for algo in (wkv.RWKV7_ALGO_CHUNKED, wkv.RWKV7_ALGO_SEQUENTIAL):
                out[algo] = tuple(wkv.wkv7_backward(*a, d["dy"], d["state_in"], None, algo=algo).values())
            x, s = d["x"].clone(), d["states"].clone()
            wkv.rwkv7_stack_forward(d["w_in"], d["w_out"], d["vecs"], x, s)
            out["stack"] = (x, s)
        return [t for o in out.values() for t in o]

    want = [call(d) for d in cases]
    torch.cuda.synchronize()
    bad = []

    def work(n):
        try:
            got = [call(cases[n]) for _ in range(10)]
            st.synchronize()
            bad.extend((n, i) for g in got for i, (t, w) in enumerate(zip(g, want[n])) if not torch.equal(t, w))
        except Exception as e:  # shown by the assertion below
            bad.append((n, e))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad
