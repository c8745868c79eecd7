"""Calls for another device than the current one, without a GPU: the tensors and the stream are stand-ins."""
import contextlib
import inspect
import re

import pytest
import torch

from linear_rnn_amd import wkv


class Like:
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


class Stream:
    cuda_stream = 4096

    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.fixture
def calls(monkeypatch):
    seen = []
    current = [0]

    class Library:
        def rwkv7_some_call(self, *args):
            seen.append((current[0], args))
            return 0

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    assert wkv._T.codes  # what is kept of torch is there
    monkeypatch.setattr(wkv, "lib", Library)
    monkeypatch.setattr(wkv._T, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    return seen


def test_the_tensors_device_is_current_for_the_call(calls):
    wkv._launch("rwkv7_some_call", [7], Like(), Stream(1))
    wkv._launch("rwkv7_some_call", [8], Like(), 4096)  # a bare handle
    assert calls == [(1, (7, 4096)), (1, (8, 4096))]


def test_a_stream_of_another_device_is_refused(calls):
    with pytest.raises(ValueError, match="the stream is on cuda:0, the tensors on cuda:1"):
        wkv._launch("rwkv7_some_call", [7], Like(), Stream(0))
    with pytest.raises(ValueError, match="current device is cuda:0"):
        wkv._launch("rwkv7_some_call", [7], Like(), None)
    assert calls == []


def test_every_entry_point_launches_so():
    """No function calls the library with whatever device is current."""
    called = set(re.findall(r"lib\(\)\.(rwkv7_\w+)", inspect.getsource(wkv)))
    assert called == {"rwkv7_wkv_prefill_algo", "rwkv7_wkv_strerror"}
