"""Host threads that share a stream share its workspace too: an operator's launches over it must not be parted by another call's."""
import contextlib
import ctypes
import threading
import time
import types

import pytest
import torch


@pytest.fixture
def api(monkeypatch):
    """The binding on a device and a library that are not there."""
    from speculative_decoding_verification_02_gb300 import api
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(api, "_workspaces", {(0, s): torch.empty(256, dtype=torch.uint8) for s in (0, 7, 8)})
    return api


def calls_at_once(first, second):
    """Runs both at the same time; how many were in the library together at most."""
    state = types.SimpleNamespace(now=0, most=0)
    guard = threading.Lock()

    def enter(*_):
        with guard:
            state.now += 1
            state.most = max(state.most, state.now)
        time.sleep(0.1)
        with guard:
            state.now -= 1
        return 0

    threads = [threading.Thread(target=f, args=(enter,)) for f in (first, second)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return state.most


def on(api, stream, old=False):
    dev = types.SimpleNamespace(index=0)
    if old:
        return lambda fn: api._check(api._call(dev, fn, 1, ctypes.c_void_p(stream)), "call")
    return lambda fn: api._with_workspace(fn, "call", api.OP_CACHE_ATTEND, b"", 1, 1, 1, dev, None, stream, 1)


@pytest.mark.parametrize("stream", [0, 7])
def test_calls_on_one_stream_follow_one_another(api, stream):
    assert calls_at_once(on(api, stream), on(api, stream)) == 1
    assert calls_at_once(on(api, stream), on(api, stream, old=True)) == 1
    assert calls_at_once(on(api, stream, old=True), on(api, stream, old=True)) == 1


def test_calls_on_other_streams_do_not_wait(api):
    assert calls_at_once(on(api, 7), on(api, 8)) == 2
    assert calls_at_once(on(api, 7, old=True), on(api, 8)) == 2


def test_a_call_that_fails_lets_the_next_one_in(api):
    def broken(*_):
        raise KeyError
    for old in (False, True):
        with pytest.raises(KeyError):
            on(api, 7, old)(broken)
    assert calls_at_once(on(api, 7), on(api, 7, old=True)) == 1
