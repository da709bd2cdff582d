"""Streams of the binding, without a GPU: whose handle a call takes, and whose memory a cache lives in."""
import contextlib
import sys
import types

import pytest
import torch


@pytest.fixture
def sdv(monkeypatch):
    import speculative_decoding_verify_02_gb300 as sdv
    monkeypatch.setattr(sdv, "_raw_stream", None)
    monkeypatch.setattr(sdv, "_device", None)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 700 + d, raising=False)
    yield sdv
    monkeypatch.undo()


def test_first_calls_of_two_threads(sdv):
    """A call that comes in between any two instructions of the first one gets its stream, too."""
    where = 0
    sys._getframe().f_trace_opcodes = True                            # before settrace, or it brings lines only
    while True:
        sdv._raw_stream = sdv._device = None
        seen = steps = 0

        def trace(frame, event, arg):
            nonlocal seen, steps
            if frame.f_code is not sdv._stream.__code__:
                return None
            frame.f_trace_opcodes = True
            if event == "opcode":
                if steps == where:
                    sys.settrace(None)
                    seen = sdv._stream(None)                          # what another thread would do here
                steps += 1
            return trace

        sys.settrace(trace)
        try:
            first = sdv._stream(None)
        finally:
            sys.settrace(None)
        assert first == 703
        if not seen:                                                  # past the last instruction
            break
        assert seen == 703
        where += 1
    assert where > 20


@pytest.mark.parametrize("given", [False, True])
def test_cache_memory_belongs_to_the_stream_that_clears_it(sdv, monkeypatch, given):
    """Memory of another stream may still be in use there when the cache is cleared."""
    current, held = ["main"], []

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream if stream is not None else current[0]
        yield
        current[0] = before

    empty = torch.empty

    def fake_empty(*shape, dtype, device):
        held.append(current[0])
        return empty(*shape, dtype=dtype)

    cleared = []
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", fake_empty)
    side = types.SimpleNamespace(cuda_stream=9)
    calls = types.SimpleNamespace(sdv_qcache_bytes=lambda *a: 0, sdv_qcache_destroy=lambda c: 0,
                                  sdv_qcache_create=lambda *a: cleared.append(a[4]) or 0)
    monkeypatch.setattr(sdv, "lib", lambda: calls)
    sdv.QuantCache(1, 2, 1, 64, n_pages=4, max_context=32, stream=side if given else None)
    assert cleared == [9 if given else 703]
    assert held == [side if given else "main"] * 3 and current == ["main"]
