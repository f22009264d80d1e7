"""Which stream and device PagedDecoder's status word is read and cleared on (no GPU needed: the library's two calls are
replaced)."""
import contextlib
import types

import pytest

import sparse_attention_row_gb300 as sar


@pytest.fixture
def world(monkeypatch):
    """A decoder on device 1 while device 0 is current; the current stream of device d is 100 + d."""
    w = types.SimpleNamespace(current=0, calls=[])

    @contextlib.contextmanager
    def device(d):
        was, w.current = w.current, d
        yield
        w.current = was

    monkeypatch.setattr(sar, "_stream", lambda s: 100 + w.current if s is None else s if isinstance(s, int) else s.cuda_stream)
    record = lambda name, result: lambda *a: w.calls.append((name, w.current, sar._stream(a[-1]))) or result  # noqa: E731
    monkeypatch.setattr(sar, "topk_workspace_init", record("init", sar.TOPK_OK))
    monkeypatch.setattr(sar, "topk_get_status", record("status", (sar.TOPK_OK, 0x80)))
    w.dec = object.__new__(sar.PagedDecoder)
    w.dec.device, w.dec.workspace = 1, None
    w.dec._torch = types.SimpleNamespace(cuda=types.SimpleNamespace(device=device))
    w.dec._get_device, w.dec._get_stream = lambda: w.current, lambda d: 100 + d
    return w


def test_status_and_reset_use_the_decoders_device_and_its_stream(world):
    assert world.dec.status() == 0x80
    world.dec.reset()
    assert world.calls == [("status", 1, 101), ("init", 1, 101)] and world.current == 0


@pytest.mark.parametrize("stream", [7, types.SimpleNamespace(cuda_stream=7)])
def test_a_stream_that_is_given_is_used(world, stream):
    world.dec.status(stream)
    world.dec.reset(stream)
    assert [c[1:] for c in world.calls] == [(1, 7), (1, 7)]


def test_on_the_current_device(world):
    world.current = 1
    world.dec.reset()
    assert world.calls == [("init", 1, 101)]
