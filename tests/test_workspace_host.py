"""Whose memory the binding's workspaces are, against a stand-in for torch (no GPU): the
allocator hands a freed buffer out again in the order of the stream that was current when it
was allocated, so that has to be the stream the call launches on, captured or not."""
import contextlib
import types

import pytest


class Device(types.SimpleNamespace):
    def __hash__(self):
        return hash((self.type, self.index))


class FakeTorch:
    """Streams are pointers; 0 is the default stream of a device."""

    uint8 = "uint8"

    def __init__(self):
        self.now, self.current, self.capturing, self.allocated = 0, {0: 7, 1: 0}, set(), []
        self._C = types.SimpleNamespace(
            _cuda_getDevice=lambda: self.now,
            _cuda_getCurrentRawStream=lambda i: self.current[i],
            _cuda_isCurrentStreamCapturing=lambda: (self.now, self.current[self.now]) in self.capturing,
            _cuda_getCurrentStream=lambda i: (self.current[i], i, 1), _cuda_setStream=self._set)
        self.cuda = types.SimpleNamespace(ExternalStream=self._external, stream=self._stream, device=self._device,
                                          default_stream=lambda d: self._stream_object(0, d))

    def _stream_object(self, ptr, device):
        return types.SimpleNamespace(stream_id=ptr, device_index=device.index, device_type=1)

    def _external(self, ptr, device=None):
        # as in torch, a null pointer asks for a new stream
        return self._stream_object(ptr or 999, device)

    def _set(self, stream_id, device_index, device_type):
        assert device_type == 1
        self.now, self.current[device_index] = device_index, stream_id

    @contextlib.contextmanager
    def _stream(self, s):
        before, stream = self.now, self.current[s.device_index]
        self._set(s.stream_id, s.device_index, 1)
        try:
            yield
        finally:
            self.current[s.device_index], self.now = stream, before

    @contextlib.contextmanager
    def _device(self, device):
        before, self.now = self.now, device.index
        try:
            yield
        finally:
            self.now = before

    def empty(self, n, dtype=None, device=None):
        buf = types.SimpleNamespace(device=device, stream=self.current[device.index], numel=lambda: n,
                                    captured=(device.index, self.current[device.index]) in self.capturing,
                                    record_stream=lambda s: None)
        self.allocated.append(buf)
        return buf


@pytest.fixture
def fake(monkeypatch):
    from __graft_entry__ import build
    build()
    import paged_kv_cache_261_gb300 as pa
    torch = FakeTorch()
    monkeypatch.setattr(pa, "_torch_module", torch)
    monkeypatch.setattr(pa, "_ws_cache", {})
    monkeypatch.setattr(pa, "_stream_ids", {}, raising=False)
    return pa, torch


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("ptr", [0, 7, 16, 32])
def test_workspace_belongs_to_the_launching_stream(fake, ptr, captured, index):
    pa, torch = fake
    dev = Device(type="cuda", index=index)
    if captured:                                  # the current stream forked into ptr, both captured
        torch.capturing = {(index, ptr), (0, 7)}
    for n in (100, 1 << 22, 200):
        buf = pa._workspace(dev, ptr, n)
        assert buf.stream == ptr and buf.device is dev and buf.numel() >= n and buf.captured == captured
    assert (torch.now, torch.current) == (0, {0: 7, 1: 0})
    # cached and grown once, or one for each captured call
    assert len(torch.allocated) == (3 if captured else 2) and len(pa._ws_cache) == (0 if captured else 1)


def test_workspace_of_a_captured_stream_that_is_not_current(fake):
    """What counts is whether the launching stream is captured: a cached buffer must not get into a graph,
    nor a graph's memory into an eager call."""
    pa, torch = fake
    dev = Device(type="cuda", index=0)
    eager = pa._workspace(dev, 16, 100)
    torch.capturing = {(0, 16)}                   # current: 7
    a, b = pa._workspace(dev, 16, 100), pa._workspace(dev, 16, 100)
    assert a is not eager and b is not a and a.captured and b.captured and a.stream == 16
    torch.capturing = {(0, 7)}
    assert pa._workspace(dev, 16, 100) is eager and not eager.captured
    assert pa._workspace(dev, 7, 100).captured


def test_failed_allocation_leaves_the_current_stream(fake, monkeypatch):
    pa, torch = fake

    def fail(*a, **kw):
        raise MemoryError

    monkeypatch.setattr(torch, "empty", fail)
    for index, ptr in ((0, 16), (0, 0), (1, 16)):
        with pytest.raises(MemoryError):
            pa._workspace(Device(type="cuda", index=index), ptr, 100)
        assert (torch.now, torch.current) == (0, {0: 7, 1: 0}) and not pa._ws_cache
