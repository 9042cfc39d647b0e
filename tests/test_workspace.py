"""Workspaces on the host, without a device: CPU buffers, and a library whose two calls write to them directly."""
import ctypes
import threading
import time

import pytest
import torch

import draft_verification_spec_gb300 as sv


class FakeLibrary:
    """spec_workspace_bytes / _init / spec_get_status on host memory; a status word holds its code."""

    def spec_workspace_bytes(self, B, K, V, dtype):
        return 1024 * B

    def spec_workspace_init(self, ptr, n, stream):
        ctypes.memset(ptr, 0, n)
        return 0

    def spec_get_status(self, ptr, stream, out):
        word = ctypes.cast(ptr, ctypes.POINTER(ctypes.c_int32))
        ctypes.cast(out, ctypes.POINTER(ctypes.c_int32))[0] = word[0]
        word[0] = 0
        return 0


@pytest.fixture
def ws(monkeypatch):
    monkeypatch.setattr(sv, "lib", FakeLibrary)
    monkeypatch.setattr(sv, "_stream_ptr", lambda stream: None)
    return sv.Workspace("cpu")


def _report(buf, code):
    buf[:4].view(torch.int32)[0] = code


def test_outgrown_buffers_stay_alive(ws):
    """A captured graph replays with the address that it was captured with."""
    import weakref
    for get in (lambda n: ws.get_step(n, None), lambda n: ws.get(-(-n // 1024), 3, 100, 0, None)):
        first = get(8192)
        address, alive = first.data_ptr(), weakref.ref(first)
        del first
        for n in (16384, 20480, 300000, 1 << 20):
            assert get(n).numel() >= n and get(1).data_ptr() == get(n).data_ptr()
        assert alive() is not None and alive().data_ptr() == address
    # and they are few and small: together less than the two that are in use
    kept = [b for b, _ in ws._outgrown]
    assert len(kept) <= 12 and sum(b.numel() for b in kept) < ws.buf.numel() + ws.step_buf.numel()


def test_threads_that_grow_a_workspace_get_one_buffer(ws, monkeypatch):
    slow = FakeLibrary.spec_workspace_init
    monkeypatch.setattr(FakeLibrary, "spec_workspace_init", lambda s, p, n, st: (time.sleep(0.05), slow(s, p, n, st))[1])
    got = []
    threads = [threading.Thread(target=lambda: got.append(ws.get_step(1 << 16, None).data_ptr())) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(set(got)) == 1 and not ws._outgrown


def test_status_of_an_outgrown_buffer_is_not_lost(ws):
    _report(ws.get_step(256, None), 7)            # a small call reports a page
    ws.get_step(1 << 20, None)                    # a larger one follows before anybody looks
    assert ws.status() == 7 and ws.status() == 0
    _report(ws.get(1, 3, 100, 0, None), 5)
    ws.get(1000, 3, 100, 0, None)
    assert ws.status() == 5 and ws.status() == 0


def test_status_names_the_gravest_report(ws):
    """Timeout before token range before page range, whichever operator's buffer holds it."""
    for first, second, want in ((5, 7, 5), (5, 4, 4), (4, 7, 4), (0, 7, 7), (0, 4, 4)):
        _report(ws.get(1, 3, 100, 0, None), first)
        _report(ws.get_step(256, None), second)
        assert ws.status() == want and ws.status() == 0


def test_reset_clears_outgrown_buffers_too(ws):
    _report(ws.get_step(256, None), 4)
    _report(ws.get_step(1 << 20, None), 7)
    ws.reset()
    assert ws.status() == 0


def test_step_operators_refuse_a_workspace_elsewhere(monkeypatch):
    """Its address would be followed on the current device."""
    from draft_verification_spec_gb300 import step
    monkeypatch.setattr(sv, "lib", FakeLibrary)
    monkeypatch.setattr(sv, "_stream_ptr", lambda stream: None)
    for device in ("cpu", "cuda:1"):
        with pytest.raises(ValueError, match="workspace must be on the current device cuda:0"):
            step._step_buffer(sv.Workspace(device), 0, 0, 256, None)
