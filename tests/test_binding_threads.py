"""CPU test of the binding's first calls from several threads at once: at whatever line of its setup the
first thread is held, another thread's calls are told what they are told alone."""
import importlib.util
import sys
import threading

import pytest
import torch


def _fresh_binding():
    """The binding as a program finds it that has made no call yet."""
    from block_scaled_w8a8_amd import bfq
    spec = importlib.util.spec_from_file_location("fresh_bfq", bfq.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _calls(b):
    i32, b16 = torch.int32, torch.bfloat16
    return (
        lambda: b.bfq_moe_route(torch.zeros(4, 16), torch.zeros((4, 2), dtype=i32), torch.zeros(4, 2)),
        lambda: b.bfq_moe_dispatch(torch.zeros((4, 256), dtype=b16), torch.zeros((4, 2), dtype=i32),
                                   rows=torch.zeros((8, 256), dtype=b16)),
        lambda: b.bfq_moe_combine_backward(torch.zeros(4, 256), 2, rows=torch.zeros((8, 256), dtype=torch.int8),
                                           rows_scales=torch.zeros(8, 2), d_weights=torch.zeros(4, 2)),
        lambda: b.bfq_gated_checkpoint(torch.zeros((4, 512), dtype=b16), h=torch.zeros((4, 256), dtype=b16)),
    )


def _told(call):
    try:
        return repr(call())
    except Exception as e:
        return f"{type(e).__name__}: {e}"


def _held_before(b, stop):
    """Four calls while another thread's first call stands before the stop-th line of the setup; the lines
    that the setup has, and what every call was told."""
    lines, held, go, out = [], threading.Event(), threading.Event(), []
    setup = b._runtime.__code__
    parts = {setup, *(c for c in setup.co_consts if hasattr(c, "co_code"))}     # and its comprehensions
    parts |= {c for p in tuple(parts) for c in p.co_consts if hasattr(c, "co_code")}

    def trace(frame, event, arg):
        if event == "call":
            return trace if frame.f_code in parts else None
        if event == "line":
            if len(lines) == stop:
                held.set()
                go.wait(20)
            lines.append(frame.f_lineno)
        return trace

    def first():
        sys.settrace(trace)
        try:
            out.append(_told(_calls(b)[0]))
        finally:
            sys.settrace(None)
            held.set()

    t = threading.Thread(target=first)
    t.start()
    assert held.wait(20)
    told = [_told(c) for c in _calls(b)]
    go.set()
    t.join()
    return len(lines), told + out + [_told(c) for c in _calls(b)]


@pytest.mark.parametrize("gpu", [False, True])
def test_first_calls_from_two_threads(monkeypatch, gpu):
    if gpu:                                  # as where the runtime is initialised; host tensors stop before it
        monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    n = stop = 0
    while stop <= n:
        n, told = _held_before(_fresh_binding(), stop)
        for got in told:
            assert got.startswith("BfqArgumentError") and "need a GPU tensor" in got, (stop, got)
        stop += 1
    assert n >= 8


def test_stream_call_is_there_before_the_device_call(monkeypatch):
    """A call that finds the device's call uses the stream's without looking again."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    b, seen = _fresh_binding(), []

    def trace(frame, event, arg):
        if frame.f_code is b._runtime.__code__:
            frame.f_trace_opcodes = True       # between the assignments of one line too
            seen.append((b._device_now, b._stream_now))
            return trace

    t = threading.Thread(target=lambda: (sys.settrace(trace), b._runtime(), sys.settrace(None)))
    t.start()
    t.join()
    assert seen and all(s is not None for d, s in seen if d is not None) and b._device_now is not None
