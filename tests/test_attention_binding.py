"""The Python side of the cache and attention calls: what it makes of its arguments before a call (no GPU needed)."""

import sys
import types

import pytest

import quantized_routed_expert_03_gb300 as qre


@pytest.mark.skipif(not hasattr(sys, "monitoring"), reason="sys.monitoring is Python 3.12's")
def test_the_current_stream_is_found_by_threads_that_ask_at_once(monkeypatch):
    """A second thread at every point of the first call of a process: none may find a half-made state."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 40 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    # a fresh copy of the function and the names that it keeps
    fresh = dict(vars(qre))
    for name in ("_raw_stream", "_current_device", "_current_stream"):
        if name in fresh:
            fresh[name] = None
    call = types.FunctionType(qre._stream.__code__.replace(), fresh)
    points = []

    def other_thread(code, offset):
        if not points or points[-1] is not None:
            points.append(None)              # (not again for the call below)
            keep = dict(fresh)
            points[-1] = call(None)
            fresh.clear()
            fresh.update(keep)               # what the first thread had left when it was interrupted

    mon = sys.monitoring
    mon.use_tool_id(mon.DEBUGGER_ID, "threads")
    try:
        mon.register_callback(mon.DEBUGGER_ID, mon.events.INSTRUCTION, other_thread)
        mon.set_local_events(mon.DEBUGGER_ID, call.__code__, mon.events.INSTRUCTION)
        first = call(None)
    finally:
        mon.set_local_events(mon.DEBUGGER_ID, call.__code__, 0)
        mon.register_callback(mon.DEBUGGER_ID, mon.events.INSTRUCTION, None)
        mon.free_tool_id(mon.DEBUGGER_ID)
    assert first == 42 and len(points) > 10 and set(points) == {42}
