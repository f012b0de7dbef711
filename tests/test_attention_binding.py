"""The Python side of the cache and attention calls: what it makes of its arguments before a call (no GPU needed)."""

import sys
import types

import pytest

import quantized_routed_expert_03_gb300 as qre
from quantized_routed_expert_03_gb300 import build as qbuild


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


@pytest.fixture(scope="module")
def pair():
    """A cache and an attention in host memory: every call below is refused before anything would run on it."""
    torch = pytest.importorskip("torch")
    from quantized_routed_expert_03_gb300.attention import Attention, KVCache
    qbuild.build()
    cache = KVCache(2, 20, 2, 16, 64, 4, 8, device="cpu")
    return torch, cache, Attention(cache, 0, 8, 4)


def ids(torch, n, kind):
    t = torch.arange(2 * n, dtype=torch.int32)
    return {"int64": t[:n].long(), "strided": t[::2], "short": t[:n - 1], "2d": t[:n].view(1, n), "float": t[:n].float()}[kind]


@pytest.mark.parametrize("kind", ["int64", "strided", "short", "2d", "float"])
def test_ids_that_are_not_int32_in_a_row_are_refused(pair, kind):
    torch, cache, att = pair
    good, bad = torch.arange(3, dtype=torch.int32), ids(torch, 3, kind)
    rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    calls = [("n_new", lambda: cache.reserve(good, bad)), ("token_pos", lambda: cache.write(0, good, bad, rows, rows)),
             ("dst", lambda: cache.fork(good, bad)), ("cu_k", lambda: att.prefill(q, rows, rows, good, bad)),
             ("seqs", lambda: att.decode(q, bad))]
    if kind != "short":
        calls += [("seqs", lambda: cache.reserve(bad, good)), ("token_seq", lambda: cache.write(0, bad, good, rows, rows)),
                  ("src", lambda: cache.fork(bad, good)), ("seqs", lambda: cache.free(bad)),
                  ("cu_q", lambda: att.prefill(q, rows, rows, bad, good))]
    for name, call in calls:
        with pytest.raises(ValueError, match=name):
            call()


def test_arrays_of_another_shape_or_type_are_refused(pair):
    torch, cache, att = pair
    i = torch.arange(3, dtype=torch.int32)
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)      # noqa: E731
    rows, q = z(3, 2, 64), z(3, 8, 64)
    for name, call in [
            ("k has", lambda: cache.write(0, i, i, z(2, 2, 64), rows)), ("k has", lambda: cache.write(0, i, i, z(3, 3, 64), rows)),
            ("v has", lambda: cache.write(0, i, i, rows, z(3, 2, 64, dtype=torch.float16))),
            ("v has", lambda: cache.write(0, i, i, rows, z(3, 2, 32))),
            ("q has", lambda: att.decode(z(3, 8, 64, dtype=torch.float32), i)), ("q has", lambda: att.decode(z(3, 4, 64), i)),
            ("o has", lambda: att.decode(q, i, o=z(2, 8, 64))), ("o has", lambda: att.decode(q, i, o=z(3, 8, 64, dtype=torch.float32))),
            ("lse has", lambda: att.decode(q, i, lse=z(3, 8))), ("lse has", lambda: att.decode(q, i, lse=z(8, 3, dtype=torch.float32).T)),
            ("k has", lambda: att.prefill(q, z(5, 8, 64), rows, i, i)), ("v has", lambda: att.prefill(q, rows, z(2, 2, 64), i, i)),
            ("k has", lambda: att.prefill(q, z(3, 2, 64, dtype=torch.float16), rows, i, i)),
            ("o has", lambda: att.prefill(q, rows, rows, i, i, o=z(3, 8, 128)))]:
        with pytest.raises(ValueError, match=name):
            call()


def test_scales_of_another_shape_or_type_are_refused(pair):
    torch, _, _ = pair
    from quantized_routed_expert_03_gb300.attention import KVCache
    for name, scales in (("k_scale", (torch.ones(2), None)), ("v_scale", (None, torch.ones((2, 2), dtype=torch.float64))),
                         ("k_scale", (torch.ones((2, 4))[:, ::2], None))):
        with pytest.raises(ValueError, match=name):
            KVCache(2, 20, 2, 16, 64, 4, 8, torch.float8_e4m3fn, *scales, device="cpu")
