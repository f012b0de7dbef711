"""What the cache and attention calls take: descriptors of derived classes and as they are, types of older and newer
torch, and defaults that follow the cache (no GPU needed: nothing below is launched)."""

import ctypes
import enum
import importlib.util
import sys

import pytest

import quantized_routed_expert_03_gb300 as qre
from test_attention_abi import A, attn, cache, lib, rows   # noqa: F401
from test_rows_abi import rope


def test_descriptors_of_derived_classes_are_taken(lib):
    class Mine(qre.qre_kv_cache):
        pass

    class Rows(qre.qre_kv_rows):
        pass
    c, r = cache(), rows()
    mine, mine_rows = Mine.from_buffer_copy(c), Rows.from_buffer_copy(r)
    qre.qre_kv_write(mine, 0, mine_rows, 0, None, None, None, None, stream=0)
    assert qre.qre_kv_workspace_size(mine) == qre.qre_kv_workspace_size(c)
    for wrong in (r, None, A, ctypes.byref(c)):
        with pytest.raises(TypeError, match="qre_kv_cache"):
            qre.qre_kv_write(wrong, 0, r, 0, None, None, None, None, stream=0)


def test_the_librarys_own_functions_know_their_descriptors(lib):
    c, r, a, p = cache(), rows(), attn(), rope()
    for f, good, rest in ((lib.qre_kv_write, (c, 0, r), (0, None, None, None, None, None)),
                          (lib.qre_kv_read, (c, 0, r), (0, None, None, None, 0, None, None, None)),
                          (lib.qre_qk_norm_rope, (p,), (0, None, None, None, None, None, None)),
                          (lib.qre_attn_decode, (a, c, 0), (0, None, 0, None, None, None, None, 0, None))):
        ways = (lambda x: x, ctypes.byref, ctypes.pointer, ctypes.addressof)
        for way in ways:
            assert f(*[way(x) if isinstance(x, ctypes.Structure) else x for x in good], *rest) == qre.QRE_OK
        for i, x in enumerate(good):
            if isinstance(x, ctypes.Structure):
                for other in (c, r, a, p):
                    if type(other) is not type(x):
                        for way in ways[:3]:
                            with pytest.raises(ctypes.ArgumentError):
                                f(*[way(other) if j == i else y for j, y in enumerate(good)], *rest)
                assert f(*[None if j == i else y for j, y in enumerate(good)], *rest) == qre.QRE_ERR_INVALID_ARG


@pytest.mark.skipif(not hasattr(sys, "monitoring"), reason="sys.monitoring is Python 3.12's")
def test_arguments_that_have_no_address_raise_nothing_on_the_way():
    """None and plain addresses are common (no log-sums, sequences 0, 1, and so on): an exception for each would take most
    of a small call's time."""
    class Address(enum.IntEnum):
        X = 48
    raised, mon = [], sys.monitoring
    mon.use_tool_id(mon.DEBUGGER_ID, "raised")
    try:
        mon.register_callback(mon.DEBUGGER_ID, mon.events.RAISE, lambda code, at, e: raised.append(code.co_name))
        mon.set_events(mon.DEBUGGER_ID, mon.events.RAISE)
        assert qre._ptr(None) is None and qre._ptr(0) == 0 and qre._ptr(A) == A
    finally:
        mon.set_events(mon.DEBUGGER_ID, 0)
        mon.register_callback(mon.DEBUGGER_ID, mon.events.RAISE, None)
        mon.free_tool_id(mon.DEBUGGER_ID)
    assert raised == []
    assert qre._ptr(Address.X) == 48 and qre._ptr(True) == 1
    for other in ("x", 1.5, object()):
        with pytest.raises(AttributeError):
            qre._ptr(other)


def test_a_torch_without_4_bit_types_has_the_other_caches(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    from quantized_routed_expert_03_gb300 import attention
    monkeypatch.delattr(torch, "float4_e2m1fn_x2", raising=False)
    spec = importlib.util.spec_from_file_location("quantized_routed_expert_03_gb300.older", attention.__file__)
    older = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(older)
    for dtype in (torch.bfloat16, torch.float16, torch.float8_e4m3fn):
        assert older.KVCache(1, 4, 2, 16, 64, 2, 4, dtype, device="cpu").k.dtype == dtype
    assert qre.QRE_E2M1 not in older.DTYPES.values()


def test_rows_are_read_in_the_caches_own_type(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    from quantized_routed_expert_03_gb300 import attention
    seen = []
    monkeypatch.setattr(attention, "qre_kv_read", lambda cache, layer, rows, *rest: seen.append(rows.dtype))
    cu = torch.tensor([0, 3], dtype=torch.int32)
    B, H = torch.bfloat16, torch.float16
    rows = {t: torch.zeros((3, 2, 64), dtype=t) for t in (B, H)}
    for kind, kw, want in ((B, {}, B), (H, {}, H), (torch.float8_e4m3fn, {}, B), (torch.float8_e4m3fn, dict(dtype=H), H),
                           (torch.float8_e4m3fn, dict(k=rows[H]), H), (torch.float8_e4m3fn, dict(v=rows[H]), H),
                           (H, dict(k=rows[H], v=rows[H]), H)):
        cache = attention.KVCache(1, 4, 2, 16, 64, 2, 4, kind, device="cpu")
        k, v = cache.read(0, None, cu, 3, **kw)
        assert k.dtype == v.dtype == want and seen.pop() == attention.DTYPES[want]


def test_common_lengths_of_sequences_in_order(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    from quantized_routed_expert_03_gb300 import attention
    seen = []
    monkeypatch.setattr(attention, "qre_kv_common_len", lambda cache, n, seqs, groups, *rest: seen.append((n, seqs, groups)))
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    for held, n in ((7, 7), (4096, 4096), (5000, 4096)):
        cache = attention.KVCache(1, 4, 2, 16, 64, held, 4, device="cpu")
        assert cache.common_len(None, cu).shape == (2,) and seen.pop() == (n, None, 2)
    with pytest.raises(ValueError, match="seqs"):
        cache.common_len(cu.long(), cu)


def test_heads_in_host_memory_are_refused(lib, monkeypatch):
    """Everything on one device, and that is not a GPU: the kernel would be given host addresses."""
    torch = pytest.importorskip("torch")
    from quantized_routed_expert_03_gb300 import attention
    ran = []
    for name in ("qre_qk_norm_rope", "qre_kv_write_rope"):
        monkeypatch.setattr(attention, name, lambda *a: ran.append(a))
    q, k = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    pos = torch.arange(3, dtype=torch.int32)
    cache = attention.KVCache(1, 4, 2, 16, 64, 2, 4, device="cpu")
    for rotary in (attention.Rotary(4, 2, 64, device="cpu"), attention.Rotary(4, 2, 64, rot_dim=0)):
        with pytest.raises(ValueError, match="GPU"):
            rotary.apply(q, k, pos)
        with pytest.raises(ValueError, match="GPU"):
            cache.write_rope(0, rotary, pos, pos, q, k, k)
    assert not ran


def test_an_odd_number_of_turned_elements_is_refused(lib):
    """(With 16 angles of its own, 33 elements were taken for 32.)"""
    torch = pytest.importorskip("torch")
    from quantized_routed_expert_03_gb300.attention import Rotary
    for kw in ({}, dict(inv_freq=torch.ones(16))):
        with pytest.raises(ValueError, match="rot_dim 33"):
            Rotary(4, 2, 64, rot_dim=33, device="cpu", **kw)
