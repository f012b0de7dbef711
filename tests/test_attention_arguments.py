"""What the cache and attention calls take: descriptors of derived classes and as they are, types of older and newer
torch, and defaults that follow the cache (no GPU needed: nothing below is launched)."""

import ctypes
import importlib.util
import os

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
