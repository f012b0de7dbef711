"""Python binding of libqre.so: the quantized routed-expert MoE layer for GB300.

Argument marshalling only.  Every function has the name of the C entry point it
calls (declared in ``include/qre.h``); every step of the layer runs in the
library's CUDA kernels.  Tensor arguments may be ``torch.Tensor`` (their
``data_ptr()`` is passed), plain integer addresses, or ``None`` for NULL.  The
stream defaults to torch's current CUDA stream.  A non-zero status raises
:class:`QreError` carrying the library's message.

There is no fallback: if ``libqre.so`` has not been built, importing works but
the first call raises, naming the build command.
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqre.so")

QRE_OK = 0
QRE_ERR_INVALID_ARG = 1
QRE_ERR_UNSUPPORTED = 2
QRE_ERR_MISALIGNED = 3
QRE_ERR_WORKSPACE = 4
QRE_ERR_CUDA = 5
QRE_ERR_TIMEOUT = 6
QRE_ERR_DEVICE_CHECK = 7

QRE_DEV_TIMEOUT = 0x1
QRE_DEV_NULL_SLOT = 0x2
QRE_DEV_BAD_SCALE = 0x4
QRE_DEV_BAD_INDEX = 0x8
QRE_DEV_FP16_RANGE = 0x10
QRE_DEV_NO_PAGE = 0x20

# qre_dtype
QRE_BF16 = 0
QRE_FP16 = 1
QRE_E4M3 = 2

# Every symbol include/qre.h declares.
EXPORTS = (
    "qre_last_error", "qre_status_string", "qre_version", "qre_workspace_size", "qre_quantize",
    "qre_quantize_gate_up",
    "qre_route", "qre_dispatch", "qre_expert_ffn", "qre_combine", "qre_validate_slots",
    "qre_cache_update", "qre_cache_copy",
    "qre_read_device_status", "qre_clear_device_status", "qre_route_noalloc", "qre_debug_wait_test",
    "qre_expert_ffn_routed", "qre_expert_ffn_shared", "qre_shared_workspace_size", "qre_stage_experts",
    "qre_read_probe", "qre_set_host_unit_cost", "qre_route_dispatch",
    "qre_kv_workspace_size", "qre_kv_reserve", "qre_kv_write", "qre_kv_fork", "qre_kv_free", "qre_kv_compact",
    "qre_attn_prefill", "qre_attn_decode_workspace_size", "qre_attn_decode",
)


class qre_layer_shape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("group", ctypes.c_int32)]


class qre_slot(ctypes.Structure):
    _fields_ = [("w_gate_up", ctypes.c_void_p), ("s_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_down", ctypes.c_void_p), ("tier", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class qre_kv_cache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "page_table", "seq_len", "ref_count", "k_scale", "v_scale")]
                + [(n, ctypes.c_int32) for n in ("n_layers", "n_pages", "n_kv_heads", "page_size", "head_dim",
                                                 "max_seqs", "max_pages", "dtype")])


class qre_kv_rows(ctypes.Structure):
    _fields_ = [("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64), ("v_token", ctypes.c_int64),
                ("v_head", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class qre_attn(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_heads", "n_kv_heads", "head_dim", "dtype")]
                + [("scale", ctypes.c_float), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                   ("reserved", ctypes.c_int32)]
                + [(n, ctypes.c_int64) for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head",
                                                 "o_token", "o_head")])


class QreError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS_NAMES.get(status, status)}: {message}")


_STATUS_NAMES = {0: "QRE_OK", 1: "QRE_ERR_INVALID_ARG", 2: "QRE_ERR_UNSUPPORTED", 3: "QRE_ERR_MISALIGNED",
                 4: "QRE_ERR_WORKSPACE", 5: "QRE_ERR_CUDA", 6: "QRE_ERR_TIMEOUT", 7: "QRE_ERR_DEVICE_CHECK"}

_lib = None

_VP, _I32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_SHAPE = ctypes.POINTER(qre_layer_shape)
_KV, _ATTN, _ROWS = ctypes.POINTER(qre_kv_cache), ctypes.POINTER(qre_attn), ctypes.POINTER(qre_kv_rows)
_SIGS = {
    "qre_last_error": ([], ctypes.c_char_p),
    "qre_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "qre_version": ([], ctypes.c_int32),
    "qre_workspace_size": ([_SHAPE, _I32, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "qre_quantize": ([_I32, _I32, _I32, _VP, _VP, _VP, _VP], ctypes.c_int),
    "qre_quantize_gate_up": ([_I32, _I32, _I32, _VP, _VP, _VP, _VP, _VP], ctypes.c_int),
    "qre_route": ([_SHAPE, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "qre_dispatch": ([_SHAPE, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "qre_expert_ffn": ([_SHAPE, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "qre_combine": ([_SHAPE, _I32, _VP, _VP, _VP, _VP, _VP, _VP], ctypes.c_int),
    "qre_validate_slots": ([_SHAPE, ctypes.POINTER(qre_slot)], ctypes.c_int),
    "qre_cache_update": ([_SHAPE, _I32, ctypes.c_float, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP],
                         ctypes.c_int),
    "qre_cache_copy": ([_SHAPE, _VP, _VP, _VP, _VP, _I32, _VP], ctypes.c_int),
    "qre_read_device_status": ([_VP, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
    "qre_clear_device_status": ([_VP], ctypes.c_int),
    "qre_route_noalloc": ([_SHAPE, _I32, _VP, _VP, _VP, _VP, _VP, _VP], ctypes.c_int),
    "qre_debug_wait_test": ([ctypes.c_uint64, ctypes.c_uint64], ctypes.c_int),
    "qre_expert_ffn_routed": ([_SHAPE, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "qre_expert_ffn_shared": ([_SHAPE, _I32, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "qre_shared_workspace_size": ([_SHAPE, _I32, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "qre_stage_experts": ([_SHAPE, ctypes.POINTER(qre_slot), ctypes.POINTER(qre_slot), _I32, _VP, _VP,
                           ctypes.POINTER(ctypes.c_int32), _VP], ctypes.c_int),
    "qre_read_probe": ([_VP, _SZ, _VP, _VP], ctypes.c_int),
    "qre_set_host_unit_cost": ([_I32], ctypes.c_int),
    "qre_route_dispatch": ([_SHAPE, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
                           ctypes.c_int),
    "qre_kv_workspace_size": ([_KV, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "qre_kv_reserve": ([_KV, _I32, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "qre_kv_write": ([_KV, _I32, _ROWS, _I32, _VP, _VP, _VP, _VP, _VP], ctypes.c_int),
    "qre_kv_fork": ([_KV, _I32, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "qre_kv_free": ([_KV, _I32, _VP, _VP], ctypes.c_int),
    "qre_kv_compact": ([_KV, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "qre_attn_prefill": ([_ATTN, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP], ctypes.c_int),
    "qre_attn_decode_workspace_size": ([_ATTN, _KV, _I32, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "qre_attn_decode": ([_ATTN, _KV, _I32, _I32, _VP, _I32, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
}


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libqre.so (once) and declares the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m quantized_routed_expert_03_gb300.build` (needs nvcc)")
    lib = ctypes.CDLL(path)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current_stream = None


def _stream(s):
    if s is None:
        # the current stream's handle without a Stream object: 0.3 us instead of 3 us of every call
        global _current_stream
        if _current_stream is None:
            import torch
            raw, device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
            _current_stream = lambda: raw(device())      # one name: other threads see all of it or nothing
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, where: str) -> None:
    if status != QRE_OK:
        raise QreError(status, where, load_library().qre_last_error().decode())


def _nbytes(t, given):
    if given is not None:
        return given
    if t is None:
        return 0
    return t.numel() * t.element_size()


def make_shape(hidden: int, inter: int, n_experts: int, top_k: int, group: int) -> qre_layer_shape:
    return qre_layer_shape(hidden, inter, n_experts, top_k, group)


def qre_version() -> int:
    return load_library().qre_version()


def qre_status_string(status: int) -> str:
    return load_library().qre_status_string(status).decode()


def qre_last_error() -> str:
    return load_library().qre_last_error().decode()


def qre_workspace_size(shape: qre_layer_shape, T: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().qre_workspace_size(ctypes.byref(shape), T, ctypes.byref(out)), "qre_workspace_size")
    return out.value


def qre_quantize(n_rows, k_dim, group, w, packed, scales, stream=None) -> None:
    _check(load_library().qre_quantize(n_rows, k_dim, group, _ptr(w), _ptr(packed), _ptr(scales),
                                       _stream(stream)), "qre_quantize")


def qre_quantize_gate_up(inter, hidden, group, w_gate, w_up, packed, scales, stream=None) -> None:
    _check(load_library().qre_quantize_gate_up(inter, hidden, group, _ptr(w_gate), _ptr(w_up), _ptr(packed),
                                               _ptr(scales), _stream(stream)), "qre_quantize_gate_up")


def qre_route(shape, T, x_bf16, w_router, bias, topk_idx, topk_w, workspace, workspace_bytes=None,
              stream=None) -> None:
    _check(load_library().qre_route(ctypes.byref(shape), T, _ptr(x_bf16), _ptr(w_router), _ptr(bias),
                                    _ptr(topk_idx), _ptr(topk_w), _ptr(workspace),
                                    _nbytes(workspace, workspace_bytes), _stream(stream)), "qre_route")


def qre_route_noalloc(shape, T, x_bf16, w_router, bias, topk_idx, topk_w, stream=None) -> None:
    """qre_route for callers that cannot allocate device memory: the logits scratch
    is a fixed array inside the library (T * n_experts <= 65,536)."""
    _check(load_library().qre_route_noalloc(ctypes.byref(shape), T, _ptr(x_bf16), _ptr(w_router), _ptr(bias),
                                            _ptr(topk_idx), _ptr(topk_w), _stream(stream)), "qre_route_noalloc")


def qre_route_dispatch(shape, T, x_bf16, w_router, bias, topk_idx, topk_w, counts, offsets, perm, inv_perm, active,
                       n_active, workspace, workspace_bytes=None, stream=None) -> None:
    _check(load_library().qre_route_dispatch(ctypes.byref(shape), T, _ptr(x_bf16), _ptr(w_router), _ptr(bias),
                                             _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(perm),
                                             _ptr(inv_perm), _ptr(active), _ptr(n_active), _ptr(workspace),
                                             _nbytes(workspace, workspace_bytes), _stream(stream)),
           "qre_route_dispatch")


def qre_dispatch(shape, T, topk_idx, counts, offsets, perm, inv_perm, active, n_active, workspace,
                 workspace_bytes=None, stream=None) -> None:
    _check(load_library().qre_dispatch(ctypes.byref(shape), T, _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                                       _ptr(perm), _ptr(inv_perm), _ptr(active), _ptr(n_active),
                                       _ptr(workspace), _nbytes(workspace, workspace_bytes), _stream(stream)),
           "qre_dispatch")


def qre_expert_ffn(shape, T, x_bf16, slots, offsets, perm, active, n_active, expert_out, workspace,
                   workspace_bytes=None, stream=None) -> None:
    _check(load_library().qre_expert_ffn(ctypes.byref(shape), T, _ptr(x_bf16), _ptr(slots), _ptr(offsets),
                                         _ptr(perm), _ptr(active), _ptr(n_active), _ptr(expert_out),
                                         _ptr(workspace), _nbytes(workspace, workspace_bytes), _stream(stream)),
           "qre_expert_ffn")


def qre_expert_ffn_routed(shape, T, x_bf16, slots, offsets, perm, active, n_active, expert_out, workspace,
                          workspace_bytes=None, stream=None) -> None:
    _check(load_library().qre_expert_ffn_routed(ctypes.byref(shape), T, _ptr(x_bf16), _ptr(slots), _ptr(offsets),
                                                _ptr(perm), _ptr(active), _ptr(n_active), _ptr(expert_out),
                                                _ptr(workspace), _nbytes(workspace, workspace_bytes),
                                                _stream(stream)), "qre_expert_ffn_routed")


def qre_expert_ffn_shared(shape, T, x_bf16, slots, expert_out, workspace, workspace_bytes=None,
                          stream=None) -> None:
    _check(load_library().qre_expert_ffn_shared(ctypes.byref(shape), T, _ptr(x_bf16), _ptr(slots),
                                                _ptr(expert_out), _ptr(workspace),
                                                _nbytes(workspace, workspace_bytes), _stream(stream)),
           "qre_expert_ffn_shared")


def qre_shared_workspace_size(shape: qre_layer_shape, T: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().qre_shared_workspace_size(ctypes.byref(shape), T, ctypes.byref(out)),
           "qre_shared_workspace_size")
    return out.value


def qre_combine(shape, T, expert_out, topk_w, inv_perm, y_f32, y_bf16, stream=None) -> None:
    _check(load_library().qre_combine(ctypes.byref(shape), T, _ptr(expert_out), _ptr(topk_w), _ptr(inv_perm),
                                       _ptr(y_f32), _ptr(y_bf16), _stream(stream)), "qre_combine")


def qre_cache_update(shape, n_slots, decay, active, n_active, scores, expert_slot, slot_expert, home, slot_mem,
                     table, copy_list, n_copies, max_copies, stream=None) -> None:
    _check(load_library().qre_cache_update(ctypes.byref(shape), n_slots, decay, _ptr(active), _ptr(n_active),
                                           _ptr(scores), _ptr(expert_slot), _ptr(slot_expert), _ptr(home),
                                           _ptr(slot_mem), _ptr(table), _ptr(copy_list), _ptr(n_copies),
                                           max_copies, _stream(stream)), "qre_cache_update")


def qre_cache_copy(shape, home, slot_mem, copy_list, n_copies, max_copies, stream=None) -> None:
    _check(load_library().qre_cache_copy(ctypes.byref(shape), _ptr(home), _ptr(slot_mem), _ptr(copy_list),
                                         _ptr(n_copies), max_copies, _stream(stream)), "qre_cache_copy")


def qre_stage_experts(shape, host_table, host_staging, host_out, table_out, stream=None) -> int:
    """Stages the host-resident experts of ``host_table`` (ctypes qre_slot array) into
    ``host_staging`` slots; ``host_out``: a host buffer of (E + 1) qre_slot (an int
    address or a tensor, kept alive until the stream passes the call); returns the
    number of experts staged."""
    n = ctypes.c_int32(0)
    _check(load_library().qre_stage_experts(ctypes.byref(shape), host_table, host_staging, len(host_staging),
                                            _ptr(host_out), _ptr(table_out), ctypes.byref(n), _stream(stream)),
           "qre_stage_experts")
    return n.value


def qre_read_probe(src, nbytes, sink, stream=None) -> None:
    """One streaming read of ``nbytes`` at ``src`` (device or host-mapped); time it with events."""
    _check(load_library().qre_read_probe(_ptr(src), nbytes, _ptr(sink), _stream(stream)), "qre_read_probe")


def qre_validate_slots(shape, host_slots) -> None:
    """host_slots: a ctypes array of qre_slot (n_experts + 1 entries) in host memory."""
    _check(load_library().qre_validate_slots(ctypes.byref(shape), host_slots), "qre_validate_slots")


def qre_debug_wait_test(wait_limit_ns: int, stall_ns: int) -> None:
    """Test hook: lower the kernels' wait limit and delay one warp of the expert
    FFN's first CTA, so that the give-up path runs (0, 0 restores the defaults)."""
    _check(load_library().qre_debug_wait_test(wait_limit_ns, stall_ns), "qre_debug_wait_test")


def qre_set_host_unit_cost(cost: int) -> None:
    """Process-wide: cut the decode kernels' work at equal cost with a host-mapped
    unit counted as ``cost`` (0 or 1: equal counts, the default)."""
    _check(load_library().qre_set_host_unit_cost(cost), "qre_set_host_unit_cost")


def make_kv_cache(k, v, page_table, seq_len, ref_count, dtype, k_scale=None, v_scale=None) -> qre_kv_cache:
    """Descriptor of a paged cache from its tensors: k, v [n_layers, n_pages, n_kv_heads, page_size, head_dim]
    (contiguous), page_table [max_seqs, max_pages], seq_len [max_seqs], ref_count [n_pages] int32.  It holds
    addresses only: keep the tensors alive."""
    L, P, H, S, D = k.shape
    assert v.shape == k.shape and k.is_contiguous() and v.is_contiguous() and page_table.is_contiguous()
    assert seq_len.numel() == page_table.shape[0] and ref_count.numel() == P
    return qre_kv_cache(_ptr(k), _ptr(v), _ptr(page_table), _ptr(seq_len), _ptr(ref_count), _ptr(k_scale),
                        _ptr(v_scale), L, P, H, S, D, page_table.shape[0], page_table.shape[1], dtype)


def _strides(t):
    if t is None:
        return 0, 0
    assert t.dim() == 3 and (t.shape[2] == 0 or t.stride(2) == 1), "[tokens, heads, head_dim] with contiguous rows"
    return t.stride(0), t.stride(1)


def make_kv_rows(dtype, k, v) -> qre_kv_rows:
    """Type and strides of new rows k, v [tokens, n_kv_heads, head_dim]."""
    return qre_kv_rows(*_strides(k), *_strides(v), dtype, 0)


def make_attn(n_heads, n_kv_heads, head_dim, dtype, scale, causal=True, window=0, q=None, k=None, v=None,
              o=None) -> qre_attn:
    """Descriptor of an attention; the strides are taken from q, k, v, o [tokens, heads, head_dim] (k and v may be
    left out for qre_attn_decode)."""
    return qre_attn(n_heads, n_kv_heads, head_dim, dtype, scale, 1 if causal else 0, window, 0, *_strides(q),
                    *_strides(k), *_strides(v), *_strides(o))


def qre_kv_workspace_size(cache: qre_kv_cache) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().qre_kv_workspace_size(ctypes.byref(cache), ctypes.byref(out)), "qre_kv_workspace_size")
    return out.value


def qre_kv_reserve(cache, n, seqs, n_new, workspace, workspace_bytes=None, stream=None) -> None:
    _check(load_library().qre_kv_reserve(ctypes.byref(cache), n, _ptr(seqs), _ptr(n_new), _ptr(workspace),
                                         _nbytes(workspace, workspace_bytes), _stream(stream)), "qre_kv_reserve")


def qre_kv_write(cache, layer, rows, n_tokens, token_seq, token_pos, k, v, stream=None) -> None:
    _check(load_library().qre_kv_write(ctypes.byref(cache), layer, ctypes.byref(rows), n_tokens, _ptr(token_seq),
                                       _ptr(token_pos), _ptr(k), _ptr(v), _stream(stream)), "qre_kv_write")


def qre_kv_fork(cache, n, src, dst, workspace, workspace_bytes=None, stream=None) -> None:
    _check(load_library().qre_kv_fork(ctypes.byref(cache), n, _ptr(src), _ptr(dst), _ptr(workspace),
                                      _nbytes(workspace, workspace_bytes), _stream(stream)), "qre_kv_fork")


def qre_kv_free(cache, n, seqs, stream=None) -> None:
    _check(load_library().qre_kv_free(ctypes.byref(cache), n, _ptr(seqs), _stream(stream)), "qre_kv_free")


def qre_kv_compact(cache, page_table_out, ref_count_out, n_live, workspace, workspace_bytes=None,
                   stream=None) -> None:
    _check(load_library().qre_kv_compact(ctypes.byref(cache), _ptr(page_table_out), _ptr(ref_count_out),
                                         _ptr(n_live), _ptr(workspace), _nbytes(workspace, workspace_bytes),
                                         _stream(stream)), "qre_kv_compact")


def qre_attn_prefill(attn, n_seqs, total_q, total_k, cu_q, cu_k, q, k, v, o, lse=None, stream=None) -> None:
    _check(load_library().qre_attn_prefill(ctypes.byref(attn), n_seqs, total_q, total_k, _ptr(cu_q), _ptr(cu_k),
                                           _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _stream(stream)),
           "qre_attn_prefill")


def qre_attn_decode_workspace_size(attn: qre_attn, cache: qre_kv_cache, n: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().qre_attn_decode_workspace_size(ctypes.byref(attn), ctypes.byref(cache), n,
                                                         ctypes.byref(out)), "qre_attn_decode_workspace_size")
    return out.value


def qre_attn_decode(attn, cache, layer, n, seqs, max_len, q, o, lse, workspace, workspace_bytes=None,
                    stream=None) -> None:
    _check(load_library().qre_attn_decode(ctypes.byref(attn), ctypes.byref(cache), layer, n, _ptr(seqs), max_len,
                                          _ptr(q), _ptr(o), _ptr(lse), _ptr(workspace),
                                          _nbytes(workspace, workspace_bytes), _stream(stream)), "qre_attn_decode")


def qre_read_device_status(stream=None) -> int:
    out = ctypes.c_int32(0)
    _check(load_library().qre_read_device_status(_stream(stream), ctypes.byref(out)), "qre_read_device_status")
    return out.value


def qre_clear_device_status(stream=None) -> None:
    _check(load_library().qre_clear_device_status(_stream(stream)), "qre_clear_device_status")


def slot_array(entries) -> ctypes.Array:
    """Host ctypes array of qre_slot from (w_gate_up, s_gate_up, w_down, s_down, tier) tuples of addresses."""
    arr = (qre_slot * len(entries))()
    for i, (wg, sg, wd, sd, tier) in enumerate(entries):
        arr[i] = qre_slot(_ptr(wg), _ptr(sg), _ptr(wd), _ptr(sd), tier, 0)
    return arr
