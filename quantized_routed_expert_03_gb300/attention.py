"""Device plumbing for attention: the paged key-value cache and the two attention calls over it.

Like ``layer``, PyTorch only allocates memory and supplies streams here; every
computation is a call into libqre.so through the binding in ``__init__``.

* :class:`KVCache` owns the pages of all layers and the device state (page table,
  lengths, reference counts): reserve, write, read, fork, free, compact.
* :class:`Rotary` norms and turns a layer's queries and keys, on arrays (``apply``)
  or on the way into the pages (``KVCache.write_rope``).
* :class:`Attention` is one layer's attention on such a cache: ``prefill`` over
  packed prompts (keys and values as they come from the projections), ``decode``
  of one new token per sequence over the pages, ``decode_shared`` where groups of
  sequences share the pages of a prefix.

Caches and attentions keep a workspace: calls on one object belong on one stream at a time.  A
result allocated here belongs to the stream that the call was given, like any
tensor made there: a program that uses it on another stream waits for the call
and, before it lets go of the tensor, tells the allocator (``record_stream``).
"""

from __future__ import annotations

import torch

from . import (QRE_BF16, QRE_E2M1, QRE_E4M3, QRE_FP16, make_attn, make_kv_cache, make_kv_rows, make_rope,
               qre_attn_decode, qre_attn_decode_shared, qre_attn_decode_shared_workspace_size,
               qre_attn_decode_workspace_size, qre_attn_prefill, qre_kv_common_len, qre_kv_compact, qre_kv_fork,
               qre_kv_free, qre_kv_read, qre_kv_reserve, qre_kv_workspace_size, qre_kv_write, qre_kv_write_rope,
               qre_qk_norm_rope)

DTYPES = {torch.bfloat16: QRE_BF16, torch.float16: QRE_FP16, torch.float8_e4m3fn: QRE_E4M3}
if hasattr(torch, "float4_e2m1fn_x2"):               # (older ones have no name for it, and the other caches without it)
    DTYPES[torch.float4_e2m1fn_x2] = QRE_E2M1


def _check_ids(device, count=None, **tensors):
    """The kernels read int32 one behind the other on the cache's device: anything else would be taken for other ids."""
    for name, t in tensors.items():
        if t.dtype != torch.int32 or not t.is_contiguous() or t.dim() != 1 or t.device != device:
            raise ValueError(f"{name} has to be a contiguous int32 tensor of one dimension on {device}, not {t.dtype} "
                             f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")
        if count is not None and t.numel() != count:
            raise ValueError(f"{name} has {t.numel()} entries, expected {count}")


def _check_array(t, name, shape, dtype, device, contiguous=False):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or (contiguous and not t.is_contiguous()):
        raise ValueError(f"{name} has to be {dtype} {tuple(shape)}{', contiguous,' if contiguous else ''} on {device}, not "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _empty(shape, dtype, device, stream):
    """An output for a call on ``stream``: memory of that stream's pool, so that nothing that another stream still does
    with a block it was given before can meet the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):        # a raw handle, 0: the default stream
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(q, stream):
    return _empty(q.shape, q.dtype, q.device, stream)


class KVCache:
    """``n_pages`` pages of ``page_size`` positions for all layers, and up to ``max_seqs`` sequences on them.

    dtype: bfloat16, float16, float8_e4m3fn, or float4_e2m1fn_x2 for codes of 4 bits with a scale for every 16 elements
    (``k`` and ``v`` are bytes then).  k_scale, v_scale: [n_layers, n_kv_heads] fp32, positive, for an E4M3 or E2M1
    cache only (None: 1).
    Sequence ids, counts and positions are contiguous int32 tensors on the device that begin at a 16-byte boundary
    (clone a slice that does not); other arguments raise ValueError; nothing here synchronizes.
    """

    def __init__(self, n_layers, n_pages, n_kv_heads, page_size, head_dim, max_seqs, max_pages,
                 dtype=torch.bfloat16, k_scale=None, v_scale=None, device="cuda"):
        self.device = torch.device(device)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.n_kv_heads, self.head_dim = n_kv_heads, head_dim
        low = DTYPES[dtype] == QRE_E2M1
        if low and head_dim % 16:
            raise ValueError(f"head_dim {head_dim} of a 4-bit cache has to be a multiple of 16")
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_dim // 16 * 9 if low else head_dim)
        self.k = torch.empty(shape, dtype=torch.uint8 if low else dtype, device=self.device)
        self.v = torch.empty_like(self.k)
        self.page_table = torch.full((max_seqs, max_pages), -1, **i32)
        self.seq_len = torch.zeros(max_seqs, **i32)
        self.ref_count = torch.zeros(n_pages, **i32)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                _check_array(t, name, (n_layers, n_kv_heads), torch.float32, self.k.device, contiguous=True)
        self.k_scale, self.v_scale = k_scale, v_scale
        self.desc = make_kv_cache(self.k, self.v, self.page_table, self.seq_len, self.ref_count, DTYPES[dtype],
                                  k_scale, v_scale)
        self.workspace = torch.empty(qre_kv_workspace_size(self.desc), dtype=torch.uint8, device=self.device)
        self.n_live = torch.zeros(1, **i32)

    def reserve(self, seqs, n_new, stream=None):
        _check_ids(self.k.device, seqs.numel(), seqs=seqs, n_new=n_new)
        qre_kv_reserve(self.desc, seqs.numel(), seqs, n_new, self.workspace, stream=stream)

    def write(self, layer, token_seq, token_pos, k, v, stream=None):
        """k, v: [tokens, n_kv_heads, head_dim], any token and head strides (views of one projection's output)."""
        _check_ids(self.k.device, token_seq.numel(), token_seq=token_seq, token_pos=token_pos)
        shape = (token_seq.numel(), self.n_kv_heads, self.head_dim)
        _check_array(k, "k", shape, k.dtype, self.k.device)
        _check_array(v, "v", shape, k.dtype, self.k.device)
        qre_kv_write(self.desc, layer, make_kv_rows(DTYPES[k.dtype], k, v), token_seq.numel(), token_seq, token_pos,
                     k, v, stream)

    def write_rope(self, layer, rotary, token_seq, token_pos, q, k, v, q_out=None, k_out=None, keep=True, stream=None):
        """Norms and turns q and k (see Rotary) and writes the keys and v; returns the queries and, if keep, the keys.
        Rows of tokens at a negative position are left as they are."""
        _check_ids(self.k.device, token_seq.numel(), token_seq=token_seq, token_pos=token_pos)
        q_out, k_out = rotary._outputs(self.k.device, token_seq.numel(), q, k, q_out, k_out, keep, stream)
        _check_array(v, "v", k.shape, k.dtype, self.k.device)
        qre_kv_write_rope(self.desc, layer, rotary._desc(q, k, v, q_out, k_out), token_seq.numel(), token_seq, token_pos,
                          q, k, v, q_out, k_out, stream)
        return q_out, k_out

    def read(self, layer, seqs, cu, total, first=None, dtype=None, k=None, v=None, stream=None):
        """The rows of sequences ``seqs`` (None: 0, 1, and so on) from positions ``first`` (None: 0) on, one sequence
        behind the other as ``cu`` [sequences + 1] says, ``total`` in all: k, v [total, n_kv_heads, head_dim].  dtype None:
        that of k or v, or the cache's, bfloat16 from an E4M3 or E2M1 cache."""
        device = self.k.device
        _check_ids(device, cu=cu)
        n = cu.numel() - 1
        for name, t in (("seqs", seqs), ("first", first)):
            if t is not None:
                _check_ids(device, n, **{name: t})
        shape = (total, self.n_kv_heads, self.head_dim)
        given = k if k is not None else v
        if given is not None:
            dtype = given.dtype
        elif dtype is None:
            dtype = self.k.dtype if self.k.dtype in (torch.bfloat16, torch.float16) else torch.bfloat16
        k = _empty(shape, dtype, device, stream) if k is None else k
        v = _empty(shape, dtype, device, stream) if v is None else v
        _check_array(k, "k", shape, dtype, device)
        _check_array(v, "v", shape, dtype, device)
        qre_kv_read(self.desc, layer, make_kv_rows(DTYPES[dtype], k, v), n, seqs, first, cu, total, k, v, stream)
        return k, v

    def common_len(self, seqs, cu_group, out=None, stream=None):
        """[groups] int32 on the device: how many leading positions each group's sequences have in common; group i is
        seqs[cu_group[i]:cu_group[i + 1]] (seqs None: sequences 0, 1, and so on, up to 4096)."""
        _check_ids(self.k.device, cu_group=cu_group)
        if seqs is not None:
            _check_ids(self.k.device, seqs=seqs)
        n = seqs.numel() if seqs is not None else min(self.page_table.shape[0], 4096)
        groups = cu_group.numel() - 1
        out = _empty((groups,), torch.int32, self.k.device, stream) if out is None else out
        _check_ids(self.k.device, groups, out=out)
        qre_kv_common_len(self.desc, n, seqs, groups, cu_group, out, stream)
        return out

    def fork(self, src, dst, stream=None):
        _check_ids(self.k.device, src.numel(), src=src, dst=dst)
        qre_kv_fork(self.desc, src.numel(), src, dst, self.workspace, stream=stream)

    def free(self, seqs, stream=None):
        _check_ids(self.k.device, seqs=seqs)
        qre_kv_free(self.desc, seqs.numel(), seqs, stream)

    def compact(self, stream=None):
        """Returns the device tensor that will hold the number of live pages."""
        qre_kv_compact(self.desc, self.page_table, self.ref_count, self.n_live, self.workspace, stream=stream)
        return self.n_live


class Rotary:
    """Norms (q_norm, k_norm: [head_dim] fp32 weights, None: none) and position rotation of heads, rot_dim elements of
    each (None: all), by the angles position * inv_freq ([rot_dim / 2] fp32; None: theta ** (-2 i / rot_dim)).
    interleaved: neighbours are the pairs, not the two halves."""

    def __init__(self, n_heads, n_kv_heads, head_dim, rot_dim=None, theta=10000.0, inv_freq=None, interleaved=False,
                 q_norm=None, k_norm=None, eps=1e-6, dtype=torch.bfloat16, device="cuda"):
        rot_dim = head_dim if rot_dim is None else rot_dim
        if rot_dim % 2:
            raise ValueError(f"rot_dim {rot_dim} is odd: elements turn in pairs")
        if inv_freq is None and rot_dim:
            i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
            inv_freq = (theta ** (-i / rot_dim)).float().to(device)
        self.n_heads, self.n_kv_heads, self.head_dim, self.dtype = n_heads, n_kv_heads, head_dim, dtype
        self.inv_freq, self.q_norm, self.k_norm = inv_freq, q_norm, k_norm
        self.interleaved, self.eps = interleaved, eps
        for name, t, n in (("inv_freq", inv_freq, rot_dim // 2), ("q_norm", q_norm, head_dim), ("k_norm", k_norm, head_dim)):
            if t is not None:
                _check_array(t, name, (n,), torch.float32, t.device, contiguous=True)

    def _outputs(self, device, tokens, q, k, q_out, k_out, keep, stream):
        if device.type != "cuda":
            raise ValueError(f"heads are normed and turned on a GPU, not on {device}")
        for name, t in (("inv_freq", self.inv_freq), ("q_norm", self.q_norm), ("k_norm", self.k_norm)):
            if t is not None and t.device != device:
                raise ValueError(f"{name} is on {t.device}, not on {device}")
        shapes = (tokens, self.n_heads, self.head_dim), (tokens, self.n_kv_heads, self.head_dim)
        _check_array(q, "q", shapes[0], self.dtype, device)
        _check_array(k, "k", shapes[1], self.dtype, device)
        q_out = _empty(shapes[0], self.dtype, device, stream) if q_out is None else q_out
        k_out = _empty(shapes[1], self.dtype, device, stream) if k_out is None and keep else k_out
        _check_array(q_out, "q_out", shapes[0], self.dtype, device)
        if k_out is not None:
            _check_array(k_out, "k_out", shapes[1], self.dtype, device)
        return q_out, k_out

    def _desc(self, q, k, v, q_out, k_out):
        return make_rope(self.n_heads, self.n_kv_heads, self.head_dim, DTYPES[self.dtype], self.inv_freq,
                         self.interleaved, self.q_norm, self.k_norm, self.eps, q, k, v, q_out, k_out)

    def apply(self, q, k, token_pos, q_out=None, k_out=None, stream=None):
        """q [tokens, n_heads, head_dim], k [tokens, n_kv_heads, head_dim] at positions token_pos; returns both, normed
        and turned.  q_out and k_out may be q and k.  Rows of tokens at a negative position are left as they are."""
        _check_ids(q.device, q.shape[0], token_pos=token_pos)
        q_out, k_out = self._outputs(q.device, q.shape[0], q, k, q_out, k_out, True, stream)
        qre_qk_norm_rope(self._desc(q, k, None, q_out, k_out), q.shape[0], token_pos, q, k, q_out, k_out, stream)
        return q_out, k_out


class Attention:
    """Layer ``layer``'s attention with ``n_heads`` query heads on ``cache``; up to ``max_batch`` sequences a decode, in up
    to ``max_groups`` groups if it is shared."""

    def __init__(self, cache, layer, n_heads, max_batch, dtype=torch.bfloat16, scale=None, window=0, max_groups=0):
        self.cache, self.layer, self.dtype, self.window = cache, layer, DTYPES[dtype], window
        self.torch_dtype = dtype
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, cache.n_kv_heads, cache.head_dim
        self.scale = self.head_dim ** -0.5 if scale is None else scale
        n = qre_attn_decode_workspace_size(self._desc(), cache.desc, max_batch)
        if max_groups:
            n = max(n, qre_attn_decode_shared_workspace_size(self._desc(), cache.desc, max_batch, max_groups))
        self.workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=cache.device)

    def _desc(self, q=None, k=None, v=None, o=None):
        return make_attn(self.n_heads, self.n_kv_heads, self.head_dim, self.dtype, self.scale, True, self.window,
                         q, k, v, o)

    def _check(self, q, o, lse):
        device = self.cache.k.device
        _check_array(q, "q", (q.shape[0], self.n_heads, self.head_dim), self.torch_dtype, device)
        if o is not None:
            _check_array(o, "o", q.shape, self.torch_dtype, device)
        if lse is not None:
            _check_array(lse, "lse", q.shape[:2], torch.float32, device, contiguous=True)
        return device

    def prefill(self, q, k, v, cu_q, cu_k, o=None, lse=None, stream=None):
        """q [tokens, n_heads, head_dim], k, v [keys, n_kv_heads, head_dim], cu_q, cu_k [sequences + 1]."""
        device = self._check(q, o, lse)
        for name, t in (("k", k), ("v", v)):
            _check_array(t, name, (k.shape[0], self.n_kv_heads, self.head_dim), self.torch_dtype, device)
        _check_ids(device, cu_q.numel(), cu_q=cu_q, cu_k=cu_k)
        o = _empty_like(q, stream) if o is None else o
        qre_attn_prefill(self._desc(q, k, v, o), cu_q.numel() - 1, q.shape[0], k.shape[0], cu_q, cu_k, q, k, v, o,
                         lse, stream)
        return o

    def decode(self, q, seqs, o=None, lse=None, max_len=0, stream=None):
        """q [sequences, n_heads, head_dim]: the newest token of each sequence, its row reserved and written before.
        seqs None: sequences 0, 1, and so on."""
        device = self._check(q, o, lse)
        if seqs is not None:
            _check_ids(device, q.shape[0], seqs=seqs)
        o = _empty_like(q, stream) if o is None else o
        qre_attn_decode(self._desc(q, o=o), self.cache.desc, self.layer, q.shape[0], seqs, max_len, q, o, lse,
                        self.workspace, stream=stream)
        return o

    def decode_shared(self, q, seqs, cu_group, common_len, o=None, lse=None, max_len=0, stream=None):
        """decode for groups of sequences with a common prefix (``KVCache.common_len``): it is read once for a group.
        max_len, an upper bound of the lengths, lets calls that are too short to gain by it go without (0: not known)."""
        device = self._check(q, o, lse)
        if seqs is not None:
            _check_ids(device, q.shape[0], seqs=seqs)
        _check_ids(device, cu_group=cu_group)
        _check_ids(device, cu_group.numel() - 1, common_len=common_len)
        o = _empty_like(q, stream) if o is None else o
        qre_attn_decode_shared(self._desc(q, o=o), self.cache.desc, self.layer, q.shape[0], seqs, cu_group.numel() - 1,
                               cu_group, common_len, max_len, q, o, lse, self.workspace, stream=stream)
        return o
