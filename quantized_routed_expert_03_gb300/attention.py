"""Device plumbing for attention: the paged key-value cache and the two attention calls over it.

Like ``layer``, PyTorch only allocates memory and supplies streams here; every
computation is a call into libqre.so through the binding in ``__init__``.

* :class:`KVCache` owns the pages of all layers and the device state (page table,
  lengths, reference counts): reserve, write, fork, free, compact.
* :class:`Attention` is one layer's attention on such a cache: ``prefill`` over
  packed prompts (keys and values as they come from the projections), ``decode``
  of one new token per sequence over the pages.

Both keep a workspace: calls on one object belong on one stream at a time.  A
result allocated here belongs to the stream that the call was given, like any
tensor made there: a program that uses it on another stream waits for the call
and, before it lets go of the tensor, tells the allocator (``record_stream``).
"""

from __future__ import annotations

import torch

from . import (QRE_BF16, QRE_E4M3, QRE_FP16, make_attn, make_kv_cache, make_kv_rows, qre_attn_decode,
               qre_attn_decode_workspace_size, qre_attn_prefill, qre_kv_compact, qre_kv_fork, qre_kv_free,
               qre_kv_reserve, qre_kv_workspace_size, qre_kv_write)

DTYPES = {torch.bfloat16: QRE_BF16, torch.float16: QRE_FP16, torch.float8_e4m3fn: QRE_E4M3}


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


def _empty_like(q, stream):
    """An output for a call on ``stream``: memory of that stream's pool, so that nothing that another stream still does
    with a block it was given before can meet the call."""
    if stream is None:
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if not isinstance(stream, torch.cuda.Stream):        # a raw handle, 0: the default stream
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        stream = torch.cuda.ExternalStream(handle, device=q.device) if handle else torch.cuda.default_stream(q.device)
    with torch.cuda.stream(stream):
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)


class KVCache:
    """``n_pages`` pages of ``page_size`` positions for all layers, and up to ``max_seqs`` sequences on them.

    k_scale, v_scale: [n_layers, n_kv_heads] fp32, for an E4M3 cache only (None: 1).
    Sequence ids, counts and positions are contiguous int32 tensors on the device that begin at a 16-byte boundary
    (clone a slice that does not); other arguments raise ValueError; nothing here synchronizes.
    """

    def __init__(self, n_layers, n_pages, n_kv_heads, page_size, head_dim, max_seqs, max_pages,
                 dtype=torch.bfloat16, k_scale=None, v_scale=None, device="cuda"):
        self.device = torch.device(device)
        i32 = dict(dtype=torch.int32, device=self.device)
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=self.device)
        self.v = torch.empty(shape, dtype=dtype, device=self.device)
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
        shape = (token_seq.numel(), self.k.shape[2], self.k.shape[4])
        _check_array(k, "k", shape, k.dtype, self.k.device)
        _check_array(v, "v", shape, k.dtype, self.k.device)
        qre_kv_write(self.desc, layer, make_kv_rows(DTYPES[k.dtype], k, v), token_seq.numel(), token_seq, token_pos,
                     k, v, stream)

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


class Attention:
    """Layer ``layer``'s attention with ``n_heads`` query heads on ``cache``; up to ``max_batch`` sequences a decode."""

    def __init__(self, cache, layer, n_heads, max_batch, dtype=torch.bfloat16, scale=None, window=0):
        self.cache, self.layer, self.dtype, self.window = cache, layer, DTYPES[dtype], window
        self.torch_dtype = dtype
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, cache.k.shape[2], cache.k.shape[4]
        self.scale = self.head_dim ** -0.5 if scale is None else scale
        n = qre_attn_decode_workspace_size(self._desc(), cache.desc, max_batch)
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
