"""ctypes binding of the paged 8-bit key/value cache: ``attn_jvp_cache_append``
(rotated keys and values into e4m3 pages) and ``attn_jvp_fwd_cache`` (O, tO and
lse of a few query tokens per sequence over them).  Argument marshalling only,
as in ``_binding``.

The cache is four tensors that the caller owns: codes ``k_cache``, ``v_cache``
(torch.float8_e4m3fn [pages, Hkv, page, 128], page a multiple of 16) and scales
``k_scale``, ``v_scale`` (float32 [pages, Hkv], powers of two); a value is its
code times its page's scale.  ``block_table`` (int32 [n_seq, width]) names the
page of each run of ``page`` tokens of a sequence; nothing needs to be
initialised before a page's first token is appended."""
from __future__ import annotations

import functools

import torch

from ._binding import _check, _ptr, load_library
from ._scored import _BF16, _F32, _I32, _all_right, _empty, _launch_scope, _tensor, _tensors

__all__ = ["attn_jvp_cache_append", "attn_jvp_fwd_cache", "fwd_cache_workspace_bytes"]


def _cache_sizes(k_cache, v_cache, k_scale, v_scale, block_table, cache_lens):
    if type(k_cache) is torch.Tensor and type(block_table) is torch.Tensor:  # the common case in one pass
        shape, table, index = k_cache.shape, block_table.shape, k_cache.get_device()
        if len(shape) == 4 and len(table) == 2 and index >= 0:
            pages, Hkv, page, d = shape
            of_scale = (pages, Hkv)
            if _all_right((k_cache, v_cache), (shape, shape), torch.float8_e4m3fn, index) \
                    and _all_right((k_scale, v_scale), (of_scale, of_scale), _F32, index) \
                    and _all_right((block_table, cache_lens), (table, table[:1]), _I32, index):
                return table[0], Hkv, pages, page, table[1], d, k_cache.device
    if not isinstance(k_cache, torch.Tensor) or not k_cache.is_cuda or k_cache.dim() != 4:
        raise ValueError("k_cache must be a CUDA [pages, Hkv, page, d] tensor")
    shape, dev = k_cache.shape, k_cache.device
    pages, Hkv, page, d = shape
    _tensors(("k_cache", "v_cache"), (k_cache, v_cache), shape, torch.float8_e4m3fn, dev)
    _tensors(("k_scale", "v_scale"), (k_scale, v_scale), (pages, Hkv), _F32, dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be an int32 [n_seq, width] tensor")
    n_seq, width = block_table.shape
    _tensor("block_table", block_table, (n_seq, width), _I32, dev)
    _tensor("cache_lens", cache_lens, (n_seq,), _I32, dev)
    return n_seq, Hkv, pages, page, width, d, dev


def attn_jvp_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cache_lens, cu_seqlens, q=None,
                          tq=None, cos=None, sin=None, interleaved=False, q_out=None, tq_out=None, stream=None):
    """Append new tokens to the cache, in place.

    k, v: bf16 [Hkv, total, 128], packed: sequence b's new tokens are rows
    ``cu_seqlens[b]`` .. ``cu_seqlens[b + 1] - 1`` and stand at positions
    ``cache_lens[b]``, ``cache_lens[b] + 1``, ...; ``cache_lens`` counts the tokens
    cached before and is left as it is.  With ``cos``, ``sin`` (float32
    [n_pos, 64], a row per position) the keys are rotated on the way: channels
    (i, i + 64) by angle i, or (2i, 2i + 1) with ``interleaved``; and ``q``, ``tq``
    (bf16 [H, total, 128], the same rows) are rotated into ``q_out``, ``tq_out``
    (allocated when omitted; they may be ``q``, ``tq`` themselves).  A page's
    scale is the smallest power of two that holds its largest value, over the
    tokens appended to it so far; a page whose first token is among the new
    ones starts afresh.  Pages that take new tokens must belong to one
    sequence.  Returns (q_out, tq_out)."""
    n_seq, Hkv, pages, page, width, d, dev = _cache_sizes(k_cache, v_cache, k_scale, v_scale, block_table, cache_lens)
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a [Hkv, total, d] tensor")
    total = k.shape[1]
    _tensors(("k", "v"), (k, v), (Hkv, total, d), _BF16, dev)
    _tensor("cu_seqlens", cu_seqlens, (n_seq + 1,), _I32, dev)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    n_pos = 0
    if cos is not None:
        n_pos = cos.shape[0] if isinstance(cos, torch.Tensor) and cos.dim() == 2 else 0
        _tensors(("cos", "sin"), (cos, sin), (n_pos, d // 2), _F32, dev)
        if n_pos < 1:
            raise ValueError("cos and sin need a row per position")
    H = Hkv
    if q is not None:
        if cos is None:
            raise ValueError("q takes part only to be rotated: cos and sin are needed")
        H = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        if H < 1 or H % Hkv:
            raise ValueError(f"q must be [H, total, d] with H a multiple of the key heads ({Hkv})")
        _tensors(("q", "tq"), (q,) if tq is None else (q, tq), (H, total, d), _BF16, dev)
        if q_out is not None or tq_out is not None:
            for name, x in (("q_out", q_out), ("tq_out", tq_out)):
                if x is not None:
                    _tensor(name, x, q.shape, _BF16, dev)
    if (q is None and (tq is not None or q_out is not None)) or (tq is None and tq_out is not None):
        raise ValueError("tq goes with q, and an output with its input")
    scope, handle = _launch_scope(stream, dev)
    with scope:
        q_out = _empty((H, total, d), _BF16, dev) if q is not None and q_out is None else q_out
        tq_out = _empty((H, total, d), _BF16, dev) if tq is not None and tq_out is None else tq_out
        rc = load_library().attn_jvp_cache_append(
            k.data_ptr(), v.data_ptr(), _ptr(q), _ptr(tq), _ptr(q_out), _ptr(tq_out), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), cache_lens.data_ptr(),
            cu_seqlens.data_ptr(), _ptr(cos), _ptr(sin),
            n_seq, H, Hkv, total, pages, page, width, n_pos, d, int(bool(interleaved)), handle)
    if rc:
        _check(rc, "attn_jvp_cache_append")
    return q_out, tq_out


def fwd_cache_workspace_bytes(n_seq: int, H: int, Hkv: int, n: int, page: int, table_width: int,
                              tangent: bool = True) -> int:
    """Device workspace with which ``attn_jvp_fwd_cache`` may spread a sequence over
    more of the current device than a cluster of CTAs (0: it would not)."""
    return int(load_library().attn_jvp_fwd_cache_workspace_bytes(int(n_seq), int(H), int(Hkv), int(n), int(page),
                                                                 int(table_width), int(bool(tangent))))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(n_seq, H, Hkv, n, page, width, tangent, device):
    """The same, with ``device`` current (part of the key: the size depends on it)."""
    return fwd_cache_workspace_bytes(n_seq, H, Hkv, n, page, width, tangent)


def attn_jvp_fwd_cache(q, tq, k_cache, v_cache, k_scale, v_scale, block_table, cache_lens, cu_seqlens=None,
                       max_seqlen=None, scale=None, softcap=0.0, slopes=None, causal=True, o=None, to=None, lse=None,
                       stream=None, want_lse=True, workspace=None):
    """O, tO, lse of the last query tokens of each sequence over its cached
    keys and values, which carry no tangent: tO is the derivative of O along
    ``tq`` (None: plain attention, and ``to`` is None).

    q, tq: bf16 [n_seq, H, n, 128], any strides that are multiples of 8 with
    the channels together; or packed [H, total, 128] with ``cu_seqlens`` (int32
    [n_seq + 1]) and ``max_seqlen`` (at least the most tokens of one sequence: a
    sequence's tokens from there on are neither computed nor written; ``total`` when
    omitted, for which the launch is then planned, so give it where it is
    known), the layout of ``attn_jvp_cache_append``.
    ``cache_lens`` (int32 [n_seq]) counts the cached tokens, the query tokens' own
    included: token t of a sequence's m stands at position cache_lens - m + t and sees the
    keys up to its own (``causal``; rows at negative positions see nothing), or
    every cached key.  ``softcap`` and ``slopes`` modify the scores as in
    ``attn_jvp_fwd_scored``.  ``workspace``: a CUDA uint8 tensor of
    ``fwd_cache_workspace_bytes`` bytes, through which few long contexts are spread
    over the whole GPU (allocated per call when omitted; an empty one: do without).
    Returns (o, to, lse), contiguous, shaped like q."""
    n_seq, Hkv, pages, page, width, d, dev = _cache_sizes(k_cache, v_cache, k_scale, v_scale, block_table, cache_lens)
    if not isinstance(q, torch.Tensor) or q.dtype is not _BF16 or q.get_device() != dev.index \
            or q.dim() != (4 if cu_seqlens is None else 3) or q.shape[-1] != d or q.stride(-1) != 1:
        raise ValueError("q must be a bf16 [n_seq, H, n, d] tensor (packed: [H, total, d]) on the cache's device with "
                         "its channels together")
    if cu_seqlens is None:
        if max_seqlen is not None:
            raise ValueError("max_seqlen belongs to cu_seqlens")
        H, n, total, strides = q.shape[1], q.shape[2], 0, q.stride()[:3]
        if q.shape[0] != n_seq:
            raise ValueError(f"q is of {q.shape[0]} sequences, the cache of {n_seq}")
    else:
        H, total = q.shape[0], q.shape[1]
        n, strides = total if max_seqlen is None else min(int(max_seqlen), total), (0, *q.stride()[:2])
        _tensor("cu_seqlens", cu_seqlens, (n_seq + 1,), _I32, dev)
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"query heads ({H}) must be a multiple of the key heads ({Hkv})")
    if tq is not None and (not isinstance(tq, torch.Tensor) or tq.shape != q.shape or tq.dtype is not _BF16
                           or tq.get_device() != dev.index or tq.stride() != q.stride()
                           and any(m > 1 and s != t for m, s, t in zip(q.shape, q.stride(), tq.stride()))):
        raise ValueError("tq must have q's shape, strides, type and device")
    if slopes is not None:
        _tensor("slopes", slopes, (H,), _F32, dev)
    shape = q.shape
    if tq is None and to is not None:
        raise ValueError("to goes with tq")
    if o is not None or to is not None:
        for name, x in (("o", o), ("to", to)):
            if x is not None:
                _tensor(name, x, shape, _BF16, dev)
    if lse is not None:
        _tensor("lse", lse, shape[:-1], _F32, dev)
    if workspace is not None:
        _tensor("workspace", workspace, (workspace.numel(),), torch.uint8, dev)
    scope, handle = _launch_scope(stream, dev)
    with scope:
        if workspace is None:
            size = _workspace_bytes(n_seq, H, Hkv, n, page, width, tq is not None, dev.index)
            workspace = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        shape = tuple(shape)
        o = _empty(shape, _BF16, dev) if o is None else o
        to = _empty(shape, _BF16, dev) if to is None and tq is not None else to
        if lse is None and want_lse:  # (packed: [H, total])
            lse = _empty(shape[:3], _F32, dev) if len(shape) == 4 else torch.empty(shape[:2], dtype=_F32, device=dev)
        rc = load_library().attn_jvp_fwd_cache(
            q.data_ptr(), _ptr(tq), o.data_ptr(), _ptr(to), _ptr(lse), k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), cache_lens.data_ptr(), _ptr(cu_seqlens),
            _ptr(slopes), n_seq, H, Hkv, n,
            total, *strides, pages, page, width, d, float(d ** -0.5 if scale is None else scale),
            float(softcap or 0.0), int(bool(causal)), _ptr(workspace), 0 if workspace is None else workspace.numel(),
            handle)
    if rc:
        _check(rc, "attn_jvp_fwd_cache")
    return o, to, lse
