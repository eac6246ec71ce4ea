"""ctypes binding of the score-modified attention + JVP: a tanh cap, a bias by
distance, an interval of visible keys per query row, and shared key heads
(``attn_jvp_fwd_scored``, ``attn_jvp_fwd_scored_stats``, ``attn_jvp_bwd_scored``),
and ``key_bounds``, which writes the usual masks as such intervals.
Argument marshalling only, as in ``_binding``."""
from __future__ import annotations

import contextlib
import functools

import torch

from ._binding import GRAD_NAMES, _check, _ptr, load_library

__all__ = ["attn_jvp_fwd_scored", "attn_jvp_fwd_scored_stats", "attn_jvp_bwd_scored", "bwd_scored_workspace_bytes",
           "key_bounds"]


_HERE = contextlib.nullcontext()
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object around it
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device  # (a tensor is on a GPU already)
try:  # an allocation without its argument parsing: 0.8 instead of 1.8 us, of which a call makes three or more
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None


def _empty(shape, dtype, device):
    """A contiguous tensor of one, three or four dimensions on ``device``, which is current."""
    if len(shape) == 1:
        strides = (1,)
    elif len(shape) == 4:
        B, H, L, d = shape
        strides = (H * L * d, L * d, d, 1)
    else:
        H, L, d = shape
        strides = (L * d, d, 1)
    if _empty_strided_cuda is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    return _empty_strided_cuda(shape, strides, dtype)


def _tensor(name, x, shape, dtype, device=None):
    """x is a contiguous CUDA tensor of this shape and type (on this device)."""
    if device is not None and type(x) is torch.Tensor and x.dtype is dtype and x.shape == shape \
            and x.get_device() == device.index and x.is_contiguous():
        return x
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != dtype or x.shape != shape \
            or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of shape {tuple(shape)}")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")
    return x


def _tensors(names, xs, shape, dtype, device):
    """Every x is such a tensor of one shape and type.  (The calls are short: what
    a check costs counts, so the common case is one pass.)"""
    if not _all_right(xs, (shape,) * len(xs), dtype, device.index):
        for name, y in zip(names, xs):
            _tensor(name, y, shape, dtype, device)


def _launch_scope(stream, device):
    """(context, handle) of a call: inside the context ``device`` is current and
    memory is allocated for the stream that the call launches on (torch's
    current stream of the device, or ``stream``), so that nothing allocated
    for the call is handed out again, or was last used, on another one."""
    if stream is None:
        here = _current_device() == device.index
        handle = _raw_stream(device.index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
        return _HERE if here else torch.cuda.device(device), handle
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _all_right(xs, shapes, dtype, index):
    for x, shape in zip(xs, shapes):
        if type(x) is not torch.Tensor or x.dtype is not dtype or x.shape != shape or x.get_device() != index \
                or not x.is_contiguous():
            return False
    return True


def _sizes(q, k, v, tq, tk, tv):
    if type(q) is torch.Tensor and type(k) is torch.Tensor:  # the common case in one pass
        qs, ks = q.shape, k.shape
        if len(qs) == len(ks) == 4 and ks[1] and not qs[1] % ks[1] and ks[0] == qs[0] and ks[3] == qs[3]:
            index = q.get_device()
            if index >= 0 and _all_right((q, tq, k, v, tk, tv), (qs, qs, ks, ks, ks, ks), _BF16, index):
                return qs[0], qs[1], ks[1], qs[2], ks[2], qs[3]
    for name, x in (("q", q), ("k", k)):
        if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 4:
            raise ValueError(f"{name} must be a CUDA [B, H, L, d] tensor")
    (B, H, Lq, d), (_, Hkv, Lk, _) = q.shape, k.shape
    if H and (Hkv < 1 or H % Hkv):
        raise ValueError(f"query heads ({H}) must be a multiple of the key heads ({Hkv})")
    _tensors(("q", "tq"), (q, tq), q.shape, _BF16, q.device)
    _tensors(("k", "v", "tk", "tv"), (k, v, tk, tv), (B, Hkv, Lk, d), _BF16, q.device)
    return B, H, Hkv, Lq, Lk, d


def _score_args(slopes, key_begin, key_end, softcap, scale, sizes, device):
    B, H, _, Lq, _, d = sizes
    if slopes is not None:
        _tensor("slopes", slopes, (H,), _F32, device)
    for name, x in (("key_begin", key_begin), ("key_end", key_end)):
        if x is not None:  # (one dimension: the same for every sequence of the batch)
            _tensor(name, x, (Lq,) if isinstance(x, torch.Tensor) and x.dim() == 1 else (B, Lq), _I32, device)
    return float(softcap or 0.0), float(d ** -0.5 if scale is None else scale)


def _per_sequence(x, B):
    return x.expand(B, x.shape[0]).contiguous() if x.dim() == 1 else x


def _fwd(entry, q, k, v, tq, tk, tv, scale, softcap, slopes, key_begin, key_end, o, to, lse, mu, stream, want_lse,
         want_mu):
    sizes = _sizes(q, k, v, tq, tk, tv)
    B, H, _, Lq, _, _ = sizes
    dev = q.device
    softcap, scale = _score_args(slopes, key_begin, key_end, softcap, scale, sizes, dev)
    if not (o is to is lse is mu is None):
        for name, x in (("o", o), ("to", to)):
            if x is not None:
                _tensor(name, x, q.shape, _BF16, dev)
        for name, x in (("lse", lse), ("mu", mu)):
            if x is not None:
                _tensor(name, x, (B, H, Lq), _F32, dev)
    scope, handle = _launch_scope(stream, dev)
    with scope:
        shape = (B, H, Lq, sizes[5])
        o = _empty(shape, _BF16, dev) if o is None else o
        to = _empty(shape, _BF16, dev) if to is None else to
        lse = _empty(shape[:3], _F32, dev) if lse is None and want_lse else lse
        mu = _empty(shape[:3], _F32, dev) if mu is None and want_mu else mu
        if key_begin is not None:
            key_begin = _per_sequence(key_begin, B)
        if key_end is not None:
            key_end = _per_sequence(key_end, B)
        rows = (o.data_ptr(), to.data_ptr(), _ptr(lse)) + ((mu.data_ptr(),) if want_mu else ())
        rc = getattr(load_library(), entry)(q.data_ptr(), k.data_ptr(), v.data_ptr(), tq.data_ptr(), tk.data_ptr(),
                                            tv.data_ptr(), *rows, _ptr(slopes), _ptr(key_begin), _ptr(key_end), *sizes,
                                            scale, softcap, handle)
    if rc:
        _check(rc, entry)
    return o, to, lse, mu


def attn_jvp_fwd_scored(q, k, v, tq, tk, tv, scale=None, softcap=0.0, slopes=None, key_begin=None, key_end=None,
                        o=None, to=None, lse=None, stream=None, want_lse=True):
    """O, tO, lse of attention whose scores are capped (``softcap`` c > 0:
    c tanh(z / c)), biased by distance (``slopes``, fp32 [H]:
    -slope |i + Lk - Lq - j|) and limited to the keys ``key_begin[b, i]`` <= j <
    ``key_end[b, i]`` of query row i (int32 [B, Lq], or [Lq] for every sequence;
    ``key_bounds`` makes them).  q, tq bf16 [B, H, Lq, 128]; k, v, tk, tv
    [B, Hkv, Lk, 128] with H a multiple of Hkv.  Rows that see nothing give
    zeros and lse = -inf, whatever their q and tq hold; k, v, tk and tv must be
    finite also where they are hidden.  Asynchronous on ``stream`` (default: the current
    stream of the tensors' device)."""
    return _fwd("attn_jvp_fwd_scored", q, k, v, tq, tk, tv, scale, softcap, slopes, key_begin, key_end, o, to, lse,
                None, stream, want_lse, False)[:3]


def attn_jvp_fwd_scored_stats(q, k, v, tq, tk, tv, scale=None, softcap=0.0, slopes=None, key_begin=None, key_end=None,
                              o=None, to=None, lse=None, mu=None, stream=None):
    """``attn_jvp_fwd_scored`` that also returns mu, for ``attn_jvp_bwd_scored``.
    Returns (o, to, lse, mu)."""
    return _fwd("attn_jvp_fwd_scored_stats", q, k, v, tq, tk, tv, scale, softcap, slopes, key_begin, key_end, o, to,
                lse, mu, stream, True, True)


def bwd_scored_workspace_bytes(B: int, H: int, Hkv: int, Lq: int, Lk: int) -> int:
    """Device workspace with which ``attn_jvp_bwd_scored`` may split its key
    side on the current device."""
    return int(load_library().attn_jvp_bwd_scored_workspace_bytes(int(B), int(H), int(Hkv), int(Lq), int(Lk)))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(B, H, Hkv, Lq, Lk, device):
    """The same (at least 1), with ``device`` current (part of the key: the size depends on it)."""
    return max(1, bwd_scored_workspace_bytes(B, H, Hkv, Lq, Lk))


def attn_jvp_bwd_scored(q, k, v, tq, tk, tv, o, to, lse, mu, dout, dtout, scale=None, softcap=0.0, slopes=None,
                        key_begin=None, key_end=None, grads=None, workspace=None, stream=None):
    """Gradients of <dout, O> + <dtout, tO> of ``attn_jvp_fwd_scored`` with
    respect to q, k, v, tq, tk, tv (slopes and cap are constants); o, to, lse,
    mu from ``attn_jvp_fwd_scored_stats`` with the same options.  All inputs must be
    finite, those of rows that see nothing too.  ``grads``: an
    optional dict of preallocated outputs; ``workspace``: a CUDA uint8 tensor
    of ``bwd_scored_workspace_bytes`` bytes (allocated per call when omitted).
    Returns a dict dq, dk, dv, dtq, dtk, dtv shaped like the inputs."""
    sizes = _sizes(q, k, v, tq, tk, tv)
    B, H, Hkv, Lq, Lk, d = sizes
    dev = q.device
    softcap, scale = _score_args(slopes, key_begin, key_end, softcap, scale, sizes, dev)
    _tensors(("o", "to", "dout", "dtout"), (o, to, dout, dtout), q.shape, _BF16, dev)
    _tensors(("lse", "mu"), (lse, mu), (B, H, Lq), _F32, dev)
    shapes = dict.fromkeys(GRAD_NAMES, (B, Hkv, Lk, d)) | {"dq": (B, H, Lq, d), "dtq": (B, H, Lq, d)}
    grads = dict(grads or {})
    for n, x in grads.items():
        if n in shapes and x is not None:
            _tensor(n, x, shapes[n], _BF16, dev)
    if workspace is not None:
        _tensor("workspace", workspace, (workspace.numel(),), torch.uint8, dev)
    scope, handle = _launch_scope(stream, dev)
    with scope:
        for n in GRAD_NAMES:
            if grads.get(n) is None:
                grads[n] = _empty(shapes[n], _BF16, dev)
        if workspace is None:
            workspace = _empty((_workspace_bytes(*sizes[:5], dev.index),), torch.uint8, dev)
        if key_begin is not None:
            key_begin = _per_sequence(key_begin, B)
        if key_end is not None:
            key_end = _per_sequence(key_end, B)
        rc = load_library().attn_jvp_bwd_scored(
            _ptr(q), _ptr(k), _ptr(v), _ptr(tq), _ptr(tk), _ptr(tv), _ptr(o), _ptr(to), _ptr(lse), _ptr(mu),
            _ptr(dout), _ptr(dtout), *(_ptr(grads[n]) for n in GRAD_NAMES), _ptr(slopes), _ptr(key_begin),
            _ptr(key_end), *sizes, scale, softcap, _ptr(workspace), workspace.numel(), handle)
    _check(rc, "attn_jvp_bwd_scored")
    return grads


def key_bounds(Lq: int, Lk: int | None = None, *, causal: bool = False, prefix: int = 0, frame: int = 0,
               window: int = 0, documents=None, device="cuda"):
    """(key_begin, key_end), int32 [Lq], of the usual masks.  Query row i stands
    at key position p = i + Lk - Lq.

    ``documents``: offsets of documents along the keys (a list or tensor,
    ascending): a row sees its own document only, and nothing before the first
    or behind the last offset.  Inside its document (else the whole sequence),
    ``causal`` hides the keys behind p except the document's first ``prefix``
    ones, ``frame`` (> 0) those behind the end of p's frame of that many keys,
    and ``window`` (> 0) all but the last ``window`` keys up to p (with ``frame``,
    the keys behind p that its frame shows stay; not with ``prefix``).
    """
    Lk = Lq if Lk is None else Lk
    if Lq < 0 or Lk < 1 or prefix < 0 or frame < 0 or window < 0 or (causal and frame):
        raise ValueError("sizes must not be negative, and a mask is causal by keys or by frames")
    if prefix and not causal:
        raise ValueError("prefix belongs to the causal mask")
    if prefix and window:
        raise ValueError("a prefix and a window are no single interval of keys")
    p = torch.arange(Lq, device=device, dtype=torch.int64) + (Lk - Lq)
    begin, end = torch.zeros_like(p), torch.full_like(p, Lk)
    inside = p >= 0 if causal or frame else torch.ones_like(p, dtype=torch.bool)  # (nothing is copied from the host)
    if documents is not None:
        cu = torch.as_tensor(documents, device=device, dtype=torch.int64)
        if cu.dim() != 1 or cu.numel() < 2:
            raise ValueError("documents are at least two offsets")
        at = torch.searchsorted(cu, p, right=True) - 1  # the last offset that is not behind p
        inside = (at >= 0) & (at < cu.numel() - 1)
        at = at.clamp(0, cu.numel() - 2)
        begin, end = cu[at], cu[at + 1].clamp(max=Lk)
    first = begin
    if causal or (window and not frame):
        end = torch.minimum(end, torch.maximum(p + 1, first + prefix) if prefix else p + 1)
    if frame:
        end = torch.minimum(end, first + (torch.div(p - first, frame, rounding_mode="floor") + 1) * frame)
    if window:
        begin = torch.maximum(first, p - window + 1)
    if causal and documents is None and prefix:
        inside = torch.ones_like(inside)
    zero = torch.zeros_like(p)
    begin, end = torch.where(inside, begin, zero), torch.where(inside, end, zero)
    return begin.to(torch.int32), end.to(torch.int32)
