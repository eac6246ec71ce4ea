"""The paged 8-bit cache in 64 bits, from its definition: appending token by
token on the host, and attention + JVP over the stored codes with elementwise
bounds on what the kernel's f16 operands and bf16 outputs may add."""
from __future__ import annotations

import numpy as np
import torch

U16 = torch.finfo(torch.float16).eps / 2  # one rounding to f16 (P and P dS)
UB = torch.finfo(torch.bfloat16).eps / 2  # one rounding to bf16 (outputs)
SLACK, FLOOR = 1.05, 2.0 ** -16


def e4m3(x):
    """The nearest e4m3 values (ties to even, saturating), as float64."""
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def exponent(amax):
    m, e = np.frexp(np.asarray(amax, dtype=np.float64))
    e = e - 9 + (m > 0.875)
    return np.clip(np.where(amax > 0, e, -100), -100, 100)


def turn(x, cos, sin, interleaved):
    """Rotation in fp32 steps, [..., 128] with cos, sin [rows, 64]."""
    x, cos, sin = (np.asarray(t, dtype=np.float32) for t in (x, cos, sin))
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return np.stack((a * cos - b * sin, b * cos + a * sin), -1).reshape(x.shape)
    a, b = x[..., :64], x[..., 64:]
    return np.concatenate((a * cos - b * sin, b * cos + a * sin), -1)


def append(x, codes, scale, table, lens, cu):
    """x [Hkv, total, 128] joins (codes [pages, Hkv, page, 128], scale [pages, Hkv]), float64 arrays, in place."""
    n_pages, _, page, _ = codes.shape
    for b, start in enumerate(lens):
        n = cu[b + 1] - cu[b]
        at = 0
        while at < n:
            p = (start + at) // page
            if p >= table.shape[1]:
                break
            kept = (start + at) % page
            take = min(n - at, page - kept)
            part = x[:, cu[b] + at: cu[b] + at + take].astype(np.float64)
            page_id = table[b, p]
            if 0 <= page_id < n_pages:
                e = exponent(np.abs(part).max((1, 2)))
                if kept:
                    e = np.maximum(e, np.log2(scale[page_id]).astype(np.int64))
                s = np.exp2(e.astype(np.float64))
                if kept:
                    codes[page_id, :, :kept] = e4m3(codes[page_id, :, :kept] * (scale[page_id] / s)[:, None, None])
                codes[page_id, :, kept: kept + take] = e4m3(part / s[:, None, None])
                scale[page_id] = s
            at += take


def attention(q, tq, k8, v8, ks, vs, table, lens, scale, softcap=0.0, slopes=None, causal=True):
    """Lists of (o, to or None, lse, bound of o, bound of to) per sequence; q, tq lists of [H, n, 128]."""
    out = []
    n_pages, Hkv, page, _ = k8.shape
    for b, length in enumerate(lens):
        qb = q[b].double()
        H, n, _ = qb.shape
        ids = table[b, : -(-length // page)].long()
        good = ((ids >= 0) & (ids < n_pages)).repeat_interleave(page)[:length]
        at = ids.clamp(0, n_pages - 1)
        k, v = (c[at].double().mul(f[at].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :length]
                .repeat_interleave(H // Hkv, 0) for c, f in ((k8, ks), (v8, vs)))
        k, v = k * good[:, None], v * good[:, None]
        k, v = torch.nan_to_num(k), torch.nan_to_num(v)
        z = scale * (qb @ k.mT)
        df = torch.ones_like(z)
        if softcap:
            t = torch.tanh(z / softcap)
            z, df = softcap * t, 1 - t * t
        i = torch.arange(length - n, length, device=z.device)[:, None]
        j = torch.arange(length, device=z.device)
        if slopes is not None:
            z = z - slopes.double()[:, None, None] * (i - j).abs()
        seen = good[None] & ((j <= i) if causal else torch.ones_like(j <= i))
        z = z.masked_fill(~seen, -float("inf"))
        if length == 0:
            zero = torch.zeros_like(qb)
            out.append((zero, None if tq is None else zero, torch.full((H, n), -float("inf")), zero, zero))
            continue
        m = z.amax(-1, keepdim=True)
        P = torch.exp(z - m.masked_fill(torch.isinf(m), 0.0))
        l = P.sum(-1, keepdim=True)
        lse = (m + torch.log(l))[..., 0]
        P = P / l.masked_fill(l == 0, 1.0)
        o = P @ v
        # f16 weights: half a step relative, and 2^-25 absolute for weights below 2^-14 of the
        # row's largest |p| x value scale; values are at most 448 scales
        eo = U16 * (P @ v.abs()) + 2.0 ** -25 * length * (P.amax(-1, keepdim=True) * v.abs().amax())
        bo = SLACK * (eo + UB * o.abs()) + FLOOR * o.abs().amax()
        if tq is None:
            out.append((o, None, lse, bo, None))
            continue
        u = df * scale * (tq[b].double() @ k.mT)
        W = P * u
        mu = W.sum(-1, keepdim=True)
        to = W @ v - mu * o
        # P dS takes two roundings' worth (P dS itself and the product before it are fp32)
        top = (P.amax(-1, keepdim=True) * u.abs().amax(-1, keepdim=True) * v.abs().amax())
        eto = U16 * (W.abs() @ v.abs()) + 2.0 ** -20 * top * length ** 0.5 + mu.abs() * eo
        out.append((o, to, lse, bo, SLACK * (eto + UB * to.abs()) + FLOOR * (W.abs() @ v.abs()).amax()))
    return out
