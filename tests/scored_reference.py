"""Attention + JVP with modified scores and its gradients in 64 bits, from the
definition, and elementwise bounds on what bf16 operands may add.

``u`` is half a bf16 step (torch.finfo(bf16).eps / 2): the most one rounding to
bf16 is off, relative to the value.  The kernels round the weights p and
p dS (forward) and the score gradients (backward) once each before their
products, and every output once; sums, statistics and exponentials are fp32.
A bound adds those roundings up in absolute value, so it holds whatever their
signs; ``SLACK`` and ``FLOOR`` leave room for the fp32 arithmetic (relative
errors of some 2^-18: exponentials of scores that are themselves sums of 128
products)."""
from __future__ import annotations

import torch

U = torch.finfo(torch.bfloat16).eps / 2
SLACK, FLOOR = 1.05, 2.0 ** -16


def scores(q, k, tq, tk, scale, softcap=0.0, slopes=None, begin=None, end=None):
    """z, dz, S (hidden keys -inf), f', f'' dz and the visible pairs; inputs [B, H, L, d] in 64 bits with the key
    heads already repeated."""
    Lq, Lk = q.shape[2], k.shape[2]
    z = scale * (q @ k.mT)
    dz = scale * (tq @ k.mT + q @ tk.mT)
    df, ddf = torch.ones_like(z), torch.zeros_like(z)
    S = z
    if softcap:
        t = torch.tanh(z / softcap)
        S, df = softcap * t, 1 - t * t
        ddf = -2.0 / softcap * t * df
    i = torch.arange(Lq, device=q.device)[:, None] + (Lk - Lq)
    j = torch.arange(Lk, device=q.device)
    if slopes is not None:
        S = S - slopes.double()[:, None, None] * (i - j).abs()
    seen = torch.ones((q.shape[0], 1, Lq, Lk), dtype=torch.bool, device=q.device)
    if begin is not None:
        seen &= (j >= begin.view(-1, Lq)[:, None, :, None])
    if end is not None:
        seen &= (j < end.view(-1, Lq)[:, None, :, None])
    return z, dz, S.masked_fill(~seen, -float("inf")), df, ddf * dz, seen


def softmax(S):
    m = S.amax(-1, keepdim=True)
    p = torch.exp(S - m.masked_fill(torch.isinf(m), 0.0))
    l = p.sum(-1, keepdim=True)
    return p / l.masked_fill(l == 0, 1.0), (m + torch.log(l))[..., 0]


def repeat(x, H):
    return x.double().repeat_interleave(H // x.shape[1], 1)


def forward(q, k, v, tq, tk, tv, scale, bounds=False, **opt):
    """o, to, lse, mu in 64 bits; with ``bounds`` also the elementwise bounds of o and to."""
    H = q.shape[1]
    q, tq = q.double(), tq.double()
    k, v, tk, tv = (repeat(x, H) for x in (k, v, tk, tv))
    _, dz, S, df, _, _ = scores(q, k, tq, tk, scale, **opt)
    P, lse = softmax(S)
    W = P * df * dz
    mu = W.sum(-1, keepdim=True)
    o = P @ v
    to = W @ v - mu * o + P @ tv
    if not bounds:
        return o, to, lse, mu[..., 0]
    eo = U * (P @ v.abs())
    eto = U * (W.abs() @ v.abs() + P @ tv.abs()) + mu.abs() * eo
    floor = lambda x: FLOOR * x.abs().amax()  # noqa: E731
    return (o, to, lse, mu[..., 0]), (SLACK * (eo + U * o.abs()) + floor(o), SLACK * (eto + U * to.abs()) + floor(to))


def backward(q, k, v, tq, tk, tv, dout, dtout, scale, bounds=False, **opt):
    """The six gradients in 64 bits (shared key heads summed over their groups); with ``bounds`` their bounds too."""
    H, Hkv = q.shape[1], k.shape[1]
    shared = lambda x: x.unflatten(1, (Hkv, H // Hkv)).sum(2)  # noqa: E731
    q, tq, do, dto = (x.double() for x in (q, tq, dout, dtout))
    k, v, tk, tv = (repeat(x, H) for x in (k, v, tk, tv))
    _, dz, S, df, ddf, _ = scores(q, k, tq, tk, scale, **opt)
    P, _ = softmax(S)
    u = df * dz
    mu = (P * u).sum(-1, keepdim=True)
    o = P @ v
    to = (P * u) @ v - mu * o + P @ tv
    A, Bc = dto @ v.mT, do @ v.mT + dto @ tv.mT
    a = (dto * o).sum(-1, keepdim=True)
    D = (do * o).sum(-1, keepdim=True) + (dto * to).sum(-1, keepdim=True) - a * mu
    dsb = P * (A - a)
    sb = P * (Bc + A * (u - mu) - a * u - D)
    zb, dzb = df * sb + ddf * dsb, df * dsb
    g = dict(dq=scale * (zb @ k + dzb @ tk), dtq=scale * (dzb @ k), dk=shared(scale * (zb.mT @ q + dzb.mT @ tq)),
             dtk=shared(scale * (dzb.mT @ q)), dv=shared(P.mT @ do + (P * (u - mu)).mT @ dto),
             dtv=shared(P.mT @ dto))
    if not bounds:
        return g
    # a and D come from outputs rounded to bf16
    eo = U * (P @ v.abs() + o.abs())
    eto = U * ((P * u).abs() @ v.abs() + P @ tv.abs() + to.abs()) + mu.abs() * U * (P @ v.abs())
    ea = (dto.abs() * eo).sum(-1, keepdim=True)
    eD = (do.abs() * eo).sum(-1, keepdim=True) + (dto.abs() * eto).sum(-1, keepdim=True) + mu.abs() * ea
    edsb, esb = P * ea, P * (eD + u.abs() * ea)
    ezb, edzb = U * zb.abs() + df * esb + ddf.abs() * edsb, U * dzb.abs() + df * edsb
    ka, tka, qa, tqa = k.abs(), tk.abs(), q.abs(), tq.abs()
    e = dict(dq=abs(scale) * (ezb @ ka + edzb @ tka), dtq=abs(scale) * (edzb @ ka),
             dk=shared(abs(scale) * (ezb.mT @ qa + edzb.mT @ tqa)), dtk=shared(abs(scale) * (edzb.mT @ qa)),
             dv=shared(U * (P.mT @ do.abs() + (P * (u - mu)).abs().mT @ dto.abs())), dtv=shared(U * (P.mT @ dto.abs())))
    return g, {n: SLACK * (e[n] + U * g[n].abs()) + FLOOR * g[n].abs().amax() for n in g}


def check(name, got, ref, bound):
    """got within the elementwise bound of ref (and finite)."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = (got.double() - ref).abs()
    worst = (err / bound.clamp_min(1e-300)).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 1.0, f"{name}: error {worst:.3f} times its bound"
    return worst
