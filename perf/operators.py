"""What the score-modified attention + JVP operators and the 8-bit paged cache
are measured on: the cases, their inputs, the operators in plain torch
operations, and the calls a user makes of them.

    fwd     O, tO and the log-sum-exp of attention whose scores may be capped
            by a tanh, get a bias by distance, and be limited to an interval of
            keys per query row (prefix, document and frame-causal masks)
    bwd     the six gradients of <dO, O> + <dtO, tO> of that forward
    append  new keys and values rotated by their positions, rounded to e4m3
            with one power-of-two scale per page and head, and written to a
            paged cache; the queries and their tangents rotated alongside
    cache   O, tO and the log-sum-exp of a few query tokens per sequence over
            such a cache, whose keys and values carry no tangent

With z = s Q K^T, dz = s (tQ K^T + Q tK^T) and cap c:
    S = c tanh(z / c) - slope |i + Lk - Lq - j|   (S = z - ... without a cap)
    dS = (1 - tanh^2(z / c)) dz,  P = softmax of S over the row's keys
    O = P V,  tO = (P .* (dS - rowsum(P .* dS))) V + P tV
"""
from __future__ import annotations

import math

import torch

own = False

D = 128  # head dimension of every case: the tensor-core kernels' only one
INF = float("inf")


# ------------------------------------------------------------------ the cases
def listed():
    """Shapes of the framework's own workloads (64x64 image tokens, a video
    latent grid of 21 frames of 30x52 tokens, 512 text tokens, 12 or 40 heads)
    and their ragged relatives."""
    return [
        # a call as small as the framework's smallest workload: launch latency decides
        dict(name="fwd_small", op="fwd", B=1, H=2, Hkv=2, Lq=128, Lk=128, cap=30.0, bias=False, mask="prefix",
             t_std=1.0),
        # a batch of 64x64 image grids, several packed into a row, with padding that sees nothing
        dict(name="fwd_image_docs_cap", op="fwd", B=2, H=12, Hkv=12, Lq=4096, Lk=4096, cap=50.0, bias=False,
             mask="docs", t_std=0.1),
        # shared key heads and a distance bias under a prefix mask, odd lengths
        dict(name="fwd_prefix_bias_gqa", op="fwd", B=1, H=12, Hkv=4, Lq=2501, Lk=2501, cap=0.0, bias=True,
             mask="prefix", t_std=1.0),
        # frame-causal video: the largest call
        dict(name="fwd_video_frames_cap", op="fwd", B=1, H=12, Hkv=12, Lq=8190, Lk=8190, cap=30.0, bias=True,
             mask="frames", t_std=1.0),
        # gradients of the packed image batch
        dict(name="bwd_image_docs_cap", op="bwd", B=1, H=12, Hkv=12, Lq=4096, Lk=4096, cap=50.0, bias=False,
             mask="docs", t_std=0.1),
        # gradients of shared key heads with a bias
        dict(name="bwd_prefix_bias_gqa", op="bwd", B=1, H=12, Hkv=4, Lq=1999, Lk=1999, cap=0.0, bias=True,
             mask="prefix", t_std=1.0),
        # video tokens over 512 text tokens: few keys, long streamed queries
        dict(name="bwd_cross_cap", op="bwd", B=1, H=12, Hkv=12, Lq=8190, Lk=512, cap=30.0, bias=False, mask="none",
             t_std=1.0),
        # a decoding step of 64 sequences appends one token each
        dict(name="append_step", op="append", B=64, H=12, Hkv=12, new=1, len=4096, page=64, interleaved=False),
        # one 30x52 frame joins each of four sequences
        dict(name="append_frame", op="append", B=4, H=12, Hkv=12, new=1560, len=6240, page=64, interleaved=True),
        # the decoding step of 64 sequences, no tangent
        dict(name="cache_step_b64", op="cache", B=64, H=12, Hkv=12, n=1, len=8192, page=64, cap=0.0, bias=False,
             tangent=False),
        # one sequence as long as the whole video, shared key heads, with tangents
        dict(name="cache_long_gqa", op="cache", B=1, H=40, Hkv=8, n=1, len=32760, page=64, cap=50.0, bias=False,
             tangent=True),
        # a few new tokens per sequence, short ragged contexts: latency
        dict(name="cache_few_rows", op="cache", B=4, H=12, Hkv=12, n=4, len=1001, page=16, cap=0.0, bias=True,
             tangent=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "append", "cache", "cache"])
    Hkv, group = rng.choice([(2, 1), (4, 3), (8, 1), (12, 1), (3, 4), (8, 5), (1, 7)])
    H = Hkv * group
    if op in ("fwd", "bwd"):
        most = 12 * 8190 * 8190 if op == "fwd" else 12 * 4096 * 4096
        mask = rng.choice(["none", "prefix", "docs", "docs_causal", "frames"])
        B = rng.choice([1, 1, 2, 3])
        # a backward pass of one key has gradients that are zero but for roundings
        Lk = _log(rng, 1 if op == "fwd" else 16, 8190)
        Lq = Lk if mask != "none" or rng.random() < 0.5 else _log(rng, 1, 8190)
        while B * H * Lq * Lk > most:
            Lq, Lk = max(1, Lq * 3 // 4), max(16, Lk * 3 // 4)
            if mask != "none":
                Lq = Lk
        return dict(op=op, B=B, H=H, Hkv=Hkv, Lq=Lq, Lk=Lk, cap=rng.choice([0.0, 15.0, 30.0, 50.0]),
                    bias=rng.random() < 0.4, mask=mask, t_std=rng.choice([0.1, 1.0]))
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        new = _log(rng, 1, 1560)
        B = max(1, min(_log(rng, 1, 64), 4 * 1560 * 24 // (new * (H + Hkv))))
        return dict(op=op, B=B, H=H, Hkv=Hkv, new=new, len=_log(rng, 1, 6240), page=page,
                    interleaved=rng.random() < 0.5)
    n = rng.choice([1, 1, 1, 2, 4, 7, 16])
    length = _log(rng, 16, 32760)
    B = max(1, min(_log(rng, 1, 64), 64 * 12 * 8192 // (length * max(Hkv, H * n // 16))))
    return dict(op=op, B=B, H=H, Hkv=Hkv, n=n, len=length, page=page, cap=rng.choice([0.0, 30.0, 50.0]),
                bias=rng.random() < 0.4, tangent=rng.random() < 0.6)


# ------------------------------------------------- what the sizes alone decide
def _bounds(case):
    """key_begin, key_end of every query row (a list each, the same for every
    sequence of the batch), or None without a mask."""
    Lq, Lk, mask = case["Lq"], case["Lk"], case["mask"]
    if mask == "none":
        return None
    rows = range(Lq)
    if mask == "prefix":  # a bidirectional prefix of a fifth, causal after it
        prefix = Lk // 5
        return [0] * Lq, [max(prefix, min(Lk, i + Lk - Lq + 1)) for i in rows]
    if mask == "frames":  # bidirectional inside a frame, all earlier frames visible
        frame = min(1560, max(1, Lk // 5))
        return [0] * Lq, [min(Lk, (i // frame + 1) * frame) for i in rows]
    cuts = sorted({math.ceil(Lk * 0.94 * (t / 5) ** 1.3) for t in range(6)})  # documents, then padding
    begin, end = [], []
    for i in rows:
        first = max((c for c in cuts if c <= i), default=0)
        after = [c for c in cuts if c > i]
        if not after:  # padding: sees nothing
            begin.append(0)
            end.append(0)
        else:
            begin.append(first)
            end.append(i + 1 if mask == "docs_causal" else after[0])
    return begin, end


def _lens(case):
    """Cached tokens of each sequence before the call's new ones (append) or
    with them (cache): ragged, the longest first, one short."""
    B, n = case["B"], case["len"]
    lens = [max(1, n - (7 * b * n) // (8 * max(1, B)) - (b % 3)) for b in range(B)]
    if B > 2:
        lens[-1] = 1 + n // 300
    return lens


def _pairs(case):
    """Visible (query row, key) pairs of one head, over the batch."""
    if case["op"] in ("fwd", "bwd"):
        b = _bounds(case)
        if b is None:
            return case["B"] * case["Lq"] * case["Lk"]
        return case["B"] * sum(max(0, e - s) for s, e in zip(*b))
    return sum(max(0, n - case["n"] + i + 1) for n in _lens(case) for i in range(case["n"]))


def work(case):
    H, Hkv, B = case["H"], case["Hkv"], case["B"]
    if case["op"] == "fwd":
        rows, keys = B * H * case["Lq"], B * Hkv * case["Lk"]
        return {"bytes": (4 * rows + 4 * keys) * D * 2 + 4 * rows, "flops": 12 * D * H * _pairs(case)}
    if case["op"] == "bwd":
        rows, keys = B * H * case["Lq"], B * Hkv * case["Lk"]
        # scores, their tangent and the two cotangent products (6), the gradients (9)
        return {"bytes": (8 * rows + 8 * keys) * D * 2 + 8 * rows, "flops": 30 * D * H * _pairs(case)}
    if case["op"] == "append":
        kv, qs = B * Hkv * case["new"] * D, B * H * case["new"] * D
        return {"bytes": 2 * kv * 2 + 2 * kv + 4 * qs * 2 + B * case["new"] * D * 4, "flops": 6 * (kv + 2 * qs)}
    tokens, rows = sum(_lens(case)), B * H * case["n"]
    parts = 4 if case["tangent"] else 2
    return {"bytes": 2 * tokens * Hkv * D + parts * rows * D * 2 + 4 * rows,
            "flops": 2 * parts * D * H * _pairs(case)}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * seed + 17)
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _slopes(case):
    """The geometric slopes of a distance bias, one per query head."""
    if not case["bias"]:
        return None
    H = case["H"]
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


def _pages(case, tokens, g):
    """A block table that hands out more pages than the tokens need, in random
    order, and the number of pages of the cache."""
    per = max(1, -(-tokens // case["page"]))
    total = case["B"] * per + 3
    order = torch.randperm(total, generator=g, device="cuda")[: case["B"] * per]
    return order.reshape(case["B"], per).to(torch.int32), total


def _filled(g, pages, case):
    """Codes and scales of pages full of normal keys (or values) whose size
    varies from page to page and channel to channel."""
    shape = (pages, case["Hkv"], case["page"], D)
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.rand((pages, case["Hkv"], 1, 1), generator=g, device="cuda") * 1.5 + 0.5
    x *= torch.rand((1, case["Hkv"], 1, D), generator=g, device="cuda") + 0.5
    scale = _scale_of(x.abs().amax((2, 3)))
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _gen(seed)
    state = dict(case=case, slopes=None, begin=None, end=None)
    B, H, Hkv = case["B"], case["H"], case["Hkv"]
    if case["op"] in ("fwd", "bwd"):
        Lq, Lk, t = case["Lq"], case["Lk"], case["t_std"]
        state["slopes"] = _slopes(case)
        state["x"] = [_normal(g, (B, H, Lq, D)), _normal(g, (B, Hkv, Lk, D)), _normal(g, (B, Hkv, Lk, D)),
                      _normal(g, (B, H, Lq, D), t), _normal(g, (B, Hkv, Lk, D), t), _normal(g, (B, Hkv, Lk, D), t)]
        bounds = _bounds(case)
        if bounds is not None:
            state["begin"], state["end"] = (torch.tensor(x, dtype=torch.int32, device="cuda").expand(B, Lq).contiguous()
                                            for x in bounds)
        if case["op"] == "bwd":  # what a training step's forward left, and the cotangents
            o, to, lse, mu = _forward(state)
            state["saved"] = [o.to(torch.bfloat16), to.to(torch.bfloat16), lse, mu]
            state["dout"], state["dtout"] = _normal(g, (B, H, Lq, D)), _normal(g, (B, H, Lq, D))
        return state
    lens = _lens(case)
    more = case["new"] if case["op"] == "append" else 0
    state["table"], pages = _pages(case, max(lens) + more, g)
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    state["k8"], state["ks"] = _filled(g, pages, case)
    state["v8"], state["vs"] = _filled(g, pages, case)
    if case["op"] == "append":
        total = B * more
        state["cu"] = torch.arange(B + 1, device="cuda", dtype=torch.int32) * more
        state["k"], state["v"] = _normal(g, (Hkv, total, D)), _normal(g, (Hkv, total, D), 2.0)
        state["q"], state["tq"] = _normal(g, (H, total, D)), _normal(g, (H, total, D))
        angle = (torch.arange(max(lens) + more, device="cuda", dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2)))
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
    else:
        state["slopes"] = _slopes(case)
        state["q"] = _normal(g, (B, H, case["n"], D))
        state["tq"] = _normal(g, (B, H, case["n"], D)) if case["tangent"] else None
    return state


# ----------------------------------------------------------- the plain forms
def _modified(z, case, slopes, distance, hidden):
    """Capped, biased and masked scores, and the cap's derivative."""
    df = None
    if case["cap"] > 0.0:
        t = torch.tanh(z / case["cap"])
        z, df = case["cap"] * t, 1.0 - t * t
    if slopes is not None:
        z = z - slopes[:, None, None] * distance
    return z.masked_fill(hidden, -INF), df


def _softmax(S):
    """P and the log-sum-exp; a row without keys has P = 0 and -inf."""
    m = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    lse = (m + torch.log(l))[..., 0]
    return p / torch.where(l > 0, l, torch.ones_like(l)), torch.where(l[..., 0] > 0, lse, torch.full_like(lse, -INF))


def _shared(x, case):
    """Key-side tensor of every query head, in fp32."""
    return x.float().repeat_interleave(case["H"] // case["Hkv"], 1)


def _grid(state):
    """|i + Lk - Lq - j| and the hidden pairs, of [B, 1, Lq, Lk] or less."""
    case = state["case"]
    i = torch.arange(case["Lq"], device="cuda")[:, None] + (case["Lk"] - case["Lq"])
    j = torch.arange(case["Lk"], device="cuda")[None]
    distance = (i - j).abs().float()
    if state["begin"] is None:
        return distance, torch.zeros((), dtype=torch.bool, device="cuda")
    return distance, ((j < state["begin"][..., None]) | (j >= state["end"][..., None]))[:, None]


def _forward(state):
    case, s = state["case"], D ** -0.5
    q, k, v, tq, tk, tv = state["x"]
    q, tq = q.float(), tq.float()
    k, v, tk, tv = (_shared(x, case) for x in (k, v, tk, tv))
    distance, hidden = _grid(state)
    S, df = _modified(s * (q @ k.mT), case, state["slopes"], distance, hidden)
    P, lse = _softmax(S)
    del S
    dS = s * (tq @ k.mT + q @ tk.mT)
    if df is not None:
        dS = dS * df
    W = P * dS
    mu = W.sum(-1, keepdim=True)
    o = P @ v
    to = W @ v - mu * o + P @ tv
    return o, to, lse, mu[..., 0]


def _plain_fwd(state):
    o, to, lse, _ = _forward(state)
    return o.to(torch.bfloat16), to.to(torch.bfloat16), lse


def _plain_bwd(state):
    """Closed form: with A = dtO V^T, B = dO V^T + dtO tV^T, u = dS,
    dS_bar = P (A - a), S_bar = P (B + A (u - mu) - a u - D), and the cap's
    chain rule z_bar = f' S_bar + f'' dz dS_bar, dz_bar = f' dS_bar."""
    case, s = state["case"], D ** -0.5
    q, k, v, tq, tk, tv = state["x"]
    q, tq, do, dto = q.float(), tq.float(), state["dout"].float(), state["dtout"].float()
    k, v, tk, tv = (_shared(x, case) for x in (k, v, tk, tv))
    distance, hidden = _grid(state)
    z = s * (q @ k.mT)
    S, df = _modified(z, case, state["slopes"], distance, hidden)
    P, _ = _softmax(S)
    del S
    dz = s * (tq @ k.mT + q @ tk.mT)
    u = dz if df is None else dz * df
    mu = (P * u).sum(-1, keepdim=True)
    dv = P.mT @ do + (P * (u - mu)).mT @ dto
    dtv = P.mT @ dto
    A = dto @ v.mT
    a = (P * A).sum(-1, keepdim=True)
    bar = do @ v.mT + dto @ tv.mT + A * (u - mu) - a * u
    zb = P * (bar - (P * bar).sum(-1, keepdim=True))
    dzb = P * (A - a)
    del bar, A, P
    if df is not None:
        t = torch.tanh(z / case["cap"])
        zb = df * (zb - (2.0 / case["cap"]) * t * dz * dzb)
        dzb = df * dzb
    dq, dtq = s * (zb @ k + dzb @ tk), s * (dzb @ k)
    dk, dtk = s * (zb.mT @ q + dzb.mT @ tq), s * (dzb.mT @ q)
    group = case["H"] // case["Hkv"]
    out = dict(dq=dq, dtq=dtq, **{n: x.unflatten(1, (-1, group)).sum(2)
                                  for n, x in (("dk", dk), ("dv", dv), ("dtk", dtk), ("dtv", dtv))})
    return {n: x.to(torch.bfloat16) for n, x in out.items()}


def _scale_of(amax):
    """The smallest power of two that brings amax to at most 448, the largest
    e4m3 value (2^-100 for zeros)."""
    mant, expo = torch.frexp(amax)  # amax = mant 2^expo, mant in [0.5, 1)
    e = expo - 9 + (mant > 0.875).to(expo.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(-100, 100)
    return torch.ldexp(torch.ones_like(amax), e)


def _rotated(x, cos, sin, interleaved):
    """Pairs of channels (2i, 2i + 1), or (i, i + 64), turned by their angles."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x[..., : D // 2], x[..., D // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _write(codes, scale, x, table, start, new):
    """x [Hkv, B * new, D] (fp32) joins one of the two caches: each touched page keeps its earlier tokens, takes the larger of its old scale
    (none if the page starts here) and its new tokens' and is rounded to it."""
    B, page = table.shape[0], codes.shape[2]
    touched = (new + page - 2) // page + 1
    first = start // page  # [B]
    slot = first[:, None] + torch.arange(touched, device="cuda")
    used = slot <= ((start + new - 1) // page)[:, None]
    # pages past a sequence's last one take part as copies of it and are not written
    index = table.gather(1, slot.clamp(max=table.shape[1] - 1).long()).long()
    token = slot[..., None] * page + torch.arange(page, device="cuda") - start[:, None, None]  # [B, touched, page]
    fresh = (token >= 0) & (token < new)
    row = torch.arange(B, device="cuda")[:, None, None] * new + token.clamp(0, new - 1)
    value = x[:, row].permute(1, 2, 0, 3, 4)  # [B, touched, Hkv, page, D]
    fresh = fresh[:, :, None, :, None]
    old_scale = scale[index]
    grown = _scale_of((value.abs() * fresh).amax((3, 4)))
    begins = (slot * page >= start[:, None])[:, :, None]
    new_scale = torch.where(begins, grown, torch.maximum(grown, old_scale))
    old = codes[index].float() * (old_scale / new_scale)[..., None, None]
    both = torch.where(fresh, value / new_scale[..., None, None], old)
    keep = (token < new)[:, :, None, :, None]  # slots behind the new tokens stay as they were
    both = torch.where(keep, both.to(torch.float8_e4m3fn).float(), codes[index].float())
    codes.view(torch.uint8)[index[used]] = both[used].to(torch.float8_e4m3fn).view(torch.uint8)
    scale[index[used]] = new_scale[used]


def _plain_append(state):
    case = state["case"]
    start, new = state["lens"].long(), case["new"]
    position = (start[:, None] + torch.arange(new, device="cuda")).flatten()
    cos, sin = state["cos"][position], state["sin"][position]
    turn = [_rotated(state[n].float(), cos, sin, case["interleaved"]) for n in ("k", "q", "tq")]
    _write(state["k8"], state["ks"], turn[0], state["table"], start, new)
    _write(state["v8"], state["vs"], state["v"].float(), state["table"], start, new)
    return dict({n: state[n] for n in ("k8", "ks", "v8", "vs")}, q=turn[1].to(torch.bfloat16),
                tq=turn[2].to(torch.bfloat16))


def _cached(codes, scale, state):
    """[B, H, tokens, D] in fp32, zeros behind each sequence's end."""
    case, table = state["case"], state["table"].long()
    x = codes[table].float() * scale[table][..., None, None]  # [B, pages, Hkv, page, D]
    x = x.transpose(1, 2).flatten(2, 3)
    live = torch.arange(x.shape[2], device="cuda") < state["lens"][:, None]
    return x.masked_fill(~live[:, None, :, None], 0.0).unflatten(1, (case["Hkv"], 1))


def _plain_cache(state):
    case, s = state["case"], D ** -0.5
    B, H, Hkv, n = case["B"], case["H"], case["Hkv"], case["n"]
    k, v = _cached(state["k8"], state["ks"], state), _cached(state["v8"], state["vs"], state)
    group = lambda x: x.float().unflatten(1, (Hkv, H // Hkv))  # noqa: E731  [B, Hkv, group, n, D]
    j = torch.arange(k.shape[3], device="cuda")
    i = state["lens"][:, None].long() - n + torch.arange(n, device="cuda")  # positions, [B, n]
    hidden = (j > i[..., None]) | (j >= state["lens"][:, None, None])
    distance = (i[..., None] - j).abs().float()[:, None]
    z = (s * (group(state["q"]) @ k.mT)).flatten(1, 2)
    S, df = _modified(z, case, state["slopes"], distance, hidden[:, None])
    P, lse = _softmax(S)
    across = lambda w: (w.unflatten(1, (Hkv, H // Hkv)) @ v).flatten(1, 2)  # noqa: E731
    o = across(P)
    if state["tq"] is None:
        return o.to(torch.bfloat16), lse
    dS = (s * (group(state["tq"]) @ k.mT)).flatten(1, 2)
    W = P * (dS if df is None else dS * df)
    to = across(W) - W.sum(-1, keepdim=True) * o
    return o.to(torch.bfloat16), to.to(torch.bfloat16), lse


# -------------------------------------------------------------- one pass of it
def run(state):
    case = state["case"]
    if own:
        import attention_forward_mode_b200 as ajvp

        if case["op"] in ("fwd", "bwd"):
            kw = dict(softcap=case["cap"], slopes=state["slopes"], key_begin=state["begin"], key_end=state["end"])
            if case["op"] == "fwd":
                return ajvp.attn_jvp_fwd_scored(*state["x"], **kw)
            return ajvp.attn_jvp_bwd_scored(*state["x"], *state["saved"], state["dout"], state["dtout"], **kw)
        if case["op"] == "append":
            q, tq = ajvp.attn_jvp_cache_append(state["k"], state["v"], state["k8"], state["v8"], state["ks"],
                                               state["vs"], state["table"], state["lens"], state["cu"],
                                               q=state["q"], tq=state["tq"], cos=state["cos"], sin=state["sin"],
                                               interleaved=case["interleaved"])
            return dict(k8=state["k8"], ks=state["ks"], v8=state["v8"], vs=state["vs"], q=q, tq=tq)
        o, to, lse = ajvp.attn_jvp_fwd_cache(state["q"], state["tq"], state["k8"], state["v8"], state["ks"],
                                             state["vs"], state["table"], state["lens"], softcap=case["cap"],
                                             slopes=state["slopes"])
        return (o, lse) if to is None else (o, to, lse)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "append": _plain_append, "cache": _plain_cache}[case["op"]](state)


# ------------------------------------------------------------------- in 64 bits
def _head(state, b, h, leaf=False):
    """Inputs of one query head in 64 bits and its score function."""
    case = state["case"]
    q, k, v, tq, tk, tv = state["x"]
    hk = h // (case["H"] // case["Hkv"])
    x = [t[b, i].double().requires_grad_(leaf) for t, i in ((q, h), (k, hk), (v, hk), (tq, h), (tk, hk), (tv, hk))]
    i = torch.arange(case["Lq"], device="cuda", dtype=torch.float64)[:, None] + (case["Lk"] - case["Lq"])
    j = torch.arange(case["Lk"], device="cuda", dtype=torch.float64)
    shift = torch.zeros((case["Lq"], case["Lk"]), dtype=torch.float64, device="cuda")
    if state["slopes"] is not None:
        shift -= state["slopes"][h].double() * (i - j).abs()
    if state["begin"] is not None:
        seen = (j >= state["begin"][b][:, None]) & (j < state["end"][b][:, None])
        shift[~seen] = -INF
    return x, shift


def _exact_rows(x, shift, cap):
    """O, tO, log-sum-exp of one head, rows without keys zero."""
    q, k, v, tq, tk, tv = x
    s = D ** -0.5
    z, dz = s * (q @ k.T), s * (tq @ k.T + q @ tk.T)
    if cap > 0.0:
        h = torch.tanh(z / cap)
        z, dz = cap * h, dz * (1 - h * h)
    lse = torch.logsumexp(z + shift, -1, keepdim=True)
    empty = torch.isinf(lse)
    P = torch.exp(z + shift - lse.masked_fill(empty, 0.0))
    centred = dz - (P * dz).sum(-1, keepdim=True)
    return P @ v, (P * centred) @ v + P @ tv, lse[..., 0]


def _exact_attention(case, state):
    B, H, Hkv = case["B"], case["H"], case["Hkv"]
    if case["op"] == "fwd":
        rows = [_exact_rows(*_head(state, b, h), case["cap"]) for b in range(B) for h in range(H)]
        return tuple(torch.stack(t).unflatten(0, (B, H)) for t in zip(*rows))
    like = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in state["x"]]
    for b in range(B):
        for h in range(H):
            x, shift = _head(state, b, h, leaf=True)
            live = ~torch.isinf(shift).all(-1)  # rows without keys are constants
            o, to, _ = _exact_rows([x[0][live], x[1], x[2], x[3][live], x[4], x[5]], shift[live], case["cap"])
            loss = ((o * state["dout"][b, h][live].double()).sum()
                    + (to * state["dtout"][b, h][live].double()).sum())
            hk = h // (H // Hkv)
            for t, at, grad in zip(like, (h, hk, hk, h, hk, hk), torch.autograd.grad(loss, x)):
                t[b, at] += grad
    return dict(zip(("dq", "dk", "dv", "dtq", "dtk", "dtv"), like))


def _exact_append(case, state):
    """Token by token of each page in 64 bits, on the host."""
    import numpy as np

    def turn(x, position):
        c, s = cos[position], sin[position]
        if case["interleaved"]:
            z = (x[..., 0::2] + 1j * x[..., 1::2]) * (c + 1j * s)
            return np.stack((z.real, z.imag), -1).reshape(x.shape)
        z = (x[..., : D // 2] + 1j * x[..., D // 2:]) * (c + 1j * s)
        return np.concatenate((z.real, z.imag), -1)

    def rounded(x):
        """The nearest e4m3 values, ties to even, saturating."""
        _, e = np.frexp(x)
        step = np.exp2(np.maximum(e - 1, -6) - 3.0)
        return np.clip(np.rint(x / step) * step, -448.0, 448.0)

    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    cos, sin = host(state["cos"]), host(state["sin"])
    lens, table, new, page = state["lens"].tolist(), state["table"].cpu().numpy(), case["new"], case["page"]
    position = np.concatenate([np.arange(n, n + new) for n in lens])
    k, v = turn(host(state["k"]), position), host(state["v"])
    out = dict(q=turn(host(state["q"]), position), tq=turn(host(state["tq"]), position))
    for x, codes, scale in ((k, "k8", "ks"), (v, "v8", "vs")):
        c, f = host(state[codes].float()), host(state[scale])
        for b, n in enumerate(lens):
            for p in range(n // page, (n + new - 1) // page + 1):
                at = table[b, p]
                lo, hi = max(n, p * page), min(n + new, (p + 1) * page)
                part = x[:, b * new + lo - n: b * new + hi - n]  # [Hkv, tokens, D]
                amax = np.abs(part).max((1, 2))
                grown = np.exp2(np.clip(np.ceil(np.log2(np.maximum(amax, 1e-300) / 448.0)), -100, 100))
                kept = lo - p * page
                both = grown if kept == 0 else np.maximum(grown, f[at])
                c[at, :, :kept] = rounded(c[at, :, :kept] * (f[at] / both)[:, None, None])
                c[at, :, kept: kept + hi - lo] = rounded(part / both[:, None, None])
                f[at] = both
        out[codes], out[scale] = c, f
    return {n: torch.from_numpy(np.ascontiguousarray(out[n])) for n in ("k8", "ks", "v8", "vs", "q", "tq")}


def _exact_cache(case, state):
    H, Hkv, n, s = case["H"], case["Hkv"], case["n"], D ** -0.5
    outs = []
    for b, length in enumerate(state["lens"].tolist()):
        pages = state["table"][b, : -(-length // case["page"])].long()
        k, v = (state[c][pages].double().mul(state[f][pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)
                [:, :length].repeat_interleave(H // Hkv, 0) for c, f in (("k8", "ks"), ("v8", "vs")))
        z = s * torch.einsum("hid,hjd->hij", state["q"][b].double(), k)
        slope = torch.ones_like(z)
        if case["cap"] > 0.0:
            h = torch.tanh(z / case["cap"])
            z, slope = case["cap"] * h, 1 - h * h
        i = torch.arange(length - n, length, device="cuda", dtype=torch.float64)[:, None]
        j = torch.arange(length, device="cuda", dtype=torch.float64)
        if state["slopes"] is not None:
            z = z - state["slopes"].double()[:, None, None] * (i - j).abs()
        z = z.masked_fill(j > i, -INF)
        lse = torch.logsumexp(z, -1, keepdim=True)
        P = torch.exp(z - lse.masked_fill(torch.isinf(lse), 0.0))
        o = torch.einsum("hij,hjd->hid", P, v)
        if state["tq"] is None:
            outs.append((o, lse[..., 0]))
            continue
        u = slope * s * torch.einsum("hid,hjd->hij", state["tq"][b].double(), k)
        outs.append((o, torch.einsum("hij,hjd->hid", P * (u - (P * u).sum(-1, keepdim=True)), v), lse[..., 0]))
    return tuple(torch.stack(t) for t in zip(*outs))


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        return _exact_attention(case, state)
    return _exact_append(case, state) if case["op"] == "append" else _exact_cache(case, state)
