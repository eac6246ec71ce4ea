"""attn_jvp_fwd_scored(_stats) and attn_jvp_bwd_scored on the GPU against the
64-bit definition: caps, biases, masks with empty rows, shared key heads, odd
lengths from one key on, split and unsplit key sides."""
import pytest
import torch

import attention_forward_mode_b200 as ajvp
import scored_reference as ref

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "tq", "tk", "tv")


def make(B, H, Hkv, Lq, Lk, seed=0, t_std=1.0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda h, n, s: (torch.randn((B, h, n, 128), generator=g, device="cuda") * s).bfloat16()  # noqa: E731
    return dict(q=draw(H, Lq, std), k=draw(Hkv, Lk, std), v=draw(Hkv, Lk, 1.0), tq=draw(H, Lq, t_std),
                tk=draw(Hkv, Lk, t_std), tv=draw(Hkv, Lk, t_std)), dict(dout=draw(H, Lq, 1.0), dtout=draw(H, Lq, 1.0))


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


def random_bounds(B, Lq, Lk, seed):
    """Intervals in no order: some empty, some reversed, some past the ends."""
    g = torch.Generator().manual_seed(seed)
    begin = torch.randint(-5, Lk + 5, (B, Lq), generator=g)
    end = begin + torch.randint(-20, Lk + 20, (B, Lq), generator=g)
    return begin.int().cuda(), end.int().cuda()


def masks(kind, B, Lq, Lk, seed):
    if kind == "none":
        return {}
    if kind == "random":
        b, e = random_bounds(B, Lq, Lk, seed)
    elif kind == "docs":
        b, e = ajvp.key_bounds(Lq, Lk, documents=[Lk // 7, Lk // 3, Lk // 2, Lk - Lk // 9], causal=seed % 2 == 0)
    elif kind == "prefix":
        b, e = ajvp.key_bounds(Lq, Lk, causal=True, prefix=Lk // 5)
    elif kind == "frames":
        b, e = ajvp.key_bounds(Lq, Lk, frame=max(1, Lk // 4))
    elif kind == "window":
        b, e = ajvp.key_bounds(Lq, Lk, causal=True, window=max(1, Lk // 6))
    else:  # every row empty
        b, e = torch.zeros(Lq, dtype=torch.int32, device="cuda"), torch.zeros(Lq, dtype=torch.int32, device="cuda")
    return dict(key_begin=b, key_end=e)


def ref_opts(kw, B):
    out = {n: kw[n] for n in ("softcap", "slopes") if n in kw}
    for n, m in (("key_begin", "begin"), ("key_end", "end")):
        if n in kw:
            x = kw[n] if kw[n].dim() == 2 else kw[n].expand(B, -1)
            out[m] = x.clamp(0)
    return out


CASES = [  # B, H, Hkv, Lq, Lk, cap, bias, mask
    (1, 1, 1, 1, 1, 0.0, False, "none"),
    (2, 2, 1, 1, 200, 30.0, True, "none"),
    (1, 2, 2, 3, 65, 5.0, False, "random"),
    (1, 4, 2, 129, 127, 0.0, True, "random"),
    (2, 2, 2, 200, 200, 30.0, False, "docs"),
    (1, 6, 2, 333, 333, 0.0, True, "docs"),
    (1, 3, 1, 257, 257, 50.0, True, "prefix"),
    (2, 2, 2, 130, 400, 0.0, False, "prefix"),
    (1, 2, 2, 400, 130, 15.0, False, "window"),
    (1, 5, 5, 511, 511, 30.0, True, "frames"),
    (1, 2, 1, 300, 300, 30.0, True, "empty"),
    (1, 2, 2, 1000, 77, 20.0, False, "none"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_backward(case):
    B, H, Hkv, Lq, Lk, cap, bias, mask = case
    inp, cot = make(B, H, Hkv, Lq, Lk, seed=Lq + 7 * Lk)
    kw = dict(softcap=cap, **({"slopes": slopes_of(H)} if bias else {}), **masks(mask, B, Lq, Lk, seed=Lq))
    x = [inp[n] for n in NAMES]
    s = 128 ** -0.5
    o, to, lse, mu = ajvp.attn_jvp_fwd_scored_stats(*x, **kw)
    (ro, rto, rlse, rmu), (eo, eto) = ref.forward(*x, s, bounds=True, **ref_opts(kw, B))
    torch.cuda.synchronize()
    assert ajvp.check_device_status() == ajvp.AJVP_OK
    ref.check("o", o, ro, eo)
    ref.check("to", to, rto, eto)
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert (o[empty] == 0).all() and (to[empty] == 0).all() and (mu[empty] == 0).all()
    # scores are fp32 sums of 128 products (some 2^-17 absolute here) and the cap's tanh adds c 2^-21
    tol = 2.0 ** -15 * (1.0 + rlse[~empty].abs())
    assert ((lse[~empty].double() - rlse[~empty]).abs() <= tol).all()
    g = ajvp.attn_jvp_bwd_scored(*x, o, to, lse, mu, cot["dout"], cot["dtout"], **kw)
    rg, eg = ref.backward(*x, cot["dout"], cot["dtout"], s, bounds=True, **ref_opts(kw, B))
    torch.cuda.synchronize()
    assert ajvp.check_device_status() == ajvp.AJVP_OK
    for n in ajvp._binding.GRAD_NAMES:
        ref.check(n, g[n], rg[n], eg[n])
