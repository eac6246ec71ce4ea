"""The paged 8-bit cache where its attention could go wrong quietly: early
tokens that hardly count, truncated rows, scales of zero, wide caps, values
that are all zero, chunks of many query tokens."""
import numpy as np
import pytest
import torch

import attention_forward_mode_b200 as ajvp
import cache_reference as ref
from test_gpu_cache import check_rows, empty_cache, filled, tables

pytestmark = pytest.mark.gpu
S = 128 ** -0.5


def leading(low, q0, far, seed=41):
    """One decoding token of each of 32 sequences over 1024 tokens, 8 heads (256 sequences and heads, a CTA each).
    The first 128 tokens, whole runs of every warp, score ``low q0`` / sqrt(128) below the others and have a score
    tangent of 8 ``far`` / sqrt(128) (``far`` a pair: its two values in turn), the others one of the order of 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_seq, Hkv, L, lead, page = 32, 8, 1024, 128, 64
    table, pages = tables(n_seq, L // page, 1, seed)
    cache, table = empty_cache(pages, Hkv, page, seed), table.cuda()
    k, v = (torch.randn((Hkv, n_seq, L, 128), generator=g, device="cuda") for _ in range(2))
    k[:, :, :lead, 0] = -low
    for i, f in enumerate(far):
        k[:, :, i:lead:len(far), 1] = f
    q, tq = (torch.randn((n_seq, Hkv, 1, 128), generator=g, device="cuda") * 0.05 for _ in range(2))
    q[..., 0], q[..., 1], tq[..., 1], tq[..., 0] = q0, 0.0, 8.0, 0.0
    cu = torch.arange(n_seq + 1, dtype=torch.int32, device="cuda") * L
    flat = lambda x: x.flatten(1, 2).bfloat16()  # noqa: E731
    ajvp.attn_jvp_cache_append(flat(k), flat(v), *cache, table, torch.zeros(n_seq, dtype=torch.int32, device="cuda"), cu)
    return q.bfloat16(), tq.bfloat16(), cache, table, torch.full((n_seq,), L, dtype=torch.int32, device="cuda")


def tangent_parts(q, tq, cache, table, L):
    """to in 64 bits, and per row: P, dS - mu, V."""
    k8, v8, ks, vs = cache
    k, v = (c[table.long()].double().mul(f[table.long()].double()[..., None, None]).transpose(1, 2).flatten(2, 3)[:, :, :L]
            for c, f in ((k8, ks), (v8, vs)))
    P = torch.softmax(S * (q.double() @ k.mT), -1)
    u = S * (tq.double() @ k.mT)
    u = u - (P * u).sum(-1, keepdim=True)
    return (P * u) @ v, P, u, v


def independent_roundings(to, P, u, v):
    """A row's rounding error in the mean square, [.., 1, 128]: weights P (dS - r) rounded to f16 and outputs to
    bf16, each off by at most half a step h relative and h / sqrt(3) in the mean, independently.  The reference r
    is a mean of dS over at least a sixteenth of the weight summed so far, so that |r - mu| <= 16 sum P |dS - mu|."""
    h = ref.U16 * (u.abs() + 16 * (P * u.abs()).sum(-1, keepdim=True)) * P
    return (h.square() @ v.square() + (ref.UB * to).square()) / 3


def as_exact_as_its_roundings(args):
    q, tq, cache, table, lens = args
    o, to, _ = ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, lens)
    rto, P, u, v = tangent_parts(q, tq, cache, table, int(lens[0]))
    mean_square = independent_roundings(rto, P, u, v).sum()
    # 256 x 128 outputs, a sum of many independent errors: twice its mean in norm is far outside
    assert (to.double() - rto).square().sum() <= 4 * mean_square


@pytest.mark.parametrize("low,far", [(16.0, 400.0), (24.0, 6000.0)])
def test_tangents_after_tokens_that_hardly_count(low, far):
    """The first tokens weigh 2^-16 (2^-24) of a later one: tO is as exact as without them."""
    as_exact_as_its_roundings(leading(low, 8.0, (far,)))


def test_the_unit_of_tangents_follows_the_weights():
    """First tokens of some 2^-60 of a later one's weight, whose score tangents are 2^30 times as large."""
    as_exact_as_its_roundings(leading(2.0 ** 14, 0.029, (2.0 ** 30, -(2.0 ** 30))))


@pytest.mark.parametrize("tangent", [True, False])
def test_rows_within_an_underestimated_max_seqlen(tangent):
    """Rows past max_seqlen are not computed; the others stand where they stand, whatever max_seqlen is."""
    counts, lens, H, most = [5, 2, 0, 9], [200, 40, 16, 333], 4, 3
    cache, table, g = filled(4, 2, 32, lens, seed=42)
    cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
    q, tq = (torch.randn((H, cu[-1], 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    o, to = torch.full_like(q, 5.0), torch.full_like(q, 5.0)
    lse = torch.full((H, cu[-1]), 5.0, device="cuda")
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ajvp.attn_jvp_fwd_cache(q, tq if tangent else None, *cache, table, dev(lens), cu_seqlens=dev(cu), max_seqlen=most,
                            o=o, to=to if tangent else None, lse=lse)
    some = [b for b, n in enumerate(counts) if n]  # (the reference takes sequences that have rows)
    rows = [slice(cu[b], cu[b + 1]) for b in some]
    want = ref.attention([q[:, r] for r in rows], [tq[:, r] for r in rows] if tangent else None, *cache, table[some],
                         [lens[b] for b in some], S)
    for r, (ro, rto, rlse, bo, bto) in zip(rows, want):
        n = min(most, r.stop - r.start)
        assert ((o[:, r][:, :n].double() - ro[:, :n]).abs() <= bo[:, :n]).all()
        if tangent:
            assert ((to[:, r][:, :n].double() - rto[:, :n]).abs() <= bto[:, :n]).all()
        assert ((lse[:, r][:, :n] - rlse.cuda()[:, :n]).abs() <= 2.0 ** -15 * (1.0 + rlse.cuda()[:, :n].abs())).all()
        assert all((x[:, r][:, n:] == 5.0).all() for x in (o, lse) + ((to,) if tangent else ()))


def test_scales_of_zero():
    """A page whose key scale is 0 holds zero keys: its tokens score 0 and count.  A value scale of 0: zero values."""
    lens, H, Hkv, page = [300, 33], 4, 2, 16
    cache, table, g = filled(2, Hkv, page, lens, seed=43)
    cache[2][table[0, 3], 0] = cache[2][table[0, 4]] = cache[2][table[1, 2], 1] = 0.0
    cache[3][table[0, 4], 1] = cache[3][table[0, 9]] = 0.0
    q, tq = (torch.randn((2, H, 3, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for t in (tq, None):
        o, to, lse = ajvp.attn_jvp_fwd_cache(q, t, *cache, table, lens_d)
        check_rows(o, to, lse, ref.attention(list(q), None if t is None else list(t), *cache, table, lens, S))
    zero = [torch.zeros_like(t.view(torch.uint8)).view(t.dtype) if t.dim() == 4 else torch.zeros_like(t) for t in cache]
    o, to, lse = ajvp.attn_jvp_fwd_cache(q[:, :, :1], tq[:, :, :1], *zero, table, lens_d)
    assert (o == 0).all() and (to == 0).all()
    want = torch.log(lens_d.double())[:, None, None]
    # scores of 0 against a reference of some -100 in log2 units (a value scale of 0 counts as a very small one):
    # fp32 holds log2 of the weights' sum to 2^-18, and lg2.approx errs by some steps more; 2^-15 as elsewhere
    assert ((lse.double() - want).abs() <= 2.0 ** -15).all()


@pytest.mark.parametrize("cap", [1e3, 1e5, 1e7, 1e20])
def test_caps_far_above_the_scores(cap):
    """A cap of 1e7 is no cap: the scores are as exact as without one."""
    lens, H = [500, 70], 6
    cache, table, g = filled(2, 2, 32, lens, seed=44)
    q, tq = (torch.randn((2, H, 2, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, to, lse = ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, lens_d, softcap=cap)
    check_rows(o, to, lse, ref.attention(list(q), list(tq), *cache, table, lens, S, cap))


def test_values_that_are_all_zero():
    """A context of zero values, large keys and small queries: O and tO are zeros, lse is what it is."""
    lens, H, page = [4096, 100], 2, 64
    cache, table, g = filled(2, 1, page, lens, seed=45)
    total = sum(lens)
    k = (torch.randn((1, total, 128), generator=g, device="cuda") * 2.0 ** 14).bfloat16()
    cu = torch.tensor([0, lens[0], total], dtype=torch.int32, device="cuda")
    ajvp.attn_jvp_cache_append(k, torch.zeros_like(k), *cache, table, torch.zeros(2, dtype=torch.int32, device="cuda"), cu)
    q = (torch.randn((2, H, 1, 128), generator=g, device="cuda") * 2.0 ** -13).bfloat16()
    tq = torch.randn((2, H, 1, 128), generator=g, device="cuda").bfloat16()
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, to, lse = ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, lens_d)
    assert (o == 0).all() and (to == 0).all()
    for b, (_, _, rlse, _, _) in enumerate(ref.attention(list(q), list(tq), *cache, table, lens, S)):
        assert ((lse[b] - rlse).abs() <= 2.0 ** -15 * (1.0 + rlse.abs())).all()


@pytest.mark.parametrize("case", [(4, 2, 300, 32, [1000, 300, 17], 30.0, True), (2, 1, 1560, 64, [4680], 0.0, True),
                                  (5, 1, 701, 16, [800, 1500], 0.0, False)],
                         ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_chunks_of_many_query_tokens(case):
    """Whole chunks and frames of queries over the cache; where a sequence is shorter than the chunk, its first
    rows stand at negative positions and see nothing."""
    H, Hkv, n, page, lens, cap, tangent = case
    cache, table, g = filled(len(lens), Hkv, page, lens, seed=46)
    q, tq = (torch.randn((len(lens), H, n, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, to, lse = ajvp.attn_jvp_fwd_cache(q, tq if tangent else None, *cache, table, lens_d, softcap=cap)
    check_rows(o, to, lse, ref.attention(list(q), list(tq) if tangent else None, *cache, table, lens, S, cap))
