"""The paged 8-bit cache on the GPU: appends equal to the definition code by
code, attention + JVP over it against 64 bits, and both together."""
import numpy as np
import pytest
import torch

import attention_forward_mode_b200 as ajvp
import cache_reference as ref

pytestmark = pytest.mark.gpu


def tables(n_seq, width, extra, seed):
    g = torch.Generator().manual_seed(seed)
    n = n_seq * width + extra
    return torch.randperm(n, generator=g)[: n_seq * width].reshape(n_seq, width).int(), n


def angles(n_pos):
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(64) / 64)
    return torch.tensor(np.cos(a), dtype=torch.float32).cuda(), torch.tensor(np.sin(a), dtype=torch.float32).cuda()


def empty_cache(pages, Hkv, page, seed):
    """A cache that holds garbage, NaN codes among it."""
    g = torch.Generator().manual_seed(seed)
    code = lambda: torch.randint(0, 256, (pages, Hkv, page, 128), generator=g, dtype=torch.uint8).cuda() \
        .view(torch.float8_e4m3fn)  # noqa: E731
    return code(), code(), torch.full((pages, Hkv), float("nan"), device="cuda"), \
        torch.full((pages, Hkv), float("nan"), device="cuda")


class Model:
    """The cache by its definition, on the host, beside the one on the GPU."""

    def __init__(self, cache):
        f = lambda t: torch.nan_to_num(t.float(), nan=0.0).cpu().double().numpy()  # noqa: E731
        self.k8, self.v8, self.ks, self.vs = (f(t) for t in cache)
        self.written = np.zeros(self.k8.shape[:3], dtype=bool)

    def append(self, k, v, table, lens, cu, rot=None):
        k, v = k.float().cpu().numpy(), v.float().cpu().numpy()
        if rot is not None:
            cos, sin, inter = rot
            pos = np.concatenate([np.arange(n, n + cu[b + 1] - cu[b]) for b, n in enumerate(lens)])
            pos = np.clip(pos, 0, cos.shape[0] - 1)
            k = ref.turn(k[:, : len(pos)], cos.cpu().numpy()[pos], sin.cpu().numpy()[pos], inter)
        ref.append(k, self.k8, self.ks, table, lens, cu)
        ref.append(v, self.v8, self.vs, table, lens, cu)
        page = self.k8.shape[2]
        for b, n in enumerate(lens):
            for t in range(n, n + cu[b + 1] - cu[b]):
                if t // page < table.shape[1] and 0 <= table[b, t // page] < self.k8.shape[0]:
                    self.written[table[b, t // page], :, t % page] = True

    def check(self, cache):
        k8, v8, ks, vs = (t.float().cpu().double().numpy() for t in cache)
        w = self.written
        assert np.array_equal(k8[w], self.k8[w]) and np.array_equal(v8[w], self.v8[w])
        used = w.any(2)
        assert np.array_equal(ks[used], self.ks[used]) and np.array_equal(vs[used], self.vs[used])


APPENDS = [  # H, Hkv, page, starts, counts per call, rotation
    (2, 2, 16, [0], [[1], [1], [14], [1], [33]], None),
    (4, 1, 32, [0, 7, 31, 64], [[1, 1, 1, 1], [5, 0, 40, 2]], "half"),
    (6, 3, 48, [0, 100], [[97, 3], [0, 1], [1, 95]], "pairs"),
    (1, 1, 128, [3, 500, 0], [[300, 0, 128], [1, 1, 1]], "half"),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"h{c[0]}-{c[1]}-page{c[2]}-{c[5]}")
def test_append_equals_the_definition(case):
    H, Hkv, page, lens, calls, rot = case
    lens = list(lens)
    g = torch.Generator(device="cuda").manual_seed(page)
    most = max(n + sum(c[b] for c in calls) for b, n in enumerate(lens))
    table, pages = tables(len(lens), -(-most // page), 3, seed=page)
    cache = empty_cache(pages, Hkv, page, seed=1)
    cos, sin = angles(most)
    model = Model(cache)
    # the first call appends the earlier tokens, so that the pages' scales and codes are defined
    start = [0] * len(lens)
    for step, counts in enumerate([list(lens)] + calls):
        total = sum(counts)
        spread = 4.0 ** step  # later tokens are larger: scales grow over earlier codes
        cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
        k, v = ((torch.randn((Hkv, total, 128), generator=g, device="cuda") * spread).bfloat16() for _ in range(2))
        q, tq = (torch.randn((H, total, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
        kw = {} if rot is None else dict(cos=cos, sin=sin, interleaved=rot == "pairs", q=q, tq=tq)
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        qo, tqo = ajvp.attn_jvp_cache_append(k, v, *cache, table.cuda(), dev(start), dev(cu), **kw)
        model.append(k, v, table.numpy(), start, cu, None if rot is None else (cos, sin, rot == "pairs"))
        model.check(cache)
        if rot is not None and total:
            pos = np.concatenate([np.arange(n, n + c) for n, c in zip(start, counts)])
            for x, y in ((q, qo), (tq, tqo)):
                want = ref.turn(x.float().cpu().numpy(), cos.cpu().numpy()[pos], sin.cpu().numpy()[pos], rot == "pairs")
                assert torch.equal(y.cpu(), torch.tensor(want).bfloat16())
        start = [n + c for n, c in zip(start, counts)]


def filled(n_seq, Hkv, page, lens, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = max(1, -(-max(lens) // page)) + 1
    table, pages = tables(n_seq, width, 2, seed)
    cache = empty_cache(pages, Hkv, page, seed)
    table = table.cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    k, v = ((torch.randn((Hkv, sum(lens), 128), generator=g, device="cuda") * spread
             * (torch.rand((Hkv, sum(lens), 1), generator=g, device="cuda") * 2 + 0.2)).bfloat16() for _ in range(2))
    ajvp.attn_jvp_cache_append(k, v, *cache, table, torch.zeros(n_seq, dtype=torch.int32, device="cuda"), cu)
    return cache, table, g


ATTN = [  # H, Hkv, n, page, lens, cap, bias, tangent, causal
    (1, 1, 1, 16, [1], 0.0, False, True, True),
    (2, 2, 1, 16, [1, 16, 17, 0], 0.0, False, False, True),
    (4, 2, 1, 64, [1000, 63, 130], 30.0, True, True, True),
    (40, 8, 1, 64, [3000, 5], 50.0, False, True, True),
    (3, 1, 7, 32, [500, 4, 64], 0.0, True, True, True),
    (7, 1, 5, 48, [777, 48], 20.0, True, False, True),
    (2, 1, 20, 128, [300, 1500], 0.0, False, True, False),
    (12, 12, 1, 16, [9000], 0.0, False, False, True),
    (16, 1, 3, 16, [4097, 33], 0.0, True, False, False),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_attention_over_the_cache(case):
    H, Hkv, n, page, lens, cap, bias, tangent, causal = case
    cache, table, g = filled(len(lens), Hkv, page, lens, seed=sum(lens))
    q, tq = (torch.randn((len(lens), H, n, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda") if bias else None
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, to, lse = ajvp.attn_jvp_fwd_cache(q, tq if tangent else None, *cache, table, lens_d, softcap=cap, slopes=slopes,
                                         causal=causal)
    want = ref.attention(list(q), list(tq) if tangent else None, *cache, table, lens, 128 ** -0.5, cap, slopes, causal)
    torch.cuda.synchronize()
    check_rows(o, to, lse, want)


def check_rows(o, to, lse, want):
    for b, (ro, rto, rlse, bo, bto) in enumerate(want):
        assert ((o[b].double() - ro).abs() <= bo).all(), (b, ((o[b].double() - ro).abs() / bo).max())
        if to is not None:
            assert ((to[b].double() - rto).abs() <= bto).all(), (b, ((to[b].double() - rto).abs() / bto).max())
        rlse = rlse.cuda()
        empty = torch.isinf(rlse)
        assert torch.equal(torch.isinf(lse[b]), empty)
        # fp32 scores of 128 products (2^-17 absolute here), the cap's tanh c 2^-21
        tol = 2.0 ** -15 * (1.0 + rlse[~empty].abs())
        assert ((lse[b][~empty].double() - rlse[~empty]).abs() <= tol).all()


LONG = [  # as ATTN; spread over the GPU through a workspace
    (1, 1, 1, 64, [32760], 30.0, True, True, True),
    (10, 2, 3, 32, [32000, 77, 0], 0.0, True, True, True),
    (16, 1, 1, 48, [30001, 4], 20.0, False, False, False),
    (40, 8, 1, 64, [17001], 0.0, False, True, True),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_long_contexts_through_a_workspace(case):
    H, Hkv, n, page, lens, cap, bias, tangent, causal = case
    cache, table, g = filled(len(lens), Hkv, page, lens, seed=sum(lens))
    q, tq = (torch.randn((len(lens), H, n, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda") if bias else None
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    size = ajvp.fwd_cache_workspace_bytes(len(lens), H, Hkv, n, page, table.shape[1], tangent)
    assert size > 0
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
    kw = dict(softcap=cap, slopes=slopes, causal=causal)
    call = lambda w: ajvp.attn_jvp_fwd_cache(q, tq if tangent else None, *cache, table, lens_d, workspace=w, **kw)  # noqa: E731
    want = ref.attention(list(q), list(tq) if tangent else None, *cache, table, lens, 128 ** -0.5, cap, slopes, causal)
    first = call(ws)
    torch.cuda.synchronize()
    assert (ws[size:] == 255).all()  # nothing behind it is written
    check_rows(*first, want)
    check_rows(*call(ws[: size // 2 // 256 * 256]), want)  # too small to be of use
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        again = call(None)
    for _ in range(3):
        for x in again:
            if x is not None:
                x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(x is y is None or torch.equal(x, y) for x, y in zip(first, again))


def test_pages_that_do_not_exist_and_ends_inside_tiles():
    """Pages outside the cache are neither written nor seen; their tokens count as hidden."""
    lens, page, Hkv, H = [200, 70], 16, 2, 4
    cache, table, g = filled(2, Hkv, page, lens, seed=31)
    n_pages = cache[0].shape[0]
    table[0, 3], table[0, 7], table[1, 4] = -1, n_pages, 2 ** 31 - 1
    q, tq = (torch.randn((2, H, 2, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, to, lse = ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, lens_d)
    want = ref.attention(list(q), list(tq), *cache, table.cpu().cuda(), lens, 128 ** -0.5)
    for b, (ro, rto, rlse, bo, bto) in enumerate(want):
        assert ((o[b].double() - ro).abs() <= bo).all() and ((to[b].double() - rto).abs() <= bto).all()
    before = [t.clone() for t in cache]
    bad = torch.full_like(table, -5)
    k = torch.randn((Hkv, 40, 128), generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, 40, 40], dtype=torch.int32, device="cuda")
    ajvp.attn_jvp_cache_append(k, k, *cache, bad, lens_d, cu)
    # past the table's capacity too
    ajvp.attn_jvp_cache_append(k, k, *cache, table, torch.full_like(lens_d, table.shape[1] * page), cu)
    torch.cuda.synchronize()
    for a, b in zip(before, cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_rows_behind_the_last_sequence_stay_as_they_were():
    Hkv, H, page, total = 1, 2, 16, 20
    cache, table, g = filled(2, Hkv, page, [30, 9], seed=32)
    cu = torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda")  # rows 12 .. 19 belong to nobody
    lens = torch.tensor([30, 9], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((Hkv, total, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    q, tq = (torch.randn((H, total, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    cos, sin = angles(64)
    out = [torch.full_like(q, 3.0) for _ in range(2)]
    wide = torch.cat([table, torch.arange(2, device="cuda", dtype=torch.int32)[:, None] + int(table.max()) + 1], 1)
    cache = [torch.cat([t, t[:4]], 0) if t.dim() == 2 else torch.cat([t.view(torch.uint8), t.view(torch.uint8)[:4]], 0)
             .view(t.dtype) for t in cache]
    ajvp.attn_jvp_cache_append(k, v, *cache, wide, lens, cu, q=q, tq=tq, cos=cos, sin=sin, q_out=out[0], tq_out=out[1])
    lens = lens + (cu[1:] - cu[:-1])
    o, to = torch.full_like(q, 5.0), torch.full_like(q, 5.0)
    lse = torch.full((H, total), 5.0, device="cuda")
    ajvp.attn_jvp_fwd_cache(out[0], out[1], *cache, wide, lens, cu_seqlens=cu, max_seqlen=7, o=o, to=to, lse=lse)
    torch.cuda.synchronize()
    assert all((t[:, 12:] == 3.0).all() for t in out) and all((t[:, 12:] == 5.0).all() for t in (o, to, lse))
    rows = [(0, 5), (5, 12)]
    want = ref.attention([out[0][:, a:b] for a, b in rows], [out[1][:, a:b] for a, b in rows], *cache, wide,
                         lens.tolist(), 128 ** -0.5)
    for (a, b), (ro, rto, rlse, bo, bto) in zip(rows, want):
        assert ((o[:, a:b].double() - ro).abs() <= bo).all() and ((to[:, a:b].double() - rto).abs() <= bto).all()
        assert ((lse[:, a:b].double() - rlse).abs() <= 2.0 ** -15 * (1.0 + rlse.abs())).all()


def test_append_then_attend_like_dense_attention():
    """Chunks joining two caches over several steps, attended after each: the same as scored attention
    over the values that the cache stands for."""
    H, Hkv, page, chunk, steps = 4, 2, 32, 48, 4
    table, pages = tables(2, -(-chunk * steps // page), 1, 33)
    cache, table = empty_cache(pages, Hkv, page, 33), table.cuda()
    g = torch.Generator(device="cuda").manual_seed(33)
    cos, sin = angles(chunk * steps)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, chunk, 2 * chunk], dtype=torch.int32, device="cuda")
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
    for step in range(steps):
        k, v = (torch.randn((Hkv, 2 * chunk, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
        q, tq = (torch.randn((H, 2 * chunk, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
        q, tq = ajvp.attn_jvp_cache_append(k, v, *cache, table, lens, cu, q=q, tq=tq, cos=cos, sin=sin, interleaved=True)
        lens += chunk
        n = (step + 1) * chunk
        packed = ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, lens, cu_seqlens=cu, max_seqlen=chunk, softcap=30.0,
                                         slopes=slopes)
        # the same rows as a strided [n_seq, H, n, d] view
        view = [t.view(H, 2, chunk, 128).transpose(0, 1) for t in (q, tq)]
        dense = ajvp.attn_jvp_fwd_cache(*view, *cache, table, lens, softcap=30.0, slopes=slopes)
        for a, b in zip(packed, dense):
            assert torch.equal(a.view(H, 2, chunk, *a.shape[2:]).transpose(0, 1), b)
        kd, vd = (c[table.long()].float().mul(f[table.long()][..., None, None]).transpose(1, 2).flatten(2, 3)[:, :, :n]
                  .contiguous().bfloat16() for c, f in ((cache[0], cache[2]), (cache[1], cache[3])))  # exact: 4 bits
        z = torch.zeros_like(kd)
        begin, end = ajvp.key_bounds(chunk, n, causal=True)
        o, to, lse = ajvp.attn_jvp_fwd_scored(view[0].contiguous(), kd, vd, view[1].contiguous(), z, z, softcap=30.0,
                                              slopes=slopes, key_begin=begin, key_end=end)
        # both are within the roundings of their weights (f16 and bf16) and outputs of the same values
        for a, b, times in ((dense[0], o, 3), (dense[1], to, 4)):
            assert (a.double() - b.double()).norm() <= times * ref.UB * b.double().norm()
        assert ((dense[2] - lse).abs() <= 2.0 ** -14 * (1 + lse.abs())).all()


def test_scales_far_apart_and_constant_tangents():
    """Pages whose values differ by powers of two, and a tangent whose dS hardly varies."""
    H, page, L = 2, 16, 320
    table, pages = tables(1, L // page, 0, 34)
    cache, table = empty_cache(pages, 1, page, 34), table.cuda()
    g = torch.Generator(device="cuda").manual_seed(34)
    size = 2.0 ** torch.randint(-12, 13, (1, L // page, 1, 1), generator=g, device="cuda").float()
    k = (torch.randn((1, L // page, page, 128), generator=g, device="cuda") * size * 0.02).view(1, L, 128).bfloat16()
    size = 2.0 ** torch.randint(-20, 21, (1, L // page, 1, 1), generator=g, device="cuda").float()
    v = (torch.randn((1, L // page, page, 128), generator=g, device="cuda") * size).view(1, L, 128).bfloat16()
    zero, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, L], dtype=torch.int32, device="cuda")
    ajvp.attn_jvp_cache_append(k, v, *cache, table, zero, cu)
    q, tq = (torch.randn((1, H, 1, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    for t in (tq, q):  # (tq = q: dS follows S)
        o, to, lse = ajvp.attn_jvp_fwd_cache(q, t, *cache, table, lens)
        ro, rto, rlse, bo, bto = ref.attention(list(q), list(t), *cache, table, [L], 128 ** -0.5)[0]
        assert ((o[0].double() - ro).abs() <= bo).all() and ((to[0].double() - rto).abs() <= bto).all()
        # scores reach some hundreds here, fp32 sums of products up to as much
        assert ((lse[0].double() - rlse).abs() <= 2.0 ** -15 * (1.0 + rlse.abs())).all()


def test_one_key_has_no_tangent():
    cache, table, g = filled(3, 2, 16, [1, 1, 1], seed=35)
    q, tq = (torch.randn((3, 4, 1, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    o, to, _ = ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, torch.ones(3, dtype=torch.int32, device="cuda"))
    # P = 1: tO is zero but for fp32 roundings of dS - r, some 2^-23 of |dS| |V|
    assert (to.abs() <= 2.0 ** -18 * 60.0 * o.abs().amax()).all()


def test_codes_past_32_bit_offsets():
    """The last pages of a cache of more than 2^31 bytes of codes."""
    page, Hkv, pages = 64, 1, (1 << 31) // (64 * 128) + 3
    if torch.cuda.get_device_properties(0).total_memory < 3 * (1 << 32):
        pytest.skip("needs 5 GB")
    k8, v8 = (torch.empty((pages, Hkv, page, 128), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, Hkv), device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(36)
    k, v = (torch.randn((1, 150, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    zero, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    ajvp.attn_jvp_cache_append(k, v, k8, v8, ks, vs, table, zero, cu)
    q, tq = (torch.randn((1, 2, 1, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    o, to, _ = ajvp.attn_jvp_fwd_cache(q, tq, k8, v8, ks, vs, table, torch.tensor([150], dtype=torch.int32, device="cuda"))
    at = table[0].long()
    ro, rto, _, bo, bto = ref.attention(list(q), list(tq), k8[at], v8[at], ks[at], vs[at],
                                        torch.arange(3, device="cuda")[None], [150], 128 ** -0.5)[0]
    assert ((o[0].double() - ro).abs() <= bo).all() and ((to[0].double() - rto).abs() <= bto).all()


def test_decoding_in_a_graph():
    """One captured step (append, attend, lengthen), replayed: the same as eager steps on a copy."""
    H, Hkv, page, steps = 4, 2, 16, 40
    table, pages = tables(2, 5, 0, 37)
    table = table.cuda()
    g = torch.Generator(device="cuda").manual_seed(37)
    cos, sin = angles(80)
    lens = [torch.tensor([7, 20], dtype=torch.int32, device="cuda") for _ in range(2)]
    caches = [[torch.zeros((pages, Hkv, page, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
               for _ in range(2)] + [torch.full((pages, Hkv), 2.0 ** -8, device="cuda") for _ in range(2)] for _ in range(2)]
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    new = [torch.empty((h, 2, 128), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, H, H)]

    def step(cache, n):
        q, tq = ajvp.attn_jvp_cache_append(new[0], new[1], *cache, table, n, cu, q=new[2], tq=new[3], cos=cos, sin=sin)
        n += 1
        return ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, n, cu_seqlens=cu, max_seqlen=1)

    def feed(i):
        for t in new:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda") * (1.0 + 0.2 * i))

    feed(0)
    step(caches[0], lens[0])
    step(caches[1], lens[1])
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    keep = [t.clone() for t in caches[0]], lens[0].clone()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        out = step(caches[0], lens[0])
    for a, b in zip(caches[0], keep[0]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # (capturing runs nothing)
    for i in range(1, steps):
        feed(i)
        graph.replay()
        want = step(caches[1], lens[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
    for a, b in zip(*caches):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert ajvp.check_device_status() == ajvp.AJVP_OK


def test_two_streams_share_a_cache():
    cache, table, g = filled(4, 2, 64, [900, 50, 1300, 2], seed=38)
    lens = torch.tensor([900, 50, 1300, 2], dtype=torch.int32, device="cuda")
    q, tq = (torch.randn((4, 6, 3, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    first = ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[ajvp.attn_jvp_fwd_cache(q, tq, *cache, table, lens, stream=s) for s in streams] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for out in pair:
            assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_queries_rotated_in_place():
    H, Hkv, page = 6, 2, 16
    g = torch.Generator(device="cuda").manual_seed(31)
    cos, sin = angles(64)
    table, pages = tables(3, 4, 1, seed=3)
    cu = torch.tensor([0, 20, 20, 27], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 9, 30], dtype=torch.int32, device="cuda")
    q, tq = (torch.randn((H, 30, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((Hkv, 30, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    for inter in (False, True):
        two = []
        for place in (False, True):
            cache = empty_cache(pages, Hkv, page, seed=2)
            for t in cache[2:]:
                t.fill_(1.0)
            a, b = q.clone(), tq.clone()
            kw = dict(q_out=a, tq_out=b) if place else dict(q_out=q.clone(), tq_out=tq.clone())
            two.append(ajvp.attn_jvp_cache_append(k, v, *cache, table.cuda(), lens, cu, q=a, tq=b, cos=cos, sin=sin,
                                                  interleaved=inter, **kw))
        assert all(torch.equal(x, y) for x, y in zip(*two))
        assert torch.equal(two[1][0][:, 27:], q[:, 27:])  # behind the last sequence


def test_tangents_of_other_strides_and_a_generous_max_seqlen():
    """One token per sequence: strides of axes of one element do not matter.  The
    most tokens of a sequence may be overestimated past all rows."""
    lens = [40, 7, 100]
    cache, table, g = filled(3, 2, 16, lens, seed=5)
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, tq = (torch.randn((3, 1, 4, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    want = ajvp.attn_jvp_fwd_cache(q.transpose(1, 2).contiguous(), tq.transpose(1, 2).contiguous(), *cache, table, lens_d)
    got = ajvp.attn_jvp_fwd_cache(q.transpose(1, 2), tq.transpose(1, 2).contiguous(), *cache, table, lens_d)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    rows = [x.squeeze(1).transpose(0, 1).contiguous() for x in (q, tq)]  # [H, total, 128]
    packed = ajvp.attn_jvp_fwd_cache(*rows, *cache, table, lens_d, cu_seqlens=cu, max_seqlen=64)
    for x, y in zip(packed[:2], want[:2]):
        assert torch.equal(x, y.squeeze(2).transpose(0, 1))
