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
    for b, (ro, rto, rlse, bo, bto) in enumerate(want):
        assert ((o[b].double() - ro).abs() <= bo).all(), (b, ((o[b].double() - ro).abs() / bo).max())
        if tangent:
            assert ((to[b].double() - rto).abs() <= bto).all(), (b, ((to[b].double() - rto).abs() / bto).max())
        rlse = rlse.cuda()
        empty = torch.isinf(rlse)
        assert torch.equal(torch.isinf(lse[b]), empty)
        # fp32 scores of 128 products (2^-17 absolute here), the cap's tanh c 2^-21
        tol = 2.0 ** -15 * (1.0 + rlse[~empty].abs())
        assert ((lse[b][~empty].double() - rlse[~empty]).abs() <= tol).all()
