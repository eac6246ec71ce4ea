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


def run(inp, cot, kw, **more):
    x = [inp[n] for n in NAMES]
    out = ajvp.attn_jvp_fwd_scored_stats(*x, **kw)
    return out, ajvp.attn_jvp_bwd_scored(*x, *out, cot["dout"], cot["dtout"], **kw, **more)


def against_reference(inp, cot, kw, out, g, scale=128 ** -0.5):
    B = inp["q"].shape[0]
    x = [inp[n] for n in NAMES]
    (ro, rto, rlse, _), (eo, eto) = ref.forward(*x, scale, bounds=True, **ref_opts(kw, B))
    ref.check("o", out[0], ro, eo)
    ref.check("to", out[1], rto, eto)
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isinf(out[2]), empty)
    assert ((out[2] - rlse)[~empty].abs() <= 2.0 ** -15 * (1.0 + rlse[~empty].abs())).all()
    rg, eg = ref.backward(*x, cot["dout"], cot["dtout"], scale, bounds=True, **ref_opts(kw, B))
    for n in ajvp.GRAD_NAMES:
        ref.check(n, g[n], rg[n], eg[n])
    assert ajvp.check_device_status() == ajvp.AJVP_OK


@pytest.mark.parametrize("kw,scale,std", [
    (dict(softcap=0.5), 128 ** -0.5, 1.0),       # scores far past the cap: the exponential's tanh
    (dict(softcap=200.0), 128 ** -0.5, 1.0),     # a cap too wide for a fixed reference
    (dict(softcap=200.0, bias=1.0), 128 ** -0.5, 1.0),
    (dict(softcap=30.0), -(128 ** -0.5), 1.0),   # negative and zero scales
    (dict(bias=1.0), -(128 ** -0.5), 1.0),
    (dict(bias=1.0), 0.0, 1.0),
    (dict(softcap=30.0), 0.0, 1.0),
    (dict(), 0.0, 1.0),
    (dict(bias=40.0), 128 ** -0.5, 1.0),         # slopes too steep for separate maxima
    (dict(bias=-0.01), 128 ** -0.5, 1.0),        # a bias that grows with distance
    (dict(softcap=30.0, bias=-0.01), 128 ** -0.5, 1.0),
    (dict(softcap=50.0, bias=1.0), 128 ** -0.5, 3.0),  # peaked rows
], ids=str)
def test_score_ranges(kw, scale, std):
    B, H, L = 1, 2, 300
    inp, cot = make(B, H, 1, L, L, seed=11, std=std)
    kw = dict(kw)
    if "bias" in kw:
        kw["slopes"] = slopes_of(H) * kw.pop("bias")
    kw.update(masks("random", B, L, L, seed=4))
    x = [inp[n] for n in NAMES]
    out = ajvp.attn_jvp_fwd_scored_stats(*x, scale=scale, **kw)
    g = ajvp.attn_jvp_bwd_scored(*x, *out, cot["dout"], cot["dtout"], scale=scale, **kw)
    against_reference(inp, cot, kw, out, g, scale)


def test_largest_bias_may_be_far():
    """Rows whose visible keys all lie far from them: the bias of the nearest is the reference."""
    B, H, L = 1, 2, 700
    inp, cot = make(B, H, H, L, L, seed=12)
    begin = torch.zeros(L, dtype=torch.int32, device="cuda")
    end = torch.full((L,), 20, dtype=torch.int32, device="cuda")
    for cap in (0.0, 30.0):
        kw = dict(softcap=cap, slopes=slopes_of(H) * 2.0, key_begin=begin, key_end=end)
        out, g = run(inp, cot, kw)
        assert torch.isfinite(out[2]).all()
        # fp32 biases of some 700 x 1 hold 2^-14 of themselves: scores, and so weights, 2^-14 x 1000 off
        (ro, rto, rlse, _), (eo, eto) = ref.forward(*(inp[n] for n in NAMES), 128 ** -0.5, bounds=True, **ref_opts(kw, B))
        ref.check("o", out[0], ro, eo + 2.0 ** -10)
        ref.check("to", out[1], rto, eto + 2.0 ** -8)
        # biases reach 87 (126 in log2 units): each fp32 step on them rounds by up to 2^-24 x 126 < 2^-17,
        # as do the sums of 128 products; where a score cancels its bias that stays, so the bound is absolute there
        assert ((out[2] - rlse).abs() <= 2.0 ** -15 * (1.0 + rlse.abs())).all()


def test_one_bound_alone_and_per_batch_bounds():
    B, H, L = 3, 2, 150
    inp, cot = make(B, H, H, L, L, seed=13)
    begin, end = random_bounds(B, L, L, 3)
    for kw in (dict(key_begin=begin), dict(key_end=end), dict(key_begin=begin, key_end=end)):
        out, g = run(inp, cot, kw)
        against_reference(inp, cot, kw, out, g)


def test_plain_options_match_the_unmasked_and_causal_entries():
    inp, _ = make(2, 2, 2, 300, 260, seed=14)
    x = [inp[n] for n in NAMES]
    a, b = ajvp.attn_jvp_fwd_scored(*x), ajvp.attn_jvp_fwd(*x)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    bounds = dict(zip(("key_begin", "key_end"), ajvp.key_bounds(300, 260, causal=True)))
    a, b = ajvp.attn_jvp_fwd_scored(*x, **bounds), ajvp.attn_jvp_fwd_causal(*x)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_split_and_unsplit_key_sides():
    """A small workspace runs the key side unsplit; both agree with the definition, and each with itself."""
    inp, cot = make(1, 4, 2, 1500, 70, seed=15)
    x = [inp[n] for n in NAMES]
    kw = dict(softcap=20.0, slopes=slopes_of(4))
    full = ajvp.bwd_scored_workspace_bytes(1, 4, 2, 1500, 70)
    least = (16 * (4 * 1500 + 64) + 255) // 256 * 256 + 256
    assert full > least  # (this shape splits)
    out = ajvp.attn_jvp_fwd_scored_stats(*x, **kw)
    got = []
    for size in (full, least, full, least):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaN bits: nothing is read before it is written
        got.append(ajvp.attn_jvp_bwd_scored(*x, *out, cot["dout"], cot["dtout"], workspace=ws, **kw))
        against_reference(inp, cot, kw, out, got[-1])
    for n in ajvp.GRAD_NAMES:
        assert torch.equal(got[0][n], got[2][n]) and torch.equal(got[1][n], got[3][n])


def test_autograd_of_shared_heads():
    B, H, Hkv, L = 1, 6, 2, 200
    inp, cot = make(B, H, Hkv, L, L, seed=16)
    begin, end = ajvp.key_bounds(L, causal=True, prefix=30)
    kw = dict(softcap=25.0, slopes=slopes_of(H), key_begin=begin, key_end=end)
    leaves = {n: inp[n].clone().requires_grad_(True) for n in NAMES}
    o, to = ajvp.attn_jvp_autograd(*(leaves[n] for n in NAMES), **kw)
    ((o.float() * cot["dout"].float()).sum() + (to.float() * cot["dtout"].float()).sum()).backward()
    _, g = run(inp, cot, kw)
    for n, gn in zip(NAMES, ("dq", "dk", "dv", "dtq", "dtk", "dtv")):
        assert torch.equal(leaves[n].grad, g[gn]), n
    # a cap alone, causal by its own argument, one output unused
    leaves = {n: inp[n].clone().requires_grad_(True) for n in NAMES}
    o, _ = ajvp.attn_jvp_autograd(*(leaves[n] for n in NAMES), softcap=25.0, causal=True)
    (o.float() * cot["dout"].float()).sum().backward()
    rg, eg = ref.backward(*(inp[n] for n in NAMES), cot["dout"], torch.zeros_like(cot["dtout"]), 128 ** -0.5, bounds=True,
                          softcap=25.0, end=ajvp.key_bounds(L, causal=True)[1].expand(B, -1))
    for n, gn in zip(NAMES, ("dq", "dk", "dv", "dtq", "dtk", "dtv")):
        ref.check(gn, leaves[n].grad, rg[gn], eg[gn])


def test_in_a_graph_beside_an_eager_call_on_another_stream():
    inp, cot = make(1, 4, 2, 400, 90, seed=17)
    x = [inp[n] for n in NAMES]
    begin, end = ajvp.key_bounds(400, 90, causal=True, prefix=40)
    kw = dict(softcap=30.0, slopes=slopes_of(4), key_begin=begin.expand(1, -1).contiguous(),
              key_end=end.expand(1, -1).contiguous())
    run(inp, cot, kw)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        out, g = run(inp, cot, kw)
    for seed in (18, 19):
        new, _ = make(1, 4, 2, 400, 90, seed=seed)
        for n in NAMES:
            inp[n].copy_(new[n])
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            out2, g2 = run(inp, cot, kw)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, out2))
        assert all(torch.equal(g[n], g2[n]) for n in g)
    # an explicit stream: what the call allocates belongs to that stream
    out3 = ajvp.attn_jvp_fwd_scored_stats(*x, stream=other, **kw)
    g3 = ajvp.attn_jvp_bwd_scored(*x, *out3, cot["dout"], cot["dtout"], stream=other.cuda_stream, **kw)
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out3, out2)) and all(torch.equal(g3[n], g2[n]) for n in g3)


def test_no_query_rows_give_zero_key_gradients():
    inp, cot = make(1, 2, 1, 4, 50, seed=20)
    e = {n: inp[n][:, :, :0].contiguous() for n in ("q", "tq")}
    z = torch.zeros((1, 2, 0), device="cuda")
    g = ajvp.attn_jvp_bwd_scored(e["q"], inp["k"], inp["v"], e["tq"], inp["tk"], inp["tv"], e["q"], e["q"], z, z, e["q"],
                                 e["q"])
    assert g["dq"].shape[2] == 0 and all((g[n] == 0).all() for n in ("dk", "dv", "dtk", "dtv"))


def test_rows_at_the_end_are_written_alone():
    """Outputs inside a larger buffer: nothing behind them changes."""
    inp, cot = make(1, 1, 1, 70, 70, seed=21)
    x = [inp[n] for n in NAMES]
    big = torch.full((2, 70 * 128 + 640), 7.0, dtype=torch.bfloat16, device="cuda")
    o, to = (t[: 70 * 128].view(1, 1, 70, 128) for t in big)
    ajvp.attn_jvp_fwd_scored(*x, o=o, to=to, softcap=20.0)
    torch.cuda.synchronize()
    assert (big[:, 70 * 128:] == 7.0).all()


@pytest.mark.parametrize("shape", [(1, 12, 4, 4100, 4100), (2, 3, 3, 2049, 515)])
def test_larger_shapes_by_the_norm(shape):
    """Relative 2-norm errors of larger calls: roundings of weights, gradients and outputs are
    independent, at most two of them per output here, each at most U and U / sqrt(3) in the mean."""
    B, H, Hkv, Lq, Lk = shape
    inp, cot = make(B, H, Hkv, Lq, Lk, seed=22)
    kw = dict(softcap=30.0, slopes=slopes_of(H), **masks("prefix", B, Lq, Lk, 0))
    out, g = run(inp, cot, kw)
    x = [inp[n] for n in NAMES]
    for h in range(0, H, max(1, H // Hkv)):  # group by group: 64-bit scores of all heads would not fit
        hs, hk = slice(h, h + H // Hkv), slice(h * Hkv // H, h * Hkv // H + 1)
        part = [x[0][:, hs], x[1][:, hk], x[2][:, hk], x[3][:, hs], x[4][:, hk], x[5][:, hk]]
        opt = ref_opts(dict(kw, slopes=kw["slopes"][hs]), B)
        ro, rto, _, _ = ref.forward(*part, 128 ** -0.5, **opt)
        rg = ref.backward(*part, cot["dout"][:, hs], cot["dtout"][:, hs], 128 ** -0.5, **opt)
        pairs = [(out[0][:, hs], ro), (out[1][:, hs], rto)]
        pairs += [(g[n][:, hs if n in ("dq", "dtq") else hk], rg[n]) for n in rg]
        for got, want in pairs:
            assert (got.double() - want).norm() <= ref.U * want.norm()


def test_more_sequences_than_a_grid_is_high():
    """70000 sequences of three rows and three keys, a bound each: as the same rows in batches of 7000."""
    B, n = 70000, 3
    inp, cot = make(B, 1, 1, n, n, seed=23)
    g = torch.Generator().manual_seed(24)
    end = torch.randint(0, n + 1, (B, n), generator=g).int().cuda()
    out, grads = run(inp, cot, dict(softcap=10.0, key_end=end))
    for b in range(0, B, 7000):
        s = slice(b, b + 7000)
        part = [{k: x[s].contiguous() for k, x in d.items()} for d in (inp, cot)]
        o2, g2 = run(*part, dict(softcap=10.0, key_end=end[s].contiguous()))
        assert all(torch.equal(x[s], y) for x, y in zip(out, o2))
        assert all(torch.equal(grads[k][s], g2[k]) for k in grads)


def test_second_derivatives_are_refused():
    inp, _ = make(1, 2, 1, 20, 20, seed=25)
    x = [inp[k].requires_grad_() for k in NAMES]
    o, to = ajvp.attn_jvp_autograd(*x, softcap=20.0)
    (dq,) = torch.autograd.grad((o.float().square() + to.float()).sum(), x[:1], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dq.float().sum().backward()


@pytest.mark.parametrize("opt", [{}, dict(softcap=30.0), dict(bias=True), dict(softcap=30.0, bias=True),
                                 dict(softcap=200.0, bias=True)], ids=lambda o: "-".join(o) + str(o.get("softcap", "")))
def test_many_units_of_different_lengths(opt):
    """40 sequences of 4 row tiles and 4 heads, every tile with an interval of its own of 0 to 9 key tiles (some
    without any): bit for bit as each sequence alone, whose few tiles are a CTA each."""
    B, H, Lq, Lk = 40, 4, 500, 555
    inp, _ = make(B, H, 2, Lq, Lk, seed=26)
    g = torch.Generator().manual_seed(27)
    begin = torch.randint(0, Lk, (B, 4), generator=g)
    length = torch.randint(0, 4, (B, 4), generator=g) * torch.randint(0, 190, (B, 4), generator=g)
    rows = lambda x: x.repeat_interleave(128, 1)[:, :Lq].int().contiguous().cuda()  # noqa: E731
    kw = dict(key_begin=rows(begin), key_end=rows(begin + length))
    if "softcap" in opt:
        kw["softcap"] = opt["softcap"]
    if "bias" in opt:
        kw["slopes"] = slopes_of(H)
    x = [inp[n] for n in NAMES]
    for _ in range(3):
        out = ajvp.attn_jvp_fwd_scored_stats(*x, **kw)
        for b in range(B):
            s = slice(b, b + 1)
            alone = ajvp.attn_jvp_fwd_scored_stats(*(t[s] for t in x), **{n: v[s] if n.startswith("key") else v
                                                                          for n, v in kw.items()})
            assert all(torch.equal(y[s], z) for y, z in zip(out, alone))
    assert ajvp.check_device_status() == ajvp.AJVP_OK


def test_outputs_allocated_either_way(monkeypatch):
    """The allocation without argument parsing is torch's own business; without it the results are the same."""
    from attention_forward_mode_b200 import _scored
    inp, cot = make(2, 4, 2, 65, 90, seed=28)
    kw = dict(softcap=20.0, key_end=torch.randint(0, 91, (2, 65), dtype=torch.int32, device="cuda"))
    out, g = run(inp, cot, kw)
    monkeypatch.setattr(_scored, "_empty_strided_cuda", None)
    out2, g2 = run(inp, cot, kw)
    for a, b in list(zip(out, out2)) + [(g[n], g2[n]) for n in g]:
        assert a.stride() == b.stride() and a.dtype == b.dtype and torch.equal(a, b)


def test_a_wait_bound_shorter_than_a_unit():
    """The bound is on single waits: a row tile of 1094 key tiles takes some 1.4 ms in all."""
    inp, _ = make(1, 2, 1, 100, 70000, seed=29)
    x = [inp[n] for n in NAMES]
    want = ajvp.attn_jvp_fwd_scored(*x, softcap=30.0)
    torch.cuda.synchronize()
    ajvp.set_wait_bound_ns(300_000)
    try:
        got = ajvp.attn_jvp_fwd_scored(*x, softcap=30.0)
        torch.cuda.synchronize()
    finally:
        ajvp.set_wait_bound_ns(0)
    assert ajvp.check_device_status() == ajvp.AJVP_OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))
