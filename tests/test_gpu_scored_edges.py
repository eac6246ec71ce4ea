"""Scored attention + JVP where it could go wrong quietly: padding that is not
finite, biases of far keys, masks made inside a captured graph, launches of
very many heads."""
import pytest
import torch

import attention_forward_mode_b200 as ajvp
import scored_reference as ref
from test_gpu_scored import NAMES, against_reference, make, ref_opts, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0), dict(softcap=200.0), dict(bias=1.0), dict(bias=40.0),
                                dict(softcap=30.0, bias=1.0), dict(softcap=200.0, bias=1.0)], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
def test_padding_rows_that_are_not_finite(kw, bad):
    """Rows that see nothing give zeros whatever their q and tq hold, also inside a tile of live rows.  The other
    rows are the definition's."""
    kw = dict(kw)
    if "bias" in kw:
        kw["slopes"] = slopes_of(4) * kw.pop("bias")
    inp, _ = make(1, 4, 2, 300, 300, seed=31)
    begin, end = ajvp.key_bounds(300, documents=[0, 40, 170, 233])  # rows 233 .. 299 are padding
    begin[50:60], end[50:60] = 90, 90  # and ten rows inside a document see nothing
    dead = end <= begin
    x = {n: t.clone() for n, t in inp.items()}
    x["q"][:, :, dead], x["tq"][:, :, dead] = bad, -bad
    o = ajvp.attn_jvp_fwd_scored_stats(*(x[n] for n in NAMES), key_begin=begin, key_end=end, **kw)
    (ro, rto, rlse, _), (eo, eto) = ref.forward(*(inp[n] for n in NAMES), 128 ** -0.5, bounds=True,
                                                **ref_opts(dict(kw, key_begin=begin, key_end=end), 1))
    ref.check("o", o[0], ro, eo)
    ref.check("to", o[1], rto, eto)
    live = ~dead
    assert ((o[2] - rlse)[:, :, live].abs() <= 2.0 ** -15 * (1.0 + rlse[:, :, live].abs())).all()
    assert torch.isfinite(o[3]).all()
    assert (o[0][:, :, dead] == 0).all() and (o[1][:, :, dead] == 0).all() and (o[3][:, :, dead] == 0).all()
    assert (o[2][:, :, dead] == -float("inf")).all()


def test_a_causal_mask_made_inside_a_captured_graph():
    """attn_jvp_autograd turns causal into bounds on the device alone: nothing is copied from the host."""
    inp, _ = make(1, 4, 2, 150, 200, seed=32)
    x = [inp[n] for n in NAMES]
    call = lambda: (*ajvp.attn_jvp_autograd(*x, softcap=20.0, causal=True),  # noqa: E731
                    *ajvp.key_bounds(150, 200, causal=True, prefix=9), *ajvp.key_bounds(150, frame=40),
                    *ajvp.key_bounds(150, causal=True, window=31))
    want = call()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        got = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_far_keys_under_a_bias_and_their_gradients(cap):
    """Rows that see only the first 20 of 700 keys: biases of up to 87 (126 in log2 units), whose fp32 roundings
    of some 2^-17 stay below those of the bf16 weights, 2^-9."""
    B, H, L = 1, 2, 700
    inp, cot = make(B, H, 1, L, L, seed=33)
    end = torch.full((L,), 20, dtype=torch.int32, device="cuda")
    kw = dict(softcap=cap, slopes=slopes_of(H) * 2.0, key_end=end)
    x = [inp[n] for n in NAMES]
    out = ajvp.attn_jvp_fwd_scored_stats(*x, **kw)
    g = ajvp.attn_jvp_bwd_scored(*x, *out, cot["dout"], cot["dtout"], **kw)
    against_reference(inp, cot, kw, out, g)


@pytest.mark.parametrize("H,B,Lq", [(65536, 1, 1), (32768, 2, 130)])
def test_very_many_heads_of_one_key(H, B, Lq):
    """H query heads share one key head and key, so that O = V; tO = tV and the log-sum-exp is the score."""
    g = torch.Generator(device="cuda").manual_seed(34)
    q, tq = (torch.randn((B, H, Lq, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v, tk, tv = (torch.randn((B, 1, 1, 128), generator=g, device="cuda").bfloat16() for _ in range(4))
    o, to, lse, mu = ajvp.attn_jvp_fwd_scored_stats(q, k, v, tq, tk, tv)
    torch.cuda.synchronize()
    assert ajvp.check_device_status() == ajvp.AJVP_OK
    assert torch.equal(o, v.expand_as(o))
    s = (q.float() * k.float()).sum(-1) * 128 ** -0.5
    assert ((lse - s).abs() <= 2.0 ** -15 * (1 + s.abs())).all()
    # tO = tV + (p dS - mu) V, with p dS = mu rounded once to bf16 as a product's operand (half a step, 2^-8 mu)
    # and the sum rounded once as an output
    err = (to.float() - tv.float()).abs()
    bound = 2.0 ** -8 * (tv.float().abs() + mu.abs()[..., None] * v.float().abs())
    assert (err <= 1.01 * bound).all()


@pytest.mark.parametrize("unit", [0, 1, 2])
def test_every_status_word_reports_a_wait_that_ran_out(unit):
    """The unmodified, the scored and the cache's kernels each set a word of their own: reported once, then clear."""
    assert ajvp.check_device_status() == ajvp.AJVP_OK
    ajvp.selftest_wait_timeout(1_000_000, unit=unit)
    assert ajvp.check_device_status() == ajvp.AJVP_ERR_TIMEOUT
    assert ajvp.check_device_status() == ajvp.AJVP_OK
    with pytest.raises(ajvp.AttnJvpError):
        ajvp.selftest_wait_timeout(1_000_000, unit=3)


def test_no_query_heads_give_zero_key_gradients():
    """H = 0 is a multiple of every Hkv: the keys' gradients are sums over nothing."""
    inp, _ = make(1, 2, 2, 4, 50, seed=35)
    e, z = torch.empty((1, 0, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 0, 4), device="cuda")
    full = {n: torch.full_like(inp["k"], 3.0) for n in ("dk", "dv", "dtk", "dtv")}
    g = ajvp.attn_jvp_bwd_scored(e, inp["k"], inp["v"], e, inp["tk"], inp["tv"], e, e, z, z, e, e, grads=full)
    assert g["dq"].shape == e.shape and all((g[n] == 0).all() for n in full)
    o, to, lse = ajvp.attn_jvp_fwd_scored(e, inp["k"], inp["v"], e, inp["tk"], inp["tv"])
    assert o.shape == to.shape == e.shape and lse.shape == z.shape
