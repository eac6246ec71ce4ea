"""Scored attention + JVP and the paged cache without a GPU: the references
against differences and torch, key_bounds against enumeration, refusals of the
C ABI and the binding, and Ulysses with score options over gloo."""
import ctypes
import os

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import cache_reference
import scored_reference as ref
from attention_forward_mode_b200 import _binding as B
from attention_forward_mode_b200 import attn_jvp_autograd, attn_jvp_cache_append, attn_jvp_fwd_cache
from attention_forward_mode_b200 import attn_jvp_fwd_scored, key_bounds
from attention_forward_mode_b200 import build as build_mod

NAMES = ("q", "k", "v", "tq", "tk", "tv")


def draw(Bn, H, Hkv, Lq, Lk, d, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, n: torch.randn((Bn, h, n, d), generator=g, dtype=torch.float64)  # noqa: E731
    return [r(H, Lq), r(Hkv, Lk), r(Hkv, Lk), r(H, Lq), r(Hkv, Lk), r(Hkv, Lk)], [r(H, Lq), r(H, Lq)]


OPTS = [dict(), dict(softcap=1.5), dict(softcap=0.7, slopes=torch.tensor([0.3, 0.05])),
        dict(slopes=torch.tensor([0.5, -0.2]), begin=torch.tensor([[0, 1, 2, 0, 4]]), end=torch.tensor([[3, 2, 2, 6, 5]]))]


@pytest.mark.parametrize("opt", OPTS, ids=["plain", "cap", "cap-bias", "bias-bounds"])
def test_reference_tangent_and_gradients(opt):
    x, (do, dto) = draw(1, 2, 1, 5, 6, 4, seed=3)
    s = 0.8

    def primal(q, k, v):
        z = torch.zeros_like
        return ref.forward(q, k, v, z(q), z(k), z(v), s, **opt)[0]

    o, to, lse, mu = ref.forward(*x, s, **opt)
    jo, jto = torch.func.jvp(primal, tuple(x[:3]), tuple(x[3:]))
    live = torch.isfinite(lse)
    assert torch.allclose(o, jo) and torch.allclose(to[live], jto[live])
    assert (o[~live] == 0).all() and (to[~live] == 0).all() and (mu[~live] == 0).all()

    g = ref.backward(*x, do, dto, s, **opt)

    def loss():
        o, to, _, _ = ref.forward(*x, s, **opt)
        return ((o * do).sum() + (to * dto).sum()).item()

    rng = np.random.default_rng(0)
    for n, t in zip(("dq", "dk", "dv", "dtq", "dtk", "dtv"), x):
        flat = t.view(-1)
        for i in rng.choice(flat.numel(), 6, replace=False):
            keep, e = flat[i].item(), 1e-5
            flat[i] = keep + e
            up = loss()
            flat[i] = keep - e
            down = loss()
            flat[i] = keep
            # central differences: e^2 times third derivatives, and 1e-16 |loss| / e of rounding
            assert abs((up - down) / (2 * e) - g[n].view(-1)[i].item()) < 1e-6, (n, i)


def test_key_bounds_enumerated():
    for Lq, Lk in ((7, 7), (4, 9), (9, 4)):
        for kw in (dict(), dict(causal=True), dict(causal=True, prefix=3), dict(frame=3), dict(causal=True, window=2),
                   dict(documents=[1, 3, 7]), dict(documents=[0, 2, 2, 6], causal=True, prefix=1),
                   dict(documents=[0, 4, 7], frame=2)):
            begin, end = key_bounds(Lq, Lk, device="cpu", **kw)
            assert begin.dtype == end.dtype == torch.int32
            for i in range(Lq):
                p = i + Lk - Lq
                seen = set(range(max(0, int(begin[i])), min(Lk, int(end[i]))))
                want = set()
                cu = kw.get("documents")
                for j in range(Lk):
                    first, last = 0, Lk
                    if cu is not None:
                        own = [(a, b) for a, b in zip(cu, cu[1:]) if a <= p < b]
                        if not own or not own[0][0] <= j < own[0][1]:
                            continue
                        first, last = own[0]
                    if kw.get("causal") and j > p and j >= first + kw.get("prefix", 0):
                        continue
                    if kw.get("frame") and (p < 0 or (j - first) // kw["frame"] > (p - first) // kw["frame"]):
                        continue
                    if kw.get("window") and j < p - kw["window"] + 1:
                        continue
                    want.add(j)
                assert seen == want, (Lq, Lk, kw, i, seen, want)
    for bad in (dict(causal=True, frame=2), dict(prefix=2), dict(frame=-1), dict(documents=[3])):
        with pytest.raises(ValueError):
            key_bounds(4, 4, device="cpu", **bad)


def test_cache_reference_rounding():
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4000, generator=g) * s for s in (0.001, 0.05, 3.0, 100.0)]).clamp(-448, 448)
    assert np.array_equal(cache_reference.e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    for amax, e in ((448.0, 0), (448.1, 1), (1.75, -8), (1.7500001, -7), (0.0, -100), (1e-40, -100), (3e38, 100)):
        assert cache_reference.exponent(np.float64(amax)) == e


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def test_scored_refusals(lib):
    p = ctypes.c_void_p(256)

    def fwd(ptr=p, H=2, Hkv=2, Lq=8, Lk=8, d=128, scale=0.1, cap=0.0, lse=None, aux=None, B_=1):
        return lib.attn_jvp_fwd_scored(ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, lse, aux, aux, aux, B_, H, Hkv, Lq, Lk, d,
                                       scale, cap, None)

    assert fwd(H=3, Hkv=2) == B.AJVP_ERR_INVALID_ARG and fwd(Hkv=0) == B.AJVP_ERR_INVALID_ARG
    assert fwd(cap=-1.0) == B.AJVP_ERR_INVALID_ARG and fwd(cap=float("nan")) == B.AJVP_ERR_INVALID_ARG
    assert fwd(cap=float("inf")) == B.AJVP_ERR_INVALID_ARG and fwd(cap=1e-42) == B.AJVP_ERR_INVALID_ARG
    assert fwd(scale=float("inf")) == B.AJVP_ERR_INVALID_ARG and fwd(Lk=0) == B.AJVP_ERR_INVALID_ARG
    assert fwd(Lq=1 << 24) == B.AJVP_ERR_TOO_LARGE and fwd(Lk=1 << 24) == B.AJVP_ERR_TOO_LARGE
    assert fwd(d=64) == B.AJVP_ERR_UNSUPPORTED_DIM and fwd(ptr=ctypes.c_void_p(24)) == B.AJVP_ERR_MISALIGNED
    assert fwd(aux=ctypes.c_void_p(6)) == B.AJVP_ERR_MISALIGNED and fwd(ptr=None) == B.AJVP_ERR_INVALID_ARG
    for empty in (dict(Lq=0), dict(B_=0), dict(H=0, Hkv=0)):
        assert fwd(ptr=None, **empty) == B.AJVP_OK
    stats = lib.attn_jvp_fwd_scored_stats
    assert stats(p, p, p, p, p, p, p, p, None, p, None, None, None, 1, 2, 2, 8, 8, 128, 0.1, 0.0, None) \
        == B.AJVP_ERR_INVALID_ARG

    def bwd(ws=p, ws_bytes=1 << 30, grad=p, Lq=8, cap=0.0, H=2):
        return lib.attn_jvp_bwd_scored(*[p] * 12, grad, p, p, p, p, p, None, None, None, 1, H, 2, Lq, 8, 128, 0.1, cap, ws,
                                       ws_bytes, None)

    assert bwd(ws=None) == B.AJVP_ERR_WORKSPACE and bwd(ws=ctypes.c_void_p(128)) == B.AJVP_ERR_WORKSPACE
    least = (16 * (2 * 8 + 64) + 255) // 256 * 256 + 256
    assert bwd(ws_bytes=least - 1) == B.AJVP_ERR_WORKSPACE
    assert bwd(grad=None) == B.AJVP_ERR_INVALID_ARG and bwd(H=3) == B.AJVP_ERR_INVALID_ARG
    assert bwd(cap=-2.0) == B.AJVP_ERR_INVALID_ARG
    size = lib.attn_jvp_bwd_scored_workspace_bytes
    if not torch.cuda.is_available():
        assert size(1, 2, 2, 8, 8) == least  # no usable device: the least
    assert size(1, 3, 2, 8, 8) == 0 and size(-1, 2, 2, 8, 8) == 0 and size(1, 2, 2, 8, 0) == 0


def test_cache_refusals(lib):
    p = ctypes.c_void_p(256)

    def append(ptr=p, q=None, tq=None, qo=None, tqo=None, cos=None, sin=None, n_seq=1, H=2, Hkv=2, total=3, pages=4,
               page=16, width=2, n_pos=0, d=128):
        return lib.attn_jvp_cache_append(ptr, ptr, q, tq, qo, tqo, ptr, ptr, ptr, ptr, ptr, ptr, ptr, cos, sin, n_seq, H,
                                         Hkv, total, pages, page, width, n_pos, d, 0, None)

    inv, big = B.AJVP_ERR_INVALID_ARG, B.AJVP_ERR_TOO_LARGE
    assert append(page=24) == inv and append(page=0) == inv and append(H=3) == inv and append(width=0) == inv
    assert append(total=-1) == inv and append(cos=p) == inv and append(cos=p, sin=p, n_pos=0) == inv
    assert append(q=p, qo=p) == inv  # without angles there is nothing to do for queries
    assert append(tq=p, tqo=p, cos=p, sin=p, n_pos=4) == inv and append(q=p, cos=p, sin=p, n_pos=4) == inv
    assert append(width=1 << 20) == big and append(page=1 << 17) == big and append(pages=1 << 31) == big
    assert append(pages=1 << 27) == big  # more than 2^31 token rows
    assert append(d=64) == B.AJVP_ERR_UNSUPPORTED_DIM and append(ptr=None) == inv
    assert append(ptr=ctypes.c_void_p(40)) == B.AJVP_ERR_MISALIGNED
    assert append(ptr=None, total=0) == B.AJVP_OK and append(ptr=None, n_seq=0) == B.AJVP_OK

    def attn(ptr=p, tq=None, to=None, cu=None, n_seq=1, H=2, Hkv=2, n=1, total=0, sb=256, sh=128, st=128, page=16, cap=0.0,
             pages=4, scale=0.1, ws=None):
        return lib.attn_jvp_fwd_cache(ptr, tq, ptr, to, None, ptr, ptr, ptr, ptr, ptr, ptr, cu, None, n_seq, H, Hkv, n,
                                      total, sb, sh, st, pages, page, 2, 128, scale, cap, 1, ws, 0, None)

    assert attn(tq=p) == inv and attn(to=p) == inv and attn(cu=p, n=4, total=3) == inv and attn(n=-1) == inv
    assert attn(cap=-1.0) == inv and attn(scale=float("nan")) == inv and attn(H=3) == inv and attn(pages=0) == inv
    assert attn(sh=100) == B.AJVP_ERR_MISALIGNED and attn(ptr=ctypes.c_void_p(24)) == B.AJVP_ERR_MISALIGNED
    assert attn(n=1 << 31) == big and attn(ptr=None) == inv
    assert attn(ws=ctypes.c_void_p(64)) == B.AJVP_ERR_WORKSPACE
    size = lib.attn_jvp_fwd_cache_workspace_bytes
    assert size(1, 3, 2, 1, 16, 9, 1) == 0 and size(1, 2, 2, 1, 24, 9, 1) == 0 and size(-1, 2, 2, 1, 16, 9, 0) == 0
    assert size(0, 2, 2, 1, 16, 9, 1) == 0 and size(1, 2, 2, 0, 16, 9, 1) == 0
    assert attn(ptr=None, n=0) == B.AJVP_OK and attn(ptr=None, n_seq=0) == B.AJVP_OK


def test_binding_refuses_what_it_cannot_pass_on(lib):
    x = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attn_jvp_fwd_scored(x, x, x, x, x, x)  # host tensors
    with pytest.raises(ValueError):
        attn_jvp_autograd(x, x, x, x, x, x, causal=True, key_end=torch.zeros(4, dtype=torch.int32))
    c = torch.zeros(2, 2, 16, 128).to(torch.float8_e4m3fn)
    s, t, n = torch.zeros(2, 2), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn_jvp_cache_append(x[0], x[0], c, c, s, s, t, n, n)
    with pytest.raises(ValueError):
        attn_jvp_fwd_cache(x, None, c, c, s, s, t, n)


def _local(q, k, v, tq, tk, tv, scale, softcap=0.0, slopes=None, key_begin=None, key_end=None):
    return ref.forward(q, k, v, tq, tk, tv, scale, softcap=softcap, slopes=slopes, begin=key_begin, end=key_end)


def _local_bwd(q, k, v, tq, tk, tv, o, to, lse, mu, dout, dtout, scale, softcap=0.0, slopes=None, key_begin=None,
               key_end=None):
    return ref.backward(q, k, v, tq, tk, tv, dout, dtout, scale, softcap=softcap, slopes=slopes, begin=key_begin,
                        end=key_end)


def _rank(rank, world, port, out):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        from attention_forward_mode_b200.ulysses import ulysses_attn_jvp, ulysses_attn_jvp_bwd, ulysses_attn_jvp_train
        x, (do, dto) = draw(2, 8, 4, 12, 8, 4, seed=5)
        begin, end = key_bounds(12, 8, device="cpu", causal=True, prefix=3)
        score = dict(softcap=2.0, slopes=torch.linspace(0.05, 0.9, 8), key_begin=begin.expand(2, 12).contiguous(),
                     key_end=end.expand(2, 12).contiguous())
        cut = lambda t: t[:, :, rank * t.shape[2] // world:(rank + 1) * t.shape[2] // world].contiguous()  # noqa: E731
        mine = [cut(t) for t in x]
        want = _local(*x, 0.5, **score)
        o, to, lse = ulysses_attn_jvp(*mine, scale=0.5, score=score,
                                      local_fn=lambda *a, **kw: _local(*a, **kw)[:3])
        same = [torch.allclose(a, cut(b), equal_nan=True) for a, b in zip((o, to), want[:2])]
        same.append(torch.allclose(lse, cut(want[2].unsqueeze(-1))[..., 0]))
        o, to, lse, ctx = ulysses_attn_jvp_train(*mine, scale=0.5, score=score, local_fwd=_local)
        g = ulysses_attn_jvp_bwd(ctx, cut(do), cut(dto), local_bwd=_local_bwd)
        full = ref.backward(*x, do, dto, 0.5, softcap=2.0, slopes=score["slopes"], begin=score["key_begin"],
                            end=score["key_end"])
        same += [torch.allclose(g[n], cut(full[n])) for n in g]
        try:
            ulysses_attn_jvp(*mine, scale=0.5, score=dict(cap=3.0), local_fn=_local)
            same.append(False)
        except ValueError:
            same.append(True)
        out[rank] = same
    finally:
        dist.destroy_process_group()


@pytest.mark.timeout(240)
@pytest.mark.parametrize("world", [2, 4])
def test_ulysses_with_score_options(world):
    import socket
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    with ctx.Manager() as m:
        out = m.dict()
        procs = [ctx.Process(target=_rank, args=(r, world, port, out)) for r in range(world)]
        for p in procs:
            p.start()
        for p in procs:
            p.join(200)
        assert all(p.exitcode == 0 for p in procs), [p.exitcode for p in procs]
        assert len(out) == world and all(all(v) for v in out.values()), dict(out)
