"""Ulysses with local steps of the caller's own and with causal score options,
on one process and over gloo ranks."""
import os

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import scored_reference as ref
from attention_forward_mode_b200 import key_bounds
from attention_forward_mode_b200.ulysses import ulysses_attn_jvp, ulysses_attn_jvp_bwd, ulysses_attn_jvp_train
from test_scored_cpu import _local, _local_bwd, draw


def test_a_local_step_of_the_callers_own_takes_any_heads():
    """Without score options it is called with the plain arguments: fewer key heads, causal or not, 3 on 2 heads."""
    for H, Hkv in ((4, 2), (3, 2)):
        x, (do, dto) = draw(1, H, Hkv, 6, 6, 4, seed=7)
        for causal in (False, True):
            seen = []

            def fwd(*a):
                seen.append(len(a))
                return x[0], x[3], x[0][..., 0], x[0][..., 1]

            o, to, lse = ulysses_attn_jvp(*x, causal=causal, local_fn=lambda *a: fwd(*a)[:3])
            assert o is x[0] and to is x[3] and seen == [7]
            *_, ctx = ulysses_attn_jvp_train(*x, causal=causal, local_fwd=fwd)
            g = ulysses_attn_jvp_bwd(ctx, do, dto, local_bwd=lambda *a: dict(n=len(a)))
            assert seen == [7, 7] and g == dict(n=13)


def _rank(rank, world, port, out):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        x, (do, dto) = draw(2, 4, 2, 8, 12, 4, seed=8)
        cut = lambda t: t[:, :, rank * t.shape[2] // world:(rank + 1) * t.shape[2] // world].contiguous()  # noqa: E731
        mine = [cut(t) for t in x]
        begin, end = key_bounds(8, 12, device="cpu", causal=True)
        score = dict(softcap=2.0)
        want = _local(*x, 0.5, **score, key_begin=begin, key_end=end)
        o, to, _, ctx = ulysses_attn_jvp_train(*mine, scale=0.5, score=score, causal=True, local_fwd=_local)
        g = ulysses_attn_jvp_bwd(ctx, cut(do), cut(dto), local_bwd=_local_bwd)
        full = ref.backward(*x, do, dto, 0.5, softcap=2.0, begin=begin, end=end)
        same = [torch.allclose(o, cut(want[0])), torch.allclose(to, cut(want[1]))]
        same += [torch.allclose(g[n], cut(full[n])) for n in g]
        o, to, _ = ulysses_attn_jvp(*mine, scale=0.5, score=score, causal=True,
                                    local_fn=lambda *a, **kw: _local(*a, **kw)[:3])
        same += [torch.allclose(o, cut(want[0])), torch.allclose(to, cut(want[1]))]
        try:
            ulysses_attn_jvp(*mine, scale=0.5, score=dict(key_end=end), causal=True, local_fn=_local)
            same.append(False)
        except ValueError:
            same.append(True)
        out[rank] = same
    finally:
        dist.destroy_process_group()


@pytest.mark.timeout(240)
def test_causal_score_options():
    import socket
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    with ctx.Manager() as m:
        out = m.dict()
        procs = [ctx.Process(target=_rank, args=(r, 2, port, out)) for r in range(2)]
        for p in procs:
            p.start()
        for p in procs:
            p.join(200)
        assert all(p.exitcode == 0 for p in procs), [p.exitcode for p in procs]
        assert len(out) == 2 and all(all(v) for v in out.values()), dict(out)
