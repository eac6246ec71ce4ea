"""Scored attention + JVP where it could go wrong quietly: padding that is not
finite, biases of far keys, masks made inside a captured graph, launches of
very many heads."""
import pytest
import torch

import attention_forward_mode_b200 as ajvp
from test_gpu_scored import NAMES, against_reference, make, slopes_of

pytestmark = pytest.mark.gpu


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
