"""How exact kvi_attn_window is for few rows: the softmax weights are two bf16 numbers each, so that
a result is off by hardly more than its own rounding.

Tolerance, beside the result's own rounding (2^-8 of it) and float32's 2^-17 (1 + size) sum p |v| that all
attention calls have: a weight's first number is off by up to 2^-8 of the weight, the second one by up to
2^-8 of that, which leaves 2^-16 of each term, so 2^-16 sum p |v|.  (Heads of more than 128 channels have one
number, and the tolerance of the other calls.)"""
import math

import pytest
import torch

from tests import attn_check as ac
from tests import step_check as sc
from tests.test_gpu_attn_window import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
REST = 2.0 ** -8  # of a rounding of the weights to bf16, as attn_check counts them


@pytest.mark.parametrize("window,sink", [(3, 0), (20, 2), (130, 4), (700, 64)])
@pytest.mark.parametrize("Hq,H,D,B", [(1, 1, 16, 1), (4, 2, 64, 16), (32, 8, 128, 16), (10, 2, 96, 24), (6, 1, 256, 8), (8, 1, 32, 5)])
@pytest.mark.parametrize("R", [1, 40])
def test_single_tokens(R, Hq, H, D, B, window, sink):
    """Single tokens, and (256 channels) prompts; one piece of the keys, and several that a cluster or a kernel joins."""
    n_q = [1] * R if D < 256 else [1 + 17 * (i % 3) for i in range(R)]
    c = Case(Hq, H, D, B, n_q, [1700 - 41 * i for i in range(R)], window, sink, seed=Hq + D + window)
    c.run()
    assert int(c.status) == 0
    G, q0 = Hq // H, 0
    for r, n in enumerate(n_q):
        seen = c.seen(r)
        for h in range(H):
            k, v = c.kv(r, h)
            unseen = ~seen.any(0)[:, None]
            hs = slice(h * G, (h + 1) * G)
            ref, lse, pv, size = sc.attend(c.q[q0:q0 + n, hs].double(), k.masked_fill(unseen, 0), v.masked_fill(unseen, 0), seen, D ** -0.5)
            ac.check_out(c.out[q0:q0 + n, hs], ref, pv, size, REST if D <= 128 else 1, (r, h))
            ac.check_lse(c.lse[q0:q0 + n, hs], lse, size)
        q0 += n



@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [3, 39, 40, 240, 270, 299])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (4, 2, 64), (6, 1, 256), (1, 1, 32)])
def test_an_infinity_among_the_values_stays_one(Hq, H, D, at, bad):
    """In a tile that all rows see and in one that only some see: the rows that see it get it, the others nothing of it."""
    c = Case(Hq, H, D, 16, [1, 1], [300, 90], 60, 40, seed=D)
    c.run()
    clean = c.out.clone()
    flat = c.pool[1].view(-1, H, D)
    flat[c.slots(0)[at], :, 3] = bad
    c.out.fill_(7)
    c.run()
    rest = torch.arange(D, device=DEV) != 3
    assert torch.equal(c.out[..., rest], clean[..., rest]) and torch.equal(c.out[1], clean[1])
    if at < 40 or at >= 240:
        want = torch.full_like(c.out[0, :, 3], bad)
        assert torch.equal(c.out[0, :, 3].isnan(), want.isnan()) and (math.isnan(bad) or torch.equal(c.out[0, :, 3], want))
    else:
        assert torch.equal(c.out[0, :, 3], clean[0, :, 3])
