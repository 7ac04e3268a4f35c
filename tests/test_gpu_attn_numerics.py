"""The 4-bit decoding step at the ends of its number range."""
import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests.test_gpu_cache4 import Step

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("e", [60, 103, 110, 126])
@pytest.mark.parametrize("Hq,H,D", [(4, 1, 64), (10, 1, 128)])
def test_large_queries(Hq, H, D, e):
    """Finite q of up to 2^127 over keys as small: ordinary scores."""
    c = Step(Hq, H, D, 16, [200, 40, 1], seed=e)
    k = (c.c.k.float().clamp(-4, 4) * 2.0 ** -e).to(torch.bfloat16)
    kvi.kvi_cache4_write(c.c.cache, 0, k, c.c.v, torch.arange(k.shape[0], device=DEV), c.c.status)
    c.c.kd = ac.dequantise(*ac.quantise(k))
    c.q = (c.q.float().clamp(-1.9, 1.9) * 2.0 ** e).to(torch.bfloat16)
    assert bool(torch.isfinite(c.q).all())
    c.run()
    c.check()


@pytest.mark.parametrize("q", [0.0, 2.0 ** -120])
@pytest.mark.parametrize("scale", [1e-6, 1e-20, 1e-38])
def test_small_queries_and_scales(q, scale):
    """Scores of next to nothing: every key weighs the same, and a masked one nothing."""
    c = Step(4, 2, 64, 16, [5, 200, 33], seed=1)
    c.a = kvi.attention(4, 2, 64, scale=scale)
    c.q = torch.full_like(c.q, q)
    c.run()
    c.check()  # (its own scale matters as little)
