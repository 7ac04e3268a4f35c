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


def test_weights_round_once():
    """P * step rounds to bf16 once.  All keys but the first, whose value is zero, weigh and hold the same, so
    that the rounding of their P * step does not average out.  An error spread evenly over half a unit of a number
    whose place between powers of two is spread evenly too is 2^-8 (0.541 / 3)^(1/2) = 0.425 * 2^-8 of it in the
    mean square: 0.601 * 2^-8 for P * step and the output together, 0.736 * 2^-8 if P had been rounded before."""
    R, G, D, n = 256, 8, 256, 32
    g = ac.gen(5)
    groups = D // 32
    k = torch.zeros(R, n, 1, D, dtype=torch.bfloat16, device=DEV)
    k[:, 1:, 0, 0] = 1
    v = torch.zeros(R, n, 1, groups, 32, device=DEV)
    v[:, 1:] = torch.exp2(4 * torch.rand(R, 1, 1, groups, 1, generator=g, device=DEV))
    k, v = k.view(R * n, 1, D), v.view(R * n, 1, D).to(torch.bfloat16)
    c = ac.Cache4(g, 1, D, n, R, k=k, v=v)
    q = torch.zeros(R, G, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = -6 * torch.rand(R, G, generator=g, device=DEV) * 0.6931 * D ** 0.5
    a, out = kvi.attention(G, 1, D), torch.empty(R, G, D, dtype=torch.bfloat16, device=DEV)
    kvi.kvi_attn_decode4(a, q, torch.full((R,), n, dtype=torch.int32, device=DEV), n,
                         torch.arange(R, dtype=torch.int32, device=DEV)[:, None], c.cache, 0, out,
                         ac.workspace(kvi.kvi_attn_decode4_workspace_bytes(a, R, n, False)), c.status)
    assert int(c.status) == 0
    p = torch.exp(q[..., 0].double() * c.kd.view(R, n, D)[:, 1, :1] * D ** -0.5)[..., None]     # [R][G][1]
    value = c.vd.view(R, n, D)[:, None, 1]                                                      # [R][1][D]
    total = 1 + (n - 1) * p
    ref = (n - 1) * p * value / total

    def rms(x):
        return float((((x - ref) / ref)[..., ::32]).square().mean().sqrt()) * 256

    def rounded(x):
        return x.to(torch.bfloat16).double()

    step = value / 7
    once, twice = (rounded((n - 1) * rounded(x * step) * 7 / total) for x in (p, rounded(p)))
    assert rms(once) < 0.64 and rms(twice) > 0.69
    assert rms(out.double()) < 0.665
