"""Forms of the attention calls that sizes alone decide on: pages of a whole
tile of keys and more, launches of joined clusters in a graph, and requests past
the first 32 that are refused."""
import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests.test_gpu_attn_prompt import Case
from tests.test_gpu_cache4 import Step

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("B", [112, 128, 256, 384])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (6, 2, 64)])
def test_prompts_over_large_pages(Hq, H, D, B):
    c = Case(Hq, H, D, B, [130, 1, 300, 40], [130, 700, 513, 39], seed=B + D)
    c.run()
    c.check()


@pytest.mark.parametrize("B", [128, 256])
def test_steps_over_large_pages(B):
    c = Step(8, 2, 128, B, [1, B - 1, B, B + 1, 1700], seed=B)
    c.run()
    c.check()


def test_joined_clusters_in_a_graph():
    """One token over the bf16 cache and over the 4-bit one, their keys in a few pieces."""
    p, s = Case(8, 2, 128, 16, [1, 1], [900, 301], seed=1), Step(8, 2, 128, 16, [900, 301], seed=2, weights=False)
    wp = ac.workspace(kvi.kvi_attn_prompt_workspace_bytes(p.a, 2, 2, 1, 900))
    ws = ac.workspace(kvi.kvi_attn_decode4_workspace_bytes(s.a, 2, 900, False))
    cache = kvi.paged_cache([p.pool], 16)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvi.kvi_attn_prompt(p.a, p.q, p.q_start, 1, p.ctx_lens, 900, p.table, cache, 0, p.out, wp, p.status, lse=p.lse)
        kvi.kvi_attn_decode4(s.a, s.q, s.ctx_lens, 900, s.table, s.c.cache, 0, s.out, ws, s.c.status)
    for seed in (3, 4):
        for x in (p, s):
            x.q.copy_(ac.randn(ac.gen(seed), *x.q.shape).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        p.check()
        s.check()


@pytest.mark.parametrize("bad", [0, 31, 32, 36, 39])
@pytest.mark.parametrize("n", [2, 40])
def test_one_of_many_requests_is_refused(n, bad):
    R = 40
    n_q, ctx = [n] * R, [n + 3 * r for r in range(R)]
    c, good = (Case(4, 1, 128, 16, n_q, ctx, seed=n) for _ in range(2))
    good.run()
    c.ctx_lens[bad] = -1
    c.run()
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE
    keep = torch.ones(R * n, dtype=torch.bool, device=DEV)
    keep[bad * n:(bad + 1) * n] = False
    assert torch.equal(c.out[keep], good.out[keep]) and torch.equal(c.lse[keep], good.lse[keep])
    assert bool((c.out[~keep] == 7).all()) and bool((c.lse[~keep] == 7).all())
