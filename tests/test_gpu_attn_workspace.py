"""One workspace for calls of many sizes, and prompts whose rows are a few of a
larger buffer."""
import math

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests.test_gpu_attn_prompt import Case
from tests.test_gpu_cache4 import Step, run_evict

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_prompts_of_falling_sizes():
    """Sized for one long prompt: then a question, single tokens and a short prompt over long contexts."""
    a = kvi.attention(8, 2, 64)
    ws = ac.workspace(kvi.kvi_attn_prompt_workspace_bytes(a, 8, 3000, 3000, 3000))
    for n_q, ctx in (([3000], [3000]), ([37], [1601]), ([1, 1, 1], [2999, 700, 3]), ([1], [3000]), ([200], [2999]), ([9] * 8, [2500] * 8)):
        c = Case(8, 2, 64, 16, n_q, ctx, seed=ctx[0])
        kvi.kvi_attn_prompt(c.a, c.q, c.q_start, c.max_q, c.ctx_lens, c.max_ctx, c.table, kvi.paged_cache([c.pool], 16), 0,
                            c.out, ws, c.status, lse=c.lse)
        c.check()


@pytest.mark.parametrize("n_q,ctx", [([1], [4099]), ([3, 0, 2], [4000, 9, 2100]), ([60], [3000]), ([40, 64], [700, 2500])])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 64), (4, 1, 128), (3, 1, 256)])
def test_rows_of_a_larger_buffer(Hq, H, D, n_q, ctx):
    """q and out have many more rows than the requests: they lie somewhere in the middle."""
    before, after = 1000, 500
    c = Case(Hq, H, D, 16, n_q, ctx, seed=D + sum(n_q))
    n = sum(n_q)
    q = torch.full((before + n + after, Hq, D), math.nan, dtype=torch.bfloat16, device=DEV)
    q[before:before + n] = c.q
    out = torch.full_like(q, 7.0)
    lse = torch.full(out.shape[:2], 7.0, device=DEV)
    size = kvi.kvi_attn_prompt_workspace_bytes(c.a, len(n_q), q.shape[0], c.max_q, c.max_ctx)
    assert size <= kvi.kvi_attn_prompt_workspace_bytes(c.a, len(n_q), len(n_q) * c.max_q, c.max_q, c.max_ctx)
    kvi.kvi_attn_prompt(c.a, q, c.q_start + before, c.max_q, c.ctx_lens, c.max_ctx, c.table, kvi.paged_cache([c.pool], 16), 0,
                        out, ac.workspace(size), c.status, lse=lse)
    c.out, c.lse = out[before:before + n], lse[before:before + n]
    c.check()
    for x in (out, lse):
        assert bool((x[:before] == 7).all()) and bool((x[before + n:] == 7).all())


def test_steps_of_falling_sizes():
    a = kvi.attention(8, 2, 64)
    ws = ac.workspace(kvi.kvi_attn_decode4_workspace_bytes(a, 6, 2049, True))
    for ctx, weights in (([2049] * 6, True), ([2048], True), ([1601], False), ([1200, 700, 2000], False), ([400, 1], True)):
        c = Step(8, 2, 64, 16, ctx, seed=ctx[0], weights=weights)
        kvi.kvi_attn_decode4(c.a, c.q, c.ctx_lens, max(ctx), c.table, c.c.cache, 0, c.out, ws, c.c.status, weights=c.w)
        c.check()


def test_evict_and_the_step_after_it():
    """Sized for the step before the eviction."""
    ctx, budget = [2049, 1500], 2048
    c = Step(4, 1, 64, 16, ctx, seed=1)
    ws = ac.workspace(max(kvi.kvi_attn_decode4_workspace_bytes(c.a, 2, 2049, True),
                          kvi.kvi_cache4_evict_workspace_bytes(1, 2, 2049)))
    w = torch.rand(2, 1, 2049, generator=ac.gen(2), device=DEV)
    pos = torch.arange(2049, dtype=torch.int32, device=DEV).expand(2, 1, -1).contiguous()
    w_out, pos_out, out = run_evict(c, ctx, budget, 4, 64, w, pos)
    before = w_out.clone()
    kvi.kvi_attn_decode4(c.a, c.q, out, budget, c.table, c.c.cache, 0, c.out, ws, c.c.status, weights=w_out)
    assert int(c.c.status) == 0 and out.tolist() == [2048, 1500]
    for r, n in enumerate(out.tolist()):  # each head's weights sum to one
        assert abs(float((w_out[r, 0, :n] - before[r, 0, :n]).double().sum()) - 4) < 1e-3
