"""kvi_attn_window against plain float64 attention: windows from one key to all,
first tokens that stay visible, blocks that no row sees, values a row must not
see, and the refusals."""
import math

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests import step_check as sc
from tests.test_gpu_attn_prompt import Case as Prompt

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case(Prompt):
    """Positions that no row of a request sees hold NaN, and blocks without a seen one are not in the table."""

    def __init__(self, Hq, H, D, B, n_q, ctx, window, sink, **kw):
        super().__init__(Hq, H, D, B, n_q, ctx, **kw)
        self.window, self.sink = window, sink
        flat = self.pool.view(2, -1, H, D)
        for r, (n, c) in enumerate(zip(n_q, ctx)):
            p = torch.arange(c, device=DEV)
            gone = (p >= sink) & (p <= c - n - window) if n else p >= 0
            flat[:, self.slots(r)[gone]] = math.nan
            for b in range((c + B - 1) // B):
                if bool(gone[b * B:(b + 1) * B].all()):
                    self.table[r, b] = -1 - b

    def slots(self, r):
        p = torch.arange(self.ctx[r], device=DEV)
        return self.table[r][p // self.B].long() * self.B + p % self.B

    def seen(self, r):
        n, c = self.n_q[r], self.ctx[r]
        i, j = torch.arange(c - n, c, device=DEV)[:, None], torch.arange(c, device=DEV)
        return (j <= i) & ((j > i - self.window) | (j < self.sink))

    def run(self, stream=None):
        n = kvi.kvi_attn_prompt_workspace_bytes(self.a, len(self.ctx), self.q.shape[0], self.max_q, self.max_ctx)
        kvi.kvi_attn_window(self.a, self.q, self.q_start, self.max_q, self.ctx_lens, self.max_ctx, self.table,
                            kvi.paged_cache([self.pool], self.B), 0, self.window, self.sink, self.out, ac.workspace(n),
                            self.status, lse=self.lse, stream=stream)

    def check(self, status=0):
        assert int(self.status) == status
        G, q0 = self.Hq // self.H, 0
        for r, n in enumerate(self.n_q):
            seen = self.seen(r)
            for h in range(self.H if n else 0):
                k, v = self.kv(r, h)
                unseen = ~seen.any(0)[:, None]
                k, v = k.masked_fill(unseen, 0), v.masked_fill(unseen, 0)
                hs = slice(h * G, (h + 1) * G)
                ref, lse, pv, size = sc.attend(self.q[q0:q0 + n, hs].double(), k, v, seen, self.D ** -0.5)
                ac.check_out(self.out[q0:q0 + n, hs], ref, pv, size, 1, (r, h))
                if self.lse is not None:
                    ac.check_lse(self.lse[q0:q0 + n, hs], lse, size)
            q0 += n


WINDOWS = [(1, 0), (1, 3), (7, 1), (40, 0), (64, 20), (100, 4), (129, 130), (300, 64), (513, 0)]


@pytest.mark.parametrize("window,sink", WINDOWS)
@pytest.mark.parametrize("Hq,H,D,B", [(1, 1, 16, 1), (4, 2, 64, 16), (8, 2, 128, 16), (10, 2, 96, 24), (6, 1, 256, 8), (3, 1, 80, 5),
                                      (128, 1, 128, 16), (2, 2, 112, 64)])
def test_layouts(Hq, H, D, B, window, sink):
    """No, one and many tokens; rows that see nothing; windows within a tile, over several, longer than the keys."""
    c = Case(Hq, H, D, B, [0, 1, 1, 7, 150, 20, 3], [5, 1, 777, 7, 470, 12, 0], window, sink, seed=Hq * D + B + window)
    c.run()
    c.check()


@pytest.mark.parametrize("window,sink", [(5, 1), (128, 0), (256, 4), (500, 200), (1024, 1000)])
@pytest.mark.parametrize("n_q,ctx", [([1], [4099]), ([1] * 3, [900, 1500, 20]), ([257], [257]), ([70], [64]),
                                     ([1, 300, 2, 0, 511], [900, 300, 2, 64, 1999]), ([1100], [2500]),
                                     ([5] * 40, [5 + 29 * i for i in range(40)])])
@pytest.mark.parametrize("Hq,H,D,B", [(4, 2, 64, 16), (8, 2, 128, 16), (5, 1, 128, 32), (2, 2, 128, 48)])
def test_lengths(Hq, H, D, B, n_q, ctx, window, sink):
    c = Case(Hq, H, D, B, n_q, ctx, window, sink, seed=len(n_q) + D + Hq)
    c.run()
    c.check()


@pytest.mark.parametrize("window,sink", [(600, 0), (1000, 130), (2000, 4)])
@pytest.mark.parametrize("n_q", [[1], [1, 2, 1, 0, 1], [1] * 40, [30], [9, 3]])
def test_pieces(n_q, window, sink):
    """Few rows whose windows are split over blocks, which a cluster or a second kernel joins."""
    c = Case(8, 2, 128, 16, n_q, [9000 - 177 * i for i in range(len(n_q))], window, sink, seed=window)
    c.run()
    c.check()
    first = c.out.clone()
    c.run()
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("n_q,ctx", [([1, 40], [700, 90]), ([200], [500])])
def test_a_window_over_everything_is_the_plain_call(n_q, ctx):
    for window, sink in ((max(ctx), 0), ((1 << 31) - 1, 0), (1, max(ctx))):
        c = Case(8, 2, 128, 16, n_q, ctx, window, sink, seed=1)
        c.run()
        c.check()
        out, lse = c.out.clone(), c.lse.clone()
        c.out.fill_(7)
        Prompt.run(c)
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [10, 200, 333, 420])
@pytest.mark.parametrize("Hq,H,D,n,window,sink", [(4, 1, 128, 300, 140, 20), (2, 2, 64, 300, 256, 0), (8, 1, 128, 40, 33, 11),
                                                  (1, 1, 128, 300, 256, 15)])
def test_unseen_values_have_no_effect(Hq, H, D, n, window, sink, at, bad):
    """An infinity or NaN in the K or V of a key touches the rows that see it and no other."""
    ctx = 440
    c = Case(Hq, H, D, 16, [n], [ctx], window, sink, seed=7)
    c.table = torch.where(c.table < 0, torch.zeros_like(c.table), c.table)
    c.run()
    c.status.zero_()
    clean = c.out.clone()
    rows = c.seen(0)[:, at]
    slot = c.slots(0)[at]
    for plane in (0, 1):
        flat = c.pool[plane].view(-1, H, D)
        keep = flat[slot].clone()
        flat[slot, :, 3] = bad
        c.out.fill_(7)
        c.run()
        assert torch.equal(c.out[~rows], clean[~rows])
        if plane == 1:
            assert not bool(torch.isfinite(c.out[rows][..., 3]).any())
            assert torch.equal(c.out[rows][..., :3], clean[rows][..., :3])
            assert torch.equal(c.out[rows][..., 4:], clean[rows][..., 4:])
        elif math.isnan(bad):
            assert bool(torch.isnan(c.out[rows]).all())
        flat[slot] = keep


@pytest.mark.parametrize("n_q", [[2, 3], [300, 260]])
def test_bad_requests_and_blocks(n_q):
    good = Case(4, 2, 128, 16, n_q + [1], [n + 40 for n in n_q] + [20], 30, 4, seed=9)
    good.run()
    c = Case(4, 2, 128, 16, n_q + [1], [n + 40 for n in n_q] + [20], 30, 4, seed=9)
    c.ctx_lens[1] = c.max_ctx + 1
    c.run()
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE
    assert torch.equal(c.out[:n_q[0]], good.out[:n_q[0]]) and torch.equal(c.out[-1:], good.out[-1:])
    assert bool((c.out[n_q[0]:-1] == 7).all())
    c = Case(4, 2, 128, 16, n_q + [1], [n + 40 for n in n_q] + [20], 30, 4, seed=9)
    c.table[1, c.ctx[1] // 16] = c.pool.shape[1]  # a block that rows see: its keys are left out
    c.run()
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE
    assert torch.equal(c.out[:n_q[0]], good.out[:n_q[0]]) and torch.equal(c.out[-1:], good.out[-1:])
    assert bool(torch.isfinite(c.out[n_q[0]:-1].float()).all())


def test_other_stream_graph_and_strides():
    c = Case(8, 2, 128, 16, [5, 200, 1], [700, 333, 2500], 256, 20, seed=10, wide=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    s.synchronize()
    c.check()
    assert bool((c.out._base[:, :4] == 7).all())
    ws = ac.workspace(kvi.kvi_attn_prompt_workspace_bytes(c.a, 3, 206, 200, 2500))
    cache, g = kvi.paged_cache([c.pool], 16), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvi.kvi_attn_window(c.a, c.q, c.q_start, 200, c.ctx_lens, 2500, c.table, cache, 0, 256, 20, c.out, ws, c.status, lse=c.lse)
    for seed in (1, 2):
        c.q.copy_(ac.randn(ac.gen(seed), *c.q.shape).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        c.check()


@pytest.mark.parametrize("n", [1, 140])
def test_offsets_past_32_bits(n):
    H, D, B = 8, 128, 16
    blocks = (1 << 31) // (B * H * D) + 64
    if torch.cuda.mem_get_info()[0] < 2 * blocks * B * H * D * 2 + (4 << 30):
        pytest.skip("not enough device memory")
    c = Case(8, 8, D, B, [n], [500], 300, 7, seed=11)
    pool = torch.empty(2, blocks, B, H, D, dtype=torch.bfloat16, device=DEV)
    live = c.table[0] >= 0
    small, table = c.pool, c.table.clone()
    c.table = torch.where(c.table >= 0, blocks - 1 - c.table, c.table).to(torch.int32)
    pool[:, c.table[0][live].long()] = small[:, table[0][live].long()]
    c.pool = pool
    c.run()
    c.check()


def test_refusals():
    c = Case(4, 2, 64, 16, [2], [20], 5, 0, seed=13)
    for window, sink, what in ((0, 0, "window"), (-1, 0, "window"), (5, -1, "sink")):
        c.window, c.sink = window, sink
        with pytest.raises(kvi.KviError, match=what):
            c.run()
    torch.cuda.synchronize()
    assert int(c.status) == 0
