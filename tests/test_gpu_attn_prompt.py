"""kvi_attn_prompt against plain float64 attention: head layouts, page sizes,
prompts of no, one and many tokens, rows that see nothing, keys past the end,
values that a row must not see, strides, streams, capture and refusals."""
import math

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    def __init__(self, Hq, H, D, B, n_q, ctx, seed=0, wide=0, lse=True, poison=True):
        g = ac.gen(seed)
        self.Hq, self.H, self.D, self.B, self.n_q, self.ctx = Hq, H, D, B, n_q, ctx
        self.a = kvi.attention(Hq, H, D)
        total = sum(n_q)
        self.q_start = torch.tensor([sum(n_q[:i]) for i in range(len(n_q) + 1)], dtype=torch.int32, device=DEV)
        self.ctx_lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.table, blocks = ac.tables(g, ctx, B)
        self.pool = ac.randn(g, 2, blocks, B, H, D).to(torch.bfloat16)
        if poison:  # what lies outside the requests' positions
            used = torch.zeros(blocks * B, dtype=torch.bool, device=DEV)
            for r, c in enumerate(ctx):
                p = torch.arange(c, device=DEV)
                used[self.table[r][p // B].long() * B + p % B] = True
            self.pool.view(2, blocks * B, H, D)[:, ~used] = math.nan
        self.q = ac.randn(g, total, Hq + wide, D).to(torch.bfloat16)[:, :Hq]
        self.out = torch.full((total, Hq + wide, D), 7.0, dtype=torch.bfloat16, device=DEV)[:, wide:]
        self.lse = torch.full((total, Hq), 7.0, device=DEV) if lse else None
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.max_q, self.max_ctx = max(n_q), max(ctx)

    def run(self, stream=None, **kw):
        n = kvi.kvi_attn_prompt_workspace_bytes(self.a, len(self.ctx), self.q.shape[0], self.max_q, self.max_ctx)
        assert n > 0
        kvi.kvi_attn_prompt(self.a, self.q, self.q_start, self.max_q, self.ctx_lens, self.max_ctx, self.table,
                            kvi.paged_cache([self.pool], self.B), 0, self.out, ac.workspace(n), self.status,
                            lse=self.lse, stream=stream, **kw)

    def kv(self, r, h):
        t = self.table[r].long().clamp(0, self.pool.shape[1] - 1)
        return (self.pool[x, t, :, h].reshape(-1, self.D)[:self.ctx[r]].double() for x in (0, 1))

    def check(self):
        assert int(self.status) == 0
        G = self.Hq // self.H
        q0 = 0
        for r, (n, c) in enumerate(zip(self.n_q, self.ctx)):
            last = torch.arange(n, device=DEV) + (c - n)
            for h in range(self.H):
                if n == 0:
                    continue
                k, v = self.kv(r, h)
                hs = slice(h * G, (h + 1) * G)
                ref, lse, _, pv, size = ac.attend(self.q[q0:q0 + n, hs].double(), k, v, last, self.D ** -0.5)
                empty = last < 0
                ref[empty] = 0
                pv[empty] = 0
                ac.check_out(self.out[q0:q0 + n, hs], ref, pv, size, 1, (r, h))
                if self.lse is not None:
                    ac.check_lse(self.lse[q0:q0 + n, hs], lse, size)
            q0 += n


LAYOUTS = [(1, 1, 16), (3, 1, 80), (4, 2, 64), (8, 8, 128), (10, 2, 96), (32, 8, 128), (6, 1, 256), (40, 2, 32),
           (128, 1, 128), (14, 2, 144)]


@pytest.mark.parametrize("B", [1, 5, 8, 16, 24, 64])
@pytest.mark.parametrize("Hq,H,D", LAYOUTS)
def test_layouts(Hq, H, D, B):
    """No, one and a few tokens; with and without memory; more tokens than keys; pages ending inside a tile."""
    c = Case(Hq, H, D, B, [0, 1, 1, 7, 33, 20, 3], [5, 1, 77, 7, 130, 12, 0], seed=Hq * D + B)
    c.run()
    c.check()


@pytest.mark.parametrize("n_q,ctx", [([1], [1]), ([1], [4099]), ([257], [257]), ([129], [1000]), ([70], [64]),
                                     ([1, 300, 2, 0, 511], [900, 300, 2, 64, 1999]), ([1025], [1153]),
                                     ([5] * 40, [5 + 29 * i for i in range(40)])])
@pytest.mark.parametrize("Hq,H,D,B", [(4, 2, 64, 16), (8, 2, 128, 16), (5, 1, 128, 32), (7, 1, 96, 48), (2, 2, 112, 16)])
def test_lengths(Hq, H, D, B, n_q, ctx):
    c = Case(Hq, H, D, B, n_q, ctx, seed=len(n_q) + D + Hq)
    c.run()
    c.check()


def test_single_tokens_many_requests():
    ctx = [1 + (37 * i) % 2300 for i in range(64)]
    c = Case(32, 8, 128, 16, [1] * 64, ctx, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("Hq,H,D,B", [(8, 2, 64, 16), (8, 2, 128, 16), (6, 1, 256, 8), (7, 1, 96, 48), (4, 4, 32, 5)])
@pytest.mark.parametrize("most", [300, 600, 1000, 1024])
def test_joined_pieces(Hq, H, D, B, most):
    """Few rows over two to eight pieces of the keys: requests with all of them, some, one and none."""
    c = Case(Hq, H, D, B, [1, 0, 2, 1, 2, 1, 2], [most, 5, 1, most // 2 + 3, most - 1, 0, 128], seed=most)
    c.run()
    c.check()
    first = c.out.clone()
    c.run()
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("n_q", [[9, 40], [200, 300]])
def test_strided_rows_without_lse(n_q):
    c = Case(8, 2, 128, 16, n_q, [n + 30 for n in n_q], seed=5, wide=4, lse=False)
    c.run()
    c.check()
    full = c.out._base
    assert bool((full[:, :4] == 7).all()), "written outside the rows"


@pytest.mark.parametrize("shift", [-60.0, 60.0])
def test_large_scores_and_late_maximum(shift):
    """Scores that grow along the keys (every tile moves the maximum), far from zero."""
    c = Case(4, 1, 64, 16, [3, 150], [1500, 700], seed=6, poison=False)
    grow = torch.linspace(0, 1, c.pool.shape[1] * c.B, device=DEV).view(1, -1, 1, 1)
    q = torch.zeros_like(c.q)
    q[..., 0] = 8
    q[..., 1:] = c.q[..., 1:] * 0.1
    c.q = q
    k = c.pool[0].view(1, -1, 1, c.D)
    k[..., 0] = (shift * (1 + grow[..., 0])).to(torch.bfloat16)
    c.run()
    c.check()


@pytest.mark.parametrize("n", [6, 150, 400])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("Hq,H,D", [(4, 1, 128), (2, 2, 64)])
def test_unseen_values_have_no_effect(Hq, H, D, bad, n):
    """An infinity or NaN in the K or V of token j touches no row before j, and the rows from j on."""
    ctx, j = n + 21, n // 2
    c = Case(Hq, H, D, 16, [n], [ctx], seed=7)
    c.run()
    clean = c.out.clone()
    p = ctx - n + j
    for plane in (0, 1):
        c.pool = c.pool.clone()
        keep = c.pool[plane, c.table[0, p // 16].long(), p % 16].clone()
        c.pool[plane, c.table[0, p // 16].long(), p % 16, :, 3] = bad
        c.out.fill_(7)
        c.run()
        assert torch.equal(c.out[:j], clean[:j])
        if plane == 1:
            assert not bool(torch.isfinite(c.out[j:, :, 3]).any())
            assert torch.equal(c.out[j:, :, :3], clean[j:, :, :3]) and torch.equal(c.out[j:, :, 4:], clean[j:, :, 4:])
        elif math.isnan(bad):
            assert bool(torch.isnan(c.out[j:]).all())
        c.pool[plane, c.table[0, p // 16].long(), p % 16] = keep


def test_scores_of_minus_infinity():
    """Keys whose scores are -inf take no part; a row with nothing else gives zeros."""
    c = Case(2, 1, 64, 16, [1, 1], [40, 3], seed=8, poison=False)
    c.q.fill_(1.0)
    flat = c.pool[0].view(-1, 1, 64)
    for r, hidden in ((0, range(5, 30)), (1, range(3))):
        for p in hidden:
            flat[int(c.table[r, p // 16]) * 16 + p % 16, 0, 0] = -math.inf
    c.run()
    k, v = c.kv(0, 0)
    seen = torch.tensor([p for p in range(40) if not 5 <= p < 30], device=DEV)
    ref, lse, _, pv, size = ac.attend(c.q[:1].double(), k[seen], v[seen], torch.tensor([len(seen) - 1], device=DEV), 0.125)
    ac.check_out(c.out[:1], ref, pv, size, 1)
    ac.check_lse(c.lse[:1], lse, size)
    assert bool((c.out[1] == 0).all()) and bool((c.lse[1] == -math.inf).all())


@pytest.mark.parametrize("n_q", [[2, 3], [300, 260]])
def test_bad_requests_are_skipped(n_q):
    for what in ("ctx", "rows", "block"):
        c = Case(4, 2, 128, 16, n_q + [1], [n + 40 for n in n_q] + [20], seed=9)
        good = Case(4, 2, 128, 16, n_q + [1], [n + 40 for n in n_q] + [20], seed=9)
        good.run()
        if what == "ctx":
            c.ctx_lens[1] = c.max_ctx + 1
        elif what == "rows":
            c.q_start[2] = c.q.shape[0] + 5
        else:
            c.table[1, 1] = c.pool.shape[1]
        c.run()
        assert int(c.status) == kvi.ERR_OUT_OF_RANGE
        assert torch.equal(c.out[:n_q[0]], good.out[:n_q[0]])
        if what == "ctx":
            assert bool((c.out[n_q[0]:n_q[0] + n_q[1]] == 7).all())
            assert torch.equal(c.out[-1:], good.out[-1:])
        elif what == "block":  # keys 16..31 of request 1 are left out
            k, v = c.kv(1, 0)
            seen = torch.cat([torch.arange(16), torch.arange(32, c.ctx[1])]).to(DEV)
            last = torch.arange(n_q[1], device=DEV) + (c.ctx[1] - n_q[1]) - 16
            ref, _, _, pv, size = ac.attend(c.q[n_q[0]:n_q[0] + n_q[1], :2].double(), k[seen], v[seen], last, 128 ** -0.5)
            ac.check_out(c.out[n_q[0]:n_q[0] + n_q[1], :2], ref, pv, size, 1)


def test_other_stream_and_graph():
    c = Case(8, 2, 128, 16, [5, 200], [700, 333], seed=10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    s.synchronize()
    c.check()
    n = kvi.kvi_attn_prompt_workspace_bytes(c.a, 2, 205, 200, 700)
    ws, cache = ac.workspace(n), kvi.paged_cache([c.pool], 16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvi.kvi_attn_prompt(c.a, c.q, c.q_start, 200, c.ctx_lens, 700, c.table, cache, 0, c.out, ws, c.status, lse=c.lse)
    for seed in (1, 2):
        c.q.copy_(ac.randn(ac.gen(seed), *c.q.shape).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        c.check()


@pytest.mark.parametrize("n", [3, 140])
def test_offsets_past_32_bits(n):
    """A pool of more than 2^31 elements per plane, used at its far end."""
    H, D, B = 8, 128, 16
    blocks = (1 << 31) // (B * H * D) + 64
    if torch.cuda.mem_get_info()[0] < 2 * blocks * B * H * D * 2 + (4 << 30):
        pytest.skip("not enough device memory")
    c = Case(8, 8, D, B, [n], [500], seed=11, poison=False)
    pool = torch.empty(2, blocks, B, H, D, dtype=torch.bfloat16, device=DEV)
    small, table = c.pool, c.table.clone()
    c.table = (blocks - 1 - table).to(torch.int32)
    pool[:, c.table[0].long()] = small[:, table[0].long()]
    c.pool = pool
    c.run()
    c.check()


def test_repeats_bit_for_bit():
    c = Case(32, 8, 128, 16, [1, 90, 600], [2000, 1200, 900], seed=12)
    c.run()
    first = c.out.clone()
    for _ in range(3):
        c.out.fill_(7)
        c.run()
        assert torch.equal(c.out, first)


def test_refusals():
    c = Case(4, 2, 64, 16, [2], [20], seed=13)
    n = kvi.kvi_attn_prompt_workspace_bytes(c.a, 1, 2, 2, 20)

    def refused(a=None, **kw):
        d = dict(q=c.q, max_q=2, max_ctx=20, table=c.table, cache=kvi.paged_cache([c.pool], 16), layer=0, out=c.out,
                 ws=ac.workspace(n), status=c.status, ctx=c.ctx_lens)
        d.update(kw)
        with pytest.raises(kvi.KviError) as e:
            kvi.kvi_attn_prompt(a or c.a, d["q"], c.q_start, d["max_q"], d["ctx"], d["max_ctx"], d["table"], d["cache"],
                                d["layer"], d["out"], d["ws"], d["status"])
        assert e.value.status == kvi.ERR_INVALID_ARG
        return kvi.kvi_last_error()

    assert "layer" in refused(layer=1)
    assert "layer" in refused(layer=-1)
    assert "max_q" in refused(max_q=3)
    assert "max_ctx" in refused(max_ctx=-1)
    assert "workspace" in refused(ws=ac.workspace(n + 16)[16:])
    assert "workspace" in refused(ws=ac.workspace(n)[:128])
    assert "scale" in refused(kvi.attention(4, 2, 64, scale=0.0))
    assert "scale" in refused(kvi.attention(4, 2, 64, scale=math.nan))
    buf = torch.zeros(2 * 4 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    assert "aligned" in refused(q=buf[4:4 + 512].view(2, 4, 64))
    assert "aligned" in refused(out=buf[1:1 + 512].view(2, 4, 64))
    torch.cuda.synchronize()
    assert int(c.status) == 0
