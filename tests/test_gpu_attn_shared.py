"""kvi_attn_shared against plain float64 attention over each request's whole table:
prefixes of one block to many, single tokens and questions, requests without rows,
head layouts, page sizes, requests that are skipped, capture and refusals."""
import math

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests.test_gpu_attn_prompt import Case as Prompt

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case(Prompt):
    """ctx: each request's keys past the prefix, its rows among them."""

    def __init__(self, Hq, H, D, B, n_q, ctx, shared, **kw):
        self.shared, first = shared, shared // B
        super().__init__(Hq, H, D, B, n_q, [c + shared for c in ctx], **kw)
        g = ac.gen(99)
        live = next((r for r, n in enumerate(n_q) if n), 0)
        for r in range(len(n_q)):
            self.table[r, :first] = self.table[live, :first]  # (a batch without rows: any table)
        used = self.table[live, :first].long()
        self.pool[:, used] = ac.randn(g, 2, first, B, H, D).to(torch.bfloat16)
        for r, n in enumerate(n_q):  # what a request without rows has is never read
            if n == 0:
                self.table[r] = -5

    def run(self, stream=None):
        n = kvi.kvi_attn_shared_workspace_bytes(self.a, len(self.ctx), self.q.shape[0], self.max_q, self.max_ctx, self.shared)
        assert n > 0
        kvi.kvi_attn_shared(self.a, self.q, self.q_start, self.max_q, self.ctx_lens, self.max_ctx, self.table,
                            kvi.paged_cache([self.pool], self.B), 0, self.shared, self.out, ac.workspace(n), self.status,
                            lse=self.lse, stream=stream)


LAYOUTS = [(1, 1, 16, 1), (4, 2, 64, 16), (8, 2, 128, 16), (32, 8, 128, 16), (10, 2, 96, 24), (6, 1, 256, 8), (3, 1, 80, 5),
           (128, 1, 128, 16), (2, 2, 112, 64)]


# (prefixes below some 32 MB less to read are attended with each request's other keys; test_many below has larger ones)
@pytest.mark.parametrize("blocks", [1, 7, 40])
@pytest.mark.parametrize("Hq,H,D,B", LAYOUTS)
def test_layouts(Hq, H, D, B, blocks):
    c = Case(Hq, H, D, B, [0, 1, 1, 7, 33, 0, 3], [0, 1, 77, 7, 130, 12, 300], blocks * B, seed=Hq * D + B)
    c.run()
    c.check()


@pytest.mark.parametrize("n_q,ctx", [([1], [1]), ([1] * 64, [1 + (37 * i) % 700 for i in range(64)]), ([257], [257]),
                                     ([5, 1, 30, 17] * 6, [40 + 9 * i for i in range(24)]), ([1, 600], [3, 700]),
                                     ([0, 0, 2], [5, 0, 2])])
@pytest.mark.parametrize("Hq,H,D,B,shared", [(8, 2, 128, 16, 1600), (8, 2, 128, 16, 10240), (4, 2, 64, 16, 416), (5, 1, 128, 32, 4096),
                                             (8, 8, 128, 16, 128), (6, 1, 256, 16, 992)])
def test_lengths(Hq, H, D, B, shared, n_q, ctx):
    c = Case(Hq, H, D, B, n_q, ctx, shared, seed=len(n_q) + D + Hq)
    c.run()
    c.check()
    first = c.out.clone()
    c.run()
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("more,long", [(0, 0), (3, 0), (0, 1500), (3, 1500)])
@pytest.mark.parametrize("Hq,H,D,B", LAYOUTS)
def test_many(Hq, H, D, B, more, long):
    """Enough requests that the prefix is read by itself: single tokens, and a few questions among them; own keys
    that are one piece, and several."""
    R = 90 if H * D > 64 else 200
    if long:
        R = min(R, 240 // H)
    n_q = [1 if i % 7 else 0 for i in range(R)]
    n_q[5:5 + more] = [9, 4, 13][:more]
    blocks = -(-(9 << 20) // ((R - 1) * H * D) // B) + 1
    ctx = [n + (37 * i) % 150 for i, n in enumerate(n_q)]
    ctx[3] += long
    c = Case(Hq, H, D, B, n_q, ctx, blocks * B, seed=Hq * D + B)
    c.run()
    c.check()
    first = c.out.clone()
    c.run()
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("Hq,H,D,B", [(6, 1, 256, 8), (3, 1, 80, 5), (40, 2, 32, 16), (10, 2, 96, 24), (4, 1, 128, 16)])
def test_a_wave_of_requests(Hq, H, D, B):
    """So many that their blocks are several waves, beside the prefix's."""
    R = 420
    n_q = [1 if i % 11 else 0 for i in range(R)]
    blocks = -(-(9 << 20) // ((R - 1) * H * D) // B) + 1
    c = Case(Hq, H, D, B, n_q, [n + (29 * i) % 90 for i, n in enumerate(n_q)], blocks * B, seed=D + B)
    c.run()
    c.check()


def test_strided_rows_without_lse():
    c = Case(8, 2, 128, 16, [9, 1, 40] * 4, [39, 5, 70] * 4, 4096, seed=5, wide=4, lse=False)
    c.run()
    c.check()
    assert bool((c.out._base[:, :4] == 7).all()), "written outside the rows"


@pytest.mark.parametrize("shared", [800, 16000])
@pytest.mark.parametrize("n_q", [[1, 1, 1], [30, 2, 5]])
def test_rows_of_a_larger_buffer(n_q, shared):
    """The batch's rows begin and end inside q; the others are left as they are."""
    c = Case(8, 2, 128, 16, n_q, [n + 50 for n in n_q], shared, seed=6)
    c.run()
    want, total = c.out.clone(), sum(n_q)
    q = torch.full((total + 200, 8, 128), math.nan, dtype=torch.bfloat16, device=DEV)
    q[90:90 + total] = c.q
    c.q, c.q_start = q, c.q_start + 90
    c.out = torch.full_like(q, 7.0)
    c.lse = torch.full((total + 200, 8), 7.0, device=DEV)
    c.run()
    assert int(c.status) == 0 and torch.equal(c.out[90:90 + total], want)
    assert bool((c.out[:90] == 7).all()) and bool((c.out[90 + total:] == 7).all())
    assert bool((c.lse[:90] == 7).all()) and bool((c.lse[90 + total:] == 7).all())


@pytest.mark.parametrize("shared", [1008, 70000])
def test_large_scores_and_late_maximum(shared):
    c = Case(4, 1, 64, 16, [3, 1, 20], [100, 1, 30], shared, seed=8, poison=False)
    grow = torch.linspace(0, 1, c.pool.shape[1] * c.B, device=DEV).view(1, -1, 1, 1)
    c.q = c.q * 0.1
    c.q[..., 0] = 8
    c.pool[0].view(1, -1, 1, c.D)[..., 0] = (-60 * (1 + grow[..., 0])).to(torch.bfloat16)
    c.run()
    c.check()


@pytest.mark.parametrize("shared", [208, 70000])
def test_values_past_the_prefix_and_past_a_row_have_no_effect(shared):
    c = Case(4, 1, 128, 16, [6, 1], [26, 4], shared, seed=7)
    c.run()
    clean = c.out.clone()
    p = c.ctx[0] - 6 + 3  # the position of row 3
    slot = int(c.table[0, p // 16]) * 16 + p % 16
    for plane in (0, 1):
        flat = c.pool[plane].view(-1, 1, 128)
        keep = flat[slot].clone()
        flat[slot, :, 3] = math.inf
        c.run()
        assert torch.equal(c.out[:3], clean[:3]) and torch.equal(c.out[6:], clean[6:])
        if plane:
            assert not bool(torch.isfinite(c.out[3:6, :, 3]).any())
            assert torch.equal(c.out[3:6, :, 4:], clean[3:6, :, 4:])
        flat[slot] = keep


@pytest.mark.parametrize("shared", [304, 24000])
@pytest.mark.parametrize("n_q", [[2, 3], [40, 60]])
def test_bad_requests_are_skipped(n_q, shared):
    """Keys that are fewer than the prefix, too many, rows outside q; a block of the prefix and of a request."""
    def case():
        return Case(4, 2, 128, 16, n_q + [1], [n + 40 for n in n_q] + [20], shared, seed=9)

    good = case()
    good.run()
    a, b = n_q[0], n_q[0] + n_q[1]
    for what in ("few", "many", "rows", "own block", "shared block"):
        c = case()
        if what == "few":
            c.ctx_lens[1] = shared + n_q[1] - 1
        elif what == "many":
            c.ctx_lens[1] = c.max_ctx + 1
        elif what == "rows":
            c.q_start[2] = c.q.shape[0] + 5
        elif what == "own block":
            c.table[1, shared // 16 + 1] = c.pool.shape[1]
        else:
            c.table[:, 3] = -1
        c.run()
        assert int(c.status) == kvi.ERR_OUT_OF_RANGE, what
        if what in ("few", "many"):
            assert bool((c.out[a:b] == 7).all())
        if what == "shared block":
            k = torch.cat([torch.arange(48), torch.arange(64, c.ctx[0])]).to(DEV)
            kk, v = c.kv(0, 0)
            last = torch.arange(a, device=DEV) + (c.ctx[0] - a) - 16
            ref, _, _, pv, size = ac.attend(c.q[:a, :2].double(), kk[k], v[k], last, 128 ** -0.5)
            ac.check_out(c.out[:a, :2], ref, pv, size, 1)
        elif what != "rows":
            assert torch.equal(c.out[:a], good.out[:a]) and torch.equal(c.out[-1:], good.out[-1:])
        else:
            assert torch.equal(c.out[:a], good.out[:a]) and bool((c.out[a:b] == 7).all())


@pytest.mark.parametrize("shared", [304, 32000])
def test_starts_that_are_no_starts(shared):
    """Row starts out of order or outside q: recorded, nothing written past them."""
    for starts in ([3, 1, 2, 0], [-4, 0, 1, 3], [0, 1, 2, 900], [900, 900, 900, 900]):
        c = Case(4, 2, 128, 16, [1, 1, 1], [9, 10, 11], shared, seed=9)
        c.q_start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        c.run()
        assert int(c.status) == kvi.ERR_OUT_OF_RANGE
        assert bool((c.out == 7).all()) or shared == 304  # (a request with a good start and end is attended there)


def test_no_prefix_is_the_plain_call():
    c = Case(8, 2, 128, 16, [1, 40], [700, 90], 0, seed=1)
    c.run()
    c.check()
    out = c.out.clone()
    Prompt.run(c)
    assert torch.equal(c.out, out)


def test_other_stream_and_graph():
    c = Case(8, 2, 128, 16, [5, 0, 1, 20], [70, 0, 33, 20], 16000, seed=10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    s.synchronize()
    c.check()
    ws = ac.workspace(kvi.kvi_attn_shared_workspace_bytes(c.a, 4, 26, 20, c.max_ctx, 16000))
    cache, g = kvi.paged_cache([c.pool], 16), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvi.kvi_attn_shared(c.a, c.q, c.q_start, 20, c.ctx_lens, c.max_ctx, c.table, cache, 0, 16000, c.out, ws, c.status, lse=c.lse)
    for seed in (1, 2):
        c.q.copy_(ac.randn(ac.gen(seed), *c.q.shape).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        c.check()
    c.q_start.zero_()  # a batch of padding alone: nothing is written
    c.out.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert int(c.status) == 0 and bool((c.out == 7).all())


def test_offsets_past_32_bits():
    H, D, B = 8, 128, 16
    blocks = (1 << 31) // (B * H * D) + 64
    if torch.cuda.mem_get_info()[0] < 2 * blocks * B * H * D * 2 + (4 << 30):
        pytest.skip("not enough device memory")
    c = Case(8, 8, D, B, [3, 1, 1], [50, 20, 30], 4800, seed=11, poison=False)
    pool = torch.empty(2, blocks, B, H, D, dtype=torch.bfloat16, device=DEV)
    small, table = c.pool, c.table.clone()
    used = table[table >= 0].long()
    c.table = (blocks - 1 - table).clamp(max=blocks - 1).to(torch.int32)
    pool[:, blocks - 1 - used] = small[:, used]
    c.pool = pool
    c.run()
    c.check()


def test_refusals():
    c = Case(4, 2, 64, 16, [2], [20], 64, seed=13)
    for shared in (-16, 8, 65, 96, 1 << 20):
        with pytest.raises(kvi.KviError, match="shared"):
            kvi.kvi_attn_shared(c.a, c.q, c.q_start, 2, c.ctx_lens, 84, c.table, kvi.paged_cache([c.pool], 16), 0, shared, c.out,
                                ac.workspace(1 << 20), c.status)
    n = kvi.kvi_attn_shared_workspace_bytes(c.a, 1, 2, 2, 84, 64)
    with pytest.raises(kvi.KviError, match="workspace"):
        kvi.kvi_attn_shared(c.a, c.q, c.q_start, 2, c.ctx_lens, 84, c.table, kvi.paged_cache([c.pool], 16), 0, 64, c.out,
                            ac.workspace(n)[:128], c.status)
    torch.cuda.synchronize()
    assert int(c.status) == 0
