"""The 4-bit cache: its bytes, rows in and out, the decoding step over it and
its eviction, against plain definitions in 64 bits."""
import math

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ------------------------------------------------------------- rows in and out

@pytest.mark.parametrize("H,D,B", [(1, 32, 16), (2, 64, 32), (8, 128, 16), (3, 96, 48), (2, 256, 16), (1, 160, 16), (2, 224, 64)])
def test_bytes_follow_the_layout(H, D, B):
    g = ac.gen(D + B)
    blocks = 5
    c = ac.Cache4(g, H, D, B, blocks)
    want = ac.pages_from(*ac.quantise(c.k), *ac.quantise(c.v), B)
    assert torch.equal(c.pool.cpu(), want)
    assert kvi.kvi_cache4_layer_bytes(H, D, blocks, B) == c.pool.numel()
    assert int(c.status) == 0


def test_rounding_and_special_values():
    """Exact ties, zeros, subnormals, the largest values, infinities and NaN."""
    H, D, B = 1, 64, 16
    rows = torch.zeros(16, H, D, dtype=torch.bfloat16, device=DEV)
    rows[0, 0, :32] = torch.arange(32, device=DEV) * 0.5 - 7          # step 1.289.. / 7
    rows[1, 0, :32] = (torch.arange(32, device=DEV) - 14) * 0.5        # step 1: every half is a tie
    rows[1, 0, 31] = 7.0
    rows[2, 0, :32] = torch.finfo(torch.bfloat16).max
    rows[3, 0, :32] = 1e-40                                            # subnormal
    rows[4, 0, 0] = 9.2e-41                                            # the smallest bf16
    rows[5, 0, 3] = math.inf
    rows[6, 0, 40] = math.nan
    rows[7, 0, :] = -0.0
    rows[8, 0, 5] = -math.inf
    c = ac.Cache4(ac.gen(1), H, D, B, 1, k=rows, v=rows.flip(0).contiguous())
    for x, back in ((c.k, torch.empty_like(rows)), (c.v, torch.empty_like(rows))):
        step, code = ac.quantise(x)
        ref = ac.dequantise(step, code).to(torch.bfloat16)
        kb, vb = torch.empty_like(rows), torch.empty_like(rows)
        kvi.kvi_cache4_read(c.cache, 0, torch.arange(16, device=DEV), kb, vb, c.status)
        got = kb if x is c.k else vb
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got.nan_to_num(0), ref.nan_to_num(0))
    assert bool(torch.isnan(ac.dequantise(*ac.quantise(rows))[5, 0, :32]).all())
    assert int(c.status) == 0


@pytest.mark.parametrize("T", [0, 1, 2, 63, 1000])
@pytest.mark.parametrize("H,D,B", [(2, 64, 16), (8, 128, 32), (1, 224, 16)])
def test_scattered_rows_and_strides(H, D, B, T):
    """Rows of a wider projection to random slots, some skipped; nothing else is touched."""
    g = ac.gen(T + D)
    blocks = T // B + 4
    wide = ac.randn(g, T, 2 * H, D).to(torch.bfloat16)
    k, v = wide[:, :H], wide[:, H:]
    slots = torch.randperm(blocks * B, generator=g, device=DEV)[:T]
    slots[2::3] = -1
    pool = torch.full((blocks, H, ac.page_bytes(B, D)), 0x5a, dtype=torch.uint8, device=DEV)
    cache, status = kvi.cache4([pool], B, H, D), torch.zeros(1, dtype=torch.int32, device=DEV)
    kvi.kvi_cache4_write(cache, 0, k, v, slots, status)
    live = slots >= 0
    back = torch.full((T, 2 * H + 1, D), 3.0, dtype=torch.bfloat16, device=DEV)
    kvi.kvi_cache4_read(cache, 0, slots, back[:, 1:1 + H], back[:, 1 + H:], status)
    assert bool((back[:, 0] == 3).all())
    for x, y in ((k, back[:, 1:1 + H]), (v, back[:, 1 + H:])):
        ref = ac.dequantise(*ac.quantise(x)).to(torch.bfloat16)
        assert torch.equal(y[live], ref[live])
        assert bool((y[~live] == 3).all())
    # every other slot still holds the pattern's values
    other = torch.ones(blocks * B, dtype=torch.bool, device=DEV)
    other[slots[live]] = False
    rest = other.nonzero().flatten()
    a, b = (torch.empty(len(rest), H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kvi.kvi_cache4_read(cache, 0, rest, a, b, status)
    assert a.unique().numel() <= 2 and b.unique().numel() <= 2   # nibbles 5 and 10
    assert int(status) == 0


def test_slots_beyond_the_pool():
    c = ac.Cache4(ac.gen(2), 2, 64, 16, 3)
    before = c.pool.clone()
    one = torch.ones(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    kvi.kvi_cache4_write(c.cache, 0, one, one, torch.tensor([48, -1], device=DEV), c.status)
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE and torch.equal(c.pool, before)
    c.status.zero_()
    out = torch.full_like(one, 5)
    kvi.kvi_cache4_read(c.cache, 0, torch.tensor([1 << 40, -9], device=DEV), out, out.clone(), c.status)
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE and bool((out == 5).all())


def test_converts_a_bf16_pool():
    g = ac.gen(3)
    blocks, B, H, D = 6, 16, 2, 128
    pool = ac.randn(g, 2, blocks, B, H, D).to(torch.bfloat16)
    c = ac.Cache4(g, H, D, B, blocks, k=pool[0].view(-1, H, D), v=pool[1].view(-1, H, D))
    out = torch.empty_like(pool)
    kvi.kvi_cache4_read(c.cache, 0, torch.arange(blocks * B, device=DEV), out[0].view(-1, H, D), out[1].view(-1, H, D), c.status)
    assert torch.equal(out.view(2, -1, H, D)[0], c.kd.to(torch.bfloat16))
    assert torch.equal(out.view(2, -1, H, D)[1], c.vd.to(torch.bfloat16))


@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("H,D", [(6, 64), (5, 96), (7, 128)])
def test_long_prefixes(H, D, first):
    """Enough rows that a thread takes several heads; runs of slots that pair up, broken by skipped and by lone rows."""
    g = ac.gen(H + D + first)
    B, T = 48, 24001
    blocks = T // B + 2
    slots = torch.arange(first, first + T, device=DEV)
    order = torch.randperm(blocks, generator=g, device=DEV)
    slots = order[slots // B] * B + slots % B
    slots[1000:1400:7] = -1
    slots[5000:5200] = slots[5000:5200].flip(0)
    k, v = (ac.randn(g, T, H, D).to(torch.bfloat16) for _ in range(2))
    pool = torch.zeros(blocks, H, ac.page_bytes(B, D), dtype=torch.uint8, device=DEV)
    cache, status = kvi.cache4([pool], B, H, D), torch.zeros(1, dtype=torch.int32, device=DEV)
    kvi.kvi_cache4_write(cache, 0, k, v, slots, status)
    kb, vb = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    kvi.kvi_cache4_read(cache, 0, slots, kb, vb, status)
    live = slots >= 0
    for x, y in ((k, kb), (v, vb)):
        assert torch.equal(y[live], ac.dequantise(*ac.quantise(x)).to(torch.bfloat16)[live])
        assert bool((y[~live] == 3).all())
    assert int(status) == 0


# ------------------------------------------------------------- decoding step

class Step:
    def __init__(self, Hq, H, D, B, ctx, seed=0, weights=True, wide=0):
        g = ac.gen(seed)
        self.Hq, self.H, self.D, self.B, self.ctx = Hq, H, D, B, ctx
        self.a = kvi.attention(Hq, H, D)
        self.table, blocks = ac.tables(g, ctx, B)
        self.c = ac.Cache4(g, H, D, B, blocks)
        used = torch.zeros(blocks * B, dtype=torch.bool, device=DEV)
        for r, n in enumerate(ctx):
            used[self.c.rows(self.table[r], n)] = True
        bad = (~used).nonzero().flatten()  # slots outside the requests read as NaN
        nan = torch.full((len(bad), H, D), math.nan, dtype=torch.bfloat16, device=DEV)
        kvi.kvi_cache4_write(self.c.cache, 0, nan, nan, bad, self.c.status)
        R = len(ctx)
        self.q = ac.randn(g, R, Hq + wide, D).to(torch.bfloat16)[:, :Hq]
        self.out = torch.full((R, Hq + wide, D), 7.0, dtype=torch.bfloat16, device=DEV)[:, wide:]
        self.ctx_lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.w0 = torch.rand(R, H, max(ctx) + 5, generator=g, device=DEV) if weights else None
        self.w = self.w0.clone() if weights else None

    def run(self, **kw):
        n = kvi.kvi_attn_decode4_workspace_bytes(self.a, len(self.ctx), max(self.ctx), self.w is not None)
        assert n > 0
        kvi.kvi_attn_decode4(self.a, self.q, self.ctx_lens, max(self.ctx), self.table, self.c.cache, 0, self.out,
                             ac.workspace(n), self.c.status, weights=self.w, **kw)

    def check(self):
        assert int(self.c.status) == 0
        G = self.Hq // self.H
        for r, n in enumerate(self.ctx):
            rows = self.c.rows(self.table[r], n)
            for h in range(self.H):
                hs = slice(h * G, (h + 1) * G)
                ref, _, p, pv, size = ac.attend(self.q[r:r + 1, hs].double(), self.c.kd[rows, h], self.c.vd[rows, h],
                                                torch.tensor([n - 1], device=DEV), self.D ** -0.5)
                ac.check_out(self.out[r:r + 1, hs], ref, pv, size, 2, (r, h))
                if self.w is not None:
                    add = p.sum((0, 1))
                    want = self.w0[r, h, :n].double() + add
                    err = (self.w[r, h, :n].double() - want).abs()
                    # the sum of the group's weights, each off by 2^-17 (1 + size) of itself, and one rounding
                    assert bool((err <= 2.0 ** -17 * (1 + size) * add + 2.0 ** -24 * want).all()), (r, h, float(err.max()))
                    assert torch.equal(self.w[r, h, n:], self.w0[r, h, n:])


@pytest.mark.parametrize("B", [16, 48])
@pytest.mark.parametrize("Hq,H,D", [(1, 1, 32), (4, 2, 64), (8, 8, 128), (32, 8, 128), (10, 2, 96), (40, 2, 128), (9, 1, 256),
                                    (17, 1, 160), (128, 1, 64), (6, 2, 192), (5, 5, 224), (33, 1, 32), (12, 1, 96)])
def test_decode_layouts(Hq, H, D, B):
    c = Step(Hq, H, D, B, [1, 16, 17, 0, 200, 47], seed=Hq + D)
    c.run()
    c.check()


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("ctx", [[1], [255], [256], [257], [5000], [40000], [3, 9000, 700], [64 * i + 1 for i in range(64)]])
def test_decode_lengths(ctx, weights):
    c = Step(8, 2, 128, 16, ctx, seed=len(ctx), weights=weights)
    c.run()
    c.check()


@pytest.mark.parametrize("Hq,H,D", [(8, 2, 64), (8, 2, 128), (40, 2, 128), (9, 1, 256), (6, 3, 96)])
@pytest.mark.parametrize("most", [400, 600, 1000, 1024, 2000])
def test_decode_joined_pieces(Hq, H, D, most):
    """Two to eight pieces a request without weights: requests with all of them, some, one and none."""
    ctx = [most, 1, 0, most // 2 + 3, 129, most - 1, 128]
    c = Step(Hq, H, D, 16, ctx, seed=most, weights=False)
    c.run()
    c.check()
    first = c.out.clone()
    c.run()
    assert torch.equal(c.out, first)
    # a request that is refused leaves the others as they are
    c.out.fill_(7)
    c.ctx_lens[3] = most + 1
    c.run()
    assert int(c.c.status) == kvi.ERR_OUT_OF_RANGE
    keep = [0, 1, 2, 4, 5, 6]
    assert torch.equal(c.out[keep], first[keep]) and bool((c.out[3] == 7).all())


def test_decode_strides_stream_and_graph():
    c = Step(8, 2, 64, 16, [700, 33], seed=4, wide=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    s.synchronize()
    c.check()
    assert bool((c.out._base[:, :3] == 7).all())
    n = kvi.kvi_attn_decode4_workspace_bytes(c.a, 2, 700, True)
    ws = ac.workspace(n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvi.kvi_attn_decode4(c.a, c.q, c.ctx_lens, 700, c.table, c.c.cache, 0, c.out, ws, c.c.status, weights=c.w)
    for seed in (1, 2):
        c.q.copy_(ac.randn(ac.gen(seed), *c.q.shape).to(torch.bfloat16))
        c.w.copy_(c.w0)
        g.replay()
        torch.cuda.synchronize()
        c.check()


def test_decode_accumulates_and_repeats():
    c = Step(8, 1, 128, 16, [1500], seed=5)
    c.run()
    once, out = c.w.clone(), c.out.clone()
    c.run()
    assert torch.equal(c.out, out)
    add = once - c.w0
    assert torch.allclose(c.w, once + add, rtol=1e-6, atol=0)
    # the group's weights sum to its heads
    assert abs(float(add.double().sum()) - 8) < 1e-3


def test_decode_bad_requests():
    c = Step(4, 2, 64, 16, [300, 40, 500], seed=6)
    good = Step(4, 2, 64, 16, [300, 40, 500], seed=6)
    good.run()
    c.ctx_lens[1] = 501
    c.run()
    assert int(c.c.status) == kvi.ERR_OUT_OF_RANGE
    assert torch.equal(c.out[0], good.out[0]) and torch.equal(c.out[2], good.out[2]) and bool((c.out[1] == 7).all())
    assert torch.equal(c.w[1], c.w0[1])
    c = Step(4, 2, 64, 16, [300, 40, 500], seed=6)
    c.table[0, 2] = -1
    c.run()
    assert int(c.c.status) == kvi.ERR_OUT_OF_RANGE
    rows = torch.cat([c.c.rows(good.table[0], 300)[:32], c.c.rows(good.table[0], 300)[48:]])
    ref, _, _, pv, size = ac.attend(c.q[:1, :2].double(), c.c.kd[rows, 0], c.c.vd[rows, 0], torch.tensor([283], device=DEV), 0.125)
    ac.check_out(c.out[:1, :2], ref, pv, size, 2)
    assert torch.equal(c.w[0, :, 32:48], c.w0[0, :, 32:48])


def test_decode_nan_rows():
    """A stored NaN reaches every head that reads it, and no other request."""
    c = Step(4, 1, 64, 16, [100, 100], seed=7)
    c.run()
    clean = c.out.clone()
    x = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    x[0, 0, 40] = math.inf
    kvi.kvi_cache4_write(c.c.cache, 0, c.c.k[:1], x, c.c.rows(c.table[0], 100)[50:51], c.c.status)
    c.run()
    assert bool(torch.isnan(c.out[0, :, 32:]).all()) and not bool(torch.isnan(c.out[0, :, :32]).any())
    assert torch.equal(c.out[1], clean[1])


def test_decode_offsets_past_32_bits():
    H, D, B = 8, 128, 16
    one = ac.page_bytes(B, D)
    blocks = (1 << 32) // (H * one) + 64
    if torch.cuda.mem_get_info()[0] < blocks * H * one + (4 << 30):
        pytest.skip("not enough device memory")
    c = Step(8, 8, D, B, [600], seed=8)
    pool = torch.empty(blocks, H, one, dtype=torch.uint8, device=DEV)
    far = (blocks - 1 - c.table).to(torch.int32)
    pool[far[0].long()] = c.c.pool[c.table[0].long()]
    cache = kvi.cache4([pool], B, H, D)
    n = kvi.kvi_attn_decode4_workspace_bytes(c.a, 1, 600, True)
    kvi.kvi_attn_decode4(c.a, c.q, c.ctx_lens, 600, far, cache, 0, c.out, ac.workspace(n), c.c.status, weights=c.w)
    c.check()
    # and rows in and out at the far end
    slots = far[0, :4].long() * B + 3
    x = ac.randn(ac.gen(1), 4, H, D).to(torch.bfloat16)
    kvi.kvi_cache4_write(cache, 0, x, x, slots, c.c.status)
    k, v = torch.empty_like(x), torch.empty_like(x)
    kvi.kvi_cache4_read(cache, 0, slots, k, v, c.c.status)
    assert torch.equal(k, ac.dequantise(*ac.quantise(x)).to(torch.bfloat16)) and torch.equal(k, v)
    assert int(c.c.status) == 0


# ------------------------------------------------------------------- eviction

def evict_reference(w, pos, n, budget, sink, recent):
    """Slots that end up at 0 .. min(n, budget)-1, by the definition."""
    if n <= budget:
        return list(range(n))
    newest = max(pos[:n])

    def rank(i):
        safe = pos[i] < sink or pos[i] > newest - recent
        x = w[i]
        return (not safe, 0 if math.isnan(x) else 1, 0.0 if math.isnan(x) else -x, i)

    kept = set(sorted(range(n), key=rank)[:budget])
    tail = iter(i for i in range(budget, n) if i in kept)
    return [i if i in kept else next(tail) for i in range(budget)]


def run_evict(c, ctx, budget, sink, recent, w, pos, max_ctx=None):
    R, H = len(ctx), c.H
    table = c.table
    lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    w_out, pos_out = torch.full_like(w, -3.0), torch.full_like(pos, -3)
    out = torch.full_like(lens, -3)
    most = max(ctx) if max_ctx is None else max_ctx
    ws = ac.workspace(kvi.kvi_cache4_evict_workspace_bytes(H, R, most))
    kvi.kvi_cache4_evict(c.c.cache, 0, lens, most, table, budget, sink, recent, w, pos, w_out, pos_out, out, ws, c.c.status)
    return w_out, pos_out, out


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special"])
@pytest.mark.parametrize("H,D,B,ctx,budget,sink,recent", [
    (2, 64, 16, [100, 30, 0, 31, 1], 30, 4, 8), (1, 128, 16, [2500], 1024, 4, 64), (3, 96, 48, [500, 400], 499, 0, 0),
    (2, 32, 16, [1100, 1025], 1, 0, 1), (1, 256, 16, [90], 80, 10, 70), (2, 64, 16, [3000, 2000], 1500, 0, 1500),
    (2, 32, 32, [7000, 4097], 4000, 4, 64), (1, 32, 64, [30001, 8193, 26000], 8192, 4, 64)])
def test_evict(H, D, B, ctx, budget, sink, recent, kind):
    c = Step(H, H, D, B, ctx, seed=budget)
    g = ac.gen(budget + len(kind))
    R, width = len(ctx), max(ctx) + 3
    w = torch.rand(R, H, width, generator=g, device=DEV)
    if kind == "ties":
        w = torch.floor(w * 4) - 1                          # -1, 0, 1, 2: many of each
        w[w == 0] *= -1.0                                   # and zeros of both signs
        w[..., ::2] = w[..., ::2].abs()
    elif kind == "equal":
        w.zero_()
    elif kind == "special":
        w[..., ::7] = math.inf
        w[..., 1::11] = math.nan
        w[..., 2::5] = -math.inf
        w[..., 3::5] = 1e-42
    pos = torch.stack([torch.stack([torch.randperm(width, generator=g, device=DEV) for _ in range(H)]) for _ in range(R)])
    pos = pos.to(torch.int32)
    before = c.c.pool.clone()
    w_out, pos_out, out = run_evict(c, ctx, budget, sink, recent, w, pos)
    assert int(c.c.status) == 0
    kb = torch.empty(before.shape[0] * B, H, D, dtype=torch.bfloat16, device=DEV)
    vb = torch.empty_like(kb)
    kvi.kvi_cache4_read(c.c.cache, 0, torch.arange(kb.shape[0], device=DEV), kb, vb, c.c.status)
    wc, pc = w.cpu(), pos.cpu()
    for r, n in enumerate(ctx):
        left = min(n, budget)
        assert int(out[r]) == left
        rows = c.c.rows(c.table[r], n)
        for h in range(H):
            src = torch.tensor(evict_reference(wc[r, h].tolist(), pc[r, h].tolist(), n, budget, sink, recent), dtype=torch.long)
            assert torch.equal(pos_out[r, h, :left].cpu(), pc[r, h, src])
            assert torch.equal(w_out[r, h, :left].cpu().view(torch.int32), wc[r, h, src].view(torch.int32))
            assert bool((pos_out[r, h, left:n] == -1).all()) and bool((w_out[r, h, left:n] == 0).all())
            assert bool((pos_out[r, h, n:] == -3).all()) and bool((w_out[r, h, n:] == -3).all())
            at = rows[src.to(DEV)] if left else rows[:0]
            assert torch.equal(kb[rows[:left], h], c.c.kd[at, h].to(torch.bfloat16))
            assert torch.equal(vb[rows[:left], h], c.c.vd[at, h].to(torch.bfloat16))
            # rows at or past the budget are never written
            assert torch.equal(kb[rows[left:], h], c.c.kd[rows[left:], h].to(torch.bfloat16))


@pytest.mark.parametrize("H,ctx,budget", [(64, [300, 290], 150), (43, [700, 200, 701], 333), (2, [300], 150)])
def test_evict_many_rows(H, ctx, budget):
    """Many heads, whose blocks move their own rows, and few, whose rows a second kernel moves."""
    c = Step(H, H, 32, 16, ctx, seed=H)
    w = torch.rand(len(ctx), H, max(ctx) + 1, generator=ac.gen(H), device=DEV)
    pos = torch.arange(max(ctx) + 1, dtype=torch.int32, device=DEV).expand(len(ctx), H, -1).contiguous()
    w_out, pos_out, out = run_evict(c, ctx, budget, 4, 16, w, pos)
    assert int(c.c.status) == 0 and out.tolist() == [min(n, budget) for n in ctx]
    wc, pc = w.cpu(), pos.cpu()
    for r, n in enumerate(ctx):
        left = min(n, budget)
        rows = c.c.rows(c.table[r], n)
        k, v = (torch.empty(left, H, 32, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kvi.kvi_cache4_read(c.c.cache, 0, rows[:left], k, v, c.c.status)
        for h in range(H):
            src = torch.tensor(evict_reference(wc[r, h].tolist(), pc[r, h].tolist(), n, budget, 4, 16), dtype=torch.long)
            assert torch.equal(pos_out[r, h, :left].cpu(), pc[r, h, src])
            assert torch.equal(k[:, h], c.c.kd[rows[src.to(DEV)], h].to(torch.bfloat16))
            assert torch.equal(v[:, h], c.c.vd[rows[src.to(DEV)], h].to(torch.bfloat16))


def test_evict_then_attend():
    """After an eviction the decoding step sees exactly the kept keys."""
    c = Step(8, 2, 128, 16, [900, 400], seed=21)
    g = ac.gen(22)
    w = torch.rand(2, 2, 905, generator=g, device=DEV)
    pos = torch.arange(905, dtype=torch.int32, device=DEV).expand(2, 2, -1).contiguous()
    w_out, pos_out, out = run_evict(c, [900, 400], 512, 4, 32, w, pos)
    n = kvi.kvi_attn_decode4_workspace_bytes(c.a, 2, 512, True)
    base = w_out.clone()
    kvi.kvi_attn_decode4(c.a, c.q, out, 512, c.table, c.c.cache, 0, c.out, ac.workspace(n), c.c.status, weights=w_out)
    assert int(c.c.status) == 0 and out.tolist() == [512, 400]
    for r in range(2):
        for h in range(2):
            keys = pos_out[r, h, :int(out[r])].long()
            assert len(set(keys.tolist())) == len(keys) and (r == 1 or keys[:4].tolist() == [0, 1, 2, 3])
            rows = c.c.rows(c.table[r], c.ctx[r])[keys]
            ref, _, p, pv, size = ac.attend(c.q[r:r + 1, 4 * h:4 * h + 4].double(), c.c.kd[rows, h], c.c.vd[rows, h],
                                            torch.tensor([len(rows) - 1], device=DEV), 128 ** -0.5)
            ac.check_out(c.out[r:r + 1, 4 * h:4 * h + 4], ref, pv, size, 2)
            add = p.sum((0, 1))
            err = (w_out[r, h, :len(rows)].double() - base[r, h, :len(rows)].double() - add).abs()
            assert bool((err <= 2.0 ** -17 * (1 + size) * add + 2.0 ** -23).all())


def test_evict_is_a_function_of_its_inputs():
    """The same call on the same inputs again (the moved rows are in place already) gives the same."""
    c = Step(2, 2, 64, 16, [800], seed=23)
    w = torch.rand(1, 2, 800, generator=ac.gen(1), device=DEV)
    pos = torch.arange(800, dtype=torch.int32, device=DEV).expand(1, 2, -1).contiguous()
    first = run_evict(c, [800], 333, 4, 16, w, pos)
    pool = c.c.pool.clone()
    again = run_evict(c, [800], 333, 4, 16, w, pos)
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and torch.equal(c.c.pool, pool)


def test_evict_bad_requests():
    c = Step(2, 2, 64, 16, [300, 200], seed=24)
    w = torch.rand(2, 2, 310, generator=ac.gen(1), device=DEV)
    pos = torch.arange(310, dtype=torch.int32, device=DEV).expand(2, 2, -1).contiguous()
    w_out, pos_out, out = run_evict(c, [301, 200], 100, 4, 16, w, pos, max_ctx=300)
    assert int(c.c.status) == kvi.ERR_OUT_OF_RANGE
    assert out.tolist() == [-3, 100] and bool((w_out[0] == -3).all()) and bool((pos_out[1, :, :100] >= 0).all())
    c.c.status.zero_()
    before = c.c.pool.clone()
    c.table[0, 0] = 10 ** 6
    run_evict(c, [300, 0], 100, 0, 0, w, pos)
    assert int(c.c.status) == kvi.ERR_OUT_OF_RANGE
    assert torch.equal(c.c.pool[c.table[0, 8:19].long()], before[c.table[0, 8:19].long()])


def test_refusals():
    c = Step(4, 2, 64, 16, [40], seed=9)
    R, H, S = 1, 2, 45
    w, pos = torch.zeros(R, H, S, device=DEV), torch.zeros(R, H, S, dtype=torch.int32, device=DEV)
    lens = c.ctx_lens

    def refused(f):
        with pytest.raises(kvi.KviError) as e:
            f()
        assert e.value.status == kvi.ERR_INVALID_ARG
        return kvi.kvi_last_error()

    def evict(**kw):
        d = dict(max_ctx=40, budget=20, sink=1, recent=2, w_out=w.clone(), pos_out=pos.clone(), out=lens.clone(),
                 ws=ac.workspace(kvi.kvi_cache4_evict_workspace_bytes(H, R, 40)), layer=0)
        d.update(kw)
        return refused(lambda: kvi.kvi_cache4_evict(c.c.cache, d["layer"], lens, d["max_ctx"], c.table, d["budget"], d["sink"],
                                                    d["recent"], w, pos, d["w_out"], d["pos_out"], d["out"], d["ws"], c.c.status))

    assert "budget" in evict(budget=0)
    assert "budget" in evict(sink=19, recent=2)
    assert "budget" in evict(sink=-1)
    assert "other buffers" in evict(w_out=w)
    assert "other buffers" in evict(pos_out=pos)
    assert "other buffers" in evict(out=lens)
    assert "max_ctx" in evict(max_ctx=46)
    assert "workspace" in evict(ws=ac.workspace(256))
    assert "layer" in evict(layer=1)

    def step(**kw):
        d = dict(a=c.a, max_ctx=40, layer=0, q=c.q, out=c.out, ws=ac.workspace(1 << 20), w=None)
        d.update(kw)
        return refused(lambda: kvi.kvi_attn_decode4(d["a"], d["q"], lens, d["max_ctx"], c.table, c.c.cache, d["layer"], d["out"],
                                                    d["ws"], c.c.status, weights=d["w"]))

    assert "layer" in step(layer=3)
    assert "max_ctx" in step(max_ctx=-1)
    assert "weights_stride" in step(max_ctx=46, w=w)
    assert "workspace" in step(ws=ac.workspace(1 << 20)[8:])
    assert "scale" in step(a=kvi.attention(4, 2, 64, scale=-1.0))
    with pytest.raises(ValueError):
        step(q=c.q.float())
    one = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    slot = torch.zeros(1, dtype=torch.int64, device=DEV)
    assert "layer" in refused(lambda: kvi.kvi_cache4_write(c.c.cache, 1, one, one, slot, c.c.status))
    assert "4-bit cache" in refused(lambda: kvi.kvi_cache4_write(
        kvi.cache4([c.c.pool], 17, 2, 64), 0, one, one, slot, c.c.status))
    assert "head_dim" in refused(lambda: kvi.kvi_cache4_write(
        kvi.cache4([c.c.pool], 16, 2, 48), 0, one.new_zeros(1, 2, 48), one.new_zeros(1, 2, 48), slot, c.c.status))
    with pytest.raises(ValueError):
        kvi.cache4([c.c.pool, c.c.pool[:1]], 16, 2, 64)
    assert kvi.kvi_cache4_layer_bytes(2, 40, 4, 16) == 0 and kvi.kvi_cache4_layer_bytes(2, 64, 4, 8) == 0
    assert kvi.kvi_attn_decode4_workspace_bytes(kvi.attention(4, 2, 80), 1, 10, False) == 0
    assert kvi.kvi_attn_prompt_workspace_bytes(kvi.attention(4, 3, 64), 1, 1, 1, 1) == 0
    assert kvi.kvi_cache4_evict_workspace_bytes(2, 0, 10) == 0
    torch.cuda.synchronize()
    assert int(c.c.status) == 0
