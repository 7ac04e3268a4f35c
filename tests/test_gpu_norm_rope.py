"""kvi_norm_rope against the definition in float64: head sizes and layouts, both
pairings, Llama 3.1 frequencies, an engine's table, rows in place and in wider
rows, pages and padding, and keys without a norm against kvi_inject_paged_ex.

Tolerance: one rounding of a result to bf16 (2^-8 of it) and float32 before it: the
sum of squares and its root within 2^-20, two products and the rotation's sums with
them, together below 2^-18 of the pair's |a| + |b|, and below the smallest normal
number where a result is next to zero."""
import math

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests import step_check as sc

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def close(got, ref, both):
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -18 * both + 2.0 ** -126
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), (int((err > tol).sum()), float((err / tol).max()), (err / tol).argmax())


class Case:
    def __init__(self, T, Hq, H, D, B=16, norm=True, interleaved=False, llama3=None, fused=True, pages=True, top=40000,
                 theta=5e5, seed=0, eps=1e-6):
        g = ac.gen(seed)
        self.T, self.Hq, self.H, self.D, self.B, self.eps, self.top = T, Hq, H, D, B, eps, top
        self.a = kvi.attention(Hq, H, D)
        self.interleaved, self.llama3, self.theta = interleaved, llama3, theta
        self.spec = kvi.rope(theta=theta, pairing=kvi.ROPE_PAIR_INTERLEAVED if interleaved else kvi.ROPE_PAIR_HALF, llama3=llama3)
        qkv = (ac.randn(g, T, Hq + 2 * H, D) * torch.exp(ac.randn(g, Hq + 2 * H, D))).to(BF)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.wq, self.wk = ((1 + 0.3 * ac.randn(g, D)).to(BF) if norm else None for _ in range(2))
        self.pos = torch.randint(0, top, (T,), generator=g, device=DEV).to(torch.int32)
        self.pos[T // 2] = 0
        self.q_out = torch.full((T, Hq, D), 7.0, dtype=BF, device=DEV)
        self.k_out, self.plain = (torch.full((T, H, D), 7.0, dtype=BF, device=DEV) for _ in range(2))
        self.pool = self.cache = self.slots = None
        if pages:
            blocks = (T + B - 1) // B + 2
            self.pool = torch.full((2, blocks, B, H, D), 7.0, dtype=BF, device=DEV)
            self.slots = torch.randperm(blocks * B, generator=g, device=DEV)[:T]
            self.slots[::5] = -1 - self.slots[::5]
            self.cache = kvi.paged_cache([self.pool], B)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, **kw):
        d = dict(q=self.q, k=self.k, q_out=self.q_out, k_out=self.k_out, k_plain=self.plain, v=self.v if self.cache else None,
                 cache=self.cache, slots=self.slots)
        d.update(kw)
        kvi.kvi_norm_rope(self.a, self.spec, self.top, self.pos, d["q"], d["k"], d["q_out"], d["k_out"], self.status,
                          q_weight=self.wq, k_weight=self.wk, eps=self.eps, k_plain=d["k_plain"], v=d["v"], cache=d["cache"],
                          slots=d["slots"], stream=kw.get("stream"))

    def reference(self, x, w):
        y = sc.normed(x, w, self.eps)
        return y, *sc.rotated(y, self.pos, sc.frequencies(self.theta, self.D, self.llama3), self.interleaved)

    def check(self, q=None, k=None):
        assert int(self.status) == 0
        _, ref, both = self.reference(self.q if q is None else q, self.wq)
        close(self.q_out, ref, both)
        y, ref, both = self.reference(self.k if k is None else k, self.wk)
        close(self.k_out, ref, both)
        close(self.plain, y, y.abs())
        if self.pool is not None:
            flat, live = self.pool.view(2, -1, self.H, self.D), self.slots >= 0
            assert torch.equal(flat[0, self.slots[live]], self.k_out[live])
            assert torch.equal(flat[1, self.slots[live]], self.v[live])
            rest = torch.ones(flat.shape[1], dtype=torch.bool, device=DEV)
            rest[self.slots[live]] = False
            assert bool((flat[:, rest] == 7).all()), "written outside the rows' slots"


@pytest.mark.parametrize("T", [1, 3, 67, 900])
@pytest.mark.parametrize("norm,interleaved", [(True, False), (True, True), (False, False), (False, True)])
@pytest.mark.parametrize("Hq,H,D", [(1, 1, 16), (3, 1, 80), (4, 2, 64), (32, 8, 128), (10, 2, 96), (6, 1, 256), (40, 2, 32), (14, 2, 144),
                                    (33, 11, 48), (128, 1, 112)])
def test_layouts(Hq, H, D, norm, interleaved, T):
    c = Case(T, Hq, H, D, norm=norm, interleaved=interleaved, seed=D + T, fused=T != 3, B=5 if D == 80 else 16)
    c.run()
    c.check()


@pytest.mark.parametrize("T", [5, 2500])
def test_llama3_frequencies_and_far_positions(T):
    c = Case(T, 8, 2, 128, llama3=(8.0, 1.0, 4.0, 8192.0), top=131072, seed=1)
    c.run()
    c.check()


def test_an_engines_own_table():
    rows, D = 300, 64
    ang = torch.outer(torch.arange(rows, dtype=torch.float64), 1e4 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D))
    cos, sin = ang.cos().float().contiguous(), ang.sin().float().contiguous()
    c = Case(200, 4, 2, D, top=rows, theta=1e4, seed=2)
    c.spec = kvi.rope(cos_table=cos, sin_table=sin, table_id=771)
    c.run()
    y = sc.normed(c.k, c.wk, c.eps)
    a, b = y.chunk(2, -1)
    cc, ss = (t.to(DEV).double()[c.pos.long()][:, None] for t in (cos, sin))
    close(c.k_out, torch.cat([a * cc - b * ss, b * cc + a * ss], -1), torch.cat([a.abs() + b.abs()] * 2, -1))
    c.pos[3], c.top = rows, 1 << 20  # its rows are all there are
    c.run()
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE


@pytest.mark.parametrize("D", [64, 128, 80])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("llama3", [None, (8.0, 1.0, 4.0, 8192.0)])
def test_unnormalised_keys_are_those_of_an_injection(D, interleaved, llama3):
    H, N, length, B = 2, 40, 7, 16
    T = N * length
    c = Case(T, 4, H, D, norm=False, interleaved=interleaved, llama3=llama3, fused=False, pages=False, seed=3)
    start = torch.randperm(N, device=DEV).to(torch.int32) * length
    c.pos = (start[:, None] + torch.arange(length, device=DEV)).flatten().to(torch.int32)
    kv = torch.stack([c.k, c.v])[None].contiguous()  # [1][2][T][H][D]
    emb, first = torch.zeros(N, 4, device=DEV), torch.arange(N, device=DEV) * length
    lens, ids = torch.full((N,), length, dtype=torch.int32, device=DEV), torch.arange(N, dtype=torch.int32, device=DEV)
    view = kvi.store_view(kvi.geometry(1, H, D, 4), kv, emb, first, lens)
    blocks = T // B + 1
    inj, own = (torch.full((2, blocks, B, H, D), 7.0, dtype=BF, device=DEV) for _ in range(2))
    table = torch.randperm(blocks, device=DEV).to(torch.int32)
    kvi.kvi_inject_paged_ex(view, ids, start, N, table, blocks,
                            kvi.paged_cache([inj], B), c.spec, c.status)
    slots = table[c.pos.long() // B].long() * B + c.pos % B
    c.run(cache=kvi.paged_cache([own], B), slots=slots, v=c.v)
    assert int(c.status) == 0 and torch.equal(own, inj)


@pytest.mark.parametrize("T", [3, 700])
def test_in_place_and_keys_alone(T):
    c = Case(T, 8, 2, 128, seed=4)
    c.run()
    c.check()
    other = Case(T, 8, 2, 128, seed=4)
    q, k = other.q.clone(), other.k.clone()
    other.run(q_out=other.q, k_out=other.k)
    assert torch.equal(other.q, c.q_out) and torch.equal(other.k, c.k_out) and torch.equal(other.pool, c.pool)
    assert torch.equal(other.v, c.v)
    other.k.copy_(k)
    other.run(q=None, q_out=None, k_out=None, k_plain=other.k)  # normalised in place, rotated into the pages
    assert torch.equal(other.k, c.plain) and torch.equal(other.pool, c.pool) and torch.equal(q, c.q)


def test_heads_of_any_size():
    """Squares beyond float32, next to nothing, zeros, and heads with an infinity or NaN."""
    c = Case(8, 4, 2, 128, pages=False, fused=False, seed=5)
    c.k[0] *= 1e30
    c.k[1] *= 1e-30
    c.k[2] = 0
    c.k[3, :, 5] = 3e38
    c.k[4, 0, 7], c.k[4, 1, 9] = math.inf, math.nan
    c.run()
    assert int(c.status) == 0
    y, ref, both = c.reference(c.k, c.wk)
    rows = torch.tensor([0, 1, 2, 3, 5, 6, 7], device=DEV)
    close(c.k_out[rows], ref[rows], both[rows])
    close(c.plain[rows], y[rows], y[rows].abs())
    assert bool(torch.isnan(c.k_out[4]).all()) and bool(torch.isnan(c.plain[4]).all())
    assert bool((c.k_out[2] == 0).all())


@pytest.mark.parametrize("T", [6, 700])
def test_bad_positions_and_slots(T):
    c = Case(T, 8, 2, 64, seed=6)
    good = Case(T, 8, 2, 64, seed=6)
    good.run()
    c.pos[1], c.pos[4] = -1, c.top
    c.run()
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE
    rows = torch.tensor([r for r in range(T) if r not in (1, 4)], device=DEV)
    assert bool((c.q_out[[1, 4]] == 7).all()) and bool((c.k_out[[1, 4]] == 7).all()) and bool((c.plain[[1, 4]] == 7).all())
    assert torch.equal(c.q_out[rows], good.q_out[rows]) and torch.equal(c.k_out[rows], good.k_out[rows])
    assert bool((c.pool.view(2, -1, 2, 64)[:, c.slots[1]] == 7).all())
    c = Case(T, 8, 2, 64, seed=6)
    c.slots[2] = c.pool.shape[1] * 16
    c.run()
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE
    assert torch.equal(c.q_out, good.q_out) and torch.equal(c.k_out, good.k_out)


def test_other_stream_and_graph():
    c = Case(300, 8, 2, 128, seed=7)
    kvi.kvi_prepare_rope_ex(c.spec, 128, c.top)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    s.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for seed in (1, 2):
        c.q.copy_(ac.randn(ac.gen(seed), *c.q.shape).to(BF))
        c.pos.copy_(torch.randint(0, c.top, (300,), generator=ac.gen(seed), device=DEV).to(torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.check()
    table_missing = kvi.rope(theta=12345.678)
    g = torch.cuda.CUDAGraph()
    with pytest.raises(kvi.KviError, match="capture"):
        with torch.cuda.graph(g):
            kvi.kvi_norm_rope(c.a, table_missing, c.top, c.pos, c.q, c.k, c.q_out, c.k_out, c.status)


def test_slots_past_32_bits():
    H, D, B = 8, 128, 16
    blocks = (1 << 31) // (B * H * D) + 64
    if torch.cuda.mem_get_info()[0] < 2 * blocks * B * H * D * 2 + (4 << 30):
        pytest.skip("not enough device memory")
    c = Case(40, 8, H, D, seed=8, pages=False)
    c.pool = torch.empty(2, blocks, B, H, D, dtype=BF, device=DEV)
    slots = blocks * B - 1 - torch.arange(40, device=DEV)
    c.run(cache=kvi.paged_cache([c.pool], B), slots=slots, v=c.v)
    assert int(c.status) == 0
    flat = c.pool.view(2, -1, H, D)
    assert torch.equal(flat[0, slots], c.k_out) and torch.equal(flat[1, slots], c.v)


def test_no_rows():
    c = Case(4, 4, 2, 64, seed=9)
    e = c.pos[:0]
    kvi.kvi_norm_rope(c.a, c.spec, 10, e, c.q[:0], c.k[:0], c.q_out[:0], c.k_out[:0], c.status)
    torch.cuda.synchronize()
    assert int(c.status) == 0 and bool((c.q_out == 7).all())
