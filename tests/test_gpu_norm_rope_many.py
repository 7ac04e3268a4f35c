"""kvi_norm_rope on many rows, where a warp stays with a part of the rows and bulk copies
bring its next ones: a warp has nine rows or more here, so that every stage of its
ring is used again.  Head sizes, parts that heads do not fill, one weight or none,
rows in place, and rows that are skipped.  Tolerances are those of the other sizes."""
import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests.test_gpu_norm_rope import Case, close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
T = 8191  # rows; warps for a part of them: 4 * 456 / parts, so 912 at most where there are two parts

LAYOUTS = [(4, 2, 64), (20, 4, 64), (36, 9, 64), (32, 8, 128), (10, 2, 128), (33, 11, 128), (17, 1, 128), (6, 1, 256), (9, 3, 256)]


def weigh(c, weights):
    """Both weights, one, or none."""
    if "q" not in weights:
        c.wq = None
    if "k" not in weights:
        c.wk = None
    return c


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", ["qk", "q", "k", ""])
@pytest.mark.parametrize("Hq,H,D", LAYOUTS)
def test_layouts(Hq, H, D, weights, interleaved):
    c = weigh(Case(T, Hq, H, D, interleaved=interleaved, seed=Hq + D), weights)
    c.run()
    c.check()


@pytest.mark.parametrize("weights", ["qk", ""])
@pytest.mark.parametrize("Hq,H,D", [(20, 4, 64), (33, 11, 128), (9, 3, 256)])
def test_outputs_of_every_kind(Hq, H, D, weights):
    """Rows alone, keys alone, pages alone, and a fact store's keys alone give the bits of all together; twice the same."""
    c = weigh(Case(T, Hq, H, D, seed=Hq), weights)
    c.run()
    c.check()
    for kw in (dict(), dict(v=None, cache=None, slots=None), dict(q=None, q_out=None), dict(k_out=None, k_plain=None), dict(k_plain=None),
               dict(q=None, q_out=None, k_out=None, v=None, cache=None, slots=None)):
        o = weigh(Case(T, Hq, H, D, seed=Hq), weights)
        o.run(**kw)
        assert int(o.status) == 0
        for name, arg in (("q_out", "q_out"), ("k_out", "k_out"), ("plain", "k_plain"), ("pool", "cache")):
            got, given = getattr(o, name), arg not in kw
            assert torch.equal(got, getattr(c, name)) if given else bool((got == 7).all()), (name, kw)


@pytest.mark.parametrize("Hq,H,D", [(20, 4, 64), (10, 2, 128), (9, 3, 256)])
def test_in_place(Hq, H, D):
    c = Case(T, Hq, H, D, seed=4)
    c.run()
    o = Case(T, Hq, H, D, seed=4)
    v = o.v.clone()
    o.run(q_out=o.q, k_out=o.k)
    assert int(o.status) == 0
    assert torch.equal(o.q, c.q_out) and torch.equal(o.k, c.k_out) and torch.equal(o.plain, c.plain)
    assert torch.equal(o.pool, c.pool) and torch.equal(o.v, v)
    o = Case(T, Hq, H, D, seed=4)
    q = o.q.clone()
    o.run(q=None, q_out=None, k_out=None, k_plain=o.k)  # normalised in place, rotated into the pages
    assert torch.equal(o.k, c.plain) and torch.equal(o.pool, c.pool) and torch.equal(o.q, q)


@pytest.mark.parametrize("Hq,H,D", [(20, 4, 64), (10, 2, 128), (9, 3, 256)])
def test_rows_that_are_skipped(Hq, H, D):
    """Positions out of range, and slots beyond the pool, in every stage."""
    good = Case(T, Hq, H, D, seed=6)
    good.run()
    c = Case(T, Hq, H, D, seed=6)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[::97] = bad[5::911] = bad[-1] = True
    c.pos[bad] = c.top
    c.pos[::291] = -1
    c.run()
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE
    for name in ("q_out", "k_out", "plain"):
        got = getattr(c, name)
        assert bool((got[bad] == 7).all()) and torch.equal(got[~bad], getattr(good, name)[~bad]), name
    want, live = good.pool.clone().view(2, -1, H, D), c.slots >= 0
    want[:, c.slots[bad & live]] = 7
    assert torch.equal(c.pool.view(2, -1, H, D), want)
    c = Case(T, Hq, H, D, seed=6)
    slots = c.slots.clone()
    c.slots[bad] = c.pool.shape[1] * c.B + torch.arange(T, device=DEV)[bad]
    c.run()
    assert int(c.status) == kvi.ERR_OUT_OF_RANGE
    assert torch.equal(c.q_out, good.q_out) and torch.equal(c.k_out, good.k_out) and torch.equal(c.plain, good.plain)
    want = good.pool.clone().view(2, -1, H, D)
    want[:, slots[bad & (slots >= 0)]] = 7
    assert torch.equal(c.pool.view(2, -1, H, D), want)


def test_rows_of_a_wide_projection_in_a_graph_on_another_stream():
    """Rows with others between them; each replay has its own rows, positions and slots."""
    c = Case(T, 20, 4, 64, seed=8)
    kvi.kvi_prepare_rope_ex(c.spec, 64, c.top)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    s.synchronize()
    with torch.cuda.graph(g, stream=s):
        c.run()
    for seed in (1, 2):
        r = ac.gen(seed)
        c.q.copy_(ac.randn(r, *c.q.shape).to(BF))
        c.k.copy_(ac.randn(r, *c.k.shape).to(BF))
        c.pos.copy_(torch.randint(0, c.top, (T,), generator=r, device=DEV).to(torch.int32))
        c.slots.copy_(c.slots.flip(0))
        c.pool.fill_(7)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        c.check()


def test_heads_of_any_size():
    """Squares beyond float32, next to nothing and zeros, and heads with an infinity or NaN, in every stage."""
    c = Case(T, 4, 2, 128, pages=False, fused=False, seed=5)
    c.k[0::7] *= 1e30
    c.k[1::7] *= 1e-30
    c.k[2::7] = 0
    c.k[3::7, :, 5] = 3e38
    c.k[4::7, 0, 7], c.k[4::7, 1, 9] = float("inf"), float("nan")
    c.run()
    assert int(c.status) == 0
    y, ref, both = c.reference(c.k, c.wk)
    rows = torch.arange(T, device=DEV) % 7 != 4
    close(c.k_out[rows], ref[rows], both[rows])
    close(c.plain[rows], y[rows], y[rows].abs())
    assert bool(torch.isnan(c.k_out[~rows]).all()) and bool(torch.isnan(c.plain[~rows]).all())
    assert bool((c.k_out[2::7] == 0).all())
