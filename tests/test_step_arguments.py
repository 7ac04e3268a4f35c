"""What the calls of a serving step refuse, without a GPU: every call here lacks its
status word or has another fault that is refused, so that nothing is launched."""
import random

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from pre_rope_kv_gb300 import build as kbuild
from tests.test_attn_arguments import WS, bf16, cache4, grows, i32


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kvi.load_library()


def i64(*shape):
    return torch.zeros(*shape, dtype=torch.int64)


POOL = bf16(2, 4, 16, 2, 64)


def attend(call, last, cache=None, lse=None, ws=WS, q=None, max_ctx=50, status=None, **kw):
    kw = {"R": 1, "table": i32(1, 4), **kw}
    q = bf16(3, 4, 64) if q is None else q
    call(kvi.attention(4, 2, 64), q, i32(kw["R"] + 1), 3, i32(kw["R"]), max_ctx, kw["table"], cache or kvi.paged_cache([POOL], 16), 0,
         *last, bf16(3, 4, 64), ws, status, lse=lse, stream=0)


@pytest.mark.parametrize("call,last", [(kvi.kvi_attn_window, (5, 1)), (kvi.kvi_attn_shared, (16,))])
def test_attention(call, last):
    with pytest.raises(kvi.KviError, match="pointer"):
        attend(call, last)
    with pytest.raises(ValueError, match="lse"):
        attend(call, last, lse=torch.zeros(3, 3))
    with pytest.raises(ValueError, match="4-bit"):
        attend(call, last, cache=cache4())
    with pytest.raises(ValueError, match="layer 0"):
        attend(call, last, cache=kvi.paged_cache([bf16(2, 4, 16, 1, 64)], 16))
    with pytest.raises(ValueError, match="ws"):
        attend(call, last, ws=WS[:32 << 20].view(-1, 512)[:, :256])
    with pytest.raises(ValueError, match="q must"):
        attend(call, last, q=torch.zeros(3, 4, 64))
    with pytest.raises(ValueError, match="block_tables"):
        attend(call, last, table=i64(1, 4))
    with pytest.raises(ValueError, match="status"):
        attend(call, last, status=i64(1))


def test_windows_and_prefixes():
    status = i32(1)
    for last, what in (((0, 1), "window"), ((-5, 1), "window"), ((5, -1), "sink")):
        with pytest.raises(kvi.KviError, match=what):
            attend(kvi.kvi_attn_window, last, status=status)
    with pytest.raises(kvi.KviError, match="2\\^30"):
        attend(kvi.kvi_attn_window, ((1 << 30) + 1, 0), status=status, max_ctx=(1 << 31) - 1)
    for shared in (-16, 8, 17, 64, 80, 1 << 30):
        with pytest.raises(kvi.KviError, match="shared"):
            attend(kvi.kvi_attn_shared, (shared,), status=status, max_ctx=64)
    with pytest.raises(kvi.KviError, match="workspace"):
        attend(kvi.kvi_attn_shared, (16,), status=status, ws=WS[:128])
    a = kvi.attention(4, 2, 64)
    assert kvi.kvi_attn_shared_workspace_bytes(a, 1, 3, 4, 50, 16) == 0
    assert kvi.kvi_attn_shared_workspace_bytes(a, 0, 3, 3, 50, 16) == 0
    assert kvi.kvi_attn_shared_workspace_bytes(a, 1, 3, 3, 50, -16) == 0


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(32, 8, 128), (8, 2, 64), (16, 1, 256), (128, 1, 96), (5, 5, 32)])
def test_a_workspace_serves_smaller_batches(q_heads, kv_heads, head_dim):
    a, rng = kvi.attention(q_heads, kv_heads, head_dim), random.Random(head_dim)

    def up_to(n):
        return min(n, max(1, int(round(n ** rng.random()))))

    def size(*x):
        return kvi.kvi_attn_shared_workspace_bytes(a, *x)

    for _ in range(500):
        R, ctx, max_q = up_to(256), up_to(60000), up_to(500)
        total, shared = rng.randint(max_q, R * max_q), rng.randrange(ctx)
        r, t = up_to(R), up_to(total)
        m, c = up_to(min(max_q, t)), up_to(ctx)
        grows(size, (R, total, max_q, ctx, shared), (r, t, m, c, min(shared, c - 1)))
        # and for the call itself, whatever form it takes: more than is asked for is not refused for its size
        need = None
        try:
            kvi.kvi_attn_shared(a, bf16(t, q_heads, head_dim) if t < 64 else torch.empty(t, q_heads, head_dim, dtype=torch.bfloat16), i32(r + 1),
                                m, i32(r), c, i32(r, 1 + c // 16), kvi.PagedCache(kvi.paged_cache([bf16(2, 1, 16, 1, 16)], 16).struct.layer_base, 1, 99, 16), 0,
                                min(shared, c - 1) // 16 * 16, torch.empty(t, q_heads, head_dim, dtype=torch.bfloat16), WS[:0], i32(1), stream=0)
        except kvi.KviError as e:
            need = str(e)
        assert need and "workspace of" in need
        assert int(need.split("workspace of ")[1].split(" ")[0]) <= size(r, t, m, c, min(shared, c - 1))


def rotate(T=3, Hq=4, H=2, D=64, status=None, spec=None, top=100, a=None, **kw):
    d = dict(positions=i32(T), q=bf16(T, Hq, D), k=bf16(T, H, D), q_out=bf16(T, Hq, D), k_out=bf16(T, H, D), eps=1e-6)
    d.update(kw)
    kvi.kvi_norm_rope(a or kvi.attention(Hq, H, D), spec or kvi.rope(theta=1e4), top, d.pop("positions"), d.pop("q"), d.pop("k"),
                      d.pop("q_out"), d.pop("k_out"), status, stream=0, **d)


def test_norm_rope():
    ok, pool = i32(1), kvi.paged_cache([POOL], 16)
    w = bf16(64)
    with pytest.raises(kvi.KviError, match="pointer"):
        rotate()
    for kw, what in ((dict(q_out=None), "together"), (dict(q=None), "together"), (dict(k_out=None), "nowhere"),
                     (dict(cache=pool), "needs v and slots"), (dict(v=bf16(3, 2, 64)), "need a cache"),
                     (dict(slots=i64(3)), "need a cache"), (dict(cache=pool, layer=1, v=bf16(3, 2, 64), slots=i64(3)), "layer"),
                     (dict(q_weight=w, eps=0.0), "eps"), (dict(k_weight=w, eps=float("nan")), "eps"), (dict(k_weight=w, eps=2.0), "eps"),
                     (dict(q=bf16(3 * 4 * 64 + 8)[4:4 + 768].view(3, 4, 64)), "aligned"),
                     (dict(k_weight=bf16(72)[1:65]), "aligned"), (dict(top=0), "max_position"), (dict(top=(1 << 22) + 1), "max_position"),
                     (dict(spec=kvi.rope(theta=0.0)), "theta"), (dict(spec=kvi.rope(theta=1e4, pairing=5)), "pairing"),
                     (dict(a=kvi.attention(4, 2, 24), D=24), "head_dim")):
        with pytest.raises(kvi.KviError, match=what):
            rotate(status=ok, **kw)
    plain = bf16(3, 2, 64)
    with pytest.raises(kvi.KviError, match="one buffer"):
        rotate(status=ok, k_out=plain, k_plain=plain)
    for kw, what in ((dict(q=bf16(2, 4, 64)), "q has"), (dict(k=bf16(3, 3, 64)), "k must"), (dict(k_out=torch.zeros(3, 2, 64)), "k_out"),
                     (dict(k_plain=bf16(3, 2, 128)[..., ::2]), "k_plain"), (dict(q_weight=torch.zeros(64)), "q_weight"),
                     (dict(k_weight=bf16(32)), "k_weight"), (dict(positions=i64(3)), "positions"), (dict(slots=i32(3)), "slots"),
                     (dict(slots=i64(2)), "slots"), (dict(cache=cache4()), "4-bit"),
                     (dict(cache=kvi.paged_cache([bf16(2, 4, 16, 1, 64)], 16)), "layer 0")):
        with pytest.raises(ValueError, match=what):
            rotate(status=ok, **kw)


def tables(status=None, block=16, shared=0, **kw):
    d = dict(ctx=i32(2), new=i32(2), table=i32(2, 4), free=i32(20), at=i64(2), at_out=i64(2), ctx_out=i32(2), q_start=i32(3),
             positions=i32(8), slots=i64(8))
    d.update(kw)
    kvi.kvi_batch_tables(d["ctx"], d["new"], d["table"], block, shared, d["free"], d["at"], d["at_out"], d["ctx_out"], d["q_start"],
                         d["positions"], d["slots"], status, stream=0)


def test_batch_tables():
    ok, one, at = i32(1), i32(2), i64(2)
    with pytest.raises(kvi.KviError, match="pointer"):
        tables()
    for kw, what in ((dict(block=0), "block_size"), (dict(shared=8), "shared"), (dict(shared=-16), "shared"), (dict(shared=80), "shared"),
                     (dict(ctx=one, ctx_out=one), "other buffers"), (dict(at=at, at_out=at), "other buffers"),
                     (dict(free=i32(0)), "num_blocks")):
        with pytest.raises(kvi.KviError, match=what):
            tables(ok, **kw)
    with pytest.raises(kvi.KviError, match="R="):
        tables(ok, ctx=i32(4097), new=i32(4097), table=i32(4097, 1), ctx_out=i32(4097), q_start=i32(4098))
    for kw, what in ((dict(ctx=i64(2)), "ctx_lens"), (dict(new=i32(1)), "new_lens"), (dict(table=i32(3, 4)), "block_tables"),
                     (dict(table=i32(2, 8)[:, ::2]), "block_tables"), (dict(free=i64(20)), "free"), (dict(at=i64(3)), "free_at"),
                     (dict(at_out=i32(2)), "free_at_out"), (dict(ctx_out=i32(1)), "ctx_out"), (dict(q_start=i32(2)), "q_start"),
                     (dict(positions=i32(7)), "positions"), (dict(slots=i32(8)), "slots")):
        with pytest.raises(ValueError, match=what):
            tables(ok, **kw)
    with pytest.raises(ValueError, match="status"):
        tables(i64(1))
