"""The attention and 4-bit cache calls refuse bad host arguments before any
CUDA work (no GPU needed), and their size queries."""
import math

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from pre_rope_kv_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kvi.load_library()


def refused(f, *a, **kw):
    with pytest.raises(kvi.KviError) as e:
        f(*a, stream=0, **kw)
    assert e.value.status == kvi.ERR_INVALID_ARG
    return kvi.kvi_last_error()


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


WS = torch.zeros(1 << 20, dtype=torch.uint8)
WS = WS[(-WS.data_ptr()) % 256:]


@pytest.mark.parametrize("a", [kvi.attention(3, 2, 64), kvi.attention(1, 2, 64), kvi.attention(2, 2, 40),
                               kvi.attention(2, 2, 272), kvi.attention(258, 2, 64), kvi.attention(2, 0, 64),
                               kvi.attention(2, 2, 64, scale=0.0), kvi.attention(2, 2, 64, scale=math.inf)])
def test_bad_attention(a):
    n, d = a.q_heads, a.head_dim
    pool = bf16(2, 4, 16, 2, 64)
    refused(kvi.kvi_attn_prompt, a, bf16(3, n, d), i32(2), 3, i32(1), 8, i32(1, 4), kvi.paged_cache([pool], 16), 0,
            bf16(3, n, d), WS, i32(1))
    assert kvi.kvi_attn_prompt_workspace_bytes(a, 1, 3, 3, 8) == 0
    assert kvi.kvi_attn_decode4_workspace_bytes(a, 1, 8, False) == 0


def prompt(**kw):
    d = dict(a=kvi.attention(4, 2, 64), q=bf16(3, 4, 64), start=i32(2), max_q=3, ctx=i32(1), max_ctx=8, table=i32(1, 4),
             cache=kvi.paged_cache([bf16(2, 4, 16, 2, 64)], 16), layer=0, out=bf16(3, 4, 64), ws=WS, status=i32(1), lse=None)
    d.update(kw)
    return refused(kvi.kvi_attn_prompt, d["a"], d["q"], d["start"], d["max_q"], d["ctx"], d["max_ctx"], d["table"],
                   d["cache"], d["layer"], d["out"], d["ws"], d["status"], lse=d["lse"])


def test_prompt_arguments():
    assert "layer" in prompt(layer=1)
    assert "max_q" in prompt(max_q=4)
    assert "max_ctx" in prompt(max_ctx=-1)
    assert "R=" in prompt(ctx=i32(5000))
    assert "workspace" in prompt(ws=WS[:16])
    assert "workspace" in prompt(ws=WS[16:])
    assert "pointer" in prompt(status=None)
    assert "pointer" in prompt(start=None)
    assert "block tables" in prompt(table=i32(1, 0))
    assert "misaligned" in prompt(lse=torch.zeros(40, dtype=torch.uint8)[2:])
    buf = bf16(3 * 4 * 64 + 8)
    assert "aligned" in prompt(q=buf[2:2 + 768].view(3, 4, 64))
    assert "aligned" in prompt(out=buf[2:2 + 768].view(3, 4, 64))
    assert "aligned" in prompt(q=torch.as_strided(bf16(4096), (3, 4, 64), (260, 64, 1)))
    assert "num_blocks" in prompt(cache=kvi.paged_cache([bf16(2, 0, 16, 2, 64)], 16))
    with pytest.raises(ValueError):
        prompt(q=bf16(3, 5, 64))
    with pytest.raises(ValueError):
        prompt(q=bf16(3, 64, 4).transpose(1, 2))
    with pytest.raises(ValueError):
        prompt(q=bf16(3, 4, 64).half())
    with pytest.raises(ValueError):
        prompt(out=bf16(2, 4, 64))


def test_layer_bytes():
    assert kvi.kvi_cache4_layer_bytes(8, 128, 10, 16) == 10 * 8 * (16 * 128 + 16 * 4 * 4)
    assert kvi.kvi_cache4_layer_bytes(1, 32, 1, 16) == 16 * 32 + 16 * 4
    for bad in [(0, 64, 1, 16), (1, 48, 1, 16), (1, 0, 1, 16), (1, 288, 1, 16), (1, 64, 0, 16), (1, 64, 1, 8), (1, 64, 1, 24)]:
        assert kvi.kvi_cache4_layer_bytes(*bad) == 0


def cache(layers=1, B=16, H=2, D=64):
    return kvi.cache4([torch.zeros(4 * kvi.kvi_cache4_layer_bytes(2, 64, 1, 16), dtype=torch.uint8) for _ in range(layers)], B, H, D)


def test_rows_arguments():
    k, slots, st = bf16(3, 2, 64), torch.zeros(3, dtype=torch.int64), i32(1)
    for f in (lambda c, l, k, v, s, t: refused(kvi.kvi_cache4_write, c, l, k, v, s, t),
              lambda c, l, k, v, s, t: refused(kvi.kvi_cache4_read, c, l, s, k, v, t)):
        assert "layer" in f(cache(), 1, k, k, slots, st)
        assert "4-bit" in f(cache(B=17), 0, k, k, slots, st)
        assert "status" in f(cache(), 0, k, k, slots, None)
        assert "aligned" in f(cache(), 0, bf16(400)[2:386].view(3, 2, 64), k, slots, st)
        assert "aligned" in f(cache(), 0, k, torch.as_strided(bf16(800), (3, 2, 64), (132, 64, 1)), slots, st)
        with pytest.raises(ValueError):
            f(cache(), 0, bf16(2, 2, 64), k, slots, st)
    with pytest.raises(ValueError):
        kvi.cache4([torch.zeros(100, dtype=torch.uint8)], 16, 2, 64)


def test_decode_arguments():
    a = kvi.attention(4, 2, 64)

    def step(**kw):
        d = dict(a=a, q=bf16(2, 4, 64), ctx=i32(2), max_ctx=8, table=i32(2, 4), cache=cache(), layer=0, out=bf16(2, 4, 64),
                 ws=WS, status=i32(1), w=None)
        d.update(kw)
        return refused(kvi.kvi_attn_decode4, d["a"], d["q"], d["ctx"], d["max_ctx"], d["table"], d["cache"], d["layer"],
                       d["out"], d["ws"], d["status"], weights=d["w"])

    assert "layer" in step(layer=-1)
    assert "max_ctx" in step(max_ctx=-2)
    assert "weights_stride" in step(w=torch.zeros(2, 2, 7))
    assert "workspace" in step(ws=WS[:0])
    assert "pointer" in step(status=None)
    assert "head_dim" in step(a=kvi.attention(4, 2, 80), q=bf16(2, 4, 80), out=bf16(2, 4, 80), cache=cache(D=80))
    with pytest.raises(ValueError):
        step(a=kvi.attention(4, 1, 64))
    with pytest.raises(ValueError):
        step(w=torch.zeros(2, 3, 8))
    assert kvi.kvi_attn_decode4_workspace_bytes(a, 0, 8, False) == 0
    assert kvi.kvi_attn_decode4_workspace_bytes(a, 2, 100, True) > kvi.kvi_attn_decode4_workspace_bytes(a, 2, 100, False)


def test_evict_arguments():
    w, p, n = torch.zeros(1, 2, 40), i32(1, 2, 40), i32(1)

    def evict(**kw):
        d = dict(max_ctx=40, budget=10, sink=1, recent=2, w2=w.clone(), p2=p.clone(), n2=n.clone(), ws=WS, status=i32(1),
                 layer=0, table=i32(1, 4))
        d.update(kw)
        return refused(kvi.kvi_cache4_evict, cache(), d["layer"], n, d["max_ctx"], d["table"], d["budget"], d["sink"],
                       d["recent"], w, p, d["w2"], d["p2"], d["n2"], d["ws"], d["status"])

    assert "budget" in evict(budget=0)
    assert "budget" in evict(sink=5, recent=6)
    assert "budget" in evict(recent=-1)
    assert "other buffers" in evict(w2=w)
    assert "other buffers" in evict(p2=p)
    assert "other buffers" in evict(n2=n)
    assert "max_ctx" in evict(max_ctx=41)
    assert "workspace" in evict(ws=WS[16:])
    assert "pointer" in evict(status=None)
    assert "layer" in evict(layer=2)
    assert "block tables" in evict(table=i32(1, 0))
    with pytest.raises(ValueError):
        evict(p2=i32(1, 2, 41))
    assert kvi.kvi_cache4_evict_workspace_bytes(2, 1, -1) == 0


def test_integers_of_another_type():
    # read as they are not, these would be other blocks, lengths or slots
    k, slots, st = bf16(3, 2, 64), torch.zeros(3, dtype=torch.int64), i32(1)
    for bad in (slots.int(), torch.zeros(6, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError):
            kvi.kvi_cache4_write(cache(), 0, k, k, bad, st, stream=0)
        with pytest.raises(ValueError):
            kvi.kvi_cache4_read(cache(), 0, bad, k, k, st, stream=0)
    for bad in (dict(ctx=i32(1).long()), dict(start=i32(2).long()), dict(start=i32(1)), dict(table=i32(1, 4).long()),
                dict(table=i32(1, 8)[:, ::2]), dict(ctx=i32(2), start=i32(3))):
        with pytest.raises(ValueError):
            prompt(**bad)
