"""Tensors of another kind, type, shape or size than a call takes are refused
by the binding (no GPU needed).  Every call here also lacks its status word, so
that nothing is launched whatever the binding lets pass."""
import random

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from pre_rope_kv_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kvi.load_library()


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


WS = torch.zeros((32 << 20) + 256, dtype=torch.uint8)
WS = WS[(-WS.data_ptr()) % 256:]


def prompt(a=None, cache=None, lse=None, ws=WS):
    a = a or kvi.attention(4, 2, 64)
    kvi.kvi_attn_prompt(a, bf16(3, a.q_heads, a.head_dim), i32(2), 3, i32(1), 8, i32(1, 4),
                        cache or kvi.paged_cache([bf16(2, 4, 16, 2, 64)], 16), 0, bf16(3, a.q_heads, a.head_dim), ws, None,
                        lse=lse, stream=0)


def test_the_calls_reach_the_library():
    for lse in (None, torch.zeros(3, 4)):
        with pytest.raises(kvi.KviError, match="pointer"):
            prompt(lse=lse)


@pytest.mark.parametrize("lse", [torch.zeros(2, 4), torch.zeros(3, 3), torch.zeros(4, 3), torch.zeros(3, 8)[:, ::2],
                                 torch.zeros(3, 4, dtype=torch.float16), torch.zeros(3, 4, dtype=torch.float64), torch.zeros(0)])
def test_log_sums(lse):
    # written as float32 [total_q][q_heads], these would be passed at their end
    with pytest.raises(ValueError, match="lse"):
        prompt(lse=lse)


@pytest.mark.parametrize("cache", [
    kvi.paged_cache([bf16(2, 4, 16, 1, 64)], 16), kvi.paged_cache([bf16(2, 4, 16, 2, 32)], 16),
    kvi.paged_cache([bf16(2, 4, 8, 2, 64)], 16), kvi.paged_cache([bf16(1, 4, 16, 2, 64)], 16),
    kvi.paged_cache([torch.zeros(2, 4, 16, 2, 64, dtype=torch.uint8)], 16),
    kvi.paged_cache([bf16(4, 2, 16, 2, 64).transpose(0, 1)], 16)])
def test_pools_of_another_layout(cache):
    with pytest.raises(ValueError, match="layer 0"):
        prompt(cache=cache)


def test_pools_of_another_layer():
    cache = kvi.paged_cache([bf16(2, 4, 16, 2, 64), bf16(2, 3, 16, 2, 64)], 16)
    with pytest.raises(kvi.KviError, match="pointer"):
        prompt(cache=cache)
    with pytest.raises(ValueError, match="layer 1"):
        kvi.kvi_attn_prompt(kvi.attention(4, 2, 64), bf16(3, 4, 64), i32(2), 3, i32(1), 8, i32(1, 4), cache, 1, bf16(3, 4, 64),
                            WS, None, stream=0)


def test_a_4_bit_pool_is_no_bf16_pool():
    one = kvi.kvi_cache4_layer_bytes(2, 64, 4, 16)
    with pytest.raises(ValueError, match="4-bit"):
        prompt(cache=kvi.cache4([torch.zeros(one, dtype=torch.uint8)], 16, 2, 64))


def cache4():
    return kvi.cache4([torch.zeros(kvi.kvi_cache4_layer_bytes(2, 64, 4, 16), dtype=torch.uint8)], 16, 2, 64)


def decode(w=None, ws=WS):
    kvi.kvi_attn_decode4(kvi.attention(4, 2, 64), bf16(1, 4, 64), i32(1), 8, i32(1, 4), cache4(), 0, bf16(1, 4, 64), ws, None,
                         weights=w, stream=0)


def evict(i=None, bad=None, ws=WS):
    t = [torch.zeros(1, 2, 40), i32(1, 2, 40), torch.zeros(1, 2, 40), i32(1, 2, 40)]  # weights and positions, in and out
    if i is not None:
        t[i] = bad
    kvi.kvi_cache4_evict(cache4(), 0, i32(1), 40, i32(1, 4), 10, 1, 2, t[0], t[1], t[2], t[3], i32(1), ws, None, stream=0)


def test_accumulated_weights_of_another_type():
    # read and written as float32, whole numbers would be other weights
    for w in (None, torch.zeros(1, 2, 40)):
        with pytest.raises(kvi.KviError, match="pointer"):
            decode(w)
    with pytest.raises(kvi.KviError, match="pointer"):
        evict()
    with pytest.raises(ValueError, match="float32"):
        decode(i32(1, 2, 40))
    for i, bad in ((0, i32(1, 2, 40)), (1, torch.zeros(1, 2, 40)), (2, i32(1, 2, 40)), (3, torch.zeros(1, 2, 40))):
        with pytest.raises(ValueError, match="float32"):
            evict(i, bad)


def test_4_bit_pools_in_pieces():
    one = kvi.kvi_cache4_layer_bytes(2, 64, 1, 16)
    kvi.cache4([torch.zeros(4, one, dtype=torch.uint8)], 16, 2, 64)
    for pool in (torch.zeros(8, one, dtype=torch.uint8)[::2], torch.zeros(4, 2 * one, dtype=torch.uint8)[:, :one]):
        with pytest.raises(ValueError, match="in one piece"):
            kvi.cache4([pool], 16, 2, 64)


@pytest.mark.parametrize("call", [prompt, decode, evict])
def test_workspaces_in_pieces(call):
    with pytest.raises(ValueError, match="ws"):
        call(ws=WS[:32 << 20].view(-1, 512)[:, :256])


def test_status_words_of_another_type():
    # the kernels write 32 bits
    k, slots, w, p = bf16(1, 2, 64), torch.zeros(1, dtype=torch.int64), torch.zeros(1, 2, 40), i32(1, 2, 40)
    a, q, n, table = kvi.attention(4, 2, 64), bf16(1, 4, 64), i32(1), i32(1, 4)
    none = WS[:0]  # (refused by the library, so that nothing is launched)
    for bad in (torch.zeros(4, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64), i32(0)):
        with pytest.raises(ValueError, match="status"):
            kvi.kvi_attn_prompt(a, q, i32(2), 1, n, 8, table, kvi.paged_cache([bf16(2, 4, 16, 2, 64)], 16), 0, q, none, bad, stream=0)
        with pytest.raises(ValueError, match="status"):
            kvi.kvi_attn_decode4(a, q, n, 8, table, cache4(), 0, q, none, bad, stream=0)
        with pytest.raises(ValueError, match="status"):
            kvi.kvi_cache4_evict(cache4(), 0, n, 40, table, 10, 1, 2, w, p, w.clone(), p.clone(), i32(1), none, bad, stream=0)
        with pytest.raises(ValueError, match="status"):
            kvi.kvi_cache4_write(cache4(), 5, k, k, slots, bad, stream=0)
        with pytest.raises(ValueError, match="status"):
            kvi.kvi_cache4_read(cache4(), 5, slots, k, k, bad, stream=0)


def grows(size, larger, smaller):
    assert size(*larger) >= size(*smaller) > 0, (larger, smaller)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(32, 8, 128), (8, 2, 64), (16, 1, 256), (128, 1, 96), (5, 5, 32)])
def test_a_workspace_serves_smaller_calls(q_heads, kv_heads, head_dim):
    """A program sizes its workspace once, for the largest call it makes."""
    a, rng = kvi.attention(q_heads, kv_heads, head_dim), random.Random(head_dim)

    def up_to(n):
        return min(n, max(1, int(round(n ** rng.random()))))

    def prompt_bytes(R, total, max_q, ctx):
        return kvi.kvi_attn_prompt_workspace_bytes(a, R, total, max_q, ctx)

    def decode_bytes(R, ctx, weights):
        return kvi.kvi_attn_decode4_workspace_bytes(a, R, ctx, weights)

    def evict_bytes(R, ctx):
        return kvi.kvi_cache4_evict_workspace_bytes(kv_heads, R, ctx)

    # a step longer, a request more; one prompt, and a question after it; an eviction and the step after it
    grows(decode_bytes, (1, 2049, True), (1, 2048, True))
    grows(decode_bytes, (64, 8192, False), (4, 8192, False))
    grows(decode_bytes, (18, 6357, True), (18, 6086, True))
    grows(prompt_bytes, (1, 8192, 8192, 8192), (1, 37, 37, 1601))
    for _ in range(4000):
        R, ctx, max_q = up_to(256), up_to(60000), up_to(5000)
        total = rng.randint(max_q, R * max_q) if rng.random() < 0.7 else max_q + up_to(60000)
        r, c = (R if rng.random() < 0.3 else up_to(R)), (ctx if rng.random() < 0.3 else up_to(ctx))
        t = total if rng.random() < 0.3 else up_to(total)
        m = min(max_q, t) if rng.random() < 0.3 else up_to(min(max_q, t))
        grows(prompt_bytes, (R, total, max_q, ctx), (r, t, m, c))
        w = rng.random() < 0.5
        grows(decode_bytes, (R, ctx, w), (r, c, w and rng.random() < 0.5))
        grows(evict_bytes, (R, ctx), (r, c))


def test_workspaces_stay_small():
    # pieces of a few rows, however large the call or the buffer q lies in
    a = kvi.attention(32, 8, 128)
    for sizes in ((1, 8192, 8192, 8192), (64, 100000, 8192, 32768), (1, 100000, 1, 100000), (1000, 100000, 37, 4000)):
        assert kvi.kvi_attn_prompt_workspace_bytes(a, *sizes) < 24 << 20
    assert kvi.kvi_attn_decode4_workspace_bytes(a, 1000, 100000, False) < 8 << 20
