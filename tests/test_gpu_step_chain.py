"""Decoding steps of a batch with a shared prefix in one CUDA graph, nothing between them: tables from
lengths, norms with rotation into the pages, attention, layer after layer and step after step, each
kernel behind the one whose results it reads.  Every step's outputs are compared with plain float64
attention over the pages, for the forms that read the prefix by itself: blocks that join its pieces to
a request's keys, and a join of its own."""
import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests import step_check as sc
from tests.test_gpu_norm_rope import close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
LAYERS, STEPS, BLOCK, THETA = 2, 6, 16, 1e4


# (users, query and KV heads, head size, keys of the prefix, room for own keys: up to 384 of them blocks join themselves, new tokens a step)
@pytest.mark.parametrize("users,Hq,H,D,shared,room,new", [(8, 8, 8, 128, 1600, 200, 1), (8, 32, 8, 128, 1600, 384, 1), (24, 16, 8, 128, 1600, 144, 1),
                                                          (8, 8, 8, 128, 1600, 900, 1), (64, 32, 8, 128, 1600, 700, 1),
                                                          (12, 32, 8, 128, 1600, 800, 9), (40, 8, 2, 64, 4096, 300, 4)])
def test_steps(users, Hq, H, D, shared, room, new):
    g = ac.gen(users + D + room)
    a, spec = kvi.attention(Hq, H, D), kvi.rope(theta=THETA)
    assert (users - 1) * shared * H * D * 4 >= 32 << 20  # (what is read less: the prefix has kernels of its own)
    limit = shared + room
    kvi.kvi_prepare_rope_ex(spec, D, limit)
    first, width = shared // BLOCK, -(-limit // BLOCK)
    blocks = first + users * (width - first) + 3
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    pool = [ac.randn(g, 2, blocks, BLOCK, H, D).to(BF) for _ in range(LAYERS)]
    cache = kvi.paged_cache(pool, BLOCK)
    table = torch.full((users, width), -9, dtype=torch.int32, device=DEV)
    table[:, :first] = order[:first]
    free = torch.full((blocks,), -3, dtype=torch.int32, device=DEV)
    free[:blocks - first] = order[first:]
    at, at_out = (torch.tensor([0, blocks - first], device=DEV) for _ in range(2))
    ctx0 = torch.full((users,), shared, dtype=torch.int32, device=DEV)
    ctx, ctx_out, q_start = ctx0.clone(), torch.empty_like(ctx0), torch.zeros(users + 1, dtype=torch.int32, device=DEV)
    news = torch.full((users,), new, dtype=torch.int32, device=DEV)
    rows, status = users * new, torch.zeros(1, dtype=torch.int32, device=DEV)
    positions, slots = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.zeros(rows, dtype=torch.int64, device=DEV)
    qkv = torch.zeros(STEPS, LAYERS, rows, Hq + 2 * H, D, dtype=BF, device=DEV)
    q = torch.zeros(rows, Hq, D, dtype=BF, device=DEV)  # one for all: a step's norms follow the last one's attention
    qs, out = (torch.zeros(STEPS, LAYERS, rows, Hq, D, dtype=BF, device=DEV) for _ in range(2))
    lse = torch.zeros(STEPS, LAYERS, rows, Hq, device=DEV)
    weights = [(1 + 0.2 * ac.randn(g, D)).to(BF) for _ in range(2)]
    ws = ac.workspace(kvi.kvi_attn_shared_workspace_bytes(a, users, rows, new, limit, shared))

    def steps():
        for i in range(STEPS):
            kvi.kvi_batch_tables(ctx, news, table, BLOCK, shared, free, at, at_out, ctx_out, q_start, positions, slots, status)
            ctx.copy_(ctx_out)
            at.copy_(at_out)
            for layer in range(LAYERS):
                x = qkv[i, layer]
                kvi.kvi_norm_rope(a, spec, limit, positions, x[:, :Hq], x[:, Hq:Hq + H], q, None, status, q_weight=weights[0],
                                  k_weight=weights[1], v=x[:, Hq + H:], cache=cache, layer=layer, slots=slots)
                kvi.kvi_attn_shared(a, q, q_start, new, ctx, limit, table, cache, layer, shared, out[i, layer], ws, status,
                                    lse=lse[i, layer])
                qs[i, layer].copy_(q)

    keep = [x.clone() for x in (ctx, at, free, table)]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        steps()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((ctx, at, free, table), keep))
    omega = sc.frequencies(THETA, D)
    for replay in range(4 if new == 1 else 2):  # (24 steps: into a block of their own)
        qkv.copy_(ac.randn(g, *qkv.shape).to(BF))
        out.fill_(7)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        assert int(status) == 0
        end = shared + (replay + 1) * STEPS * new
        assert ctx.tolist() == [end] * users
        for i in range(STEPS):
            keys = end - (STEPS - 1 - i) * new
            j = torch.arange(keys, device=DEV)
            pos = torch.arange(keys - new, keys, device=DEV).repeat(users)
            seen = j <= torch.arange(keys - new, keys, device=DEV)[:, None]
            for layer in range(LAYERS):
                flat = pool[layer].view(2, -1, H, D)
                ref, both = sc.rotated(sc.normed(qkv[i, layer, :, :Hq], weights[0], 1e-6), pos, omega, False)
                close(qs[i, layer], ref, both)
                for r in range(0, users, 5):
                    where = table[r][j // BLOCK].long() * BLOCK + j % BLOCK
                    ref, both = sc.rotated(sc.normed(qkv[i, layer, r * new:(r + 1) * new, Hq:Hq + H], weights[1], 1e-6), pos[:new], omega, False)
                    close(flat[0, where[-new:]], ref, both)
                    assert torch.equal(flat[1, where[-new:]], qkv[i, layer, r * new:(r + 1) * new, Hq + H:])
                    for h in range(0, H, 3):
                        hs, rs = slice(h * Hq // H, (h + 1) * Hq // H), slice(r * new, (r + 1) * new)
                        ref, log_sum, pv, size = sc.attend(qs[i, layer, rs, hs].double(), flat[0, where, h].double(), flat[1, where, h].double(),
                                                           seen, a.scale)
                        ac.check_out(out[i, layer, rs, hs], ref, pv, size, 1, (replay, i, layer, r, h))
                        ac.check_lse(lse[i, layer, rs, hs], log_sum, size)
