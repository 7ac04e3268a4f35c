"""Many users over one memory: a serving loop without the host in between.

The attention side of a model whose layers alternate between full attention and a
sliding window, on random weights:

  1. one conversation's facts are retrieved and injected once, into blocks that
     all users' tables share (kvi_retrieve_topk, kvi_place, kvi_inject_paged);
     the system's own tokens behind them fill the last block (kvi_norm_rope);
  2. each step's tables, rows, positions and slots come from the users' lengths
     on the GPU (kvi_batch_tables): first a question each, then single tokens;
     a user who has finished gives the blocks back;
  3. queries and keys are normalised and rotated, and K and V go to the pages,
     in one pass (kvi_norm_rope);
  4. full layers read the memory once for all users (kvi_attn_shared), the others
     see a window and the first tokens (kvi_attn_window).

The generation steps are one CUDA graph, replayed.

    python examples/serve_shared_memory.py
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import pre_rope_kv_gb300 as kvi  # noqa: E402


def run(layers=2, q_heads=8, kv_heads=2, head_dim=64, embed_dim=256, facts=200, k=24, users=6, question=37, steps=20,
        window=96, sink=16, block=16, theta=1e4, seed=0, watch=None):
    """Returns the state at the end; watch(state) is called after each step."""
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    status = torch.zeros(1, dtype=torch.int32, device=dev)
    a, spec = kvi.attention(q_heads, kv_heads, head_dim), kvi.rope(theta=theta)

    # ---- 1. the memory: k facts, and system tokens up to a whole block
    fact_len = 8 + torch.arange(facts, device=dev, dtype=torch.int32) % 16
    fact_start = torch.cumsum(fact_len.long(), 0) - fact_len
    kv = randn(layers, 2, int(fact_len.sum()), kv_heads, head_dim).to(torch.bfloat16)
    emb = torch.nn.functional.normalize(randn(facts, embed_dim), dim=-1)
    view = kvi.store_view(kvi.geometry(layers, kv_heads, head_dim, embed_dim), kv, emb, fact_start, fact_len)
    ids, pos = (torch.zeros(k, dtype=torch.int32, device=dev) for _ in range(2))
    scores = torch.zeros(k, device=dev)
    ws = torch.empty(kvi.kvi_workspace_bytes(1, facts, k), dtype=torch.uint8, device=dev)
    query = torch.nn.functional.normalize(randn(embed_dim), dim=-1)
    kvi.kvi_retrieve_topk(view, query, k, ids, scores, ws, status)
    kvi.kvi_place(view, ids, k, 0, pos, status)
    memory = int(fact_len[ids.long()].sum())
    system = 8 + (-(memory + 8)) % block
    shared = memory + system
    room = shared + question + steps
    width = (room + block - 1) // block
    blocks = shared // block + users * (width - shared // block) + 4
    limit = width * block
    kvi.kvi_prepare_rope_ex(spec, head_dim, limit)
    pool = [torch.zeros(2, blocks, block, kv_heads, head_dim, dtype=torch.bfloat16, device=dev) for _ in range(layers)]
    cache = kvi.paged_cache(pool, block)
    order = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    prefix = order[:shared // block].contiguous()
    kvi.kvi_inject_paged_ex(view, ids, pos, k, prefix, prefix.numel(), cache, spec, status)
    weights = [[(1 + 0.2 * randn(head_dim)).to(torch.bfloat16) for _ in range(2)] for _ in range(layers)]  # of q, k
    at = memory + torch.arange(system, device=dev)
    for layer in range(layers):
        own = randn(system, 2 * kv_heads, head_dim).to(torch.bfloat16)
        kvi.kvi_norm_rope(a, spec, limit, at.to(torch.int32), None, own[:, :kv_heads], None, None, status, k_weight=weights[layer][1],
                          v=own[:, kv_heads:], cache=cache, layer=layer, slots=prefix[at // block].long() * block + at % block)

    # ---- the users: their tables begin with the memory's blocks; the others are free
    table = torch.zeros(users, width, dtype=torch.int32, device=dev)
    table[:, :prefix.numel()] = prefix
    free = torch.zeros(blocks, dtype=torch.int32, device=dev)
    free[:blocks - prefix.numel()] = order[prefix.numel():]
    free_at, free_after = (torch.tensor([0, blocks - prefix.numel()], device=dev) for _ in range(2))
    ctx = torch.full((users,), shared, dtype=torch.int32, device=dev)
    ctx_after, new = torch.empty_like(ctx), torch.empty_like(ctx)
    q_start = torch.zeros(users + 1, dtype=torch.int32, device=dev)

    def buffers(rows, longest):
        wide = q_heads + 2 * kv_heads
        need = max(kvi.kvi_attn_shared_workspace_bytes(a, users, rows, longest, room, shared),
                   kvi.kvi_attn_prompt_workspace_bytes(a, users, rows, longest, room))
        return dict(rows=rows, longest=longest, positions=torch.zeros(rows, dtype=torch.int32, device=dev),
                    slots=torch.zeros(rows, dtype=torch.int64, device=dev), ws=torch.empty(need, dtype=torch.uint8, device=dev),
                    qkv=[torch.zeros(rows, wide, head_dim, dtype=torch.bfloat16, device=dev) for _ in range(layers)],
                    q=[torch.zeros(rows, q_heads, head_dim, dtype=torch.bfloat16, device=dev) for _ in range(layers)],
                    out=[torch.zeros(rows, q_heads, head_dim, dtype=torch.bfloat16, device=dev) for _ in range(layers)])

    def step(b):
        """A step of all users, from `new` and the projections b["qkv"]."""
        kvi.kvi_batch_tables(ctx, new, table, block, shared, free, free_at, free_after, ctx_after, q_start, b["positions"],
                             b["slots"], status)
        ctx.copy_(ctx_after)
        free_at.copy_(free_after)
        for layer in range(layers):
            qkv, q = b["qkv"][layer], b["q"][layer]
            kvi.kvi_norm_rope(a, spec, limit, b["positions"], qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], q, None, status,
                              q_weight=weights[layer][0], k_weight=weights[layer][1], v=qkv[:, q_heads + kv_heads:], cache=cache,
                              layer=layer, slots=b["slots"])
            if layer % 2 == 0:
                kvi.kvi_attn_shared(a, q, q_start, b["longest"], ctx, room, table, cache, layer, shared, b["out"][layer], b["ws"], status)
            else:
                kvi.kvi_attn_window(a, q, q_start, b["longest"], ctx, room, table, cache, layer, window, sink, b["out"][layer], b["ws"],
                                    status)

    state = dict(a=a, spec=spec, theta=theta, pool=pool, table=table, block=block, shared=shared, window=window, sink=sink, weights=weights, ctx=ctx,
                 q_start=q_start, free=free, free_at=free_at, blocks=blocks, status=status, memory=memory)

    def seen(b):
        if watch:
            watch(dict(state, **b))

    # ---- 2 to 4: questions of different lengths, then tokens; the rows are as many in each step, and padded
    asked = torch.randint(1, question + 1, (users,), generator=g, device=dev).to(torch.int32)
    b = buffers(int(asked.sum()) + 3, question)
    new.copy_(asked)
    for x in b["qkv"]:
        x.copy_(randn(*x.shape))
    step(b)
    seen(b)
    b = buffers(users, 1)
    new.fill_(1)
    graph = torch.cuda.CUDAGraph()
    keep = [x.clone() for x in (ctx, free_at, free, table)]
    with torch.cuda.graph(graph):
        step(b)
    for x, y in zip((ctx, free_at, free, table), keep):  # (recording ran nothing)
        assert torch.equal(x, y)
    for i in range(steps):
        if users > 1 and i == steps // 2:
            new[-1] = -1  # the last user has finished
        elif users > 1 and i == steps // 2 + 1:
            new[-1] = 0
        for x in b["qkv"]:
            x.copy_(randn(*x.shape))
        graph.replay()
        seen(b)
    if int(status):
        raise RuntimeError(f"device status {int(status)}: {kvi.kvi_status_str(int(status))}")
    return dict(state, **b)


def main():
    r = run()
    print(f"{r['memory']} tokens of memory in {r['shared'] // r['block']} shared blocks; users' lengths {r['ctx'].tolist()}; "
          f"{int(r['free_at'][1] - r['free_at'][0])} of {r['blocks']} blocks free")


if __name__ == "__main__":
    main()
