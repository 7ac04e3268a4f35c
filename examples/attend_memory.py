"""A request from retrieval to generation over injected memory.

The attention side of a serving step, layer by layer, on random weights:

  1. the question's facts are retrieved and injected into the paged bf16 cache
     (kvi_retrieve_and_inject);
  2. the prompt's own keys and values are written behind them and the prompt
     attends to memory and itself (kvi_attn_prompt);
  3. the cache is converted to 4 bits (kvi_cache4_write on the pool's planes);
  4. tokens are generated over the 4-bit cache, each step storing its K/V
     (kvi_cache4_write) and accumulating every key's softmax weight
     (kvi_attn_decode4);
  5. when a layer holds more keys than its budget it is cut back to the keys
     that drew most weight (kvi_cache4_evict).

    python examples/attend_memory.py
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import pre_rope_kv_gb300 as kvi  # noqa: E402


def run(layers=2, q_heads=8, kv_heads=2, head_dim=64, embed_dim=256, facts=200, k=12, prompt=37, steps=24, budget=160,
        sink=4, recent=16, block=16, theta=1e4, seed=0):
    """Returns what the last steps computed (for a caller that checks it)."""
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # ---- a store of facts of 8 to 23 tokens, and a pool that holds one request
    fact_len = 8 + torch.arange(facts, device=dev, dtype=torch.int32) % 16
    fact_start = torch.cumsum(fact_len.long(), 0) - fact_len
    tokens = int(fact_len.sum())
    geom = kvi.geometry(layers, kv_heads, head_dim, embed_dim)
    kv = randn(layers, 2, tokens, kv_heads, head_dim).to(torch.bfloat16)
    emb = torch.nn.functional.normalize(randn(facts, embed_dim), dim=-1)
    room = k * 23 + prompt + steps
    blocks = (room + block - 1) // block + 2
    pool = [torch.zeros(2, blocks, block, kv_heads, head_dim, dtype=torch.bfloat16, device=dev) for _ in range(layers)]
    cache = kvi.paged_cache(pool, block)
    table = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)[None]
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def slots(first, n):
        p = torch.arange(first, first + n, device=dev)
        return table[0, p // block].long() * block + p % block

    # ---- 1. memory: positions 0 .. memory-1
    view = kvi.store_view(geom, kv, emb, fact_start, fact_len)
    views = torch.frombuffer(bytearray(kvi.pack_store_views([view])), dtype=torch.uint8).to(dev)
    question = torch.nn.functional.normalize(randn(1, embed_dim), dim=-1)
    ids, pos = (torch.zeros(1, k, dtype=torch.int32, device=dev) for _ in range(2))
    scores = torch.zeros(1, k, device=dev)
    ws = torch.empty(kvi.kvi_workspace_bytes(1, facts, k), dtype=torch.uint8, device=dev)
    start = torch.zeros(1, dtype=torch.int32, device=dev)
    table_lens = torch.full((1,), blocks, dtype=torch.int32, device=dev)
    kvi.kvi_retrieve_and_inject(geom, 1, views, facts, question, k, start, table, table_lens, blocks, cache, theta, ids,
                                scores, pos, ws, status)
    memory = int(fact_len[ids[0].long()].sum())

    # ---- 2. the prompt: its K/V behind the memory, its attention over both
    a = kvi.attention(q_heads, kv_heads, head_dim)
    ctx = memory + prompt
    ctx_lens = torch.tensor([ctx], dtype=torch.int32, device=dev)
    q_start = torch.tensor([0, prompt], dtype=torch.int32, device=dev)
    ws = torch.empty(kvi.kvi_attn_prompt_workspace_bytes(a, 1, prompt, prompt, ctx), dtype=torch.uint8, device=dev)
    prompt_out = []
    for layer in range(layers):
        qkv = randn(prompt, q_heads + 2 * kv_heads, head_dim).to(torch.bfloat16)  # a fused projection's output
        flat = pool[layer].view(2, -1, kv_heads, head_dim)
        flat[0, slots(memory, prompt)] = qkv[:, q_heads:q_heads + kv_heads]
        flat[1, slots(memory, prompt)] = qkv[:, q_heads + kv_heads:]
        out = torch.empty(prompt, q_heads, head_dim, dtype=torch.bfloat16, device=dev)
        kvi.kvi_attn_prompt(a, qkv[:, :q_heads], q_start, prompt, ctx_lens, ctx, table, cache, layer, out, ws, status)
        prompt_out.append((qkv[:, :q_heads], out))

    # ---- 3. the cache in 4 bits: the same blocks, 4.5 bits an element
    one = kvi.kvi_cache4_layer_bytes(kv_heads, head_dim, blocks, block)
    pool4 = [torch.zeros(one, dtype=torch.uint8, device=dev) for _ in range(layers)]
    cache4 = kvi.cache4(pool4, block, kv_heads, head_dim)
    every = torch.full((blocks * block,), -1, dtype=torch.int64, device=dev)  # rows that hold nothing: skipped
    every[slots(0, ctx)] = slots(0, ctx)
    for layer in range(layers):
        flat = pool[layer].view(2, -1, kv_heads, head_dim)
        kvi.kvi_cache4_write(cache4, layer, flat[0], flat[1], every, status)

    # ---- 4 and 5. generation; per layer a weight and a position for every slot
    weights = [torch.zeros(1, kv_heads, room, device=dev) for _ in range(layers)]
    where = [torch.arange(room, dtype=torch.int32, device=dev).expand(1, kv_heads, -1).contiguous() for _ in range(layers)]
    lens = [ctx_lens.clone() for _ in range(layers)]
    held, position, evictions = ctx, ctx, 0
    ws = torch.empty(max(kvi.kvi_attn_decode4_workspace_bytes(a, 1, room, True),
                         kvi.kvi_cache4_evict_workspace_bytes(kv_heads, 1, room)), dtype=torch.uint8, device=dev)
    last = []
    for _ in range(steps):
        if held >= budget + recent:  # a layer is over its budget: cut back to it
            for layer in range(layers):
                w2, p2, n2 = torch.zeros_like(weights[layer]), torch.full_like(where[layer], -1), torch.empty_like(ctx_lens)
                kvi.kvi_cache4_evict(cache4, layer, lens[layer], held, table, budget, sink, recent, weights[layer],
                                     where[layer], w2, p2, n2, ws, status)
                weights[layer], where[layer], lens[layer] = w2, p2, n2
            held, evictions = budget, evictions + 1
        last = []
        for layer in range(layers):
            qkv = randn(1, q_heads + 2 * kv_heads, head_dim).to(torch.bfloat16)
            kvi.kvi_cache4_write(cache4, layer, qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:],
                                 slots(held, 1), status)
            weights[layer][:, :, held] = 0
            where[layer][:, :, held] = position
            lens[layer] += 1
            out = torch.empty(1, q_heads, head_dim, dtype=torch.bfloat16, device=dev)
            kvi.kvi_attn_decode4(a, qkv[:, :q_heads], lens[layer], held + 1, table, cache4, layer, out, ws, status,
                                 weights=weights[layer])
            last.append((qkv[:, :q_heads], out))
        held, position = held + 1, position + 1
    if int(status):
        raise RuntimeError(f"device status {int(status)}: {kvi.kvi_status_str(int(status))}")
    return dict(a=a, pool=pool, cache4=cache4, table=table, block=block, memory=memory, ctx=ctx, prompt=prompt_out,
                held=held, position=position, evictions=evictions, weights=weights, where=where, last=last,
                slots=slots, facts=ids)


def main():
    r = run()
    print(f"{r['facts'].numel()} facts injected ({r['memory']} tokens), prompt to position {r['ctx']}, "
          f"generated to {r['position']}, {r['evictions']} evictions, {r['held']} keys held")
    heavy = r["weights"][0][0, 0, :r["held"]].topk(5)
    print("most attended positions of layer 0, head 0:",
          [int(r["where"][0][0, 0, i]) for i in heavy.indices], [round(float(v), 2) for v in heavy.values])


if __name__ == "__main__":
    main()
