"""A serving step around injected memory: the operators, their workloads and their plain forms.

What a step runs before and in its attention, from the requests' lengths on:

  tables  block tables, slots and positions of a step's new rows, made from the
          requests' lengths on the GPU; blocks come from a ring of free ones and
          those of finished requests go back to it;
  rotate  queries and keys normalised per head (or not), rotated to their
          positions and, with the values, put into the paged cache in one pass;
          where asked the keys before rotation too, as a fact store keeps them;
  window  causal attention of packed prompts (or single tokens) over the paged
          cache in which a row sees the last keys and a few first ones;
  shared  attention of a batch whose requests share a long prefix (one memory,
          many users), the prefix computed once for all.

`run` computes them in plain torch (`own` false) or through this package
(`own` true); `exact` gives the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
POSITIONS = 40960  # positions that the rotation's coefficients are kept for


# ------------------------------------------------------------------ workloads

def listed():
    tables = dict(op="tables", block=16)
    rotate = dict(op="rotate", q_heads=32, kv_heads=8, head_dim=128, block=16, norm=True, pages=True, plain=False,
                  fused=True, interleaved=False, llama3=False)
    window = dict(op="window", q_heads=32, kv_heads=8, head_dim=128, block=16, lse=False, fused=False)
    shared = dict(op="shared", q_heads=32, kv_heads=8, head_dim=128, block=16, lse=False, fused=False)
    return [
        # one decoding step of 64 users, three of whom have finished; the rows padded to a captured graph's 72: latency
        dict(tables, name="tables_step", requests=64, new_lo=1, new_hi=1, ctx_lo=700, ctx_hi=2300, shared=0, gone=3,
             pad=8, spread=1),
        # 16 ragged prompts behind one memory of 100 blocks
        dict(tables, name="tables_prompts", requests=16, new_lo=1, new_hi=2048, ctx_lo=1600, ctx_hi=1600, shared=1600,
             gone=0, pad=0, spread=2),
        # many requests of odd lengths in larger pages, a ninth of them finished
        dict(tables, name="tables_many", requests=1000, new_lo=1, new_hi=500, ctx_lo=0, ctx_hi=900, shared=0, gone=111,
             block=32, pad=77, spread=3),
        # the rows of one decoding step of 64 users: latency
        dict(rotate, name="rotate_step", tokens=64, skip=0),
        # a small model without norms, Llama 3.1 frequencies, neighbouring pairs, rows alone (for a 4-bit cache): latency
        dict(rotate, name="rotate_small", q_heads=4, kv_heads=2, head_dim=64, tokens=131, norm=False, pages=False,
             interleaved=True, llama3=True, skip=0),
        # a long prompt whose keys also go into a fact store before rotation; some rows are padding
        dict(rotate, name="rotate_prompt", tokens=8192, plain=True, skip=9),
        # one token each of 64 users with long caches
        dict(window, name="window_single_tokens", requests=64, q_lo=1, q_hi=1, mem_lo=2000, mem_hi=16000, window=1024,
             sink=4, spread=4),
        # ragged prompts behind a system prefix of 64 tokens that stays visible, q taken from a fused projection
        dict(window, name="window_packed", requests=16, q_lo=1, q_hi=2048, mem_lo=0, mem_hi=1600, window=512, sink=64,
             lse=True, fused=True, spread=5),
        # a whole long prompt
        dict(window, name="window_whole", requests=1, q_lo=8192, q_hi=8192, mem_lo=0, mem_hi=0, window=2048, sink=4,
             spread=6),
        # a few users' single tokens over the memory of one conversation: latency
        dict(shared, name="shared_few", requests=8, q_lo=1, q_hi=1, prefix=1600, mem_lo=20, mem_hi=200, spread=7),
        # 64 users' single tokens over a large memory
        dict(shared, name="shared_users", requests=64, q_lo=1, q_hi=1, prefix=10240, mem_lo=30, mem_hi=700, spread=8),
        # the questions of 24 users over the same memory
        dict(shared, name="shared_questions", requests=24, q_lo=5, q_hi=37, prefix=10240, mem_lo=0, mem_hi=100, lse=True,
             fused=True, spread=9),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["tables", "rotate", "window", "window", "shared", "shared"])
    block = rng.choice([16, 16, 32, 64])
    if op == "tables":
        requests = _log(rng, 1, 2000)
        hi = _log(rng, 1, min(4000, 200000 // requests))
        shared = rng.choice([0, 0, 3 * block, 64 * block])
        ctx = shared + _log(rng, 1, 1500)
        return dict(op=op, block=block, requests=requests, new_lo=rng.choice([0, 1, hi]) if hi < 64 else 1, new_hi=hi,
                    ctx_lo=shared, ctx_hi=ctx, shared=shared, gone=rng.randrange(0, 1 + requests // 4),
                    pad=rng.choice([0, 5, 64]), spread=rng.randrange(1 << 20))
    kv_heads = rng.choice([1, 2, 4, 8])
    c = dict(op=op, kv_heads=kv_heads, q_heads=kv_heads * rng.choice([1, 2, 4, 5, 8]), block=block,
             head_dim=rng.choice([64, 128, 128]))
    if op == "rotate":
        return dict(c, tokens=_log(rng, 1, 7000), norm=rng.random() < 0.7, pages=rng.random() < 0.7,
                    plain=rng.random() < 0.4, fused=rng.random() < 0.6, interleaved=rng.random() < 0.3,
                    llama3=rng.random() < 0.3, skip=rng.choice([0, 0, 3, 17]))
    c.update(lse=rng.random() < 0.5, fused=rng.random() < 0.5, spread=rng.randrange(1 << 20))
    if op == "window":
        if rng.random() < 0.4:  # single tokens over long caches
            requests = _log(rng, 1, 64)
            hi = _log(rng, 100, 16000)
            return dict(c, requests=requests, q_lo=1, q_hi=1, mem_lo=hi // rng.choice([1, 3]), mem_hi=hi,
                        window=_log(rng, 1, 4096), sink=rng.choice([0, 1, 4, 64]))
        requests = _log(rng, 1, 16)
        top = max(1, min(8192, int(math.sqrt(8192 * 8192 * 32 / (2.0 * requests * c["q_heads"])))))
        q_hi = _log(rng, 1, top)
        mem_hi = _log(rng, 1, min(top, 2000))
        return dict(c, requests=requests, q_lo=_log(rng, 1, q_hi), q_hi=q_hi, mem_lo=rng.choice([0, mem_hi]),
                    mem_hi=mem_hi, window=_log(rng, 1, 4096), sink=rng.choice([0, 1, 4, 64, 200]))
    requests = _log(rng, 1, 64)
    q_hi = _log(rng, 1, max(1, min(200, 700 // requests)))
    mem_hi = _log(rng, 1, 700)
    return dict(c, requests=requests, q_lo=rng.choice([1, q_hi]), q_hi=q_hi, prefix=block * _log(rng, 1, 10240 // block),
                mem_lo=rng.choice([0, mem_hi]), mem_hi=mem_hi)


def _lens(c):
    """Per-request lengths of a case: (new rows, keys before them); of the shared form without its prefix."""
    rs = np.random.RandomState(c["spread"])
    r = c["requests"]
    lo, hi = ("new_lo", "new_hi") if c["op"] == "tables" else ("q_lo", "q_hi")
    low = math.log(max(c[lo], 0.5))
    n = np.clip(np.rint(np.exp(low + rs.uniform(size=r) * (math.log(c[hi]) - low))), c[lo], c[hi]).astype(np.int64)
    n[rs.randint(r)] = c[hi]
    if c["op"] != "tables":
        return n, rs.randint(c["mem_lo"], c["mem_hi"] + 1, r)
    ctx = rs.randint(c["ctx_lo"], c["ctx_hi"] + 1, r)
    n[rs.permutation(r)[:c["gone"]]] = -1
    return n, ctx


def _blocks(keys, block):
    return (keys + block - 1) // block


def work(c):
    if c["op"] == "tables":
        n, ctx = _lens(c)
        live = np.maximum(n, 0)
        taken = int(np.sum(_blocks(ctx + live, c["block"]) - _blocks(ctx, c["block"])))
        back = int(np.sum((_blocks(ctx, c["block"]) - c["shared"] // c["block"])[n < 0]))
        rows = int(live.sum())
        # lengths in and out, starts; a slot and a position per row; blocks from the ring to a table, and back
        return {"bytes": 16 * len(n) + 12 * (rows + c["pad"]) + 8 * taken + 8 * back, "flops": 4 * rows}
    h, d, hq = c["kv_heads"], c["head_dim"], c["q_heads"]
    if c["op"] == "rotate":
        t = c["tokens"]
        live = t - (t // c["skip"] if c["skip"] else 0)
        row = 2 * d
        wide = hq + h                                           # q and k in, q out
        moved = t * row * (wide + hq + (h if c["plain"] else 0)) + (live * row * 3 * h if c["pages"] else t * row * h)
        return {"bytes": moved + 12 * t, "flops": t * wide * d * (7 if c["norm"] else 3)}
    n, mem = _lens(c)
    rows = int(n.sum())
    out = rows * hq * (d * 4 + (4 if c["lse"] else 0))
    if c["op"] == "shared":
        pairs = rows * c["prefix"] + int(np.sum(n * mem + n * (n + 1) // 2))
        return {"bytes": (c["prefix"] + int(np.sum(n + mem))) * h * d * 4 + out, "flops": pairs * hq * d * 4}
    pairs = keys = 0
    for a, b in zip(n.tolist(), mem.tolist()):
        p = np.arange(b, a + b)
        low = np.maximum(0, p - c["window"] + 1)
        pairs += int(np.sum(p + 1 - low + np.minimum(c["sink"], low)))
        keys += a + b - int(low[0]) + min(c["sink"], int(low[0]))
    return {"bytes": keys * h * d * 4 + out, "flops": pairs * hq * d * 4}


# --------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, n, heads, d):
    """K-like or V-like rows: Gaussian, the channels of different sizes."""
    size = torch.exp(0.5 * torch.randn(heads, d, generator=g, device=DEV))
    out = torch.empty(n, heads, d, device=DEV, dtype=torch.bfloat16)
    for i in range(0, n, 1 << 16):
        m = min(1 << 16, n - i)
        out[i:i + m] = (torch.randn(m, heads, d, generator=g, device=DEV) * size).to(torch.bfloat16)
    return out


def _tables(g, ctx, block, shared=0):
    """Shuffled block tables [R][width] int32 for these lengths, the first `shared` blocks the same in all
    rows, and the blocks that they use."""
    need = _blocks(ctx, block) - shared
    width = int(max(1, need.max() + shared))
    total = int(need.sum()) + shared
    ids = torch.randperm(total + 3, generator=g, device=DEV).to(torch.int32)
    first = torch.from_numpy(np.cumsum(need) - need).to(DEV)
    col = torch.arange(width, device=DEV)
    at = torch.where(col[None] < shared, col[None], shared + first[:, None] + (col[None] - shared)).clamp_(max=total)
    inside = col[None] < torch.from_numpy(need + shared).to(DEV)[:, None]
    return torch.where(inside, ids[at], torch.zeros_like(ids[at])).contiguous(), total + 3


def prepare(case, seed):
    c, g = case, _generator(seed)
    return {"tables": _prepare_tables, "rotate": _prepare_rotate}.get(c["op"], _prepare_attention)(c, g)


def _prepare_tables(c, g):
    n, ctx = _lens(c)
    b, r = c["block"], c["requests"]
    live = np.maximum(n, 0)
    table, used = _tables(g, ctx, b, c["shared"] // b)
    need = int(np.sum(_blocks(ctx + live, b) - _blocks(ctx, b)))
    blocks = used + need + 40
    width = int(max(1, _blocks(ctx + live, b).max()))
    s = {"case": c, "rows": int(live.sum()) + c["pad"], "blocks": blocks}
    s["table"] = torch.zeros(r, width, dtype=torch.int32, device=DEV)
    s["table"][:, :min(width, table.shape[1])] = table[:, :width]
    # the ring of free blocks, anywhere in its circle; what it holds elsewhere means nothing
    head = int(torch.randint(0, 5 * blocks, (1,), generator=g, device=DEV))
    spare = (used + torch.randperm(blocks - used, generator=g, device=DEV)).to(torch.int32)
    s["free"] = torch.full((blocks,), -1, dtype=torch.int32, device=DEV)
    s["free"][(head + torch.arange(blocks - used, device=DEV)) % blocks] = spare
    s["at"] = torch.tensor([head, head + blocks - used], dtype=torch.int64, device=DEV)
    s["at_out"] = torch.zeros_like(s["at"])
    s["ctx"], s["new"] = (torch.from_numpy(x.astype(np.int32)).to(DEV) for x in (ctx, n))
    s["ctx_out"] = torch.zeros_like(s["ctx"])
    s["q_start"] = torch.zeros(r + 1, dtype=torch.int32, device=DEV)
    s["positions"] = torch.zeros(s["rows"], dtype=torch.int32, device=DEV)
    s["slots"] = torch.zeros(s["rows"], dtype=torch.int64, device=DEV)
    if own:
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def _prepare_rotate(c, g):
    t, hq, h, d, b = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"], c["block"]
    s = {"case": c}
    qkv = _rows(g, t, hq + 2 * h, d)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
    if not c["fused"]:
        s["q"], s["k"], s["v"] = (x.contiguous() for x in (s["q"], s["k"], s["v"]))
    if t > 256:  # prompts: runs of positions
        s["positions"] = (torch.arange(t, device=DEV) + int(torch.randint(0, 2000, (1,), generator=g, device=DEV))).to(torch.int32)
    else:
        s["positions"] = torch.randint(0, POSITIONS, (t,), generator=g, device=DEV).to(torch.int32)
    s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None
                        for _ in range(2))
    s["q_out"] = torch.zeros(t, hq, d, dtype=torch.bfloat16, device=DEV)
    s["k_out"] = None if c["pages"] else torch.zeros(t, h, d, dtype=torch.bfloat16, device=DEV)
    s["plain"] = torch.zeros(t, h, d, dtype=torch.bfloat16, device=DEV) if c["plain"] else None
    s["slots"] = s["pool"] = None
    if c["pages"]:
        blocks = _blocks(t, b) + 2
        order = torch.randperm(blocks, generator=g, device=DEV)
        row = torch.arange(t, device=DEV)
        s["slots"] = order[row // b] * b + row % b if t > 256 else torch.randperm(blocks * b, generator=g, device=DEV)[:t]
        if c["skip"]:
            s["slots"][c["skip"] - 1::c["skip"]] = -1
        s["pool"] = torch.zeros(2, blocks, b, h, d, dtype=torch.bfloat16, device=DEV)
    if own:
        import pre_rope_kv_gb300 as kvi
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["attention"] = kvi.attention(hq, h, d)
        s["spec"] = kvi.rope(theta=500000.0, pairing=kvi.ROPE_PAIR_INTERLEAVED if c["interleaved"] else kvi.ROPE_PAIR_HALF,
                             llama3=(8.0, 1.0, 4.0, 8192.0) if c["llama3"] else None)
        kvi.kvi_prepare_rope_ex(s["spec"], d, POSITIONS)
        s["cache"] = kvi.paged_cache([s["pool"]], b) if c["pages"] else None
    return s


def _prepare_attention(c, g):
    h, d, b, hq, r = c["kv_heads"], c["head_dim"], c["block"], c["q_heads"], c["requests"]
    n, mem = _lens(c)
    prefix = c["prefix"] if c["op"] == "shared" else 0
    ctx = prefix + mem + n
    s = {"case": c, "max_q": int(n.max()), "max_ctx": int(ctx.max())}
    s["table"], blocks = _tables(g, ctx, b, prefix // b)
    s["ctx"] = torch.from_numpy(ctx.astype(np.int32)).to(DEV)
    total = int(n.sum())
    s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)
    wide = hq + 2 * h if c["fused"] else hq  # q as a part of a fused q, k, v projection
    s["q"] = torch.randn(total, wide, d, generator=g, device=DEV).to(torch.bfloat16)[:, :hq]
    s["out"] = torch.zeros(total, hq, d, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros(total, hq, device=DEV) if c["lse"] else None
    s["pool"] = torch.empty(2, blocks, b, h, d, dtype=torch.bfloat16, device=DEV)
    for plane in s["pool"]:
        plane.copy_(_rows(g, blocks * b, h, d).view(blocks, b, h, d))
    if own:
        import pre_rope_kv_gb300 as kvi
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["attention"] = kvi.attention(hq, h, d)
        s["cache"] = kvi.paged_cache([s["pool"]], b)
        if prefix:
            need = kvi.kvi_attn_shared_workspace_bytes(s["attention"], r, total, s["max_q"], s["max_ctx"], prefix)
        else:
            need = kvi.kvi_attn_prompt_workspace_bytes(s["attention"], r, total, s["max_q"], s["max_ctx"])
        s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ operators

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import pre_rope_kv_gb300 as kvi
    c = s["case"]
    if c["op"] == "tables":
        kvi.kvi_batch_tables(s["ctx"], s["new"], s["table"], c["block"], c["shared"], s["free"], s["at"], s["at_out"],
                             s["ctx_out"], s["q_start"], s["positions"], s["slots"], s["status"])
        return _tables_results(s)
    if c["op"] == "rotate":
        kvi.kvi_norm_rope(s["attention"], s["spec"], POSITIONS, s["positions"], s["q"], s["k"], s["q_out"], s["k_out"],
                          s["status"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, k_plain=s["plain"],
                          v=s["v"] if c["pages"] else None, cache=s["cache"], layer=0, slots=s["slots"])
        return {"q": s["q_out"], "k": s["k_out"], "plain": s["plain"], "pool": s["pool"]}
    if c["op"] == "window":
        kvi.kvi_attn_window(s["attention"], s["q"], s["q_start"], s["max_q"], s["ctx"], s["max_ctx"], s["table"], s["cache"],
                            0, c["window"], c["sink"], s["out"], s["ws"], s["status"], lse=s["lse"])
    else:
        kvi.kvi_attn_shared(s["attention"], s["q"], s["q_start"], s["max_q"], s["ctx"], s["max_ctx"], s["table"], s["cache"],
                            0, c["prefix"], s["out"], s["ws"], s["status"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _tables_results(s):
    return {"table": s["table"], "free": s["free"], "at": s["at_out"], "ctx": s["ctx_out"], "q_start": s["q_start"],
            "positions": s["positions"], "slots": s["slots"]}


def _run_plain(s):
    return {"tables": _plain_tables, "rotate": _plain_rotate, "window": _plain_window, "shared": _plain_shared}[s["case"]["op"]](s)


def _plain_tables(s):
    c = s["case"]
    b, first, blocks = c["block"], c["shared"] // c["block"], s["blocks"]
    ctx, new = s["ctx"].long(), s["new"].long()
    gone, n = new < 0, new.clamp_min(0)
    had, has = (ctx + b - 1) // b, (ctx + n + b - 1) // b
    start = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)])
    need = has - had
    need_at = need.cumsum(0) - need
    back = torch.where(gone, (had - first).clamp_min(0), torch.zeros_like(had))
    back_at = back.cumsum(0) - back
    # tables: each new column takes the next free block
    col = torch.arange(s["table"].shape[1], device=DEV)
    fresh = (col >= had[:, None]) & (col < has[:, None])
    taken = s["free"][(s["at"][0] + need_at[:, None] + col - had[:, None]) % blocks]
    returned = gone[:, None] & (col >= first) & (col < had[:, None])
    ring = torch.where(returned, (s["at"][1] + back_at[:, None] + col - first) % blocks, blocks)
    free = torch.cat([s["free"], s["free"][:1]]).scatter_(0, ring.flatten(), s["table"].flatten())[:-1]
    s["table"] = torch.where(fresh, taken, s["table"])
    s["free"] = free
    s["at_out"] = s["at"] + torch.stack([need.sum(), back.sum()])
    s["ctx_out"] = torch.where(gone, 0, ctx + n).to(torch.int32)
    s["q_start"] = start.to(torch.int32)
    # rows
    row = torch.arange(s["rows"], device=DEV)
    of = torch.searchsorted(start, row, right=True) - 1
    real = of < len(n)
    of = of.clamp_max(len(n) - 1)
    p = ctx[of] + row - start[of]
    at = torch.where(real, p // b, torch.zeros_like(p))
    s["positions"] = torch.where(real, p, 0).to(torch.int32)
    s["slots"] = torch.where(real, s["table"][of, at].long() * b + p % b, -1)
    return _tables_results(s)


def _angles(c, positions):
    """cos and sin of position * frequency, from 64 bits."""
    d = c["head_dim"]
    w = 500000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=DEV) / d)
    if c["llama3"]:
        turns = 8192.0 * w / (2 * math.pi)  # of the original context
        keep = ((turns - 1.0) / 3.0).clamp(0, 1)
        w = keep * w + (1 - keep) * w / 8.0
    a = positions.double()[:, None, None] * w
    return a.cos().float(), a.sin().float()


def _plain_rotate(s):
    c = s["case"]
    cos, sin = _angles(c, s["positions"])

    def turned(x):
        a, b = (x[..., 0::2], x[..., 1::2]) if c["interleaved"] else x.chunk(2, -1)
        y = (a * cos - b * sin, b * cos + a * sin)
        return torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1)

    def normed(x, w):
        x = x.float()
        return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()

    q, k = normed(s["q"], s["wq"]), normed(s["k"], s["wk"])
    s["q_out"] = turned(q).to(torch.bfloat16)
    rotated = turned(k).to(torch.bfloat16)
    if c["plain"]:
        s["plain"] = k.to(torch.bfloat16)
    if c["pages"]:
        flat = s["pool"].view(2, -1, *s["k"].shape[1:])
        live = s["slots"] >= 0
        flat[0, s["slots"][live]] = rotated[live]
        flat[1, s["slots"][live]] = s["v"][live]
    else:
        s["k_out"] = rotated
    return {"q": s["q_out"], "k": s["k_out"], "plain": s["plain"], "pool": s["pool"]}


def _softmax(score, seen):
    """(weights, sum of exp(score - top), top) of scores [..., keys] where seen; top is finite."""
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min_(-3e38)
    p = score.sub_(top).exp_()
    return p, p.sum(-1, keepdim=True), top


def _padded(s):
    """Padded queries [R][H][G][n][D] float32, which of them are real [R][n], their rows in q, and their positions."""
    c = s["case"]
    start = s["q_start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(s["max_q"], device=DEV)
    real = i < n[:, None]
    at = torch.where(real, start[:-1, None] + i, torch.zeros_like(i))
    q = s["q"][at].float().view(c["requests"], s["max_q"], c["kv_heads"], -1, c["head_dim"]).permute(0, 2, 3, 1, 4)
    return q * (1.0 / math.sqrt(c["head_dim"])), real, at, s["ctx"].long()[:, None] - n[:, None] + i


def _put(s, o, lse, real, at):
    """Results o [R][H][G][n][D] and lse [R][H][G][n][1] into the state's rows."""
    rows = at[real]
    s["out"][rows] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real].to(torch.bfloat16)
    if s["lse"] is not None:
        s["lse"][rows] = lse[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[real]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_window(s):
    c = s["case"]
    q, real, at, p = _padded(s)
    keys = s["pool"][:, s["table"].long()].flatten(2, 3)[:, :, :s["max_ctx"]]      # [2][R][keys][H][D]
    k, v = (x.transpose(1, 2).unsqueeze(2).float() for x in keys)                  # [R][H][1][keys][D]
    j = torch.arange(k.shape[3], device=DEV)
    seen = (j <= p[..., None]) & ((j < c["sink"]) | (j > p[..., None] - c["window"]))
    w, total, top = _softmax(torch.matmul(q, k.transpose(-1, -2)), seen[:, None, None])
    return _put(s, torch.matmul(w, v) / total.clamp_min(1e-38), top + total.log(), real, at)


def _plain_shared(s):
    c = s["case"]
    q, real, at, p = _padded(s)
    r, h, g, n, d = q.shape
    first = c["prefix"] // c["block"]
    # the prefix once for all: every request's rows of a head together
    k0, v0 = (x.flatten(0, 1)[:c["prefix"]].transpose(0, 1).float() for x in s["pool"][:, s["table"][0, :first].long()])
    rows = q.permute(1, 0, 2, 3, 4).reshape(h, r * g * n, d)
    w0, t0, m0 = (x.view(h, r, g, n, -1).transpose(0, 1) for x in
                  _softmax(torch.matmul(rows, k0.transpose(-1, -2)), torch.ones(1, dtype=torch.bool, device=DEV)))
    o0 = torch.matmul(w0.transpose(0, 1).reshape(h, r * g * n, -1), v0).view(h, r, g, n, d).transpose(0, 1)
    # each request's own keys
    keys = s["pool"][:, s["table"][:, first:].long()].flatten(2, 3)[:, :, :s["max_ctx"] - c["prefix"]]
    k1, v1 = (x.transpose(1, 2).unsqueeze(2).float() for x in keys)
    seen = c["prefix"] + torch.arange(k1.shape[3], device=DEV) <= p[..., None]
    w1, t1, m1 = _softmax(torch.matmul(q, k1.transpose(-1, -2)), seen[:, None, None])
    o1 = torch.matmul(w1, v1)
    top = torch.maximum(m0, m1)
    f0, f1 = (m0 - top).exp(), (m1 - top).exp()
    total = t0 * f0 + t1 * f1
    return _put(s, (o0 * f0 + o1 * f1) / total, top + total.log(), real, at)


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "rotate": _exact_rotate}.get(case["op"], _exact_attention)(case, s)


def _exact_tables(c, s):
    """Request after request, on the host."""
    b, blocks = c["block"], s["blocks"]
    table, free = s["table"].cpu().numpy(), s["free"].cpu().numpy()
    head, tail = s["at"].tolist()
    ctx_out, starts = [], [0]
    positions, slots = np.zeros(s["rows"], np.int32), np.full(s["rows"], -1, np.int64)
    for r, (ctx, n) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
        if n < 0:
            for col in range(c["shared"] // b, -(-ctx // b)):
                free[tail % blocks] = table[r, col]
                tail += 1
            ctx, n = 0, 0
        else:
            for col in range(-(-ctx // b), -(-(ctx + n) // b)):
                table[r, col] = free[head % blocks]
                head += 1
        p = np.arange(ctx, ctx + n)
        at = slice(starts[-1], starts[-1] + n)
        positions[at] = p
        slots[at] = table[r, p // b].astype(np.int64) * b + p % b
        ctx_out.append(ctx + n)
        starts.append(starts[-1] + n)
    new = {"table": table, "free": free, "at": np.array([head, tail]), "ctx": np.array(ctx_out, np.int32),
           "q_start": np.array(starts, np.int32), "positions": positions, "slots": slots}
    return {k: torch.from_numpy(v).to(DEV) for k, v in new.items()}


def _exact_rotate(c, s):
    d, half = c["head_dim"], c["head_dim"] // 2
    w = []
    for i in range(half):
        f = math.pow(500000.0, -2.0 * i / d)
        if c["llama3"]:
            wavelength = 2.0 * math.pi / f
            if wavelength > 8192.0:
                f /= 8.0
            elif wavelength >= 2048.0:
                mix = (8192.0 / wavelength - 1.0) / 3.0
                f = mix * f + (1.0 - mix) * f / 8.0
        w.append(f)
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * torch.tensor(w, dtype=torch.float64, device=DEV))[:, None]
    pairs = torch.arange(d, device=DEV).view(half, 2) if c["interleaved"] else torch.arange(d, device=DEV).view(2, half).T

    def normed(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * weight.double()
        return x

    def turned(x):
        z = torch.complex(x[..., pairs[:, 0]], x[..., pairs[:, 1]]) * turn
        y = torch.empty_like(x)
        y[..., pairs[:, 0]], y[..., pairs[:, 1]] = z.real, z.imag
        return y

    k = normed(s["k"], s["wk"])
    out = {"q": turned(normed(s["q"], s["wq"])), "k": None if c["pages"] else turned(k), "plain": k if c["plain"] else None,
           "pool": None}
    if c["pages"]:
        out["pool"] = s["pool"].double()
        flat = out["pool"].view(2, -1, *k.shape[1:])
        slots = s["slots"].cpu()
        live = torch.nonzero(slots >= 0).flatten().to(DEV)
        flat[0].index_copy_(0, s["slots"][live], turned(k)[live])
        flat[1].index_copy_(0, s["slots"][live], s["v"].double()[live])
    return out


def _exact_attention(c, s):
    h, d, b = c["kv_heads"], c["head_dim"], c["block"]
    group = c["q_heads"] // h
    n_q = np.diff(s["q_start"].cpu().numpy()).tolist()
    ctx = s["ctx"].tolist()
    sees_all = c["op"] == "shared"
    if sum(n * min(x, 10 ** 9 if sees_all else c["window"] + c["sink"] + 1024 + n % 1024) for n, x in zip(n_q, ctx)) * c["q_heads"] * d > 6e11:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["out"].shape[:2], dtype=torch.float64, device=DEV)
    start = 0
    for r, (n, keys) in enumerate(zip(n_q, ctx)):
        blocks = s["table"][r, :_blocks(keys, b)].long()
        for j in range(h):
            k, v = (s["pool"][x, blocks, :, j].reshape(-1, d)[:keys].double() for x in (0, 1))
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                last = torch.arange(keys - n + i, keys - n + i + m, device=DEV)[:, None]
                low = 0 if sees_all else max(0, int(last[0]) - c["window"] + 1)
                at = torch.arange(low, int(last[-1]) + 1, device=DEV)
                if low:
                    at = torch.cat([torch.arange(min(c["sink"], low), device=DEV), at])
                hidden = at > last
                if not sees_all:
                    hidden |= (at >= c["sink"]) & (at <= last - c["window"])
                score = torch.einsum("ngd,kd->gnk", s["q"][start + i:start + i + m, j * group:(j + 1) * group].double(), k[at])
                score = (score / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                log_sum = torch.logsumexp(score, -1)
                out[start + i:start + i + m, j * group:(j + 1) * group] = \
                    torch.einsum("gnk,kd->ngd", torch.exp(score - log_sum[..., None]), v[at])
                lse[start + i:start + i + m, j * group:(j + 1) * group] = log_sum.T
        start += n
    return {"out": out, "lse": lse if c["lse"] else None}
