"""Attention over injected memory: the operators, their workloads and their plain forms.

What runs once the memory facts of a request lie in the paged cache:

  prompt  attention of the request's own tokens (packed prompts of different
          lengths, causal, grouped heads) over the paged bf16 cache that holds
          the injected memory and the prompt itself;
  store   rows of K and V written into a cache held in 4 bits, and read back;
  decode  attention of one new token per request over the 4-bit cache, where
          asked adding each key's softmax weight to its accumulated weight;
  evict   reduction of a 4-bit cache to a budget of keys by that accumulated
          weight, followed by the decoding step over what is left.

`run` computes them in plain torch (`own` false) or through this package
(`own` true); `exact` gives the same from the definitions in 64 bits.

Layout of a 4-bit page, for one block of B tokens and one KV head (bytes, with
G = D / 32 groups of 32 channels, each with a bf16 step; an element is
step * (nibble - 8)):
  K codes  [B][4][G] words: word (t, g) holds channels 32 g + 8 t + n, n = 0..7,
           nibble n
  V codes  [B / 2][8][G] words: word (s, g) holds channels 32 g + 4 s + j of
           tokens 2 i (nibble j) and 2 i + 1 (nibble 4 + j)
  K steps  [B][G] bf16
  V steps  [B / 2][G][2] bf16
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ workloads

def listed():
    prompt = dict(op="prompt", q_heads=32, kv_heads=8, head_dim=128, block=16, lse=False, fused=False)
    store = dict(op="store", kv_heads=8, head_dim=128, block=16)
    decode = dict(op="decode", q_heads=32, kv_heads=8, head_dim=128, block=16)
    evict = dict(op="evict", q_heads=32, kv_heads=8, head_dim=128, block=16, sink=4, recent=64)
    return [
        # one user's short question behind 50 injected facts (64-token system prefix first): latency
        dict(prompt, name="prompt_question", requests=1, q_lo=37, q_hi=37, mem_lo=1564, mem_hi=1564, spread=1),
        # a small model with two KV heads: odd prompts behind a few facts: latency
        dict(prompt, name="prompt_small_heads", q_heads=4, kv_heads=2, head_dim=64, requests=3, q_lo=5, q_hi=131,
             mem_lo=0, mem_hi=80, spread=2, lse=True),
        # 64 concurrent users, one token each, over the bf16 cache
        dict(prompt, name="prompt_single_tokens", requests=64, q_lo=1, q_hi=1, mem_lo=700, mem_hi=2300, spread=3),
        # a batch of ragged prompts, with and without memory, q taken from a fused projection
        dict(prompt, name="prompt_packed", requests=16, q_lo=1, q_hi=2048, mem_lo=0, mem_hi=1600, spread=4, lse=True,
             fused=True),
        # a whole long prompt without memory: the dense causal case
        dict(prompt, name="prompt_whole", requests=1, q_lo=8192, q_hi=8192, mem_lo=0, mem_hi=0, spread=5),
        # the K/V of one decoding step of 64 users
        dict(store, name="store_step", tokens=64, skip=0),
        # conversion of a whole memory prefix, some rows left out
        dict(store, name="store_prefix", tokens=65537, skip=9),
        # one user's decoding step
        dict(decode, name="decode_one", requests=1, ctx_lo=1601, ctx_hi=1601, weights=False, spread=6),
        # 64 users' decoding step, weights accumulated for a later eviction
        dict(decode, name="decode_weights", requests=64, ctx_lo=700, ctx_hi=2300, weights=True, spread=7),
        # long contexts in larger pages
        dict(decode, name="decode_long", requests=16, ctx_lo=24000, ctx_hi=32768, block=32, weights=False, spread=8),
        # one user's cache cut back to 1024 keys
        dict(evict, name="evict_one", requests=1, ctx_lo=1601, ctx_hi=1601, budget=1024, spread=9),
        # 64 users' caches cut back to 2000 keys
        dict(evict, name="evict_many", requests=64, ctx_lo=1900, ctx_hi=4100, budget=2000, spread=10),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(max(v, lo), hi)
    return v - 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["prompt", "prompt", "store", "decode", "decode", "evict"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    c = dict(op=op, kv_heads=kv_heads, block=rng.choice([16, 16, 32, 64]), head_dim=rng.choice([64, 128, 128]))
    if op == "store":
        return dict(c, tokens=_log(rng, 1, 65000), skip=rng.choice([0, 0, 3, 17]))
    c.update(q_heads=kv_heads * group, spread=rng.randrange(1 << 20))
    if op == "prompt":
        requests = _log(rng, 1, 64)
        # the padded scores of the plain form stay below those of the listed cases
        top = max(1, min(8192, int(math.sqrt(8192 * 8192 * 32 / (2.0 * requests * c["q_heads"])))))
        q_hi = _log(rng, 1, top)
        mem_hi = _log(rng, 1, min(top, 4000))
        return dict(c, requests=requests, q_lo=_log(rng, 1, q_hi), q_hi=q_hi, mem_lo=rng.choice([0, mem_hi // 2, mem_hi]),
                    mem_hi=mem_hi, lse=rng.random() < 0.5, fused=rng.random() < 0.5)
    requests = _log(rng, 1, 64)
    top = min(32768, 16 * 28000 * 8 // (requests * kv_heads))
    if op == "decode":
        hi = _log(rng, 1, top)
        return dict(c, requests=requests, ctx_lo=rng.choice([hi, max(1, hi // 2)]), ctx_hi=hi, weights=rng.random() < 0.5)
    hi = _log(rng, 130, min(top, 8000))
    budget = _log(rng, 80, hi)
    return dict(c, requests=requests, ctx_lo=rng.choice([hi, max(1, hi // 2)]), ctx_hi=hi, budget=budget,
                sink=rng.choice([0, 4]), recent=rng.choice([0, 1, 64]))


def _lens(c):
    """Per-request lengths of a case: (query tokens, keys)."""
    rs = np.random.RandomState(c["spread"])
    r = c["requests"]
    if c["op"] == "prompt":
        u = rs.uniform(size=r)
        q = np.clip(np.rint(np.exp(math.log(c["q_lo"]) + u * (math.log(c["q_hi"]) - math.log(c["q_lo"])))), c["q_lo"], c["q_hi"])
        q = q.astype(np.int64)
        q[rs.randint(r)] = c["q_hi"]
        return q, q + rs.randint(c["mem_lo"], c["mem_hi"] + 1, r)
    return np.ones(r, np.int64), rs.randint(c["ctx_lo"], c["ctx_hi"] + 1, r)


def work(c):
    h, d = c["kv_heads"], c["head_dim"]
    page = h * (d + d // 8)  # bytes of one token's K and V in 4 bits, with their steps
    if c["op"] == "store":
        t = c["tokens"]
        live = t - (t // c["skip"] if c["skip"] else 0)
        return {"bytes": live * (2 * 2 * h * d * 2 + 2 * page) + 8 * t, "flops": live * 2 * h * d * 4}
    q, ctx = _lens(c)
    hq = c["q_heads"]
    if c["op"] == "prompt":
        pairs = int(np.sum(q * ctx - q * (q - 1) // 2))
        return {"bytes": int(np.sum(ctx)) * h * d * 4 + int(np.sum(q)) * hq * (d * 4 + (4 if c["lse"] else 0)),
                "flops": pairs * hq * d * 4}
    n = int(np.sum(ctx))
    step = lambda keys: keys * page + len(ctx) * hq * d * 4  # noqa: E731
    if c["op"] == "decode":
        return {"bytes": step(n) + (n * h * 8 if c["weights"] else 0), "flops": n * hq * d * 4}
    left = int(np.sum(np.minimum(ctx, c["budget"])))
    # every weight and position read; the kept ones written and, in the decoding step, the weights updated
    return {"bytes": n * h * 8 + n * h * 8 + left * h * 8 + step(left), "flops": left * hq * d * 4}


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


def _tables(g, ctx, block):
    """Shuffled block tables [R][max_blocks] int32 for these lengths, and the pool's blocks."""
    need = (ctx + block - 1) // block
    width = int(max(1, need.max()))
    total = int(need.sum()) + 3
    ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    first = torch.from_numpy(np.cumsum(need) - need).to(DEV)
    col = torch.arange(width, device=DEV)
    at = (first[:, None] + col[None, :]).clamp_(max=total - 1)
    table = torch.where(col[None, :] < torch.from_numpy(need).to(DEV)[:, None], ids[at], torch.zeros_like(ids[at]))
    return table.contiguous(), total


def _quantise(x):
    """Steps and codes of rows [..., D]: groups of 32 channels, step = bf16(max |x| / 7),
    code = x / step rounded to the nearest, ties to even, from -7 to 7; 0 where the step is 0."""
    v = x.float().unflatten(-1, (-1, 32))
    step = (v.abs().amax(-1) / 7).to(torch.bfloat16)
    s = step.float().unsqueeze(-1)
    code = torch.where(s > 0, torch.round(v / s), torch.zeros_like(v)).clamp_(-7, 7)
    return step, code.flatten(-2).to(torch.int8)


def _pack(k, v, block):
    """The 4-bit pages [blocks][H][bytes] of rows k, v [blocks * block][H][D]."""
    n, h, d = k.shape
    groups, blocks = d // 32, n // block
    parts = []
    for x, is_v in ((k, False), (v, True)):
        step, code = _quantise(x)
        nib = (code + 8).to(torch.uint8)
        if not is_v:
            # [blk][B][H][G][4 t][8 n] -> [blk][H][B][t][G][n]
            a = nib.view(blocks, block, h, groups, 4, 8).permute(0, 2, 1, 4, 3, 5).reshape(blocks, h, -1, 2)
            s = step.view(blocks, block, h, groups).permute(0, 2, 1, 3)
        else:
            # [blk][B/2][2][H][G][8 s][4 j] -> [blk][H][B/2][s][G][2][j]
            a = nib.view(blocks, block // 2, 2, h, groups, 8, 4).permute(0, 3, 1, 5, 4, 2, 6).reshape(blocks, h, -1, 2)
            s = step.view(blocks, block // 2, 2, h, groups).permute(0, 3, 1, 4, 2)
        parts.append((a[..., 0] | (a[..., 1] << 4), s.reshape(blocks, h, -1).contiguous().view(torch.uint8)))
    return torch.cat([parts[0][0], parts[1][0], parts[0][1], parts[1][1]], dim=-1).contiguous()


def _unpack(pages, block, d):
    """(K, V) values, float32, of pages [..., bytes]: each [..., block, D]."""
    groups = d // 32
    lead = pages.shape[:-1]
    kc, vc, ks, vs = pages.split([block * d // 2, block * d // 2, 2 * block * groups, 2 * block * groups], dim=-1)

    def values(c):
        return torch.stack([c & 15, c >> 4], dim=-1).flatten(-2).float() - 8

    k = values(kc).view(*lead, block, 4, groups, 8).transpose(-3, -2)
    k = k * ks.contiguous().view(torch.bfloat16).view(*lead, block, groups, 1, 1).float()
    v = values(vc).view(*lead, block // 2, 8, groups, 2, 4)
    v = v * vs.contiguous().view(torch.bfloat16).view(*lead, block // 2, 1, groups, 2, 1).float()
    v = v.movedim(-2, -4).movedim(-2, -3)  # [..., B/2, 2, G, 8, 4]
    return k.reshape(*lead, block, d), v.reshape(*lead, block, d)


def prepare(case, seed):
    c, g = case, _generator(seed)
    h, d, b = c["kv_heads"], c["head_dim"], c["block"]
    s = {"case": c}
    if c["op"] == "store":
        t = c["tokens"]
        blocks = (t + b - 1) // b + 2
        s["k"], s["v"] = _rows(g, t, h, d), _rows(g, t, h, d)
        slots = torch.randperm(blocks * b, generator=g, device=DEV)[:t]
        if t > 64:  # a prefix lies in whole blocks, one after another
            order = torch.randperm(blocks, generator=g, device=DEV)
            row = torch.arange(t, device=DEV)
            slots = order[row // b] * b + row % b
        if c["skip"]:
            slots[c["skip"] - 1::c["skip"]] = -1
        s["slots"] = slots
        s["pool"] = torch.zeros(blocks, h, b * (d + d // 8), dtype=torch.uint8, device=DEV)
        s["k_back"], s["v_back"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    else:
        q_len, ctx = _lens(c)
        hq, r = c["q_heads"], c["requests"]
        s["table"], blocks = _tables(g, ctx, b)
        s["ctx"] = torch.from_numpy(ctx.astype(np.int32)).to(DEV)
        s["max_q"], s["max_ctx"] = int(q_len.max()), int(ctx.max())
        total = int(q_len.sum())
        s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)).to(DEV)
        wide = hq + 2 * h if c.get("fused") else hq  # q as a part of a fused q, k, v projection
        s["q"] = torch.randn(total, wide, d, generator=g, device=DEV).to(torch.bfloat16)[:, :hq]
        s["out"] = torch.zeros(total, hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(total, hq, device=DEV) if c.get("lse") else None
        k, v = _rows(g, blocks * b, h, d), _rows(g, blocks * b, h, d)
        if c["op"] == "prompt":
            s["pool"] = torch.stack([k.view(blocks, b, h, d), v.view(blocks, b, h, d)])
        else:
            s["pool"] = _pack(k, v, b)
        del k, v
        if c.get("weights") or c["op"] == "evict":
            width = s["max_ctx"] + 7
            s["weights"] = torch.rand(r, h, width, generator=g, device=DEV).square_()
            if c["op"] == "evict":
                # a quarter of the keys have no weight yet: ties
                s["weights"] *= torch.rand(r, h, width, generator=g, device=DEV) > 0.25
                s["pos"] = torch.argsort(torch.rand(r, h, width, generator=g, device=DEV) +
                                         2.0 * (torch.arange(width, device=DEV) >= s["ctx"][:, None, None]), dim=-1).to(torch.int32)
                s["weights_out"], s["pos_out"] = torch.zeros_like(s["weights"]), torch.zeros_like(s["pos"])
                s["ctx_out"] = torch.zeros_like(s["ctx"])
        else:
            s["weights"] = None
    if own:
        import pre_rope_kv_gb300 as kvi
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if c["op"] != "store":
            s["attention"] = kvi.attention(hq, h, d)
        if c["op"] == "prompt":
            s["cache"] = kvi.paged_cache([s["pool"]], b)
            n = kvi.kvi_attn_prompt_workspace_bytes(s["attention"], r, total, s["max_q"], s["max_ctx"])
        else:
            s["cache"] = kvi.cache4([s["pool"]], b, h, d)
            n = 0
        if c["op"] in ("decode", "evict"):
            n = kvi.kvi_attn_decode4_workspace_bytes(s["attention"], r, s["max_ctx"], s["weights"] is not None)
        if c["op"] == "evict":
            n = max(n, kvi.kvi_cache4_evict_workspace_bytes(h, r, s["max_ctx"]))
        s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ operators

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import pre_rope_kv_gb300 as kvi
    c = s["case"]
    if c["op"] == "prompt":
        kvi.kvi_attn_prompt(s["attention"], s["q"], s["q_start"], s["max_q"], s["ctx"], s["max_ctx"], s["table"],
                            s["cache"], 0, s["out"], s["ws"], s["status"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "store":
        kvi.kvi_cache4_write(s["cache"], 0, s["k"], s["v"], s["slots"], s["status"])
        kvi.kvi_cache4_read(s["cache"], 0, s["slots"], s["k_back"], s["v_back"], s["status"])
        return {"k": s["k_back"], "v": s["v_back"]}
    if c["op"] == "decode":
        kvi.kvi_attn_decode4(s["attention"], s["q"], s["ctx"], s["max_ctx"], s["table"], s["cache"], 0, s["out"],
                             s["ws"], s["status"], weights=s["weights"])
        return {"out": s["out"], "weights": s["weights"]}
    kvi.kvi_cache4_evict(s["cache"], 0, s["ctx"], s["max_ctx"], s["table"], c["budget"], c["sink"], c["recent"],
                         s["weights"], s["pos"], s["weights_out"], s["pos_out"], s["ctx_out"], s["ws"], s["status"])
    kvi.kvi_attn_decode4(s["attention"], s["q"], s["ctx_out"], min(s["max_ctx"], c["budget"]), s["table"], s["cache"],
                         0, s["out"], s["ws"], s["status"], weights=s["weights_out"])
    return {"ctx": s["ctx_out"], "pos": s["pos_out"], "weights": s["weights_out"], "out": s["out"]}


def _attend(q, k, v, seen):
    """Softmax attention in float32: q [..., G, n, D], k and v [..., 1, keys, D],
    seen [..., 1, n, keys].  Returns the output, the log of the sum and the weights;
    a row that sees nothing gives zeros and minus infinity."""
    score = torch.matmul(q * (1.0 / math.sqrt(q.shape[-1])), k.transpose(-1, -2))
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min_(-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= total.clamp_min(1e-38)
    return torch.matmul(p, v), (top + total.log()).squeeze(-1), p


def _run_plain(s):
    return {"prompt": _plain_prompt, "store": _plain_store, "decode": _plain_decode, "evict": _plain_evict}[s["case"]["op"]](s)


def _plain_prompt(s):
    c = s["case"]
    h, d, b, r = c["kv_heads"], c["head_dim"], c["block"], c["requests"]
    group = c["q_heads"] // h
    keys = s["pool"][:, s["table"].long()].flatten(2, 3)[:, :, :s["max_ctx"]]      # [2][R][keys][H][D]
    k, v = (x.transpose(1, 2).unsqueeze(2).float() for x in keys)                  # [R][H][1][keys][D]
    start = s["q_start"].long()
    n_q = start[1:] - start[:-1]
    i = torch.arange(s["max_q"], device=DEV)
    real = i[None] < n_q[:, None]                                                  # [R][n]
    at = torch.where(real, start[:-1, None] + i[None], torch.zeros_like(i[None]))
    q = s["q"][at].float().view(r, s["max_q"], h, group, d).permute(0, 2, 3, 1, 4)  # [R][H][G][n][D]
    last = s["ctx"].long()[:, None] - n_q[:, None] + i[None]                       # the last key a row sees
    seen = torch.arange(k.shape[3], device=DEV)[None, None, :] <= last[:, :, None]
    o, lse, _ = _attend(q, k, v, seen[:, None, None])
    s["out"][at[real]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real].to(torch.bfloat16)
    if s["lse"] is not None:
        s["lse"][at[real]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[real]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_store(s):
    live = s["slots"] >= 0
    out = {}
    for name in ("k", "v"):
        step, code = _quantise(s[name])
        back = (code.float().unflatten(-1, (-1, 32)) * step.float().unsqueeze(-1)).flatten(-2).to(torch.bfloat16)
        out[name] = s[name + "_back"] = torch.where(live[:, None, None], back, s[name + "_back"])
    return out


def _plain_step(s, k, v, ctx, weights):
    """One decoding step over values k, v [R][H][keys][D]; adds to weights [R][H][width]."""
    c = s["case"]
    h, r = c["kv_heads"], c["requests"]
    q = s["q"].float().view(r, h, -1, 1, c["head_dim"])
    seen = torch.arange(k.shape[2], device=DEV)[None] < ctx[:, None]
    o, _, p = _attend(q, k.unsqueeze(2), v.unsqueeze(2), seen[:, None, None, None])
    s["out"].copy_(o.reshape(r, c["q_heads"], -1))
    if weights is not None:
        weights[:, :, :k.shape[2]] += p.sum((2, 3))


def _values(s):
    """K and V values [R][H][keys][D] that the block tables reach."""
    c = s["case"]
    k, v = _unpack(s["pool"][s["table"].long()], c["block"], c["head_dim"])        # [R][blocks][H][B][D]
    return (x.transpose(1, 2).flatten(2, 3)[:, :, :s["max_ctx"]] for x in (k, v))


def _plain_decode(s):
    k, v = _values(s)
    _plain_step(s, k, v, s["ctx"], s["weights"])
    return {"out": s["out"], "weights": s["weights"]}


def _plain_evict(s):
    c = s["case"]
    w, pos = s["weights"], s["pos"]
    slot = torch.arange(w.shape[-1], device=DEV).expand_as(w)
    ctx = s["ctx"].long()[:, None, None]
    new = ctx.clamp(max=c["budget"])
    here = slot < ctx
    newest = torch.where(here, pos, torch.full_like(pos, -1)).amax(-1, keepdim=True)
    safe = (pos < c["sink"]) | (pos > newest - c["recent"])
    key = torch.where(safe, torch.full_like(w, math.inf), w).masked_fill(~here, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(here).scatter_(-1, order, slot < new)
    src = slot.clone()
    src[(slot < new) & ~kept] = slot[(slot >= new) & kept]     # both in the order of (request, head, slot)
    s["weights_out"].copy_(torch.where(slot < new, w.gather(-1, src), torch.where(here, 0.0, s["weights_out"])))
    s["pos_out"].copy_(torch.where(slot < new, pos.gather(-1, src), torch.where(here, -1, s["pos_out"])))
    s["ctx_out"].copy_(new[:, 0, 0])
    top = min(s["max_ctx"], c["budget"])
    k, v = (x.gather(2, src[:, :, :top, None].expand(-1, -1, -1, x.shape[-1])) for x in _values(s))
    _plain_step(s, k, v, s["ctx_out"], s["weights_out"])
    return {"ctx": s["ctx_out"], "pos": s["pos_out"], "weights": s["weights_out"], "out": s["out"]}


# ------------------------------------------------- the definitions in 64 bits

def _exact_values(pool, table, n, block, d, head):
    """K and V of one request and head, float64 [n][D], element by element from the page layout."""
    i = torch.arange(n, device=DEV)[:, None]
    ch = torch.arange(d, device=DEV)[None, :]
    groups, g, x = d // 32, ch // 32, ch % 32
    page = pool[table.long(), head]                                                # [blocks][bytes]
    blk, off = i // block, i % block
    k_byte = off * (d // 2) + ((x // 8) * groups + g) * 4 + (x % 8) // 2
    v_byte = block * d // 2 + (off // 2) * d + ((x // 4) * groups + g) * 4 + (off % 2) * 2 + (x % 4) // 2
    steps = page[:, block * d:].contiguous().view(torch.bfloat16).double()
    out = []
    for byte, step in ((k_byte, off * groups + g), (v_byte, block * groups + ((off // 2) * groups + g) * 2 + off % 2)):
        two = page[blk, byte].to(torch.int64)
        out.append((((two >> (4 * (x % 2))) & 15) - 8).double() * steps[blk, step])
    return out


def _exact_rows(q, k, v, last):
    """q [n][G][D] over k, v [keys][D], row i up to key last[i]: output and log of the sum."""
    score = torch.einsum("ngd,kd->gnk", q, k) / math.sqrt(q.shape[-1])
    score.masked_fill_(torch.arange(len(k), device=DEV)[None, None] > last[None, :, None], -math.inf)
    lse = torch.logsumexp(score, -1)
    p = torch.exp(score - lse[..., None]).nan_to_num(0.0)
    return torch.einsum("gnk,kd->ngd", p, v), lse.T, p


def exact(case, seed):
    c, s = case, prepare(case, seed)
    h, d, b = c["kv_heads"], c["head_dim"], c["block"]
    if c["op"] == "store":
        out = {}
        for name in ("k", "v"):
            rows = s[name].double().view(c["tokens"], h, d // 32, 32)
            step = (rows.abs().max(-1, keepdim=True).values / 7).to(torch.bfloat16).double()
            back = torch.where(step > 0, torch.round(rows / step) * step, torch.zeros_like(rows)).reshape(c["tokens"], h, d)
            back[s["slots"] < 0] = 0
            out[name] = back
        return out
    group = c["q_heads"] // h
    q_len, ctx = _lens(c)
    if c["op"] == "prompt" and float(np.sum(q_len * ctx)) * c["q_heads"] * d > 6e11:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["out"].shape[:2], dtype=torch.float64, device=DEV)
    w = s["weights"].double() if s.get("weights") is not None else None
    if c["op"] == "evict":
        w_in, pos_in, w, pos, ctx_out = s["weights"].cpu().numpy(), s["pos"].cpu().numpy(), s["weights_out"].double(), s["pos_out"], s["ctx_out"]
    start = 0
    for r in range(c["requests"]):
        n, keys = int(q_len[r]), int(ctx[r])
        for j in range(h):
            q = s["q"][start:start + n, j * group:(j + 1) * group].double()
            if c["op"] == "prompt":
                k, v = (s["pool"][x, s["table"][r].long(), :, j].reshape(-1, d)[:keys].double() for x in (0, 1))
                last = torch.arange(n, device=DEV) + (keys - n)
                for i in range(0, n, 1024):
                    o, l, _ = _exact_rows(q[i:i + 1024], k, v, last[i:i + 1024])
                    out[start + i:start + i + 1024, j * group:(j + 1) * group][:len(o)] = o
                    lse[start + i:start + i + 1024, j * group:(j + 1) * group][:len(o)] = l
                continue
            k, v = _exact_values(s["pool"], s["table"][r], keys, b, d, j)
            if c["op"] == "evict":
                left = min(keys, c["budget"])
                p, x = pos_in[r, j, :keys].astype(np.int64), w_in[r, j, :keys].astype(np.float64)
                safe = (p < c["sink"]) | (p >= p.max() + 1 - c["recent"])
                kept = np.sort(np.lexsort((np.arange(keys), -x, ~safe))[:left])
                src = np.arange(left)
                src[np.setdiff1d(src, kept)] = kept[kept >= left]
                at = torch.from_numpy(src).to(DEV)
                k, v = k[at], v[at]
                w[r, j, :keys], pos[r, j, :keys] = 0, -1
                w[r, j, :left], pos[r, j, :left] = s["weights"][r, j, at].double(), s["pos"][r, j, at]
                ctx_out[r] = left
            o, _, p = _exact_rows(q, k, v, torch.full((1,), len(k) - 1, device=DEV))
            out[start, j * group:(j + 1) * group] = o[0]
            if w is not None:
                w[r, j, :len(k)] += p.sum((0, 1))
        start += n
    if c["op"] == "prompt":
        return {"out": out, "lse": lse if c["lse"] else None}
    if c["op"] == "decode":
        return {"out": out, "weights": w}
    return {"ctx": ctx_out, "pos": pos, "weights": w, "out": out}
