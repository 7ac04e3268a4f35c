"""Plain float64 references of a serving step's operators: attention with any mask,
norms with rotation, and block tables made request by request."""
import math

import torch

DEV = "cuda"


def attend(q, k, v, seen, scale):
    """q [n][G][D], k and v [keys][D] (float64), seen [n][keys].  Returns out, lse, sum p |v| and
    the largest sum |q k| scale; a row that sees nothing gives zeros and minus infinity."""
    s = torch.einsum("ngd,kd->ngk", q, k) * scale
    size = float((torch.einsum("ngd,kd->ngk", q.abs(), k.abs()) * scale)[seen[:, None].expand_as(s)].max()) if bool(seen.any()) else 0.0
    hidden = ~seen[:, None]
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(hidden, torch.zeros_like(s), torch.exp(s - lse[..., None]))
    p = torch.where(torch.isinf(lse)[..., None], torch.zeros_like(p), p)
    v = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))
    return torch.einsum("ngk,kd->ngd", p, v), lse, torch.einsum("ngk,kd->ngd", p, v.abs()), size


def frequencies(theta, D, llama3=None):
    """omega_i, i < D / 2, from the header's description."""
    out = []
    for i in range(D // 2):
        w = theta ** (-2.0 * i / D)
        if llama3:
            factor, low, high, original = llama3
            length = 2 * math.pi / w
            if length > original / low:
                w /= factor
            elif length >= original / high:
                g = (original / length - low) / (high - low)
                w = g * w + (1 - g) * w / factor
        out.append(w)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def normed(x, weight, eps):
    x = x.double()
    return x if weight is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def rotated(y, positions, omega, interleaved):
    """(rotated rows, |a| + |b| of each element's pair) of y [T][H][D] float64."""
    ang = positions.double()[:, None, None] * omega
    c, s = ang.cos(), ang.sin()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else y.chunk(2, -1)
    parts = (a * c - b * s, b * c + a * s)
    both = a.abs() + b.abs()
    if interleaved:
        return torch.stack(parts, -1).flatten(-2), both.repeat_interleave(2, -1)
    return torch.cat(parts, -1), torch.cat([both, both], -1)


def tables(ctx, new, table, block, shared, free, at, total_rows):
    """kvi_batch_tables on lists: (table, free, at, ctx_out, q_start, positions, slots, errors), errors
    a set of 'capacity' and 'range'."""
    R, width, n_blocks = len(ctx), len(table[0]), len(free)
    table, given, free = [list(t) for t in table], list(free), list(free)
    errors = set()
    head, tail = at
    ring = 0 <= head <= tail <= head + n_blocks
    if not ring:
        errors.add("range")
    avail = tail - head if ring else 0
    good, need, back = [], [], []
    for c, n in zip(ctx, new):
        end = c + max(n, 0)
        ok = 0 <= c <= width * block and not (n > 0 and c < shared)
        if not ok:
            errors.add("range")
        elif end > width * block:
            errors.add("capacity")
            ok = False
        good.append(ok)
        need.append(-(-end // block) - -(-c // block) if ok and n > 0 else 0)
        back.append(max(0, -(-c // block) - shared // block) if ok and n < 0 else 0)
    returns = ring and sum(back) <= n_blocks - avail
    if ring and not returns:
        errors.add("capacity")
    asked_blocks = asked_rows = taken = returned = 0
    ctx_out, q_start, positions, slots = [], [0], [], []
    for r in range(R):
        n = max(new[r], 0) if good[r] else 0
        first = asked_blocks
        asked_blocks += need[r]
        asked_rows += n
        got = n > 0 and (need[r] == 0 or asked_blocks <= avail) and asked_rows <= total_rows
        if n > 0 and not got:
            errors.add("capacity")
        if got:
            for i in range(need[r]):
                table[r][-(-ctx[r] // block) + i] = given[(head + first + i) % n_blocks]
            taken += need[r]
            for p in range(ctx[r], ctx[r] + n):
                block_id = table[r][p // block]
                inside = 0 <= block_id < n_blocks
                if not inside:
                    errors.add("range")
                positions.append(p)
                slots.append(block_id * block + p % block if inside else -1)
        if returns and good[r] and new[r] < 0:
            for i in range(back[r]):
                free[(tail + returned + i) % n_blocks] = table[r][shared // block + i]
            returned += back[r]
            ctx_out.append(0)
        else:
            ctx_out.append(ctx[r] + n if got else ctx[r])
        q_start.append(len(slots))
    positions += [0] * (total_rows - len(positions))
    slots += [-1] * (total_rows - len(slots))
    return table, free, [head + taken, tail + returned], ctx_out, q_start, positions, slots, errors
