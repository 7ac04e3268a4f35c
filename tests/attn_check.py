"""Plain float64 references and inputs for the attention and 4-bit cache tests.

Tolerances.  A result differs from the exact one by
  - its own rounding to bf16 (8 significant bits, so half a unit in the last
    place is at most 2^-8 of the number): 2^-8 |out|;
  - the rounding of the softmax weights P to bf16 before the second product:
    at most 2^-8 of each term, so 2^-8 sum p |v| (twice that over the 4-bit
    cache, where P * step rounds again);
  - float32 arithmetic: a score is off by at most a few 2^-24 of sum |q k| scale
    (its largest over the keys: `size`), exp2 by 2^-22, the sums by a few ulps:
    together below 2^-17 (1 + size) of sum p |v|.
"""
import math

import numpy as np
import torch

import pre_rope_kv_gb300 as kvi

DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def tables(g, ctx, block, extra=3, width=None):
    """Shuffled tables [R][width] (unused entries: an id far outside) and the number of blocks."""
    need = [(c + block - 1) // block for c in ctx]
    total = sum(need) + extra
    ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    t = torch.full((len(ctx), width or max(1, max(need))), -7, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(need):
        t[r, :n] = ids[at:at + n]
        at += n
    return t, total


def attend(q, k, v, last, scale):
    """q [n][G][D], k and v [keys][D] (float64), row i sees keys 0..last[i].
    Returns out, lse, weights [n][G][keys], sum p |v|, the largest sum |q k| scale."""
    n, G, D = q.shape
    keys = k.shape[0]
    if keys == 0:
        z = torch.zeros(n, G, D, dtype=torch.float64, device=q.device)
        return z, torch.full((n, G), -math.inf, dtype=torch.float64, device=q.device), \
            torch.zeros(n, G, 0, dtype=torch.float64, device=q.device), z, 0.0
    s = torch.einsum("ngd,kd->ngk", q, k) * scale
    size = float((torch.einsum("ngd,kd->ngk", q.abs(), k.abs()) * scale).max()) if n else 0.0
    hidden = torch.arange(keys, device=q.device)[None, None] > last[:, None, None]
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(hidden, torch.zeros_like(s), torch.exp(s - lse[..., None]))
    return (torch.einsum("ngk,kd->ngd", p, v), lse, p, torch.einsum("ngk,kd->ngd", p, v.abs()), size)


def check_out(got, ref, pv, size, p_roundings, what=""):
    tol = 2.0 ** -8 * ref.abs() + (p_roundings * 2.0 ** -8 + 2.0 ** -17 * (1 + size)) * pv + 1e-30
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol)[bad].max()),
                                 bad.nonzero()[0].tolist())


def check_lse(got, ref, size):
    empty = torch.isinf(ref)
    assert torch.equal(torch.isinf(got) & (got < 0), empty)
    err = (got.double() - ref)[~empty].abs()
    assert err.numel() == 0 or float(err.max()) <= 2.0 ** -17 * (1 + size)


# ------------------------------------------------------------ the 4-bit format

def quantise(x):
    """(step bf16 [..., G], code int64 [..., D]) of bf16 rows, from the definition."""
    v = x.double().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1)
    step = (top / 7).to(torch.bfloat16)
    s = step.double().unsqueeze(-1)
    ok = torch.isfinite(v).all(-1, keepdim=True)
    code = torch.where((s > 0) & ok, torch.round(v / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(v))
    step = torch.where(ok.squeeze(-1), step, torch.full_like(step, math.nan))
    return step, code.clamp(-7, 7).flatten(-2).long()


def dequantise(step, code):
    return (code.double().unflatten(-1, (-1, 32)) * step.double().unsqueeze(-1)).flatten(-2)


def page_bytes(B, D):
    return B * D + B * (D // 32) * 4


def pages_from(step_k, code_k, step_v, code_v, B):
    """The layout of kvi_cache4_layer_bytes' comment, byte by byte, on the host:
    rows [blocks * B][H][...] -> uint8 [blocks][H][page bytes]."""
    n, H, D = code_k.shape
    G, blocks = D // 32, n // B
    out = np.zeros((blocks, H, page_bytes(B, D)), np.uint8)
    nib = [(c.cpu().numpy() + 8).astype(np.uint8).reshape(blocks, B, H, D) for c in (code_k, code_v)]
    st = [s.cpu().contiguous().view(torch.int16).numpy().view(np.uint16).reshape(blocks, B, H, G) for s in (step_k, step_v)]
    for off in range(B):
        for d in range(D):
            g, x = d // 32, d % 32
            word = (off * 4 + x // 8) * G + g
            out[:, :, word * 4 + (x % 8) // 2] |= nib[0][:, off, :, d] << (4 * (x % 2))
            word = (off // 2 * 8 + x // 4) * G + g
            n4 = x % 4 + 4 * (off % 2)
            out[:, :, B * D // 2 + word * 4 + n4 // 2] |= nib[1][:, off, :, d] << (4 * (n4 % 2))
        for g in range(G):
            for base, s in ((B * D + (off * G + g) * 2, st[0]),
                            (B * D + B * G * 2 + ((off // 2 * G + g) * 2 + off % 2) * 2, st[1])):
                out[:, :, base] = s[:, off, :, g] & 255
                out[:, :, base + 1] = s[:, off, :, g] >> 8
    return torch.from_numpy(out)


class Cache4:
    """A 4-bit pool of random rows, made by kvi_cache4_write, and its values."""

    def __init__(self, g, H, D, B, blocks, k=None, v=None):
        n = blocks * B
        size = torch.exp(0.5 * randn(g, H, D))
        self.k = (randn(g, n, H, D) * size).to(torch.bfloat16) if k is None else k
        self.v = (randn(g, n, H, D) * size.flip(-1)).to(torch.bfloat16) if v is None else v
        self.pool = torch.full((blocks, H, page_bytes(B, D)), 0xff, dtype=torch.uint8, device=DEV)
        self.cache = kvi.cache4([self.pool], B, H, D)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        kvi.kvi_cache4_write(self.cache, 0, self.k, self.v, torch.arange(n, device=DEV), self.status)
        self.kd, self.vd = (dequantise(*quantise(x)) for x in (self.k, self.v))
        self.B, self.H, self.D = B, H, D

    def rows(self, table, ctx):
        """Slots of a request's positions."""
        p = torch.arange(ctx, device=DEV)
        return table[p // self.B].long() * self.B + p % self.B


def workspace(n):
    return torch.full((max(n, 256),), 0xff, dtype=torch.uint8, device=DEV)  # nothing may need initial values
