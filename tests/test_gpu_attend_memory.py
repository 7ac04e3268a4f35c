"""The example's whole path: injected memory, prompt attention, the 4-bit
cache, generation and eviction together, its outputs against float64."""
import pytest
import torch

import pre_rope_kv_gb300 as kvi
from examples import attend_memory
from tests import attn_check as ac

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(q_heads=8, kv_heads=8, head_dim=128, block=32, prompt=150, steps=40, budget=96),
                                dict(layers=1, q_heads=20, kv_heads=4, head_dim=96, k=3, prompt=1, steps=70, budget=40, recent=8)])
def test_request_from_memory_to_eviction(kw):
    r = attend_memory.run(**kw)
    a = r["a"]
    G, H, D = a.q_heads // a.kv_heads, a.kv_heads, a.head_dim
    assert r["evictions"] > 0
    for layer, (q, out) in enumerate(r["prompt"]):  # over the bf16 pool
        flat = r["pool"][layer].view(2, -1, H, D)[:, r["slots"](0, r["ctx"])].double()
        last = torch.arange(q.shape[0], device="cuda") + r["memory"]
        for h in range(H):
            hs = slice(h * G, (h + 1) * G)
            ref, _, _, pv, size = ac.attend(q[:, hs].double(), flat[0, :, h], flat[1, :, h], last, D ** -0.5)
            ac.check_out(out[:, hs], ref, pv, size, 1, (layer, h))
    n = r["held"]
    for layer, (q, out) in enumerate(r["last"]):    # over what is left of the 4-bit cache
        k, v = (torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvi.kvi_cache4_read(r["cache4"], layer, r["slots"](0, n), k, v, status)
        for h in range(H):
            where = r["where"][layer][0, h, :n]
            assert len(set(where.tolist())) == n and int(where.max()) == r["position"] - 1
            assert set(range(4)) <= set(where.tolist())                    # the sinks stay
            # (reading back rounds each element to bf16 once: 2^-8 of it in K and V)
            hs = slice(h * G, (h + 1) * G)
            ref, _, _, pv, size = ac.attend(q[:, hs].double(), k[:, h].double(), v[:, h].double(),
                                            torch.tensor([n - 1], device="cuda"), D ** -0.5)
            extra = 2.0 ** -8 * (2 * size + 1) * pv
            assert bool(((out[:, hs].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -7 + 2.0 ** -17 * (1 + size)) * pv
                         + extra).all())
