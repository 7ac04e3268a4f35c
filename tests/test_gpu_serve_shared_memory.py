"""The serving loop of examples/serve_shared_memory.py: every step's positions, slots,
pages and attention against plain references, and blocks that come back."""
import pytest
import torch

from examples import serve_shared_memory
from tests import attn_check as ac
from tests import step_check as sc
from tests.test_gpu_norm_rope import close

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Watch:
    def __init__(self):
        self.ctx = None
        self.steps = 0

    def __call__(self, s):
        self.steps += 1
        assert int(s["status"]) == 0
        a, block = s["a"], s["block"]
        Hq, H, D = a.q_heads, a.kv_heads, a.head_dim
        users = s["table"].shape[0]
        n_q = (s["q_start"][1:] - s["q_start"][:-1]).tolist()
        ctx = s["ctx"].tolist()
        rows = int(s["q_start"][-1])
        omega = sc.frequencies(s["theta"], D)
        # positions and slots
        for r in range(users):
            q0, n = int(s["q_start"][r]), n_q[r]
            p = torch.arange(ctx[r] - n, ctx[r], device=DEV)
            assert torch.equal(s["positions"][q0:q0 + n].long(), p)
            assert torch.equal(s["slots"][q0:q0 + n], s["table"][r][p // block].long() * block + p % block)
            if self.ctx is not None:
                assert ctx[r] in (self.ctx[r] + n, 0) and (ctx[r] or n == 0)
        assert bool((s["slots"][rows:] == -1).all())
        self.ctx = ctx
        # blocks: each user's own are nobody else's, and none is free
        first = s["shared"] // block
        own = [s["table"][r, first:-(-ctx[r] // block)].tolist() if ctx[r] else [] for r in range(users)]
        head, tail = s["free_at"].tolist()
        free = [int(s["free"][i % s["blocks"]]) for i in range(head, tail)]
        used = s["table"][0, :first].tolist() + sum(own, []) + free
        assert sorted(used) == list(range(s["blocks"]))
        for layer, pool in enumerate(s["pool"]):
            flat = pool.view(2, -1, H, D)
            qkv = s["qkv"][layer][:rows]
            wq, wk = s["weights"][layer]
            pos, slots = s["positions"][:rows], s["slots"][:rows]
            for got, x, w in ((s["q"][layer][:rows], qkv[:, :Hq], wq), (flat[0, slots], qkv[:, Hq:Hq + H], wk)):
                ref, both = sc.rotated(sc.normed(x, w, 1e-6), pos, omega, False)
                close(got, ref, both)
            assert torch.equal(flat[1, slots], qkv[:, Hq + H:])
            for r in range(users):
                q0, n = int(s["q_start"][r]), n_q[r]
                if n == 0:
                    continue
                at = torch.arange(ctx[r], device=DEV)
                at = s["table"][r][at // block].long() * block + at % block
                i, j = torch.arange(ctx[r] - n, ctx[r], device=DEV)[:, None], torch.arange(ctx[r], device=DEV)
                seen = j <= i
                if layer % 2:
                    seen &= (j > i - s["window"]) | (j < s["sink"])
                for h in range(H):
                    hs = slice(h * Hq // H, (h + 1) * Hq // H)
                    ref, _, pv, size = sc.attend(s["q"][layer][q0:q0 + n, hs].double(), flat[0, at, h].double(), flat[1, at, h].double(),
                                                 seen, a.scale)
                    ac.check_out(s["out"][layer][q0:q0 + n, hs], ref, pv, size, 1, (layer, r, h))


@pytest.mark.parametrize("kw", [dict(), dict(users=40, head_dim=128, kv_heads=8, q_heads=32, k=100, facts=400, block=32, steps=9, window=200,
                                             seed=1), dict(users=1, question=1, block=8, steps=5)])
def test_a_run(kw):
    w = Watch()
    r = serve_shared_memory.run(watch=w, **kw)
    assert w.steps == 1 + kw.get("steps", 20)
    users = kw.get("users", 6)
    assert r["ctx"].tolist().count(0) == (1 if users > 1 else 0)
