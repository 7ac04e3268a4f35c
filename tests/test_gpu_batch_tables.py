"""kvi_batch_tables against tables made request by request: lengths of every kind,
finished requests, rings that wrap, prefixes, padding, and what does not fit."""
import random

import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import step_check as sc

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    def __init__(self, ctx, new, block=16, shared=0, width=None, spare=10, head=0, pad=0, rows=None, seed=0):
        rng = random.Random(seed)
        self.ctx, self.new, self.block, self.shared = list(ctx), list(new), block, shared
        need = sum(-(-(c + n) // block) - -(-c // block) for c, n in zip(ctx, new) if n > 0)
        held = [-(-c // block) for c in ctx]
        width = width or max(1, max(-(-(c + max(n, 0)) // block) for c, n in zip(ctx, new)))
        first = shared // block
        total = first + sum(max(0, h - first) for h in held) + max(0, need + spare)
        ids = list(range(total))
        rng.shuffle(ids)
        prefix, at = ids[:first], first
        self.table = []
        for h in held:
            own = max(0, min(h, width) - first)
            self.table.append((prefix[:min(first, width)] + ids[at:at + own] + [-9] * width)[:width])
            at += own
        self.free = [-3] * total
        for i, b in enumerate(ids[at:]):
            self.free[(head + i) % total] = b
        self.at = [head, head + total - at]
        self.rows = sum(max(n, 0) for n in new) + pad if rows is None else rows

    def run(self):
        def dev(x, t=torch.int32):
            return torch.tensor(x, dtype=t, device=DEV)

        self.t = dict(ctx=dev(self.ctx), new=dev(self.new), table=dev(self.table), free=dev(self.free), at=dev(self.at, torch.int64),
                      at_out=dev([-1, -1], torch.int64), ctx_out=dev([-7] * len(self.ctx)), q_start=dev([-7] * (len(self.ctx) + 1)),
                      positions=dev([-7] * self.rows), slots=dev([-7] * self.rows, torch.int64), status=dev([0]))
        self.call()

    def call(self, stream=None):
        t = self.t
        kvi.kvi_batch_tables(t["ctx"], t["new"], t["table"], self.block, self.shared, t["free"], t["at"], t["at_out"], t["ctx_out"],
                             t["q_start"], t["positions"], t["slots"], t["status"], stream=stream)

    def check(self):
        table, free, at, ctx, q_start, positions, slots, errors = sc.tables(
            self.ctx, self.new, self.table, self.block, self.shared, self.free, self.at, self.rows)
        t = {k: v.tolist() for k, v in self.t.items()}
        assert t["q_start"] == q_start and t["ctx_out"] == ctx
        assert t["positions"] == positions and t["slots"] == slots
        assert t["table"] == table and t["free"] == free and t["at_out"] == at
        codes = {"capacity": kvi.ERR_CAPACITY, "range": kvi.ERR_OUT_OF_RANGE}
        assert t["status"][0] in ({codes[e] for e in errors} or {0})
        assert t["ctx"] == self.ctx and t["new"] == self.new and t["at"] == self.at
        return errors


@pytest.mark.parametrize("block", [1, 16, 24])
@pytest.mark.parametrize("R", [1, 2, 63, 64, 257, 1000, 4096])
def test_requests(R, block):
    rng = random.Random(R + block)
    ctx = [rng.choice([0, 1, block - 1, block, block + 1, rng.randrange(0, 300)]) for _ in range(R)]
    new = [rng.choice([1, 1, 0, -1, block, rng.randrange(0, 60), 2 * block + 1]) for _ in range(R)]
    c = Case(ctx, new, block, head=rng.randrange(0, 10 ** 12), pad=rng.choice([0, 1, 70]), seed=R)
    c.run()
    assert not c.check()


@pytest.mark.parametrize("head", [0, 3, 10 ** 15 + 7])
def test_prefixes_and_long_prompts(head):
    c = Case([64, 64, 70, 64, 100, 64], [2048, 1, 5000, -1, -1, 0], 16, shared=64, head=head, pad=5)
    c.run()
    assert not c.check()


@pytest.mark.parametrize("R", [3, 40, 700])
def test_blocks_that_run_out(R):
    """Requests are served in order; later ones that need no block still get their rows."""
    rng = random.Random(R)
    for spare in (-1, -5, -R, 0):
        c = Case([rng.randrange(0, 40) for _ in range(R)], [rng.choice([1, 1, 20, -1]) for _ in range(R)], 16, spare=spare, seed=R)
        c.run()
        errors = c.check()
        assert errors == ({"capacity"} if spare < 0 and c.at[1] - c.at[0] < sum(
            -(-(a + n) // 16) - -(-a // 16) for a, n in zip(c.ctx, c.new) if n > 0) else set())


def test_rows_that_run_out():
    for rows in (0, 1, 5, 24):
        c = Case([5, 0, 30, 2], [5, 10, 5, 5], rows=rows)
        c.run()
        assert c.check() == {"capacity"}


def test_lengths_that_do_not_fit():
    c = Case([5, -1, 30, 100, 47, 2, 3], [5, 10, 19, 5, 1, 5, 0], width=3, shared=0)
    c.new[-1] = 2 ** 31 - 1
    c.run()
    assert c.check() == {"capacity", "range"}
    c = Case([32, 31, 0, 40, 10], [1, 1, 0, -1, -1], shared=32)  # rows before the prefix's end
    c.run()
    assert c.check() == {"range"}


def test_rings_that_are_none():
    for at in ([-1, 5], [9, 3], [0, 10 ** 6]):
        c = Case([5, 40], [1, -1])
        c.at = at
        c.run()
        assert c.check() == {"range"}
        assert c.t["ctx_out"].tolist() == [6, 40]  # (the first has room in its last block)


def test_more_returned_than_the_ring_holds():
    c = Case([5, 40], [30, -1])
    c.at = [0, len(c.free)]
    c.run()
    assert c.check() == {"capacity"}


def test_block_ids_outside_the_pool():
    c = Case([5, 40, 17], [30, 10, -1])
    c.table[0][0] = len(c.free)
    c.free[1] = -1
    c.run()
    assert c.check() == {"range"}


def test_steps_in_a_graph_on_another_stream():
    """Two captured steps hand their lengths and ring to each other; replays go on with them."""
    a = Case([17, 5, 90, 33], [1, 1, 1, 1], width=12, spare=40, head=77, pad=3)
    a.run()
    t = a.t
    for name in ("table", "free", "ctx", "at", "status"):
        t[name].copy_(torch.tensor(dict(table=a.table, free=a.free, ctx=a.ctx, at=a.at, status=[0])[name]))
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        a.call()
        t["ctx"].copy_(t["ctx_out"])
        t["at"].copy_(t["at_out"])
    state = (a.ctx, a.table, a.free, a.at)
    for step in range(20):
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        ctx, table, free, at = state
        table, free, at, ctx, q_start, positions, slots, errors = sc.tables(ctx, [1, 1, 1, 1], table, 16, 0, free, at, a.rows)
        state = (ctx, table, free, at)
        assert t["slots"].tolist() == slots and t["positions"].tolist() == positions and t["q_start"].tolist() == q_start
        assert t["table"].tolist() == table and t["at"].tolist() == at and t["ctx"].tolist() == ctx and not errors
    assert int(t["status"]) == 0
