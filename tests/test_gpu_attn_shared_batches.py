"""kvi_attn_shared on batches whose row starts are no good as a whole, or in part: what is
written and what is not is the same whether the prefix is read by itself or with each
request's other keys."""
import pytest
import torch

import pre_rope_kv_gb300 as kvi
from tests import attn_check as ac
from tests.test_gpu_attn_shared import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (layout, keys in the prefix, own keys, rows of the requests): the plain kernels for few rows and for many, with one
# piece of keys and several; a prefix of its own whose pieces the requests' blocks join, a third kernel for few rows, for many
FORMS = {
    "rows": ((4, 2, 128, 16), 96, 40, [1, 2, 1, 3]),
    "rows in a cluster": ((4, 2, 128, 16), 608, 40, [1, 1, 1, 2]),
    "rows in pieces": ((4, 2, 128, 16), 3200, 40, [1, 1, 1, 2]),
    "rows in many pieces": ((2, 1, 256, 16), 9600, 40, [1, 1, 1, 2]),
    "tiles": ((4, 2, 128, 16), 96, 40, [40, 9, 30, 70]),
    "tiles in pieces": ((4, 2, 128, 16), 3200, 40, [40, 9, 30, 70]),
    "prefix, joined by blocks": ((4, 2, 128, 16), 32000, 200, [1, 2, 1, 3]),
    "prefix, joined by a kernel": ((4, 2, 128, 16), 32000, 900, [1, 2, 1, 3]),
    "prefix, questions": ((4, 2, 128, 16), 32000, 900, [40, 9, 30, 70]),
}


def batch(form):
    (Hq, H, D, B), shared, own, n_q = FORMS[form]
    return Case(Hq, H, D, B, n_q, [n + own + 5 * i for i, n in enumerate(n_q)], shared, seed=Hq * D + shared)


@pytest.mark.parametrize("form", FORMS)
def test_a_batch_that_ends_past_q_is_left_out(form):
    """Its end is past q's, and no more rows than its requests can have; the others' rows are good."""
    good = batch(form)
    good.run()
    good.check()
    for lost in (1, 2):
        c = batch(form)
        total = c.q.shape[0]
        assert total + lost <= len(c.n_q) * c.max_q
        c.q_start[-1] = total + lost
        c.run()
        assert int(c.status) == kvi.ERR_OUT_OF_RANGE
        assert bool((c.out == 7).all()) and bool((c.lse == 7).all())


@pytest.mark.parametrize("form", FORMS)
def test_starts(form):
    """A batch's first and last start decide on all of it; of those between, on the requests beside them."""
    good = batch(form)
    good.run()
    n, total = good.n_q, good.q.shape[0]
    s = [sum(n[:i]) for i in range(5)]
    far = 4 * good.max_q + 1
    #        starts                                 requests whose rows are written
    cases = [([-1] + s[1:], []),
             ([total + 1] + s[1:], []),
             (s[:4] + [-3], []),
             (s[:4] + [far], []),                           # past q, and more than the requests can have
             ([s[4], s[3], s[2], s[1], s[0]], []),
             ([s[0], s[1], total + 9, s[3], s[4]], [0, 3]),
             ([s[0], -5, s[2], s[3], s[4]], [2, 3]),
             ([s[0], s[1], s[1], s[3], s[4]], [0, 3]),      # (of other requests, other rows)
             ([s[1], s[1], s[2], s[3], s[4]], [1, 2, 3])]
    for starts, written in cases:
        c = batch(form)
        c.q_start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        c.run()
        touched = torch.zeros(total, dtype=torch.bool, device=DEV)
        for r in written:
            at = slice(s[r], s[r + 1])
            touched[at] = True
            assert torch.equal(c.out[at], good.out[at]) and torch.equal(c.lse[at], good.lse[at]), (starts, r)
        others = [r for r in range(4) if r not in written and 0 <= starts[r] < starts[r + 1] <= total]
        if written and others:  # (rows that a request now has instead of another)
            for r in others:
                touched[starts[r]:starts[r + 1]] = True
        assert bool((c.out[~touched] == 7).all()) and bool((c.lse[~touched] == 7).all()), starts
        usable = all(0 <= a <= b <= total and b - a <= c.max_q for a, b in zip(starts, starts[1:]))
        assert int(c.status) == (0 if usable else kvi.ERR_OUT_OF_RANGE), starts
