"""Padding items of kda_pages_fork: -1 as parent or child, whatever the other is, leaves the item out altogether."""
import random

import pytest
import torch

from tests.latent_testutil import PoolModel
from tests.test_pages_gpu import Both, _i32

pytestmark = pytest.mark.gpu


class Padded(PoolModel):
    """A padding item names no row."""

    def fork(self, parents, children):
        super().fork(parents, [-1 if p == -1 else c for p, c in zip(parents, children)])


def pool(*args, **kw):
    b = Both(*args, **kw)
    b.m = Padded(len(b.m.lens), b.m.table.shape[1], len(b.m.ref), b.m.ps)
    return b


def test_a_child_named_by_padding_items_is_still_served():
    b = pool(4, 4, 12, 16)
    b.call("reserve", [0, 2], [20, 33])
    b.call("fork", [-1, 0], [1, 1])
    assert b.m.bits == 0 and int(b.pt.lens[1]) == 20
    b.call("fork", [-1, -1, 2, -1], [3, 3, 3, 3])
    assert b.m.bits == 0 and int(b.pt.lens[3]) == 33
    b.call("truncate", [1], [0])
    b.call("fork", [-1, 0, 2], [1, 1, 1])          # of two that are none, the first
    assert b.m.bits == 1 and int(b.pt.lens[1]) == 20
    b.call("truncate", [1], [0])
    b.call("fork", [9, 0], [1, 1])                  # a bad parent is no padding: the row is named
    assert b.m.bits == 1 and int(b.pt.lens[1]) == 0


@pytest.mark.parametrize("seed", range(4))
def test_histories_of_mostly_padding_forks(seed):
    r = random.Random(100 + seed)
    ps = r.choice([16, 64])
    b = pool(10, 6, 50, ps, seed=seed)
    for _ in range(40):
        b.call("reserve", [r.randrange(10)], [r.randint(1, 5 * ps)])
        n = r.randint(2, 12)
        b.call("fork", [r.choice([-1, -1, r.randint(0, 9)]) for _ in range(n)], [r.randint(-1, 9) for _ in range(n)])
        b.call("truncate", [r.randrange(10)], [0])
    b.call("compact")


def test_stale_children_in_a_replayed_graph():
    """A call of fixed size: the items that are not used keep the children of the step before."""
    b = pool(6, 4, 20, 16)
    b.call("reserve", [0], [40])
    parents, children, st = _i32([-1, -1, -1]), _i32([3, 4, 5]), _i32([0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.kda.kda_pages_fork(b.pt, b.cache, parents, children, b.ws, st)
    for pa, ch in (([-1, -1, -1], [3, 4, 5]), ([-1, 0, -1], [4, 4, 5]), ([-1, -1, 0], [5, 5, 5]), ([0, -1, -1], [3, 5, 4])):
        parents.copy_(_i32(pa))
        children.copy_(_i32(ch))
        g.replay()
        b.m.fork(pa, ch)
        for s, d in b.m.copies:
            b.want[:, d] = b.want[:, s].clone()
        torch.cuda.synchronize()
        b.same(int(st.item()), (pa, ch))
        assert b.m.bits == 0
