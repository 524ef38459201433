"""The page pool's operations against a plain model on the host: tables, lengths, counts and page contents, exactly."""
import random

import numpy as np
import pytest
import torch

from tests.latent_testutil import PoolModel

pytestmark = pytest.mark.gpu


def _kda():
    import hybrid_linear_attention_decode_gb300 as kda
    kda.load_library()
    return kda


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    def __init__(self, max_seqs, max_pages, num_pages, ps, layers=2, rank=128, rope=16, seed=0, page_major=False, items=64):
        self.kda = _kda()
        self.m = PoolModel(max_seqs, max_pages, num_pages, ps)
        self.pt = self.kda.PageTable.empty(max_seqs, max_pages, num_pages, ps)
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (num_pages, layers, ps, rank + rope) if page_major else (layers, num_pages, ps, rank + rope)
        pages = torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
        self.pages = pages.transpose(0, 1) if page_major else pages
        self.want = self.pages.clone()
        self.cache = self.kda.LatentCache(self.pages, rank)
        self.ws = torch.empty(self.kda.kda_pages_workspace_bytes(self.pt, items), dtype=torch.uint8, device="cuda")
        self.ws.fill_(0xa5)

    def call(self, op, *arrays, stream=None):
        st = _i32([0])
        if op == "truncate":
            self.kda.kda_pages_truncate(self.pt, *[_i32(x) for x in arrays], self.ws, st)
        elif op == "compact":
            self.kda.kda_pages_compact(self.pt, self.cache, self.ws, st)
        else:
            getattr(self.kda, "kda_pages_" + op)(self.pt, self.cache, *[_i32(x) for x in arrays], self.ws, st)
        getattr(self.m, op)(*arrays)
        for s, d in self.m.copies:
            self.want[:, d] = self.want[:, s].clone()
        torch.cuda.synchronize()
        self.same(int(st.item()), op)

    def same(self, bits, what):
        assert bits == self.m.bits, (what, bits, self.m.bits)
        assert np.array_equal(self.pt.lens.cpu().numpy(), self.m.lens), what
        assert np.array_equal(self.pt.refcount.cpu().numpy(), self.m.ref), what
        assert np.array_equal(self.pt.table.cpu().numpy(), self.m.table), what
        assert torch.equal(self.pages, self.want), what


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("page_major", [False, True])
def test_random_histories(seed, page_major):
    r = random.Random(seed)
    ps = r.choice([16, 32, 64])
    b = Both(24, 9, 110, ps, seed=seed, page_major=page_major)
    for _ in range(60):
        op = r.choice(["reserve", "reserve", "reserve", "truncate", "fork", "compact"])
        k = r.randint(1, 12)
        rows = [r.choice([-1] + list(range(24))) if r.random() < 0.9 else r.choice([-2, 24, 99]) for _ in range(k)]
        if op == "reserve":
            b.call(op, rows, [int(b.m.lens[x]) + r.randint(-3, 3 * ps) if 0 <= x < 24 else 5 for x in rows])
        elif op == "truncate":
            b.call(op, rows, [r.randint(-1, max(1, int(b.m.lens[x]) + 1)) if 0 <= x < 24 else 0 for x in rows])
        elif op == "fork":
            b.call(op, [r.randint(-1, 24) for _ in rows], rows)
        else:
            b.call(op)


def test_growth_takes_the_lowest_pages_in_order_and_stops_at_the_last():
    b = Both(4, 50, 10, 16)
    b.call("reserve", [2, 0], [40, 17])            # 3 and 2 pages
    assert b.m.table[2, :3].tolist() == [0, 1, 2] and b.m.table[0, :2].tolist() == [3, 4]
    b.call("reserve", [1, 3], [16 * 6, 16])        # 6 of the 5 left: refused, and so is what comes behind it
    assert b.m.bits == 32 and b.m.lens[1] == 0
    b.call("reserve", [3, 1], [16 * 5, 0])         # exactly the rest; growth by nothing
    assert b.m.bits == 0 and int((b.pt.refcount > 0).sum()) == 10
    b.call("truncate", [2], [0])
    b.call("reserve", [1], [48])


def test_shared_last_page_is_copied_before_it_grows():
    b = Both(6, 8, 30, 32)
    b.call("reserve", [0], [100])
    b.call("fork", [0, 0], [1, 2])
    b.call("truncate", [1, 2], [70, 64])           # row 1 now ends inside a page that rows 0 and 2... share
    b.call("reserve", [1, 2], [71, 65])
    b.call("truncate", [0, 1, 2], [40, 40, 40])    # all three inside the same shared page
    b.call("reserve", [0, 1, 2], [41, 42, 43])     # each takes a copy; the shared page ends up free
    b.call("compact")


def test_sizes_beyond_one_plan_sweep():
    """Several pages and more than one item for each thread of the plan CTA (1024)."""
    b = Both(1500, 12, 9000, 16, layers=1, rank=128, rope=0, items=1500)
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 100, 1500).tolist()
    b.call("reserve", list(range(1500)), lens)
    b.call("truncate", list(range(0, 1500, 2)), [0] * 750)
    b.call("fork", list(range(1, 1500, 2))[:700], list(range(0, 1500, 2))[:700])
    b.call("truncate", list(range(1, 1500, 3)), [0] * 500)
    b.call("compact")


def test_copy_pages_exact_and_contained():
    b = Both(2, 2, 20, 64, layers=3, rope=64, rank=512)
    st = _i32([0])
    b.kda.kda_pages_copy(b.cache, _i32([3, -1, 3, 7, 2]), _i32([4, 5, 9, -1, 19]), st)
    for s, d in ((3, 4), (3, 9), (2, 19)):
        b.want[:, d] = b.want[:, s].clone()
    b.same(int(st.item()), "copy")
    b.kda.kda_pages_copy(b.cache, _i32([20, 1, -2]), _i32([0, 21, 6]), st)
    torch.cuda.synchronize()
    assert int(st.item()) == b.kda.KDA_DEV_BAD_PAGE and torch.equal(b.pages, b.want)


def test_bad_table_entries_are_flagged_and_skipped():
    b = Both(4, 4, 12, 16)
    b.call("reserve", [0, 1], [40, 20])
    b.pt.table[0, 2] = 12
    st = _i32([0])
    b.kda.kda_pages_fork(b.pt, b.cache, _i32([0]), _i32([2]), b.ws, st)      # its partial page is the bad one
    torch.cuda.synchronize()
    assert int(st.item()) == b.kda.KDA_DEV_BAD_PAGE and int(b.pt.lens[2]) == 0
    st.zero_()
    b.kda.kda_pages_truncate(b.pt, _i32([0]), _i32([0]), b.ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == b.kda.KDA_DEV_BAD_PAGE
    assert int(b.pt.refcount.sum()) == 3                                      # row 1's two and the page that row 0 lost sight of
    b.pt.lens[3] = 65
    st.zero_()
    b.kda.kda_pages_compact(b.pt, b.cache, b.ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == b.kda.KDA_DEV_BAD_SEQLENS


def test_captured_reserve_append_cycle():
    """Growth by one token inside a replayed graph: lengths go up on the device."""
    kda = _kda()
    b = Both(3, 6, 16, 16)
    st, rows, goal = _i32([0]), _i32([0, 2]), _i32([1, 1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_pages_reserve(b.pt, b.cache, rows, goal, b.ws, st)
    for n in range(1, 40):
        goal.fill_(n)
        g.replay()
        b.m.reserve([0, 2], [n, n])
        torch.cuda.synchronize()
        b.same(int(st.item()), n)
