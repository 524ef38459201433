"""What queries get that see rows, keys or values that are not finite, as include/kda.h states it."""
import math

import pytest
import torch

from tests.latent_testutil import F64, attend, check
from tests.test_latent_gpu import Problem, Prompt

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


def place(p, b, j):
    """The cache row of token j of sequence b."""
    return p.pages[0, int(p.pt.table[b, j // p.page]), j % p.page]


def without(p, b, j, t):
    """The 64-bit answer for query t of sequence b as if the cache had no token j."""
    kv = torch.cat([p.rows64(b)[:j], p.rows64(b)[j + 1:]])
    seen = torch.ones(p.H, len(kv), dtype=torch.bool, device="cuda")
    if p.nq[b] - 1 - t:
        seen[:, -(p.nq[b] - 1 - t):] = False
    q = p.q[sum(p.nq[:b]) + t].to(F64)
    return attend(q, kv, kv[:, :p.rank], seen, p.scale, p.dtype)


# the row: the newest of one token, or an earlier one in the first, a middle and the last tile
ROWS = [(0, 199), (0, 0), (0, 100), (0, 195), (1, 64), (1, 10)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("b,j", ROWS)
def test_decode_row_of_one_token_or_before_the_drafts(b, j, dtype):
    p = Problem([200, 65], [1, 1], H=12, rank=256, rope=64, page=32, dtype=dtype, seed=60)
    p.q[:, :, 300] = torch.where(torch.arange(12, device="cuda") % 2 == 0, 1.0, -1.0).to(dtype)
    p.q[:, :, 7] = p.q[:, :, 300]
    p.run()
    clean, clean_l = p.out.clone(), p.lse.clone()
    row = place(p, b, j)
    old = row.clone()
    for at in (300, 7):                       # a rotary channel and a latent one
        row[at] = NAN
        p.run()
        assert bool(torch.isnan(p.out[b]).all()) and bool(torch.isnan(p.lse[b]).all())
        assert torch.equal(p.out[1 - b], clean[1 - b]) and torch.equal(p.lse[1 - b], clean_l[1 - b])
        row[at] = INF                         # scores +inf for the even heads, -inf for the odd ones
        p.run()
        assert bool(torch.isnan(p.out[b, ::2]).all()) and bool(torch.isnan(p.lse[b, ::2]).all())
        row.copy_(old)
        o, l, to, tl = without(p, b, j, 0)
        keep = [c for c in range(256) if c != at]
        check(p.out[b, 1::2][:, keep], o[1::2][:, keep], to[1::2][:, keep], "weight 0")
        check(p.lse[b, 1::2], l[1::2], tl[1::2], "weight 0")
        assert torch.equal(p.out[1 - b], clean[1 - b])


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_decode_row_among_several_drafts_makes_all_nan(value, tree):
    p = Problem([200, 30], [3, 1], H=12, rank=128, seed=61)
    mask = torch.tensor([1, 3, 5, 1], dtype=torch.int64, device="cuda") if tree else None
    p.run(tree=mask)
    clean, clean_l = p.out.clone(), p.lse.clone()
    place(p, 0, 198)[5] = value               # drafted token 1: the tree's third query does not see it
    if tree:
        place(p, 1, 29)[140] = value          # with a tree, the one token of a sequence counts as drafted, too
    p.run(tree=mask)
    bad = [1, 3] if tree else [1, 2]
    good = [i for i in range(4) if i not in bad]
    assert bool(torch.isnan(p.out[bad]).all()) and bool(torch.isnan(p.lse[bad]).all())
    assert torch.equal(p.out[good], clean[good]) and torch.equal(p.lse[good], clean_l[good])


@pytest.mark.parametrize("H", [3, 96])
def test_prefill_keys_and_values_that_are_seen(H):
    p = Prompt([200], [400], H=H, seed=62)    # queries 0..199 see keys 0..200 + i
    p.q[:, :, 3] = 1
    p.run()
    clean, clean_l = p.out.clone(), p.lse.clone()
    late = range(150, 200)                    # the queries that see key 350
    for j, see in ((20, range(200)), (350, late)):
        rest = [i for i in range(200) if i not in see]
        see = list(see)
        old = p.k[j, 1].clone()
        p.k[j, 1, 3] = NAN
        p.run()
        assert bool(torch.isnan(p.out[see, 1]).all()) and bool(torch.isnan(p.lse[see, 1]).all())
        p.k[j, 1, 3] = INF
        p.run()
        assert bool(torch.isnan(p.out[see, 1]).all())
        p.k[j, 1, 3] = -INF                   # weight 0: as if the key were not there
        p.run()
        p.k[j, 1] = old
        key = torch.cat([p.k[:, 1], p.r], 1).to(F64)
        seen = torch.arange(400, device="cuda")[None] <= torch.arange(200, device="cuda")[:, None] + 200
        seen[:, j] = False
        o, l, to, tl = attend(p.q[:, 1].to(F64), key, p.v[:, 1].to(F64), seen, p.scale, p.dtype)
        check(p.out[:, 1], o, to)
        check(p.lse[:, 1], l, tl)
        old = p.v[j, 2].clone()
        for value in (NAN, INF, -INF):
            p.v[j, 2, 9] = value
            p.run()
            assert bool((~torch.isfinite(p.out[see, 2, 9])).all())
            assert torch.equal(p.out[rest, 2], clean[rest, 2]) and torch.equal(p.lse[rest, 2], clean_l[rest, 2])
        p.v[j, 2] = old
    p.run()
    assert torch.equal(p.out, clean) and torch.equal(p.lse, clean_l)
