"""kda_kv_decode and kda_kv_evict against 64-bit softmax and the rules of eviction, and a run of the whole set."""
import math

import numpy as np
import pytest
import torch

import hybrid_linear_attention_decode_gb300 as kda
from tests.kv_testutil import DEV, F64, Pages, attention, check, cu_of, evicted, i32, rotated, status

pytestmark = pytest.mark.gpu


def queries(T, H, d, dtype, seed=5, strided=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H + 3 if strided else H, d, generator=g, device=DEV).to(dtype)
    return x[:, 2:H + 2] if strided else x


def decode(p, q, nq, layer=0, rows=None, tree=None, decay=None, scale=None, max_slots=None, cu="from", max_tokens=None,
           out=None, lse=None, stream=None, ws=None, st=None):
    T, H, d = q.shape
    n = len(nq)
    mt = max_tokens or max([1] + list(nq))
    out = torch.full((T, H, d), 5.0, dtype=q.dtype, device=DEV) if out is None else out
    lse = torch.full((T, H), 5.0, device=DEV) if lse is None else lse
    slots = 0 if decay is None else p.cache.data.shape[1] * p.page if max_slots is None else max_slots
    if ws is None:  # with bytes that are not finite numbers, as a workspace need not be initialised
        ws = torch.full((max(16, kda.kda_kv_decode_workspace_bytes(p.cache, H, n, mt, slots)),), 255, dtype=torch.uint8,
                        device=DEV)
    st = status() if st is None else st
    kda.kda_kv_decode(p.cache, layer, p.pt, rows, cu_of(nq) if cu == "from" else cu, mt, q, out, lse,
                      1 / math.sqrt(d) if scale is None else scale, ws, st, tree_mask=tree, weight_decay=decay,
                      max_slots=slots or None, stream=stream)
    return out, lse, st


def compare(p, q, nq, out, lse, layer=0, rows=None, tree=None, scale=None, sums=None, decay=1.0):
    """All sequences against 64 bits; sums: the cache's weights before the call."""
    d, at = q.shape[2], 0
    for b, k in enumerate(nq):
        row = b if rows is None else rows[b]
        t = None if tree is None else tree[at:at + k].tolist()
        n = 0 if row < 0 else p.lens[row]
        o, l, add = attention(p, layer, max(row, 0), q[at:at + k], 1 / math.sqrt(d) if scale is None else scale, t, n)
        check(out[at:at + k], *o, ("out", b))
        check(lse[at:at + k], *l, ("lse", b))
        if sums is not None and n and k:
            pid, slot = p.places(row)
            was = sums[layer, pid, :, slot].to(F64).t()
            got = p.cache.weights[layer, pid, :, slot].to(F64).t()
            ref = decay * was + add[0]
            check(got, ref, add[1] + 2 * 2.0 ** -24 * (ref.abs() + was.abs()) + 2.0 ** -126, ("sums", b))
        at += k


LENS = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,G,d,page", [
    (8, 4, 128, 64), (1, 1, 16, 16), (2, 7, 24, 16), (2, 16, 64, 32), (3, 5, 80, 64), (1, 8, 96, 16), (4, 1, 120, 128),
    (1, 32, 128, 16), (2, 8, 192, 192), (1, 12, 256, 32), (2, 2, 248, 64), (1, 256, 64, 64), (128, 2, 32, 16), (1, 17, 40, 1024)])
def test_one_token(dtype, kv, G, d, page):
    p = Pages(LENS, kv, d, page, dtype=dtype, layers=2, transposed=True, seed=kv + d)
    p.poison()
    nq = [1] * len(LENS)
    q = queries(len(LENS), kv * G, d, dtype, strided=True)
    out, lse, st = decode(p, q, nq, layer=1)
    compare(p, q, nq, out, lse, layer=1)
    assert int(st) == 0
    again, lse2, _ = decode(p, q, nq, layer=1, cu=None)  # the same without cu_tokens, bit for bit
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d,page", [(136, 16), (160, 64), (184, 32), (192, 16), (192, 64), (200, 128)])
@pytest.mark.parametrize("kv,G,tokens", [(8, 1, 1), (2, 4, 3), (1, 8, 4), (3, 12, 5)])
def test_wide_heads(d, page, kv, G, tokens):
    """Heads between 128 and 256 channels, each number of rows of a unit, sums of weights."""
    lens = [tokens, 31, 32, 33, 700, 0, 95, 5000]
    nq = [tokens] * len(lens)
    p = Pages(lens, kv, d, page, stats=True, seed=d)
    p.poison()
    sums = p.cache.weights.clone()
    q = queries(sum(nq), kv * G, d, torch.bfloat16, strided=True)
    out, lse, st = decode(p, q, nq, decay=0.5)
    compare(p, q, nq, out, lse, sums=sums, decay=0.5)
    assert int(st) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,G,d,page,tokens", [(8, 4, 128, 16, 5), (2, 8, 64, 64, 3), (1, 16, 128, 32, 8), (1, 5, 96, 64, 64),
                                                (2, 1, 256, 16, 7), (1, 33, 72, 64, 4), (4, 2, 128, 64, 20)])
def test_drafted_chains_and_trees(dtype, kv, G, d, page, tokens):
    rng = np.random.default_rng(tokens + d)
    lens = [tokens, tokens + 1, 63, 64, 65, 66, 129, 0, 400, 2]
    nq = [int(rng.integers(0, tokens + 1)) for _ in lens]
    nq[0], nq[4], nq[6] = tokens, min(tokens, 3), tokens
    p = Pages(lens, kv, d, page, dtype=dtype, seed=d)
    q = queries(sum(nq), kv * G, d, dtype)
    out, lse, st = decode(p, q, nq)
    compare(p, q, nq, out, lse)
    masks = []
    for k in nq:
        for j in range(k):
            m = int(rng.integers(0, 1 << 62)) & ((1 << (j + 1)) - 1)
            masks.append(m if rng.random() < 0.8 else 0)
    tree = torch.tensor(masks, dtype=torch.int64, device=DEV)
    out, lse, st2 = decode(p, q, nq, tree=tree)
    compare(p, q, nq, out, lse, tree=tree)
    assert int(st) == 0 and int(st2) == 0


@pytest.mark.parametrize("kv,G,d,page,tokens", [(2, 32, 128, 64, 5), (1, 128, 64, 16, 3), (1, 9, 200, 32, 10), (4, 16, 96, 128, 1)])
def test_more_rows_than_a_unit(kv, G, d, page, tokens):
    """More than 64 rows of a sequence on a key-value head, and calls that mix few and many of them."""
    lens = [700, 64, 33, 2000, 5]
    nq = [tokens, 1, tokens, 1, min(tokens, 5)]
    p = Pages(lens, kv, d, page, seed=G)
    p.poison()
    q = queries(sum(nq), kv * G, d, torch.bfloat16)
    out, lse, st = decode(p, q, nq)
    compare(p, q, nq, out, lse)
    assert int(st) == 0


@pytest.mark.parametrize("kv,G,d,page,lens", [
    (2, 4, 128, 64, [50000]), (1, 1, 64, 16, [100001]), (4, 8, 128, 128, [9000, 1, 20000, 333]), (1, 16, 256, 64, [30000, 5]),
    (8, 4, 128, 32, [int(x) for x in np.random.default_rng(1).integers(1, 900, 90)]),
    (2, 2, 64, 16, [int(x) for x in np.random.default_rng(2).integers(0, 40, 700)])])
def test_long_and_many(kv, G, d, page, lens):
    p = Pages(lens, kv, d, page, seed=len(lens))
    p.poison(float("inf"))
    nq = [1] * len(lens)
    q = queries(len(lens), kv * G, d, torch.bfloat16)
    out, lse, st = decode(p, q, nq)
    assert int(st) == 0
    few = range(len(lens)) if len(lens) < 9 else list(range(0, len(lens), 13)) + [len(lens) - 1]
    for b in few:
        o, l, _ = attention(p, 0, b, q[b:b + 1], 1 / math.sqrt(d))
        check(out[b:b + 1], *o, b)
        check(lse[b:b + 1], *l, b)
    assert bool(torch.isfinite(out).all())


def test_thousands_of_entries_with_repeats_and_padding():
    """65535 entries, most of them padding; table rows repeat; the others' outputs are those of a small call."""
    p = Pages([100, 0, 333, 17], 2, 64, 16)
    n = 65535
    rows = torch.full((n,), -1, dtype=torch.int32)
    at = torch.randperm(n, generator=torch.Generator().manual_seed(1))[:1500]
    rows[at] = torch.randint(0, 4, (1500,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    q = queries(n, 4, 64, torch.bfloat16)
    out, lse, st = decode(p, q, [1] * n, rows=rows.cuda(), cu=None)
    assert int(st) == 0
    pad = rows.cuda() < 0
    assert bool((out[pad] == 0).all()) and bool((lse[pad] == -math.inf).all())
    for b in at[:12].tolist():
        row = int(rows[b])
        o, l, _ = attention(p, 0, row, q[b:b + 1], 1 / 8)
        check(out[b:b + 1], *o)
        check(lse[b:b + 1], *l)


def test_padding_bad_entries_and_rows_behind():
    lens = [100, 70, 5, 200]
    p = Pages(lens, 2, 64, 16, max_seqs=5)
    p.pt.lens[4] = 10 ** 6
    rows = [3, -1, 1, 77, 4, 3, 2]
    nq = [2, 2, 1, 1, 1, 1, 0]
    q = queries(10, 8, 64, torch.bfloat16)
    out, lse, st = decode(p, q, nq, rows=i32(rows))
    assert int(st) == kda.KDA_DEV_BAD_SLOT | kda.KDA_DEV_BAD_SEQLENS
    zero = [x if x in (0, 1, 2, 3) else -1 for x in rows]  # bad rows are like empty ones
    compare(p, q, nq, out, lse, rows=zero)
    assert bool((out[8:] == 5).all()) and bool((lse[8:] == 5).all())
    # bad cu_tokens: those sequences' rows stay as they were
    out, lse, st = decode(p, q[:4], [1, 1], cu=i32([0, 1, 50]), max_tokens=2)
    assert int(st) == kda.KDA_DEV_BAD_SEQLENS and bool((out[1:] == 5).all()) and not bool((out[0] == 5).any())


def test_bad_pages_read_as_zeros():
    p = Pages([100, 70], 2, 64, 16)
    good = p.pt.table.clone()
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1, p.cache.data.shape[1]):
        p.pt.table.copy_(good)
        p.pt.table[0, 2] = bad
        q = queries(2, 4, 64, torch.bfloat16)
        out, lse, st = decode(p, q, [1, 1])
        assert int(st) == kda.KDA_DEV_BAD_PAGE
        p.pt.table.copy_(good)
        k, v = p.cache.keys.clone(), p.cache.values.clone()
        p.cache.keys[0, good[0, 2].long()] = 0
        p.cache.values[0, good[0, 2].long()] = 0
        compare(p, q, [1, 1], out, lse)
        p.cache.keys.copy_(k)
        p.cache.values.copy_(v)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_non_finite_rows(dtype):
    """What a query does not see does not matter to it; a seen NaN key spoils the query, a seen NaN value its channel or,
    among several drafted tokens, the query."""
    p = Pages([90, 90, 90, 90], 1, 64, 16, dtype=dtype)
    for x, row, j in ((p.cache.keys, 0, 88), (p.cache.values, 1, 88), (p.cache.values, 2, 40), (p.cache.keys, 3, 89)):
        pid, slot = p.places(row)
        x[0, pid[j], 0, slot[j], 3] = float("nan")
    q = queries(12, 4, 64, dtype)
    tree = torch.tensor([1, 2, 4] * 4, dtype=torch.int64, device=DEV)  # query t sees the old ones and drafted token t
    out, lse, st = decode(p, q, [3] * 4, tree=tree)
    assert int(st) == 0
    bad, badl = torch.isnan(out), torch.isnan(lse)
    for row, t in ((0, 1), (1, 1), (3, 2)):
        assert bool(bad[3 * row + t].all()) and bool(badl[3 * row + t].all())
        for other in range(3):
            if other != t:
                assert not bool(bad[3 * row + other].any()) and not bool(badl[3 * row + other].any())
    assert bool(bad[6:9, :, 3].all()) and int(bad[6:9].sum()) == 12 and not bool(badl[6:9].any())
    out, lse, _ = decode(p, q[:4], [1] * 4)
    assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(lse[3]).all())
    assert int(torch.isnan(out[1]).sum()) == 4 and not bool(torch.isnan(lse[1]).any())


def test_infinite_scores():
    p = Pages([50, 50], 1, 64, 16, dtype=torch.float16)
    pid, slot = p.places(0)
    p.cache.keys[0, pid[7], 0, slot[7]] = float("-inf")
    q = torch.ones(2, 1, 64, dtype=torch.float16, device=DEV)
    out, lse, _ = decode(p, q, [1, 1])
    assert bool(torch.isfinite(out).all())  # a score of -infinity has weight 0
    k = p.cache.keys.clone()
    p.cache.keys[0, pid[7], 0, slot[7]] = float("inf")
    out, lse, _ = decode(p, q, [1, 1])
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all()) and bool(torch.isfinite(out[1]).all())
    p.cache.keys.copy_(k)
    p.cache.keys[0, pid, 0, slot] = float("-inf")
    out, lse, _ = decode(p, q, [1, 1])
    assert float(lse[0, 0]) == -math.inf and bool((out[0] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1e-30, 1e-4, 8.0, 300.0])
def test_scales(dtype, scale):
    p = Pages([700, 64, 130], 2, 64, 16, dtype=dtype)
    q = queries(3, 8, 64, dtype)
    out, lse, _ = decode(p, q, [1] * 3, scale=scale)
    compare(p, q, [1] * 3, out, lse, scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens", [1, 7, 16])
def test_scores_past_fp32_by_the_scale(dtype, tokens):
    """Products that fp32 holds, scores that it does not: +infinity makes a query NaN, -infinity weighs nothing."""
    d, n = 64, 100
    p = Pages([n, n, n, n], 1, d, 16, dtype=dtype)
    for b, signs in enumerate(("-", "-0", "-+", "0")):  # of the keys, in turn; a key is 0 or +-(6e4, 0, ...)
        pid, slot = p.places(b)
        for j in range(n):
            c = signs[j % len(signs)] if j < n - tokens else signs[-1]
            p.cache.keys[0, pid[j], 0, slot[j]] = 0
            p.cache.keys[0, pid[j], 0, slot[j], 0] = {"-": -6e4, "0": 0.0, "+": 6e4}[c]
    q = torch.zeros(4 * tokens, 4, d, dtype=dtype, device=DEV)
    q[:, :, 0] = 6e4
    out, lse, st = decode(p, q, [tokens] * 4, scale=1e30)  # 3.6e9 * 1e30
    assert int(st) == 0
    out, lse = out.view(4, tokens, 4, d), lse.view(4, tokens, 4)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    assert bool(out[2].isnan().all()) and bool(lse[2].isnan().all())
    for b in (1, 3):  # weights of the zero scores are equal
        pid, slot = p.places(b)
        zero = p.cache.keys[0, pid, 0, slot, 0] == 0
        for t in range(tokens):
            seen = zero.clone()
            seen[n - tokens + t + 1:] = False
            v = p.cache.values[0, pid, 0, slot].to(F64)[seen]
            k = int(seen.sum())
            # weights rounded to the type and exponentials of 2^-22, a sum of k terms, one rounding
            u = torch.finfo(dtype).eps / 2
            tol = u * v.mean(0).abs() + (u + 2.0 ** -20 + k * 2.0 ** -24) * v.abs().mean(0) + torch.finfo(dtype).smallest_normal
            for h in range(4):
                check(out[b, t, h], v.mean(0), tol)
                assert abs(float(lse[b, t, h]) - math.log(k)) <= 2.0 ** -20 + 4 * 2.0 ** -24 * math.log(k)


def test_long_tail_of_small_weights():
    """One large weight whose value is near zero, and 30000 of e^-20 of it that make up the output."""
    for dtype in (torch.float16, torch.bfloat16):
        p = Pages([30001], 1, 64, 64, dtype=dtype)
        p.cache.keys.zero_()
        p.cache.values.fill_(1000.0)
        pid, slot = p.places(0)
        p.cache.keys[0, pid[77], 0, slot[77], 0] = 16.0
        p.cache.values[0, pid[77], 0, slot[77]] = 2.0 ** -14
        q = torch.zeros(1, 2, 64, dtype=dtype, device=DEV)
        q[..., 0] = 1.25
        out, lse, _ = decode(p, q, [1], scale=1.0)
        compare(p, q, [1], out, lse, scale=1.0)


# ------------------------------------------------------------------------------------------------- sums of weights
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,G,d,page,tokens,decay", [(8, 4, 128, 64, 1, 1.0), (2, 7, 64, 16, 1, 0.9), (1, 16, 96, 32, 3, 0.0),
                                                      (3, 1, 24, 16, 2, 1.0), (1, 40, 128, 64, 4, 0.5), (2, 2, 256, 192, 5, 1.0)])
def test_sums(dtype, kv, G, d, page, tokens, decay):
    lens = [0, 1, 5, 64, 65, 130, 700, 16]
    nq = [min(tokens, 1 + i % tokens) for i in range(len(lens))]
    p = Pages(lens, kv, d, page, stats=True, dtype=dtype, layers=2, transposed=True, seed=d)
    before = p.cache.data.clone()
    sums = p.cache.weights.clone()
    q = queries(sum(nq), kv * G, d, dtype)
    out, lse, st = decode(p, q, nq, layer=1, decay=decay)
    assert int(st) == 0
    compare(p, q, nq, out, lse, layer=1, sums=sums, decay=decay)
    # nothing but the sums of tokens in the call's layer has changed
    after = p.cache.weights.clone()
    for b in range(len(lens)):
        pid, slot = p.places(b)
        after[1, pid, :, slot] = sums[1, pid, :, slot]
    assert torch.equal(after, sums)
    p.cache.weights.copy_(sums)
    assert torch.equal(p.cache.data.view(torch.int16), before.view(torch.int16))
    plain, lse2, _ = decode(p, q, nq, layer=1)
    compare(p, q, nq, plain, lse2, layer=1)


def test_sums_of_long_and_many():
    lens = [40000, 3, 900, 17]
    p = Pages(lens, 2, 128, 64, stats=True)
    sums, nq = p.cache.weights.clone(), [1] * 4
    q = queries(4, 8, 128, torch.bfloat16)
    out, lse, st = decode(p, q, nq, decay=1.0)
    compare(p, q, nq, out, lse, sums=sums)
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 300, 120)]
    p = Pages(lens, 1, 64, 16, stats=True)
    sums, nq = p.cache.weights.clone(), [1] * 120
    q = queries(120, 4, 64, torch.bfloat16)
    out, lse, st = decode(p, q, nq, decay=1.0)
    compare(p, q, nq, out, lse, sums=sums)
    assert int(st) == 0


def test_shared_pages_slots_past_the_bound_padding_and_nan():
    lens = [100, 70, 60, 40]
    p = Pages(lens, 2, 64, 16, stats=True)
    p.pt.refcount[p.pt.table[0, 1].long()] = 2
    pid, slot = p.places(3)
    p.cache.keys[0, pid[5], 1, slot[5], 0] = float("nan")  # head 1 of row 3
    sums, q, nq = p.cache.weights.clone(), queries(5, 4, 64, torch.bfloat16), [1, 1, 1, 1, 1]
    rows = [0, -1, 1, 3, 2]
    out, lse, st = decode(p, q, nq, rows=i32(rows), decay=1.0, max_slots=215)  # 100 + 70 + 40 fit, 60 more do not
    assert int(st) == kda.KDA_DEV_BAD_SEQLENS
    keep = p.cache.weights.clone()
    pid2, slot2 = p.places(2)
    assert torch.equal(keep[0, pid2, :, slot2], sums[0, pid2, :, slot2])
    shared = p.pt.table[0, 1].long()
    assert torch.equal(keep[0, shared], sums[0, shared])
    assert torch.equal(keep[0, pid, 1, slot], sums[0, pid, 1, slot])  # a NaN lse adds nothing
    assert not torch.equal(keep[0, pid, 0, slot], sums[0, pid, 0, slot])
    for b, row in ((0, 0), (2, 1), (4, 2)):
        o, l, add = attention(p, 0, row, q[b:b + 1], 1 / 8)
        check(out[b:b + 1], *o)
        if row < 2:
            pid3, slot3 = p.places(row)
            mine = pid3 != shared
            got, was = (x[0, pid3[mine], :, slot3[mine]].to(F64).t() for x in (keep, sums))
            check(got, was + add[0][:, mine], add[1][:, mine] + 2.0 ** -22 * (1 + was))


def test_sums_skip_bad_pages():
    p = Pages([100], 1, 64, 16, stats=True)
    sums = p.cache.weights.clone()
    p.pt.table[0, 3] = -5
    out, lse, st = decode(p, queries(1, 4, 64, torch.bfloat16), [1], decay=0.0)
    assert int(st) == kda.KDA_DEV_BAD_PAGE
    touched = (p.cache.weights != sums).flatten(2).any(-1)[0]
    assert set(torch.nonzero(touched)[:, 0].tolist()) == set(p.pt.table[0, [0, 1, 2, 4, 5, 6]].tolist())


# ------------------------------------------------------------------------------------------------- eviction
def evict_and_compare(p, keep, rows=None, first=0, since=None, expect=0, skip=(), max_len=0):
    """The call against the rules, every word of the cache; skip: entries that are left as they are."""
    cache, L, kv = p.cache, p.cache.data.shape[0], p.heads
    want = cache.data.clone()
    ref = p.pt.refcount.cpu().numpy()
    w, pos = cache.weights.cpu().numpy(), cache.positions.cpu().numpy()
    t = p.pt.table.cpu().numpy()
    view = kda.KvCache(want, kv, p.d, p.page, True)
    expect_lens = []
    for i in range(len(keep)):
        row = i if rows is None else rows[i]
        if i in skip or row < 0:
            expect_lens.append(None if i in skip else 0)
            continue
        n = p.lens[row]
        expect_lens.append(min(n, keep[i]))
        if n <= keep[i]:
            continue
        j = np.arange(n)
        pid, slot = t[row, j // p.page], j % p.page
        for l in range(L):
            for h in range(kv):
                moves = evicted(w[l, pid, h, slot], pos[l, pid, h, slot], ref[pid] > 1, keep[i], first,
                                None if since is None else since[i])
                if not moves:
                    continue
                a, b = (torch.tensor(x, device=DEV) for x in zip(*moves))
                pa, sa, pb, sb = (torch.from_numpy(pid).cuda().long()[a], a % p.page,
                                  torch.from_numpy(pid).cuda().long()[b], b % p.page)
                for x in (view.keys, view.values, view.weights.view(torch.int32), view.positions):
                    x[l, pb, h, sb] = x[l, pa, h, sa].clone()
    new, st = torch.full((len(keep),), -9, dtype=torch.int32, device=DEV), status()
    kda.kda_kv_evict(cache, p.pt, None if rows is None else i32(rows), i32(keep), new, st, first=first,
                     since=None if since is None else i32(since), max_len=max_len)
    assert int(st) == expect
    for got, n in zip(new.tolist(), expect_lens):
        assert n is None or got == n
    assert torch.equal(cache.data.view(torch.int16), want.view(torch.int16))
    return new.tolist()


def heavy(p, seed=0, ties=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.exp(3 * torch.randn(p.cache.weights.shape, generator=g, device=DEV))
    if ties:
        w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < ties, torch.full_like(w, 0.25), w)
    p.cache.weights.copy_(w)
    p.cache.positions.copy_(torch.randint(0, 100000, w.shape, generator=g, device=DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,d,page,layers", [(8, 128, 64, 3), (1, 16, 16, 1), (2, 24, 16, 2), (3, 80, 192, 1), (2, 256, 32, 2)])
@pytest.mark.parametrize("ties", [0.0, 0.7, 1.0])
def test_evict(dtype, kv, d, page, layers, ties):
    lens = [0, 1, 2, 16, 17, 31, 32, 33, 64, 100, 255, 256, 257, 500, 513]
    p = Pages(lens, kv, d, page, stats=True, dtype=dtype, layers=layers, transposed=layers > 1, seed=d)
    heavy(p, ties=ties)
    keep = [3, 0, 1, 16, 1, 30, 31, 32, 63, 37, 128, 255, 32, 511, 512]
    evict_and_compare(p, keep)


@pytest.mark.parametrize("lens,keep", [([5000], [1000]), ([70000], [4096]), ([70000], [69999]), ([20001, 3000], [1, 2999]),
                                       ([200000], [120000]), ([1048576], [8192])])
@pytest.mark.parametrize("ties", [0.0, 0.9])
def test_evict_long_rows(lens, keep, ties):
    """Few units of many slots: clusters of CTAs, and keys that no longer fit shared memory."""
    p = Pages(lens, 2 if lens[0] < 200000 else 1, 16, 64, stats=True)
    heavy(p, ties=ties)
    evict_and_compare(p, keep, first=100, since=[99000] * len(lens))


def test_evict_bound_of_lengths():
    """Rows up to the bound are shortened; longer ones are flagged unless they stay as they are anyway."""
    p = Pages([300, 200, 201, 199], 2, 32, 16, stats=True)
    heavy(p)
    new = evict_and_compare(p, [300, 50, 60, 70], max_len=200, expect=kda.KDA_DEV_BAD_SEQLENS, skip=(2,))
    assert new == [300, 50, 201, 70]


@pytest.mark.parametrize("room", [70, 300, 9000, 20000])
def test_evict_of_short_rows_in_wide_tables(room):
    p = Pages([100, 2000, 513, 64] * 40, 2, 16, 16, stats=True)
    p.pt.table = torch.nn.functional.pad(p.pt.table, (0, max(0, room - p.pt.table.shape[1])), value=-1).contiguous()
    heavy(p, ties=0.5)
    evict_and_compare(p, [50, 1500, 512, 3] * 40, first=7)


def test_evict_many_units():
    lens = [int(x) for x in np.random.default_rng(5).integers(1, 200, 150)]
    p = Pages(lens, 4, 32, 16, stats=True, layers=2)
    heavy(p)
    evict_and_compare(p, [max(1, n // 2) for n in lens])


def test_evict_protects():
    p = Pages([300, 300, 300], 2, 64, 16, stats=True)
    heavy(p)
    for b in range(3):  # positions 0..299 in some order
        pid, slot = p.places(b)
        perm = torch.randperm(300, generator=torch.Generator().manual_seed(b)).to(torch.int32).cuda()
        p.cache.positions[0, pid, :, slot] = perm[:, None].expand(-1, 2)
    p.pt.refcount[p.pt.table[1, [0, 5, 18]].long()] = 2  # shared pages: kept, never written
    before = p.cache.data[0, p.pt.table[1, [0, 5, 18]].long()].clone()
    evict_and_compare(p, [40, 100, 7], first=4, since=[280, 250, 290])  # row 2: more protected ones than places
    assert torch.equal(before.view(torch.int16), p.cache.data[0, p.pt.table[1, [0, 5, 18]].long()].view(torch.int16))
    # the beginning and the newest are still there in row 0
    pid, slot = p.places(0, 40)
    for h in range(2):
        left = set(p.cache.positions[0, pid, h, slot].tolist())
        assert left >= {0, 1, 2, 3} | set(range(280, 300)) and len(left) == 40


def test_evict_odd_sums():
    """NaN counts as least, -0 as 0, infinities as what they are, negative numbers below 0."""
    p = Pages([64], 1, 16, 16, stats=True)
    heavy(p)
    pid, slot = p.places(0)
    w = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1.0, -1e-40, 1e-40] * 8, device=DEV)
    p.cache.weights[0, pid, 0, slot] = w
    for keep in (60, 50, 42, 33, 30, 17, 9, 8, 3):
        p.cache.weights[0, pid, 0, slot] = w
        evict_and_compare(p, [keep])


def test_evict_thousands_of_padding_entries():
    p = Pages([100, 80], 2, 64, 16, stats=True)
    heavy(p)
    n = 5000
    rows = [-1] * n
    rows[1234], rows[4999] = 1, 0
    keep = [5] * n
    new = evict_and_compare(p, keep, rows=rows)
    assert [x for x in new if x] == [5, 5] and new[1234] == 5 and new[4999] == 5


def test_evict_refused_rows_stay():
    p = Pages([100, 80, 90, 60, 70], 2, 64, 16, stats=True, max_seqs=6)
    heavy(p)
    p.pt.lens[5] = 10 ** 7
    p.pt.table[2, 4] = -3
    new = evict_and_compare(p, [50, 10, 20, -1, 70, 9, 5, 8], rows=[0, -1, 2, 3, 4, 5, 99, 1],
                            expect=kda.KDA_DEV_BAD_SLOT | kda.KDA_DEV_BAD_SEQLENS | kda.KDA_DEV_BAD_PAGE, skip=(2, 3, 5, 6))
    assert new == [50, 0, 90, 60, 70, 0, 0, 8]


# ------------------------------------------------------------------------------------------------- the pool with these pages
def test_pool_operations_carry_whole_pages():
    p = Pages([20, 33, 16], 2, 24, 16, stats=True, layers=2, max_seqs=6, spare=9, transposed=True)
    heavy(p)
    p.pt.table = torch.cat([p.pt.table, torch.full((6, 4), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    ws = torch.empty(kda.kda_pages_workspace_bytes(p.pt, 4), dtype=torch.uint8, device=DEV)
    st = status()

    def tokens(row, n):
        j = torch.arange(n, device=DEV)
        pid, slot = p.pt.table[row].long()[j // 16], j % 16
        return [x[:, pid, :, slot].clone() for x in (p.cache.keys, p.cache.values, p.cache.weights, p.cache.positions)]
    was = tokens(1, 33)
    kda.kda_pages_fork(p.pt, p.cache, i32([1, 1]), i32([4, 5]), ws, st)
    assert p.pt.lens.tolist() == [20, 33, 16, 0, 33, 33]
    for row in (4, 5):
        assert all(torch.equal(a, b) for a, b in zip(tokens(row, 33), was))
    kda.kda_pages_reserve(p.pt, p.cache, i32([4, 0]), i32([35, 50]), ws, st)
    assert all(torch.equal(a, b) for a, b in zip(tokens(4, 33), was))
    kda.kda_pages_truncate(p.pt, i32([1, 5]), i32([0, 0]), ws, st)
    kept = tokens(4, 35), tokens(0, 20), tokens(2, 16)
    kda.kda_pages_compact(p.pt, p.cache, ws, st)
    assert int(p.pt.table.max()) == int((p.pt.refcount > 0).sum()) - 1
    for (row, n), was in zip(((4, 35), (0, 20), (2, 16)), kept):
        assert all(torch.equal(a, b) for a, b in zip(tokens(row, n), was))
    kda.kda_pages_copy(p.cache, i32([0, -1]), i32([int(p.pt.refcount.shape[0]) - 1, 3]), st)
    words = p.cache.data.transpose(0, 1).view(torch.int16)
    assert torch.equal(words[0], words[-1]) and int(st) == 0


# ------------------------------------------------------------------------------------------------- a run of them together
def test_a_run_as_it_is_served():
    """Two sequences: prompts appended, steps that add up weights, evictions whenever a budget is passed, pages given back.
    Each step's outputs are those of 64-bit attention over the tokens that are still there, and which ones these are
    follows from the sums that the kernels kept."""
    torch.manual_seed(0)
    kv, H, d, page, layers = 2, 8, 64, 16, 2
    cache = kda.KvCache.empty(layers, 40, page, kv, d, stats=True)
    pt = kda.PageTable.empty(2, 12, 40, page)
    rope = kda.Rope.make(d, 10000.0)
    st, pw = status(), torch.empty(kda.kda_pages_workspace_bytes(pt, 2), dtype=torch.uint8, device=DEV)
    ws = torch.empty(kda.kda_kv_decode_workspace_bytes(cache, H, 2, 1, 640), dtype=torch.uint8, device=DEV)
    p = Pages([1], kv, d, page)  # its helpers over this cache
    p.cache, p.pt = cache, pt
    seen = [37, 70]   # tokens so far, which are also the next positions
    held = [37, 70]
    budget, slack = 64, 5
    kda.kda_pages_reserve(pt, cache, i32([0, 1]), i32(held), pw, st)
    for l in range(layers):
        x = torch.randn(107, 2 * kv, d, device=DEV).to(torch.bfloat16)
        kda.kda_kv_append(cache, l, pt, None, cu_of(held), x[:, :kv], x[:, kv:], i32(list(range(37)) + list(range(70))), st,
                          rope=rope)
    evictions = 0
    for step in range(14):
        held = [h + 1 for h in held]
        kda.kda_pages_reserve(pt, cache, i32([0, 1]), i32(held), pw, st)
        for l in range(layers):
            x = torch.randn(2, H + 2 * kv, d, device=DEV).to(torch.bfloat16)
            qr = torch.empty(2, H, d, dtype=torch.bfloat16, device=DEV)
            kda.kda_kv_append(cache, l, pt, None, i32([0, 1, 2]), x[:, H:H + kv], x[:, H + kv:], i32(seen), st, rope=rope,
                              q=x[:, :H], q_out=qr)
            check(qr, *rotated(rope, x[:, :H], i32(seen)))
            sums = cache.weights.clone()
            out, lse = torch.empty_like(qr), torch.empty(2, H, device=DEV)
            kda.kda_kv_decode(cache, l, pt, None, None, 1, qr, out, lse, 0.125, ws, st, weight_decay=1.0)
            p.lens = held
            compare(p, qr, [1, 1], out, lse, layer=l, scale=0.125, sums=sums)
        seen = [s + 1 for s in seen]
        if max(held) > budget + slack:
            p.lens = held
            new = evict_and_compare(p, [budget, budget], first=2, since=[s - 8 for s in seen])
            kda.kda_pages_truncate(pt, i32([0, 1]), i32(new), pw, st)
            held = new
            evictions += 1
            assert pt.lens.tolist() == held and int((pt.refcount > 0).sum()) == sum(-(-h // page) for h in held)
            for b in range(2):  # the newest eight and the first two are there in every layer and head
                pid, slot = p.places(b, held[b])
                for l in range(layers):
                    for h in range(kv):
                        left = cache.positions[l, pid, h, slot].tolist()
                        assert set(left) >= {0, 1} | set(range(seen[b] - 8, seen[b])) and len(set(left)) == held[b]
    assert evictions >= 2 and int(st) == 0


def test_captured_step_follows_its_inputs():
    """Append, decode with sums and evict in one graph, replayed on other lengths and values; two graphs with a workspace
    each on two streams at once."""
    kv, H, d, page = 2, 8, 64, 16
    rope = kda.Rope.make(d)

    def state(seed):
        p = Pages([100, 100, 77], kv, d, page, stats=True, seed=seed, spare=20)  # pages for all lengths below
        s = dict(p=p, x=torch.randn(3, H + 2 * kv, d, device=DEV).to(torch.bfloat16), pos=i32([99, 39, 76]), st=status(),
                 qr=torch.empty(3, H, d, dtype=torch.bfloat16, device=DEV), keep=i32([90, 90, 60]),
                 new=torch.empty(3, dtype=torch.int32, device=DEV), cu=i32([0, 1, 2, 3]),
                 ws=torch.empty(kda.kda_kv_decode_workspace_bytes(p.cache, H, 3, 1, 5000), dtype=torch.uint8, device=DEV))
        s["out"], s["lse"] = torch.empty_like(s["qr"]), torch.empty(3, H, device=DEV)
        return s

    def step(s):
        x, p = s["x"], s["p"]
        kda.kda_kv_append(p.cache, 0, p.pt, None, s["cu"], x[:, H:H + kv], x[:, H + kv:], s["pos"], s["st"], rope=rope,
                          q=x[:, :H], q_out=s["qr"])
        kda.kda_kv_decode(p.cache, 0, p.pt, None, s["cu"], 1, s["qr"], s["out"], s["lse"], 0.125, s["ws"], s["st"],
                          weight_decay=1.0, max_slots=5000)
        kda.kda_kv_evict(p.cache, p.pt, None, s["keep"], s["new"], s["st"], first=3)

    def fields(s):
        return [s["p"].cache.data.view(torch.int16), s["out"], s["lse"], s["new"], s["qr"]]
    states = [state(1), state(2)]
    start = [s["p"].cache.data.clone() for s in states]
    for s in states:
        step(s)  # everything is loaded before the capture
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    for lens in ([100, 40, 77], [33, 16, 70], [1, 100, 64]):
        want = []
        for s, d0 in zip(states, start):
            s["p"].cache.data.copy_(d0)
            s["p"].pt.lens.copy_(i32(lens))
            s["x"].copy_(torch.randn(s["x"].shape, device=DEV))
            step(s)
            want.append([f.clone() for f in fields(s)])
            s["p"].cache.data.copy_(d0)
            s["out"].zero_()
            s["new"].zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip(states, want):
            assert all(torch.equal(a, b) for a, b in zip(fields(s), w)) and int(s["st"]) == 0


def test_calls_of_other_sizes_share_one_workspace():
    """What is enough for the largest is enough for all; nothing is kept in it between calls."""
    p = Pages([700, 64, 33, 1500], 2, 64, 16, stats=True)
    nbytes = kda.kda_kv_decode_workspace_bytes(p.cache, 64, 4, 8, 4000)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    for H, nq, decay in ((64, [8, 8, 8, 8], 1.0), (2, [1, 1, 1, 1], None), (64, [1, 2, 0, 3], 0.5), (8, [5, 1, 1, 1], None),
                         (32, [1, 1, 1, 1], 1.0)):
        assert kda.kda_kv_decode_workspace_bytes(p.cache, H, 4, max(nq), 4000 if decay else 0) <= nbytes
        sums = p.cache.weights.clone()
        q = queries(sum(nq), H, 64, torch.bfloat16, seed=H)
        out, lse, st = decode(p, q, nq, decay=decay, max_slots=4000 if decay else None, ws=ws)
        compare(p, q, nq, out, lse, sums=sums if decay else None, decay=decay)
        assert int(st) == 0 and (decay or torch.equal(sums, p.cache.weights))


def test_calls_on_a_given_stream_and_repeats_are_the_same():
    p = Pages([3000, 70, 900], 4, 128, 64, stats=True)
    q = queries(3, 16, 128, torch.bfloat16)
    first, lse, _ = decode(p, q, [1, 1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, l2, _ = decode(p, q, [1, 1, 1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, first) and torch.equal(lse, l2)
    start, got = p.cache.weights.clone(), []
    for _ in range(3):
        p.cache.weights.copy_(start)
        decode(p, q, [1, 1, 1], decay=1.0)
        got.append(p.cache.weights.clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_pages_past_32_bits():
    """A pool of more than 2^32 words, the row's tokens in its last pages."""
    kv, d, page = 8, 128, 64
    words = kda.KvCache.words(page, kv, d, True)
    num = (1 << 32) // words + 40
    data = torch.empty(1, num, words, dtype=torch.bfloat16, device=DEV)
    p = Pages([1], kv, d, page, stats=True)
    p.cache = kda.KvCache(data, kv, d, page, True)
    ids = [num - 1, num - 3, 5, num - 2]
    p.pt = kda.PageTable(i32([ids]), i32([200]), torch.ones(num, dtype=torch.int32, device=DEV), page)
    p.lens = [200]
    data[0, ids] = torch.randn(4, words, device=DEV).to(torch.bfloat16)
    p.cache.weights[0, ids] = torch.rand(4, kv, page, device=DEV)
    p.cache.positions[0, ids] = 7
    r = kda.Rope.make(d)
    x, st = torch.randn(2, 48, d, device=DEV).to(torch.bfloat16), status()
    kda.kda_kv_append(p.cache, 0, p.pt, None, i32([0, 2]), x[:, 32:40], x[:, 40:], i32([198, 199]), st, rope=r)
    pid, slot = p.places(0)
    check(p.cache.keys[0, pid[198:], :, slot[198:]], *rotated(r, x[:, 32:40], i32([198, 199])))
    q, sums = queries(1, 32, d, torch.bfloat16), p.cache.weights.clone()
    out, lse, _ = decode(p, q, [1], decay=1.0, max_slots=1000)
    compare(p, q, [1], out, lse, sums=sums)
    keys = p.cache.data[0, ids].clone()
    new = torch.empty(1, dtype=torch.int32, device=DEV)
    kda.kda_kv_evict(p.cache, p.pt, None, i32([100]), new, st)
    small = Pages([200], kv, d, page, stats=True)
    small.cache.data[0, small.pt.table[0, :4].long()] = keys
    kda.kda_kv_evict(small.cache, small.pt, None, i32([100]), new, st)
    assert int(st) == 0
    assert torch.equal(p.cache.data[0, ids].view(torch.int16),
                       small.cache.data[0, small.pt.table[0, :4].long()].view(torch.int16))
