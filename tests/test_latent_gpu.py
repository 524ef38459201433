"""Latent attention over the paged cache (kda_latent_append, _decode, _prefill) against plain 64-bit forms.

Tolerances are those of latent_testutil.attend, derived there from the number of roundings."""
import math

import numpy as np
import pytest
import torch

from tests.latent_testutil import F64, attend, check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def _kda():
    import hybrid_linear_attention_decode_gb300 as kda
    kda.load_library()
    return kda


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Problem:
    """A cache in random page order, queries, and the 64-bit answer."""

    def __init__(self, lens, nq, H=4, rank=128, rope=64, page=64, dtype=BF, layers=1, layer=0, seed=0, spare=3,
                 page_major=False, scale=None, width=None, uniform=False):
        self.kda = _kda()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.nq, self.H, self.rank, self.page, self.layer, self.dtype = lens, nq, H, rank, page, layer, dtype
        self.d = rank + rope
        k = [-(-x // page) for x in lens]
        num = sum(k) + spare
        shape = (num, layers, page, self.d) if page_major else (layers, num, page, self.d)
        pages = torch.randn(*shape, generator=g, device="cuda").to(dtype)
        self.pages = pages.transpose(0, 1) if page_major else pages
        rng = np.random.default_rng(seed)
        perm = rng.permutation(num)
        width = width or max(k + [1]) + 1
        t = np.full((len(lens), width), -1, np.int32)
        ref = np.zeros(num, np.int32)
        at = 0
        for i, c in enumerate(k):
            t[i, :c] = perm[at:at + c]
            ref[perm[at:at + c]] = 1
            at += c
        self.used = set(perm[:at].tolist())
        self.cache = self.kda.LatentCache(self.pages, rank)
        self.pt = self.kda.PageTable(_i32(t), _i32(lens), _i32(ref), page)
        self.T = sum(nq)
        self.q = torch.randn(self.T, H, self.d, generator=g, device="cuda").to(dtype)
        self.cu = None if uniform else _cu(nq)
        self.scale = scale or 1 / math.sqrt(192)
        self.status = _i32([0])
        self.out = torch.full((self.T, H, rank), -7.0, dtype=dtype, device="cuda")
        self.lse = torch.full((self.T, H), -7.0, device="cuda")

    def rows64(self, b):
        n = self.lens[b]
        pos = torch.arange(n, device="cuda")
        return self.pages[self.layer, self.pt.table[b].long()[pos // self.page], pos % self.page].to(F64)

    def run(self, rows=None, tree=None, q=None, status=0, stream=None):
        n = len(self.nq)
        nbytes = self.kda.kda_latent_decode_workspace_bytes(self.cache, self.H, n, max(self.nq))
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.kda.kda_latent_decode(self.cache, self.layer, self.pt, rows, self.cu, max(self.nq),
                                   self.q if q is None else q, self.out, self.lse, self.scale, ws, self.status,
                                   tree_mask=tree, stream=stream)
        torch.cuda.synchronize()
        assert int(self.status.item()) == status

    def seen(self, b, tree=None):
        """[nq, len] bool: what each query of sequence b sees."""
        k, n = self.nq[b], self.lens[b]
        j = torch.arange(n, device="cuda") - (n - k)
        t = torch.arange(k, device="cuda")
        if tree is None:
            return j[None, :] <= t[:, None]
        c0 = sum(self.nq[:b])
        m = tree[c0:c0 + k, None]
        return (j[None, :] < 0) | ((m >> j.clamp(min=0)[None, :]) & 1 == 1)

    def expect(self, b, tree=None, rows=None):
        c0, k, H = sum(self.nq[:b]), self.nq[b], self.H
        kv = self.rows64(b) if rows is None else rows
        q = self.q[c0:c0 + k].to(F64).reshape(k * H, self.d)
        seen = self.seen(b, tree).repeat_interleave(H, 0)
        o, l, to, tl = attend(q, kv, kv[:, :self.rank], seen, self.scale, self.dtype)
        return [x.reshape(k, H, *x.shape[1:]) for x in (o, l, to, tl)]

    def verify(self, tree=None, only=None):
        for b in range(len(self.nq)) if only is None else only:
            c0, k = sum(self.nq[:b]), self.nq[b]
            if k == 0:
                continue
            o, l, to, tl = self.expect(b, tree)
            check(self.out[c0:c0 + k], o, to, f"out of sequence {b}")
            check(self.lse[c0:c0 + k], l, tl, f"lse of sequence {b}")


DECODE = [
    # lens, nq, H, rank, rope, page, dtype
    ([1], [1], 1, 128, 64, 64, BF),
    ([1, 2, 15, 16, 17], [1] * 5, 3, 128, 16, 16, FP),
    ([63, 64, 65, 127, 128, 129], [1] * 6, 16, 256, 32, 32, BF),
    ([0, 5, 0, 700], [1] * 4, 5, 128, 0, 128, BF),
    ([1013], [1], 32, 512, 64, 64, BF),
    ([2500, 31, 999], [1] * 3, 32, 512, 64, 64, FP),
    ([1500, 77], [1] * 2, 64, 512, 64, 256, BF),
    ([777, 4001], [1] * 2, 128, 512, 64, 128, BF),
    ([333, 900, 64], [1] * 3, 65, 384, 48, 16, FP),
    ([300, 301, 8, 2], [5, 3, 8, 1], 20, 512, 64, 16, BF),
    ([600, 70], [8, 8], 32, 512, 64, 64, FP),
    ([400], [64], 7, 128, 64, 64, BF),
    ([64, 3], [64, 5], 32, 256, 64, 32, BF),   # the drafted tokens reach before the sequence: empty rows
    ([20000], [1], 16, 512, 64, 64, BF),
    ([40] * 200, [1] * 200, 16, 128, 64, 16, BF),
    ([130 + 7 * i for i in range(70)], [1 + i % 3 for i in range(70)], 32, 256, 64, 64, FP),
]


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_matches_64_bits(case):
    lens, nq, H, rank, rope, page, dt = DECODE[case]
    p = Problem(lens, nq, H, rank, rope, page, dt, seed=case)
    p.run()
    p.verify()


def test_decode_without_cu_tokens_lse_or_refcount_of_use():
    p = Problem([100, 0, 257], [2, 2, 2], H=8, uniform=True, seed=5)
    keep = p.lse
    p.lse = None
    p.run()
    p.lse = keep
    a = p.out.clone()
    p.run()
    assert torch.equal(a, p.out)  # the same call gives the same bits
    p.verify()


def test_decode_strided_queries_layers_and_page_major_cache():
    p = Problem([300, 41], [2, 1], H=6, rank=256, rope=32, page=32, layers=3, layer=2, page_major=True, seed=6)
    big = torch.full((p.T, 9, 2 * p.d), float("nan"), dtype=p.dtype, device="cuda")
    big[:, 1:7, 8:8 + p.d] = p.q
    p.run(q=big[:, 1:7, 8:8 + p.d])
    p.verify()


@pytest.mark.parametrize("H,page,dt", [(32, 16, BF), (5, 64, FP), (128, 128, BF)])
def test_decode_tree_masks(H, page, dt):
    nq = [8, 1, 0, 5, 33]
    p = Problem([500, 64, 10, 5, 90], nq, H=H, rank=512, page=page, dtype=dt, seed=H)
    rng = np.random.default_rng(H)
    masks = []
    for k in nq:
        anc = []
        for j in range(k):
            par = int(rng.integers(-1, j)) if j else -1
            anc.append((anc[par] if par >= 0 else 0) | (1 << j))
        masks += anc
    masks[3] = 0                      # sees the earlier tokens only
    masks[9] = 0                      # (sequence 3 has no earlier tokens: this query sees nothing)
    masks[11] = 0b10110               # not itself
    tree = torch.tensor(masks, dtype=torch.int64, device="cuda")
    p.run(tree=tree)
    p.verify(tree=tree)
    assert bool((p.out[9] == 0).all()) and bool((p.lse[9] == -math.inf).all())


def test_decode_tree_of_64_uses_the_top_bit():
    p = Problem([100], [64], H=2, seed=9)
    tree = torch.tensor([1 << j if j < 63 else -(1 << 63) for j in range(64)], dtype=torch.int64, device="cuda")
    p.run(tree=tree)
    p.verify(tree=tree)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_decode_unseen_rows_may_hold_anything(value, page):
    """Pages in no table, the tail of each last page, and drafted tokens that a query does not see."""
    lens, nq = [100, 17, 200], [1, 4, 8]
    p = Problem(lens, nq, H=16, rank=256, page=page, seed=11)
    p.run()
    clean, clean_l = p.out.clone(), p.lse.clone()
    for pg in range(p.pages.shape[1]):
        if pg not in p.used:
            p.pages[0, pg] = value
    for b, n in enumerate(lens):
        if n % page:
            p.pages[0, int(p.pt.table[b, n // page]), n % page:] = value
    p.run()
    assert torch.equal(p.out, clean) and torch.equal(p.lse, clean_l)
    # the last drafted token of the chains of 4 and 8: only the last query sees it
    for b in (1, 2):
        j = lens[b] - 1
        p.pages[0, int(p.pt.table[b, j // page]), j % page, 3] = value
    p.run()
    last = [4, 12]
    others = [i for i in range(p.T) if i not in last]
    assert torch.equal(p.out[others], clean[others]) and torch.equal(p.lse[others], clean_l[others])
    assert bool(torch.isnan(p.out[last]).all())


@pytest.mark.parametrize("before", [0, 7, 35, 64, 100])
def test_decode_marks_of_drafts_in_two_tiles(before):
    """60 drafted tokens over two tiles, each of which holds a row that is not finite; queries see both, one or none."""
    p = Problem([before + 60], [60], H=48, rank=128, page=16, seed=before)
    bad = (3, 59)
    free = [j for j in range(60) if j not in bad]
    masks = [sum(1 << j for j in free if j <= t or t in bad) | sum(1 << bad[i] for i in range(2) if t % 4 >> i & 1)
             for t in range(60)]
    tree = torch.tensor(masks, dtype=torch.int64, device="cuda")
    none = torch.tensor([m & ~(1 << 3) & ~(1 << 59) for m in masks], dtype=torch.int64, device="cuda")
    p.run(tree=none)
    clean = p.out.clone()
    for j in bad:
        p.pages[0, int(p.pt.table[0, (before + j) // 16]), (before + j) % 16, 2] = float("nan")
    for _ in range(20):
        p.run(tree=tree)
        for t in range(60):
            if t % 4:
                assert bool(torch.isnan(p.out[t]).all()), t
            else:
                assert torch.equal(p.out[t], clean[t]), t


def test_decode_one_bad_query_stays_alone():
    p = Problem([150, 90], [2, 2], H=20, rank=128, seed=12)
    p.run()
    clean = p.out.clone()
    p.q[1, 7] = float("nan")
    p.q[3, 19, 5] = float("inf")
    p.run()
    assert bool(torch.isnan(p.out[1, 7]).all())
    keep = torch.ones(p.T, p.H, dtype=torch.bool, device="cuda")
    keep[1, 7] = keep[3, 19] = False
    assert torch.equal(p.out[keep], clean[keep])


def test_decode_large_scores_and_a_rising_maximum():
    """Scores of several hundred that grow along the sequence: the running maximum moves at every tile."""
    p = Problem([900], [1], H=32, rank=512, seed=13, scale=1.0)
    rows = p.pages[0, p.pt.table[0, :15].long()]
    rows *= torch.linspace(0.05, 1.0, 15, device="cuda").to(p.dtype)[:, None, None]
    p.pages[0, p.pt.table[0, :15].long()] = rows
    p.run()
    p.verify()


def test_decode_rows_padding_repeats_and_rows_behind_the_last_sequence():
    p = Problem([64, 200, 33], [1, 2, 1], H=8, seed=14)
    nq, order = [2, 1, 1, 2], [1, -1, 1, 0]
    extra = 3
    q = torch.randn(sum(nq) + extra, 8, p.d, device="cuda").to(p.dtype)
    out = torch.full((q.shape[0], 8, p.rank), -7.0, dtype=p.dtype, device="cuda")
    lse = torch.full((q.shape[0], 8), -7.0, device="cuda")
    ws = torch.empty(p.kda.kda_latent_decode_workspace_bytes(p.cache, 8, 4, 2), dtype=torch.uint8, device="cuda")
    p.kda.kda_latent_decode(p.cache, 0, p.pt, _i32(order), _cu(nq), 2, q, out, lse, p.scale, ws, p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    c0 = 0
    for k, r in zip(nq, order):
        if r < 0:
            assert bool((out[c0:c0 + k] == 0).all()) and bool((lse[c0:c0 + k] == -math.inf).all())
        else:
            kv = p.rows64(r)
            j = torch.arange(p.lens[r], device="cuda") - (p.lens[r] - k)
            seen = (j[None, :] <= torch.arange(k, device="cuda")[:, None]).repeat_interleave(8, 0)
            o, l, to, tl = attend(q[c0:c0 + k].to(F64).reshape(k * 8, -1), kv, kv[:, :p.rank], seen, p.scale, p.dtype)
            check(out[c0:c0 + k].reshape(k * 8, -1), o, to)
            check(lse[c0:c0 + k].reshape(k * 8), l, tl)
        c0 += k
    assert bool((out[c0:] == -7).all()) and bool((lse[c0:] == -7).all())


def test_decode_bad_tables_are_flagged_and_contained():
    kda = _kda()
    p = Problem([64, 200, 33, 50], [1] * 4, H=8, seed=15)
    p.pt.lens[0] = 10 ** 6          # longer than the table
    p.pt.lens[2] = -4
    p.run(status=kda.KDA_DEV_BAD_SEQLENS)
    p.verify(only=[1, 3])
    assert bool((p.out[[0, 2]] == 0).all()) and bool((p.lse[[0, 2]] == -math.inf).all())
    p.pt.lens.copy_(_i32([64, 200, 33, 50]))
    p.status.zero_()
    p.pt.table[1, 1] = p.pages.shape[1]
    p.pt.table[3, 0] = -1
    p.run(status=kda.KDA_DEV_BAD_PAGE)
    p.verify(only=[0, 2])
    zero = p.pages.shape[1]
    for b in (1, 3):                # a bad page's tokens read as zero rows
        t = p.pt.table[b].clone()
        n = p.lens[b]
        pos = torch.arange(n, device="cuda")
        pg = t.long()[pos // 64]
        bad = (pg < 0) | (pg >= zero)
        kv = p.pages[0, pg.clamp(0, zero - 1), pos % 64].to(F64) * (~bad)[:, None]
        o, l, to, tl = p.expect(b, rows=kv)
        check(p.out[b:b + 1], o, to)
        check(p.lse[b:b + 1], l, tl)
    p = Problem([64, 200], [1, 1], H=8, seed=16)
    p.run(rows=_i32([5, 1]), status=kda.KDA_DEV_BAD_SLOT)
    p.verify(only=[1])
    assert bool((p.out[0] == 0).all())
    # cu_tokens that run backwards or past the end: those sequences are left alone
    p = Problem([64, 200, 30], [1, 1, 1], H=8, seed=17)
    p.cu = _i32([0, 1, 0, 9])
    p.run(status=kda.KDA_DEV_BAD_SEQLENS)
    p.verify(only=[0])
    assert bool((p.out[1:] == -7).all())


def test_decode_on_a_side_stream_and_in_a_replayed_graph():
    p = Problem([500, 130], [1, 1], H=16, rank=512, seed=18)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.run(stream=s)
    p.verify()
    ws = torch.empty(p.kda.kda_latent_decode_workspace_bytes(p.cache, 16, 2, 1), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.kda.kda_latent_decode(p.cache, 0, p.pt, None, p.cu, 1, p.q, p.out, p.lse, p.scale, ws, p.status)
    for lens in ([500, 130], [64, 0], [1, 129], [333, 65]):  # lengths are read at replay
        p.lens = lens
        p.pt.lens.copy_(_i32(lens))
        p.out.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        p.verify()


def test_decode_thousands_of_entries_mostly_padding():
    """6000 entries, of which 37 have a sequence (some the same), of 0 to 900 tokens."""
    lens = [0, 1, 900, 64, 129, 500, 65]
    p = Problem(lens, [1] * len(lens), H=8, rank=128, seed=21)
    n = 6000
    at = list(range(0, n, 167)) + [n - 1]
    rows = np.full(n, -1, np.int32)
    rows[at] = np.arange(len(at)) % len(lens)
    q = torch.zeros(n, 8, p.d, dtype=p.dtype, device="cuda")
    q[at] = torch.randn(len(at), 8, p.d, device="cuda").to(p.dtype)
    out, lse = torch.full((n, 8, 128), -7.0, dtype=p.dtype, device="cuda"), torch.full((n, 8), -7.0, device="cuda")
    ws = torch.empty(p.kda.kda_latent_decode_workspace_bytes(p.cache, 8, n, 1), dtype=torch.uint8, device="cuda")
    p.kda.kda_latent_decode(p.cache, 0, p.pt, _i32(rows), None, 1, q, out, lse, p.scale, ws, p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    for i in at:
        kv = p.rows64(int(rows[i]))
        seen = torch.ones(8, kv.shape[0], dtype=torch.bool, device="cuda")
        o, l, to, tl = attend(q[i].to(F64), kv, kv[:, :128], seen, p.scale, p.dtype)
        check(out[i], o, to, f"out of entry {i}")
        check(lse[i], l, tl, f"lse of entry {i}")
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((out[rest] == 0).all()) and bool((lse[rest] == -math.inf).all())


def test_calls_on_two_streams_at_once():
    """Decode, prefill and a second decode with its own workspace, queued on three streams, give what they give alone."""
    a = Problem([3000, 70, 900], [2, 1, 4], H=32, rank=512, seed=22)
    b = Problem([1200] * 9, [1] * 9, H=64, rank=256, seed=23)
    c = Prompt([700, 90], [1500, 90], H=16, seed=24)
    for x in (a, b, c):
        x.run()
    want = [(x.out.clone(), x.lse.clone()) for x in (a, b, c)]
    ws = [torch.empty(x.kda.kda_latent_decode_workspace_bytes(x.cache, x.H, len(x.nq), max(x.nq)), dtype=torch.uint8,
                      device="cuda") for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for x in (a, b, c):
        x.out.fill_(-7)
        x.lse.fill_(-7)
    torch.cuda.synchronize()
    for _ in range(8):
        for x, w, s in zip((a, b), ws, streams):
            x.kda.kda_latent_decode(x.cache, 0, x.pt, None, x.cu, max(x.nq), x.q, x.out, x.lse, x.scale, w, x.status, stream=s)
        c.kda.kda_latent_prefill(c.cu_q, c.cu_k, 700, c.q, c.k, c.r, c.v, c.out, c.lse, c.scale, c.status, stream=streams[2])
    torch.cuda.synchronize()
    for x, (out, lse) in zip((a, b, c), want):
        assert int(x.status.item()) == 0
        assert torch.equal(x.out, out) and torch.equal(x.lse, lse)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_ordered_by_events_across_streams(captured):
    """Rows appended on one stream, read by decodes of two layers on two streams, which a third call waits for."""
    kda = _kda()
    lens = [700, 64, 1]
    p = Problem(lens, [1, 1, 1], H=32, rank=512, layers=2, seed=25)
    old = p.pages.clone()
    new = torch.randn(2, 3, p.d, device="cuda").to(p.dtype)
    cu = _cu([1, 1, 1])
    out = torch.zeros(2, 3, 32, 512, dtype=p.dtype, device="cuda")
    lse = torch.zeros(2, 3, 32, device="cuda")
    ws = [torch.empty(kda.kda_latent_decode_workspace_bytes(p.cache, 32, 3, 1), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    last = torch.tensor([int(p.pt.table[b, (n - 1) // 64]) for b, n in enumerate(lens)])
    src, dst = _i32([int(last[0])]), _i32([min(set(range(p.pages.shape[1])) - p.used)])
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        for layer in range(2):
            kda.kda_latent_append(p.cache, layer, p.pt, None, cu, new[layer, :, :512], new[layer, :, 512:], p.status)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kda.kda_latent_decode(p.cache, 1, p.pt, None, cu, 1, p.q, out[1], lse[1], p.scale, ws[1], p.status)
        kda.kda_latent_decode(p.cache, 0, p.pt, None, cu, 1, p.q, out[0], lse[0], p.scale, ws[0], p.status)
        main.wait_stream(side)
        kda.kda_pages_copy(p.cache, src, dst, p.status)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(g):
            step()
    for k in range(6):
        p.pages.copy_(old)
        new.copy_(torch.randn(2, 3, p.d, device="cuda"))
        out.zero_()
        g.replay() if captured else step()
        torch.cuda.synchronize()
        assert int(p.status.item()) == 0
        assert torch.equal(p.pages[:, int(dst)], p.pages[:, int(src)])
        for layer in range(2):
            p.layer = layer
            for b, n in enumerate(lens):
                assert torch.equal(p.pages[layer, int(last[b]), (n - 1) % 64], new[layer, b])
                o, l, to, tl = p.expect(b)
                check(out[layer, b:b + 1], o, to, f"step {k}, layer {layer}, sequence {b}")
                check(lse[layer, b:b + 1], l, tl)


def test_decode_rows_at_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements, read at its far end."""
    kda = _kda()
    rank, rope, page = 512, 64, 64
    num = (1 << 31) // (page * 576) + 40
    cache = kda.LatentCache(torch.empty(1, num, page, 576, dtype=BF, device="cuda"), rank)
    lens = [150, 64 * 3]
    t = _i32([[num - 1, num - 7, num - 20], [3, num - 2, 0]])
    pt = kda.PageTable(t, _i32(lens), torch.ones(num, dtype=torch.int32, device="cuda"), page)
    new = torch.randn(sum(lens), 576, device="cuda").to(BF)
    st = _i32([0])
    kda.kda_latent_append(cache, 0, pt, None, _cu(lens), new[:, :512], new[:, 512:], st)
    q = torch.randn(2, 32, 576, device="cuda").to(BF)
    out, lse = torch.empty(2, 32, 512, dtype=BF, device="cuda"), torch.empty(2, 32, device="cuda")
    ws = torch.empty(kda.kda_latent_decode_workspace_bytes(cache, 32, 2, 1), dtype=torch.uint8, device="cuda")
    kda.kda_latent_decode(cache, 0, pt, None, None, 1, q, out, lse, 0.07, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    at = 0
    for b, n in enumerate(lens):
        kv = new[at:at + n].to(F64)
        at += n
        o, l, to, tl = attend(q[b].to(F64), kv, kv[:, :512], torch.ones(32, n, dtype=torch.bool, device="cuda"), 0.07, BF)
        check(out[b], o, to)
        check(lse[b], l, tl)


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("page,rank,rope,dt", [(16, 128, 0, BF), (64, 512, 64, FP), (128, 256, 48, BF)])
def test_append_writes_exactly_its_rows(page, rank, rope, dt):
    kda = _kda()
    lens, new = [70, 1, 300, 40, 5], [70, 0, 37, 40, 1]
    p = Problem(lens, [1] * 5, rank=rank, rope=rope, page=page, dtype=dt, layers=2, layer=1, seed=20)
    T = sum(new) + 2
    src = torch.randn(T, rank + rope + 16, device="cuda").to(dt)
    lat, rp = src[:, 8:8 + rank], src[:, 8 + rank:8 + rank + rope] if rope else None
    want = p.pages.clone()
    order, c0 = [0, 1, 2, -1, 4], 0
    for b, k in enumerate(new):
        for i in range(k):
            pos = lens[b] - k + i
            if order[b] >= 0:
                want[1, int(p.pt.table[b, pos // page]), pos % page] = src[c0 + i, 8:8 + rank + rope]
        c0 += k
    st = _i32([0])
    kda.kda_latent_append(p.cache, 1, p.pt, _i32(order), _cu(new), lat, rp, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(p.pages, want)


def test_append_flags_bad_rows_lengths_and_pages():
    kda = _kda()
    for spoil, bit in (("row", kda.KDA_DEV_BAD_SLOT), ("len", kda.KDA_DEV_BAD_SEQLENS), ("page", kda.KDA_DEV_BAD_PAGE),
                       ("cu", kda.KDA_DEV_BAD_SEQLENS)):
        p = Problem([10, 20], [1, 1], seed=21)
        want = p.pages.clone()
        rows, cu = _i32([0, 1]), _cu([3, 4])
        src = torch.randn(7, p.d, device="cuda").to(p.dtype)
        if spoil == "row":
            rows[0] = 2
        elif spoil == "len":
            p.pt.lens[0] = 2     # three tokens cannot be the last of two: the first has no place
        elif spoil == "page":
            p.pt.table[0, 0] = 10 ** 6
        else:
            cu[2] = 99           # past the tokens
        st = _i32([0])
        kda.kda_latent_append(p.cache, 0, p.pt, rows, cu, src[:, :p.rank], src[:, p.rank:], st)
        torch.cuda.synchronize()
        assert int(st.item()) == bit, spoil
        if spoil != "cu":
            for i in range(4):
                want[0, int(p.pt.table[1, 0]), 16 + i] = src[3 + i]
        if spoil == "len":
            for i in (1, 2):
                want[0, int(p.pt.table[0, 0]), i - 1] = src[i]
        if spoil == "cu":
            for i in range(3):
                want[0, int(p.pt.table[0, 0]), 7 + i] = src[i]
        assert torch.equal(p.pages, want), spoil


# ------------------------------------------------------------------------------------------------ prefill
class Prompt:
    def __init__(self, nq, nk, H=2, nope=128, rope=64, dv=128, dtype=BF, causal=True, seed=0, extra_q=0, extra_k=0):
        self.kda = _kda()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.nq, self.nk, self.H, self.nope, self.dv, self.dtype, self.causal = nq, nk, H, nope, dv, dtype, causal
        Tq, Tk = sum(nq) + extra_q, sum(nk) + extra_k

        def rn(*s):
            return torch.randn(*s, generator=g, device="cuda").to(dtype)

        self.q, self.k, self.r, self.v = rn(Tq, H, nope + rope), rn(Tk, H, nope), rn(Tk, rope), rn(Tk, H, dv)
        self.cu_q, self.cu_k = _cu(nq), _cu(nk)
        self.scale = 1 / math.sqrt(nope + rope)
        self.out = torch.full((Tq, H, dv), -7.0, dtype=dtype, device="cuda")
        self.lse = torch.full((Tq, H), -7.0, device="cuda")
        self.status = _i32([0])

    def run(self, status=0, stream=None, **other):
        a = dict(q=self.q, k=self.k, r=self.r, v=self.v)
        a.update(other)
        self.kda.kda_latent_prefill(self.cu_q, self.cu_k, max(self.nq), a["q"], a["k"], a["r"], a["v"], self.out, self.lse,
                                    self.scale, self.status, causal=self.causal, stream=stream)
        torch.cuda.synchronize()
        assert int(self.status.item()) == status

    def verify(self, only=None, heads=None):
        q0 = k0 = 0
        for b, (n, m) in enumerate(zip(self.nq, self.nk)):
            if n and (only is None or b in only):
                j, i = torch.arange(m, device="cuda"), torch.arange(n, device="cuda")
                seen = (j[None, :] <= i[:, None] + (m - n)) if self.causal else torch.ones(n, m, dtype=torch.bool,
                                                                                         device="cuda")
                for h in range(self.H) if heads is None else heads:
                    key = torch.cat([self.k[k0:k0 + m, h], self.r[k0:k0 + m]], 1).to(F64)
                    o, l, to, tl = attend(self.q[q0:q0 + n, h].to(F64), key, self.v[k0:k0 + m, h].to(F64), seen,
                                          self.scale, self.dtype)
                    check(self.out[q0:q0 + n, h], o, to, f"out of sequence {b}, head {h}")
                    check(self.lse[q0:q0 + n, h], l, tl, f"lse of sequence {b}, head {h}")
            q0 += n
            k0 += m


PREFILL = [
    # nq, nk, H, nope, rope, dv, dtype, causal
    ([1], [1], 1, 128, 64, 128, BF, True),
    ([1, 2, 63], [1, 2, 63], 2, 64, 32, 64, FP, True),
    ([64, 65, 127, 128], [64, 65, 127, 128], 2, 128, 64, 128, BF, True),
    ([129, 255, 256, 257], [129, 255, 256, 257], 1, 128, 64, 128, FP, True),
    ([300], [300], 3, 128, 48, 64, BF, False),
    ([5, 0, 130], [700, 9, 131], 2, 128, 64, 128, BF, True),
    ([200, 10], [600, 0], 2, 64, 16, 128, BF, True),       # no keys at all
    ([200, 10], [600, 0], 2, 64, 16, 128, FP, False),
    ([150, 300], [20, 140], 2, 128, 64, 128, BF, True),    # fewer keys than queries: the first queries see none
    ([1000], [1000], 4, 128, 64, 128, BF, True),
    ([1], [3000], 4, 128, 64, 128, BF, True),
    ([33, 513, 700], [833, 513, 1700], 32, 128, 64, 128, BF, True),
    ([400, 30], [1111, 900], 5, 128, 64, 128, FP, False),
]


@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_prefill_matches_64_bits(case):
    nq, nk, H, nope, rope, dv, dt, causal = PREFILL[case]
    p = Prompt(nq, nk, H, nope, rope, dv, dt, causal, seed=case)
    p.run()
    p.verify()


# The same with so many heads that a CTA has two query tiles (small calls have one)
WIDE = [
    # nq, nk, nope, rope, dv, dtype, causal
    ([1, 2, 63, 64, 65], [1, 2, 63, 64, 65], 128, 64, 128, BF, True),
    ([127, 128, 129, 255, 256, 257], [127, 128, 129, 255, 256, 257], 128, 64, 128, FP, True),
    ([300, 511, 512, 513], [300, 511, 512, 513], 64, 32, 64, BF, True),
    ([300, 140], [300, 900], 128, 48, 64, BF, False),
    ([200, 10, 0, 290], [600, 0, 5, 20], 64, 16, 128, BF, True),
    ([400, 385], [1111, 385], 128, 64, 128, FP, False),
]


@pytest.mark.parametrize("case", range(len(WIDE)))
def test_prefill_two_query_tiles_match_64_bits(case):
    nq, nk, nope, rope, dv, dt, causal = WIDE[case]
    p = Prompt(nq, nk, 96, nope, rope, dv, dt, causal, seed=100 + case)
    p.run()
    p.verify(heads=[0, 50, 95])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_prefill_two_query_tiles_unseen_keys_and_values_may_hold_anything(value):
    p = Prompt([150, 100, 260], [150, 130, 460], H=96, seed=132)
    p.run()
    clean, clean_l = p.out.clone(), p.lse.clone()
    p.v[120, 1, 3] = value           # queries 120.. of the first sequence see key 120
    p.k[279, 7] = value              # only the second sequence's last query sees its last key
    p.v[280 + 300, 90] = value       # queries 100.. of the third see its key 300
    p.v[280 + 459, 40, 100] = value  # only its last query sees its last key
    p.run()
    keep = torch.ones(510, 96, dtype=torch.bool, device="cuda")
    keep[120:150, 1] = keep[249, 7] = keep[350:, 90] = keep[509, 40] = False
    assert torch.equal(p.out[keep], clean[keep]) and torch.equal(p.lse[keep], clean_l[keep])
    assert bool((~torch.isfinite(p.out[120:150, 1, 3])).all()) and bool(torch.isnan(p.out[249, 7]).all())
    assert bool((~torch.isfinite(p.out[350:, 90])).all()) and bool((~torch.isfinite(p.out[509, 40, 100])).all())


def test_prefill_two_query_tiles_rising_maximum_and_bad_query():
    p = Prompt([700], [700], H=96, seed=134)
    ramp = torch.linspace(0.05, 1, 700, device="cuda")
    p.k.copy_(p.k.float() * ramp[:, None, None])
    p.r.copy_(p.r.float() * ramp[:, None])
    p.scale = 1.5
    p.run()
    p.verify(heads=[3, 77])
    clean = p.out.clone()
    p.q[300, 5, 9] = float("nan")
    p.run()
    keep = torch.ones(700, 96, dtype=torch.bool, device="cuda")
    keep[300, 5] = False
    assert torch.equal(p.out[keep], clean[keep]) and bool(torch.isnan(p.out[300, 5]).all())


def test_prefill_long_sequence_sampled_heads():
    p = Prompt([4500], [5000], H=6, seed=30)
    p.run()
    p.verify(heads=[0, 5])


def test_prefill_of_a_sequence_does_not_depend_on_the_others():
    """Bit for bit, where the calls are cut alike (the same bound of 700 queries: two query tiles a CTA)."""
    p = Prompt([300, 90, 700], [300, 400, 1700], H=96, seed=46)
    p.run()
    q0 = k0 = 0
    for n, m in zip(p.nq, p.nk):
        out = torch.empty(n, 96, 128, dtype=p.dtype, device="cuda")
        p.kda.kda_latent_prefill(_cu([n]), _cu([m]), 700, p.q[q0:q0 + n], p.k[k0:k0 + m], p.r[k0:k0 + m], p.v[k0:k0 + m],
                                 out, None, p.scale, p.status)
        torch.cuda.synchronize()
        assert torch.equal(out, p.out[q0:q0 + n])
        q0 += n
        k0 += m


def test_prefill_strided_inputs_and_rows_behind_the_last_sequence():
    p = Prompt([140, 77], [240, 177], H=3, seed=31, extra_q=5, extra_k=9)
    Tq, Tk = p.q.shape[0], p.k.shape[0]
    nan = float("nan")
    kv = torch.full((Tk, 4, 264), nan, dtype=p.dtype, device="cuda")
    kv[:, 1:, :128], kv[:, 1:, 128:256] = p.k, p.v
    qq = torch.full((Tq, 3, 256), nan, dtype=p.dtype, device="cuda")
    qq[:, :, 64:] = p.q
    rr = torch.full((Tk, 72), nan, dtype=p.dtype, device="cuda")
    rr[:, 8:] = p.r
    kv[417:] = nan
    rr[417:] = nan
    p.run(q=qq[:, :, 64:], k=kv[:, 1:, :128], v=kv[:, 1:, 128:256], r=rr[:, 8:])
    p.verify()
    assert bool((p.out[217:] == -7).all()) and bool((p.lse[217:] == -7).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_prefill_unseen_keys_and_values_may_hold_anything(value):
    nq, nk = [150, 100, 260], [150, 130, 260]
    p = Prompt(nq, nk, H=2, seed=32)
    p.run()
    clean, clean_l = p.out.clone(), p.lse.clone()
    # key 120 of the first sequence: its queries 0..119 do not see it; the whole third sequence: the second's do not
    p.v[120, 1, 3] = value
    p.k[280:, 0] = value
    p.v[280:] = value
    p.run()
    keep = torch.ones(510, 2, dtype=torch.bool, device="cuda")
    keep[120:150, 1] = False
    keep[250:] = False
    assert torch.equal(p.out[keep], clean[keep]) and torch.equal(p.lse[keep], clean_l[keep])
    assert bool((~torch.isfinite(p.out[120:150, 1, 3])).all())
    p.r[149] = value                 # the last key of the first sequence: its last query alone
    p.run()
    keep[149] = False
    assert torch.equal(p.out[keep], clean[keep])
    assert bool(torch.isnan(p.out[149]).all())


@pytest.mark.parametrize("nq,nk,dims", [(1, 129, (128, 64, 128)), (7, 1000, (64, 16, 64)), (100, 600, (128, 64, 128)),
                                        (128, 128 * 9, (64, 32, 128)), (384, 2048, (128, 48, 64)), (257, 257, (64, 64, 64))])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_few_queries_over_many_keys(nq, nk, dims, causal):
    """A last query tile that stands alone: its even and odd key tiles are joined at the end."""
    p = Prompt([nq, 3], [nk, 300], H=3, nope=dims[0], rope=dims[1], dv=dims[2], causal=causal, seed=nq + nk, dtype=FP)
    p.run()
    p.verify()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prefill_few_queries_unseen_values_may_hold_anything(value):
    p = Prompt([100, 50], [700, 333], H=2, seed=38)
    p.run()
    clean = p.out.clone()
    p.v[650, 0, 7] = value           # queries 50.. of the first sequence see key 650
    p.v[700 + 300, 1] = value        # queries 17.. of the second see its key 300
    p.run()
    keep = torch.ones(150, 2, dtype=torch.bool, device="cuda")
    keep[50:100, 0] = keep[117:, 1] = False
    assert torch.equal(p.out[keep], clean[keep])
    assert bool((~torch.isfinite(p.out[50:100, 0, 7])).all()) and bool((~torch.isfinite(p.out[117:, 1])).all())


def test_prefill_rising_maximum_over_alternating_key_tiles():
    """Odd key tiles of 128 score far above the even ones (and the other way round): each half has its own maximum."""
    for odd in (0, 1):
        p = Prompt([60], [128 * 6 + 40], H=2, seed=39 + odd)
        k = p.k.float().view(-1, 2, 128)
        tile = (torch.arange(k.shape[0], device="cuda") // 128) % 2
        p.k.copy_((k * torch.where(tile == odd, 6.0, 0.05)[:, None, None]).view_as(p.k))
        p.run()
        p.verify()


@pytest.mark.parametrize("layout", ["head-major", "odd"])
def test_prefill_and_decode_of_other_layouts(layout):
    """[H, T, d] tensors, and strides that are multiples of 8 and of nothing else."""
    def lay(x):
        T, H, d = x.shape
        if layout == "head-major":
            y = torch.empty(H, T, d, dtype=x.dtype, device="cuda").transpose(0, 1)
        else:
            y = torch.empty(T * (H * (d + 8) + 24), dtype=x.dtype, device="cuda").as_strided((T, H, d),
                                                                                        (H * (d + 8) + 24, d + 8, 1))
        y.copy_(x)
        return y
    p = Prompt([200, 130], [300, 130], H=3, seed=44)
    p.run(q=lay(p.q), k=lay(p.k), v=lay(p.v))
    p.verify()
    d = Problem([300, 41, 129], [2, 1, 4], H=6, rank=256, rope=64, seed=45)
    d.run(q=lay(d.q))
    d.verify()


def test_prefill_one_bad_query_stays_alone():
    p = Prompt([300], [300], H=2, seed=33)
    p.run()
    clean = p.out.clone()
    p.q[17, 0] = float("nan")
    p.q[200, 1, 3] = float("inf")
    p.run()
    keep = torch.ones(300, 2, dtype=torch.bool, device="cuda")
    keep[17, 0] = keep[200, 1] = False
    assert torch.equal(p.out[keep], clean[keep]) and bool(torch.isnan(p.out[17, 0]).all())


def test_prefill_large_scores_and_a_rising_maximum():
    p = Prompt([700], [700], H=2, seed=34)
    ramp = torch.linspace(0.05, 1, 700, device="cuda")
    p.k.copy_(p.k.float() * ramp[:, None, None])
    p.r.copy_(p.r.float() * ramp[:, None])
    p.scale = 1.5
    p.run()
    p.verify()


def test_prefill_bad_tables_are_flagged_and_contained():
    kda = _kda()
    p = Prompt([100, 50, 60], [100, 50, 60], seed=35)
    p.cu_q[3] = 9999
    p.run(status=kda.KDA_DEV_BAD_SEQLENS)
    p.verify(only=[0, 1])
    assert bool((p.out[150:] == -7).all())
    p = Prompt([100, 50, 60], [100, 50, 60], seed=36)
    p.cu_k[1] = 160                  # the second sequence's keys run backwards
    p.nk = [160, 50, 60]
    p.run(status=kda.KDA_DEV_BAD_SEQLENS)
    assert bool((p.out[100:150] == -7).all())


def test_prefill_on_a_side_stream_and_in_a_replayed_graph():
    p = Prompt([200, 100], [200, 180], seed=37)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.run(stream=s)
    p.verify()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.kda.kda_latent_prefill(p.cu_q, p.cu_k, 250, p.q, p.k, p.r, p.v, p.out, p.lse, p.scale, p.status)
    for nq, nk in (([200, 100], [200, 180]), ([250, 50], [300, 80])):
        p.nq, p.nk = nq, nk
        p.cu_q.copy_(_cu(nq))
        p.cu_k.copy_(_cu(nk))
        p.out.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        p.verify()


# ------------------------------------------------------------------------------------------------ together
def test_prompt_decode_drafts_forks_and_compaction_together():
    """A serving run: a prompt by the expanded form, its rows appended; then tokens decoded by the absorbed form,
    a drafted tree verified and cut back, a fork, and a compaction.  Both forms answer from the same layer: the
    absorbed queries are q_nope W_K^h (fp64 here, rounded to the type once), and W_V^h o~ is compared with the
    64-bit attention over the expanded keys and values of the same rounded rows."""
    kda = _kda()
    H, nope, rope, dv, rank, page = 4, 128, 64, 128, 256, 32
    g = torch.Generator(device="cuda").manual_seed(40)
    wk = (torch.randn(H, nope, rank, generator=g, device="cuda") / 16).to(F64)
    wv = (torch.randn(H, dv, rank, generator=g, device="cuda") / 16).to(F64)
    pt = kda.PageTable.empty(6, 40, 60, page)
    cache = kda.LatentCache.empty(2, 60, page, rank, rope)
    ws = torch.empty(kda.kda_pages_workspace_bytes(pt, 4), dtype=torch.uint8, device="cuda")
    st = _i32([0])
    scale = 1 / math.sqrt(nope + rope)
    rows_of = {0: [], 2: []}

    def fresh(k):
        x = torch.randn(k, rank + rope, generator=g, device="cuda").to(BF)
        return x, torch.randn(k, H, nope + rope, generator=g, device="cuda").to(BF)

    def expand(x):
        c = x[:, :rank].to(F64)
        return torch.einsum("tr,hnr->thn", c, wk), torch.einsum("tr,hvr->thv", c, wv)

    def absorbed(q):
        return torch.cat([torch.einsum("thn,hnr->thr", q[..., :nope].to(F64), wk), q[..., nope:].to(F64)], -1).to(BF)

    def decode(rows, nq, q, tree=None):
        qa = absorbed(q)
        out, lse = torch.empty(len(q), H, rank, dtype=BF, device="cuda"), torch.empty(len(q), H, device="cuda")
        w = torch.empty(kda.kda_latent_decode_workspace_bytes(cache, H, len(nq), max(nq)), dtype=torch.uint8,
                        device="cuda")
        kda.kda_latent_decode(cache, 1, pt, _i32(rows), _cu(nq), max(nq), qa, out, lse, scale, w, st, tree_mask=tree)
        c0 = 0
        for r, k in zip(rows, nq):
            kv = torch.cat(rows_of[r]).to(F64)
            n = len(kv)
            j = torch.arange(n, device="cuda") - (n - k)
            if tree is None:
                seen = j[None, :] <= torch.arange(k, device="cuda")[:, None]
            else:
                seen = (j[None, :] < 0) | ((tree[c0:c0 + k, None] >> j.clamp(min=0)[None, :]) & 1 == 1)
            o, l, to, tl = attend(qa[c0:c0 + k].to(F64).reshape(k * H, -1), kv, kv[:, :rank],
                                  seen.repeat_interleave(H, 0), scale, BF)
            check(out[c0:c0 + k].reshape(k * H, -1), o, to, "decode")
            check(lse[c0:c0 + k].reshape(k * H), l, tl, "decode")
            c0 += k
        return out

    # two prompts
    lens = [100, 45]
    kda.kda_pages_reserve(pt, cache, _i32([0, 2]), _i32(lens), ws, st)
    x, q = fresh(sum(lens))
    kda.kda_latent_append(cache, 1, pt, _i32([0, 2]), _cu(lens), x[:, :rank], x[:, rank:], st)
    rows_of[0], rows_of[2] = [x[:100]], [x[100:]]
    kn, v = (t.to(BF) for t in expand(x))
    out = torch.empty(145, H, dv, dtype=BF, device="cuda")
    kda.kda_latent_prefill(_cu(lens), _cu(lens), 100, q, kn, x[:, rank:], v, out, None, scale, st)
    for a, e in ((0, 100), (100, 145)):
        seen = torch.ones(e - a, e - a, dtype=torch.bool, device="cuda").tril()
        for h in range(H):
            key = torch.cat([kn[a:e, h], x[a:e, rank:]], 1).to(F64)
            o, _, to, _ = attend(q[a:e, h].to(F64), key, v[a:e, h].to(F64), seen, scale, BF)
            check(out[a:e, h], o, to, "prefill")
    # the absorbed form over the cache gives what the expanded form gave for the last prompt token
    last = decode([0, 2], [1, 1], q[[99, 144]])
    both = torch.einsum("thr,hvr->thv", last.to(F64), wv)
    # both sides round inputs, weights and outputs to bf16: a few roundings of 2^-8 of values near 1
    assert float((both - out[[99, 144]].to(F64)).abs().max()) < 16 * 2.0 ** -8
    # three decoded tokens each
    for step in range(3):
        lens = [n + 1 for n in lens]
        kda.kda_pages_reserve(pt, cache, _i32([0, 2]), _i32(lens), ws, st)
        x, q = fresh(2)
        kda.kda_latent_append(cache, 1, pt, _i32([0, 2]), _cu([1, 1]), x[:, :rank], x[:, rank:], st)
        rows_of[0].append(x[:1])
        rows_of[2].append(x[1:])
        decode([0, 2], [1, 1], q)
    # a drafted tree of 4 on row 0, of which the first two are kept
    kda.kda_pages_reserve(pt, cache, _i32([0]), _i32([lens[0] + 4]), ws, st)
    x, q = fresh(4)
    kda.kda_latent_append(cache, 1, pt, _i32([0]), _cu([4]), x[:, :rank], x[:, rank:], st)
    rows_of[0].append(x)
    decode([0], [4], q, tree=torch.tensor([1, 3, 5, 9], dtype=torch.int64, device="cuda"))
    lens[0] += 2
    rows_of[0][-1] = x[:2]
    kda.kda_pages_truncate(pt, _i32([0]), _i32([lens[0]]), ws, st)
    # two branches of row 0, each with a token of its own; the parent goes on too
    kda.kda_pages_fork(pt, cache, _i32([0, 0]), _i32([1, 5]), ws, st)
    for r in (1, 5):
        rows_of[r] = list(rows_of[0])
    rows = [0, 1, 5]
    kda.kda_pages_reserve(pt, cache, _i32(rows), _i32([lens[0] + 1] * 3), ws, st)
    x, q = fresh(3)
    kda.kda_latent_append(cache, 1, pt, _i32(rows), _cu([1, 1, 1]), x[:, :rank], x[:, rank:], st)
    for i, r in enumerate(rows):
        rows_of[r].append(x[i:i + 1])
    decode(rows, [1, 1, 1], q)
    # the parent ends, the pool is compacted, the rest goes on
    kda.kda_pages_truncate(pt, _i32([0]), _i32([0]), ws, st)
    kda.kda_pages_compact(pt, cache, ws, st)
    used = int((pt.refcount > 0).sum())
    assert bool((pt.refcount[:used] > 0).all()) and used < 60
    _, q = fresh(3)
    decode([1, 5, 2], [1, 1, 1], q)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
