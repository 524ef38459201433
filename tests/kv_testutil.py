"""Plain 64-bit forms of rotary positions, grouped-query attention and eviction, shared by the tests."""
import math

import numpy as np
import torch

import hybrid_linear_attention_decode_gb300 as kda
from tests.latent_testutil import F64, attend, check, unit  # noqa: F401

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cu_of(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]).tolist())


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def fraction(turns, positions):
    """Angles in radians, [T, dim / 2] in 64 bits: whole turns taken out with Python's integers."""
    out = [[((int(p) * (int(t) % (1 << 64))) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for t in turns.tolist()]
           for p in positions.tolist()]
    return torch.tensor(out, dtype=F64, device=positions.device).reshape(len(positions), len(turns))


def rotated(rope, x, positions, inverse=False):
    """x [T, H, D] turned in 64 bits, and how far a kernel may be off.

    With e = 2^-24: the angle is rounded to fp32 as a part of pi (pi e) and the sine and cosine have 2 units in the last
    place (4 e), scaled (e); two products and a sum (3 e): under 16 e of (|x1| + |x2|) scale.  Then one rounding to the type.
    """
    y, mag = x.to(F64).clone(), torch.zeros(x.shape, dtype=F64, device=x.device)
    half = rope.turns.shape[0]
    a = fraction(rope.turns, positions)[:, None] * (-1 if inverse else 1)
    at = torch.arange(half, device=x.device)
    one = rope.offset + (2 * at if rope.interleaved else at)
    two = one + (1 if rope.interleaved else half)
    x1, x2 = y[..., one], y[..., two]
    y[..., one] = (x1 * a.cos() - x2 * a.sin()) * rope.scale
    y[..., two] = (x2 * a.cos() + x1 * a.sin()) * rope.scale
    mag[..., one] = mag[..., two] = (x1.abs() + x2.abs()) * abs(rope.scale)
    tol = torch.where(mag > 0, unit(x.dtype) * y.abs() + 16 * 2.0 ** -24 * mag + torch.finfo(x.dtype).smallest_normal, 0)
    return y, tol


class Pages:
    """A cache and its table, filled at random, and the rows of a sequence."""

    def __init__(self, lens, heads, d, page, stats=False, dtype=torch.bfloat16, layers=1, spare=3, seed=0, max_seqs=None,
                 transposed=False, fill=None):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        num = sum(need) + spare
        words = kda.KvCache.words(page, heads, d, stats)
        shape = (num, layers, words) if transposed else (layers, num, words)
        data = torch.randn(shape, generator=g, device=DEV).to(dtype) if fill is None else torch.full(shape, fill, dtype=dtype,
                                                                                                     device=DEV)
        self.cache = kda.KvCache(data.transpose(0, 1) if transposed else data, heads, d, page, stats)
        rows = max_seqs or max(1, len(lens))
        t = np.full((rows, max([1] + need) + 2), -1, np.int32)
        ref = np.zeros(num, np.int32)
        perm, at = rng.permutation(num), 0
        for b, k in enumerate(need):
            t[b, :k] = perm[at:at + k]
            ref[t[b, :k]] = 1
            at += k
        full = np.zeros(rows, np.int32)
        full[:len(lens)] = lens
        self.pt = kda.PageTable(*[torch.from_numpy(x).cuda() for x in (t, full, ref)], page)
        self.lens, self.page, self.heads, self.d = list(lens), page, heads, d
        if stats:
            self.cache.weights.copy_(torch.rand(self.cache.weights.shape, generator=g, device=DEV))
            self.cache.positions.zero_()

    def places(self, row, n=None):
        """Pages and slots in them of a row's tokens."""
        j = torch.arange(self.lens[row] if n is None else n, device=DEV)
        return self.pt.table[row].long()[j // self.page], j % self.page

    def rows(self, row, layer, head, n=None):
        p, s = self.places(row, n)
        return self.cache.keys[layer, p, head, s].to(F64), self.cache.values[layer, p, head, s].to(F64)

    def poison(self, value=float("nan")):
        """Everything that no row holds becomes `value` (keys and values alone)."""
        held = torch.zeros(self.cache.data.shape[1], self.page, dtype=torch.bool, device=DEV)
        for b in range(len(self.lens)):
            held[self.places(b)] = True
        for x in (self.cache.keys, self.cache.values):
            x.masked_fill_(~held[None, :, None, :, None], value)


def seen_by(nq, n, tree=None):
    """[nq, n] bool: which slots each query sees; tree: bits of drafted tokens by query."""
    seen = torch.ones(nq, n, dtype=torch.bool, device=DEV)
    for t in range(nq):
        for i in range(nq):
            if 0 <= n - nq + i < n:
                seen[t, n - nq + i] = bool((tree[t] >> i) & 1) if tree is not None else i <= t
    return seen


def attention(pages, layer, row, q, scale, tree=None, n=None):
    """q [nq, H, d] of one sequence: out, lse with their tolerances, and the weights [heads, n] with theirs."""
    nq, H, d = q.shape
    G = H // pages.heads
    n = pages.lens[row] if n is None else n
    seen = seen_by(nq, n, tree)
    out = torch.zeros(2, nq, H, d, dtype=F64, device=DEV)
    lse = torch.zeros(2, nq, H, dtype=F64, device=DEV)
    add = torch.zeros(2, pages.heads, n, dtype=F64, device=DEV)
    e = 2.0 ** -24
    for h in range(H):
        k, v = pages.rows(row, layer, h // G, n)
        o, l, to, tl = attend(q[:, h].to(F64), k, v, seen, scale, q.dtype)
        out[0, :, h], lse[0, :, h], out[1, :, h], lse[1, :, h] = o, l, to, tl
        if n:
            s = (scale * (q[:, h].to(F64) @ k.t())).masked_fill(~seen, -math.inf)
            p = torch.exp(s - torch.where(torch.isinf(l), torch.zeros_like(l), l)[:, None])
            add[0, h // G] += p.sum(0)
            # a weight's own score and the row's lse are off by at most tl each; the exponential and the sums add 2^-20
            add[1, h // G] += (p * (2 * tl[:, None] + 2.0 ** -20 + H * nq * e)).sum(0)
    return out, lse, add


def evicted(weights, positions, shared, keep, first=0, since=None):
    """Slots that stay, by the rules: (from, to) pairs of the moves.  weights fp32, positions int, shared bool: numpy [len]."""
    n = len(weights)
    since = 2 ** 31 - 1 if since is None else since
    prot = (positions < first) | (positions >= since) | shared
    w = weights.astype(np.float64)
    order = sorted(range(n), key=lambda j: (not prot[j], 0 if prot[j] else (1 if np.isnan(w[j]) else 0),
                                            0 if prot[j] or np.isnan(w[j]) else -w[j], j))
    kept = set(order[:keep])
    holes = [j for j in range(min(keep, n)) if j not in kept]
    sources = [j for j in range(keep, n) if j in kept]
    assert len(holes) == len(sources)
    return list(zip(sources, holes))
