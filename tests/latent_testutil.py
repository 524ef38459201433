"""Plain 64-bit forms of latent attention and a plain model of the page pool, shared by the tests."""
import math

import numpy as np
import torch

F64 = torch.float64


def unit(dtype) -> float:
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


def attend(q, keys, values, seen, scale, dtype):
    """q [R, d], keys [n, d], values [n, dv], seen [R, n] bool, all in 64 bits: (out, lse, tol_out, tol_lse).

    Tolerances, from the kernels' arithmetic (u: one rounding to the 16-bit type, e: 2^-24):
      scores   fp32 sums of d products: |ds| <= 4 d e scale sum_k |q_k x_k| (any order of a d-term sum gives d e;
               4 covers the product scale * log2(e) and accumulation that truncates where rounding would do half)
      weights  rounded to the type (u), exp2 to 2^-22, and both numerator and denominator move by ds:
               the weighted sum moves by (u + 2 ds + 2^-20) sum_j p_j |v_j|, fp32 accumulation adds n e of it at most
      output   one rounding, u |out|, and the smallest step of the type
      lse      ds, the logarithm's and exponentials' 2^-20, and 4 e |lse|
    """
    R, n = seen.shape
    dv = values.shape[1]
    if n == 0:
        z = torch.zeros(R, dv, dtype=F64, device=q.device)
        return z, torch.full((R,), -math.inf, dtype=F64, device=q.device), z, torch.zeros(R, dtype=F64, device=q.device)
    s = scale * (q @ keys.t())
    mag = (scale * (q.abs() @ keys.abs().t())).masked_fill(~seen, 0).amax(1)
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m).masked_fill(~seen, 0)
    l = p.sum(1, keepdim=True)
    w = p / torch.where(l == 0, torch.ones_like(l), l)
    out, a = w @ values, w @ values.abs()
    lse = (m + torch.log(l))[:, 0]
    e = 2.0 ** -24
    ds = 4 * q.shape[1] * e * mag
    u = unit(dtype)
    tol = u * out.abs() + (u + 2 * ds[:, None] + 2.0 ** -20 + n * e) * a * 1.01 + torch.finfo(dtype).smallest_normal
    return out, lse, tol, ds + 2.0 ** -20 + 4 * e * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())


def check(got, ref, tol, what=""):
    got = got.to(F64)
    assert torch.equal(torch.isinf(got), torch.isinf(ref)), what
    fin = torch.isfinite(ref)
    bad = ~((got - ref).abs() <= tol)
    bad &= fin
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - ref)[fin].abs().max()),
                                 [tuple(x) for x in torch.nonzero(bad)[:4].tolist()])


class PoolModel:
    """The page pool's rules, one item after another on the host; pages hold tokens' numbers instead of rows."""

    def __init__(self, max_seqs, max_pages, num_pages, ps):
        self.table = np.full((max_seqs, max_pages), -1, np.int32)
        self.lens = np.zeros(max_seqs, np.int32)
        self.ref = np.zeros(num_pages, np.int32)
        self.ps, self.copies, self.bits = ps, [], 0

    def _begin(self):
        self.free = [p for p in range(len(self.ref)) if self.ref[p] <= 0]
        self.taken, self.copies, self.bits, self.old = 0, [], 0, (self.table.copy(), self.lens.copy(), self.ref.copy())

    def _take(self, k):
        """k pages, or None; the demand counts in either case."""
        at = self.taken
        self.taken += k
        if k and self.taken > len(self.free):
            self.bits |= 32
            return None
        return self.free[at:at + k]

    def _named(self, rows, i):
        r = rows[i]
        if r < 0 or r >= len(self.lens) or r in rows[:i]:
            self.bits |= 1
            return False
        return True

    def reserve(self, rows, new_lens):
        self._begin()
        rows = list(rows)
        table, lens, ref = self.old
        for i, (r, nl) in enumerate(zip(rows, new_lens)):
            if r == -1 or not self._named(rows, i):
                continue
            n = int(lens[r])
            if nl < n or nl > self.table.shape[1] * self.ps:
                self.bits |= 2
                continue
            have, want = -(-n // self.ps), -(-nl // self.ps)
            copy = nl > n and n % self.ps != 0 and ref[table[r][have - 1]] > 1
            got = self._take(want - have + copy)
            if got is None:
                continue
            if copy:
                old = int(table[r][have - 1])
                self.copies.append((old, got[0]))
                self.ref[old] -= 1
                self.table[r, have - 1] = got[0]
                self.ref[got[0]] = 1
                got = got[1:]
            for j, p in enumerate(got):
                self.table[r, have + j] = p
                self.ref[p] = 1
            self.lens[r] = nl

    def truncate(self, rows, keep):
        self._begin()
        rows = list(rows)
        for i, (r, k) in enumerate(zip(rows, keep)):
            if r == -1 or not self._named(rows, i):
                continue
            if k < 0 or k > self.old[1][r]:
                self.bits |= 2
                continue
            for j in range(-(-k // self.ps), -(-int(self.old[1][r]) // self.ps)):
                self.ref[self.table[r, j]] -= 1
                self.table[r, j] = -1
            self.lens[r] = k

    def fork(self, parents, children):
        self._begin()
        children = list(children)
        table, lens, _ = self.old
        for i, (p, c) in enumerate(zip(parents, children)):
            if p == -1 or c == -1:
                continue
            if p < 0 or p >= len(self.lens):
                self.bits |= 1
                continue
            if not self._named(children, i):
                continue
            if lens[c] != 0:
                self.bits |= 2
                continue
            n = int(lens[p])
            full = n // self.ps
            got = self._take(int(n % self.ps != 0))
            if got is None:
                continue
            for j in range(full):
                self.table[c, j] = table[p, j]
                self.ref[table[p, j]] += 1
            if got:
                self.table[c, full] = got[0]
                self.ref[got[0]] = 1
                self.copies.append((int(table[p, full]), got[0]))
            self.lens[c] = n

    def compact(self):
        self._begin()
        used = [p for p in range(len(self.ref)) if self.ref[p] > 0]
        k = len(used)
        src = [p for p in used if p >= k]
        dst = [p for p in range(k) if self.ref[p] <= 0]
        to = dict(zip(src, dst))
        self.copies = list(to.items())
        for s, d in self.copies:
            self.ref[d] = self.ref[s]
            self.ref[s] = 0
        for s in range(len(self.lens)):
            for j in range(-(-int(self.lens[s]) // self.ps)):
                self.table[s, j] = to.get(int(self.table[s, j]), int(self.table[s, j]))
