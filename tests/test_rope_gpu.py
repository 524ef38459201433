"""kda_rope_apply and kda_kv_append against 64-bit rotations with exact angles."""
import math

import pytest
import torch

import hybrid_linear_attention_decode_gb300 as kda
from tests.kv_testutil import DEV, F64, Pages, check, cu_of, fraction, i32, rotated, status, unit

pytestmark = pytest.mark.gpu
FAR = [0, 1, 2, 3, 17, -1, -4096, 131071, 1000003, 2 ** 31 - 1, -2 ** 31]


def make(dim, offset=0, interleaved=False, scale=1.0, base=10000.0, **kw):
    return kda.Rope.make(dim, base, offset=offset, interleaved=interleaved, scale=scale, **kw)


def randn(*shape, dtype=torch.bfloat16, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,dim,offset", [
    (1, 1, 8, 2, 0), (11, 3, 16, 16, 0), (11, 1, 64, 64, 0), (11, 32, 192, 64, 128), (5, 7, 80, 32, 8), (5, 5, 24, 6, 9),
    (3, 2, 128, 126, 1), (40, 9, 128, 64, 0), (2, 1024, 32, 32, 0), (1, 2, 1024, 256, 504), (3, 300, 72, 30, 11),
    (700, 33, 128, 128, 0), (3000, 5, 256, 256, 0), (2500, 17, 64, 48, 16)])
def test_apply(dtype, interleaved, T, H, D, dim, offset):
    r = make(dim, offset, interleaved, scale=1.0 if H % 2 else 1.3)
    x = randn(T, H, D, dtype=dtype, seed=T + D)
    pos = i32([FAR[i % len(FAR)] if i < 2 * len(FAR) else 37 * i for i in range(T)])
    ref, tol = rotated(r, x, pos)
    out = torch.full_like(x, float("nan"))
    kda.kda_rope_apply(r, x, pos, out)
    check(out, ref, tol, "out of place")
    y = x.clone()
    kda.kda_rope_apply(r, y, pos, y)
    assert torch.equal(y, out)
    kda.kda_rope_apply(r, x, pos, out, inverse=True)
    check(out, *rotated(r, x, pos, inverse=True), "inverse")


def test_strided_views_and_what_lies_between():
    """The rotary part of latent queries as a view, and heads as a transposed axis; gaps stay as they are."""
    r = make(64, 0, True)
    q = randn(6, 4, 192)
    whole, pos = q.clone(), i32([5, 6, 7, 900, 901, 70000])
    part = q[..., 128:]
    ref, tol = rotated(r, part, pos)
    kda.kda_rope_apply(r, part, pos, part)
    check(q[..., 128:], ref, tol)
    assert torch.equal(q[..., :128], whole[..., :128])
    x = randn(4, 6, 64).transpose(0, 1)  # [6, 4, 64], heads outermost
    wide = torch.full((6, 4, 72), 7.0, dtype=torch.bfloat16, device=DEV)
    kda.kda_rope_apply(r, x, pos, wide[..., :64])
    check(wide[..., :64], *rotated(r, x, pos))
    assert bool((wide[..., 64:] == 7).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_inverse(interleaved):
    """The gradient of sum(w * rotated(x)) is w rotated by -angle (times scale); against the formula's and differences."""
    r = make(32, 16, interleaved, scale=1.25)
    x, w, pos = randn(9, 3, 64, dtype=torch.float16), randn(9, 3, 64, dtype=torch.float16, seed=1), i32(list(range(3, 12)))
    g = torch.empty_like(w)
    kda.kda_rope_apply(r, w, pos, g, inverse=True)

    def f(z):  # in 64 bits, written with complex numbers
        a = torch.polar(torch.full((9, 16), 1.25, dtype=F64, device=DEV), fraction(r.turns, pos))[:, None]
        p = z[..., 16:48]
        pair = torch.complex(p[..., 0::2].contiguous(), p[..., 1::2].contiguous()) if interleaved else torch.complex(
            p[..., :16].contiguous(), p[..., 16:].contiguous())
        t = pair * a
        p = torch.stack([t.real, t.imag], -1).flatten(-2) if interleaved else torch.cat([t.real, t.imag], -1)
        return (w.to(F64) * torch.cat([z[..., :16], p, z[..., 48:]], -1)).sum()

    z = x.to(F64).requires_grad_(True)
    (exact,) = torch.autograd.grad(f(z), z)
    tol = unit(torch.float16) * exact.abs() + 16 * 2.0 ** -24 * 1.25 * 2 * w.abs().max().to(F64)
    check(g, exact, tol + torch.finfo(torch.float16).smallest_normal)
    for t, h, c in ((0, 0, 16), (4, 1, 33), (8, 2, 47), (2, 2, 3)):
        e = torch.zeros_like(z)
        e[t, h, c] = 0.5
        d = (f(x.to(F64) + e) - f(x.to(F64) - e))  # linear in x: the difference is exact up to 64-bit rounding
        assert abs(float(d) - float(g[t, h, c])) <= float(tol[t, h, c]) + 2.0 ** -14


def test_non_finite_values_stay_in_their_pairs():
    r = make(64)
    x, pos = randn(2, 2, 128), i32([3, 4])
    x[0, 0, 5] = float("nan")
    x[1, 1, 100] = float("inf")
    out = torch.empty_like(x)
    kda.kda_rope_apply(r, x, pos, out)
    bad = ~torch.isfinite(out)
    assert torch.nonzero(bad).tolist() == [[0, 0, 5], [0, 0, 37], [1, 1, 100]]


# ------------------------------------------------------------------------------------------------- append
def run_append(p, rope, new, H, dtype, rows=None, seed=3, q_in_place=False, layer=0, extra=0, packed=True, cu=None, st=None):
    T = sum(new) + extra
    kv, d = p.heads, p.d
    x = randn(T, H + 2 * kv, d, dtype=dtype, seed=seed) if packed else None
    q, k, v = ((x[:, :H], x[:, H:H + kv], x[:, H + kv:]) if packed else
               [randn(T, h, d, dtype=dtype, seed=seed + i) for i, h in enumerate((H, kv, kv))])
    pos = i32([(7 * i * i + 11) % 150000 for i in range(T)])
    qo = torch.full((T, H, d), 9.0, dtype=dtype, device=DEV) if H else None
    if q_in_place:
        q = q.contiguous()
        qo, q0 = q, q.clone()
    st = status() if st is None else st
    kda.kda_kv_append(p.cache, layer, p.pt, rows, cu_of(new) if cu is None else cu, k, v, pos, st, rope=rope,
                      q=q if H else None, q_out=qo)
    return (q0 if q_in_place else q), k, v, pos, qo, st


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,H,d,page,dim,offset,interleaved,stats,lens,new", [
    (8, 32, 128, 64, 128, 0, False, True, [5, 64, 65, 1, 200], [1, 1, 1, 1, 1]),
    (8, 32, 128, 16, 64, 0, False, False, [700, 33, 90], [700, 3, 0]),
    (1, 7, 64, 32, 32, 32, True, True, [17, 40], [17, 39]),
    (3, 0, 24, 16, 10, 5, False, True, [40, 16, 1], [33, 16, 1]),
    (2, 2, 256, 128, 256, 0, True, False, [300], [299]),
    (128, 256, 16, 16, 16, 0, False, True, [9, 3], [3, 2]),
    (4, 20, 80, 192, 48, 16, False, True, [500, 191, 193, 4], [7, 190, 2, 0]),
    (8, 8, 96, 64, 96, 0, True, False, [2000, 1500], [1999, 1500]),
    (2, 6, 40, 16, 14, 26, True, True, [100], [100])])
def test_append(dtype, kv, H, d, page, dim, offset, interleaved, stats, lens, new):
    r = make(dim, offset, interleaved, scale=1.1, base=500000.0)
    p = Pages(lens, kv, d, page, stats=stats, dtype=dtype, layers=2, transposed=True)
    before = p.cache.data.clone()
    q, k, v, pos, qo, st = run_append(p, r, new, H, dtype, layer=1, packed=kv != 2)
    assert int(st) == 0
    ref, tol = rotated(r, k, pos)
    if H:
        check(qo, *rotated(r, q, pos), "queries")
    after, at = p.cache.data.clone(), 0
    p.cache.data.copy_(before)
    for b, (n, m) in enumerate(zip(lens, new)):
        j = torch.arange(n - m, n, device=DEV)
        pid, slot = p.pt.table[b].long()[j // page], j % page
        got = kda.KvCache(after, kv, d, page, stats)
        check(got.keys[1, pid, :, slot], ref[at:at + m], tol[at:at + m], "keys")
        assert torch.equal(got.values[1, pid, :, slot], v[at:at + m])
        p.cache.keys[1, pid, :, slot] = got.keys[1, pid, :, slot]
        p.cache.values[1, pid, :, slot] = v[at:at + m]
        if stats:
            p.cache.weights[1, pid, :, slot] = 0
            p.cache.positions[1, pid, :, slot] = pos[at:at + m, None].expand(-1, kv)
        at += m
    assert torch.equal(p.cache.data.view(torch.int16), after.view(torch.int16))  # nothing else was written


def test_append_without_rope_copies():
    p = Pages([20, 3], 2, 64, 16)
    before = p.cache.keys.clone()
    _, k, v, _, _, st = run_append(p, None, [4, 3], 0, torch.bfloat16)
    assert int(st) == 0
    for b, (n, a, m) in enumerate(((20, 0, 4), (3, 4, 3))):
        pid, slot = p.places(b)
        assert torch.equal(p.cache.keys[0, pid[n - m:], :, slot[n - m:]], k[a:a + m])
        assert torch.equal(p.cache.values[0, pid[n - m:], :, slot[n - m:]], v[a:a + m])
        assert torch.equal(p.cache.keys[0, pid[:n - m], :, slot[:n - m]], before[0, pid[:n - m], :, slot[:n - m]])


def test_append_padding_bad_entries_and_rows_behind():
    r = make(64)
    p = Pages([20, 30, 40, 50], 2, 64, 16, stats=True)
    p.pt.table[3, 3] = 99  # tokens 48 and 49 of row 3
    before = p.cache.data.clone()
    # entries: padding, row 1, a row outside, row 3 (with a bad page), more tokens than row 0 has; two tokens behind
    q, k, v, pos, qo, st = run_append(p, r, [2, 3, 1, 4, 21], 4, torch.bfloat16, rows=i32([-1, 1, 7, 3, 0]), extra=2)
    assert int(st) == kda.KDA_DEV_BAD_SLOT | kda.KDA_DEV_BAD_PAGE | kda.KDA_DEV_BAD_SEQLENS
    ref, tol = rotated(r, q, pos)
    check(qo[:31], ref[:31], tol[:31])
    assert bool((qo[31:] == 9).all())
    touched = (p.cache.data.view(torch.int16) != before.view(torch.int16)).any(-1)[0]
    pid, _ = p.places(0)
    want = set(p.pt.table[1, 1:2].tolist()) | {int(p.pt.table[3, 2])} | set(pid.tolist())
    assert set(torch.nonzero(touched)[:, 0].tolist()) == want
    pid, slot = p.places(1)
    check(p.cache.keys[0, pid[27:], :, slot[27:]], *[x[2:5] for x in rotated(r, k, pos)])
    pid, slot = p.pt.table[3, 2].long().expand(2), torch.tensor([14, 15], device=DEV)
    check(p.cache.keys[0, pid, :, slot], *[x[6:8] for x in rotated(r, k, pos)])
    pid, slot = p.places(0)
    check(p.cache.keys[0, pid, :, slot], *[x[11:31] for x in rotated(r, k, pos)])


def test_append_of_flagged_tables_leaves_all():
    p = Pages([20, 30], 2, 64, 16, stats=True)
    before = p.cache.data.clone()
    _, _, _, _, qo, st = run_append(p, make(64), [4, 4], 4, torch.bfloat16, cu=i32([0, 4, 99]))
    assert int(st) == kda.KDA_DEV_BAD_SEQLENS and bool((qo[4:] == 9).all()) and not bool((qo[:4] == 9).any())
    pid, slot = p.places(0)
    before.view(torch.int16)[0, pid[16:].unique()] = p.cache.data.view(torch.int16)[0, pid[16:].unique()]
    assert torch.equal(before.view(torch.int16), p.cache.data.view(torch.int16))


def test_queries_in_place_and_far_rows_of_the_input():
    r = make(64, interleaved=True)
    p = Pages([9, 9], 2, 64, 16)
    q, _, _, pos, qo, st = run_append(p, r, [2, 3], 6, torch.bfloat16, q_in_place=True)
    check(qo, *rotated(r, q, pos))
    # tokens 2^31 elements and more apart
    k = torch.zeros(3, (1 << 30) + 8, dtype=torch.bfloat16, device=DEV)
    k[:, :128] = randn(3, 128)
    view = k[:, :128].unflatten(1, (2, 64))
    st = status()
    kda.kda_kv_append(p.cache, 0, p.pt, None, i32([0, 2, 3]), view, view, i32([4, 5, 6]), st, rope=r)
    ref, tol = rotated(r, view, i32([4, 5, 6]))
    pid, slot = p.places(0)
    check(p.cache.keys[0, pid[7:], :, slot[7:]], ref[:2], tol[:2])
    pid, slot = p.places(1)
    check(p.cache.keys[0, pid[8:], :, slot[8:]], ref[2:], tol[2:])
    assert int(st) == 0


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts"])
def test_scalings_reach_the_kernel(scaling):
    r = make(64, scaling=scaling, factor=8.0, original=4096.0)
    x, pos = randn(4, 2, 64), i32([0, 5000, 32000, 131071])
    w = [10000.0 ** (-2 * i / 64) for i in range(32)]
    if scaling == "linear":
        w = [t / 8 for t in w]
    if scaling == "ntk":
        w = [(10000.0 * 8 ** (64 / 62)) ** (-2 * i / 64) for i in range(32)]
    if scaling == "parts":
        g = [min(1.0, max(0.0, (4096 * t / (2 * math.pi) - 1) / 31)) for t in w]
        w = [a * t + (1 - a) * t / 8 for a, t in zip(g, w)]
    a = pos.to(F64)[:, None, None] * torch.tensor(w, dtype=F64, device=DEV)
    one, two = x[..., :32].to(F64), x[..., 32:].to(F64)
    ref = torch.cat([one * a.cos() - two * a.sin(), two * a.cos() + one * a.sin()], -1)
    out = torch.empty_like(x)
    kda.kda_rope_apply(r, x, pos, out)
    tol = unit(x.dtype) * ref.abs() + (16 * 2.0 ** -24 + 131071 * 2.0 ** -50) * (one.abs() + two.abs()).repeat(1, 1, 2)
    check(out, ref, tol + 2.0 ** -126)
