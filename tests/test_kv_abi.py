"""Refusals of the key-value attention, eviction and rotary calls, without a GPU: every one returns before a CUDA call."""
import ctypes
import math

import pytest
import torch

import hybrid_linear_attention_decode_gb300 as kda
from tests.test_latent_abi import P, ref, table


@pytest.fixture(scope="module")
def lib():
    from hybrid_linear_attention_decode_gb300 import build as kbuild
    kbuild.build()
    return kda.load_library()


WORDS = 64 * 8 * 260


def cache(**kw):
    f = dict(heads=8, head_dim=128, page_size=64, layers=2, dtype=0, stats=1, num_pages=100, layer_stride=100 * WORDS,
             page_stride=WORDS, pages=P)
    f.update(kw)
    return kda._KvCache(**f)


def rope(**kw):
    f = dict(dim=128, offset=0, interleaved=0, scale=1.0, turns=P)
    f.update(kw)
    return kda._Rope(**f)


def decode(lib, c=None, t=None, layer=0, n=2, rows=None, cu=P, T=2, mt=1, H=32, q=P, ts=32 * 128, hs=128, tree=None,
           scale=0.1, out=P, lse=P, add=1, decay=1.0, slots=1000, ws=P, nbytes=1 << 40, st=P):
    return lib.kda_kv_decode(ref(c or cache()), layer, ref(t or table()), n, rows, cu, T, mt, H, q, ts, hs, tree, scale, out,
                             lse, add, decay, slots, ws, nbytes, st, None)


def append(lib, c=None, t=None, layer=0, n=1, rows=None, cu=P, T=2, k=P, ks=(1024, 128), v=P, vs=(1024, 128), pos=P,
           r=None, H=32, q=P, qs=(4096, 128), qo=P, st=P):
    return lib.kda_kv_append(ref(c or cache()), layer, ref(t or table()), n, rows, cu, T, k, *ks, v, *vs, pos,
                             ref(rope() if r is None else r or None), H, q, *qs, qo, st, None)


def apply(lib, r=None, dtype=0, T=3, H=4, D=192, pos=P, inv=0, x=P, xs=(768, 192), out=P + (1 << 20), os=(768, 192)):
    return lib.kda_rope_apply(ref(r or rope(dim=64, offset=128)), dtype, T, H, D, pos, inv, x, *xs, out, *os, None)


def evict(lib, c=None, t=None, n=2, rows=None, keep=P, first=0, since=None, most=0, new=P, st=P):
    return lib.kda_kv_evict(ref(c or cache()), ref(t or table()), n, rows, keep, first, since, most, new, st, None)


BAD_CACHE = [(dict(pages=None), 1), (dict(dtype=2), 1), (dict(stats=2), 1), (dict(head_dim=8), 2), (dict(head_dim=264), 2),
             (dict(head_dim=100), 2), (dict(heads=0), 2), (dict(heads=129), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
             (dict(page_size=2048), 2), (dict(layers=0), 1), (dict(num_pages=0), 1), (dict(num_pages=1 << 40), 1),
             (dict(pages=P + 8), 1), (dict(page_stride=WORDS + 4), 1), (dict(page_stride=WORDS - 8), 1),
             (dict(layer_stride=WORDS), 1), (dict(layer_stride=-8), 1), (dict(layer_stride=99 * WORDS), 1),
             (dict(page_stride=1 << 40), 1)]


@pytest.mark.parametrize("bad", range(len(BAD_CACHE)))
def test_bad_caches(lib, bad):
    kw, rc = BAD_CACHE[bad]
    c, out = cache(**kw), kda._LatentCache()
    assert decode(lib, c) == rc and kda.kda_last_error_string()
    assert append(lib, c) == rc and evict(lib, c) == rc and lib.kda_kv_cache_pages(ref(c), ref(out)) == rc
    assert lib.kda_kv_decode_workspace_bytes(ref(c), 32, 1, 1, 0) == 0


@pytest.mark.parametrize("kw", [dict(table=None), dict(lens=None), dict(max_seqs=0), dict(max_pages=0), dict(num_pages=99),
                                dict(page_size=32), dict(table=P + 2), dict(max_pages=1 << 30)])
def test_bad_tables(lib, kw):
    t = table(**kw)
    assert decode(lib, t=t) == 1 and append(lib, t=t) == 1 and evict(lib, t=t) == 1 and kda.kda_last_error_string()


@pytest.mark.parametrize("kw,rc", [
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(n=-1), 1), (dict(n=70000), 1), (dict(mt=0), 1), (dict(mt=65), 1),
    (dict(H=0), 1), (dict(H=257), 1), (dict(H=36), 1), (dict(H=264), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1),
    (dict(cu=None, T=3), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(q=P + 2), 1), (dict(out=P + 8), 1), (dict(ts=4), 1),
    (dict(ts=-4096), 1), (dict(hs=120), 1), (dict(tree=P + 4), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=1e31), 1), (dict(decay=1.5), 1), (dict(decay=-0.5), 1),
    (dict(decay=float("nan")), 1), (dict(c=cache(stats=0)), 1), (dict(t=table(refcount=None)), 1), (dict(slots=-1), 1),
    (dict(ws=None), 3), (dict(nbytes=0), 3), (dict(ws=P + 8), 3), (dict(lse=P + 2), 1), (dict(rows=P + 1), 1),
    (dict(st=P + 2), 1)])
def test_decode_refuses(lib, kw, rc):
    assert decode(lib, **kw) == rc and kda.kda_last_error_string()


def test_decode_without_sums_needs_no_stats_or_counts(lib):
    assert decode(lib, c=cache(stats=0), t=table(refcount=None), add=0, nbytes=0) == 3


@pytest.mark.parametrize("kw", [
    dict(layer=2), dict(n=-1), dict(T=-1), dict(cu=None), dict(k=None), dict(v=None), dict(pos=None), dict(k=P + 4),
    dict(v=P + 8), dict(q=P + 2), dict(qo=None), dict(qo=P + 2), dict(ks=(1020, 128)), dict(ks=(120, 128)), dict(vs=(1024, 120)),
    dict(qs=(4096, 64)), dict(H=0), dict(H=1025), dict(r=False), dict(r=rope(dim=0)), dict(r=rope(dim=130)),
    dict(r=rope(dim=64, offset=72)), dict(r=rope(dim=63)), dict(r=rope(offset=-2)), dict(r=rope(interleaved=2)),
    dict(r=rope(scale=0.0)), dict(r=rope(scale=float("nan"))), dict(r=rope(turns=None)), dict(r=rope(turns=P + 4)),
    dict(rows=P + 2), dict(qs=(8192, 128))])
def test_append_refuses(lib, kw):
    assert append(lib, **kw) == 1 and kda.kda_last_error_string()


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=2), 1), (dict(H=0), 2), (dict(H=1025), 2), (dict(D=4), 2), (dict(D=196), 2), (dict(D=2048), 2),
    (dict(r=rope(dim=64, offset=136)), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(pos=None), 1), (dict(x=None), 1),
    (dict(out=None), 1), (dict(x=P + 8), 1), (dict(out=P + 2), 1), (dict(pos=P + 2), 1), (dict(xs=(764, 192)), 1),
    (dict(xs=(184, 192)), 1), (dict(os=(768, 184)), 1), (dict(os=(-768, 192)), 1), (dict(out=P, os=(1536, 192)), 1),
    (dict(xs=(1 << 37, 192)), 1)])
def test_rope_refuses(lib, kw, rc):
    assert apply(lib, **kw) == rc and kda.kda_last_error_string()


@pytest.mark.parametrize("kw", [dict(c=cache(stats=0, page_stride=64 * 8 * 256, layer_stride=100 * 64 * 8 * 256)), dict(n=-1),
                                dict(n=65536), dict(first=-1), dict(most=-1), dict(most=(1 << 20) + 1), dict(keep=None), dict(new=None), dict(keep=P + 2),
                                dict(since=P + 1), dict(rows=P + 2), dict(t=table(refcount=None)), dict(st=P + 3),
                                dict(n=60000, c=cache(layers=200))])
def test_evict_refuses(lib, kw):
    assert evict(lib, **kw) == 1 and kda.kda_last_error_string()


def test_empty_calls_are_ok(lib):
    assert decode(lib, n=0, T=0) == 0 and decode(lib, T=0) == 0
    assert append(lib, n=0) == 0 and append(lib, T=0) == 0 and apply(lib, T=0) == 0 and evict(lib, n=0) == 0


def test_pool_calls_take_the_pages_and_latent_calls_do_not(lib):
    small = cache(heads=1, head_dim=64, stats=0, page_stride=64 * 128, layer_stride=100 * 64 * 128)
    out = kda._LatentCache()
    assert lib.kda_kv_cache_pages(ref(small), ref(out)) == 0 and (out.rank, out.rope) == (128, 0)
    t, need = table(), lib.kda_pages_workspace_bytes(ref(table()), 1)
    assert lib.kda_pages_reserve(ref(t), ref(out), 1, P, P, None, need, P, None) == 3  # only the workspace is missing
    assert lib.kda_latent_append(ref(out), 0, ref(t), 1, None, P, 1, P, 128, None, 0, P, None) == 1
    assert "kda_kv_cache" in kda.kda_last_error_string()
    assert lib.kda_latent_decode_workspace_bytes(ref(out), 4, 1, 1) == 0
    out.rank = 1 << 20
    assert lib.kda_pages_reserve(ref(t), ref(out), 1, P, P, P, need, P, None) == 1


def test_workspace_grows_with_every_size(lib):
    # (its size needs the GPU's number of multiprocessors; without one the fallback is the same for all calls)
    c = cache()
    at = [lib.kda_kv_decode_workspace_bytes(ref(c), *a) for a in
          ((32, 1, 1, 0), (32, 9, 1, 0), (32, 9, 8, 0), (32, 9, 8, 5000), (32, 9, 8, 500000))]
    assert all(x > 0 for x in at) and at == sorted(at)


def test_turns(lib):
    """theta_i against the formulas, to the 2^-52 of a double; whole turns fall out."""
    def theta(**kw):
        return [(int(t) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for t in kda.Rope.make(device="cpu", **kw).turns]
    base = [10000.0 ** (-2 * i / 64) for i in range(32)]

    def close(a, b):
        assert all(abs(x - y) <= 2.0 ** -50 * y + 2.0 ** -60 for x, y in zip(a, b, strict=True))
    close(theta(dim=64, base=10000.0), base)
    close(theta(dim=64, base=10000.0, scaling="linear", factor=8.0), [t / 8 for t in base])
    close(theta(dim=64, base=10000.0, scaling="ntk", factor=8.0), [(10000.0 * 8 ** (64 / 62)) ** (-2 * i / 64) for i in range(32)])
    g = [min(1.0, max(0.0, (4096 * t / (2 * math.pi) - 1) / 31)) for t in base]
    assert 0.0 in g and 1.0 in g and any(0 < x < 1 for x in g)
    close(theta(dim=64, base=10000.0, scaling="parts", factor=8.0, original=4096, low=1.0, high=32.0),
          [x * t + (1 - x) * t / 8 for x, t in zip(g, base)])
    r = kda.Rope.of([0.0, 1.0, 2 * math.pi + 1.0, 7.5], device="cpu")
    got = [(int(t) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for t in r.turns]
    assert got[0] == 0 and all(abs(x - y) < 1e-14 for x, y in zip(got[1:], [1.0, 1.0, 7.5 - 2 * math.pi]))


def test_turns_refuse(lib):
    for kw in (dict(dim=63), dict(dim=0), dict(dim=258), dict(base=0.5), dict(base=float("nan")), dict(factor=0.5, scaling="linear"),
               dict(scaling="ntk", dim=2), dict(scaling="parts"), dict(scaling="parts", original=100.0, low=2.0, high=2.0)):
        with pytest.raises(kda.KdaError):
            kda.Rope.make(**{**dict(dim=64, device="cpu"), **kw})
    with pytest.raises(ValueError):
        kda.Rope.make(64, scaling="cubic", device="cpu")
    for bad in ([-1.0], [float("nan")], [float("inf")], [2.0 ** 20]):
        with pytest.raises(kda.KdaError):
            kda.Rope.of(bad, device="cpu")
    assert lib.kda_rope_turns(64, 10000.0, 4, 1.0, 0.0, 0.0, 0.0, ctypes.c_void_p(P)) == 1
    assert lib.kda_rope_turns(64, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, None) == 1


def test_binding_refuses_cpu_tensors_types_and_shapes(lib):
    c = kda.KvCache.empty(1, 4, 16, 2, 64, stats=True, device="cpu")
    t = kda.PageTable.empty(2, 3, 4, 16, device="cpu")
    one, x = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    r = kda.Rope.make(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_kv_append(c, 0, t, None, torch.zeros(2, dtype=torch.int32), x, x, one, one)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_kv_evict(c, t, None, one, one, one)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_rope_apply(r, x, one, x)
    with pytest.raises(TypeError):
        kda.KvCache(c.data.float(), 2, 64, 16, True).kv()
    with pytest.raises(ValueError):
        kda.KvCache(c.data, 2, 64, 16, False).kv()
    with pytest.raises(ValueError):
        kda.KvCache.empty(1, 4, 16, 2, 64, device="cpu").weights
    with pytest.raises(ValueError):
        kda.Rope(r.turns.float()).c()


def test_views_are_the_pages():
    c = kda.KvCache.empty(2, 3, 16, 4, 24, stats=True, device="cpu")
    c.keys[1, 2, 3, 15, 23] = 1
    c.values[0, 1, 2, 3, 4] = 2
    c.weights[1, 0, 3, 5] = 0.5
    c.positions[1, 0, 3, 6] = -7
    size = 4 * 16 * 24
    assert c.data[1, 2, size - 1] == 1 and c.data[0, 1, size + (2 * 16 + 3) * 24 + 4] == 2
    words = c.data.view(torch.int32)
    assert words[1, 0, size + 3 * 32 + 16 + 6] == -7
    assert c.data.view(torch.float32)[1, 0, size + 3 * 32 + 5] == 0.5
    assert int((c.data != 0).sum()) == 2 + 1 + 2  # 0.5 has one word that is not zero, -7 two
    key = c.kv()
    assert key is c.kv() and (key.layers, key.num_pages) == (2, 3)
    c.data.transpose_(0, 1)
    assert (c.kv().layers, c.kv().num_pages) == (3, 2) and c.c().rank == 4 * 52


def test_rope_notices_strides():
    turns = torch.arange(64)
    r = kda.Rope(turns[:16])
    assert r.c().dim == 32 and r.c() is r.c()
    r.turns = turns[::2][:16]  # the same address and shape
    with pytest.raises(ValueError, match="contiguous"):
        r.c()
