"""Refusals of the latent attention and page pool calls, without a GPU: every one returns before a CUDA call."""
import ctypes

import pytest
import torch

import hybrid_linear_attention_decode_gb300 as kda

P = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    from hybrid_linear_attention_decode_gb300 import build as kbuild
    kbuild.build()
    return kda.load_library()


def cache(**kw):
    f = dict(rank=512, rope=64, page_size=64, layers=2, dtype=0, reserved=0, num_pages=100,
             layer_stride=100 * 64 * 576, page_stride=64 * 576, pages=P)
    f.update(kw)
    return kda._LatentCache(**f)


def table(**kw):
    f = dict(max_seqs=4, max_pages=10, page_size=64, reserved=0, num_pages=100, table=P, lens=P, refcount=P)
    f.update(kw)
    return kda._PageTable(**f)


def ref(x):
    return None if x is None else ctypes.byref(x)


BAD_CACHE = [(dict(pages=None), 1), (dict(dtype=2), 1), (dict(rank=0), 2), (dict(rank=576), 2), (dict(rank=200), 2),
             (dict(rope=8), 2), (dict(rope=80), 2), (dict(rope=-16), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
             (dict(page_size=0), 2), (dict(page_size=2048), 2), (dict(layers=0), 1), (dict(num_pages=0), 1),
             (dict(num_pages=1 << 40), 1), (dict(pages=P + 8), 1), (dict(page_stride=64 * 576 + 4), 1),
             (dict(page_stride=64 * 576 - 8), 1), (dict(layer_stride=64 * 576), 1), (dict(layer_stride=-8), 1),
             (dict(layer_stride=99 * 64 * 576), 1)]
BAD_TABLE = [dict(table=None), dict(lens=None), dict(max_seqs=0), dict(max_pages=0), dict(num_pages=99),
             dict(page_size=32), dict(table=P + 2), dict(max_pages=1 << 30)]


def decode(lib, c=None, t=None, layer=0, n=2, rows=None, cu=P, T=2, mt=1, H=32, q=P, ts=32 * 576, hs=576, tree=None,
           scale=0.1, out=P, lse=P, ws=P, nbytes=1 << 40, st=P):
    return lib.kda_latent_decode(ref(c or cache()), layer, ref(t or table()), n, rows, cu, T, mt, H, q, ts, hs, tree, scale,
                                 out, lse, ws, nbytes, st, None)


@pytest.mark.parametrize("bad", range(len(BAD_CACHE)))
def test_bad_caches(lib, bad):
    kw, rc = BAD_CACHE[bad]
    c = cache(**kw)
    assert decode(lib, c) == rc and kda.kda_last_error_string()
    assert lib.kda_latent_append(ref(c), 0, ref(table()), 1, None, P, 1, P, 512, P, 64, P, None) == rc
    assert lib.kda_latent_decode_workspace_bytes(ref(c), 32, 1, 1) == 0
    assert lib.kda_pages_copy(ref(c), 1, P, P, P, None) == rc
    for name in ("kda_pages_reserve", "kda_pages_fork"):
        assert getattr(lib, name)(ref(table()), ref(c), 1, P, P, P, 1 << 40, P, None) == rc
    assert lib.kda_pages_compact(ref(table()), ref(c), P, 1 << 40, P, None) == rc


@pytest.mark.parametrize("bad", range(len(BAD_TABLE)))
def test_bad_tables(lib, bad):
    t = table(**BAD_TABLE[bad])
    assert decode(lib, t=t) == 1 and kda.kda_last_error_string()
    assert lib.kda_latent_append(ref(cache()), 0, ref(t), 1, None, P, 1, P, 512, P, 64, P, None) == 1
    assert lib.kda_pages_reserve(ref(t), ref(cache()), 1, P, P, P, 1 << 40, P, None) == 1


@pytest.mark.parametrize("kw,rc", [
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(n=-1), 1), (dict(n=70000), 1), (dict(mt=0), 1), (dict(mt=65), 1),
    (dict(H=0), 1), (dict(H=129), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(cu=None, T=3), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(q=P + 2), 1), (dict(out=P + 8), 1), (dict(ts=4), 1), (dict(ts=-576), 1), (dict(hs=568), 1),
    (dict(tree=P + 4), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(ws=None), 3), (dict(nbytes=0), 3), (dict(ws=P + 8), 3), (dict(lse=P + 2), 1),
    (dict(rows=P + 1), 1), (dict(st=P + 2), 1)])
def test_decode_refuses(lib, kw, rc):
    assert decode(lib, **kw) == rc and kda.kda_last_error_string()


def test_empty_calls_are_ok(lib):
    assert decode(lib, n=0, T=0) == 0 and decode(lib, T=0) == 0
    assert lib.kda_latent_append(ref(cache()), 0, ref(table()), 0, None, None, 0, None, 512, None, 64, None, None) == 0
    assert lib.kda_pages_copy(ref(cache()), 0, None, None, None, None) == 0
    for name in ("kda_pages_reserve", "kda_pages_fork"):
        assert getattr(lib, name)(ref(table()), ref(cache()), 0, None, None, None, 0, None, None) == 0
    assert prefill(lib, nseq=0) == 0 and prefill(lib, num_q=0) == 0 and prefill(lib, max_q=0) == 0


def prefill(lib, dtype=0, H=8, nope=128, rope=64, dv=128, nseq=2, cu_q=P, cu_k=P, num_q=10, num_k=20, max_q=5, q=P,
            qs=(8 * 192, 192), k=P, ks=(8 * 128, 128), r=P, rs=64, v=P, vs=(8 * 128, 128), scale=0.1, out=P, lse=P, st=P):
    return lib.kda_latent_prefill(dtype, H, nope, rope, dv, nseq, cu_q, cu_k, num_q, num_k, max_q, 1, q, *qs, k, *ks, r, rs,
                                  v, *vs, scale, out, lse, st, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=3), 1), (dict(H=0), 1), (dict(H=129), 1), (dict(nope=96), 2), (dict(nope=256), 2), (dict(rope=0), 2),
    (dict(rope=72), 2), (dict(dv=32), 2), (dict(nseq=-1), 1), (dict(num_q=-1), 1), (dict(num_k=1 << 31), 1),
    (dict(max_q=-1), 1), (dict(cu_q=None), 1), (dict(cu_k=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(r=None), 1),
    (dict(v=None), 1), (dict(out=None), 1), (dict(q=P + 8), 1), (dict(v=P + 2), 1), (dict(qs=(8 * 192, 190)), 1),
    (dict(ks=(0, 128)), 1), (dict(rs=-64), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(lse=P + 1), 1),
    (dict(st=P + 1), 1)])
def test_prefill_refuses(lib, kw, rc):
    assert prefill(lib, **kw) == rc and kda.kda_last_error_string()


def test_append_and_pages_refuse(lib):
    def append(layer=0, n=1, cu=P, T=1, lat=P, ls=512, rp=P, rs=64, rows=None):
        return lib.kda_latent_append(ref(cache()), layer, ref(table()), n, rows, cu, T, lat, ls, rp, rs, P, None)
    for kw in (dict(layer=2), dict(n=-1), dict(T=-1), dict(cu=None), dict(lat=None), dict(rp=None), dict(lat=P + 4),
               dict(T=2, ls=504), dict(T=2, rs=60), dict(rows=P + 2)):
        assert append(**kw) == 1, kw
    t, c = table(), cache()
    assert lib.kda_pages_reserve(ref(table(refcount=None)), ref(c), 1, P, P, P, 1 << 40, P, None) == 1
    assert lib.kda_pages_reserve(ref(t), ref(c), -1, P, P, P, 1 << 40, P, None) == 1
    assert lib.kda_pages_reserve(ref(t), ref(c), 1, None, P, P, 1 << 40, P, None) == 1
    assert lib.kda_pages_truncate(ref(t), 1, P, P + 2, P, 1 << 40, P, None) == 1
    need = lib.kda_pages_workspace_bytes(ref(t), 5)
    assert need > 0 and lib.kda_pages_workspace_bytes(ref(t), -1) == 0
    assert lib.kda_pages_fork(ref(t), ref(c), 5, P, P, P, need - 1, P, None) == 3
    assert lib.kda_pages_fork(ref(t), ref(c), 5, P, P, None, need, P, None) == 3
    assert lib.kda_pages_copy(ref(c), 1, None, P, P, None) == 1
    assert lib.kda_pages_copy(ref(c), -1, P, P, P, None) == 1


def test_binding_refuses_cpu_tensors_types_and_shapes(lib):
    c = kda.LatentCache(torch.zeros(1, 4, 16, 144, dtype=torch.bfloat16), 128)
    t = kda.PageTable.empty(2, 3, 4, 16, device="cpu")
    st = torch.zeros(1, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_latent_append(c, 0, t, None, torch.zeros(2, dtype=torch.int32), c.pages[0, 0, :1, :128],
                              c.pages[0, 0, :1, 128:], st)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_pages_copy(c, one, one, st)
    with pytest.raises(TypeError):
        kda.LatentCache(torch.zeros(1, 4, 16, 144), 128).c()
    with pytest.raises(ValueError):
        kda.LatentCache(torch.zeros(1, 4, 144, 16, dtype=torch.float16).transpose(2, 3), 128).c()
    with pytest.raises(ValueError):
        kda.PageTable(t.table, t.lens.long(), t.refcount, 16).c()
    with pytest.raises(ValueError):
        kda._rows_of(torch.zeros(3, 4, dtype=torch.float16), "x", torch.bfloat16, (3, 4))
    with pytest.raises(ValueError):
        kda._rows_of(torch.zeros(4, 3).t(), "x", torch.float32, (3, 4))
    x = torch.zeros(5, 2, 8)[:, :1, :4]
    assert kda._rows_of(x, "x", torch.float32, (5, 1, 4))[1:] == (16, 4)
    assert kda._rows_of(x[:1], "x", torch.float32, (1, 1, 4))[1:] == (4, 4)


def test_limits_of_scales_tokens_and_keys(lib):
    for bad in (1e-31, 1e-45, 2e30):
        assert decode(lib, scale=bad) == 1 and prefill(lib, scale=bad) == 1
    # a table of 2^31 - 64 tokens at most, whatever the page size; too small a workspace is looked at after it
    for size, most in ((16, (1 << 27) - 4), (64, (1 << 25) - 1), (1024, (1 << 21) - 1)):
        c = cache(page_size=size, page_stride=size * 576, layer_stride=100 * size * 576)
        assert decode(lib, c, table(page_size=size, max_pages=most), nbytes=0) == 3
        assert decode(lib, c, table(page_size=size, max_pages=most + 1), nbytes=0) == 1
    assert prefill(lib, num_k=(1 << 31) - 255) == 1 and "num_k" in kda.kda_last_error_string()
    big = dict(H=128, nseq=65535, num_q=1 << 22)
    assert prefill(lib, max_q=2049, **big) == 1 and "2^26" in kda.kda_last_error_string()
    assert prefill(lib, max_q=2048, out=None, **big) == 1 and "2^26" not in kda.kda_last_error_string()


def test_structs_follow_tensors_changed_in_place():
    c = kda.LatentCache(torch.zeros(2, 4, 16, 144, dtype=torch.bfloat16), 128)
    assert (c.c().layers, c.c().num_pages, c.c().layer_stride) == (2, 4, 4 * 16 * 144)
    c.pages.transpose_(0, 1)
    assert (c.c().layers, c.c().num_pages, c.c().layer_stride) == (4, 2, 16 * 144)
    c.rank = 112
    assert (c.c().rank, c.c().rope) == (112, 32)
    t = kda.PageTable.empty(4, 6, 9, 16, device="cpu")
    assert (t.c().max_seqs, t.c().max_pages) == (4, 6)
    t.table.resize_(3, 8)
    t.lens.resize_(3)
    assert (t.c().max_seqs, t.c().max_pages) == (3, 8)
    t.table.resize_(2, 8)
    with pytest.raises(ValueError):
        t.c()
