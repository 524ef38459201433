"""Counts and strides so large that an index or a product would wrap around are refused, before any CUDA call."""
import pytest

import hybrid_linear_attention_decode_gb300 as kda
from tests.test_latent_abi import P, cache, decode, prefill, ref, table

BIG, MOST = (1 << 31) - 1, 1 << 30


@pytest.fixture(scope="module")
def lib():
    from hybrid_linear_attention_decode_gb300 import build as kbuild
    kbuild.build()
    return kda.load_library()


def append(lib, c=None, t=None, n=1, T=1, ls=512, rs=64):
    return lib.kda_latent_append(ref(c or cache()), 0, ref(t or table()), n, None, P, T, P, ls, P, rs, P, None)


def test_overlapping_pages_are_refused_where_their_extent_passes_64_bits(lib):
    """(num_pages - 1) * page_stride is 2^64 here; layers and pages at the same stride overlap."""
    num, far = (1 << 28) + 1, 1 << 36
    c, t = cache(num_pages=num, page_stride=far, layer_stride=far), table(num_pages=num)
    assert decode(lib, c, t, nbytes=0) == 1 and "latent cache" in kda.kda_last_error_string()
    assert append(lib, c, t) == 1
    assert lib.kda_pages_compact(ref(t), ref(c), P, 0, P, None) == 1
    assert lib.kda_latent_decode_workspace_bytes(ref(c), 32, 1, 1) == 0
    # a layout of 2^44 elements is looked at further: what is missing is the workspace
    c = cache(layers=1, num_pages=(1 << 8) + 1, page_stride=far, layer_stride=0)
    assert decode(lib, c, table(num_pages=257), nbytes=0) == 3
    c = cache(layers=1, num_pages=(1 << 8) + 2, page_stride=far, layer_stride=0)
    assert decode(lib, c, table(num_pages=258), nbytes=0) == 1


def test_items_and_table_rows_whose_indices_would_wrap_are_refused(lib):
    c, t = cache(), table()
    for n in (BIG, MOST + 1):
        assert append(lib, n=n) == 1 and "n or num_tokens" in kda.kda_last_error_string()
        for name in ("kda_pages_reserve", "kda_pages_fork"):
            assert getattr(lib, name)(ref(t), ref(c), n, P, P, P, 0, P, None) == 1, name
        assert lib.kda_pages_truncate(ref(t), n, P, P, P, 0, P, None) == 1
        assert lib.kda_pages_copy(ref(c), n, P, P, P, None) == 1
        assert lib.kda_pages_workspace_bytes(ref(t), n) == 0
        wide = table(max_seqs=n)
        assert lib.kda_pages_compact(ref(wide), ref(c), P, 0, P, None) == 1
        assert lib.kda_pages_workspace_bytes(ref(wide), 1) == 0
        assert decode(lib, t=wide, nbytes=0) == 1 and append(lib, t=wide) == 1
    assert lib.kda_pages_truncate(ref(t), MOST, P, P, P, 0, P, None) == 3
    assert lib.kda_pages_workspace_bytes(ref(table(max_seqs=MOST)), MOST) > 0


def test_strides_that_reach_too_far_are_refused(lib):
    far = 1 << 36
    T = (1 << 28) + 1
    assert append(lib, T=T, ls=far) == 1 and append(lib, T=T, rs=far) == 1
    assert decode(lib, n=1 << 15, cu=P, T=T, ts=far) == 1 and "strides" in kda.kda_last_error_string()
    assert decode(lib, H=128, T=2, ts=8, hs=far, nbytes=0) == 3    # 127 * 2^36 is below 2^44
    for kw in (dict(num_q=T, qs=(far, 192)), dict(num_k=T, ks=(far, 128)), dict(num_k=T, rs=far), dict(num_k=T, vs=(far, 128))):
        assert prefill(lib, **kw) == 1 and "strides" in kda.kda_last_error_string(), kw
