"""kda_kv_decode's bound on slots: sums of weights without one are refused, before any CUDA call."""
import pytest

import hybrid_linear_attention_decode_gb300 as kda
from tests.test_kv_abi import cache, decode, lib, ref  # noqa: F401


@pytest.mark.parametrize("n,T", [(1, 1), (2, 2), (65535, 65535)])
def test_sums_need_a_bound(lib, n, T):  # noqa: F811
    """A workspace that was asked for with a bound of 0 has no room for sums."""
    need = lib.kda_kv_decode_workspace_bytes(ref(cache()), 32, n, 1, 0)
    assert need > 0
    for nbytes in (need, 1 << 40):
        assert decode(lib, n=n, T=T, slots=0, add=1, nbytes=nbytes) == 1
        assert "max_slots" in kda.kda_last_error_string()
    # what is missing is the workspace: a bound of 0 is what calls without sums have, and a bound of 1 needs more room
    assert decode(lib, n=n, T=T, slots=0, add=0, nbytes=need - 1) == 3
    assert decode(lib, n=n, T=T, slots=1, add=1, nbytes=need) == 3


def test_empty_calls_need_none(lib):  # noqa: F811
    assert decode(lib, n=0, T=0, slots=0) == 0 and decode(lib, T=0, slots=0) == 0
