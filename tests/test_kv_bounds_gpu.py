"""kda_kv_decode's bound on slots on the GPU: none at all, one that all sequences pass, and workspaces of exactly the size."""
import pytest
import torch

import hybrid_linear_attention_decode_gb300 as kda
from tests.kv_testutil import DEV, Pages, status
from tests.test_kv_gpu import compare, queries

pytestmark = pytest.mark.gpu


def call(p, q, slots, ws, decay=1.0):
    out, lse, st = torch.full_like(q, 5.0), torch.full(q.shape[:2], 5.0, device=DEV), status()
    kda.kda_kv_decode(p.cache, 0, p.pt, None, None, 1, q, out, lse, 0.125, ws, st, weight_decay=decay, max_slots=slots)
    return out, lse, int(st)


@pytest.mark.parametrize("lens", [[0, 0, 0], [40, 0, 100]])
def test_sums_without_a_bound_are_refused(lens):
    p = Pages(lens, 2, 64, 16, stats=True)
    q, before = queries(3, 8, 64, torch.bfloat16), p.cache.data.clone()
    nbytes = kda.kda_kv_decode_workspace_bytes(p.cache, 8, 3, 1, 0)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
    with pytest.raises(kda.KdaError, match="max_slots"):
        call(p, q, 0, ws)
    out, lse, st = call(p, q, 0, ws, decay=None)  # without sums it is what a call has
    compare(p, q, [1, 1, 1], out, lse)
    assert st == 0 and torch.equal(p.cache.data.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("slots", [1, 39, 40, 64, 139, 140, 1000])
@pytest.mark.parametrize("lens", [[0, 0, 0], [40, 0, 100]])
def test_nothing_is_written_behind_the_workspace(lens, slots):
    """Bounds that no, some and all sequences keep, in a workspace of exactly the size; pads on both sides stay as they were."""
    p = Pages(lens, 2, 64, 16, stats=True)
    q, sums = queries(3, 8, 64, torch.bfloat16), p.cache.weights.clone()
    nbytes, pad = kda.kda_kv_decode_workspace_bytes(p.cache, 8, 3, 1, slots), 1 << 20
    room = torch.full((nbytes + 2 * pad,), 0xa5, dtype=torch.uint8, device=DEV)
    out, lse, st = call(p, q, slots, room[pad:pad + nbytes])
    assert bool((room[:pad] == 0xa5).all()) and bool((room[pad + nbytes:] == 0xa5).all())
    compare(p, q, [1, 1, 1], out, lse)
    assert st == (kda.KDA_DEV_BAD_SEQLENS if sum(lens) > slots else 0)
    for b, n in enumerate(lens):
        pid, slot = p.places(b)
        same = torch.equal(p.cache.weights[0, pid, :, slot], sums[0, pid, :, slot])
        assert same == (n == 0 or sum(lens[:b + 1]) > slots)
