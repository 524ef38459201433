"""kda_kv_append: rows of the inputs that no sequence has, before the first and behind the last, are not touched."""
import pytest
import torch

import hybrid_linear_attention_decode_gb300 as kda
from tests.kv_testutil import DEV, Pages, check, i32, rotated, status
from tests.test_rope_gpu import make, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu", [[3, 4, 6], [1, 1, 9], [5, 5, 5], [0, 2, 4], [8, 9, 9]])
@pytest.mark.parametrize("dim", [64, 30])
def test_rows_of_no_sequence(cu, dim):
    T, H, kv, d = 9, 4, 2, 64
    p = Pages([20, 33], kv, d, 16, stats=True)
    before, r = p.cache.data.clone(), make(dim)
    x, pos = randn(T, H + 2 * kv, d), i32(list(range(100, 100 + T)))
    qo, st = torch.full((T, H, d), 9.0, dtype=torch.bfloat16, device=DEV), status()
    kda.kda_kv_append(p.cache, 0, p.pt, None, i32(cu), x[:, H:H + kv], x[:, H + kv:], pos, st, rope=r, q=x[:, :H], q_out=qo)
    assert int(st) == 0
    live = slice(cu[0], cu[2])
    ref, tol = rotated(r, x[:, :H], pos)
    check(qo[live], ref[live], tol[live])
    assert bool((qo[:cu[0]] == 9).all()) and bool((qo[cu[2]:] == 9).all())
    keys, ktol = rotated(r, x[:, H:H + kv], pos)
    want = before.clone()
    view = kda.KvCache(want, kv, d, 16, True)
    for b in range(2):
        pid, slot = (t[p.lens[b] - (cu[b + 1] - cu[b]):] for t in p.places(b))
        mine = slice(cu[b], cu[b + 1])
        check(p.cache.keys[0, pid, :, slot], keys[mine], ktol[mine])
        view.keys[0, pid, :, slot] = p.cache.keys[0, pid, :, slot]
        view.values[0, pid, :, slot] = x[mine, H + kv:]
        view.weights[0, pid, :, slot] = 0.0
        view.positions[0, pid, :, slot] = pos[mine, None].expand(-1, kv)
    assert torch.equal(p.cache.data.view(torch.int16), want.view(torch.int16))
