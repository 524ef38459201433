"""kda_kv_decode: a sequence's results do not depend on what the other sequences of the call hold."""
import pytest
import torch

import hybrid_linear_attention_decode_gb300 as kda
from tests.kv_testutil import DEV, Pages, cu_of, status
from tests.test_kv_gpu import queries

pytestmark = pytest.mark.gpu


def run(p, q, nq, tokens, tree=None, sums=False):
    T, H, d = q.shape
    n, slots = len(nq), sum(p.lens) if sums else 0
    out, lse, st = torch.empty_like(q), torch.empty(T, H, device=DEV), status()
    ws = torch.empty(kda.kda_kv_decode_workspace_bytes(p.cache, H, n, tokens, slots), dtype=torch.uint8, device=DEV)
    was = p.cache.data.clone()
    kda.kda_kv_decode(p.cache, 0, p.pt, None, cu_of(nq), tokens, q, out, lse, d ** -0.5, ws, st, tree_mask=tree,
                      weight_decay=1.0 if sums else None, max_slots=slots)
    added = p.cache.weights.clone() if sums else None
    p.cache.data.copy_(was)
    assert int(st) == 0
    return out, lse, added


# units of 8, 16, 32 and 64 rows, several rows a group, more rows than a unit; heads whose queries stay in registers and not
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,G,d,tokens", [(1, 1, 64, 8), (1, 2, 128, 8), (2, 4, 64, 8), (1, 8, 128, 8), (1, 8, 96, 8), (1, 5, 256, 3),
                                           (1, 16, 192, 4), (1, 40, 64, 3)])
@pytest.mark.parametrize("how", ["large", "infinite", "nan"])
def test_queries_of_others(dtype, kv, G, d, tokens, how):
    """Sequences with the full number of queries and ones with fewer, two by two, so that the rows behind a sequence's last
    query were another one's before it; then other queries for those with the full number.  The others' outputs, log sums and
    sums of weights stay, bit for bit."""
    n = 800 // kv
    nq = [tokens if b % 4 < 2 else 1 + b % (tokens - 1) for b in range(n)]
    lens = [300 + 37 * (b % 11) for b in range(n)]
    p = Pages(lens, kv, d, 64, stats=True, dtype=dtype, seed=d)
    q = queries(sum(nq), kv * G, d, dtype)
    few = torch.cat([torch.full((k,), k < tokens, device=DEV) for k in nq])
    other = q.clone()
    if how == "large":
        other[~few] = (20 * torch.randn(other[~few].shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)).to(dtype)
    else:
        other[~few, :, ::7] = float("inf") if how == "infinite" else float("nan")
    a, b = run(p, q, nq, tokens, sums=True), run(p, other, nq, tokens, sums=True)
    assert torch.equal(a[0][few], b[0][few]) and torch.equal(a[1][few], b[1][few])
    for row in [r for r in range(n) if nq[r] < tokens][::17]:
        pid, slot = p.places(row)
        assert torch.equal(a[2][0, pid, :, slot], b[2][0, pid, :, slot])
    if how == "large":
        assert not torch.equal(a[0][~few], b[0][~few])


def test_keys_and_values_of_others():
    """Pages that a sequence shares a tile's buffers with, and rows behind the end of its last page, hold other things."""
    lens, nq = [1 + 97 * (b % 13) for b in range(700)], [1 + b % 3 for b in range(700)]
    p = Pages([max(a, b) for a, b in zip(lens, nq)], 1, 128, 16, stats=True, seed=7)
    q = queries(sum(nq), 8, 128, torch.bfloat16)
    a = run(p, q, nq, 3, sums=True)
    few = torch.cat([torch.full((k,), b % 2 == 0, device=DEV) for b, k in enumerate(nq)])
    for b in range(1, 700, 2):
        pid, slot = p.places(b)
        p.cache.keys[0, pid, :, slot] *= 30
        p.cache.values[0, pid, :, slot] = float("nan")
    p.poison(float("inf"))
    b = run(p, q, nq, 3, sums=True)
    assert torch.equal(a[0][few], b[0][few]) and torch.equal(a[1][few], b[1][few])
    for row in range(0, 700, 34):
        pid, slot = p.places(row)
        assert torch.equal(a[2][0, pid, :, slot], b[2][0, pid, :, slot])
