"""Latent attention where the weights or the scores span the type's range.

Every head has one key of weight 1 whose values are zero and a tail of keys of weight 2^-level, whose values are the whole
output.  Tolerance: that of latent_testutil.attend, and in fp16 the rounding of weights held as multiples of 2^-24 after a
factor 2^9, half a step each: 2^-34 of the largest weight, so 2^-34 sum_j |v_j| of the normalised output at most."""
import math

import pytest
import torch

from tests.latent_testutil import F64, attend, check
from tests.test_latent_gpu import Problem, Prompt

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
LEVELS = [14 + 0.5 * i for i in range(27)]  # 2^-14 .. 2^-27


def extra(values, seen, dtype):
    if dtype is BF:
        return 0.0
    return 2.0 ** -34 * (seen.to(F64) @ values.abs())


def tail(shape, dtype, seed):
    """Values from 500 to 1000, whose sign is the channel's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = 500 + 500 * torch.rand(*shape, generator=g, device="cuda")
    return (v * (1 - 2 * (torch.arange(shape[-1], device="cuda") % 2))).to(dtype)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("count,nq", [(1, 1), (90, 1), (30, 3)])
def test_decode_tail_of_small_weights(dtype, where, count, nq):
    lens = [130, 700, 1500][:count] * (count // 3) if count >= 3 else [3000]
    H, rank = len(LEVELS), 128
    p = Problem(lens, [nq] * len(lens), H=H, rank=rank, rope=64, page=64, dtype=dtype, seed=50, scale=1.0)
    p.pages[..., :rank] = tail((*p.pages.shape[:3], rank), dtype, 51)
    p.pages[..., rank:] = 0
    p.pages[..., rank] = -1
    for b, n in enumerate(lens):
        j = {"first": 0, "middle": n // 2, "last": n - nq}[where]
        p.pages[0, int(p.pt.table[b, j // 64]), j % 64] = 0
    p.q[:] = 0
    p.q[:, :, rank] = (torch.tensor(LEVELS, device="cuda") * math.log(2)).to(dtype)
    p.run()
    c0 = 0
    for b in range(len(lens)):
        kv = p.rows64(b)
        seen = p.seen(b).repeat_interleave(H, 0)
        o, l, to, tl = attend(p.q[c0:c0 + nq].to(F64).reshape(nq * H, -1), kv, kv[:, :rank], seen, 1.0, dtype)
        check(p.out[c0:c0 + nq].reshape(nq * H, rank), o, to + extra(kv[:, :rank], seen, dtype), f"out of sequence {b}")
        check(p.lse[c0:c0 + nq].reshape(nq * H), l, tl, f"lse of sequence {b}")
        c0 += nq


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("at", [0, 400])
@pytest.mark.parametrize("nq,nk,H", [([600, 50], [600, 900], 27), ([600, 300], [600, 900], 108), ([20], [3000], 27)])
def test_prefill_tail_of_small_weights(dtype, at, nq, nk, H):
    p = Prompt(nq, nk, H=H, dtype=dtype, seed=52)
    p.scale = 1.0
    p.q[:] = 0
    level = torch.tensor((LEVELS * 4)[:H], device="cuda")
    p.q[:, :, p.nope] = (level * math.log(2)).to(dtype)
    p.r[:] = 0
    p.r[:, 0] = -1
    p.v.copy_(tail(tuple(p.v.shape), dtype, 53))
    k0 = 0
    for m in nk:
        p.r[k0 + at] = 0
        p.v[k0 + at] = 0
        k0 += m
    p.run()
    q0 = k0 = 0
    for n, m in zip(nq, nk):
        seen = torch.arange(m, device="cuda")[None, :] <= torch.arange(n, device="cuda")[:, None] + (m - n)
        for h in range(0, H, 1 if H == 27 else 5):
            key, v = torch.cat([p.k[k0:k0 + m, h], p.r[k0:k0 + m]], 1).to(F64), p.v[k0:k0 + m, h].to(F64)
            o, l, to, tl = attend(p.q[q0:q0 + n, h].to(F64), key, v, seen, 1.0, dtype)
            check(p.out[q0:q0 + n, h], o, to + extra(v, seen, dtype), f"out, head {h}")
            check(p.lse[q0:q0 + n, h], l, tl, f"lse, head {h}")
        q0 += n
        k0 += m


@pytest.mark.parametrize("dtype", [FP, BF])
def test_scores_whose_fp32_step_is_many_units_of_log2_stay_finite(dtype):
    """Scores of 2^29 and one step (64) above, times scale log2 e = 0.104: the outputs are means of the values all the same."""
    p = Problem([300] * 200, [1] * 200, H=8, rank=128, dtype=dtype, seed=54)
    p.pages[..., 128:] = 0
    p.pages[..., 128] = 2 ** 15
    p.pages[..., 129] = (torch.rand(p.pages.shape[:3], device="cuda") < 0.5).to(dtype)
    for b in range(200):
        p.pages[0, int(p.pt.table[b, 0]), :, 129] = 0
    p.q[:] = 0
    p.q[..., 128] = 2 ** 14
    p.q[..., 129] = 64
    p.run()
    top = p.pages[..., :128].abs().max().to(F64)
    assert bool((p.out.to(F64).abs() <= top * (1 + 2.0 ** -6)).all()) and bool(torch.isfinite(p.lse).all())
    a = Prompt([700], [700], H=2, dtype=dtype, seed=55)
    a.r[:] = 0
    a.r[:, 0] = 2 ** 15
    a.r[128:, 1] = (torch.rand(572, device="cuda") < 0.5).to(dtype)
    a.q[:] = 0
    a.q[..., a.nope] = 2 ** 14
    a.q[..., a.nope + 1] = 64
    a.run()
    top = a.v.abs().max().to(F64)
    assert bool((a.out.to(F64).abs() <= top * (1 + 2.0 ** -6)).all()) and bool(torch.isfinite(a.lse).all())
