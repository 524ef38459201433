"""Grouped-query attention over the paged cache as a serving program calls it, with plain forms to measure against.

A page holds keys and values of `page` tokens for every key-value head and, where the program evicts, two more numbers
for each token and head: its accumulated attention weight and its position.

  rope    rotary positions of queries, keys or latent rows: half or interleaved, part of the head, scaled
  append  new tokens' keys (rotated on the way) and values into their pages, their queries rotated beside
  decode  attention of the newest tokens over the pages: one a sequence, or drafted chains and trees; optionally
          each cached token's weight is added to its sum
  evict   each head keeps the tokens with the largest sums; they move to the front, the rest can be truncated

`own` false computes them with elementary torch operations, true calls the package's kernels.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a lone chat in its first thousand tokens: latency counts
        dict(name="kv_decode_one", op="decode", n=1, heads=32, kv=8, d=128, page=64, lo=1013, hi=1013, tokens=1,
             tree=False, weigh=False, dtype="bf16", lens_seed=1),
        # the decode batch of the framework's own benchmark, ragged lengths
        dict(name="kv_decode_batch64", op="decode", n=64, heads=32, kv=8, d=128, page=64, lo=500, hi=8192, tokens=1,
             tree=False, weigh=False, dtype="bf16", lens_seed=2),
        # few sequences with very long contexts, few key-value heads: the split over the length
        dict(name="kv_decode_long", op="decode", n=3, heads=32, kv=4, d=128, page=128, lo=60000, hi=131072, tokens=1,
             tree=False, weigh=False, dtype="bf16", lens_seed=3),
        # verification of drafted trees of up to 5 tokens, small pages
        dict(name="kv_decode_tree", op="decode", n=16, heads=32, kv=8, d=128, page=16, lo=2000, hi=16384, tokens=5,
             tree=True, weigh=False, dtype="fp16", lens_seed=4),
        # a batch that keeps its caches short: every step adds up the weights
        dict(name="kv_decode_weights", op="decode", n=48, heads=64, kv=8, d=64, page=32, lo=1000, hi=4200, tokens=1,
             tree=False, weigh=True, dtype="bf16", lens_seed=5),
        # rotary parts of latent attention's queries, one token for each of 64 sequences at far positions
        dict(name="rope_latent_step", op="rope", tokens=64, heads=32, d=192, dim=64, offset=128, interleaved=True,
             scaling="parts", factor=32.0, theta=10000.0, original=4096, far=131072, dtype="bf16"),
        # queries of the four-sequence prefill workload, whole heads in the half layout
        dict(name="rope_prompts", op="rope", tokens=22528, heads=32, d=128, dim=128, offset=0, interleaved=False,
             scaling="none", factor=1.0, theta=500000.0, original=8192, far=8192, dtype="bf16"),
        # one new token for each of 256 sequences: query, key and value of one projection
        dict(name="kv_append_step", op="append", n=256, heads=32, kv=8, d=128, page=64, lo=1, hi=1, past=700,
             dim=128, offset=0, interleaved=False, scaling="none", factor=1.0, theta=500000.0, original=8192,
             stats=True, dtype="bf16", lens_seed=8),
        # the prompts of the prefill workload
        dict(name="kv_append_prompts", op="append", n=4, heads=32, kv=8, d=128, page=64, lo=2000, hi=8192, past=300,
             dim=64, offset=0, interleaved=False, scaling="ntk", factor=4.0, theta=10000.0, original=8192,
             stats=False, dtype="fp16", lens_seed=9),
        # a running batch that is brought back to its budget every few steps
        dict(name="kv_evict_step", op="evict", n=64, kv=8, d=128, page=64, layers=4, lo=2049, hi=2112, keep=2048,
             first=4, recent=64, dtype="bf16", lens_seed=10),
        # prompts cut to their heavy tokens after prefill
        dict(name="kv_evict_prompts", op="evict", n=6, kv=8, d=128, page=64, layers=8, lo=2000, hi=8192, keep=1024,
             first=4, recent=128, dtype="bf16", lens_seed=11),
        # one long context cut to a sixteenth, few heads: the selection itself
        dict(name="kv_evict_long", op="evict", n=1, kv=4, d=128, page=128, layers=2, lo=120000, hi=131072, keep=8192,
             first=4, recent=1024, dtype="bf16", lens_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng, d):
    dim = rng.choice([d, d, d // 2])
    scaling, factor = rng.choice([("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("parts", 16.0)])
    return dict(dim=dim, offset=rng.choice([0, d - dim]), interleaved=rng.random() < 0.5, scaling=scaling, factor=factor,
                theta=rng.choice([10000.0, 500000.0]), original=rng.choice([2048, 4096, 8192]))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "rope", "append", "evict", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    seed = rng.randrange(1 << 30)
    d = rng.choice([64, 128, 128, 256, 96])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if op == "decode":
        n = _log(rng, 1, 96)
        tokens = rng.choice([1, 1, 1, 2, 5, 8])
        hi = _log(rng, 40, max(41, min(100000, 200000 * 8 * 128 // (n * kv * d))))
        return dict(op=op, n=n, heads=kv * group, kv=kv, d=d, page=page, lo=max(tokens, hi // rng.choice([1, 2, 8])),
                    hi=hi, tokens=tokens, tree=tokens > 1 and rng.random() < 0.6, weigh=rng.random() < 0.3,
                    dtype=dtype, lens_seed=seed)
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 12000), heads=kv * rng.choice([1, 2, 5, 8]) if d < 256 else kv, d=d,
                    far=rng.choice([100, 8192, 131072, 1000000]), dtype=dtype, **_draw_rope(rng, d))
    if op == "append":
        n = _log(rng, 1, 200)
        hi = _log(rng, 1, max(2, 8000 // n))
        return dict(op=op, n=n, heads=kv * min(group, 8), kv=kv, d=d, page=page, lo=max(1, hi // 2), hi=hi,
                    past=_log(rng, 1, 900), stats=rng.random() < 0.5, dtype=dtype, lens_seed=seed, **_draw_rope(rng, d))
    n = _log(rng, 1, 40)
    layers = rng.choice([1, 2, 3])
    hi = _log(rng, 30, max(31, min(60000, 400000 * 8 // (n * kv * layers))))
    return dict(op=op, n=n, kv=kv, d=d, page=page, layers=layers, lo=max(1, hi // rng.choice([1, 3])), hi=hi,
                keep=max(1, hi // rng.choice([2, 5, 16])), first=rng.choice([0, 1, 4]), recent=rng.choice([0, 1, 32]),
                dtype=dtype, lens_seed=seed)


def _new_lens(case):
    """Tokens that the call brings, by sequence."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "decode":
        r.random()
        return [r.randint(max(1, case["tokens"] - 3), case["tokens"]) if case["tree"] else case["tokens"]
                for _ in range(case["n"])]
    if case["hi"] == 8192 and case["n"] == 4:  # the prefill workload's prompts
        return [2048, 4096, 8192, 8192]
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


def _total_lens(case):
    """Tokens of each sequence, those that the call brings among them."""
    r = random.Random(case["lens_seed"] + 1)
    if case["op"] in ("decode", "evict"):
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    return [k + r.randint(case["past"] // 2, case["past"]) for k in _new_lens(case)]


def _pages_of(lens, page):
    return [-(-x // page) for x in lens]


def _has_stats(case):
    return case["op"] == "evict" or case.get("weigh", False) or case.get("stats", False)


# ---------------------------------------------------------------------------------------------------- inputs
def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _inv_freq(case):
    """Radians a position for each pair, in 64 bits."""
    dim, f = case["dim"], case["factor"]
    base = case["theta"] * f ** (dim / (dim - 2)) if case["scaling"] == "ntk" else case["theta"]
    w = torch.tensor([base ** (-2.0 * i / dim) for i in range(dim // 2)], dtype=torch.float64)
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "parts":
        g = ((case["original"] * w / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        w = w / f * (1 - g) + w * g
    return w


def _rope_scale(case):
    """What a program that scales by parts multiplies rotated values with."""
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def _parts(data, case):
    """Views of the pages: keys, values [layers, pages, kv, page, d], and the stats' words [layers, pages, kv, 2, page]."""
    layers, num, _ = data.shape
    kv, page, d = case["kv"], case["page"], case["d"]
    size = kv * page * d
    k, v = (data[..., i * size:(i + 1) * size].view(layers, num, kv, page, d) for i in (0, 1))
    if not _has_stats(case):
        return k, v, None
    return k, v, data.view(torch.int32)[..., size:].view(layers, num, kv, 2, page)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        x = torch.empty(*shape, dtype=dt, device="cuda")
        for part in x.view(-1).split(1 << 28):
            part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
        return x

    s = dict(case=dict(case))
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] in ("rope", "append"):
        s["inv_freq"] = _inv_freq(case).cuda()
        s["mult"] = _rope_scale(case)
        if own:
            import hybrid_linear_attention_decode_gb300 as kda
            s["rope"] = kda.Rope.make(case["dim"], case["theta"], offset=case["offset"], interleaved=case["interleaved"],
                                      scaling=case["scaling"], factor=case["factor"], original=case["original"],
                                      low=1.0, high=32.0, scale=s["mult"])
    if case["op"] == "rope":
        x = randn(case["tokens"], case["heads"], case["d"])
        pos = rng.integers(0, case["far"], case["tokens"])
        s.update(x=x, out=torch.empty_like(x), pos=torch.from_numpy(pos.astype(np.int32)).cuda())
        return s
    lens, page, layers = _total_lens(case), case["page"], case.get("layers", 1)
    H, kv, d = case.get("heads", 0), case["kv"], case["d"]
    pages = _pages_of(lens, page)
    num = sum(pages) + 8
    stats = _has_stats(case)
    data = randn(layers, num, kv * page * (2 * d + (4 if stats else 0)))
    perm = rng.permutation(num)
    t = np.full((len(lens), max(pages) + 2), -1, dtype=np.int32)
    ref = np.zeros(num, dtype=np.int32)
    ends = np.cumsum(pages)
    for i, k in enumerate(pages):
        t[i, :k] = perm[ends[i] - k:ends[i]]
    ref[perm[:ends[-1]]] = 1
    s["table"], s["ref"] = torch.from_numpy(t).cuda(), torch.from_numpy(ref).cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s.update(lens_h=lens, data=data)
    s["keys"], s["values"], s["words"] = _parts(data, case)
    if stats:
        # sums of a running program: most tokens little, some much, the newest nothing yet
        w = torch.exp(2 * torch.randn(layers, num, kv, page, generator=g, device="cuda"))
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.05] = 0
        s["words"][:, :, :, 0] = w.view(torch.int32)
        s["words"][:, :, :, 1] = 0
    if case["op"] == "decode":
        nq = _new_lens(case)
        tq = sum(nq)
        s.update(nq=nq, cu_q=_cu(nq), q=randn(tq, H, d), scale=1.0 / math.sqrt(d),
                 out=torch.empty(tq, H, d, dtype=dt, device="cuda"),
                 lse=torch.empty(tq, H, dtype=torch.float32, device="cuda"), tree=None)
        if case["tree"]:
            r = random.Random(seed)
            rows = []
            for k in nq:
                anc = []
                for j in range(k):
                    p = r.randint(-1, j - 1) if j else -1
                    anc.append((anc[p] if p >= 0 else 0) | (1 << j))
                rows += anc
            s["tree"] = torch.tensor(rows, dtype=torch.int64, device="cuda")
    elif case["op"] == "append":
        new = _new_lens(case)
        tq = sum(new)
        x = randn(tq, H + 2 * kv, d)  # one projection's output
        pos = np.concatenate([np.arange(a - k, a) for a, k in zip(lens, new)])
        s.update(nq=new, cu_q=_cu(new), q=x[:, :H], k=x[:, H:H + kv], v=x[:, H + kv:],
                 q_out=torch.empty(tq, H, d, dtype=dt, device="cuda"),
                 pos=torch.from_numpy(pos.astype(np.int32)).cuda())
    else:
        # positions in the order that earlier evictions left
        for b, n in enumerate(lens):
            p = torch.from_numpy(rng.permutation(pages[b] * page).astype(np.int32)).cuda()
            s["words"][:, s["table"][b, :pages[b]].long(), :, 1] = p.view(1, pages[b], 1, page)
        s.update(keep=torch.full((len(lens),), case["keep"], dtype=torch.int32, device="cuda"),
                 since=s["lens"] - case["recent"], new_lens=torch.empty_like(s["lens"]))
    if stats and case["op"] != "append":
        s["kept"] = s["words"].clone()
    if own:
        import hybrid_linear_attention_decode_gb300 as kda
        s["cache"] = kda.KvCache(data, kv, d, page, stats)
        s["pt"] = kda.PageTable(s["table"], s["lens"], s["ref"], page)
        if case["op"] == "decode":
            nbytes = kda.kda_kv_decode_workspace_bytes(s["cache"], H, case["n"], max(s["nq"]),
                                                       num * page if case["weigh"] else 0)
            s["ws"] = torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if "kept" in s:  # the sums (and positions) as they were before the first pass
        s["words"].copy_(s["kept"])
    if own:
        return {"decode": _own_decode, "rope": _own_rope, "append": _own_append, "evict": _own_evict}[op](s)
    return {"decode": _plain_decode, "rope": _plain_rope, "append": _plain_append, "evict": _plain_evict}[op](s)


def _outputs(s):
    """The pages whole: keys, values, sums and positions."""
    w = s["words"]
    return [s["keys"], s["values"]] + ([] if w is None else [w[:, :, :, 0].view(torch.float32), w[:, :, :, 1]])


def _own_decode(s):
    import hybrid_linear_attention_decode_gb300 as kda
    kda.kda_kv_decode(s["cache"], 0, s["pt"], None, s["cu_q"], max(s["nq"]), s["q"], s["out"], s["lse"], s["scale"],
                      s["ws"], s["status"], tree_mask=s["tree"], weight_decay=1.0 if s["case"]["weigh"] else None)
    return [s["out"], s["lse"]] + ([s["words"][:, :, :, 0].view(torch.float32)] if s["case"]["weigh"] else [])


def _own_rope(s):
    import hybrid_linear_attention_decode_gb300 as kda
    kda.kda_rope_apply(s["rope"], s["x"], s["pos"], s["out"])
    return s["out"]


def _own_append(s):
    import hybrid_linear_attention_decode_gb300 as kda
    kda.kda_kv_append(s["cache"], 0, s["pt"], None, s["cu_q"], s["k"], s["v"], s["pos"], s["status"], rope=s["rope"],
                      q=s["q"], q_out=s["q_out"])
    return _outputs(s) + [s["q_out"]]


def _own_evict(s):
    import hybrid_linear_attention_decode_gb300 as kda
    kda.kda_kv_evict(s["cache"], s["pt"], None, s["keep"], s["new_lens"], s["status"], first=s["case"]["first"],
                     since=s["since"])
    return _outputs(s) + [s["new_lens"]]


def _plain_decode(s):
    c, at = s["case"], 0
    H, kv, page, d = c["heads"], c["kv"], c["page"], c["d"]
    G = H // kv
    out, lse = s["out"], s["lse"]
    for b, (n, k) in enumerate(zip(s["lens_h"], s["nq"])):
        ids = s["table"][b, :-(-n // page)].long()
        keys, vals = (x[0][ids].transpose(0, 1).reshape(kv, -1, d)[:, :n].float() for x in (s["keys"], s["values"]))
        q = s["q"][at:at + k].float().reshape(k, kv, G, d).permute(1, 0, 2, 3).reshape(kv, k * G, d)
        x = torch.matmul(q, keys.transpose(1, 2)) * s["scale"]
        if k > 1:
            j = torch.arange(k, device="cuda")
            if s["tree"] is not None:
                seen = (s["tree"][at:at + k, None] >> j[None, :]) & 1 == 1
            else:
                seen = j[None, :] <= j[:, None]
            x[:, :, n - k:] = x[:, :, n - k:].masked_fill(~seen.repeat_interleave(G, 0)[None], float("-inf"))
        m = x.amax(dim=-1, keepdim=True)
        p = torch.exp(x - m)
        z = p.sum(dim=-1, keepdim=True)
        p = p / z
        o = torch.matmul(p, vals)
        out[at:at + k] = o.reshape(kv, k, G, d).transpose(0, 1).reshape(k, H, d).to(out.dtype)
        lse[at:at + k] = (m + torch.log(z)).reshape(kv, k, G).transpose(0, 1).reshape(k, H)
        if c["weigh"]:
            w = torch.zeros(kv, len(ids) * page, device="cuda")
            w[:, :n] = p.sum(dim=1)
            sums = s["words"][0, :, :, 0].view(torch.float32)
            sums[ids] += w.view(kv, len(ids), page).transpose(0, 1)
        at += k
    return [out, lse] + ([s["words"][:, :, :, 0].view(torch.float32)] if c["weigh"] else [])


def _plain_rotate(s, x):
    """x [T, H, d] rotated by its tokens' angles, in its type."""
    c = s["case"]
    a = s["pos"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = ((f(a) * s["mult"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    y = x.float().clone()
    r = y[..., c["offset"]:c["offset"] + c["dim"]]
    half = c["dim"] // 2
    one, two = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
    a, b = one * cos - two * sin, two * cos + one * sin
    one.copy_(a)
    two.copy_(b)
    return y.to(x.dtype)


def _plain_rope(s):
    s["out"].copy_(_plain_rotate(s, s["x"]))
    return s["out"]


def _plain_append(s):
    c = s["case"]
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
    slot = s["lens"].long()[b] - (s["cu_q"].long()[b + 1] - t)
    pid, row = s["table"][b, slot // c["page"]].long(), slot % c["page"]
    s["keys"][0][pid, :, row] = _plain_rotate(s, s["k"])
    s["values"][0][pid, :, row] = s["v"]
    if s["words"] is not None:
        s["words"][0][pid, :, 0, row] = 0
        s["words"][0][pid, :, 1, row] = s["pos"][:, None].expand(-1, c["kv"])
    s["q_out"].copy_(_plain_rotate(s, s["q"]))
    return _outputs(s) + [s["q_out"]]


def _plain_evict(s):
    c = s["case"]
    kv, page, d, layers = c["kv"], c["page"], c["d"], c["layers"]
    units = layers * kv
    for b, n in enumerate(s["lens_h"]):
        keep = min(c["keep"], n)
        s["new_lens"][b] = keep
        if keep == n:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        words = s["words"][:, ids]                                       # [layers, pages, kv, 2, page]
        words = words.permute(0, 2, 3, 1, 4).reshape(units, 2, -1)[..., :n]
        pos = words[:, 1]
        rank = words[:, 0].long()                                        # sums are not negative: ordered as their bits
        rank = torch.where((pos < c["first"]) | (pos >= s["since"][b]), torch.full_like(rank, 1 << 32), rank)
        order = rank * (1 << 24) + ((1 << 24) - 1 - torch.arange(n, device="cuda"))
        least = order.sort(dim=1, descending=True).values[:, keep - 1:keep]
        chosen = order >= least
        unit, hole = torch.nonzero(~chosen[:, :keep], as_tuple=True)
        _, source = torch.nonzero(chosen[:, keep:], as_tuple=True)       # as many in each unit, in the same order
        source = source + keep
        l, h = unit // kv, unit % kv
        src, dst = (l, ids[source // page], h, source % page), (l, ids[hole // page], h, hole % page)
        for x in (s["keys"], s["values"]):
            x[dst] = x[src]
        w = s["words"].transpose(3, 4)
        w[dst] = w[src]
    return _outputs(s) + [s["new_lens"]]


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        return {"bytes": case["tokens"] * (4 * case["heads"] * case["d"] + 4),
                "flops": 3 * case["tokens"] * case["heads"] * case["dim"]}
    lens, kv, d = _total_lens(case), case["kv"], case["d"]
    if op == "append":
        t, H = sum(_new_lens(case)), case["heads"]
        return {"bytes": t * (4 * (H + 2 * kv) * d + 4 + (8 * kv if case["stats"] else 0)),
                "flops": 3 * t * (H + kv) * case["dim"]}
    if op == "decode":
        new, H = _new_lens(case), case["heads"]
        tq = sum(new)
        seen = sum(k * n - k * (k - 1) // 2 for n, k in zip(lens, new))
        return {"bytes": sum(lens) * kv * (4 * d + (8 if case["weigh"] else 0)) + tq * H * (4 * d + 4),
                "flops": 4 * H * seen * d}
    units, moved = case["layers"] * kv, 0
    for n in lens:
        keep = min(case["keep"], n)
        # with the kept tokens spread evenly, this share of them lies behind the first `keep` slots
        moved += keep * (n - keep) // n
    return {"bytes": units * (8 * sum(lens) + 2 * moved * (4 * d + 8)), "flops": 0}


# ---------------------------------------------------------------------------------------------------- in 64 bits
def _turned(case, x, pos):
    """x [T, H, d] with each pair multiplied, as a complex number, by scale * exp(i angle)."""
    y = x.to(torch.float64)
    lo, dim = case["offset"], case["dim"]
    part = y[..., lo:lo + dim]
    angle = torch.outer(pos.to(torch.float64), _inv_freq(case).to(x.device))
    factor = torch.polar(torch.full_like(angle, _rope_scale(case)), angle)[:, None]
    if case["interleaved"]:
        z = torch.view_as_complex(part.reshape(*part.shape[:-1], dim // 2, 2).contiguous()) * factor
        y[..., lo:lo + dim] = torch.view_as_real(z).reshape(part.shape)
    else:
        z = torch.complex(part[..., :dim // 2].contiguous(), part[..., dim // 2:].contiguous()) * factor
        y[..., lo:lo + dim] = torch.cat([z.real, z.imag], dim=-1)
    return y


def exact(case, seed):
    """Rotations and attention from their definitions in 64 bits; what only moves has no such value."""
    if case["op"] == "evict":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(case, s["x"], s["pos"])
    f64 = torch.float64
    if case["op"] == "append":
        keys = s["keys"].to(f64)
        rows, at = _turned(case, s["k"], s["pos"]), 0
        for b, (n, k) in enumerate(zip(s["lens_h"], s["nq"])):
            slot = torch.arange(n - k, n, device="cuda")
            keys[0, s["table"][b].long()[slot // case["page"]], :, slot % case["page"]] = rows[at:at + k]
            at += k
        return [keys, None] + ([None, None] if case["stats"] else []) + [_turned(case, s["q"], s["pos"])]
    if work(case)["flops"] > 4e12:
        return None
    H, kv, page = case["heads"], case["kv"], case["page"]
    out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=f64, device="cuda")
    sums = s["words"][:, :, :, 0].view(torch.float32).to(f64) if case["weigh"] else None
    t0 = 0
    for b, k in enumerate(s["nq"]):
        n = s["lens_h"][b]
        slot = torch.arange(n, device="cuda")
        where, row = s["table"][b].long()[slot // page], slot % page
        for h in range(kv):
            key, val = s["keys"][0, where, h, row].to(f64), s["values"][0, where, h, row].to(f64)
            mine = slice(h * (H // kv), (h + 1) * (H // kv))
            for t in range(k):
                logits = s["scale"] * (key @ s["q"][t0 + t, mine].to(f64).t())          # [slots, group]
                for j in range(k):
                    if not ((int(s["tree"][t0 + t]) >> j) & 1 if s["tree"] is not None else j <= t):
                        logits[n - k + j] = -math.inf
                total = torch.logsumexp(logits, dim=0)
                share = torch.exp(logits - total)
                out[t0 + t, mine] = share.t() @ val
                lse[t0 + t, mine] = total
                if sums is not None:
                    sums[0, where, h, row] += share.sum(dim=1)
        t0 += k
    return [out, lse] + ([] if sums is None else [sums])
