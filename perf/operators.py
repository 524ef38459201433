"""The latent-attention operators as a serving program calls them, with plain forms to measure them against.

Latent attention keeps one row per token and layer, c_t | r_t (a latent vector of `rank` values and a rotary key
of `rope` values shared by all heads), in pages of a cache:

  append   new tokens' rows are written into the pages that a page table names
  decode   the absorbed form: queries of rank + rope values attend the rows themselves and sum the latents;
           one token a sequence, or a tree of drafted tokens
  prefill  the expanded form for prompts: keys k_nope | r and values per head
  pages    forking sequences, truncating and growing them, and compacting the page pool

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
        dict(name="decode_one", op="decode", n=1, heads=32, rank=512, rope=64, page=64, lo=1013, hi=1013, tokens=1,
             tree=False, dtype="bf16", lens_seed=1),
        # the decode batch of the framework's own benchmark, ragged lengths
        dict(name="decode_batch64", op="decode", n=64, heads=32, rank=512, rope=64, page=64, lo=500, hi=8192,
             tokens=1, tree=False, dtype="bf16", lens_seed=2),
        # verification of drafted trees of up to 8 tokens, small pages
        dict(name="decode_tree", op="decode", n=16, heads=32, rank=512, rope=64, page=16, lo=2000, hi=16384,
             tokens=8, tree=True, dtype="fp16", lens_seed=3),
        # all heads on one GPU over long contexts
        dict(name="decode_heads128", op="decode", n=8, heads=128, rank=512, rope=64, page=128, lo=16000, hi=32768,
             tokens=1, tree=False, dtype="bf16", lens_seed=4),
        # a few short prompts
        dict(name="prefill_short", op="prefill", n=3, heads=32, nope=128, rope=64, v=128, lo=33, hi=200, past=0,
             causal=True, dtype="bf16", lens_seed=5),
        # the framework's four-sequence prefill workload
        dict(name="prefill_varlen4", op="prefill", n=4, heads=32, nope=128, rope=64, v=128, lo=0, hi=0, past=0,
             causal=True, dtype="bf16", lens_seed=0),
        # one long prompt
        dict(name="prefill_long", op="prefill", n=1, heads=32, nope=128, rope=64, v=128, lo=11111, hi=11111, past=0,
             causal=True, dtype="fp16", lens_seed=6),
        # later chunks of prompts whose beginnings are in the cache already
        dict(name="prefill_resumed", op="prefill", n=4, heads=32, nope=128, rope=64, v=128, lo=300, hi=1100,
             past=8192, causal=True, dtype="bf16", lens_seed=7),
        # one new token for each of 256 sequences
        dict(name="append_step", op="append", n=256, rank=512, rope=64, page=64, lo=1, hi=1, past=700, dtype="bf16",
             lens_seed=8),
        # the rows of the prefill workload's prompts
        dict(name="append_prompts", op="append", n=4, rank=512, rope=64, page=64, lo=2000, hi=8192, past=300,
             dtype="bf16", lens_seed=9),
        # 48 branches of running sequences: shared pages, private copies of the last, partly filled ones
        dict(name="pages_fork", op="fork", n=64, forks=48, rank=512, rope=64, page=64, layers=8, lo=200, hi=1500,
             dtype="bf16", lens_seed=10),
        # a fragmented pool brought back to a dense one
        dict(name="pages_compact", op="compact", n=64, forks=0, rank=512, rope=64, page=64, layers=2, lo=600, hi=2200,
             dtype="bf16", lens_seed=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "fork", "compact"])
    dtype = rng.choice(["bf16", "fp16"])
    seed = rng.randrange(1 << 30)
    if op == "decode":
        n = _log(rng, 1, 96)
        heads = rng.choice([4, 16, 20, 32, 64, 128])
        tokens = rng.choice([1, 1, 2, 5, 8])
        hi = _log(rng, 40, max(41, min(60000, 400000 // n)))
        return dict(op=op, n=n, heads=heads, rank=rng.choice([128, 256, 512, 512]), rope=rng.choice([32, 64, 64]),
                    page=rng.choice([16, 32, 64, 128]), lo=max(tokens, hi // rng.choice([1, 2, 8])), hi=hi,
                    tokens=tokens, tree=tokens > 1 and rng.random() < 0.6, dtype=dtype, lens_seed=seed)
    if op == "prefill":
        n = _log(rng, 1, 12)
        hi = _log(rng, 20, 7000 // n)
        past = rng.choice([0, 0, _log(rng, 1, 4000)])
        return dict(op=op, n=n, heads=rng.choice([4, 16, 32]), nope=rng.choice([64, 128, 128]),
                    rope=rng.choice([32, 64, 64]), v=rng.choice([64, 128, 128]), lo=max(1, hi // rng.choice([1, 3])),
                    hi=hi, past=past, causal=rng.random() < 0.8, dtype=dtype, lens_seed=seed)
    page = rng.choice([16, 32, 64, 128])
    rank, rope = rng.choice([(128, 32), (256, 64), (512, 64), (512, 64)])
    if op == "append":
        n = _log(rng, 1, 200)
        hi = _log(rng, 1, max(2, 20000 // n))
        return dict(op=op, n=n, rank=rank, rope=rope, page=page, lo=max(1, hi // 2), hi=hi, past=_log(rng, 1, 900),
                    dtype=dtype, lens_seed=seed)
    n = _log(rng, 2, 80)
    hi = _log(rng, 30, 2000)
    layers = rng.choice([1, 2, 3])
    return dict(op=op, n=n, forks=rng.randint(1, n) if op == "fork" else 0, rank=rank, rope=rope, page=page,
                layers=layers, lo=max(1, hi // 3), hi=hi, dtype=dtype, lens_seed=seed)


def _new_lens(case):
    """Tokens that the call brings, by sequence."""
    if case["op"] == "prefill" and case["hi"] == 0:
        return [2048, 4096, 8192, 8192]
    r = random.Random(case["lens_seed"])
    if case["op"] == "decode":
        r.random()
        return [r.randint(max(1, case["tokens"] - 3), case["tokens"]) if case["tree"] else case["tokens"]
                for _ in range(case["n"])]
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


def _total_lens(case):
    """Tokens of each sequence, those that the call brings among them."""
    r = random.Random(case["lens_seed"] + 1)
    if case["op"] in ("decode", "fork", "compact"):
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    return [k + (r.randint(case["past"] // 2, case["past"]) if case["past"] else 0) for k in _new_lens(case)]


def _pages_of(lens, page):
    return [-(-x // page) for x in lens]


# ---------------------------------------------------------------------------------------------------- inputs
def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _table(lens, page, rows, width, num_pages, rng):
    """Pages in random order for the first len(lens) rows of a table; the rest is -1."""
    perm = rng.permutation(num_pages)
    t = np.full((rows, width), -1, dtype=np.int32)
    ref = np.zeros(num_pages, dtype=np.int32)
    at = 0
    for i, k in enumerate(_pages_of(lens, page)):
        t[i, :k] = perm[at:at + k]
        ref[perm[at:at + k]] = 1
        at += k
    full = np.zeros(rows, dtype=np.int32)
    full[:len(lens)] = lens
    return [torch.from_numpy(x).cuda() for x in (t, full, ref)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    s = dict(case=dict(case))
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "prefill":
        nq, nk = _new_lens(case), _total_lens(case)
        H, tq, tk = case["heads"], sum(nq), sum(nk)
        s.update(nq=nq, nk=nk, cu_q=_cu(nq), cu_k=_cu(nk), q=randn(tq, H, case["nope"] + case["rope"]),
                 kv=randn(tk, H, case["nope"] + case["v"]), rope=randn(tk, case["rope"]),
                 out=torch.empty(tq, H, case["v"], dtype=dt, device="cuda"),
                 lse=torch.empty(tq, H, dtype=torch.float32, device="cuda"),
                 scale=1.0 / math.sqrt(case["nope"] + case["rope"]))
        return s
    lens, page = _total_lens(case), case["page"]
    width = max(_pages_of(lens, page)) + 2
    used = sum(_pages_of(lens, page))
    num_pages = used + (case.get("forks", 0) + 8 if case["op"] != "compact" else used // 2 + 8)
    extra_rows = case.get("forks", 0)
    s["table"], s["lens"], s["ref"] = _table(lens, page, len(lens) + extra_rows, width, num_pages, rng)
    s["lens_h"] = lens
    d = case["rank"] + case["rope"]
    s["pages"] = randn(case.get("layers", 1), num_pages, page, d)
    if case["op"] == "decode":
        nq = _new_lens(case)
        tq, H = sum(nq), case["heads"]
        s.update(nq=nq, cu_q=_cu(nq), q=randn(tq, H, d), scale=1.0 / math.sqrt(192.0),
                 out=torch.empty(tq, H, case["rank"], dtype=dt, device="cuda"),
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
        s.update(nq=new, cu_q=_cu(new), latent=randn(sum(new), case["rank"]), rope=randn(sum(new), case["rope"]))
    else:
        s["kept"] = [s["table"].clone(), s["lens"].clone(), s["ref"].clone()]
        if case["op"] == "fork":
            s["parents"] = torch.tensor(rng.integers(0, len(lens), case["forks"]), dtype=torch.int32, device="cuda")
            s["children"] = torch.arange(len(lens), len(lens) + case["forks"], dtype=torch.int32, device="cuda")
    if own:
        import hybrid_linear_attention_decode_gb300 as kda
        s["cache"] = kda.LatentCache(s["pages"], case["rank"])
        s["pt"] = kda.PageTable(s["table"], s["lens"], s["ref"], page)
        if case["op"] == "decode":
            nbytes = kda.kda_latent_decode_workspace_bytes(s["cache"], case["heads"], case["n"], max(s["nq"]))
            s["ws"] = torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")
        elif case["op"] in ("fork", "compact"):
            s["ws"] = torch.empty(kda.kda_pages_workspace_bytes(s["pt"], max(1, case["forks"])), dtype=torch.uint8,
                                  device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"decode": _own_decode, "prefill": _own_prefill, "append": _own_append, "fork": _own_fork,
                "compact": _own_compact}[op](s)
    return {"decode": _plain_decode, "prefill": _plain_prefill, "append": _plain_append, "fork": _plain_fork,
            "compact": _plain_compact}[op](s)


def _own_decode(s):
    import hybrid_linear_attention_decode_gb300 as kda
    kda.kda_latent_decode(s["cache"], 0, s["pt"], None, s["cu_q"], max(s["nq"]), s["q"], s["out"], s["lse"],
                          s["scale"], s["ws"], s["status"], tree_mask=s["tree"])
    return [s["out"], s["lse"]]


def _own_prefill(s):
    import hybrid_linear_attention_decode_gb300 as kda
    c = s["case"]
    kda.kda_latent_prefill(s["cu_q"], s["cu_k"], max(s["nq"]), s["q"], s["kv"][..., :c["nope"]], s["rope"],
                           s["kv"][..., c["nope"]:], s["out"], s["lse"], s["scale"], s["status"], causal=c["causal"])
    return [s["out"], s["lse"]]


def _own_append(s):
    import hybrid_linear_attention_decode_gb300 as kda
    kda.kda_latent_append(s["cache"], 0, s["pt"], None, s["cu_q"], s["latent"], s["rope"], s["status"])
    return [s["pages"]]


def _restore(s):
    """The bookkeeping as it was before the first pass (the page contents that a pass writes are the same each time)."""
    for have, kept in zip((s["table"], s["lens"], s["ref"]), s["kept"]):
        have.copy_(kept)


def _own_fork(s):
    import hybrid_linear_attention_decode_gb300 as kda
    _restore(s)
    kda.kda_pages_fork(s["pt"], s["cache"], s["parents"], s["children"], s["ws"], s["status"])
    return [s["pages"], s["table"], s["lens"], s["ref"]]


def _own_compact(s):
    import hybrid_linear_attention_decode_gb300 as kda
    _restore(s)
    kda.kda_pages_compact(s["pt"], s["cache"], s["ws"], s["status"])
    return [s["pages"], s["table"], s["lens"], s["ref"]]


def _softmax_sum(x, v):
    """Rows of scores (masked ones at -inf) to weighted sums of v, and the logarithm of the rows' sums."""
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(x - m)
    z = e.sum(dim=-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(z == 0, torch.ones_like(z), z)
    return o, (m + torch.log(z))[..., 0]


def _plain_decode(s):
    c, at = s["case"], 0
    H, page = c["heads"], c["page"]
    out, lse = s["out"], s["lse"]
    for b, (n, k) in enumerate(zip(s["lens_h"], s["nq"])):
        rows = s["pages"][0][s["table"][b, :-(-n // page)].long()].reshape(-1, c["rank"] + c["rope"])[:n].float()
        x = torch.matmul(s["q"][at:at + k].float().reshape(k * H, -1), rows.t()) * s["scale"]
        x = x.reshape(k, H, n)
        if k > 1 or s["tree"] is not None:
            j = torch.arange(k, device="cuda")
            if s["tree"] is not None:
                seen = (s["tree"][at:at + k, None] >> j[None, :]) & 1 == 1
            else:
                seen = j[None, :] <= j[:, None]
            x[:, :, n - k:] = x[:, :, n - k:].masked_fill(~seen[:, None, :], float("-inf"))
        o, z = _softmax_sum(x.reshape(k * H, n), rows[:, :c["rank"]])
        out[at:at + k] = o.reshape(k, H, -1).to(out.dtype)
        lse[at:at + k] = z.reshape(k, H)
        at += k
    return [out, lse]


def _plain_prefill(s):
    c = s["case"]
    out, lse = s["out"], s["lse"]
    q0 = k0 = 0
    for n, m in zip(s["nq"], s["nk"]):
        rope = s["rope"][k0:k0 + m].float()
        hidden = None
        if c["causal"]:
            hidden = (torch.arange(m, device="cuda")[None, :]
                      > torch.arange(n, device="cuda")[:, None] + (m - n))
        step = max(1, min(c["heads"], (1 << 28) // max(1, n * m)))
        for h in range(0, c["heads"], step):
            e = min(c["heads"], h + step)
            q = s["q"][q0:q0 + n, h:e].float().transpose(0, 1)
            kv = s["kv"][k0:k0 + m, h:e].float().transpose(0, 1)
            x = torch.matmul(q[..., :c["nope"]], kv[..., :c["nope"]].transpose(1, 2))
            x += torch.matmul(q[..., c["nope"]:], rope.t())
            x *= s["scale"]
            if hidden is not None:
                x.masked_fill_(hidden, float("-inf"))
            o, z = _softmax_sum(x, kv[..., c["nope"]:])
            out[q0:q0 + n, h:e] = o.transpose(0, 1).to(out.dtype)
            lse[q0:q0 + n, h:e] = z.transpose(0, 1)
        q0 += n
        k0 += m
    return [out, lse]


def _plain_append(s):
    c = s["case"]
    t = torch.arange(s["latent"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
    pos = s["lens"].long()[b] - (s["cu_q"].long()[b + 1] - t)
    pid = s["table"][b, pos // c["page"]].long()
    s["pages"][0][pid, pos % c["page"]] = torch.cat([s["latent"], s["rope"]], dim=1)
    return [s["pages"]]


def _plain_fork(s):
    _restore(s)
    page = s["case"]["page"]
    par, chi = s["parents"].long(), s["children"].long()
    n = s["lens"][par].long()
    part = n % page != 0
    new = torch.nonzero(s["ref"] == 0)[:, 0][torch.cumsum(part, 0) - 1]
    rows = s["table"][par]
    at = torch.arange(rows.shape[1], device="cuda")
    last = part[:, None] & (at[None, :] == (n // page)[:, None])
    shared = (at[None, :] < (n // page)[:, None])
    src = rows[last].long()
    dst = new[part]
    s["pages"][:, dst] = s["pages"][:, src]
    s["ref"].index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    s["ref"][dst] = 1
    s["table"][chi] = torch.where(last, new[:, None].to(torch.int32), rows)
    s["lens"][chi] = s["lens"][par]
    return [s["pages"], s["table"], s["lens"], s["ref"]]


def _plain_compact(s):
    _restore(s)
    ref = s["ref"]
    n = ref.shape[0]
    used = ref > 0
    at = torch.arange(n, device="cuda")
    k = used.sum()
    src = torch.nonzero(used & (at >= k))[:, 0]
    dst = torch.nonzero(~used & (at < k))[:, 0]
    s["pages"][:, dst] = s["pages"][:, src]
    to = at.clone()
    to[src] = dst
    ref[dst] = ref[src]
    ref[src] = 0
    t = s["table"]
    t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()].to(torch.int32), t))
    return [s["pages"], t, s["lens"], ref]


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    op, lens = case["op"], _total_lens(case)
    new = _new_lens(case) if op in ("decode", "prefill", "append") else None
    if op == "decode":
        d, H, tq = case["rank"] + case["rope"], case["heads"], sum(new)
        seen = sum(k * n - k * (k - 1) // 2 for n, k in zip(lens, new))
        return {"bytes": 2 * d * sum(lens) + tq * H * (2 * d + 2 * case["rank"] + 4),
                "flops": 2 * H * seen * (d + case["rank"])}
    if op == "prefill":
        H, tq, tk = case["heads"], sum(new), sum(lens)
        dq = case["nope"] + case["rope"]
        seen = sum((k * n - k * (k - 1) // 2) if case["causal"] else k * n for n, k in zip(lens, new))
        return {"bytes": 2 * tq * H * (dq + case["v"]) + 4 * tq * H
                + 2 * tk * (H * (case["nope"] + case["v"]) + case["rope"]),
                "flops": 2 * H * seen * (dq + case["v"])}
    row = 2 * (case["rank"] + case["rope"])
    if op == "append":
        return {"bytes": 2 * row * sum(new), "flops": 0}
    page, k = case["page"], _pages_of(lens, case["page"])
    meta = 4 * (sum(k) + len(lens))
    if op == "fork":
        # every fork of a partly filled sequence copies one page in each layer: taken as all of them
        return {"bytes": 2 * case["forks"] * case["layers"] * page * row + meta, "flops": 0}
    # with the used pages spread evenly, a third of them lies behind the dense part
    moved = sum(k) * (1 - sum(k) / (sum(k) + sum(k) // 2 + 8))
    return {"bytes": 2 * int(moved) * case["layers"] * page * row + 2 * meta, "flops": 0}


# ---------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The attention outputs from their definition in 64 bits: sums of exponentials over the keys a query sees."""
    if case["op"] not in ("decode", "prefill"):
        return None
    s = prepare(case, seed)
    if work(case)["flops"] > 6e12:
        return None
    f64 = torch.float64
    if case["op"] == "decode":
        out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=f64, device="cuda")
        t0 = 0
        for b, k in enumerate(s["nq"]):
            n = s["lens_h"][b]
            pos = torch.arange(n, device="cuda")
            kv = s["pages"][0, s["table"][b].long()[pos // case["page"]], pos % case["page"]].to(f64)
            for t in range(k):
                keep = torch.ones(n, dtype=torch.bool, device="cuda")
                for j in range(k):
                    if s["tree"] is not None:
                        keep[n - k + j] = bool((int(s["tree"][t0 + t]) >> j) & 1)
                    else:
                        keep[n - k + j] = j <= t
                rows = kv[keep]
                logits = s["scale"] * (rows @ s["q"][t0 + t].to(f64).t())          # [keys, heads]
                top = logits.max(dim=0).values
                w = torch.exp(logits - top)
                out[t0 + t] = (w.t() @ rows[:, :case["rank"]]) / w.sum(dim=0)[:, None]
                lse[t0 + t] = top + torch.log(w.sum(dim=0))
            t0 += k
        return [out, lse]
    out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=f64, device="cuda")
    q0 = k0 = 0
    for n, m in zip(s["nq"], s["nk"]):
        r = s["rope"][k0:k0 + m].to(f64)
        for h in range(case["heads"]):
            key = torch.cat([s["kv"][k0:k0 + m, h, :case["nope"]].to(f64), r], dim=1)
            val = s["kv"][k0:k0 + m, h, case["nope"]:].to(f64)
            for a in range(0, n, 2048):
                e = min(n, a + 2048)
                stop = e + m - n if case["causal"] else m
                logits = s["scale"] * (s["q"][q0 + a:q0 + e, h].to(f64) @ key[:stop].t())
                if case["causal"]:
                    late = (torch.arange(stop, device="cuda")[None]
                            - torch.arange(a, e, device="cuda")[:, None]) > m - n
                    logits[late] = -math.inf
                top = logits.max(dim=1).values
                w = torch.exp(logits - top[:, None])
                out[q0 + a:q0 + e, h] = (w @ val[:stop]) / w.sum(dim=1)[:, None]
                lse[q0 + a:q0 + e, h] = top + torch.log(w.sum(dim=1))
        q0 += n
        k0 += m
    return [out, lse]
