"""Attention over the keys of a request and the paged cache that holds them:
the calls that are measured, their plain forms and their definition in 64 bits.

  prompt    causal attention over packed prompts (grouped heads)
  cached    one new token per sequence over a paged key-value cache
  selected  attention over the keys that the index selected, from the cache
  fork      sequences that share another's pages, and their release
  compact   live pages of a fragmented cache moved to its front

A case's sequence lengths follow from its sizes and its number "ragged"; the
values follow from the seed.
"""
import random

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a few short turns that arrive together: launch latency
        {"name": "prompt short turns", "op": "prompt", "n_seq": 7, "q_len": 117, "prefix": 0, "Hq": 32, "Hkv": 8,
         "D": 128, "ragged": 1},
        # an ordinary prefill batch, each sequence with its earlier chunks behind it, narrow heads
        {"name": "prompt chunks", "op": "prompt", "n_seq": 4, "q_len": 2048, "prefix": 2500, "Hq": 32, "Hkv": 4,
         "D": 64, "ragged": 2},
        # one long prompt
        {"name": "prompt long", "op": "prompt", "n_seq": 1, "q_len": 16384, "prefix": 0, "Hq": 16, "Hkv": 2,
         "D": 128, "ragged": 0},
        # one conversation's next token
        {"name": "cached single", "op": "cached", "n_seq": 1, "length": 1021, "page": 16, "Hq": 32, "Hkv": 8, "D": 128,
         "kv": "bf16", "ragged": 0},
        # a serving batch of unlike lengths on an 8-bit cache
        {"name": "cached batch fp8", "op": "cached", "n_seq": 48, "length": 8192, "page": 64, "Hq": 64, "Hkv": 8,
         "D": 128, "kv": "fp8", "ragged": 3},
        # few sequences with long prefixes
        {"name": "cached long", "op": "cached", "n_seq": 4, "length": 131072, "page": 64, "Hq": 32, "Hkv": 8,
         "D": 128, "kv": "bf16", "ragged": 0},
        # a decode step: one query's 2048 keys of a 128K prefix, one key head
        {"name": "selected step", "op": "selected", "rows": 1, "prefix": 131072, "k": 2048, "page": 64, "Hq": 64,
         "Hkv": 1, "D": 128, "kv": "bf16"},
        # an odd chunk near the start of a prompt (rows with fewer keys than k), 8-bit cache
        {"name": "selected early fp8", "op": "selected", "rows": 509, "prefix": 1400, "k": 1000, "page": 32, "Hq": 32,
         "Hkv": 8, "D": 128, "kv": "fp8"},
        # a whole prefill chunk at 128K
        {"name": "selected chunk", "op": "selected", "rows": 8192, "prefix": 131072, "k": 2048, "page": 64, "Hq": 32,
         "Hkv": 1, "D": 128, "kv": "bf16"},
        # two conversations branch, one layer
        {"name": "fork few", "op": "fork", "n_fork": 2, "n_layers": 1, "n_pages": 256, "page": 16, "Hkv": 8, "D": 128,
         "n_seq": 5, "length": 500, "ragged": 4},
        # many samples branch from their prompts, all layers of a small model
        {"name": "fork many", "op": "fork", "n_fork": 64, "n_layers": 16, "n_pages": 384, "page": 64, "Hkv": 8,
         "D": 128, "n_seq": 24, "length": 700, "ragged": 5},
        # a cache after half of its sequences have left
        {"name": "compact", "op": "compact", "n_layers": 4, "n_pages": 1024, "page": 64, "Hkv": 8, "D": 128,
         "n_seq": 40, "length": 2000, "ragged": 6},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["prompt", "cached", "selected", "fork", "compact"])
    ragged = rng.randrange(1, 1 << 20)
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    if op == "prompt":
        q_len = _log(rng, 1, 4000)
        return {"op": op, "n_seq": rng.randint(1, max(1, min(12, 9000 // q_len))), "q_len": q_len,
                "prefix": rng.choice([0, _log(rng, 1, 3000)]), "Hq": Hq, "Hkv": Hkv, "D": D, "ragged": ragged}
    if op == "cached":
        length = _log(rng, 1, 60000)
        return {"op": op, "n_seq": rng.randint(1, max(1, min(96, 120000 // length))), "length": length,
                "page": rng.choice([16, 32, 64, 128, 256]), "Hq": Hq, "Hkv": Hkv, "D": D,
                "kv": rng.choice(["bf16", "fp8"]), "ragged": ragged}
    if op == "selected":
        k = _log(rng, 1, 2048)
        return {"op": op, "rows": _log(rng, 1, max(1, min(4096, 2000000 // (k * Hkv)))), "prefix": _log(rng, 1, 131072),
                "k": k, "page": rng.choice([16, 32, 64, 128, 256]), "Hq": Hq, "Hkv": Hkv, "D": D,
                "kv": rng.choice(["bf16", "fp8"])}
    page = rng.choice([16, 32, 64, 128])
    length = _log(rng, 1, 1500)
    n_seq = rng.randint(2, 24)
    n_fork = rng.randint(1, 48)
    n_pages = n_seq * (length // page + 1) + n_fork + rng.randint(0, 60)
    case = {"op": op, "n_layers": rng.randint(1, max(1, min(8, 65536 // (n_pages * page)))), "n_pages": n_pages,
            "page": page, "Hkv": Hkv, "D": D, "n_seq": n_seq, "length": length, "ragged": ragged}
    if op == "fork":
        case["n_fork"] = n_fork
    return case


def _lens(n, most, ragged, least=1):
    """n lengths up to `most`, the first of them `most` itself; all alike where ragged is 0."""
    if not ragged:
        return [most] * n
    r = random.Random(ragged)
    return [most] + [r.randint(min(least, most), most) for _ in range(n - 1)]


def _prompt_lens(c):
    ql = _lens(c["n_seq"], c["q_len"], c["ragged"])
    pre = _lens(c["n_seq"], c["prefix"], c["ragged"] + 1 if c["ragged"] else 0, 0) if c["prefix"] else [0] * c["n_seq"]
    return ql, [a + b for a, b in zip(ql, pre)]


def _cum(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def work(c):
    op = c["op"]
    if op == "prompt":
        ql, kl = _prompt_lens(c)
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(ql, kl))
        return {"bytes": sum(ql) * c["Hq"] * (c["D"] * 4 + 4) + sum(kl) * c["Hkv"] * c["D"] * 4,
                "flops": 4 * pairs * c["Hq"] * c["D"]}
    row = 2 * c["Hkv"] * (c["D"] * 2 if c.get("kv", "bf16") == "bf16" else c["D"] + 4)  # one token's K and V
    if op == "cached":
        n = sum(_lens(c["n_seq"], c["length"], c["ragged"]))
        return {"bytes": n * row + c["n_seq"] * c["Hq"] * (c["D"] * 4 + 4), "flops": 4 * n * c["Hq"] * c["D"]}
    if op == "selected":
        first = c["prefix"] - c["rows"]
        keys = sum(min(c["k"], max(1, first + i + 1)) for i in range(c["rows"]))
        return {"bytes": min(keys, max(c["prefix"], 1)) * row + c["rows"] * (c["k"] * 4 + c["Hq"] * (c["D"] * 4 + 4)),
                "flops": 4 * keys * c["Hq"] * c["D"]}
    lens = _lens(c["n_seq"], c["length"], c["ragged"])
    tables = sum(-(-n // c["page"]) for n in lens) * 4 + c["n_pages"] * 8
    if op == "fork":
        slots = sum(lens[i % c["n_seq"]] % c["page"] for i in range(c["n_fork"]))
        return {"bytes": 2 * slots * c["n_layers"] * row + tables, "flops": 0}
    live, _, gone = _pages(c)
    holes = sum(1 for p in range(len(live)) if p in gone)
    return {"bytes": 2 * holes * c["page"] * c["n_layers"] * row + 2 * tables, "flops": 0}


def _pages(c):
    """The pages of a cache in use: those of the sequences that stay (by sequence), and the set that is free."""
    lens = _lens(c["n_seq"], c["length"], c["ragged"])
    need = [-(-n // c["page"]) for n in lens]
    order = list(range(c["n_pages"]))
    random.Random(c["ragged"] + 7).shuffle(order)
    at = _cum(need)
    rows = [order[at[s]:at[s + 1]] for s in range(c["n_seq"])]
    stay = [s for s in range(c["n_seq"]) if c["op"] != "compact" or s % 2 == 0]
    live = [p for s in stay for p in rows[s]]
    return live, {s: rows[s] for s in stay}, set(range(c["n_pages"])) - set(live)


# ------------------------------------------------------------------ inputs
def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF16)


def _pool(g, pages, c):
    """K or V pages: bf16 values, or e4m3 codes with one scale for each token and head."""
    x = torch.empty(pages, c["page"], c["Hkv"], c["D"], dtype=BF16, device=DEV).normal_(generator=g)
    # some channels are larger than the others, as in trained models' keys
    x[..., :4] *= 3
    if c["kv"] == "bf16":
        return x, None
    s = (x.abs().amax(-1).float() / 448).clamp_min(1e-12)
    return (x.float() / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def _tables(g, lens, page, width):
    """Page tables over a pool whose pages are in no order; -1 behind a sequence's last page."""
    need = [-(-n // page) for n in lens]
    total = sum(need)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = _cum(need)
    for i, n in enumerate(need):
        table[i, :n] = order[at[i]:at[i + 1]]
    return table, total


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = c["op"], dict(c)
    if op == "prompt":
        ql, kl = _prompt_lens(c)
        s |= {"q": _normal(g, sum(ql), c["Hq"], c["D"], scale=1.5), "k": _normal(g, sum(kl), c["Hkv"], c["D"]),
              "v": _normal(g, sum(kl), c["Hkv"], c["D"]), "cu_q": _int(_cum(ql)), "cu_k": _int(_cum(kl))}
        # the plain form's plan: each packed token's sequence and position
        s["q_max"], s["k_max"] = max(ql), max(kl)
    elif op == "cached":
        lens = _lens(c["n_seq"], c["length"], c["ragged"])
        width = -(-max(lens) // c["page"])
        s["tables"], total = _tables(g, lens, c["page"], width)
        s["lens"] = _int(lens)
        s["q"] = _normal(g, c["n_seq"], c["Hq"], c["D"], scale=1.5)
        (s["k"], s["ks"]), (s["v"], s["vs"]) = _pool(g, total, c), _pool(g, total, c)
    elif op == "selected":
        n, T, k = max(c["prefix"], c["rows"]), c["rows"], c["k"]
        width = -(-n // c["page"])
        s["tables"], total = _tables(g, [n], c["page"], width)
        s["lens"] = _int([n])
        s["q"] = _normal(g, T, c["Hq"], c["D"], scale=1.5)
        (s["k"], s["ks"]), (s["v"], s["vs"]) = _pool(g, total, c), _pool(g, total, c)
        # the newest T positions; each row's ids are distinct, at most its position, in no order, -1 behind them
        pos = n - T + torch.arange(T, device=DEV)[:, None]
        gap = ((pos + 1).double() / k).clamp_min(1)
        ids = torch.rand(T, k, generator=g, device=DEV) * (gap - 1) + torch.arange(k, device=DEV) * gap
        ids = torch.where(torch.arange(k, device=DEV) <= pos, ids.long().clamp_max(n), n)
        ids = ids.gather(1, torch.rand(T, k, generator=g, device=DEV).argsort(1))
        ids = ids.gather(1, (ids > pos).to(torch.int8).argsort(dim=1, stable=True))
        s["ids"] = torch.where(ids > pos, -1, ids).to(torch.int32)
    else:
        _, rows, free = _pages(c)
        lens = _lens(c["n_seq"], c["length"], c["ragged"])
        n_rows = c["n_seq"] + c.get("n_fork", 0)
        width = max(-(-n // c["page"]) for n in lens)
        s["k"] = torch.empty(c["n_layers"], c["n_pages"], c["page"], c["Hkv"], c["D"], dtype=BF16, device=DEV)
        s["k"].normal_(generator=g)
        s["v"] = torch.empty_like(s["k"]).normal_(generator=g)
        s["tables"] = _int([rows.get(i, []) + [-1] * (width - len(rows.get(i, []))) for i in range(n_rows)])
        s["lens"] = _int([lens[i] if i in rows else 0 for i in range(n_rows)])
        s["refs"] = _int([int(p not in free) for p in range(c["n_pages"])])
        if op == "fork":
            s["src"] = _int([i % c["n_seq"] for i in range(c["n_fork"])])
            s["dst"] = _int([c["n_seq"] + i for i in range(c["n_fork"])])
        else:
            s["kept"] = (s["tables"].clone(), s["refs"].clone())
    return s


# -------------------------------------------------------------- plain forms
def _attend(q, k, v, seen):
    """q [B, Lq, Hkv, G, D], k and v [B, Lk, Hkv, D], seen [B, Lq, Lk], in float32: softmax over the seen keys.
    Returns o [B, Lq, Hkv, G, D] and the log of the sum [B, Lq, Hkv, G]; zeros and -inf where nothing is seen."""
    B, Lq, Hkv, G, D = q.shape
    x = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Lq, D) @ k.permute(0, 2, 3, 1)
    x = x.view(B, Hkv, G, Lq, -1).mul_(D ** -0.5)
    x.masked_fill_(~seen[:, None, None], -torch.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.clamp_min(torch.finfo(m.dtype).min)).exp_()
    tot = p.sum(-1, keepdim=True)
    o = p.reshape(B, Hkv, G * Lq, -1) @ v.permute(0, 2, 1, 3)
    o = o.view(B, Hkv, G, Lq, D) / tot.where(tot > 0, 1)
    lse = (m + tot.log()).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4), lse.permute(0, 3, 1, 2)


def _plain_prompt(s):
    q, cu_q, cu_k = s["q"], s["cu_q"].long(), s["cu_k"].long()
    Nq, Hq, D = q.shape
    Hkv = s["Hkv"]
    lq, lk = cu_q.diff(), cu_k.diff()
    i = torch.arange(s["q_max"], device=DEV)
    j = torch.arange(s["k_max"], device=DEV)
    qi = (cu_q[:-1, None] + i).clamp_max(Nq - 1)
    kj = (cu_k[:-1, None] + j).clamp_max(s["k"].shape[0] - 1)
    seen = j[None, None] <= (lk - lq)[:, None, None] + i[None, :, None]
    seen &= (j < lk[:, None])[:, None]
    o, lse = _attend(q[qi].float().view(*qi.shape, Hkv, Hq // Hkv, D), s["k"][kj].float(), s["v"][kj].float(), seen)
    real = i < lq[:, None]
    return {"out": o.reshape(*qi.shape, Hq, D)[real].to(BF16), "lse": lse.reshape(*qi.shape, Hq)[real]}


def _values(pool, scale, at):
    """The float32 rows [..., Hkv, D] of a pool at token slots `at` (page * page size + offset)."""
    x = pool.flatten(0, 1)[at]
    if scale is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * scale.flatten(0, 1)[at][..., None]


def _plain_cached(s):
    q, lens = s["q"], s["lens"].long()
    B, Hq, D = q.shape
    j = torch.arange(s["tables"].shape[1] * s["page"], device=DEV)
    at = s["tables"].long().clamp_min(0)[:, j // s["page"]] * s["page"] + j % s["page"]
    seen = (j < lens[:, None])[:, None]
    o, lse = _attend(q.float().view(B, 1, s["Hkv"], -1, D), _values(s["k"], s["ks"], at),
                     _values(s["v"], s["vs"], at), seen)
    return {"out": o.reshape(B, Hq, D).to(BF16), "lse": lse.reshape(B, Hq)}


def _plain_selected(s):
    q, ids = s["q"], s["ids"].long()
    T, Hq, D = q.shape
    real = ids.clamp_min(0)
    at = s["tables"][0].long()[real // s["page"]] * s["page"] + real % s["page"]
    o, lse = _attend(q.float().view(T, 1, s["Hkv"], -1, D), _values(s["k"], s["ks"], at),
                     _values(s["v"], s["vs"], at), (ids >= 0)[:, None])
    return {"out": o.reshape(T, Hq, D).to(BF16), "lse": lse.reshape(T, Hq)}


def _plain_fork(s):
    tables, lens, refs, page = s["tables"], s["lens"], s["refs"], s["page"]
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src]
    full, part = n // page, n % page
    # free pages, lowest first: one for each part page, then as many that stay as they are
    order = (refs > 0).to(torch.int8).argsort(stable=True)
    need = part > 0
    rank = torch.where(need, need.cumsum(0) - 1, need.sum() + (~need).cumsum(0) - 1)
    fresh = order[rank]
    old = tables[src].gather(1, full[:, None].long().clamp_max(tables.shape[1] - 1)).squeeze(1).long().clamp_min(0)
    j = torch.arange(tables.shape[1], device=DEV)
    shared = j < full[:, None]
    row = torch.where(shared, tables[src], -1)
    row = torch.where((j == full[:, None]) & need[:, None], fresh[:, None].to(torch.int32), row)
    refs.index_add_(0, tables[src].long().clamp_min(0).flatten(), shared.flatten().to(torch.int32))
    refs.index_add_(0, fresh, need.to(torch.int32))
    tables[dst], lens[dst] = row, n
    filled = (torch.arange(page, device=DEV) < part[:, None])[None, :, :, None, None]
    s["k"][:, fresh] = torch.where(filled, s["k"][:, old], s["k"][:, fresh])
    s["v"][:, fresh] = torch.where(filled, s["v"][:, old], s["v"][:, fresh])


def _plain_free(s, seqs):
    tables, lens, refs = s["tables"], s["lens"], s["refs"]
    at = seqs.long()
    used = torch.arange(tables.shape[1], device=DEV) * s["page"] < lens[at][:, None]
    refs.index_add_(0, tables[at].long().clamp_min(0).flatten(), -used.flatten().to(torch.int32))
    tables[at], lens[at] = -1, 0


def _plain_compact(s):
    tables, refs = s["tables"], s["refs"]
    live = refs > 0
    page = torch.arange(refs.numel(), device=DEV)
    front = page < live.sum()
    move, to = page[live & ~front], page[~live & front]
    s["k"][:, to] = s["k"][:, move]
    s["v"][:, to] = s["v"][:, move]
    new = page.clone()
    new[move] = to
    tables.copy_(torch.where(tables >= 0, new[tables.long().clamp_min(0)].to(torch.int32), tables))
    refs[to] = refs[move]
    refs[move] = 0


def run(s):
    op = s["op"]
    if op == "fork":
        if own:
            from ivf_top_key_b200 import cache_fork, cache_free
            cache_fork(s["k"], s["v"], s["tables"], s["lens"], s["refs"], s["src"], s["dst"])
        else:
            _plain_fork(s)
        forked = (s["tables"].clone(), s["lens"].clone(), s["refs"].clone())
        if own:
            cache_free(s["tables"], s["lens"], s["refs"], s["dst"], page_size=s["page"])
        else:
            _plain_free(s, s["dst"])
        return {"k": s["k"], "v": s["v"], "forked": forked, "freed": (s["tables"], s["lens"], s["refs"])}
    if op == "compact":
        s["tables"].copy_(s["kept"][0])  # the fragmented state again
        s["refs"].copy_(s["kept"][1])
        if own:
            from ivf_top_key_b200 import cache_compact
            cache_compact(s["k"], s["v"], s["tables"], s["lens"], s["refs"])
        else:
            _plain_compact(s)
        return {"k": s["k"], "v": s["v"], "tables": s["tables"], "lens": s["lens"], "refs": s["refs"]}
    if not own:
        return {"prompt": _plain_prompt, "cached": _plain_cached, "selected": _plain_selected}[op](s)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    if op == "prompt":
        from ivf_top_key_b200 import attend_prompt
        out = attend_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out_lse=lse)
    elif op == "cached":
        from ivf_top_key_b200 import attend_cached
        out = attend_cached(s["q"], s["k"], s["v"], s["tables"], s["lens"], k_scale=s["ks"], v_scale=s["vs"],
                            out_lse=lse)
    else:
        from ivf_top_key_b200 import attend_selected
        out = attend_selected(s["q"], s["ids"], s["k"], s["v"], s["tables"], s["lens"], k_scale=s["ks"],
                              v_scale=s["vs"], out_lse=lse)
    return {"out": out, "lse": lse}


# ------------------------------------------------- the definition in 64 bits
def _one(q, k, v):
    """One query's heads [Hq, D] over keys [n, Hkv, D], in float64: out [Hq, D], log of the sum [Hq]."""
    Hkv = k.shape[1]
    if not len(k):
        return torch.zeros_like(q), torch.full((len(q),), -torch.inf, dtype=q.dtype, device=q.device)
    x = torch.einsum("hgd,nhd->hgn", q.view(Hkv, -1, q.shape[-1]), k) / q.shape[-1] ** 0.5
    lse = torch.logsumexp(x, -1)
    o = torch.einsum("hgn,nhd->hgd", torch.exp(x - lse[..., None]), v)
    return o.reshape(q.shape), lse.reshape(-1)


def _dequantised(pool, scale):
    if scale is None:
        return pool.double()
    return pool.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    outs, lses = [], []
    if op == "prompt":
        G = c["Hq"] // c["Hkv"]
        ql, kl = _prompt_lens(c)
        q0, k0 = _cum(ql), _cum(kl)
        out = torch.empty(sum(ql), c["Hq"], c["D"], dtype=torch.float64, device=DEV)
        lse = torch.empty(sum(ql), c["Hq"], dtype=torch.float64, device=DEV)
        for b in range(c["n_seq"]):
            k, v = (s[n][k0[b]:k0[b + 1]].double() for n in ("k", "v"))
            for a in range(0, ql[b], 1024):  # 1024 queries at a time
                rows = torch.arange(a, min(a + 1024, ql[b]), device=DEV)
                last = kl[b] - ql[b] + int(rows[-1]) + 1
                hidden = torch.arange(last, device=DEV) > kl[b] - ql[b] + rows[:, None]
                for h in range(c["Hq"]):
                    x = s["q"][q0[b] + rows, h].double() @ k[:last, h // G].T / c["D"] ** 0.5
                    x[hidden] = -torch.inf
                    y = torch.logsumexp(x, -1)
                    out[q0[b] + rows, h] = torch.exp(x - y[:, None]) @ v[:last, h // G]
                    lse[q0[b] + rows, h] = y
        return {"out": out, "lse": lse}
    if op == "cached":
        for b, n in enumerate(_lens(c["n_seq"], c["length"], c["ragged"])):
            at = s["tables"][b, :-(-n // c["page"])].long()
            k, v = (_dequantised(s[p][at], s[t] if s[t] is None else s[t][at]).flatten(0, 1)[:n]
                    for p, t in (("k", "ks"), ("v", "vs")))
            o, y = _one(s["q"][b].double(), k, v)
            outs.append(o)
            lses.append(y)
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    if op == "selected":
        at = s["tables"][0].long()
        k, v = (_dequantised(s[p][at], s[t] if s[t] is None else s[t][at]).flatten(0, 1)
                for p, t in (("k", "ks"), ("v", "vs")))
        count = (s["ids"] >= 0).sum(1).tolist()
        for t in range(c["rows"]):
            ids = s["ids"][t, :count[t]].long()
            o, y = _one(s["q"][t].double(), k[ids], v[ids])
            outs.append(o)
            lses.append(y)
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    lens = s["lens"].tolist()
    table = s["tables"].tolist()
    k, v = s["k"].clone(), s["v"].clone()
    used = {p for row in table for p in row if p >= 0}
    free = [p for p in range(c["n_pages"]) if p not in used]
    if op == "fork":
        for a in s["src"].tolist():
            part = lens[a] % c["page"]
            if part:
                new, old = free.pop(0), table[a][lens[a] // c["page"]]
                k[:, new, :part], v[:, new, :part] = k[:, old, :part], v[:, old, :part]
        return {"k": k.double(), "v": v.double(), "forked": None, "freed": None}
    for p in sorted(used):
        if p >= len(used):
            new = free.pop(0)
            k[:, new], v[:, new] = k[:, p], v[:, p]
    return {"k": k.double(), "v": v.double(), "tables": None, "lens": None, "refs": None}
