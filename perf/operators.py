"""The cache side of a speculative round, measured: the round's keys and values written into a paged
cache, attention of the round's tokens over it, the attention weight its entries gather, and the
eviction of the entries that gathered least.

Layout: key and value pages [num_pages, Hkv, page_size, D] (or the same with slots before heads), a
page table [B, max_pages], entry j of row b in slot j % page_size of page page_table[b, j // page_size],
and accumulated attention weights [num_pages, Hkv, page_size]. Row b holds prefix_len[b] entries before
the round and num[b] of the round's N tokens (a chain of drafts, or a tree of candidates).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------

def case(name, op, B, N, Hq, Hkv, D, lo, hi, page, layout="hnd", dtype="bf16", **more):
    c = dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, page=page, layout=layout, dtype=dtype,
             tree=False)
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One user, one new token on a short context: the call's latency.
        case("attend_one_token_one_row", "attend", 1, 1, 32, 8, 128, 1023, 1023, 16),
        # A decode step of a serving batch: one token a row, contexts of very different lengths.
        case("attend_decode_batch", "attend", 64, 1, 32, 8, 128, 17, 8191, 16),
        # One long document, a single sequence split over the whole GPU; heads of 64.
        case("attend_long_context", "attend", 1, 5, 16, 2, 64, 262000, 262000, 64, "nhd", "f16"),
        # The verification pass of a batch with eight drafts a row, ragged draft lengths.
        case("attend_round_batch", "attend", 64, 9, 32, 8, 128, 100, 8000, 32),
        # Verification of candidate trees of 31 nodes a row, eight query heads to a key head.
        case("attend_tree_batch", "attend", 24, 31, 32, 4, 128, 500, 6000, 16, "nhd", tree=True),
        # The weight that the kept tokens of a round gave to every entry: one row, then a batch.
        case("weigh_one_row", "weigh", 1, 5, 32, 8, 128, 3001, 3001, 16),
        case("weigh_round_batch", "weigh", 64, 9, 32, 8, 128, 100, 8000, 32, dtype="f16"),
        # A few rows just over their budget, and a batch cut to half of its long contexts.
        case("evict_few_rows", "evict", 3, 1, 8, 8, 128, 1030, 1501, 16, budget=1024, recent=100),
        case("evict_batch_to_half", "evict", 32, 1, 8, 8, 128, 2000, 8190, 16, "nhd", budget=2048,
             recent=256),
        case("evict_one_head", "evict", 16, 1, 1, 1, 64, 5000, 16000, 64, budget=4096, recent=64,
             dtype="f16"),
        # A decode step's keys and values, and those of a batch's kept tree paths.
        case("append_decode", "append", 64, 1, 32, 8, 128, 17, 8191, 16),
        case("append_paths", "append", 512, 31, 32, 8, 128, 10, 300, 16, "nhd", tree=True),
    ]


def draw(rng):
    spread = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["attend", "attend", "attend", "weigh", "evict", "append"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    page = rng.choice([16, 16, 32, 64, 128])
    layout, dtype = rng.choice(["hnd", "nhd"]), rng.choice(["bf16", "bf16", "f16"])
    tree = False
    if op == "evict":
        group, N = 1, 1
    elif rng.random() < 0.3:
        N, tree = rng.randint(2, 65), op in ("attend", "append")
    else:
        N = rng.randint(1, 9)
    hi = spread(20, 60000)
    # Entries of all rows times heads and their width, held below the largest listed cases.
    most = 64 * 3000 * 8 * 128 // (hi * Hkv * D)
    if op == "attend" and N * group > 72:
        most = most * 72 // (N * group)
    B = spread(1, max(1, min(200, most)))
    c = case(None, op, B, N, Hkv * group, Hkv, D, max(1, int(hi * rng.uniform(0.02, 1.0))), hi, page,
             layout, dtype, tree=tree)
    if op == "evict":
        c["budget"] = max(2, int(hi * rng.uniform(0.3, 0.95)))
        c["recent"] = int(c["budget"] * rng.choice([0.0, 0.05, 0.25, 1.0]))
    return c


def lengths(c):
    """Per row: the entries before the round, and the round's tokens (both by the case alone)."""
    prefix, num = [], []
    for b in range(c["B"]):
        f = (0.5 + b * 0.6180339887498949) % 1.0
        prefix.append(c["lo"] + int(round((c["hi"] - c["lo"]) * f)))
        num.append(c["N"] - int((c["N"] * 0.75) * ((0.37 + b * 0.7548776662466927) % 1.0)))
    return prefix, num


def parents_of(c):
    """Candidate trees [B, N]: each node hangs on one of the nodes shortly before it."""
    g = np.random.RandomState(c["B"] * 131 + c["N"])
    p = np.full((c["B"], c["N"]), -1, np.int32)
    for i in range(1, c["N"]):
        p[:, i] = np.maximum(0, i - 1 - g.randint(0, 6, c["B"]))
    return p


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------

def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = TYPES[c["dtype"]]
    B, N, H, D, ps = c["B"], c["N"], c["Hkv"], c["D"], c["page"]
    prefix, num = lengths(c)
    ends = [p + (0 if c["op"] == "evict" else N) for p in prefix]
    pages = [-(-e // ps) for e in ends]
    max_pages, total = max(pages), sum(pages) + 3
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    used = torch.tensor(pages, device=dev)
    first = torch.cumsum(used, 0) - used
    at = torch.arange(max_pages, device=dev)
    table = torch.where(at[None] < used[:, None],
                        perm[(first[:, None] + at[None]).clamp(max=total - 1)], 0).to(torch.int32)
    shape = (total, H, ps, D) if c["layout"] == "hnd" else (total, ps, H, D)

    def pool(channels):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(t)
        if channels is not None:
            x *= channels.to(t)
        return x if c["layout"] == "hnd" else x.transpose(1, 2)

    # Keys have a few channels that are larger than the others.
    loud = torch.exp(0.5 * torch.randn((D,), generator=g, device=dev))
    s = dict(case=c, k=pool(loud / loud.square().mean().sqrt()), v=pool(None), table=table,
             prefix=torch.tensor(prefix, dtype=torch.int32, device=dev),
             num=torch.tensor(num, dtype=torch.int32, device=dev), parents=None)
    if c["tree"]:
        s["parents"] = torch.from_numpy(parents_of(c)).to(dev)
    heads = c["Hq"] + 2 * H
    # The round's queries, keys and values as one projection writes them: [B, N, Hq + 2 Hkv, D].
    qkv = torch.randn((B, N, heads, D), generator=g, device=dev, dtype=torch.float32)
    qkv[:, :, :c["Hq"]] *= 2.0
    qkv = qkv.to(t)
    s["q"] = qkv[:, :, :c["Hq"]]
    s["k_new"], s["v_new"] = qkv[:, :, c["Hq"]:c["Hq"] + H], qkv[:, :, c["Hq"] + H:]
    if c["op"] in ("weigh", "evict"):
        # What entries have gathered so far: most little, a few much.
        w = torch.rand((total, H, ps), generator=g, device=dev).clamp(min=1e-7)
        s["weight"] = 0.05 / w
    if c["op"] == "weigh":
        s["lse"] = plain_attend(s)[1]
    if c["op"] == "append":
        s["weight"] = torch.rand((total, H, ps), generator=g, device=dev)
        s["path"] = None
        if c["tree"]:     # a path of ascending nodes for each row, root first
            r = torch.rand((B, N), generator=g, device=dev)
            r[:, 0] = -1.0
            take = torch.argsort(r, dim=1)
            k = torch.arange(N, device=dev)[None] < s["num"][:, None]
            take = torch.where(k, take, N)
            take = torch.sort(take, dim=1)[0]
            s["path"] = torch.where(take < N, take, -1).to(torch.int32)
    if own:
        import speculative_decoding_verification_55_gb300 as sv
        s["cache"] = sv.PagedCache(s["k"], s["v"], s["table"], s.get("weight"))
        s["out_len"] = torch.empty((B,), dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import speculative_decoding_verification_55_gb300 as sv
        c, cache = s["case"], s["cache"]
        if op == "attend":
            return sv.attend(s["q"], cache, s["prefix"], s["num"], s["parents"])
        if op == "weigh":
            sv.spec_verify_kv_weights(s["q"], s["lse"], cache, s["prefix"], s["num"])
            return s["weight"]
        if op == "evict":
            sv.spec_verify_kv_evict(cache, s["prefix"], c["budget"], c["recent"], s["out_len"])
            return s["k"], s["v"], s["weight"], s["out_len"]
        sv.spec_verify_kv_append(s["k_new"], s["v_new"], cache, s["prefix"], s["num"], s["path"],
                                 s["out_len"])
        return s["k"], s["v"], s["weight"], s["out_len"]
    return {"attend": plain_attend, "weigh": plain_weigh, "evict": plain_evict,
            "append": plain_append}[op](s)


def places(s, L):
    """Page and slot of entries 0..L-1 of every row, [B, L] each."""
    ps = s["case"]["page"]
    j = torch.arange(L, device=s["k"].device)
    page = s["table"][:, (j // ps).clamp(max=s["table"].shape[1] - 1)].long()
    return page, (j % ps)[None].expand_as(page)


def gathered(pages, page, slot):
    """Entries of every row and head: [B, L, H, ...]."""
    h = torch.arange(pages.shape[1], device=pages.device)
    return pages[page[..., None], h, slot[..., None]]


def visible(s, L):
    """Which entries each of the round's tokens attends: [B, N, L]."""
    c = s["case"]
    j = torch.arange(L, device=s["k"].device)
    i = torch.arange(c["N"], device=s["k"].device)
    at = j[None] - s["prefix"][:, None]                            # place in the round, [B, L]
    if s["parents"] is None:
        return at[:, None] <= i[None, :, None]
    # A node sees itself and all above it: the parent relation, squared until it reaches the root.
    seen = ((s["parents"][:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (c["N"] - 1).bit_length())):
        seen = (torch.matmul(seen, seen) > 0).float()
    seen = seen.bool()
    inside = (at >= 0) & (at < c["N"])
    tail = torch.gather(seen, 2, at.clamp(0, c["N"] - 1)[:, None].expand(-1, c["N"], -1))
    return (at < 0)[:, None] | (inside[:, None] & tail)


def scores(s, L, page, slot):
    """Scaled scores [B, Hkv, N, group, L] in fp32, -inf where a token does not look."""
    c = s["case"]
    B, N, H, D = c["B"], c["N"], c["Hkv"], c["D"]
    k = gathered(s["k"], page, slot).float()                        # [B, L, H, D]
    q = s["q"].float().reshape(B, N, H, c["Hq"] // H, D).permute(0, 2, 1, 3, 4)
    x = torch.matmul(q.reshape(B, H, -1, D), k.permute(0, 2, 3, 1)) / math.sqrt(D)
    return x.reshape(B, H, N, -1, L)


def plain_attend(s):
    c = s["case"]
    B, N, H, D = c["B"], c["N"], c["Hkv"], c["D"]
    L = s["table"].shape[1] * c["page"]
    page, slot = places(s, L)
    see = visible(s, L) & (torch.arange(N, device=page.device)[None, :, None] < s["num"][:, None, None])
    x = scores(s, L, page, slot).masked_fill_(~see[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.where(m > -math.inf, x.sub_(m), -math.inf).exp_()
    total = x.sum(-1, keepdim=True)
    lse = torch.where(total > 0, m + torch.log(total), 0.0)
    v = gathered(s["v"], page, slot).float()
    inside = torch.arange(L, device=page.device)[None] < (s["prefix"] + s["num"])[:, None]
    v = torch.where(inside[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)
    o = torch.matmul(x.reshape(B, H, -1, L), v).reshape(B, H, N, -1, D) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, c["Hq"], D).to(s["k"].dtype)
    return o, lse.squeeze(-1).permute(0, 2, 1, 3).reshape(B, N, c["Hq"])


def plain_weigh(s):
    """Token d of the round's num[b] kept ones attended the entries before prefix_len[b] + d + 1."""
    c = s["case"]
    B, N, H = c["B"], c["N"], c["Hkv"]
    L = s["table"].shape[1] * c["page"]
    page, slot = places(s, L)
    lse = s["lse"].reshape(B, N, H, -1).permute(0, 2, 1, 3)[..., None]
    kept = torch.arange(N, device=page.device)[None, :, None] < s["num"][:, None, None]
    see = (visible(s, L) & kept)[:, None, :, None]
    p = torch.where(see, torch.exp(scores(s, L, page, slot) - lse), 0.0).sum((2, 3))     # [B, H, L]
    inside = torch.arange(L, device=page.device)[None] < (s["prefix"] + s["num"])[:, None]
    b, j = torch.nonzero(inside, as_tuple=True)
    h = torch.arange(H, device=page.device)
    s["weight"].index_put_((page[b, j][:, None], h[None], slot[b, j][:, None]), p[b, :, j],
                           accumulate=True)
    return s["weight"]


def plain_evict(s):
    """Of a row with more than `budget` entries the last `recent` stay and, per head, of the others the
    budget - recent with the largest weight (of equal ones the first); they move up in their order."""
    c = s["case"]
    H = c["Hkv"]
    n, budget, recent = s["prefix"], c["budget"], c["recent"]
    L = s["table"].shape[1] * c["page"]
    page, slot = places(s, L)
    j = torch.arange(L, device=page.device)
    w = gathered(s["weight"], page, slot).permute(0, 2, 1)                          # [B, H, L]
    old = (j[None] < (n - recent)[:, None])[:, None].expand_as(w)
    order = torch.sort(torch.where(old, w, -math.inf), dim=2, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(2, order, j.expand_as(order))
    keep = (old & (rank < budget - recent)) | (~old & (j[None] < n[:, None])[:, None])
    keep = torch.where((n > budget)[:, None, None], keep, (j[None] < n[:, None])[:, None])
    src = torch.sort((~keep).to(torch.int8), dim=2, stable=True)[1][:, :, :budget]  # kept ones, in order
    new_len = torch.minimum(n, torch.full_like(n, budget))
    inside = (j[None, :src.shape[2]] < new_len[:, None])[:, None].expand_as(src)
    b, h, d = torch.nonzero(inside, as_tuple=True)
    a = src[b, h, d]
    frm, to = (page[b, a], h, slot[b, a]), (page[b, d], h, slot[b, d])
    for x in (s["k"], s["v"], s["weight"]):
        x[to] = x[frm]
    return s["k"], s["v"], s["weight"], new_len


def plain_append(s):
    c = s["case"]
    L = s["table"].shape[1] * c["page"]
    page, slot = places(s, L)
    h = torch.arange(c["Hkv"], device=page.device)[None]
    b, d = torch.nonzero(torch.arange(c["N"], device=page.device)[None] < s["num"][:, None], as_tuple=True)
    i = d if s["path"] is None else s["path"][b, d].long()
    j = s["prefix"][b].long() + d
    to = (page[b, j][:, None], h, slot[b, j][:, None])
    s["k"][to] = s["k_new"][b, i]
    s["v"][to] = s["v_new"][b, i]
    s["weight"][to] = 0.0
    return s["k"], s["v"], s["weight"], s["prefix"] + s["num"]


# ------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------------

def work(case):
    c = case
    prefix, num = lengths(c)
    row = c["Hkv"] * c["D"] * 2                           # one entry's keys (or values), all heads
    entries = sum(p + k for p, k in zip(prefix, num))
    q = sum(num) * c["Hq"] * c["D"] * 2
    pairs = sum(k * (p + (k + 1) / 2) for p, k in zip(prefix, num)) * c["Hq"]
    if c["op"] == "attend":
        return {"bytes": 2 * entries * row + 2 * q + sum(num) * c["Hq"] * 4, "flops": 4 * pairs * c["D"]}
    if c["op"] == "weigh":
        return {"bytes": entries * row + q + sum(num) * c["Hq"] * 4 + 2 * entries * c["Hkv"] * 4,
                "flops": 2 * pairs * c["D"]}
    if c["op"] == "evict":
        # Weights read and written; the kept entries behind a row's first dropped one move, and that
        # lies, of equally likely ones, at about (old + 1) / (dropped + 1).
        seen = sum(p for p in prefix if p > c["budget"])
        moved = sum(c["budget"] - min(c["budget"], (p - c["recent"] + 1) // (p - c["budget"] + 1) - 1)
                    for p in prefix if p > c["budget"])
        return {"bytes": seen * c["Hkv"] * 4 + moved * (c["Hkv"] * 4 + 4 * row), "flops": 0}
    return {"bytes": sum(num) * (4 * row + c["Hkv"] * 4), "flops": 0}


# ------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ------------------------------------------------------------------------------------------------

def row_entries(pages, table_row, n, ps):
    """The first n entries of a row in order, [H, n, ...]."""
    ids = table_row[:-(-n // ps)].long()
    x = pages[ids].transpose(0, 1)                        # [H, pages, slots, ...]
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :n]


def put_entries(pages, table_row, lo, x, ps):
    """Writes x [H, m, ...] to the entries lo.. of a row."""
    for a in range(x.shape[1]):
        j = lo + a
        pages[int(table_row[j // ps]), :, j % ps] = x[:, a]


def ancestors(par, i):
    line = [i]
    while par[line[-1]] >= 0:
        line.append(int(par[line[-1]]))
    return line


def exact(case, seed):
    c = case
    prefix, num = lengths(c)
    H, D, ps, N = c["Hkv"], c["D"], c["page"], c["N"]
    G = c["Hq"] // H
    if c["op"] in ("evict", "append"):                    # moved, not computed
        return None
    s = prepare(c, seed)
    tab = s["table"]
    out = torch.zeros((c["B"], N, H, G, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["B"], N, H, G), dtype=torch.float64, device="cuda")
    weight = s["weight"].double() if c["op"] == "weigh" else None
    par = parents_of(c) if c["tree"] else None
    for b, (p, k) in enumerate(zip(prefix, num)):
        n = p + k
        see = torch.ones((k, n), dtype=torch.bool)
        for i in range(k):
            see[i, p:] = False
            see[i, [p + a for a in (ancestors(par[b], i) if c["tree"] else range(i + 1))]] = True
        see = see.cuda()
        K = row_entries(s["k"], tab[b], n, ps).double()
        q = s["q"][b, :k].double().reshape(k, H, G, D).permute(1, 0, 2, 3)
        x = (q.reshape(H, k * G, D) @ K.transpose(1, 2)).reshape(H, k, G, n) * D ** -0.5
        x = x.masked_fill(~see[None, :, None], -math.inf)
        if c["op"] == "weigh":
            given = s["lse"][b, :k].double().reshape(k, H, G).permute(1, 0, 2)
            w = torch.exp(x - given[..., None]).sum((1, 2))
            ids = tab[b][:-(-n // ps)].long()
            pad = torch.zeros((H, len(ids) * ps), dtype=torch.float64, device="cuda")
            pad[:, :n] = w
            weight.index_add_(0, ids, pad.reshape(H, len(ids), ps).transpose(0, 1))
            continue
        z = torch.logsumexp(x, -1)
        V = row_entries(s["v"], tab[b], n, ps).double()
        o = torch.exp(x - z[..., None]).reshape(H, k * G, n) @ V
        out[b, :k] = o.reshape(H, k, G, D).permute(1, 0, 2, 3)
        lse[b, :k] = z.permute(1, 0, 2)
    if c["op"] == "weigh":
        return weight
    return out.reshape(c["B"], N, c["Hq"], D), lse.reshape(c["B"], N, c["Hq"])
