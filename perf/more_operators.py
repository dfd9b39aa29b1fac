"""What a serving batch adds to a round, measured: attention of rows that share the front of their
contexts (a common prompt or document), the shaping of a round's logits before they are verified
(penalties for repeated tokens, biases, grammar masks), and the token counts that penalties read.

Attention: pages [num_pages, Hkv, page_size, D] (or slots before heads), a page table [B, max_pages]; row b
holds prefix_len[b] entries before the round and the round's num[b] of N tokens. Rows group_start[g] up to
group_start[g + 1] - 1 have their first shared_len[b] entries, whole pages, in common: their page tables
begin with the same pages.

Logits [B, N, V]: position i of row b follows the row's own text and the round's tokens before position i
(a chain of drafts: tokens 0 .. i - 1; a tree: the node's ancestors and itself). counts [B, V] int16 hold the
text: 32768 (the sign) for a token of the prompt, plus its occurrences in the output.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------

def shared(name, B, G, lone, N, Hq, Hkv, D, slo, shi, olo, ohi, page, layout="hnd", dtype="bf16", tree=False):
    """G groups and `lone` rows in none; shared entries slo..shi a group, own ones olo..ohi a row."""
    c = dict(op="shared", B=B, G=G, lone=lone, N=N, Hq=Hq, Hkv=Hkv, D=D, slo=slo, shi=shi, olo=olo, ohi=ohi,
             page=page, layout=layout, dtype=dtype, tree=tree)
    if name:
        c["name"] = name
    return c


def shape(name, B, N, V, dtype="bf16", history=1000, mask="none", width=100, bias=0, tree=False):
    """mask: narrow (`width` tokens allowed), open (`width` tokens barred), even (half of them) or none."""
    c = dict(op="shape", B=B, N=N, V=V, dtype=dtype, history=history, mask=mask, width=width, bias=bias, tree=tree)
    if name:
        c["name"] = name
    return c


def count(name, B, M, V, prompt):
    c = dict(op="count", B=B, M=M, V=V, prompt=prompt)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # Four answers to one question, a token each: the call's latency.
        shared("shared_four_answers", 4, 1, 0, 1, 32, 8, 128, 1024, 1024, 3, 50, 16),
        # A decode step of a batch that serves one product: the same long instructions for everyone.
        shared("shared_decode_batch", 64, 1, 0, 1, 32, 8, 128, 8000, 8000, 17, 1000, 16),
        # The verification pass of two products' batches with eight drafts a row, and of some other rows.
        shared("shared_round_batch", 64, 2, 6, 9, 32, 8, 128, 3000, 6000, 100, 1000, 32),
        # Candidate trees of 31 nodes a row over three shared documents.
        shared("shared_tree_batch", 24, 3, 0, 31, 32, 4, 128, 2000, 5000, 100, 1500, 16, "nhd", tree=True),
        # Many small groups (samples of one question each) with heads of 64.
        shared("shared_many_groups", 200, 40, 10, 5, 16, 2, 64, 300, 2500, 20, 400, 64, "nhd", "f16"),
        # Questions about one very long document, one key head of 256.
        shared("shared_long_document", 8, 1, 0, 1, 8, 1, 256, 131072, 131072, 5, 300, 64),
        # One row's next token with a grammar: the call's latency.
        shape("shape_one_row", 1, 1, 32000, "f32", 500, "narrow", 40, 8),
        # A round of a batch, penalties alone, logits in fp32.
        shape("shape_penalties", 256, 8, 152064, "f32", 4000),
        # A round of a batch that answers in a grammar: few tokens allowed at each position.
        shape("shape_narrow_masks", 64, 6, 128256, "bf16", 2000, "narrow", 300, 16),
        # Candidate trees inside a string of such an answer: nearly every token is allowed.
        shape("shape_open_masks_tree", 32, 31, 128256, "bf16", 2000, "open", 400, 0, True),
        # The tokens that a round emitted, and prompts of new requests.
        count("count_emitted", 1024, 9, 256000, False),
        count("count_prompts", 64, 30000, 128256, True),
    ]


def draw(rng):
    spread = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["shared", "shared", "shared", "shape", "shape", "shape", "count"])
    if op == "shared":
        D, Hkv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
        tree = rng.random() < 0.25
        N = rng.randint(2, 65) if tree else rng.randint(1, 9)
        shi, ohi = spread(20, 60000), spread(1, 3000)
        # Entries of all rows with their heads, and the products of all query rows, stay below the listed ones'.
        most = min(64 * 9000 * 8 * 128 // ((shi + ohi) * Hkv * D),
                   64 * 9 * 32 * 7000 * 128 // ((shi + ohi) * Hkv * group * N * D))
        B = spread(1, max(1, min(300, most)))
        lone = rng.randint(0, B) if rng.random() < 0.4 else 0
        G = spread(1, max(1, B - lone))
        return shared(None, B, G, lone, N, Hkv * group, Hkv, D, max(1, int(shi * rng.uniform(0.1, 1.0))), shi,
                      max(1, int(ohi * rng.uniform(0.02, 1.0))), ohi, rng.choice([16, 16, 32, 64, 128]),
                      rng.choice(["hnd", "nhd"]), rng.choice(["bf16", "bf16", "f16"]), tree)
    V = rng.choice([256, 32000, 128256, 152064, 256000, spread(100, 256000)])
    if op == "count":
        prompt = rng.random() < 0.5
        M = spread(1, 30000) if prompt else rng.randint(1, 66)
        return count(None, spread(1, max(1, min(1024, 250000000 // V, 2500000 // M))), M, V, prompt)
    tree = rng.random() < 0.25
    N = rng.randint(2, 65) if tree else rng.randint(1, 9)
    B = spread(1, max(1, min(1024, 300000000 // (N * V))))
    return shape(None, B, N, V, rng.choice(["bf16", "bf16", "f32"]), spread(1, 30000),
                 rng.choice(["narrow", "open", "even", "none", "none"]), spread(1, max(1, min(3000, V // 4))),
                 rng.choice([0, 0, rng.randint(1, 300)]), tree)


def spaced(i, step):
    """Numbers spread over [0, 1), the same ones for the same case."""
    return (0.5 + i * step) % 1.0


def groups(c):
    """Per group its first row (and the end of the last), and per row the shared entries, those before the
    round and the round's tokens (all by the case alone). Lone rows come first and last."""
    B, G, ps = c["B"], c["G"], c["page"]
    inside = B - c["lone"]
    G = min(G, max(1, inside))
    weights = [0.2 + spaced(g, 0.6180339887498949) for g in range(G)]
    start, at = [], 0.0
    front = c["lone"] // 2
    for g in range(G + 1):
        start.append(front + int(round(inside * at / sum(weights))))
        at += weights[g] if g < G else 0.0
    common, prefix, num = [0] * B, [], []
    for g in range(G):
        s = c["slo"] + int(round((c["shi"] - c["slo"]) * spaced(g, 0.7548776662466927)))
        for b in range(start[g], start[g + 1]):
            common[b] = -(-s // ps) * ps
    for b in range(B):
        prefix.append(common[b] + c["olo"] + int(round((c["ohi"] - c["olo"]) * spaced(b, 0.6180339887498949))))
        num.append(c["N"] - int((c["N"] * 0.75) * ((0.37 + b * 0.7548776662466927) % 1.0)))
    return start, common, prefix, num


def positions(c):
    return [c["N"] - int((c["N"] * 0.75) * ((0.37 + b * 0.7548776662466927) % 1.0)) for b in range(c["B"])]


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
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"shared": prepare_shared, "shape": prepare_shape, "count": prepare_count}[case["op"]](case, g)


def prepare_shared(c, g):
    dev, t = "cuda", TYPES[c["dtype"]]
    B, N, H, D, ps = c["B"], c["N"], c["Hkv"], c["D"], c["page"]
    start, common, prefix, num = groups(c)
    pages = [-(-(p + N) // ps) for p in prefix]
    max_pages = max(pages) + 2
    table = np.zeros((B, max_pages), np.int64)
    total, of_group = 0, {}
    for b in range(B):
        front = common[b] // ps
        if front:
            first = max(x for x in start[:-1] if x <= b)
            if first not in of_group:
                of_group[first] = np.arange(total, total + front)
                total += front
            table[b, :front] = of_group[first]
        table[b, front:pages[b]] = np.arange(total, total + pages[b] - front)
        total += pages[b] - front
    total += 3
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    held = torch.arange(max_pages, device=dev)[None] < torch.tensor(pages, device=dev)[:, None]
    table = torch.where(held, perm[torch.from_numpy(table).to(dev)], 0).to(torch.int32)
    shape = (total, H, ps, D) if c["layout"] == "hnd" else (total, ps, H, D)

    def pool(channels):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(t)
        if channels is not None:
            x *= channels.to(t)
        return x if c["layout"] == "hnd" else x.transpose(1, 2)

    # Keys have a few channels that are larger than the others.
    loud = torch.exp(0.5 * torch.randn((D,), generator=g, device=dev))
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case=c, k=pool(loud / loud.square().mean().sqrt()), v=pool(None), table=table,
             prefix=torch.tensor(prefix, **i32), num=torch.tensor(num, **i32),
             start=torch.tensor(start, **i32), common=torch.tensor(common, **i32), parents=None)
    if c["tree"]:
        s["parents"] = torch.from_numpy(parents_of(c)).to(dev)
    # The round's queries, keys and values as one projection writes them: [B, N, Hq + 2 Hkv, D].
    qkv = torch.randn((B, N, c["Hq"] + 2 * H, D), generator=g, device=dev, dtype=torch.float32)
    qkv[:, :, :c["Hq"]] *= 2.0
    s["q"] = qkv.to(t)[:, :, :c["Hq"]]
    if own:
        import speculative_decoding_verification_55_gb300 as sv
        s["cache"] = sv.PagedCache(s["k"], s["v"], s["table"])
    return s


def text(shape, V, g):
    """Tokens as texts have them: the frequent ones have low numbers."""
    u = torch.rand(shape, generator=g, device="cuda")
    return torch.exp(u * math.log(V)).long().sub_(1).clamp_(0, V - 1)


def packed(allowed):
    """[B, N, V] truth values as words of 32 bits, the lowest bit first."""
    B, N, V = allowed.shape
    allowed = torch.nn.functional.pad(allowed, (0, -V % 32))
    words = torch.zeros((B, N, allowed.shape[2] // 32), dtype=torch.int32, device=allowed.device)
    for k in range(32):
        words |= allowed[:, :, k::32].int() << k
    return words


def prepare_shape(c, g):
    dev, B, N, V = "cuda", c["B"], c["N"], c["V"]
    logits = torch.randn((B, N, V), generator=g, device=dev)
    logits.mul_(2.5).sub_(1.1 * torch.log(1.0 + torch.arange(V, device=dev)))
    s = dict(case=c, logits=logits.to(TYPES[c["dtype"]]), parents=None, mask=None, bias_tokens=None, bias=None)
    del logits
    s["num"] = torch.tensor(positions(c), dtype=torch.int32, device=dev)
    # The round's tokens: what the drafter found likely, some of it in the text before.
    s["tokens"] = text((B, N), V, g).to(torch.int32)
    if c["tree"]:
        s["parents"] = torch.from_numpy(parents_of(c)).to(dev)
    half = max(1, c["history"] // 2)
    counts = torch.zeros((B, V), dtype=torch.int32, device=dev)
    counts.scatter_add_(1, text((B, half), V, g), torch.ones((B, half), dtype=torch.int32, device=dev))
    prompt = torch.zeros((B, V), dtype=torch.bool, device=dev)
    prompt.scatter_(1, text((B, half), V, g), True)
    s["counts"] = torch.where(prompt, counts - 32768, counts).to(torch.int16)
    u = torch.rand((3, B), generator=g, device=dev)
    s["repetition"] = 1.0 + 0.3 * u[0]
    s["frequency"], s["presence"] = 0.5 * u[1], 0.6 * u[2]
    if c["bias"]:
        s["bias_tokens"] = torch.randint(0, V, (B, c["bias"]), generator=g, device=dev, dtype=torch.int32)
        s["bias"] = 4.0 * torch.randn((B, c["bias"]), generator=g, device=dev)
    if c["mask"] == "even":
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, N, -(-V // 32)), generator=g, device=dev, dtype=torch.int32)
    elif c["mask"] != "none":
        narrow = c["mask"] == "narrow"
        allowed = torch.full((B, N, V), not narrow, dtype=torch.bool, device=dev)
        allowed.scatter_(2, torch.randint(0, V, (B, N, c["width"]), generator=g, device=dev), narrow)
        s["mask"] = packed(allowed)
    return s


def prepare_count(c, g):
    dev, B, M, V = "cuda", c["B"], c["M"], c["V"]
    tokens = text((B, M), V, g).to(torch.int32)
    lo = 0.2 if c["prompt"] else 0.0
    num = (1 + (M - 1) * (lo + (1 - lo) * torch.rand((B,), generator=g, device=dev))).round().to(torch.int32)
    used = torch.arange(M, device=dev)[None] < num[:, None]
    s = dict(case=c, tokens=torch.where(used, tokens, -1), num=num)
    s["counts"] = torch.zeros((B, V), dtype=torch.int16, device=dev)
    if not c["prompt"]:
        s["counts"].scatter_(1, text((B, 500), V, g), 3)
        s["counts"].scatter_(1, text((B, 500), V, g), -32768)
    return s


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import speculative_decoding_verification_55_gb300 as sv
        if op == "shared":
            return sv.attend_shared(s["q"], s["cache"], s["prefix"], s["common"], s["start"], s["num"], s["parents"])
        if op == "shape":
            sv.spec_verify_shape_logits(s["logits"], num_positions=s["num"], tokens=s["tokens"],
                                        tree_parents=s["parents"], counts=s["counts"], repetition=s["repetition"],
                                        frequency=s["frequency"], presence=s["presence"],
                                        bias_tokens=s["bias_tokens"], bias=s["bias"], mask=s["mask"])
            return s["logits"]
        sv.spec_verify_count_tokens(s["tokens"], s["num"], s["counts"], s["case"]["prompt"])
        return s["counts"]
    return {"shared": plain_attend, "shape": plain_shape, "count": plain_count}[op](s)


def seen_in_tree(parents, N):
    """Which nodes a node has above it or is, [B, N, N]: the parent relation, squared until it is all in."""
    i = torch.arange(N, device=parents.device)
    seen = ((parents[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (N - 1).bit_length())):
        seen = (torch.matmul(seen, seen) > 0).float()
    return seen.bool()


def plain_attend(s):
    c = s["case"]
    B, N, H, D = c["B"], c["N"], c["Hkv"], c["D"]
    dev, L = s["q"].device, s["table"].shape[1] * c["page"]
    j, i = torch.arange(L, device=dev), torch.arange(N, device=dev)
    page, slot = s["table"][:, j // c["page"]].long(), (j % c["page"])[None].expand(B, L)
    h = torch.arange(H, device=dev)
    k = s["k"][page[..., None], h, slot[..., None]].float()              # [B, L, H, D]
    at = j[None] - s["prefix"][:, None]                                  # place in the round
    if s["parents"] is None:
        see = at[:, None] <= i[None, :, None]
    else:
        tail = torch.gather(seen_in_tree(s["parents"], N), 2, at.clamp(0, N - 1)[:, None].expand(-1, N, -1))
        see = (at < 0)[:, None] | (((at >= 0) & (at < N))[:, None] & tail)
    see = see & (i[None, :, None] < s["num"][:, None, None])             # [B, N, L]
    q = s["q"].float().reshape(B, N, H, -1, D).permute(0, 2, 1, 3, 4)
    x = torch.matmul(q.reshape(B, H, -1, D), k.permute(0, 2, 3, 1)) / math.sqrt(D)
    del k
    x = x.reshape(B, H, N, -1, L).masked_fill_(~see[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.where(m > -math.inf, x.sub_(m), -math.inf).exp_()
    total = x.sum(-1, keepdim=True)
    lse = torch.where(total > 0, m + torch.log(total), 0.0)
    v = s["v"][page[..., None], h, slot[..., None]].float()
    inside = j[None] < (s["prefix"] + s["num"])[:, None]
    v = torch.where(inside[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)
    o = torch.matmul(x.reshape(B, H, -1, L), v).reshape(B, H, N, -1, D) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, c["Hq"], D).to(s["q"].dtype)
    return o, lse.squeeze(-1).permute(0, 2, 1, 3).reshape(B, N, c["Hq"])


def plain_shape(s):
    c, z = s["case"], s["logits"]
    B, N, V = z.shape
    dev = z.device
    i = torch.arange(N, device=dev)
    before = (i[None] < i[:, None])[None].expand(B, N, N) if s["parents"] is None else seen_in_tree(s["parents"], N)
    counts = s["counts"].int()
    uses = (counts & 32767)[:, None].expand(B, N, V).float()             # a copy below
    uses = uses.scatter_add(2, s["tokens"].long()[:, None].expand(B, N, N), before.float())
    seen = (uses > 0) | (counts < 0)[:, None]
    x = z.float()
    r = s["repetition"][:, None, None]
    y = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    y -= s["frequency"][:, None, None] * uses
    y -= torch.where(uses > 0, s["presence"][:, None, None], 0.0)
    if s["bias"] is not None:
        bias = torch.zeros((B, V), device=dev).scatter_add_(1, s["bias_tokens"].long(), s["bias"])
        y += bias[:, None]
    if s["mask"] is not None:
        v = torch.arange(V, device=dev)
        y = torch.where((s["mask"][:, :, v // 32] >> (v % 32).int()) & 1 != 0, y, -math.inf)
    s["logits"].copy_(torch.where((i[None] < s["num"][:, None])[..., None], y, x))
    return s["logits"]


def plain_count(s):
    c, counts = s["case"], s["counts"]
    M = c["M"]
    used = torch.arange(M, device=counts.device)[None] < s["num"][:, None]
    used = used & (s["tokens"] >= 0) & (s["tokens"] < c["V"])
    at = torch.where(used, s["tokens"], 0).long()
    new = torch.zeros(counts.shape, dtype=torch.int32, device=counts.device).scatter_add_(1, at, used.int())
    old = counts.int()
    if c["prompt"]:
        out = torch.where(new > 0, (old & 32767) - 32768, old)
    else:
        out = ((old & 32767) + new).clamp_(max=32767)
        out = torch.where(old < 0, out - 32768, out)
    counts.copy_(out.to(torch.int16))
    return counts


# ------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "shared":
        start, common, prefix, num = groups(c)
        row = c["Hkv"] * c["D"] * 2                       # one entry's keys (or values), all heads
        first = {start[g] for g in range(len(start) - 1) if start[g] < start[g + 1]}
        entries = sum(p + k - s for p, k, s in zip(prefix, num, common)) + sum(common[b] for b in first)
        pairs = sum(k * (p + (k + 1) / 2) for p, k in zip(prefix, num)) * c["Hq"]
        q = sum(num) * c["Hq"] * c["D"] * 2
        return {"bytes": 2 * entries * row + 2 * q + sum(num) * c["Hq"] * 4, "flops": 4 * pairs * c["D"]}
    if c["op"] == "count":
        tokens = c["B"] * c["M"] * (0.6 if c["prompt"] else 0.5)
        return {"bytes": tokens * 4 + c["B"] * 4 + 4 * distinct(c["M"] * 0.6, c["V"]) * c["B"], "flops": 0}
    rows, V, size = sum(positions(c)), c["V"], 4 if c["dtype"] == "f32" else 2
    words = 0 if c["mask"] == "none" else rows * -(-V // 32) * 4
    open_ = {"none": 1.0, "even": 0.5, "open": 1.0 - c["width"] / V, "narrow": min(1.0, c["width"] / V)}[c["mask"]]
    touched = distinct(c["history"], V) + c["bias"]
    # The counts, the masks, the barred logits written, and the penalised or biased allowed ones read and written.
    return {"bytes": c["B"] * 2 * V + words + rows * V * (1 - open_) * size + 2 * rows * touched * open_ * size
            + c["B"] * 8 * c["bias"], "flops": 0}


def distinct(n, V):
    """Different ones among n tokens of `text`: token t has probability log((t + 2) / (t + 1)) / log(V)."""
    t = np.arange(1, V, dtype=np.float64)
    return float((1.0 - np.exp(n * np.log1p(-np.log1p(1.0 / t) / math.log(V)))).sum())


# ------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ------------------------------------------------------------------------------------------------

def ancestors(par, i):
    line = [i]
    while par[line[-1]] >= 0:
        line.append(int(par[line[-1]]))
    return line


def exact(case, seed):
    c = case
    if c["op"] == "count":                                # whole numbers
        return None
    s = prepare(c, seed)
    return exact_attend(c, s) if c["op"] == "shared" else exact_shape(c, s)


def exact_attend(c, s):
    _, _, prefix, num = groups(c)
    H, D, ps, N = c["Hkv"], c["D"], c["page"], c["N"]
    G = c["Hq"] // H
    out = torch.zeros((c["B"], N, H, G, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["B"], N, H, G), dtype=torch.float64, device="cuda")
    par = parents_of(c) if c["tree"] else None
    for b, (p, k) in enumerate(zip(prefix, num)):
        n = p + k
        see = torch.ones((k, n), dtype=torch.bool)
        for i in range(k):
            see[i, p:] = False
            see[i, [p + a for a in (ancestors(par[b], i) if c["tree"] else range(i + 1))]] = True
        ids = s["table"][b][:-(-n // ps)].long()

        def entries(pages):                               # the row's entries in order, [H, n, D]
            x = pages[ids].transpose(0, 1)
            return x.reshape(H, -1, D)[:, :n].double()

        q = s["q"][b, :k].double().reshape(k, H, G, D).permute(1, 0, 2, 3).reshape(H, k * G, D)
        x = (q @ entries(s["k"]).transpose(1, 2)).reshape(H, k, G, n) * D ** -0.5
        x = x.masked_fill(~see.cuda()[None, :, None], -math.inf)
        z = torch.logsumexp(x, -1)
        o = torch.exp(x - z[..., None]).reshape(H, k * G, n) @ entries(s["v"])
        out[b, :k] = o.reshape(H, k, G, D).permute(1, 0, 2, 3)
        lse[b, :k] = z.permute(1, 0, 2)
    return out.reshape(c["B"], N, c["Hq"], D), lse.reshape(c["B"], N, c["Hq"])


def exact_shape(c, s):
    B, N, V = c["B"], c["N"], c["V"]
    if B * N > 4000:
        return None
    z = s["logits"].double()
    par = parents_of(c) if c["tree"] else None
    tokens, words = s["tokens"].cpu().numpy(), s["mask"]
    pen = [s[x].cpu().double().tolist() for x in ("repetition", "frequency", "presence")]
    bit = torch.arange(32, device="cuda", dtype=torch.int32)
    for b, m in enumerate(positions(c)):
        r, f, p = (x[b] for x in pen)
        base = s["counts"][b].int()
        for i in range(m):
            said = [int(tokens[b, a]) for a in (ancestors(par[b], i) if par is not None else range(i))]
            n = (base & 32767).double()
            n.index_add_(0, torch.tensor(said, device="cuda", dtype=torch.long),
                         torch.ones(len(said), dtype=torch.float64, device="cuda"))
            at = torch.nonzero((n > 0) | (base < 0)).flatten()
            x, k = z[b, i, at], n[at]
            z[b, i, at] = torch.where(x > 0, x / r, x * r) - f * k - p * (k > 0)
            if s["bias"] is not None:
                z[b, i].index_add_(0, s["bias_tokens"][b].long(), s["bias"][b].double())
            if words is not None:
                barred = ((words[b, i][:, None] >> bit) & 1 == 0).flatten()[:V]
                z[b, i, barred] = -math.inf
    return z
