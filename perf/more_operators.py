"""Operators for many requests on one base model, as a serving program calls them, for timing and comparison.

  shared    attention of one new token per sequence where groups of sequences share a long prefix (a system
            prompt, a document), held once in the paged cache: each group's prefix is read once for all of it
  project   a projection shared by all requests, with the low-rank adapter of each request's own beside it
  logprobs  from rows of logits: the log probability and rank of a given token, the entropy, and the most
            probable tokens with their log probabilities

`run` computes the plain form in 32 bits, or calls the library where `own` is set; `exact` restates each
operator in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# (query heads, kv heads, head dim) of this repository's decoders and encoder, and plain multi-head attention
HEADS = [(14, 2, 64), (32, 8, 64), (16, 8, 128), (32, 8, 128), (8, 8, 128), (4, 2, 16)]
# (inputs, outputs) of their projections: fused q|k|v, o, fused gate|up, down
PROJECTIONS = [(896, 1152), (896, 896), (896, 9728), (4864, 896), (2048, 2048), (2048, 16384), (8192, 2048),
               (1024, 4096), (2048, 1024), (64, 128)]
VOCABS = [256, 32000, 50257, 128256, 151936]


def listed():
    share = dict(op="shared", page=16, row_major=False, type="bf16", groups=1)
    adapt = dict(op="project", type="bf16", out="same", bias=False, runs=False)
    score = dict(op="logprobs", type="f32", temperature=1.0, pad=0)
    return [
        # a few answers to one short prompt: latency
        dict(share, name="shared few", heads=14, kv_heads=2, dim=64, batch=4, prefix=700, tail=40),
        # the 64-sequence decode step of the 1B decoder under a common system prompt
        dict(share, name="shared batch 64", heads=32, kv_heads=8, dim=64, batch=64, prefix=8192, tail=512),
        # several documents with questions to each, prefixes that end inside pages
        dict(share, name="shared documents", heads=16, kv_heads=8, dim=128, batch=75, prefix=12001, tail=333, groups=5,
             type="f16", page=64, row_major=True),
        # many users on one very long context
        dict(share, name="shared long", heads=32, kv_heads=8, dim=128, batch=128, prefix=32768, tail=700, page=64),
        # one token of one request through a small projection: latency
        dict(adapt, name="project one row", inputs=896, outputs=1152, rows=1, rank=8, adapters=4, bias=True),
        # a decode step's widest projection, each request with an adapter of its own or none
        dict(adapt, name="project batch 64", inputs=2048, outputs=16384, rows=64, rank=16, adapters=40),
        # a ragged batch of prompts of several requests, rows of one request together
        dict(adapt, name="project prompts", inputs=1024, outputs=4096, rows=777, rank=32, adapters=9, type="f16", out="f32",
             runs=True),
        # a long prompt through the down projection
        dict(adapt, name="project prompt 4096", inputs=8192, outputs=2048, rows=4096, rank=64, adapters=3, runs=True),
        # the token just sampled, with alternatives
        dict(score, name="logprobs one row", rows=1, vocab=151936, top=5),
        # a decode step of 64 requests at the sampler's temperature
        dict(score, name="logprobs batch 64", rows=64, vocab=128256, top=20, temperature=0.7),
        # an odd vocabulary in padded rows
        dict(score, name="logprobs odd vocabulary", rows=517, vocab=50257, top=1, type="f16", pad=47),
        # a prompt's tokens scored at once
        dict(score, name="logprobs prompt", rows=2048, vocab=151936, top=10, type="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["shared", "project", "logprobs"])
    if op == "shared":
        heads, kv_heads, dim = rng.choice(HEADS)
        c = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                 row_major=rng.random() < 0.3, type=rng.choice(["bf16", "bf16", "f16"]), batch=log(1, 256),
                 prefix=log(1, 40000), tail=log(1, 3000))
        c["groups"] = min(c["batch"], rng.choice([1, 1, 2, 3, 8]))
        while c["batch"] * heads * dim * (c["prefix"] + c["tail"]) > 1.7e10 or c["batch"] * c["tail"] * heads * dim > 1.5e9:
            c["prefix"], c["tail"] = max(1, c["prefix"] * 4 // 5), max(1, c["tail"] * 2 // 3)
        return c
    if op == "project":
        inputs, outputs = rng.choice(PROJECTIONS)
        c = dict(op=op, inputs=inputs, outputs=outputs, rows=log(1, 4096), rank=rng.choice([8, 16, 32, 64, 128]),
                 adapters=log(1, 64), type=rng.choice(["bf16", "bf16", "f16"]), out=rng.choice(["same", "same", "f32"]),
                 bias=rng.random() < 0.4, runs=rng.random() < 0.5)
        while c["rows"] * inputs * outputs > 6.8e10:
            c["rows"] = c["rows"] * 2 // 3
        if c["rows"] > 512:
            c["runs"] = True          # prompts come as runs of rows
        return c
    c = dict(op=op, vocab=rng.choice(VOCABS), rows=log(1, 4096), top=rng.choice([0, 1, 5, 20, 32]),
             type=rng.choice(["f32", "f32", "bf16", "f16"]), temperature=rng.choice([1.0, 1.0, 0.7, 1.3]),
             pad=rng.choice([0, 0, 3, 64]))
    while c["rows"] * c["vocab"] > 3e8:
        c["rows"] = c["rows"] * 2 // 3
    return c


def spread(longest, n):
    """n lengths up to `longest`, spread over (0, longest], the first the longest."""
    return [min(longest, max(1, round(longest * (1.0 - (b * 0.6180339887) % 1.0)))) for b in range(n)]


def layout(case):
    """Per group its rows and shared keys; per row its own keys beyond them."""
    n, g = case["batch"], case["groups"]
    weight = spread(1000, g)
    rows = [1 + (n - g) * w // sum(weight) for w in weight]
    rows[0] += n - sum(rows)
    return rows, spread(case["prefix"], g), spread(case["tail"], n)


def owners(case):
    """The adapter of each row (-1: none), in no order or in runs of rows."""
    n, k = case["rows"], case["adapters"]
    if case["runs"]:
        parts = spread(1000, min(n, 2 * k + 1))
        out = [(p * 7) % (k + 1) - 1 if p else 0 for p, w in enumerate(parts) for _ in range(1 + n * w // sum(parts))]
        return (out + [k - 1] * n)[:n]
    return [(i * 2654435761 >> 7) % (k + 1) - 1 if i else 0 for i in range(n)]


def work(case):
    if case["op"] == "shared":
        nh, nk, d = case["heads"], case["kv_heads"], case["dim"]
        rows, shared, tails = layout(case)
        keys = sum(m * p for m, p in zip(rows, shared)) + sum(tails)
        return {"bytes": (sum(shared) + sum(tails)) * nk * d * 4 + case["batch"] * nh * (d * 4 + 4), "flops": 4 * nh * d * keys}
    if case["op"] == "project":
        k, n, m, r = case["inputs"], case["outputs"], case["rows"], case["rank"]
        who = owners(case)
        used, with_one = len({a for a in who if a >= 0}), sum(a >= 0 for a in who)
        return {"bytes": 2 * (n * k + used * r * (n + k) + m * k) + m * n * (4 if case["out"] == "f32" else 2)
                + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k + 2 * with_one * r * (n + k)}
    n, v = case["rows"], case["vocab"]
    return {"bytes": n * v * (4 if case["type"] == "f32" else 2) + n * (16 + 8 * case["top"]), "flops": 8 * n * v}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["type"]]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = {"case": case}
    if case["op"] == "shared":
        nh, nk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
        rows, shared, tails = layout(case)
        s["rows"], s["prefix_keys"] = rows, shared
        past = [p for m, p in zip(rows, shared) for _ in range(m)]
        # table rows: the groups' prefixes, then the sequences, which own pages from the end of the prefix on
        spans = [(0, p) for p in shared] + [(p, p + t) for p, t in zip(past, tails)]
        per = [(a // page, -(-b // page)) for a, b in spans]
        pages, width = sum(b - a for a, b in per) + 3, max(b for _, b in per) + 1
        shape = (pages, page, nk, d) if case["row_major"] else (pages, nk, page, d)
        s["k"], s["v"] = (normal(*shape, dtype=dt) for _ in range(2))
        if case["row_major"]:
            s["k"], s["v"] = s["k"].transpose(1, 2), s["v"].transpose(1, 2)   # [page][head][row][dim] either way
        at = torch.arange(width)[None]
        held = (at >= torch.tensor([a for a, _ in per])[:, None]) & (at < torch.tensor([b for _, b in per])[:, None])
        table = torch.full((len(per), width), -1, dtype=torch.int32)
        table[held] = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[:pages - 3].cpu()
        s["table"] = table.to(dev)
        if own:
            from gqa_transformer_decode_gb300 import runtime
            s["cache"] = runtime.PagedKV(s["k"], s["v"], s["table"])
        cu = [0]
        for m in rows:
            cu.append(cu[-1] + m)
        s["groups"], s["shared"], s["prefixes"] = ints(cu), ints(shared), ints(list(range(len(rows))))
        s["seqs"] = ints([len(rows) + b for b in range(case["batch"])])
        s["lens"] = ints([p + t for p, t in zip(past, tails)])
        s["longest_tail"] = max(tails)
        s["scale"] = 1.0 / math.sqrt(d)
        # queries sharp enough that some keys count far more than others
        s["q"] = normal(case["batch"], nh, d, dtype=dt, scale=2.0)
    elif case["op"] == "project":
        k, n, r = case["inputs"], case["outputs"], case["rank"]
        s["x"] = normal(case["rows"], k, dtype=dt)
        s["w"] = normal(n, k, dtype=dt, scale=0.02)
        s["a"] = normal(case["adapters"], r, k, dtype=dt, scale=k ** -0.5)
        s["b"] = normal(case["adapters"], n, r, dtype=dt, scale=0.02)
        s["s"] = torch.rand(case["adapters"], generator=g, device=dev) * 1.5 + 0.5
        s["bias"] = normal(n, dtype=dt, scale=0.02) if case["bias"] else None
        s["ids"] = ints(owners(case))
        s["out"] = torch.float32 if case["out"] == "f32" else dt
        if own:
            from gqa_transformer_decode_gb300 import runtime
            s["adapters"] = runtime.Adapters(s["a"], s["b"], s["s"])
    else:
        n, v = case["rows"], case["vocab"]
        # a broad floor and a few likely tokens, of which one is often the given one
        x = normal(n, v + case["pad"], scale=2.0)
        likely = torch.randint(v, (n, 12), generator=g, device=dev)
        x.scatter_add_(1, likely, normal(n, 12, scale=4.0).abs() + 4.0)
        x = x.to(dt)
        s["logits"] = x[:, :v]
        pick = torch.randint(v, (n,), generator=g, device=dev)
        s["ids"] = torch.where(torch.rand(n, generator=g, device=dev) < 0.7, likely[:, 0], pick).to(torch.int32)
        s["top"], s["temperature"] = case["top"], case["temperature"]
    return s


# ---- the plain forms --------------------------------------------------------------------------------------


def plain_shared(s):
    page, nk = s["k"].shape[2], s["k"].shape[1]
    q = s["q"].float()
    b, nh, d = q.shape
    grouped = q.view(b, nk, nh // nk, d)
    lens, start = s["lens"].long(), torch.repeat_interleave(
        s["shared"].long(), (s["groups"][1:] - s["groups"][:-1]).long(), output_size=b)
    # the rows' own keys, from the end of the prefix on
    key = start[:, None] + torch.arange(s["longest_tail"], device=q.device)
    ok = key < lens[:, None]
    own_rows = s["table"][s["seqs"].long()]
    at = own_rows.gather(1, (key // page).clamp(max=own_rows.shape[1] - 1)).clamp(min=0).long()
    k, v = (s[x][at, :, key % page].float() for x in "kv")             # [B][T][NKV][D]
    score = torch.einsum("bkgd,btkd->bkgt", grouped, k) * s["scale"]
    score = score.masked_fill(~ok[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    acc = torch.einsum("bkgt,btkd->bkgd", p, v)
    # each group's prefix, once for its rows
    r = 0
    for i, (m, n) in enumerate(zip(s["rows"], s["prefix_keys"])):
        key = torch.arange(n, device=q.device)
        at = s["table"][s["prefixes"][i].long(), key // page].long()
        k, v = (s[x][at, :, key % page].float() for x in "kv")         # [T][NKV][D]
        score = torch.einsum("bkgd,tkd->bkgt", grouped[r:r + m], k).mul_(s["scale"])
        new = torch.maximum(top[r:r + m], score.amax(-1, keepdim=True))
        old = (top[r:r + m] - new).exp()
        p = score.sub_(new).exp_()
        total[r:r + m] = total[r:r + m] * old + p.sum(-1, keepdim=True)
        acc[r:r + m] = acc[r:r + m] * old + torch.einsum("bkgt,tkd->bkgd", p, v)
        top[r:r + m] = new
        r += m
    return (acc / total).reshape(b, nh, d).to(s["q"].dtype), (top + total.log()).reshape(b, nh)


def plain_project(s):
    x, n, r = s["x"].float(), s["a"].shape[0], s["a"].shape[1]
    y = x @ s["w"].float().T
    # every row's products with every adapter, of which its own stay
    t = (x @ s["a"].float().flatten(0, 1).T).view(-1, n, r)
    mine = s["ids"][:, None] == torch.arange(n, device=x.device)
    t = torch.where(mine[:, :, None], t * s["s"][None, :, None], 0.0)
    y += t.flatten(1) @ s["b"].float().transpose(1, 2).flatten(0, 1)
    if s["bias"] is not None:
        y += s["bias"].float()
    return y.to(s["out"])


def plain_logprobs(s):
    logits = s["logits"].float()
    n, v = logits.shape
    x = logits / s["temperature"]
    x = x - x.amax(-1, keepdim=True)
    e = x.exp()
    total = e.sum(-1, keepdim=True)
    entropy = total.log()[:, 0] - (e * x).sum(-1) / total[:, 0]
    lp = x - total.log()
    given = s["ids"].long()[:, None]
    mine = logits.gather(1, given)
    before = (logits > mine) | ((logits == mine) & (torch.arange(v, device=x.device) < given))
    # equal logits stand in the order of their indices
    best = logits.sort(dim=-1, descending=True, stable=True).indices[:, :s["top"]] if s["top"] else given[:, :0]
    return lp.gather(1, given)[:, 0], before.sum(-1).to(torch.int32), entropy, best.to(torch.int32), lp.gather(1, best)


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "shared":
        if own:
            return s["cache"].decode_shared(s["q"], s["lens"], s["groups"], s["shared"], s["prefixes"], seqs=s["seqs"],
                                            scale=s["scale"], return_lse=True)
        return plain_shared(s)
    if op == "project":
        if own:
            return s["adapters"].project(s["x"], s["w"], s["ids"], bias=s["bias"], out_dtype=s["out"])
        return plain_project(s)
    if own:
        from gqa_transformer_decode_gb300 import runtime
        return tuple(runtime.logprobs(s["logits"], s["ids"], top=s["top"], temperature=s["temperature"]))
    return plain_logprobs(s)


# ---- the same in 64 bits, row by row ----------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "shared":
        page, nk, nh, d = case["page"], case["kv_heads"], case["heads"], case["dim"]
        q = s["q"].double()
        out = torch.zeros_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
        cu, shared, lens = (s[x].tolist() for x in ("groups", "shared", "lens"))

        def held(row, first, last):
            """Keys and values of positions first .. last - 1 of a table row, [NKV][n][D]."""
            i = torch.arange(first, last, device=q.device)
            at = s["table"][row].long()[i // page]
            return (s[x][at, :, i % page].transpose(0, 1).double() for x in "kv")
        for i in range(case["groups"]):
            k0, v0 = held(i, 0, shared[i])
            for b in range(cu[i], cu[i + 1]):
                k1, v1 = held(case["groups"] + b, shared[i], lens[b])
                for h in range(nk):
                    rows = slice(h * (nh // nk), (h + 1) * (nh // nk))
                    score = torch.cat((q[b, rows] @ k0[h].T, q[b, rows] @ k1[h].T), -1) * s["scale"]
                    lse[b, rows] = torch.logsumexp(score, -1)
                    p = torch.softmax(score, -1)
                    out[b, rows] = p[:, :shared[i]] @ v0[h] + p[:, shared[i]:] @ v1[h]
        return out, lse
    if case["op"] == "project":
        x = s["x"].double()
        y = x @ s["w"].double().T
        for a in range(case["adapters"]):
            at = (s["ids"] == a).nonzero()[:, 0]
            low = x[at] @ s["a"][a].double().T
            y[at] += low @ s["b"][a].double().T * float(s["s"][a])
        return y if s["bias"] is None else y + s["bias"].double()
    n, v = case["rows"], case["vocab"]
    parts = []
    for r in range(0, n, 256):
        raw = s["logits"][r:r + 256]
        given = s["ids"][r:r + 256].long()
        x = raw.double() / case["temperature"]
        lse = torch.logsumexp(x, -1)
        logp = x - lse[:, None]
        entropy = -(logp.exp() * logp).sum(-1)
        row = torch.arange(len(raw), device=x.device)
        index = torch.arange(v, device=x.device)
        mine = raw[row, given][:, None].double()
        rank = (raw.double() > mine).sum(-1) + ((raw.double() == mine) & (index < given[:, None])).sum(-1)
        left = raw.double().clone()
        best = torch.empty(len(raw), case["top"], dtype=torch.int32, device=x.device)
        for j in range(case["top"]):
            first = torch.where(left == left.amax(-1, keepdim=True), index, v).amin(-1)
            best[:, j] = first
            left[row, first] = -math.inf
        parts.append((logp[row, given], rank.to(torch.int32), entropy, best, logp[row[:, None], best.long()]))
    return tuple(torch.cat(x) for x in zip(*parts))
