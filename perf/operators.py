"""The paged-cache operators as a serving program calls them, for timing and comparison.

Three operators work on one pool of key/value pages shared by many sequences:

  append   per-head RMS norm of q and k (optional), rotary embedding, and the
           store of the K/V rows of new tokens into their sequences' pages
  decode   attention of one new token per sequence over its pages
  prefill  attention of several new tokens per sequence (a ragged batch, each
           chunk standing on the keys already cached)

Both attentions are causal and take a sliding window with a few first tokens
(sinks) that stay visible.  `run` computes the plain form in 32 bits, or calls
the library where `own` is set; `exact` restates each operator in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# (query heads, kv heads, head dim) of this repository's decoders and encoder, and plain multi-head attention
HEADS = [(14, 2, 64), (32, 8, 64), (16, 8, 128), (32, 8, 128), (8, 8, 128), (4, 2, 16)]


def listed():
    base = dict(page=16, row_major=False, type="bf16", ragged=False, window=0, sinks=0)
    q05 = dict(base, heads=14, kv_heads=2, dim=64)     # the 0.5B decoder
    l1b = dict(base, heads=32, kv_heads=8, dim=64)     # the 1B decoder
    d128 = dict(base, heads=16, kv_heads=8, dim=128)   # the 128-wide heads with q/k norms
    return [
        # one token of one sequence between two projections: latency alone
        dict(q05, name="append one token", op="append", batch=1, new=1, past=516, input="f32", norm=False),
        # a decode step of 64 sequences at different lengths
        dict(l1b, name="append batch 64", op="append", batch=64, new=1, past=4095, ragged=True, input="f32", norm=False),
        # a 4096-token prompt straight from the f32 projections
        dict(l1b, name="append prompt 4096", op="append", batch=1, new=4096, past=0, input="f32", norm=False),
        # ragged prompts with q/k norms from bf16 projections into pages that hold a row's heads side by side
        dict(d128, name="append normed prompts", op="append", batch=9, new=2047, past=1000, ragged=True, page=64,
             row_major=True, input="bf16", norm=True),
        # the greedy loop of one short conversation
        dict(q05, name="decode one short", op="decode", batch=1, new=1, past=516),
        # the 64-sequence decode step at contexts of up to 4096 tokens
        dict(l1b, name="decode batch 64", op="decode", batch=64, new=1, past=4095, ragged=True),
        # one user with a very long document
        dict(base, heads=32, kv_heads=8, dim=128, name="decode one long", op="decode", batch=1, new=1, past=131070,
             type="f16", page=64),
        # streaming generation: long sequences of which a window and the first tokens count
        dict(d128, name="decode windowed", op="decode", batch=32, new=1, past=16383, ragged=True, window=1024, sinks=4,
             page=32, row_major=True),
        # drafted tokens checked at once, a few sequences
        dict(q05, name="prefill drafts", op="prefill", batch=4, new=9, past=700, ragged=True),
        # the 2048-token prompt of the 1B decoder
        dict(l1b, name="prefill prompt 2048", op="prefill", batch=1, new=2048, past=0, page=64),
        # chunks of several prompts, each on what is cached already
        dict(d128, name="prefill chunks", op="prefill", batch=5, new=1000, past=5001, ragged=True, type="f16", page=32),
        # a long prompt under a window
        dict(d128, name="prefill windowed", op="prefill", batch=1, new=8192, past=0, window=1024, sinks=4, page=128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "decode", "prefill"])
    heads, kv_heads, dim = rng.choice(HEADS)
    c = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
             row_major=rng.random() < 0.3, type=rng.choice(["bf16", "bf16", "f16"]), ragged=rng.random() < 0.7,
             window=0, sinks=0)
    if op == "append":
        c["batch"] = log(1, 64)
        c["new"] = 1 if rng.random() < 0.4 else max(1, log(1, 8192) // c["batch"])
        c["past"] = rng.choice([0, log(1, 8000)])
        c["input"] = rng.choice(["f32", "bf16", "f16"])
        c["norm"] = rng.random() < 0.5
    else:
        if rng.random() < 0.4:
            c["window"], c["sinks"] = log(16, 4096), rng.choice([0, 1, 4, 17])
        if op == "decode":
            c["batch"], c["new"], c["past"] = log(1, 128), 1, log(1, 100000)
            while work(c)["bytes"] > 5e8 or c["batch"] * c["past"] * kv_heads * dim > 3e8:
                c["past"] = c["past"] * 2 // 3
        else:
            c["batch"], c["new"], c["past"] = log(1, 12), log(2, 6000), rng.choice([0, log(1, 8000)])
            while c["batch"] ** 2 * c["new"] * (c["new"] + c["past"]) * heads > 1e9:
                c["new"], c["past"] = max(2, c["new"] * 2 // 3), c["past"] * 4 // 5
    return c


def spread(longest, n, ragged):
    """n lengths up to `longest`: all the same, or spread over (0, longest] with the first the longest."""
    if not ragged:
        return [longest] * n
    return [min(longest, max(1, round(longest * (1.0 - (b * 0.6180339887) % 1.0)))) for b in range(n)]


def lengths(case):
    """(new tokens, keys cached before them) of each sequence."""
    n = case["batch"]
    new = spread(case["new"], n, case["ragged"])
    past = spread(case["past"], n, case["ragged"])[::-1] if case["past"] else [0] * n
    return new, past


def visible_pairs(case):
    """Number of (new token, visible key) pairs."""
    total = 0
    w, k = case["window"], case["sinks"]
    for n, p in zip(*lengths(case)):
        lo, hi = p + 1, p + n   # keys at or before each new token, first and last
        if not w:
            total += (lo + hi) * n // 2
            continue
        # a token with m keys at or before it sees min(m, w) of the window and min(sinks, m - w) below it
        a = min(max(w - lo + 1, 0), n)                       # tokens with m <= w
        total += (lo + lo + a - 1) * a // 2 + (n - a) * w
        m0 = max(lo, w + 1)
        b = min(max(w + k - m0 + 1, 0), n - a)               # tokens with w < m <= w + sinks
        total += b * (m0 - w + m0 + b - 1 - w) // 2 + (n - a - b) * k
    return total


def visible_keys(case):
    """Number of keys that some new token sees."""
    total = 0
    w, k = case["window"], case["sinks"]
    for n, p in zip(*lengths(case)):
        lo = max(0, p + 1 - w) if w else 0
        total += p + n - lo + min(k, lo)
    return total


def work(case):
    nh, nk, d = case["heads"], case["kv_heads"], case["dim"]
    new, past = lengths(case)
    n = sum(new)
    if case["op"] == "append":
        size = 4 if case["input"] == "f32" else 2
        rows = len({p + i for m, p in zip(new, past) for i in range(m)})
        return {"bytes": n * (nh + 2 * nk) * d * (size + 2) + rows * d * 4 + n * 8 + (4 * d if case["norm"] else 0),
                "flops": n * (nh + nk) * d * (7 if case["norm"] else 3)}
    return {"bytes": visible_keys(case) * nk * d * 4 + n * nh * (d * 4 + 4), "flops": 4 * nh * d * visible_pairs(case)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["type"]]
    nh, nk, d, page, batch = case["heads"], case["kv_heads"], case["dim"], case["page"], case["batch"]
    new, past = lengths(case)
    per = [-(-(m + p) // page) for m, p in zip(new, past)]
    n, pages, width = sum(new), sum(per) + 3, max(per) + 1

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    # a pool that other requests have used before, and pages dealt out in no order
    shape = (pages, page, nk, d) if case["row_major"] else (pages, nk, page, d)
    pool = [normal(*shape, dtype=dt) for _ in range(2)]
    if case["row_major"]:
        pool = [x.transpose(1, 2) for x in pool]   # [page][head][row][dim] whatever the memory order
    dealt = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32)
    counts = torch.tensor(per)
    at = torch.arange(width)[None, :] < counts[:, None]
    table[at] = dealt[:sum(per)].cpu()
    s = {"case": case, "k": pool[0], "v": pool[1], "table": table.to(dev)}
    if own:
        from gqa_transformer_decode_gb300 import runtime
        s["cache"] = runtime.PagedKV(s["k"], s["v"], s["table"])
    s["lens"] = torch.tensor([m + p for m, p in zip(new, past)], dtype=torch.int32, device=dev)
    s["window"], s["sinks"], s["scale"] = case["window"], case["sinks"], 1.0 / math.sqrt(d)
    if case["op"] == "append":
        src = DTYPES[case["input"]]
        s["qkv"] = normal(n, (nh + 2 * nk) * d, dtype=src)
        s["seqs"] = torch.tensor([b for b, m in enumerate(new) for _ in range(m)], dtype=torch.int32, device=dev)
        s["positions"] = torch.tensor([p + i for m, p in zip(new, past) for i in range(m)], dtype=torch.int32, device=dev)
        turn = torch.arange(max(m + p for m, p in zip(new, past)), dtype=torch.float64, device=dev)[:, None] \
            * (1e6 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=dev) / d))[None, :]
        s["cos"], s["sin"] = turn.cos().float(), turn.sin().float()
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"], s["k_norm"] = ((1 + normal(d, scale=0.1)).to(torch.bfloat16) for _ in range(2))
    else:
        # queries sharp enough that some keys count far more than others
        s["q"] = normal(n, nh, d, dtype=dt, scale=2.0)
        if case["op"] == "prefill":
            cu = [0]
            for m in new:
                cu.append(cu[-1] + m)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
            s["keys"] = sum(m + p for m, p in zip(new, past))
    return s


# ---- the plain forms --------------------------------------------------------------------------------------


def turned(x, norm, cos, sin, eps):
    """RMS norm over the last axis (where given) and rotate-half, in 32 bits."""
    if norm is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * norm.float()
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def plain_append(s, q, k, v):
    page = s["k"].shape[2]
    pos = s["positions"].long()
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    dt = s["k"].dtype
    at = s["table"][s["seqs"].long(), pos // page].long()
    s["k"][at, :, pos % page] = turned(k.float(), s["k_norm"], cos, sin, 1e-6).to(dt)
    s["v"][at, :, pos % page] = v.to(dt)
    return turned(q.float(), s["q_norm"], cos, sin, 1e-6).to(dt), s["k"], s["v"]


def sees(pos, key, window, sinks):
    """Whether a token at `pos` sees the key at position `key`."""
    ok = key <= pos
    if window:
        ok = ok & ((key > pos - window) | (key < sinks))
    return ok


def plain_decode(s):
    page, nk = s["k"].shape[2], s["k"].shape[1]
    q = s["q"].float()
    b, nh, d = q.shape
    key = torch.arange(int(s["table"].shape[1]) * page, device=q.device)
    at = s["table"].clamp(min=0).long()[:, key // page]
    k, v = (s[x][at, :, key % page].float() for x in "kv")            # [B][T][NKV][D]
    ok = sees(s["lens"][:, None] - 1, key[None, :], s["window"], s["sinks"])
    score = torch.einsum("bkgd,btkd->bkgt", q.view(b, nk, nh // nk, d), k) * s["scale"]
    score = score.masked_fill(~ok[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bkgt,btkd->bkgd", p, v.masked_fill(~ok[:, :, None, None], 0.0)) / total.clamp(min=1e-37)
    return out.view(b, nh, d).to(s["q"].dtype), (top + total.log()).view(b, nh)


def plain_prefill(s):
    page, nk = s["k"].shape[2], s["k"].shape[1]
    q = s["q"].float()
    n, nh, d = q.shape
    lens, cu = s["lens"].long(), s["cu"].long()
    which = torch.arange(lens.numel(), device=q.device)
    # every query row and every key as (sequence, position)
    rseq = torch.repeat_interleave(which, cu[1:] - cu[:-1], output_size=n)
    rpos = torch.arange(n, device=q.device) - cu[rseq + 1] + lens[rseq]
    kseq = torch.repeat_interleave(which, lens, output_size=s["keys"])
    kpos = torch.arange(s["keys"], device=q.device) - (lens.cumsum(0) - lens)[kseq]
    at = s["table"][kseq, kpos // page].long()
    k, v = (s[x][at, :, kpos % page].float() for x in "kv")            # [T][NKV][D]
    ok = (rseq[:, None] == kseq[None, :]) & sees(rpos[:, None], kpos[None, :], s["window"], s["sinks"])
    score = torch.einsum("nkgd,tkd->kgnt", q.view(n, nk, nh // nk, d), k) * s["scale"]
    score = score.masked_fill_(~ok, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("kgnt,tkd->nkgd", p, v) / total.clamp(min=1e-37).permute(2, 0, 1, 3)
    return out.reshape(n, nh, d).to(s["q"].dtype), (top + total.log()).permute(2, 0, 1, 3).reshape(n, nh)


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "append":
        nh, nk, d = s["case"]["heads"], s["k"].shape[1], s["k"].shape[3]
        q, k, v = s["qkv"].view(-1, nh + 2 * nk, d).split((nh, nk, nk), 1)
        if own:
            q = s["cache"].append(k, v, s["seqs"], s["positions"], s["cos"], s["sin"], q=q, q_norm=s["q_norm"],
                                  k_norm=s["k_norm"], eps=1e-6)
            return q, s["k"], s["v"]
        return plain_append(s, q, k, v)
    if op == "decode":
        if own:
            return s["cache"].decode(s["q"], s["lens"], window=s["window"], sinks=s["sinks"], scale=s["scale"],
                                     return_lse=True)
        return plain_decode(s)
    if own:
        return s["cache"].prefill(s["q"], s["cu"], s["lens"], window=s["window"], sinks=s["sinks"], scale=s["scale"],
                                  return_lse=True)
    return plain_prefill(s)


# ---- the same in 64 bits, sequence by sequence ------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    page, nk, d, nh = case["page"], case["kv_heads"], case["dim"], case["heads"]
    new, past = lengths(case)
    if case["op"] == "append":
        rows = s["qkv"].double().view(-1, nh + 2 * nk, d)
        turn = torch.complex(s["cos"].double(), s["sin"].double())
        kp, vp = s["k"].double(), s["v"].double()
        table = s["table"].cpu()
        qs, r = [], 0
        for b, (m, p) in enumerate(zip(new, past)):
            x = rows[r:r + m]
            r += m
            heads = []
            for part, w in ((x[:, :nh], s["q_norm"]), (x[:, nh:nh + nk], s["k_norm"])):
                if w is not None:
                    part = part / (part.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
                z = torch.complex(part[..., :d // 2].contiguous(), part[..., d // 2:].contiguous()) * turn[p:p + m, None]
                heads.append(torch.cat((z.real, z.imag), -1))
            qs.append(heads[0])
            for first in range(p // page * page, p + m, page):
                i0, i1 = max(first, p), min(first + page, p + m)
                at = int(table[b, first // page])
                kp[at, :, i0 - first:i1 - first] = heads[1][i0 - p:i1 - p].transpose(0, 1)
                vp[at, :, i0 - first:i1 - first] = x[i0 - p:i1 - p, nh + nk:].transpose(0, 1)
        return torch.cat(qs), kp, vp
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    r = 0
    for b, (m, p) in enumerate(zip(new, past)):
        held = s["table"][b, :-(-(m + p) // page)].long()
        pos = torch.arange(p, p + m, device=q.device)[:, None]
        key = torch.arange(p + m, device=q.device)[None, :]
        hidden = (key > pos) | ((key <= pos - case["window"]) & (key >= case["sinks"]) if case["window"] else key > pos)
        for h in range(nk):
            k, v = (s[x][held, h].reshape(-1, d)[:p + m].double() for x in "kv")
            for j in range(h * (nh // nk), (h + 1) * (nh // nk)):
                score = (q[r:r + m, j] @ k.T * s["scale"]).masked_fill(hidden, -math.inf)
                lse[r:r + m, j] = torch.logsumexp(score, -1)
                out[r:r + m, j] = torch.softmax(score, -1) @ v
        r += m
    return out, lse
