"""The operators around the paged KV cache and their measured cases.

Four operators of one decode step, in the order a serving program calls them:

  qk_norm_rope      RMSNorm of every query and key head, the rotation by position, and the write of
                    the new K and V rows into the paged cache (fp32, bf16, or e4m3 with a scale per
                    kv head)
  attention_q8      block-causal grouped-query attention that reads the e4m3 cache
  attention_shared  the same attention over a bf16 cache for a batch whose sequences all start with
                    one shared prefix, whose pages are stored once
  sample            the next token of every row of logits by temperature, top-k, top-p and min-p,
                    from given uniform numbers

`run` computes them from elementary torch operations, or with `own` by the library's calls.
"""
import math

import torch

own = False

PAGE = 64
HEADS = ((32, 8, 128), (40, 8, 128), (8, 2, 128))   # query heads, kv heads, head_dim


def listed():
    return [
        # one new token of one chat, bf16 cache: the call's latency is the figure
        dict(name="qkv write, 1 token", op="qk_norm_rope", batch=1, m=1, ctx=500, hq=32, hkv=8, hd=128, dtype="bf16",
             cache="bf16", norm=True, ragged=False),
        # a verify forward of 64 chats, 33 rows each, into an e4m3 cache
        dict(name="qkv write, 64 x 33 rows, e4m3", op="qk_norm_rope", batch=64, m=33, ctx=479, hq=32, hkv=8, hd=128,
             dtype="bf16", cache="e4m3", norm=True, ragged=False),
        # a padded prefill: prompts of 1..2048 tokens, five query heads per kv head
        dict(name="qkv write, ragged prefill 8 x 2048, e4m3", op="qk_norm_rope", batch=8, m=2048, ctx=0, hq=40, hkv=8,
             hd=128, dtype="bf16", cache="e4m3", norm=True, ragged=True),
        # single-token decode of one short chat
        dict(name="q8 decode, 1 x 1000 keys", op="attention_q8", batch=1, m=1, ctx=999, ragged=False, block=1, hq=32,
             hkv=8),
        # single-token decode of a full batch of chats of many lengths
        dict(name="q8 decode, 64 ragged to 8192", op="attention_q8", batch=64, m=1, ctx=8191, ragged=True, block=1,
             hq=32, hkv=8),
        # the draft forward of a diffusion block of 32 after long documents
        dict(name="q8 block of 32, 8 x 16384", op="attention_q8", batch=8, m=32, ctx=16384, ragged=False, block=32,
             hq=32, hkv=8),
        # four chats under one short system prompt
        dict(name="shared decode, 4, prefix 1000", op="attention_shared", batch=4, m=1, prefix=1000, ctx=90, block=1,
             hq=32, hkv=8),
        # 64 questions about one long document
        dict(name="shared decode, 64, prefix 16384", op="attention_shared", batch=64, m=1, prefix=16384, ctx=511,
             block=1, hq=32, hkv=8),
        # draft blocks of 32 for 16 chats under one long instruction, five query heads per kv head
        dict(name="shared block of 32, 16, prefix 4133", op="attention_shared", batch=16, m=32, prefix=4133, ctx=300,
             block=32, hq=40, hkv=8),
        # one row of a small vocabulary
        dict(name="sample, 1 x 5000", op="sample", rows=1, vocab=5000, dtype="f32", filters="all"),
        # a batch of chats with settings of their own each
        dict(name="sample, 64 x 151936, own settings", op="sample", rows=64, vocab=151936, dtype="f32",
             filters="mixed"),
        # many samples of one model by temperature alone, bf16 logits (equal logits are common)
        dict(name="sample, 300 x 151936, temperature", op="sample", rows=300, vocab=151936, dtype="bf16",
             filters="none"),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("qk_norm_rope", "attention_q8", "attention_shared", "sample"))
    hq, hkv, hd = rng.choice(HEADS)
    if op == "qk_norm_rope":
        if rng.random() < 0.25:
            hq, hkv, hd = rng.choice(((4, 4, 64), (16, 4, 64)))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        batch = _log(rng, 1, 64)
        m = _log(rng, 1, 8192 // batch)
        ctx = _log(rng, 1, 16384 // batch)
        return dict(op=op, batch=batch, m=m, ctx=ctx, hq=hq, hkv=hkv, hd=hd, dtype=dtype,
                    cache=rng.choice((dtype, "e4m3")), norm=rng.random() < 0.8, ragged=rng.random() < 0.4)
    if op == "sample":
        vocab = rng.choice((151936, _log(rng, 300, 151936), _log(rng, 300, 151936)))
        return dict(op=op, rows=_log(rng, 1, min(300, 45000000 // vocab)), vocab=vocab, dtype=rng.choice(("f32", "bf16")),
                    filters=rng.choice(("all", "mixed", "mixed", "none")))
    m = rng.choice((1, 1, 1, 2, 8, 16, 32, 33))
    block = rng.choice((1, m, 8)) if m > 8 else 1
    batch = _log(rng, 1, 64)
    if op == "attention_q8":
        return dict(op=op, batch=batch, m=m, ctx=_log(rng, 1, 16384 * 8 // max(8, batch)), ragged=rng.random() < 0.5,
                    block=block, hq=hq, hkv=hkv)
    # rows that read the prefix x its length: no more than the largest listed case
    return dict(op=op, batch=batch, m=m, prefix=_log(rng, 60, min(16384, 16 * 32 * 4133 // (batch * m))),
                ctx=_log(rng, 1, 511), block=block, hq=hq, hkv=hkv)


DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _pages(g, count, total):
    """`count` distinct page ids of a pool of `total` pages, in no order."""
    return torch.randperm(total, generator=g, device="cuda")[:count].to(torch.int32)


def _lens(g, batch, ctx, ragged):
    if not ragged:
        return torch.full((batch,), ctx, dtype=torch.int32, device="cuda")
    lens = torch.randint(max(0, ctx // 8), ctx + 1, (batch,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = ctx
    return lens


def _kv(g, n_pages, hkv, hd, dtype):
    """Filled pages, K about twice as large as V, made in parts (a cache of some hundred MB)."""
    pool = torch.empty(n_pages, 2, hkv, PAGE, hd, dtype=dtype, device="cuda")
    for at in range(0, n_pages, 2048):
        part = _randn(g, min(2048, n_pages - at), 2, hkv, PAGE, hd)
        pool[at:at + 2048].copy_(part)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        x = _randn(g, rows, vocab) * 2.0
        # a few likely tokens in each row, as a trained model gives them
        at = torch.randint(0, vocab, (rows, 12), generator=g, device="cuda")
        x.scatter_add_(1, at, 4.0 + 6.0 * torch.rand(rows, 12, generator=g, device="cuda"))
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["u"] = torch.rand(rows, generator=g, device="cuda")
        s["temperature"] = 0.5 + torch.rand(rows, generator=g, device="cuda")
        k = torch.randint(1, 200, (rows,), generator=g, device="cuda", dtype=torch.int32)
        p = 0.5 + 0.49 * torch.rand(rows, generator=g, device="cuda")
        q = 0.2 * torch.rand(rows, generator=g, device="cuda")
        if case["filters"] == "mixed":   # a third of the rows leaves each filter off, one in eight is greedy
            k *= (torch.rand(rows, generator=g, device="cuda") > 0.33).to(torch.int32)
            p = torch.where(torch.rand(rows, generator=g, device="cuda") > 0.33, p, torch.ones_like(p))
            q = torch.where(torch.rand(rows, generator=g, device="cuda") > 0.33, q, torch.zeros_like(q))
            s["temperature"] *= (torch.rand(rows, generator=g, device="cuda") > 0.125).float()
        off = case["filters"] == "none"
        s["top_k"], s["top_p"], s["min_p"] = (None, None, None) if off else (k, p, q)
        s["tokens"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["prob"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        return s
    batch, m, hq, hkv = case["batch"], case["m"], case["hq"], case["hkv"]
    hd = case.get("hd", 128)
    ctx = case["ctx"]
    pps = (ctx + m + PAGE - 1) // PAGE
    if case["op"] == "qk_norm_rope":
        dtype = DTYPES[case["dtype"]]
        n_pages = batch * pps + 1
        s["lens"] = _lens(g, batch, ctx, case["ragged"])
        # q, k and v are parts of one projection's output, as a forward has them
        qkv = (_randn(g, batch, m, hq + 2 * hkv, hd) * 1.5).to(dtype)
        s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        s["q_gain"] = (1.0 + 0.2 * _randn(g, hd)).to(dtype) if case["norm"] else None
        s["k_gain"] = (1.0 + 0.2 * _randn(g, hd)).to(dtype) if case["norm"] else None
        i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
        pos = torch.arange(pps * PAGE, device="cuda", dtype=torch.float64)
        angle = pos[:, None] * 10000.0 ** (-2.0 * i / hd)
        s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()   # [positions, hd / 2, 2]
        s["page_table"] = _pages(g, batch * pps, n_pages).view(batch, pps)
        s["pool"] = torch.zeros(n_pages, 2, hkv, PAGE, hd, device="cuda").to(DTYPES[case["cache"]])
        s["q_out"] = torch.zeros(batch, m, hq, hd, dtype=dtype, device="cuda")
        q8 = case["cache"] == "e4m3"
        s["k_scale"] = 0.02 + 0.02 * torch.rand(hkv, generator=g, device="cuda") if q8 else None
        s["v_scale"] = 0.02 + 0.02 * torch.rand(hkv, generator=g, device="cuda") if q8 else None
        rows = torch.randint(1, m + 1, (batch,), generator=g, device="cuda", dtype=torch.int32) if case["ragged"] else None
        s["rows"] = rows
        live = torch.arange(m, device="cuda")[None, :] < (m if rows is None else rows[:, None])
        s["live"] = live.expand(batch, m).nonzero()   # (sequence, row) of every row that is not padding
        return s
    s["q"] = _randn(g, batch, m, hq, hd).to(torch.bfloat16)
    s["lens"] = _lens(g, batch, ctx, case.get("ragged", True))
    s["out"] = torch.empty(batch, m, hq, hd, dtype=torch.bfloat16, device="cuda")
    s["max_len"] = ctx + m
    if case["op"] == "attention_q8":
        n_pages = batch * pps + 1
        s["pool"] = _kv(g, n_pages, hkv, hd, torch.float8_e4m3fn)
        s["k_scale"] = 0.8 + 0.4 * torch.rand(hkv, generator=g, device="cuda")
        s["v_scale"] = 0.8 + 0.4 * torch.rand(hkv, generator=g, device="cuda")
        s["page_table"] = _pages(g, batch * pps, n_pages).view(batch, pps)
        return s
    shared = (case["prefix"] + PAGE - 1) // PAGE
    n_pages = batch * pps + shared + 1
    s["pool"] = _kv(g, n_pages, hkv, hd, torch.bfloat16)
    every = _pages(g, batch * pps + shared, n_pages)
    s["shared_pages"], s["page_table"] = every[:shared].contiguous(), every[shared:].view(batch, pps).contiguous()
    return s


# ------------------------------------------------------------------------------- plain forms --


def _norm_rope(x, gain, eps, cos, sin):
    """x [batch, m, heads, hd] in 32 bits: RMSNorm of each head, then the rotation of the pairs (i, i + hd / 2)."""
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gain.float()
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_qk_norm_rope(s):
    pos = s["lens"][:, None].long() + torch.arange(s["m"], device="cuda")
    cs = s["rope"][pos.clamp(max=s["rope"].shape[0] - 1)][:, :, None]   # positions behind a padded row's end are not read
    q = _norm_rope(s["q"].float(), s["q_gain"], 1e-6, cs[..., 0], cs[..., 1])
    k = _norm_rope(s["k"].float(), s["k_gain"], 1e-6, cs[..., 0], cs[..., 1])
    kv = torch.stack((k, s["v"].float()), 2)   # [batch, m, 2, hkv, hd]
    if s["k_scale"] is not None:
        kv = (kv / torch.stack((s["k_scale"], s["v_scale"]))[:, :, None]).clamp(-448.0, 448.0)
    b, i = s["live"][:, 0], s["live"][:, 1]
    at = pos[b, i]
    page = s["page_table"][b, at // PAGE].long()
    s["q_out"][b, i] = q[b, i].to(s["q_out"].dtype)
    new = kv[b, i].to(s["pool"].dtype)
    pool = s["pool"]
    if pool.dtype == torch.float8_e4m3fn:
        pool, new = pool.view(torch.uint8), new.view(torch.uint8)
    pool[page, :, :, at % PAGE] = new
    return {"q": s["q_out"], "pool": s["pool"]}


def _visible(s, keys):
    """[batch, m, keys]: which keys (counted from the sequence's own first one) a row sees."""
    row = torch.arange(s["m"], device="cuda")
    end = torch.clamp(row // s["block"] * s["block"] + s["block"], max=s["m"])
    return torch.arange(keys, device="cuda") < (s["lens"][:, None] + end)[:, :, None]


def _rows(s):
    """Queries as [batch, hkv, m * G, hd] in 32 bits, scaled."""
    b, m, hq, hd = s["q"].shape
    g = hq // s["hkv"]
    q = s["q"].float().view(b, m, s["hkv"], g, hd).permute(0, 2, 1, 3, 4).reshape(b, s["hkv"], m * g, hd)
    return q / math.sqrt(hd)


def _back(s, o):
    b, m, hq, hd = s["q"].shape
    return o.view(b, s["hkv"], m, hq // s["hkv"], hd).permute(0, 2, 1, 3, 4).reshape(b, m, hq, hd).to(torch.bfloat16)


def _paged(pool, table, which):
    """K (0) or V (1) of every sequence: [batch, hkv, keys, hd] in 32 bits."""
    part = pool[:, which]
    if part.dtype == torch.float8_e4m3fn:
        part = part.view(torch.uint8)[table.long()].view(torch.float8_e4m3fn)
    else:
        part = part[table.long()]
    b, pages, hkv, page, hd = part.shape
    return part.float().permute(0, 2, 1, 3, 4).reshape(b, hkv, pages * page, hd)


def _masked_scores(s, q, k):
    seen = _visible(s, k.shape[2])[:, None, :, None, :]
    b, hkv, rows, _ = q.shape
    score = (q @ k.transpose(2, 3)).view(b, hkv, s["m"], rows // s["m"], k.shape[2])
    return torch.where(seen, score, float("-inf")).view(b, hkv, rows, k.shape[2])


def _plain_attention_q8(s):
    k = _paged(s["pool"], s["page_table"], 0) * s["k_scale"][:, None, None]
    score = _masked_scores(s, _rows(s), k)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    v = _paged(s["pool"], s["page_table"], 1) * s["v_scale"][:, None, None]
    return _back(s, (p @ v) / p.sum(-1, keepdim=True))


def _plain_attention_shared(s):
    q = _rows(s)
    b, hkv, rows, hd = q.shape
    every = q.permute(1, 0, 2, 3).reshape(hkv, b * rows, hd)
    own_score = _masked_scores(s, q, _paged(s["pool"], s["page_table"], 0))
    sk = _paged(s["pool"], s["shared_pages"][None], 0)[0][:, :s["prefix"]]
    sv = _paged(s["pool"], s["shared_pages"][None], 1)[0][:, :s["prefix"]]
    score = every @ sk.transpose(1, 2)
    top = torch.maximum(score.amax(-1).view(hkv, b, rows).transpose(0, 1), own_score.amax(-1))[..., None]
    p = torch.exp(score - top.transpose(0, 1).reshape(hkv, b * rows, 1))
    own_p = torch.exp(own_score - top)
    o = (p @ sv).view(hkv, b, rows, hd).transpose(0, 1) + own_p @ _paged(s["pool"], s["page_table"], 1)
    total = p.sum(-1).view(hkv, b, rows).transpose(0, 1) + own_p.sum(-1)
    return _back(s, o / total[..., None])


def _plain_sample(s):
    # in 64 bits: sums over a vocabulary, and values next to the borders of the filters
    x = s["logits"].double()
    rows, vocab = x.shape
    t = s["temperature"].double()[:, None]
    top = x.amax(1, keepdim=True)
    w = torch.where(t > 0, torch.exp((x - top) / torch.where(t > 0, t, 1.0)), (x == top).double())
    greedy = (t > 0).logical_not()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(vocab, device="cuda")[None]
    keep = torch.where(greedy, rank < 1, True)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((k <= 0) | (rank < k))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        ws = ws * keep
        before = torch.cumsum(ws, 1) - ws
        keep = keep & ((p >= 1) | (before < p * ws.sum(1, keepdim=True)) | (rank < 1))
    if s["min_p"] is not None:
        keep = keep & (w.gather(1, order) >= s["min_p"].double()[:, None])
    kept = torch.zeros_like(w).scatter_(1, order, keep.double()) * w
    run_sum = torch.cumsum(kept, 1)
    total = run_sum[:, -1:]
    token = (run_sum <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    s["tokens"].copy_(token[:, 0])
    s["prob"].copy_((kept.gather(1, token) / total)[:, 0])
    return {"tokens": s["tokens"], "prob": s["prob"]}


# ------------------------------------------------------------------------------------ one pass --


def _own(s):
    import self_speculation_b200 as nb

    op = s["op"]
    if op == "qk_norm_rope":
        nb.nld_qk_norm_rope(s["q"], s["k"], s["v"], s["q_gain"], s["k_gain"], 1e-6, s["rope"], s["lens"], s["q_out"],
                            s["pool"], s["page_table"], rows=s["rows"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"q": s["q_out"], "pool": s["pool"]}
    if op == "attention_q8":
        nb.nld_attention_q8(s["q"], s["pool"], s["k_scale"], s["v_scale"], s["page_table"], s["lens"], s["block"],
                            s["max_len"], s["out"])
        return s["out"]
    if op == "attention_shared":
        if "workspace" not in s:   # kept with the plan, as a serving loop keeps it
            size = nb.nld_attention_shared_workspace_size(s["batch"], s["m"], s["hq"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        nb.nld_attention_shared(s["q"], s["pool"], s["shared_pages"], s["prefix"], s["page_table"], s["lens"], s["block"],
                                s["max_len"], s["out"], s["workspace"])
        return s["out"]
    nb.nld_sample(s["logits"], s["u"], s["tokens"], s["prob"], temperature=s["temperature"], top_k=s["top_k"],
                  top_p=s["top_p"], min_p=s["min_p"])
    return {"tokens": s["tokens"], "prob": s["prob"]}


def run(state):
    if own:
        return _own(state)
    return {"qk_norm_rope": _plain_qk_norm_rope, "attention_q8": _plain_attention_q8,
            "attention_shared": _plain_attention_shared, "sample": _plain_sample}[state["op"]](state)


def work(case):
    op = case["op"]
    if op == "sample":
        n = case["rows"] * case["vocab"]
        # every logit is read once; an exponential and a few comparisons each
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["rows"] * 24, "flops": 4 * n}
    batch, m, hq, hkv = case["batch"], case["m"], case["hq"], case["hkv"]
    if op == "qk_norm_rope":
        hd = case["hd"]
        live = batch * (m + 1) // 2 if case["ragged"] else batch * m
        el = 4 if case["dtype"] == "f32" else 2
        kv = 1 if case["cache"] == "e4m3" else el
        # q, k, v read; q and the cache rows written; the table's rows of each token
        return {"bytes": live * hd * (el * (2 * hq + 2 * hkv) + kv * 2 * hkv) + live * hd * 4,
                "flops": live * hd * (hq + hkv) * 8}
    keys = batch * ((case["ctx"] * 9 // 16 if case.get("ragged", True) else case["ctx"]) + m)
    rows = 2 * batch * m * hq * 128 * 2   # queries read and outputs written
    if op == "attention_q8":
        return {"bytes": keys * hkv * 2 * 128 + rows, "flops": keys * m * hq * 4 * 128}
    return {"bytes": (keys + case["prefix"]) * hkv * 2 * 128 * 2 + rows,
            "flops": (keys * m + batch * m * case["prefix"]) * hq * 4 * 128}


# --------------------------------------------------------------------- the definitions in 64 bits --


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "qk_norm_rope":
        return _exact_qk_norm_rope(s)
    b, m, hq, hd = s["q"].shape
    group = hq // s["hkv"]
    out = torch.empty(b, m, hq, hd, dtype=torch.float64, device="cuda")
    for i in range(b):
        n = int(s["lens"][i])
        k, v = _rows_of(s, s["page_table"][i], n + m)
        if case["op"] == "attention_shared":
            k0, v0 = _rows_of(s, s["shared_pages"], case["prefix"])
            k, v = torch.cat((k0, k)), torch.cat((v0, v))
        before = k.shape[0] - m   # keys that every row sees
        for j in range(0, m, case["block"]):
            rows = s["q"][i, j:j + case["block"]].double()
            end = before + min(j + case["block"], m)
            for h in range(s["hkv"]):
                q = rows[:, h * group:(h + 1) * group].reshape(-1, hd)
                p = torch.softmax(q @ k[:end, h].T * hd ** -0.5, -1)
                out[i, j:j + case["block"], h * group:(h + 1) * group] = (p @ v[:end, h]).view(-1, group, hd)
    return out


def _rows_of(s, pages, n):
    """The first n K rows and V rows of a list of pages, [n, hkv, hd] in 64 bits."""
    got = torch.cat([s["pool"][int(p)].double() for p in pages[:(n + PAGE - 1) // PAGE]], 2)[:, :, :n].transpose(1, 2)
    if "k_scale" in s:
        return got[0] * s["k_scale"].double()[None, :, None], got[1] * s["v_scale"].double()[None, :, None]
    return got[0], got[1]


def _exact_qk_norm_rope(s):
    q_out, pool = s["q_out"].double(), s["pool"].double()
    half = s["hd"] // 2
    for b in range(s["batch"]):
        n = s["m"] if s["rows"] is None else int(s["rows"][b])
        first = int(s["lens"][b])
        cs = torch.view_as_complex(s["rope"][first:first + n].double().contiguous())[:, None]

        def turned(x, gain):
            x = x[b, :n].double()
            if gain is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain.double()
            z = torch.complex(x[..., :half], x[..., half:]) * cs
            return torch.cat((z.real, z.imag), -1)

        q_out[b, :n] = turned(s["q"], s["q_gain"])
        k, v = turned(s["k"], s["k_gain"]), s["v"][b, :n].double()
        if s["k_scale"] is not None:
            k, v = k / s["k_scale"].double()[:, None], v / s["v_scale"].double()[:, None]
        for at in range(first // PAGE, (first + n - 1) // PAGE + 1):
            lo, hi = max(first, at * PAGE), min(first + n, (at + 1) * PAGE)
            page = int(s["page_table"][b, at])
            slots = slice(lo - at * PAGE, hi - at * PAGE)
            pool[page, 0, :, slots] = k[lo - first:hi - first].transpose(0, 1)
            pool[page, 1, :, slots] = v[lo - first:hi - first].transpose(0, 1)
    return {"q": q_out, "pool": pool}


def _exact_sample(s):
    tokens, probs = [], []
    for r in range(s["rows"]):
        x = s["logits"][r].double()
        t = float(s["temperature"][r])
        ids = torch.argsort(x, descending=True, stable=True)   # likeliest first, equal ones by index
        if t <= 0:
            tokens.append(int(ids[0]))
            probs.append(1.0)
            continue
        w = ((x[ids] - x[ids[0]]) / t).exp()
        if s["top_k"] is not None:
            k = int(s["top_k"][r])
            least = float(s["min_p"][r])
            p = float(s["top_p"][r])
            if k > 0:
                w = w[:k]
            n = w.numel()
            if p < 1:
                before = torch.cat((w.new_zeros(1), w.cumsum(0)[:-1]))
                n = max(1, int((before < p * w.sum()).sum()))
            w = w[:n]
            w = w[w >= least]
        ids, at = ids[:w.numel()].sort()
        w = w[at]
        c = w.cumsum(0)
        j = int(torch.searchsorted(c, float(s["u"][r]) * c[-1], right=True))
        tokens.append(int(ids[j]))
        probs.append(float(w[j] / c[-1]))
    return {"tokens": torch.tensor(tokens), "prob": torch.tensor(probs, dtype=torch.float64)}
