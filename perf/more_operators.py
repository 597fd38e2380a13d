"""Measured cases of a serving step's operators: paging, an 8-bit K/V cache, attention, sampling.

Four kinds of case:

  plan    block tables, slots and offsets of a step from the requests' lengths (memq_page_plan)
  cache   quantising keys and values into the paged cache, a scale for every 16 tokens of a head,
          and reading them back (memq_kv_cache_append, memq_kv_cache_read)
  attn    causal attention of each sequence's new tokens over that cache (memq_attn_paged)
  sample  one token a row of logits: temperature, top-k, top-p, min-p (memq_sample)

``own`` selects the framework's kernels; otherwise ``run`` evaluates the formulas with
elementary torch operations.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 16  # tokens that share a scale


def listed():
    return [
        # one request's next token: the bookkeeping of the smallest decode step
        dict(name="plan_1", kind="plan", seqs=1, chunk=1, page=64, pages=512, max_len=8192),
        # a large batch between two steps: decodes, prompt chunks, finished requests, rejected drafts
        dict(name="plan_1024", kind="plan", seqs=1024, chunk=512, page=32, pages=131072, max_len=32768),
        # one step's rows of a decode batch, most of them into blocks that hold rows already
        dict(name="cache_256x1_f32", kind="cache", seqs=256, t=1, start=1000, kv_heads=8, heads=40, d=128,
             page=64, type="f32"),
        # a prompt of odd length, written in one call
        dict(name="cache_1x16381_bf16", kind="cache", seqs=1, t=16381, start=0, kv_heads=8, heads=40, d=128,
             page=64, type="bf16"),
        # the smallest call: one token of one sequence, precise types
        dict(name="attn_1x1_kv2048", kind="attn", seqs=1, t=1, kv=2048, heads=40, kv_heads=8, d=128, page=64,
             type="f32", ragged=False),
        # one token over a long cache: few rows, a long axis
        dict(name="attn_1x1_kv131071", kind="attn", seqs=1, t=1, kv=131071, heads=64, kv_heads=8, d=128,
             page=64, type="bf16", ragged=False),
        # a serving batch of single tokens, every length another
        dict(name="attn_64x1_kv16384", kind="attn", seqs=64, t=1, kv=16384, heads=64, kv_heads=8, d=128,
             page=64, type="bf16", ragged=True),
        # ragged chunks, narrow heads, an odd number of them to a key head, small pages
        dict(name="attn_7x61_kv1999", kind="attn", seqs=7, t=61, kv=1999, heads=14, kv_heads=2, d=64, page=16,
             type="f32", ragged=True),
        # a chunk of a long prompt
        dict(name="attn_1x2048_kv16384", kind="attn", seqs=1, t=2048, kv=16384, heads=64, kv_heads=8, d=128,
             page=128, type="bf16", ragged=False),
        # one row of the logits of a small vocabulary
        dict(name="sample_1x32000", kind="sample", rows=1, vocab=32000, type="f32"),
        # eight requests, an odd vocabulary
        dict(name="sample_8x128259", kind="sample", rows=8, vocab=128259, type="f32"),
        # a large batch with every request's own settings
        dict(name="sample_256x131072", kind="sample", rows=256, vocab=131072, type="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["plan", "cache", "attn", "attn", "sample"])
    page, typ = rng.choice([16, 32, 64, 128]), rng.choice(["f32", "bf16"])
    if kind == "plan":
        seqs = _log(rng, 1, 1024)
        chunk = _log(rng, 1, 512)
        return dict(kind=kind, seqs=seqs, chunk=chunk, page=page, max_len=rng.choice([4096, 32768]),
                    pages=rng.choice([1, 2, 4]) * seqs * 1024 // page + 64)
    if kind == "sample":
        vocab = _log(rng, 1000, 262144)
        return dict(kind=kind, rows=_log(rng, 1, min(256, 2 ** 25 // vocab)), vocab=vocab, type=typ)
    d, kv_heads, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
    if kind == "cache":
        seqs = _log(rng, 1, 256)
        return dict(kind=kind, seqs=seqs, t=_log(rng, 1, max(1, 16384 // seqs)), start=rng.choice([0, 7, 1000]),
                    kv_heads=kv_heads, heads=kv_heads * group, d=d, page=page, type=typ)
    seqs, heads = _log(rng, 1, 64), kv_heads * group
    kv = _log(rng, 1, min(131072, 2 ** 20 // seqs))
    # the score matrix bounds the query rows; a third of the draws are single tokens
    most = max(1, min(2048, kv, 2 ** 29 // (seqs * heads * kv)))
    if rng.random() < 0.5:
        most = min(most, 8)
    t = 1 if rng.random() < 0.3 else _log(rng, 1, most)
    return dict(kind=kind, seqs=seqs, t=t, kv=kv, heads=heads, kv_heads=kv_heads, d=d, page=page, type=typ,
                ragged=rng.random() < 0.7)


def _lengths(case):
    """(new tokens, cached rows) of each sequence, the new tokens' own rows included."""
    out = []
    for b in range(case["seqs"]):
        f = 1.0 - 0.75 * ((b * 0.6180339887) % 1.0) if case["ragged"] else 1.0
        g = 1.0 - 0.75 * ((b * 0.4142135624) % 1.0) if case["ragged"] else 1.0
        t = max(1, round(case["t"] * g))
        out.append((t, max(t, round(case["kv"] * f))))
    return out


def _requests(case):
    """(cached, keep, new) of each request of a plan: fixed by the case."""
    out, page = [], case["page"]
    room = case["pages"] * page // (2 * case["seqs"])
    for b in range(case["seqs"]):
        f, g = (0.37 + b * 0.6180339887) % 1.0, (0.11 + b * 0.4142135624) % 1.0
        cached = max(1, min(int(room * f), case["max_len"] - case["chunk"]))
        keep, new = cached, 1
        if case["seqs"] > 1:
            if g < 0.05:  # finished
                keep, new = 0, 0
            elif g < 0.1:  # another request takes its place
                keep, new = 0, max(1, int(case["chunk"] * f))
            elif g < 0.2:  # rejected drafts
                keep, new = max(0, cached - 1 - b % 5), 4
            elif g < 0.25:  # a chunk of a prompt
                new = max(1, int(case["chunk"] * (1 - f)))
            elif g < 0.3:  # idle
                new = 0
        out.append((cached, keep, new))
    return out


def _pow2_scale(top):
    """The least power of two with top <= 448 * scale."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(top > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return torch.ldexp(torch.ones_like(top), e)


def _paged_rows(g, pages, n_kv, page, d, used, values):
    """A pool of which the rows `used` (pool rows, in whole blocks) hold quantised `values`
    [len(used), n_kv, d]; the others hold whatever was there before."""
    dev = "cuda"
    cache = torch.randint(0, 256, (pages, n_kv, page, d), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.zeros(pages, n_kv, page // BLOCK, device=dev)
    x = values.view(-1, BLOCK, n_kv, d)
    s = _pow2_scale(x.abs().amax((1, 3)))
    first = used.view(-1, BLOCK)[:, 0]
    scales.permute(0, 2, 1)[first // page, first % page // BLOCK] = s
    codes = (x / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    cache.permute(0, 2, 1, 3)[used // page, used % page] = codes.view(-1, n_kv, d)
    return cache, scales


def _up(n, m):
    return -(-n // m) * m


def _pages_of(g, lens, page, extra):
    """Random pages for the rows of each sequence: the table, and every row's place in the pool."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g, device="cuda")[: sum(need)].to(torch.int32).cpu()
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    rows, at = [], 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        rows.append((order[at:at + k].long()[:, None] * page + torch.arange(page)).reshape(-1))
        at += k
    return pages, table.to("cuda"), rows


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    empty = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
    kind = case["kind"]
    if kind == "plan":
        req, page, pages = _requests(case), case["page"], case["pages"]
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
        have = [-(-c // page) for c, _, _ in req]
        table = torch.full((len(req), case["max_len"] // page), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(have):
            table[b, :k] = order[at:at + k]
            at += k
        free = torch.full((pages,), -1, dtype=torch.int32)
        free[: pages - at] = order[at:]
        n = len(req)
        n_tok = _up(max(1, sum(r[2] for r in req)), 8)
        return dict(case=case, cached=i32([r[0] for r in req]), keep=i32([r[1] for r in req]),
                    new=i32([r[2] for r in req]), table=table.to(dev), free=free.to(dev), n_free=i32([pages - at]),
                    n_tok=n_tok, slots=empty(n_tok), positions=empty(n_tok), cu_q=empty(n + 1), kv_len=empty(n),
                    granted=empty(n), n_free_out=empty(1))
    if kind == "sample":
        rows, v = case["rows"], case["vocab"]
        logits = 2.0 * randn(rows, v)
        # what the model thinks of: some tokens stand out, by more in some rows than in others
        likely = torch.randint(0, v, (rows, 48), generator=g, device=dev)
        lift = 6 + 8 * torch.rand(rows, 1, generator=g, device=dev)
        logits.scatter_add_(1, likely, lift * torch.rand(rows, 48, generator=g, device=dev))
        pick = lambda xs: torch.tensor(xs, device=dev)[  # noqa: E731
            torch.randint(0, len(xs), (rows,), generator=g, device=dev)]
        if rows == 1:
            temperature, top_k, top_p, min_p = pick([0.8]), pick([50]), pick([0.95]), pick([0.0])
        else:
            temperature, top_k = pick([0.0, 0.6, 0.7, 0.9, 1.0, 1.0, 1.2]), pick([0, 0, 20, 50, 64, 500])
            top_p, min_p = pick([1.0, 0.8, 0.9, 0.95, 0.99]), pick([0.0, 0.0, 0.02, 0.1])
        return dict(case=case, logits=logits.to(DTYPES[case["type"]]), temperature=temperature,
                    top_k=top_k.to(torch.int32), top_p=top_p, min_p=min_p,
                    u=torch.rand(rows, generator=g, device=dev), out=empty(rows))
    heads, n_kv, d, page = case["heads"], case["kv_heads"], case["d"], case["page"]
    dt = DTYPES[case["type"]]
    if kind == "cache":
        # every sequence has `start` rows (a few more or less) and gets t; q, k and v come out of one projection
        starts = [max(0, case["start"] - b % 37) for b in range(case["seqs"])]
        lens = [s + case["t"] for s in starts]
        pages, _, rows = _pages_of(g, lens, page, 3)
        new = torch.cat([r[s:s + case["t"]] for r, s in zip(rows, starts)]).to(dev)
        back = torch.cat([r[s // BLOCK * BLOCK: s + case["t"]] for r, s in zip(rows, starts)]).to(dev)
        held = torch.cat([r[s // BLOCK * BLOCK: _up(s, BLOCK)] for r, s in zip(rows, starts)]).to(dev)
        n = new.numel()
        qkv = (randn(n, heads + 2 * n_kv, d) * torch.exp(0.3 * randn(n, heads + 2 * n_kv, 1))).to(dt)
        s = dict(case=case, k=qkv[:, heads:heads + n_kv], v=qkv[:, heads + n_kv:], slots=new.to(torch.int32),
                 back=back.to(torch.int32), out_k=torch.empty(back.numel(), n_kv, d, dtype=torch.bfloat16, device=dev),
                 out_v=torch.empty(back.numel(), n_kv, d, dtype=torch.bfloat16, device=dev))
        for x in "kv":
            s[x + "_cache"], s[x + "_scales"] = _paged_rows(g, pages, n_kv, page, d, held, randn(held.numel(), n_kv, d))
        return s
    lens = _lengths(case)
    n_tok = sum(t for t, _ in lens)
    pages, table, rows = _pages_of(g, [kv for _, kv in lens], page, 3)
    used = torch.cat([r[: _up(kv, BLOCK)] for r, (_, kv) in zip(rows, lens)]).to(dev)
    cu = [0]
    for t, _ in lens:
        cu.append(cu[-1] + t)
    qkv = randn(n_tok, heads + 2 * n_kv, d).to(dt)
    s = dict(case=case, q=qkv[:, :heads], table=table, kv_len=i32([kv for _, kv in lens]), cu_q=i32(cu),
             scale=d ** -0.5, max_t=max(t for t, _ in lens), max_kv=max(kv for _, kv in lens),
             out=torch.empty(n_tok, heads, d, dtype=dt, device=dev))
    for x in "kv":
        values = randn(used.numel(), n_kv, d) * torch.exp(0.3 * randn(used.numel(), n_kv, 1))
        s[x + "_cache"], s[x + "_scales"] = _paged_rows(g, pages, n_kv, page, d, used, values)
    return s


def _plan(s):
    page, n_tok, table, free = s["case"]["page"], s["n_tok"], s["table"], s["free"]
    cached, keep, new = s["cached"].long(), s["keep"].long(), s["new"].long()
    have, need = (cached + page - 1) // page, (keep + new + page - 1) // page
    push, pop = (have - need).clamp(min=0), (need - have).clamp(min=0)
    ends = torch.cumsum(pop, 0)
    stack = s["n_free"].long() + push.sum()
    granted = (pop == 0) | (ends <= stack)
    pop = torch.where(granted, pop, torch.zeros_like(pop))
    col = torch.arange(table.shape[1], device=table.device)[None]
    first = torch.cumsum(push, 0) - push
    gone = (col >= need[:, None]) & (col < have[:, None])
    at = s["n_free"].long() + first[:, None] + col - need[:, None]
    free[at[gone]] = table[gone]
    fresh = (col >= have[:, None]) & (col < need[:, None]) & granted[:, None]
    at = stack - 1 - ((ends - pop)[:, None] + col - have[:, None])
    table[fresh] = free[at[fresh]]
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    tok = torch.arange(n_tok, device=table.device)
    b = torch.searchsorted(cu[1:], tok, right=True).clamp(max=new.numel() - 1)
    live = tok < cu[-1]
    pos = keep[b] + tok - cu[b]
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    minus = torch.full_like(tok, -1)
    out = {"slots": torch.where(live & granted[b], slot, minus), "positions": torch.where(live, pos, minus),
           "cu_q": cu, "kv_len": torch.where(granted, keep + new, cached),
           "granted": granted, "n_free": (stack - pop.sum()).view(1)}
    out = {k: v.to(torch.int32) for k, v in out.items()}
    return dict(out, table=table, free=free)


def _values(cache, scales, rows):
    """The values that the pool's rows stand for: [n, n_kv, d]."""
    page = cache.shape[2]
    codes = cache.permute(0, 2, 1, 3)[rows // page, rows % page].view(torch.float8_e4m3fn).float()
    return codes * scales.permute(0, 2, 1)[rows // page, rows % page // BLOCK][:, :, None]


def _cache(s):
    out, slots = {}, s["slots"].long()
    for x in "kv":
        cache, scales, new = s[x + "_cache"], s[x + "_scales"], s[x].float()
        page = cache.shape[2]
        blk = slots // BLOCK
        lead = torch.ones_like(blk, dtype=torch.bool)
        lead[1:] = blk[1:] != blk[:-1]
        run = torch.cumsum(lead, 0) - 1
        blk = blk[lead]
        n_kv = new.shape[1]
        top = torch.zeros(blk.numel(), n_kv, device=new.device)
        top = top.scatter_reduce(0, run[:, None].expand(-1, n_kv), new.abs().amax(2), "amax")
        fresh = torch.zeros(blk.numel(), device=new.device).scatter_reduce(0, run, (slots % BLOCK == 0).float(), "amax")
        where = (blk * BLOCK // page, blk * BLOCK % page // BLOCK)
        old = scales.permute(0, 2, 1)[where]
        scale = _pow2_scale(top)
        scale = torch.where((fresh == 0)[:, None], torch.maximum(scale, old), scale)
        scales.permute(0, 2, 1)[where] = scale
        # rows that are there take the new scale
        rows = blk[:, None] * BLOCK + torch.arange(BLOCK, device=blk.device)
        view = cache.permute(0, 2, 1, 3)
        codes = view[rows // page, rows % page].view(torch.float8_e4m3fn).float()
        grown = (codes * (old / scale)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        moved = ((fresh == 0)[:, None] & (scale > old))[:, None, :, None]
        view[rows // page, rows % page] = torch.where(moved, grown, view[rows // page, rows % page])
        codes = (new / scale[run][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        view[slots // page, slots % page] = codes
        out[x] = _values(cache, scales, s["back"].long()).to(torch.bfloat16)
        out[x + "_scales"] = scales
    return out


def _attn(s):
    q = s["q"].float()
    n_tok, heads, d = q.shape
    n_kv, page = s["k_cache"].shape[1:3]
    table, kv_len, cu = s["table"].long(), s["kv_len"].long(), s["cu_q"].long()
    seqs, group = table.shape[0], heads // n_kv
    key = torch.arange(s["max_kv"], device=q.device)
    rows = table[:, key // page].clamp(min=0) * page + key % page
    held = key[None] < kv_len[:, None]
    k, v = (torch.where(held[:, :, None, None], _values(s[x + "_cache"], s[x + "_scales"], rows.view(-1)).view(
        seqs, -1, n_kv, d), torch.zeros((), device=q.device)).transpose(1, 2) for x in "kv")
    tok = torch.arange(n_tok, device=q.device)
    b = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[b]
    pad = torch.zeros(seqs, s["max_t"], heads, d, device=q.device)
    pad[b, i] = q
    pad = pad.view(seqs, -1, n_kv, group, d).transpose(1, 2).reshape(seqs, n_kv, -1, d)
    x = torch.matmul(pad, k.transpose(2, 3)).view(seqs, n_kv, s["max_t"], group, -1) * s["scale"]
    pos = (kv_len - (cu[1:] - cu[:-1]))[:, None] + torch.arange(s["max_t"], device=q.device)[None]
    seen = held[:, None, :] & (key[None, None] <= pos[:, :, None])
    x = x.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    top = x.amax(4, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(4, keepdim=True)
    o = torch.matmul(p.view(seqs, n_kv, -1, p.shape[4]), v).view(seqs, n_kv, s["max_t"], group, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 2, 1, 3, 4).reshape(seqs, s["max_t"], heads, d)[b, i].to(s["out"].dtype)


def _sample(s):
    # 64 bits: the draw and the cut of top-p fall next to borders between tokens
    x, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    rows, v = x.shape
    t = s["temperature"].double()[:, None]
    w = torch.exp((x - x[:, :1]) / torch.where(t > 0, t, torch.ones_like(t)))
    place = torch.arange(v, device=x.device)[None]
    k = torch.where((s["top_k"] > 0), s["top_k"].long(), torch.full_like(s["top_k"].long(), v))[:, None]
    k = torch.where(t > 0, k, torch.ones_like(k))
    w = torch.where(place < k, w, torch.zeros_like(w))
    run = torch.cumsum(w, 1)
    p = s["top_p"].double()[:, None]
    keep = (run - w < p * run[:, -1:]) | (p >= 1)
    keep &= w >= s["min_p"].double()[:, None]
    keep |= place == 0
    w = torch.where(keep, w, torch.zeros_like(w))
    by_token = torch.zeros_like(w).scatter_(1, order, w)
    run = torch.cumsum(by_token, 1)
    past = run > s["u"].double()[:, None] * run[:, -1:]
    return past.to(torch.int32).argmax(1).to(torch.int32)


def run(state):
    s, kind = state, state["case"]["kind"]
    if not own:
        return {"plan": _plan, "cache": _cache, "attn": _attn, "sample": _sample}[kind](s)
    import quantized_decode_memq_gb300 as memq
    if kind == "plan":
        slots, positions, cu_q, kv_len, granted, n_free = memq.memq_page_plan(
            s["cached"], s["new"], s["table"], s["free"], s["n_free"], s["case"]["page"], s["n_tok"], keep=s["keep"],
            slots=s["slots"], positions=s["positions"], cu_q=s["cu_q"], kv_len=s["kv_len"], granted=s["granted"],
            n_free_out=s["n_free_out"])
        return {"slots": slots, "positions": positions, "cu_q": cu_q, "kv_len": kv_len, "granted": granted,
                "n_free": n_free, "table": s["table"], "free": s["free"]}
    if kind == "cache":
        memq.memq_kv_cache_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scales"],
                                  s["v_scales"])
        out = {}
        for x in "kv":
            out[x] = memq.memq_kv_cache_read(s[x + "_cache"], s[x + "_scales"], s["back"], out=s["out_" + x])
            out[x + "_scales"] = s[x + "_scales"]
        return out
    if kind == "attn":
        return memq.memq_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"],
                                    s["kv_len"], s["cu_q"], s["scale"], out=s["out"])
    return memq.memq_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                            min_p=s["min_p"], out=s["out"])


def work(case):
    kind = case["kind"]
    if kind == "plan":
        page, req = case["page"], _requests(case)
        moved = sum(abs(-(-c // page) - -(-(k + n) // page)) for c, k, n in req)
        tokens = sum(r[2] for r in req)
        # lengths in; lengths, offsets and grants out; moved pages in and out; two numbers a token out
        return {"bytes": len(req) * 6 * 4 + moved * 8 + tokens * 8, "flops": 4 * tokens}
    size = 4 if case["type"] == "f32" else 2
    if kind == "sample":
        e = case["rows"] * case["vocab"]
        return {"bytes": e * size + case["rows"] * 24, "flops": 4 * e}
    n_kv, d = case["kv_heads"], case["d"]
    if kind == "cache":
        n, width = case["seqs"] * case["t"], 2 * n_kv * d
        # rows in, codes out; then codes in, bf16 values out; slots; scales twice
        return {"bytes": n * (width * (size + 1 + 1 + 2) + 12) + 16 * n * n_kv // BLOCK, "flops": 4 * n * width}
    lens, heads = _lengths(case), case["heads"]
    rows = sum(t for t, _ in lens) * heads
    pairs = sum(heads * (t * kv - t * (t - 1) // 2) for t, kv in lens)
    return {"bytes": sum(kv * d + _up(kv, BLOCK) * 4 // BLOCK for _, kv in lens) * n_kv * 2 + rows * d * 2 * size,
            "flops": pairs * 4 * d}


_E4M3 = None


def _decoded():
    """The 256 values of E4M3."""
    global _E4M3
    if _E4M3 is None:
        bits = torch.arange(256, device="cuda")
        e, f = (bits >> 3) & 15, bits & 7
        val = torch.where(e == 0, f.double() / 512, (8 + f).double() * torch.exp2(e.double() - 10))
        _E4M3 = torch.where(bits >= 128, -val, val)
    return _E4M3


def _to_e4m3(v):
    """To the nearest value of three fraction bits, exponents from -6 on."""
    _, e = torch.frexp(v)
    unit = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(v / unit) * unit


def _exact_plan(s, case):
    page, n_tok = case["page"], s["n_tok"]
    table, free = s["table"].tolist(), s["free"].tolist()
    stack = s["n_free"].item()
    req = list(zip(s["cached"].tolist(), s["keep"].tolist(), s["new"].tolist()))
    size = lambda n: (n + page - 1) // page  # noqa: E731
    for b, (cached, keep, new) in enumerate(req):
        for c in range(size(keep + new), size(cached)):
            free[stack] = table[b][c]
            stack += 1
    slots, positions, cu, kv_len, granted, asked, left = [], [], [0], [], [], 0, stack
    for b, (cached, keep, new) in enumerate(req):
        want = max(0, size(keep + new) - size(cached))
        asked += want
        ok = want == 0 or asked <= stack
        if ok:
            for c in range(size(cached), size(cached) + want):
                left -= 1
                table[b][c] = free[left]
        for i in range(keep, keep + new):
            positions.append(i)
            slots.append(table[b][i // page] * page + i % page if ok else -1)
        cu.append(cu[-1] + new)
        kv_len.append(keep + new if ok else cached)
        granted.append(int(ok))
    slots += [-1] * (n_tok - len(slots))
    positions += [-1] * (n_tok - len(positions))
    out = {"slots": slots, "positions": positions, "cu_q": cu, "kv_len": kv_len, "granted": granted, "n_free": [left],
           "table": table, "free": free}
    return {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in out.items()}


def _exact_cache(s, case):
    out, slots = {}, s["slots"].long()
    block, place = slots // BLOCK, slots % BLOCK
    for x in "kv":
        cache, scales, new = s[x + "_cache"], s[x + "_scales"].double(), s[x].double()
        pages, n_kv, page, d = cache.shape
        codes = _decoded()[cache.long()].transpose(1, 2).reshape(-1, BLOCK, n_kv, d)
        old = scales.transpose(1, 2).reshape(-1, n_kv)
        touched, which = torch.unique(block, return_inverse=True)
        rows = torch.zeros(touched.numel(), BLOCK, n_kv, d, dtype=torch.float64, device="cuda")
        rows[which, place] = new
        ours = torch.zeros(touched.numel(), BLOCK, dtype=torch.bool, device="cuda")
        ours[which, place] = True
        afresh = ours[:, 0]
        # the least power of two that takes the largest element to 448 or less
        top = rows.abs().amax((1, 3)).clamp(min=2.0 ** -100)
        scale = torch.exp2(torch.round(torch.log2(top)) - 7)
        for _ in range(3):
            scale = torch.where(top <= 224 * scale, scale / 2, scale)
        scale = scale.clamp(min=2.0 ** -100)
        scale = torch.where(afresh[:, None], scale, torch.maximum(scale, old[touched]))
        before = codes[touched] * (old[touched] / scale)[:, None, :, None]
        codes[touched] = torch.where(ours[:, :, None, None], _to_e4m3(rows / scale[:, None, :, None]),
                                     torch.where(afresh[:, None, None, None], codes[touched], _to_e4m3(before)))
        old[touched] = scale
        back = s["back"].long()
        out[x] = codes.view(-1, n_kv, d)[back] * old[back // BLOCK][:, :, None]
        out[x + "_scales"] = old.view(pages, page // BLOCK, n_kv).transpose(1, 2).contiguous()
    return out


def _exact_attn(s, case):
    heads, n_kv, d, page = case["heads"], case["kv_heads"], case["d"], case["page"]
    group, first = heads // n_kv, 0
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, (t, kv) in enumerate(_lengths(case)):
        ids = s["table"][b, : -(-kv // page)].long()
        step = max(1, 2 ** 27 // (kv * group))
        for h in range(n_kv):
            k, v = ((_decoded()[s[x + "_cache"][ids, h].long()]
                     * s[x + "_scales"][ids, h].double().repeat_interleave(BLOCK, 1)[:, :, None]).view(-1, d)[:kv]
                    for x in "kv")
            for i in range(0, t, step):
                n = min(step, t - i)
                at = slice(first + i, first + i + n), slice(h * group, (h + 1) * group)
                x = torch.einsum("ihd,kd->ihk", s["q"][at].double(), k) * s["scale"]
                last = kv - t + i + torch.arange(n, device="cuda")
                x += torch.where(torch.arange(kv, device="cuda")[None] > last[:, None], -math.inf, 0.0)[:, None]
                out[at] = torch.einsum("ihk,kd->ihd", torch.softmax(x, 2), v)
        first += t
    return out


def _exact_sample(s, case):
    tokens = []
    rows = zip(s["logits"].double(), s["temperature"].tolist(), s["top_k"].tolist(), s["top_p"].tolist(),
               s["min_p"].tolist(), s["u"].tolist())
    for x, t, k, p, floor, u in rows:
        if t <= 0:
            tokens.append((x == x.max()).nonzero()[0, 0])
            continue
        # token indices, the likeliest first, the lowest first among equals
        order = torch.argsort(-x, stable=True)[: k if 0 < k <= x.numel() else x.numel()]
        prob = torch.softmax(x[order] / t, 0)
        ahead = torch.cumsum(prob, 0) - prob
        n = max(1, int((ahead < p).sum())) if p < 1 else prob.numel()
        n = max(1, min(n, int((prob[:n] >= floor * prob[0]).sum())))
        kept, perm = torch.sort(order[:n])
        mass = torch.cumsum(prob[:n][perm], 0)
        tokens.append(kept[min(n - 1, int((mass <= u * mass[-1]).sum()))])
    return torch.stack(tokens).to(torch.int32)


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "cache": _exact_cache, "attn": _exact_attn, "sample": _exact_sample}[case["kind"]](s, case)
