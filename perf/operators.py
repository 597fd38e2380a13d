"""Measured cases of the operators around latent attention over a quantised, paged cache.

Three kinds of case, one per operator:

  norm    residual addition, RMSNorm and the q8_1 activation (memq_add_rmsnorm_q8_1)
  cache   quantising latent rows as they are written to the paged cache, and reading them back
          (memq_mla_cache_append, memq_mla_cache_read)
  attn    a chunk of new tokens attending, causally, to the E4M3 latent cache through a block
          table, queries in the latent space (memq_mla_attn_paged)

``own`` selects the framework's kernels; otherwise ``run`` evaluates the formulas with
elementary torch operations.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
D_HEAD = 256  # width of a head before absorption: the score scale is (D_HEAD + rope)^-1/2


def listed():
    return [
        # one token's hidden row between two layers of a decode step
        dict(name="norm_1x5120", kind="norm", rows=1, ncols=5120),
        # eight rows (drafted tokens, or eight sequences) at the widest projection
        dict(name="norm_8x17408", kind="norm", rows=8, ncols=17408),
        # a long prompt's rows
        dict(name="norm_4096x8192", kind="norm", rows=4096, ncols=8192),
        # the latent rows of one decode step of eight tokens
        dict(name="cache_8_f32", kind="cache", n=8, rank=512, rope=0, page=64, type="f32", pool=32768),
        # a prompt of odd length with the decoupled position part, written in one call
        dict(name="cache_16381_bf16", kind="cache", n=16381, rank=512, rope=64, page=64, type="bf16",
             pool=65536),
        # the smallest call: one token of one sequence over 2048 cached rows
        dict(name="attn_1x1_kv2048", kind="attn", seqs=1, t=1, kv=2048, heads=64, rank=512, rope=0,
             page=64, type="f32", ragged=False),
        # one token over a long cache: few rows, a long axis
        dict(name="attn_1x1_kv32768", kind="attn", seqs=1, t=1, kv=32768, heads=64, rank=512, rope=0,
             page=64, type="f32", ragged=False),
        # eight drafted tokens of one sequence
        dict(name="attn_1x8_kv32768", kind="attn", seqs=1, t=8, kv=32768, heads=64, rank=512, rope=64,
             page=64, type="bf16", ragged=False),
        # a serving batch of single tokens, every length another
        dict(name="attn_48x1_kv16384", kind="attn", seqs=48, t=1, kv=16384, heads=64, rank=512,
             rope=64, page=64, type="bf16", ragged=True),
        # few heads, ragged chunks and small pages
        dict(name="attn_7x61_kv1999", kind="attn", seqs=7, t=61, kv=1999, heads=16, rank=256, rope=32,
             page=16, type="bf16", ragged=True),
        # a chunk of a long prompt
        dict(name="attn_1x2048_kv8192", kind="attn", seqs=1, t=2048, kv=8192, heads=64, rank=512,
             rope=64, page=128, type="bf16", ragged=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["norm", "cache", "attn", "attn"])
    if kind == "norm":
        ncols = 32 * _log(rng, 16, 544)
        return dict(kind=kind, rows=_log(rng, 1, min(4096, 2 ** 25 // ncols)), ncols=ncols)
    rank, rope = rng.choice([128, 256, 512]), rng.choice([0, 32, 64, 128])
    page, typ = rng.choice([16, 32, 64, 128]), rng.choice(["f32", "bf16"])
    if kind == "cache":
        return dict(kind=kind, n=_log(rng, 1, 8192), rank=rank, rope=rope, page=page, type=typ,
                    pool=rng.choice([8192, 32768]))
    heads = rng.choice([8, 16, 24, 40, 64, 96, 128])
    seqs, kv = _log(rng, 1, 48), _log(rng, 1, 32768)
    # the score matrix bounds the query rows; a third of the draws are single tokens
    most = max(1, min(2048, kv, 2 ** 29 // (seqs * heads * kv)))
    if rng.random() < 0.5:
        most = min(most, 8)
    t = 1 if rng.random() < 0.3 else _log(rng, 1, most)
    return dict(kind=kind, seqs=seqs, t=t, kv=kv, heads=heads, rank=rank, rope=rope, page=page, type=typ,
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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if case["kind"] == "norm":
        rows, n = case["rows"], case["ncols"]
        return dict(case=case, x=randn(rows, n), res=4 * randn(rows, n), w=1 + 0.1 * randn(n),
                    h=torch.empty(rows, n, device=dev),
                    qs=torch.empty(rows, n, dtype=torch.int8, device=dev),
                    d=torch.empty(rows, n // 32, device=dev),
                    y=torch.empty(rows, n // 32, 32, dtype=torch.bfloat16, device=dev))
    rank, rope, page, dt = case["rank"], case["rope"], case["page"], DTYPES[case["type"]]
    width = rank + rope
    if case["kind"] == "cache":
        n, pages = case["n"], case["pool"] // page
        return dict(case=case, latent=(randn(n, rank) * torch.exp(0.3 * randn(n, 1))).to(dt),
                    k_pe=randn(n, rope).to(dt) if rope else None,
                    slots=torch.randperm(pages * page, generator=g, device=dev)[:n].to(torch.int32),
                    cache=torch.zeros(pages, page, width, dtype=torch.uint8, device=dev),
                    scales=torch.zeros(pages, page, device=dev),
                    out=torch.empty(n, width, dtype=torch.bfloat16, device=dev))
    lens = _lengths(case)
    heads, n_tok = case["heads"], sum(t for t, _ in lens)
    need = [-(-kv // page) for _, kv in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev)[: sum(need)].to(torch.int32).cpu()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    slots, at = [], 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        slots.append((order[at:at + k].long()[:, None] * page + torch.arange(page)).reshape(-1)[: lens[b][1]])
        at += k
    slots = torch.cat(slots).to(dev)
    # rows that no sequence owns hold whatever was there before
    cache = torch.randint(0, 256, (pages * page, width), generator=g, device=dev, dtype=torch.uint8)
    scales = torch.full((pages * page,), float("nan"), device=dev)
    rows = randn(slots.numel(), width) * torch.exp(0.3 * randn(slots.numel(), 1))
    s = rows.abs().amax(1) / 448
    cache[slots] = (rows / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scales[slots] = s
    cu = [0]
    for t, _ in lens:
        cu.append(cu[-1] + t)
    return dict(case=case, q_lat=randn(n_tok, heads, rank).to(dt),
                q_pe=randn(n_tok, heads, rope).to(dt) if rope else None,
                cache=cache.view(pages, page, width), scales=scales.view(pages, page),
                table=table.to(dev), kv_len=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=dev),
                cu_q=torch.tensor(cu, dtype=torch.int32, device=dev), scale=(D_HEAD + rope) ** -0.5,
                max_t=max(t for t, _ in lens), max_kv=max(kv for _, kv in lens),
                out=torch.empty(n_tok, heads, rank, dtype=torch.bfloat16, device=dev))


def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _norm(s):
    h = s["x"] + s["res"]
    rr = 1 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)
    z = (h * rr.float()) * s["w"]
    blk = z.view(z.shape[0], -1, 32)
    d = blk.abs().amax(2, keepdim=True) / 127
    v = (blk / torch.where(d == 0, torch.ones_like(d), d)).double()
    qs = torch.sign(v) * torch.floor(v.abs() + 0.5)  # ties away from zero
    return {"h": h, "y": (qs.float() * d).to(torch.bfloat16)}


def _cache(s):
    x = s["latent"].float()
    if s["k_pe"] is not None:
        x = torch.cat([x, s["k_pe"].float()], 1)
    scale = x.abs().amax(1) / 448
    codes = (x / torch.where(scale == 0, torch.ones_like(scale), scale)[:, None]).to(torch.float8_e4m3fn)
    slots = s["slots"].long()
    cache, scales = s["cache"].view(-1, x.shape[1]), s["scales"].view(-1)
    cache[slots] = codes.view(torch.uint8)
    scales[slots] = scale
    return {"values": (_e4m3(cache[slots]) * scales[slots][:, None]).to(torch.bfloat16), "scales": s["scales"]}


def _attn(s):
    q = s["q_lat"].float()
    rank = q.shape[2]
    if s["q_pe"] is not None:
        q = torch.cat([q, s["q_pe"].float()], 2)
    n_tok, heads, width = q.shape
    table, kv_len, cu = s["table"].long(), s["kv_len"].long(), s["cu_q"].long()
    seqs, page = table.shape[0], s["cache"].shape[1]
    key = torch.arange(s["max_kv"], device=q.device)
    slot = table[:, key // page].clamp(min=0) * page + key % page
    held = key[None] < kv_len[:, None]
    c = _e4m3(s["cache"].view(-1, width)[slot]) * s["scales"].view(-1)[slot][:, :, None]
    c = torch.where(held[:, :, None], c, torch.zeros_like(c))
    tok = torch.arange(n_tok, device=q.device)
    b = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[b]
    pad = torch.zeros(seqs, s["max_t"], heads, width, device=q.device)
    pad[b, i] = q
    x = torch.matmul(pad.view(seqs, -1, width), c.transpose(1, 2)).view(seqs, s["max_t"], heads, -1) * s["scale"]
    pos = (kv_len - (cu[1:] - cu[:-1]))[:, None] + torch.arange(s["max_t"], device=q.device)[None]
    seen = held[:, None, :] & (key[None, None] <= pos[:, :, None])
    x = x.masked_fill(~seen[:, :, None, :], float("-inf"))
    top = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p.view(seqs, -1, p.shape[3]), c[:, :, :rank]).view(seqs, s["max_t"], heads, rank)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    return o[b, i].to(torch.bfloat16)


def run(state):
    kind = state["case"]["kind"]
    if own:
        import quantized_decode_memq_gb300 as memq
        if kind == "norm":
            h, _, qs, d = memq.memq_add_rmsnorm_q8_1(state["x"], state["res"], state["w"], EPS, h=state["h"],
                                                     qs=state["qs"], d=state["d"], want_z=False)
            y = torch.mul(qs.view(state["y"].shape), d.unsqueeze(2), out=state["y"])
            return {"h": h, "y": y}
        if kind == "cache":
            memq.memq_mla_cache_append(state["latent"], state["k_pe"], state["slots"], state["cache"],
                                       state["scales"])
            values = memq.memq_mla_cache_read(state["cache"], state["scales"], state["slots"], out=state["out"])
            return {"values": values, "scales": state["scales"]}
        return memq.memq_mla_attn_paged(state["q_lat"], state["q_pe"], state["cache"], state["scales"],
                                        state["table"], state["kv_len"], state["cu_q"], state["scale"],
                                        out=state["out"])
    if kind == "norm":
        return _norm(state)
    return _cache(state) if kind == "cache" else _attn(state)


def work(case):
    if case["kind"] == "norm":
        e = case["rows"] * case["ncols"]
        # x, the residual and the weight in; the sum, the codes and their scales out
        return {"bytes": e * (4 + 4 + 4 + 1 + 4 / 32) + 4 * case["ncols"], "flops": 8 * e}
    width, size = case["rank"] + case["rope"], 4 if case["type"] == "f32" else 2
    if case["kind"] == "cache":
        # rows in, codes and scales out; then codes and scales in, bf16 values out
        return {"bytes": case["n"] * (width * size + 4 + width + 4 + width + 4 + 4 + 2 * width),
                "flops": case["n"] * width * 4}
    lens = _lengths(case)
    heads = case["heads"]
    rows = sum(t for t, _ in lens) * heads
    pairs = sum(heads * (t * kv - t * (t - 1) // 2) for t, kv in lens)
    return {"bytes": sum(kv for _, kv in lens) * (width + 4) + rows * (width * size + case["rank"] * 2),
            "flops": pairs * 2 * (width + case["rank"])}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        h = s["x"].double() + s["res"].double()
        z = h * torch.rsqrt((h ** 2).sum(1, keepdim=True) / case["ncols"] + EPS) * s["w"].double()
        z = z.unflatten(1, (-1, 32))
        step = z.abs().max(2, keepdim=True).values / 127
        n = z / step.clamp(min=1e-300)
        whole = torch.trunc(n)
        return {"h": h, "y": (whole + torch.trunc(2 * (n - whole))) * step}
    if case["kind"] == "cache":
        x = s["latent"].double()
        if s["k_pe"] is not None:
            x = torch.cat((x, s["k_pe"].double()), 1)
        step = x.abs().max(1, keepdim=True).values / 448
        v = x / step.clamp(min=1e-300)
        # E4M3: three fraction bits, exponents from -6 on
        _, e = torch.frexp(v)
        unit = torch.exp2((e - 4).clamp(min=-9).double())
        scales = torch.zeros(case["pool"], dtype=torch.float64, device="cuda")
        scales[s["slots"].long()] = step[:, 0]
        return {"values": torch.round(v / unit) * unit * step, "scales": scales.view(s["scales"].shape)}
    rank, page = case["rank"], case["page"]
    bits = torch.arange(256, device="cuda")
    e, f = (bits >> 3) & 15, bits & 7
    val = torch.where(e == 0, f.double() / 512, (8 + f).double() * torch.exp2(e.double() - 10))
    val = torch.where(bits >= 128, -val, val)
    outs, first = [], 0
    for b, (t, kv) in enumerate(_lengths(case)):
        ids = s["table"][b, : -(-kv // page)].long()
        c = val[s["cache"][ids].reshape(-1, s["cache"].shape[2])[:kv].long()]
        c = c * s["scales"][ids].reshape(-1)[:kv, None].double()
        step = max(1, 2 ** 27 // (kv * case["heads"]))
        for i in range(0, t, step):
            n = min(step, t - i)
            q = s["q_lat"][first + i: first + i + n].double()
            if s["q_pe"] is not None:
                q = torch.cat((q, s["q_pe"][first + i: first + i + n].double()), 2)
            last = kv - t + i + torch.arange(n, device="cuda")
            x = torch.einsum("ihd,kd->ihk", q, c) * s["scale"]
            x += torch.where(torch.arange(kv, device="cuda")[None] > last[:, None], -math.inf, 0.0)[:, None]
            outs.append(torch.einsum("ihk,kd->ihd", torch.softmax(x, 2), c[:, :rank]))
        first += t
    return torch.cat(outs)
