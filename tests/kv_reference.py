"""Plain f64 evaluation of the K/V cache's operations, the page plan and the sampler, for the tests, with
bounds of what the attention kernels may be off.

Written from the formulas; imports nothing from the product."""
from __future__ import annotations

import numpy as np

from paged_reference import E4M3, bf16, to_e4m3

BLOCK = 16


def scale_of(top: float) -> float:
    """The least power of two, 2^-100 at least, with top <= 448 * scale."""
    scale = 2.0 ** -100
    while top > 448 * scale:
        scale *= 2
    return scale


def append(k, v, slots, caches, scales, page):
    """k, v f32 [n, n_kv, d]; caches (codes [pages, n_kv, page, d] twice) and scales (f32 [pages, n_kv, page /
    16] twice) are changed."""
    pool = caches[0].shape[0] * page
    runs = []
    for r, s in enumerate(slots):
        if s < 0 or s >= pool:
            continue
        if runs and runs[-1][-1] == r - 1 and slots[r - 1] // BLOCK == s // BLOCK:
            runs[-1].append(r)
        else:
            runs.append([r])
    for run in runs:
        block = slots[run[0]] // BLOCK
        p, j = block * BLOCK // page, block * BLOCK % page // BLOCK
        places = [int(slots[r]) % BLOCK for r in run]
        for h in range(k.shape[1]):
            fin = [np.isfinite(k[r, h]).all() and np.isfinite(v[r, h]).all() for r in run]
            for x, cache, scale in ((k, caches[0], scales[0]), (v, caches[1], scales[1])):
                rows = cache[p, h, j * BLOCK:(j + 1) * BLOCK]
                new = scale_of(max([float(np.abs(x[r, h]).max()) for r, f in zip(run, fin) if f], default=0.0))
                old = float(scale[p, h, j])
                if 0 not in places and 0 < old < np.inf:
                    new = max(new, 2.0 ** np.ceil(np.log2(old)))
                    if new != old:
                        others = [i for i in range(BLOCK) if i not in places]
                        nan = (rows[others] & 127) == 127
                        moved = to_e4m3((np.where(nan, 0, E4M3[rows[others]]) * (old / new)).astype(np.float32))
                        rows[others] = np.where(nan, 0x7f, moved)
                scale[p, h, j] = new
                for r, i, f in zip(run, places, fin):
                    rows[i] = to_e4m3(x[r, h].astype(np.float64) / new) if f else (0x7f if x is k else 0)


def values(cache, scales, slots):
    """f64 [n, n_kv, d] of the rows that the slots name; a negative slot gives zeros."""
    page = cache.shape[2]
    out = np.zeros((len(slots), cache.shape[1], cache.shape[3]))
    for r, s in enumerate(slots):
        if s >= 0:
            p, i = s // page, s % page
            out[r] = E4M3[cache[p, :, i]] * scales[p, :, i // BLOCK, None].astype(np.float64)
    return out


def attend(q, k, v, t, scale, p_terms, out_eps, vs):
    """Attention of the last t tokens of a sequence: q f64 [t, nh, d] (the exact inputs), k, v f64 [kv,
    n_kv, d], vs f64 [kv, n_kv], the values' scales.  Returns (out [t, nh, d], bound of |kernel - out|).

    The bound adds up what the kernels' roundings can do (f16 rounds by 2^-11 of a number, by 2^-25 below
    2^-14; f32 by 2^-24):
      query     f32: the remainder's rounding, 2^-22 |q|, and 2^-39 of the row's largest; bf16: the latter
      scores    sums of d products on the tensor cores, 2^-17 of the sum of |products|; then three products
                and the argument of exp2, of |s log2 e| + |reference| + 15 at most, 4 x 2^-24 of that;
                exp2 itself 2^-22
      weights   u = exp(s) vs: 2^-11 u (two terms 2^-22 u), and 2^-25 against 2^9 at a reference that is
                at most the largest u: 2^-34 max u; |codes| <= 448 multiply it
      sums      a term of n is rounded n times at most: (kv / 16 + 64) 2^-23 of the sum of |terms|, for the
                weights and the outputs
      output    one rounding to its type
    """
    exact_q = np.array_equal(q, bf16(q.astype(np.float32)).astype(np.float64))
    kv, n_kv, d = k.shape
    nh = q.shape[1]
    group = nh // n_kv
    out, bound = np.zeros((2, t, nh, d))
    p_eps = 2.0 ** -22 if p_terms == 2 else 2.0 ** -11
    for i in range(t):
        seen = kv - t + i + 1
        if seen <= 0:
            continue
        for h in range(n_kv):
            ci, vi, si = k[:seen, h], v[:seen, h], vs[:seen, h]
            qi = q[i, h * group:(h + 1) * group]
            s = scale * qi @ ci.T
            mag = abs(scale) * np.abs(qi) @ np.abs(ci).T
            ds = 2.0 ** -39 * np.abs(qi).max(1)[:, None] * np.abs(ci).sum(1)[None] * abs(scale)
            if not exact_q:
                ds = ds + 2.0 ** -22 * mag
            ref = 1.45 * np.abs(s).max(1, keepdims=True) + np.abs(np.log2(np.maximum(si, 2.0 ** -100))).max() + 15
            ds = ds + 2.0 ** -17 * mag + 4 * 2.0 ** -24 * (1.45 * np.abs(s) + ref) + 2.0 ** -22
            p = np.exp(s - s.max(1, keepdims=True))
            total = p.sum(1, keepdims=True)
            o = p @ vi / total
            u = p * si
            du = p_eps * u + 2.0 ** -34 * u.max(1, keepdims=True)
            a = np.abs(vi)
            codes = a / np.maximum(si, 2.0 ** -200)[:, None]
            grow = np.expm1(np.minimum(ds, 50.0))
            b = ((p * grow) @ a + (p * grow).sum(1, keepdims=True) * np.abs(o)) / total
            b += du @ codes / total + (kv / 16 + 64) * 2.0 ** -23 * (p @ a / total + np.abs(o))
            at = slice(h * group, (h + 1) * group)
            out[i, at] = o
            bound[i, at] = b * (1 + out_eps) + out_eps * np.abs(o) + 2.0 ** -90
    return out, bound


def plan(cached, keep, new, table, free, n_free, page, n_tok):
    """The page plan, request by request; table and free are changed.  Returns (slots, positions, cu_q,
    kv_len, granted, n_free)."""
    need = lambda n: -(-n // page)  # noqa: E731
    n, room = len(cached), table.shape[1] * page
    cu = np.minimum(np.r_[0, np.cumsum(new)], n_tok)
    fits = [keep[b] + new[b] <= room and sum(new[:b + 1]) <= n_tok for b in range(n)]
    stack = n_free
    for b in range(n):
        if fits[b]:
            for c in range(need(keep[b] + new[b]), need(cached[b])):
                free[stack] = table[b, c]
                stack += 1
    slots, positions = np.full(n_tok, -1), np.full(n_tok, -1)
    kv_len, granted, asked, left = np.array(cached), np.zeros(n, int), 0, stack
    for b in range(n):
        want = max(0, need(keep[b] + new[b]) - need(cached[b])) if fits[b] else 0
        asked += want
        granted[b] = fits[b] and (want == 0 or asked <= stack)
        if granted[b]:
            for c in range(need(cached[b]), need(cached[b]) + want):
                left -= 1
                table[b, c] = free[left]
            kv_len[b] = keep[b] + new[b]
        for i in range(cu[b + 1] - cu[b]):
            positions[cu[b] + i] = keep[b] + i
            if granted[b]:
                slots[cu[b] + i] = table[b, (keep[b] + i) // page] * page + (keep[b] + i) % page
    return slots, positions, cu, kv_len, granted, left


def sample(logits, temperature, k, p, min_p, u):
    """The tokens that the sampler may give for one row: the draw's own, and those at borders that its
    weights, each within 2^-41, cannot tell apart."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    v = len(x)
    top = x.max()
    if not temperature > 0 or top == -np.inf:
        best = np.flatnonzero(x == top)
        if top == -np.inf and not np.isnan(logits).all():
            best = np.flatnonzero(logits == -np.inf)
        return {int(best[0])}
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / max(float(temperature), 1e-30)))
    order = np.lexsort((np.arange(v), -x))
    if 0 < k < v:
        order = order[:k]
    if p <= 0:
        order = order[:1]
    eps = len(order) * 2.0 ** -41
    got = set()
    for dp in (-eps, eps):
        kept = order
        if 0 < p < 1:
            cum = np.cumsum(w[order])
            kept = order[:max(1, int((cum - w[order] < p * cum[-1] + dp).sum()))]
        for df in (-2.0 ** -41, 2.0 ** -41) if min_p > 0 else (0.0,):
            some = kept[(w[kept] >= min(float(min_p), 1.0) + df) | (np.arange(len(kept)) == 0) | (w[kept] == 1)]
            some = np.sort(some)
            some = some[w[some] > 0]
            cum = np.cumsum(w[some])
            for du in (-eps, eps):
                goal = max(0.0, float(min(max(u, 0.0), 1.0)) * cum[-1] + du)
                got.add(int(some[min(len(some) - 1, int((cum <= goal).sum()))]))
    return got
