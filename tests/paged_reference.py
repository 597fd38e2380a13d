"""Plain f64 evaluation of the paged latent cache's operations, for the tests: the cache's
quantisation, its read, and causal attention over it, with bounds of what the kernels may be off.

Written from the formulas; imports nothing from the product."""
from __future__ import annotations

import numpy as np

U24 = 2.0 ** -24


def e4m3_table() -> np.ndarray:
    """The 256 values of E4M3 (bias 7, subnormals below 2^-6, 0x7F / 0xFF NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


E4M3 = e4m3_table()


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """f32 -> E4M3 codes: nearest, ties to even, saturating at 448."""
    v = np.abs(x.astype(np.float64))
    _, e = np.frexp(v)
    unit = np.exp2(np.maximum(e - 4, -9).astype(np.float64))  # spacing of the codes around v
    q = np.minimum(np.rint(v / unit) * unit, 448.0)
    code = np.searchsorted(E4M3[:127], q)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def bf16(x: np.ndarray) -> np.ndarray:
    """f32 rounded to bf16 (nearest, ties to even), as f32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def quantise(rows: np.ndarray):
    """(codes, scales) of f32 rows: scale = max|x| / 448 and code = e4m3(x / scale), f32 divisions; a
    row that is not finite has zero codes and a NaN scale."""
    rows = rows.astype(np.float32)
    ok = np.isfinite(rows).all(1)
    safe = np.where(ok[:, None], rows, np.float32(0))
    scale = np.abs(safe).max(1) / np.float32(448)
    div = np.where(scale == 0, np.float32(1), scale)
    codes = np.where(scale[:, None] == 0, np.uint8(0), to_e4m3(safe / div[:, None]))
    return codes, np.where(ok, scale, np.float32(np.nan)).astype(np.float32)


def attend(q, codes, scales, t, rank, scale, out_eps):
    """Attention of the last t tokens of a sequence: q f64 [t, nh, width] (the exact inputs), codes
    uint8 [kv, width], scales f32 [kv].  Returns (out [t, nh, rank], bound of |kernel - out|).

    The bound adds up, per output, what the kernel's roundings can do:
      query terms  |dq| <= 1.13 * 2^-8 |q| + 2^-17 max|q|   (0 in the first term for a bf16 query)
      scores       f32 sums of 576 products and more: 2^-17 of the sum of |products|, and the
                   argument of exp2: 2^-20 (|s| + 2)
      weights      u = exp(s) * scale: 1.07 * 2^-7 u + 2^-14 max u
      sums         f32 sums of weights and of outputs over the keys: 2^-16 of the sum of |terms|
      output       one rounding to its type: out_eps |out|
    """
    exact_q = np.array_equal(q, bf16(q.astype(np.float32)).astype(np.float64))
    kv = codes.shape[0]
    nh, width = q.shape[1], q.shape[2]
    c = E4M3[codes] * scales[:, None].astype(np.float64)
    out = np.zeros((t, nh, rank))
    bound = np.zeros((t, nh, rank))
    for i in range(t):
        seen = kv - t + i + 1
        if seen <= 0:
            continue
        ci, si = c[:seen], scales[:seen].astype(np.float64)
        s = scale * q[i] @ ci.T                                        # [nh, seen]
        mag = abs(scale) * np.abs(q[i]) @ np.abs(ci).T
        dq = 2.0 ** -17 * np.abs(q[i]).max(1)[:, None] * np.abs(ci).sum(1)[None] * abs(scale)
        if not exact_q:
            dq = dq + 1.13 * 2.0 ** -8 * mag
        ds = dq + 2.0 ** -17 * mag + 2.0 ** -20 * (np.abs(s) + 2)
        p = np.exp(s - s.max(1, keepdims=True))
        total = p.sum(1, keepdims=True)
        o = p @ ci[:, :rank] / total
        u = p * si
        du = 1.07 * 2.0 ** -7 * u + 2.0 ** -14 * u.max(1, keepdims=True)
        a = np.abs(ci[:, :rank])
        mean = p @ a / total                                           # of |v|
        codes_abs = np.abs(E4M3[codes[:seen, :rank]])
        grow = np.expm1(np.minimum(ds, 50.0))
        b = ((p * grow) @ a + (p * grow).sum(1, keepdims=True) * np.abs(o)) / total
        b += du @ codes_abs / total + 2.0 ** -16 * (mean + np.abs(o))
        out[i] = o
        bound[i] = b * (1 + out_eps) + out_eps * np.abs(o) + 1e-30
    return out, bound


def attend_batch(q, table, kv_len, cu_q, codes, scales, rank, scale, out_eps):
    """attend() of every sequence: q f64 [n_tok, nh, width], codes [pages, page, width]."""
    page = codes.shape[1]
    out = np.full(q.shape[:2] + (rank,), np.nan)
    bound = np.full_like(out, np.nan)
    for b in range(len(kv_len)):
        t, kv = cu_q[b + 1] - cu_q[b], kv_len[b]
        ids = table[b, : -(-kv // page)]
        cb = codes[ids].reshape(-1, codes.shape[2])[:kv]
        sb = scales[ids].reshape(-1)[:kv]
        out[cu_q[b]:cu_q[b + 1]], bound[cu_q[b]:cu_q[b + 1]] = attend(
            q[cu_q[b]:cu_q[b + 1]], cb, sb, t, rank, scale, out_eps)
    return out, bound
