"""GPU parity of the paged latent cache (append, read), causal attention over it, and
memq_add_rmsnorm_q8_1.

The cache's writes and reads are compared bit for bit with the IEEE evaluation of their formulas; the
attention with the f64 reference within the bound that paged_reference.attend derives from the
kernel's roundings; the producer bit for bit with memq_rmsnorm_q8_1 on the sum."""
import numpy as np
import pytest
import torch

import paged_reference as ref
from gpu_helpers import to_dev

pytestmark = pytest.mark.gpu

EPS_OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -22}


@pytest.fixture(scope="module")
def memq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_decode_memq_gb300 import build
    build.build()
    import quantized_decode_memq_gb300 as m
    m.memq_device_fault()
    return m


# ------------------------------------------------------------------------------- the producer
@pytest.mark.parametrize("rows,ncols", [(1, 32), (1, 5120), (8, 17408), (3, 160), (5, 8224), (1, 32768), (4097, 64),
                                       (2, 1056), (40, 2080), (3, 4096), (19, 8192), (20, 8192), (300, 16416),
                                       (1, 4128), (25, 32768), (600, 1536), (1600, 5152)])
def test_add_rmsnorm_is_the_producer_on_the_sum(memq, rows, ncols):
    g = torch.Generator("cuda").manual_seed(rows * ncols)
    x = torch.randn(rows, ncols, device="cuda", generator=g)
    res = 3 * torch.randn(rows, ncols, device="cuda", generator=g)
    w = torch.randn(ncols, device="cuda", generator=g)
    h, z, qs, d = memq.memq_add_rmsnorm_q8_1(x, res, w, 1e-5)
    assert torch.equal(h, x + res)
    z2, qs2, d2 = memq.memq_rmsnorm_q8_1(h, w, 1e-5)
    assert torch.equal(z, z2) and torch.equal(qs, qs2) and torch.equal(d, d2)
    for target in (res, x):  # the residual updated in place, over either input
        a, b = x.clone(), res.clone()
        t = b if target is res else a
        h3, z3, qs3, d3 = memq.memq_add_rmsnorm_q8_1(a, b, w, 1e-5, h=t, want_z=False)
        assert h3 is t and z3 is None
        assert torch.equal(t, h) and torch.equal(qs3, qs) and torch.equal(d3, d)
        assert torch.equal(b if t is a else a, res if t is a else x)


@pytest.mark.parametrize("rows,ncols", [(6, 5120), (6, 96), (6, 17408), (400, 2048)])
def test_add_rmsnorm_special_values(memq, rows, ncols):
    """Rows that are not finite, overflow in the sum, or are denormal: the producer's bits all the same."""
    g = torch.Generator("cuda").manual_seed(ncols)
    x = torch.randn(rows, ncols, device="cuda", generator=g)
    x[0, 5], x[1, 7] = float("inf"), float("nan")
    x[2] *= 1e-39
    x[3] = 3e38
    x[4] *= 1e18
    res = torch.where(x.abs() > 1e17, x, 0.25 * x)
    w = torch.randn(ncols, device="cuda", generator=g)
    w[:32], w[32:64], w[64:96] = 1e-38, 1e30, 0
    h, z, qs, d = memq.memq_add_rmsnorm_q8_1(x, res, w)
    bits = lambda t: t.view(torch.int32)
    assert torch.equal(bits(h), bits(x + res))
    z2, qs2, d2 = memq.memq_rmsnorm_q8_1(h, w)
    assert torch.equal(bits(z), bits(z2)) and torch.equal(qs, qs2) and torch.equal(bits(d), bits(d2))


def test_add_rmsnorm_vector_in_place_is_not_a_copy(memq):
    x, w = torch.randn(64, device="cuda"), torch.ones(64, device="cuda")
    h = torch.zeros(64, device="cuda")
    assert memq.memq_add_rmsnorm_q8_1(x, x, w, h=h)[0] is h and torch.equal(h, x + x)
    for bad in (torch.zeros(128, device="cuda")[::2], torch.zeros(2, 4, 16, device="cuda").transpose(0, 1)):
        with pytest.raises(ValueError):
            memq.memq_add_rmsnorm_q8_1(x, x, w, h=bad)
    with pytest.raises((TypeError, ValueError)):
        memq.memq_add_rmsnorm_q8_1(x, x, w, h=[0.0] * 64)


def test_add_rmsnorm_edges(memq):
    w = torch.ones(64, device="cuda")
    h, z, qs, d = memq.memq_add_rmsnorm_q8_1(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"), w)
    assert qs.shape == (0, 64)
    x = torch.randn(64, device="cuda")
    h, _, qs, d = memq.memq_add_rmsnorm_q8_1(x, -x, w)  # a zero row, given as a vector
    assert torch.all(h == 0) and torch.all(qs == 0) and torch.all(d == 0)
    with pytest.raises(ValueError):
        memq.memq_add_rmsnorm_q8_1(x, torch.randn(32, device="cuda"), w)
    with pytest.raises(TypeError):
        memq.memq_add_rmsnorm_q8_1(x.double(), x, w)


# ------------------------------------------------------------------------------- the cache
def rows_of(rng, n, width):
    return (rng.normal(0, 1, (n, width)) * np.exp(rng.normal(0, 0.5, (n, 1)))).astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rank,rope", [(128, 0), (256, 32), (512, 64), (512, 128), (128, 128), (512, 0)])
@pytest.mark.parametrize("n", [1, 37])
def test_cache_write_and_read(memq, n, rank, rope, dtype):
    rng = np.random.default_rng(n + rank + rope)
    x = rows_of(rng, n, rank + rope)
    if n > 9:
        x[3] = 0                       # a zero row
        x[4] *= np.float32(1e-30)
        x[5] *= np.float32(1e30)
        x[6, rank // 2] = np.inf       # rows that are not finite
        x[7, -1] = np.nan
        x[8] = np.float32(1e-45)       # the scale underflows to zero
    if dtype is torch.bfloat16:
        x = ref.bf16(x)
    pages, page = 7, 16
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    cache = torch.full((pages, page, rank + rope), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, page), -3.0, device="cuda")
    xd = to_dev(x).to(dtype)
    if n > 2:
        slots[1] = -1                  # padding
    memq.memq_mla_cache_append(xd[:, :rank].contiguous(), xd[:, rank:].contiguous() if rope else None, to_dev(slots),
                               cache, scales)
    codes, want = ref.quantise(x)
    c, s = cache.cpu().numpy().reshape(-1, rank + rope), scales.cpu().numpy().reshape(-1)
    kept = slots >= 0
    assert np.array_equal(ref.E4M3[c[slots[kept]]], ref.E4M3[codes[kept]])
    assert np.array_equal(s[slots[kept]], want[kept], equal_nan=True)
    others = np.setdiff1d(np.arange(pages * page), slots[kept])
    assert np.all(c[others] == 0x55) and np.all(s[others] == -3)
    for out_type in (torch.float32, torch.bfloat16):
        got = memq.memq_mla_cache_read(cache, scales, to_dev(slots), dtype=out_type)
        val = (ref.E4M3[codes] * want[:, None].astype(np.float64)).astype(np.float32)
        val[~kept] = 0
        expect = torch.from_numpy(val).to(out_type).float().numpy()
        assert np.array_equal(got.float().cpu().numpy(), expect, equal_nan=True)
    assert memq.memq_device_fault() == 0


def test_cache_slots_out_of_range_and_repeated(memq):
    cache = torch.zeros(2, 16, 128, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, 16, device="cuda")
    x = torch.randn(3, 128, device="cuda")
    slots = torch.tensor([5, 32, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    memq.memq_mla_cache_append(x, None, slots, cache, scales)
    assert memq.memq_device_fault() == 32
    assert scales.count_nonzero() == 1 and scales[0, 5] > 0
    got = memq.memq_mla_cache_read(cache, scales, slots, dtype=torch.float32)
    assert memq.memq_device_fault() == 32
    assert torch.all(got[1:] == 0) and got[0].abs().max() > 0
    again = memq.memq_mla_cache_read(cache, scales, torch.full((6,), 5, dtype=torch.int32, device="cuda"),
                                     dtype=torch.float32)
    assert torch.equal(again, got[:1].expand(6, 128))
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    memq.memq_mla_cache_append(x[:0], None, empty, cache, scales)
    assert memq.memq_mla_cache_read(cache, scales, empty).shape == (0, 128)
    assert memq.memq_device_fault() == 0


# ------------------------------------------------------------------------------- the attention
class Batch:
    """A paged cache with `lens` = [(new tokens, cached rows)] in it; everything that no sequence owns
    is NaN codes and NaN scales, table entries that are not needed are -1."""

    def __init__(self, lens, nh, rank, rope, page, dtype=torch.bfloat16, seed=0, row_scale=0.5, q_scale=1.0,
                 lead=0, tail=0, spare=0):
        rng = np.random.default_rng(seed)
        self.lens, self.rank, self.width, self.nh = lens, rank, rank + rope, nh
        need = [-(-kv // page) for _, kv in lens]
        pages = sum(need) + 2
        ids = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(need + [1]) + spare), -1, np.int32)
        self.codes = np.full((pages, page, self.width), 0x7F, np.uint8)
        self.scales = np.full((pages, page), np.nan, np.float32)
        at = 0
        for b, (t, kv) in enumerate(lens):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            x = (rng.normal(0, 1, (kv, self.width)) * np.exp(row_scale * rng.normal(0, 1, (kv, 1)))).astype(np.float32)
            c, s = ref.quantise(x)
            slot = (self.table[b, :need[b], None] * page + np.arange(page)).reshape(-1)[:kv]
            self.codes.reshape(-1, self.width)[slot] = c
            self.scales.reshape(-1)[slot] = s
        self.kv_len = np.array([kv for _, kv in lens], np.int32)
        self.cu = (lead + np.r_[0, np.cumsum([t for t, _ in lens])]).astype(np.int32)
        q = (rng.normal(0, 1, (self.cu[-1] + tail, nh, self.width)) * q_scale).astype(np.float32)
        self.q = ref.bf16(q) if dtype is torch.bfloat16 else q
        self.dtype, self.scale = dtype, 1.5 / np.sqrt(self.width)

    def device(self):
        q = to_dev(self.q).to(self.dtype)
        self.d = (q[..., :self.rank].contiguous(), q[..., self.rank:].contiguous() if self.width > self.rank else None,
                  to_dev(self.codes), to_dev(self.scales), to_dev(self.table), to_dev(self.kv_len), to_dev(self.cu))
        return self.d

    def run(self, memq, out_type=torch.bfloat16, fill=None, **kw):
        args = self.device()
        out = torch.full(self.q.shape[:2] + (self.rank,), float("nan") if fill is None else fill, dtype=out_type,
                         device="cuda")
        got = memq.memq_mla_attn_paged(*args, self.scale, out=out, **kw)
        torch.cuda.synchronize()
        return got

    def reference(self, out_type=torch.bfloat16):
        return ref.attend_batch(self.q.astype(np.float64), self.table, self.kv_len, self.cu, self.codes, self.scales,
                                self.rank, self.scale, EPS_OUT[out_type])

    def check(self, memq, out_type=torch.bfloat16):
        got = self.run(memq, out_type).double().cpu().numpy()
        want, bound = self.reference(out_type)
        own = ~np.isnan(want)
        err = np.abs(got - want)
        assert np.all(np.isfinite(got[own]))
        assert np.all(err[own] <= bound[own]), f"worst {np.max(err[own] / np.maximum(bound[own], 1e-30)):.3f} of the bound"
        assert memq.memq_device_fault() == 0
        return float(np.max(err[own] / np.maximum(bound[own], 1e-30), initial=0))


LENS = {
    "one": [(1, 1)],
    "edges": [(1, 127), (1, 128), (1, 129), (1, 15), (1, 16), (1, 17)],
    "from_empty": [(5, 5), (130, 130)],
    "holes": [(0, 7), (3, 0), (2, 1), (17, 300), (0, 0), (1, 64)],
    "long": [(1, 4097), (2, 3000)],
    "chunk": [(61, 517), (9, 1000)],
}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("nh,rank,rope,page", [(64, 512, 64, 64), (1, 128, 0, 16), (24, 256, 32, 32)])
def test_attention_lengths(memq, lens, nh, rank, rope, page):
    Batch(LENS[lens], nh, rank, rope, page, seed=nh).check(memq)


@pytest.mark.parametrize("nh", [1, 2, 3, 16, 40, 63, 64, 65, 96, 128, 200])
def test_attention_heads(memq, nh):
    Batch([(1, 300), (7, 150)], nh, 256, 64, 64, seed=nh).check(memq)


@pytest.mark.parametrize("rank", [128, 256, 512])
@pytest.mark.parametrize("rope", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype,out_type", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                            (torch.float32, torch.bfloat16)])
def test_attention_widths_and_types(memq, rank, rope, dtype, out_type):
    Batch([(3, 400), (1, 77)], 20, rank, rope, 16, dtype, seed=rank + rope).check(memq, out_type)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_attention_pages(memq, page):
    Batch([(2, 1500), (1, 3), (4, 1024)], 16, 128, 32, page, seed=page, spare=3).check(memq)


def test_attention_many_sequences(memq):
    rng = np.random.default_rng(5)
    lens = [(int(t), int(t + k)) for t, k in zip(rng.integers(0, 4, 700), rng.integers(0, 150, 700))]
    Batch(lens, 8, 128, 0, 16, seed=6).check(memq)


def test_attention_few_long_items_split_over_all_sms(memq):
    """One item over every CTA (parts beyond a warp), and items that share a CTA."""
    Batch([(1, 40000)], 16, 128, 32, 64, seed=7).check(memq)
    Batch([(1, 9000), (1, 8000), (1, 7000)], 32, 128, 0, 64, seed=8).check(memq, torch.float32)


def test_attention_scales_far_apart(memq):
    """Row scales over ten decades, zero rows among them: the scale is part of the weight's range."""
    b = Batch([(2, 700)], 8, 256, 64, 64, seed=9, row_scale=3.0, q_scale=0.3)
    b.codes[b.table[0, 2], 5] = 0
    b.scales[b.table[0, 2], 5] = 0
    b.check(memq)


@pytest.mark.parametrize("size", [2.0 ** -6, 2.0 ** -12, 2.0 ** -20, 2.0 ** -40])
@pytest.mark.parametrize("least", [0.0, 1e-42, 1e-37, 1e-30])
def test_attention_zero_and_tiny_rows_among_small_ones(memq, size, least):
    """Rows whose scale is zero or nearly weigh as any other, whatever the others' scale is."""
    b = Batch([(1, 8), (2, 200)], 5, 128, 32, 16, seed=25, row_scale=0.0, q_scale=0.5 / size)
    b.scales *= np.float32(size)
    for slot in (0, 3, 7):
        for page in (b.table[0, 0], b.table[1, 0], b.table[1, 9]):
            b.scales[page, slot] = least
            if least == 0:
                b.codes[page, slot] = 0
    got = b.run(memq, torch.float32).double().cpu().numpy()
    want, bound = b.reference(torch.float32)
    # a scale below 2^-64 counts as 2^-64: up to 448 * 2^-64 off in the output
    assert np.all(np.abs(got - want) <= bound + 448 * 2.0 ** -64)
    assert memq.memq_device_fault() == 0


def test_attention_over_zero_rows_only(memq):
    b = Batch([(1, 8), (3, 300)], 3, 128, 0, 16, seed=26)
    b.scales[:] = 0
    b.codes[:] = 0
    for out_type in (torch.float32, torch.bfloat16):
        assert torch.all(b.run(memq, out_type) == 0)


def test_attention_sink_and_long_tail(memq):
    """One key far above thousands that carry half of the sum: small weights must not be flushed."""
    b = Batch([(1, 12000)], 4, 128, 0, 64, seed=10, row_scale=0.0)
    c, s = b.codes.reshape(-1, 128), b.scales.reshape(-1)
    first = b.table[0, 0] * 64
    q = b.q[0].astype(np.float64)
    key = q.sum(0) / np.linalg.norm(q.sum(0))                    # scores high for every head
    row = (key * 8).astype(np.float32)
    c[first], s[first] = (v[0] for v in ref.quantise(row[None]))
    top = b.scale * (q @ (ref.E4M3[c[first]] * s[first]))
    b.q *= np.float32(9.0 / top.min())                           # e^9 = 8103 against 11999 keys
    b.q = ref.bf16(b.q)
    tail = np.setdiff1d((b.table[0][:, None] * 64 + np.arange(64)).reshape(-1)[:12000], [first])
    s[tail] *= np.float32(0.02)                                  # the others' scores are near zero
    b.check(memq)


def test_attention_large_scores(memq):
    """Scores of hundreds: the reference moves often, weights underflow."""
    Batch([(3, 900)], 16, 256, 32, 32, seed=11, q_scale=60.0).check(memq)


def test_rows_outside_the_sequences_are_left_alone(memq):
    b = Batch([(2, 40), (3, 7)], 5, 128, 32, 16, seed=12, lead=3, tail=4)
    got = b.run(memq, fill=7.0).float().cpu().numpy()
    assert np.all(got[:3] == 7) and np.all(got[b.cu[-1]:] == 7)
    want, bound = b.reference()
    sl = slice(3, b.cu[-1])
    assert np.all(np.abs(got[sl] - want[sl]) <= bound[sl])


def test_not_finite_rows_reach_only_who_sees_them(memq):
    """A NaN row of the chunk itself: tokens before it are unaffected, tokens from it on are NaN.  A
    query row with an infinity is NaN alone."""
    b = Batch([(6, 200), (2, 90)], 8, 128, 32, 16, seed=13)
    clean = b.run(memq).float().cpu().numpy()
    pos = 200 - 6 + 3
    b.scales[b.table[0, pos // 16], pos % 16] = np.nan
    b.codes[b.table[0, pos // 16], pos % 16] = 0
    got = b.run(memq).float().cpu().numpy()
    want, bound = b.reference()
    seen = np.r_[0:3, 6:8]
    assert np.all(np.abs(got[seen] - want[seen]) <= bound[seen])
    assert np.array_equal(got[6:], clean[6:]) and np.all(np.isnan(got[3:6]))
    b = Batch([(6, 200), (2, 90)], 8, 128, 32, 16, seed=13)
    for bad in (np.inf, np.nan, np.float32(3e38)):
        b.q[1, 4, 17] = bad
        got = b.run(memq).float().cpu().numpy()
        assert np.all(np.isnan(got[1, 4]))
        got[1, 4] = clean[1, 4]
        assert np.array_equal(got, clean)
    assert memq.memq_device_fault() == 0


def test_empty_calls(memq):
    b = Batch([(2, 40)], 4, 128, 0, 16, seed=14)
    q, _, cache, scales, table, kv, cu = b.device()
    assert memq.memq_mla_attn_paged(q[:0], None, cache, scales, table, kv, torch.zeros_like(cu), 1.0).shape == (0, 4, 128)
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    out = torch.full((2, 4, 128), 5.0, device="cuda")
    memq.memq_mla_attn_paged(q, None, cache, scales, table[:0], z, torch.zeros(1, dtype=torch.int32, device="cuda"), 1.0,
                             out=out)
    assert torch.all(out == 5)


def test_same_call_same_bits_and_reused_workspace(memq):
    b = Batch([(1, 5000), (9, 700)], 64, 256, 64, 64, seed=15)
    ws = torch.full((memq.memq_mla_attn_paged_workspace(256),), 0xFF, dtype=torch.uint8, device="cuda")
    first = b.run(memq, torch.float32, workspace=ws)
    small = Batch([(1, 20)], 4, 256, 64, 64, seed=16)
    small.run(memq, workspace=ws)
    assert torch.equal(b.run(memq, torch.float32, workspace=ws), first)


def test_captured_call_serves_other_lengths(memq):
    b = Batch([(3, 1000), (3, 200)], 16, 256, 32, 32, seed=17)
    args = b.device()
    out = torch.empty(b.q.shape[:2] + (256,), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(memq.memq_mla_attn_paged_workspace(256), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        memq.memq_mla_attn_paged(*args, b.scale, out=out, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            memq.memq_mla_attn_paged(*args, b.scale, out=out, workspace=ws)
    st.synchronize()
    for kv, cu in (([1000, 200], [0, 3, 6]), ([37, 129], [0, 1, 6]), ([0, 3], [0, 2, 4]), ([513, 200], [0, 6, 6])):
        b.kv_len, b.cu = np.array(kv, np.int32), np.array(cu, np.int32)
        args[5].copy_(to_dev(b.kv_len))
        args[6].copy_(to_dev(b.cu))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        want, bound = b.reference()
        own = ~np.isnan(want)
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - want)[own] <= bound[own]) and np.all(np.isnan(got[~own]))


def test_two_streams_at_once(memq):
    bs = [Batch([(4, 3000)], 64, 512, 64, 64, seed=18), Batch([(1, 9000), (2, 100)], 32, 512, 0, 64, seed=19)]
    alone = [b.run(memq, torch.float32) for b in bs]
    sts = [torch.cuda.Stream() for _ in bs]
    outs = [[], []]
    for b in bs:
        b.device()
    torch.cuda.synchronize()
    for _ in range(5):
        for i, b in enumerate(bs):
            o = torch.empty_like(alone[i])
            outs[i].append(memq.memq_mla_attn_paged(*b.d, b.scale, out=o, stream=sts[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


def test_workspace_is_memory_of_the_stream_that_uses_it(memq, monkeypatch):
    """Also when the default stream is named inside another stream's context: memory of that other
    stream would be handed out again while the call still runs."""
    b = Batch([(1, 40)], 4, 128, 0, 16, seed=27)
    args = b.device()
    out = torch.empty(b.q.shape[:2] + (128,), device="cuda")
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    seen, empty = [], torch.empty

    def recording(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)
    monkeypatch.setattr(torch, "empty", recording)
    for use in (torch.cuda.default_stream(), 0, other, other.cuda_stream, None):
        with torch.cuda.stream(side):
            memq.memq_mla_attn_paged(*args, b.scale, out=out, stream=use)
        torch.cuda.synchronize()
    assert seen == [0, 0, other.cuda_stream, other.cuda_stream, side.cuda_stream]


def test_input_faults_are_reported_and_contained(memq):
    """Lengths past the table, page indexes outside the pool, offsets that descend: the fault bit is
    set, nothing outside the arrays is touched, and other sequences are right."""
    def run(change, good):
        b = Batch([(2, 100), (3, 60)], 8, 128, 32, 16, seed=20)
        want, bound = b.reference()
        change(b)
        got = b.run(memq).double().cpu().numpy()
        assert memq.memq_device_fault() == 32
        assert np.all(np.abs(got - want)[good] <= bound[good])
    run(lambda b: b.kv_len.__setitem__(0, 10 ** 6), slice(2, 5))
    run(lambda b: b.kv_len.__setitem__(1, -5), slice(0, 2))
    run(lambda b: b.table.__setitem__((0, 3), b.codes.shape[0]), slice(2, 5))
    run(lambda b: b.table.__setitem__((1, 1), -1), slice(0, 2))
    run(lambda b: b.cu.__setitem__(slice(None), [0, 2, 99]), slice(0, 2))
    run(lambda b: b.cu.__setitem__(slice(None), [3, 2, 1]), slice(0, 0))
    assert memq.memq_device_fault() == 0


def test_rows_past_four_gigabytes(memq):
    """A pool of 8 M rows of 640 bytes: slots, codes and boxes beyond 2^32 bytes."""
    rank, rope, page, pages = 512, 128, 128, 64 * 1024
    cache = torch.empty(pages, page, rank + rope, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, page, device="cuda")
    b = Batch([(2, 300)], 4, rank, rope, page, seed=21)
    n = b.table.shape[1]
    far = np.array([pages - 1, pages - 7, pages // 2 + 3][:n], np.int32)
    rows = np.concatenate([ref.E4M3[b.codes[p]] * b.scales[p][:, None].astype(np.float64) for p in b.table[0]])[:300]
    x = rows.astype(np.float32)
    slots = (far[:, None] * page + np.arange(page)).reshape(-1)[:300].astype(np.int32)
    assert slots.astype(np.int64).max() * (rank + rope) > 1 << 32
    xd = to_dev(x)
    memq.memq_mla_cache_append(xd[:, :rank].contiguous(), xd[:, rank:].contiguous(), to_dev(slots), cache, scales)
    back = memq.memq_mla_cache_read(cache, scales, to_dev(slots), dtype=torch.float32).cpu().numpy()
    codes, sc = ref.quantise(x)
    assert np.array_equal(back, (ref.E4M3[codes] * sc[:, None].astype(np.float64)).astype(np.float32))
    q, pe, *_ = b.device()
    got = memq.memq_mla_attn_paged(q, pe, cache, scales, to_dev(far[None]), to_dev(b.kv_len), to_dev(b.cu), b.scale)
    want, bound = ref.attend(b.q.astype(np.float64), codes, sc, 2, rank, b.scale, 2.0 ** -8)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)
    assert memq.memq_device_fault() == 0


def test_refusals_of_the_binding(memq):
    b = Batch([(2, 40)], 4, 128, 32, 16, seed=22)
    q, pe, cache, scales, table, kv, cu = b.device()
    run = memq.memq_mla_attn_paged
    for args in ((q[0], pe, cache, scales, table, kv, cu), (q, None, cache, scales, table, kv, cu),
                 (q, pe[:1], cache, scales, table, kv, cu), (q, pe, cache[0], scales, table, kv, cu),
                 (q, pe, cache, scales[:1], table, kv, cu), (q, pe, cache, scales, table[0], kv, cu),
                 (q, pe, cache, scales, table, kv, cu[:1]),
                 (q.transpose(0, 1), pe, cache, scales, table, kv, cu)):
        with pytest.raises(ValueError):
            run(*args, 1.0)
    for args in ((q.half(), pe, cache, scales, table, kv, cu), (q, pe.float(), cache, scales, table, kv, cu),
                 (q, pe, cache, scales, table.long(), kv, cu)):
        with pytest.raises(TypeError):
            run(*args, 1.0)
    with pytest.raises(memq.MemqError):  # a workspace too small
        run(q, pe, cache, scales, table, kv, cu, 1.0, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(memq.MemqError):
        run(q, pe, cache, scales, table, kv, cu, float("inf"))
    with pytest.raises(ValueError):
        memq.memq_mla_cache_append(q[:, 0].contiguous(), None, kv, cache, scales)
    with pytest.raises(ValueError):
        memq.memq_mla_cache_read(cache[..., :144].contiguous(), scales, kv)
    assert memq.memq_device_fault() == 0


def test_a_layer_step(memq):
    """The operators as a decode step uses them: residual and norm, the new tokens' latent rows into the
    cache, absorbed queries, attention over the pages, decompression; against the same in f64."""
    rng = np.random.default_rng(23)
    nh, d_nope, rank, rope, page, t, kv = 16, 128, 512, 64, 32, 4, 150
    b = Batch([(t, kv)], nh, rank, rope, page, torch.float32, seed=24)
    q_nope = rng.normal(0, 1, (t, nh, d_nope)).astype(np.float32)
    wk = (rng.normal(0, 1, (nh, rank, d_nope)) / np.sqrt(d_nope)).astype(np.float32)
    wv = (rng.normal(0, 1, (nh, 128, rank)) / np.sqrt(rank)).astype(np.float32)
    _, pe, cache, scales, table, kv_len, cu = b.device()
    x, res = rng.normal(0, 1, (2, t, 1024)).astype(np.float32)
    h, _, qs, d = memq.memq_add_rmsnorm_q8_1(to_dev(x), to_dev(res), torch.ones(1024, device="cuda"))
    assert torch.equal(h, to_dev(x) + to_dev(res)) and qs.abs().max() == 127

    new = rows_of(rng, t, rank + rope)
    pos = np.arange(kv - t, kv)
    slots = b.table[0, pos // page] * page + pos % page
    memq.memq_mla_cache_append(to_dev(new[:, :rank]), to_dev(new[:, rank:]), to_dev(slots.astype(np.int32)), cache, scales)
    c, s = ref.quantise(new)
    b.codes.reshape(-1, rank + rope)[slots], b.scales.reshape(-1)[slots] = c, s
    q_lat = memq.memq_mla_absorb_q(to_dev(q_nope), to_dev(wk))
    o_lat = memq.memq_mla_attn_paged(q_lat, pe, cache, scales, table, kv_len, cu, b.scale,
                                     out=torch.empty(t, nh, rank, device="cuda"))
    out = memq.memq_mla_decompress_v(o_lat, to_dev(wv)).double().cpu().numpy()

    b.q = np.concatenate([q_lat.cpu().numpy(), b.q[..., rank:]], 2)
    q_ref = np.einsum("thd,hrd->thr", q_nope.astype(np.float64), wk.astype(np.float64))
    assert np.abs(b.q[..., :rank] - q_ref).max() <= 2e-5 * np.einsum("thd,hrd->thr", np.abs(q_nope), np.abs(wk)).max()
    want, bound = b.reference(torch.float32)
    assert np.all(np.abs(o_lat.double().cpu().numpy() - want) <= bound)
    w64 = wv.astype(np.float64)
    final = np.einsum("thr,hvr->thv", want, w64)
    slack = np.einsum("thr,hvr->thv", bound + 2e-5 * np.abs(want), np.abs(w64))
    assert np.all(np.abs(out - final) <= slack)

    # the cache read back in f32 is what the gathered attention reads
    rows = memq.memq_mla_cache_read(cache, scales, torch.arange(cache.shape[0] * page, dtype=torch.int32, device="cuda"),
                                    dtype=torch.float32)
    idx = (b.table[0, np.arange(kv) // page] * page + np.arange(kv) % page)[: kv - t + 1].astype(np.int32)
    first = memq.memq_mla_attn_gathered(q_lat[:1].contiguous(), pe[:1].contiguous(), rows, to_dev(idx[None]), b.scale)
    assert np.all(np.abs(first.double().cpu().numpy() - want[:1]) <= bound[:1])
    assert memq.memq_device_fault() == 0


@pytest.mark.parametrize("ncols", [4128, 6176, 8192, 8224, 12288, 14368, 16384, 24576, 32768])
def test_add_rmsnorm_clusters_started_at_once(memq, ncols):
    """Rows shared by clusters of five to eight CTAs, launch behind launch on two streams, so that CTAs of
    a cluster start while others still run: every launch gives the same bits."""
    rows = 18 if ncols <= 8192 else 333
    g = torch.Generator("cuda").manual_seed(ncols)
    x, res = torch.randn(2, rows, ncols, device="cuda", generator=g)
    w = torch.randn(ncols, device="cuda", generator=g)
    z, qs, d = memq.memq_rmsnorm_q8_1(x + res, w)
    sts = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(12):
        for st in sts:
            with torch.cuda.stream(st):
                outs.append(memq.memq_add_rmsnorm_q8_1(x, res, w))
    torch.cuda.synchronize()
    for h2, z2, qs2, d2 in outs:
        assert torch.equal(h2, x + res) and torch.equal(z2, z) and torch.equal(qs2, qs) and torch.equal(d2, d)


@pytest.mark.parametrize("cu", [[0, 5, 0, 5, 0], [3, 2, 5, 5, 5], [0, 5, 5, 5, 4], [5, 5, 5, 5, -1]])
def test_offsets_that_descend_write_nothing(memq, cu):
    """They would name the same tokens over and over: the call reports them and leaves the outputs alone."""
    b = Batch([(2, 100), (3, 60), (0, 40), (0, 9)], 8, 128, 32, 16, seed=28)
    assert b.q.shape[0] == 5
    b.cu = np.array(cu, np.int32)
    assert torch.all(b.run(memq, fill=7.0) == 7)
    assert memq.memq_device_fault() == 32
    b.cu = np.array([0, 2, 5, 5, 5], np.int32)
    b.check(memq)
