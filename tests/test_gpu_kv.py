"""GPU parity of the paged K/V cache (append, read), the attention over it and the page plan.

Writes and plans are compared bit for bit with their definitions; the attention with the f64 reference
within the bound that kv_reference.attend derives from the kernels' roundings."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from gpu_helpers import to_dev
from paged_reference import E4M3, bf16

pytestmark = pytest.mark.gpu

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}


@pytest.fixture(scope="module")
def memq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_decode_memq_gb300 import build
    build.build()
    import quantized_decode_memq_gb300 as m
    m.memq_device_fault()
    return m


# ------------------------------------------------------------------------------- the cache
class Pool:
    """Random codes and scales, as a pool that was in use."""

    def __init__(self, rng, pages, n_kv, page, d):
        self.page = page
        self.codes = [rng.integers(0, 256, (pages, n_kv, page, d)).astype(np.uint8) for _ in range(2)]
        self.scales = [np.exp2(rng.integers(-12, 4, (pages, n_kv, page // 16))).astype(np.float32) for _ in range(2)]

    def device(self):
        return [to_dev(x.copy()) for x in (*self.codes, *self.scales)]


def rows_of(rng, *shape):
    return (rng.normal(0, 1, shape) * np.exp(rng.normal(0, 1, shape[:-1] + (1,)))).astype(np.float32)


def run_append(memq, pool, k, v, slots, dtype=torch.float32):
    dev = pool.device()
    memq.memq_kv_cache_append(to_dev(k).to(dtype), to_dev(v).to(dtype), to_dev(np.asarray(slots, np.int32)), *dev)
    r = (lambda x: x) if dtype is torch.float32 else bf16
    with np.errstate(invalid="ignore"):
        ref.append(r(k), r(v), slots, pool.codes, pool.scales, pool.page)
    for got, want in zip(dev, (*pool.codes, *pool.scales)):
        assert np.array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))
    return dev


SLOTS = {
    "one": [37],
    "fresh block": list(range(32, 48)),
    "a prompt from the middle of a block": list(range(21, 70)),
    "a decode batch": [5, 17, 48, 64 + 31, 64 + 32, 128 + 3],
    "drafts": [8, 9, 10, 40, 41, 42, 43, 100],
    "padding": [-1, -1, 16, 17, -1, 90, -1],
    "a page behind a later one": list(range(112, 128)) + list(range(0, 16)),
    "twice the same": [50, 50, 51, 50, 52] + [60] * 37 + [61],
    "holes and downwards": [35, 33, 45, 34],
    "nothing": [],
}


@pytest.mark.parametrize("name", SLOTS)
@pytest.mark.parametrize("n_kv,d,page,dtype", [(1, 64, 16, torch.float32), (3, 128, 64, torch.float32),
                                              (2, 64, 128, torch.bfloat16), (8, 128, 32, torch.bfloat16)])
def test_append(memq, name, n_kv, d, page, dtype):
    rng = np.random.default_rng(len(name) + d)
    slots = SLOTS[name]
    pool = Pool(rng, 256 // page, n_kv, page, d)
    k, v = rows_of(rng, 2, len(slots), n_kv, d)
    dev = run_append(memq, pool, k, v, slots, dtype)
    back = np.array([0, 37, -1, 37, 255] + [s for s in slots if s >= 0], np.int32)
    for i in range(2):
        want = ref.values(pool.codes[i], pool.scales[i], back)
        for t in (torch.float32, torch.bfloat16):
            got = memq.memq_kv_cache_read(dev[i], dev[2 + i], to_dev(back), dtype=t).float().cpu().numpy()
            w = want.astype(np.float32)
            assert np.array_equal(got, w if t is torch.float32 else np.where(np.isnan(w), w, bf16(w)), equal_nan=True)
    assert memq.memq_device_fault() == 0


def test_append_long_prompts(memq):
    """More rows than a warp serves one at a time: windows of 16, blocks that begin anywhere in them."""
    rng = np.random.default_rng(3)
    pool = Pool(rng, 300, 8, 16, 64)
    order = rng.permutation(300)
    slots = np.concatenate([order[:200, None] * 16 + np.arange(16)])[:].reshape(-1)[5:2500]
    slots = np.r_[slots, -np.ones(70, int), order[210] * 16 + 3, order[211:290] * 16 + rng.integers(0, 16, 79)]
    k, v = rows_of(rng, 2, len(slots), 8, 64)
    run_append(memq, pool, k, v, slots, torch.bfloat16)


def test_append_scales(memq):
    """Scales at the borders of a binade, zero rows, rows that grow, shrink or are not finite."""
    rng = np.random.default_rng(4)
    pool = Pool(rng, 8, 2, 16, 64)
    pool.scales[0][3], pool.scales[0][4], pool.scales[0][5] = 0.0, np.nan, np.inf
    pool.scales[1][3], pool.scales[1][4] = 0.3, -1.0
    k, v = rows_of(rng, 2, 40, 2, 64)
    slots = np.r_[0:16, 17:21, 33:35, 50:52, 66:70, 80 + 1, 96:104, 112:114, 127]
    assert len(slots) == 40
    k[0, 0, 0], k[1, 0] = 448.0, 0
    k[0:16, 0] = np.clip(k[0:16, 0], -448, 448)
    k[0:16, 1], v[0:16, 0] = 0, np.float32(1e-44)
    v[3, 1, 7] = np.float32(448.00003)
    v[16:20] *= 1e5
    k[16:20] *= 1e-6
    v[20] = np.float32(3e38)
    k[24, 0, 5], v[25, 1, 6], k[26, 0, 0] = np.inf, np.nan, -np.inf
    k[30:38, 1] = np.nan
    run_append(memq, pool, k, v, slots)
    assert memq.memq_device_fault() == 0


def test_append_takes_parts_of_a_projection(memq):
    rng = np.random.default_rng(5)
    for dtype in (torch.float32, torch.bfloat16):
        pool = Pool(rng, 4, 2, 64, 128)
        qkv = torch.randn(33, 9, 128, device="cuda").to(dtype)
        k, v = qkv[:, 4:6], qkv[:, 7:9]
        slots = np.r_[70:103]
        dev = pool.device()
        memq.memq_kv_cache_append(k, v, to_dev(slots.astype(np.int32)), *dev)
        ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(), slots, pool.codes, pool.scales, 64)
        for got, want in zip(dev, (*pool.codes, *pool.scales)):
            assert np.array_equal(got.cpu().numpy(), want)
        one = qkv[:1, :2].expand(16, 2, 128)  # one row for all
        memq.memq_kv_cache_append(one, one, torch.arange(16, dtype=torch.int32, device="cuda"), *dev)
        got = memq.memq_kv_cache_read(dev[0], dev[2], torch.arange(16, dtype=torch.int32, device="cuda"))
        assert torch.equal(got, got[:1].expand_as(got)) and got.abs().max() > 0


def test_cache_slots_out_of_range(memq):
    rng = np.random.default_rng(6)
    pool = Pool(rng, 4, 2, 16, 64)
    k, v = rows_of(rng, 2, 4, 2, 64)
    dev = run_append(memq, pool, k, v, [64, 5, 2 ** 31 - 1, -7])
    assert memq.memq_device_fault() == 32
    got = memq.memq_kv_cache_read(dev[0], dev[2], to_dev(np.array([64, 5, 2 ** 31 - 1, -7], np.int32)), dtype=torch.float32)
    assert memq.memq_device_fault() == 32
    assert torch.all(got[[0, 2, 3]] == 0) and torch.any(got[1] != 0)


# ------------------------------------------------------------------------------- attention
class Batch:
    """Sequences (t, kv) over random pages; the pool's other rows hold anything."""

    def __init__(self, lens, nh, n_kv, d, page, dtype=torch.bfloat16, seed=0, spread=0.5, extra=3):
        rng = np.random.default_rng(seed)
        self.lens, self.dtype, self.scale, self.page = lens, dtype, d ** -0.5, page
        need = [-(-kv // page) for _, kv in lens]
        pages = max(1, sum(need)) + extra
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(1, *need)), -1, np.int32)
        self.codes = [rng.integers(0, 256, (pages, n_kv, page, d)).astype(np.uint8) for _ in range(2)]
        self.scales = [np.full((pages, n_kv, page // 16), np.nan, np.float32) for _ in range(2)]
        at = 0
        for b, (_, kv) in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            slots = self.slots(b, kv)
            for i in range(2):
                x = (rng.normal(0, 1, (kv, n_kv, d)) * np.exp(spread * rng.normal(0, 1, (kv, n_kv, 1)))).astype(np.float32)
                for j in range(0, kv, 16):
                    rows = x[j:j + 16]
                    s = np.array([ref.scale_of(float(np.abs(rows[:, h]).max())) for h in range(n_kv)])
                    p, o = slots[j] // page, slots[j] % page
                    self.scales[i][p, :, o // 16] = s
                    self.codes[i][p, :, o:o + len(rows)] = ref.to_e4m3(rows / s[:, None]).transpose(1, 0, 2)
        self.kv_len = np.array([kv for _, kv in lens], np.int32)
        self.cu = np.r_[0, np.cumsum([t for t, _ in lens])].astype(np.int32)
        self.q = rng.normal(0, 1, (int(self.cu[-1]), nh, d)).astype(np.float32)
        if dtype is torch.bfloat16:
            self.q = bf16(self.q)

    def slots(self, b, n):
        j = np.arange(n)
        return self.table[b, j // self.page].astype(np.int64) * self.page + j % self.page

    def device(self):
        return [to_dev(self.q).to(self.dtype), *(to_dev(x) for x in (*self.codes, *self.scales, self.table, self.kv_len,
                                                                    self.cu))]

    def run(self, memq, out_type=None, fill=None, **kw):
        out = None
        if out_type is not None or fill is not None:
            out = torch.full(self.q.shape, fill or 0.0, dtype=out_type or self.dtype, device="cuda")
        return memq.memq_attn_paged(*self.device(), self.scale, out=out, **kw)

    def reference(self, out_type=None):
        out_type = out_type or self.dtype
        want, bound = np.full((2,) + self.q.shape, np.nan)
        for b, (t, kv) in enumerate(self.lens):
            s = self.slots(b, kv)
            k, v = (ref.values(self.codes[i], self.scales[i], s) for i in range(2))
            vs = self.scales[1][s // self.page, :, s % self.page // 16].astype(np.float64)
            at = slice(self.cu[b], self.cu[b] + t)
            want[at], bound[at] = ref.attend(self.q[at].astype(np.float64), k, v, t, self.scale,
                                             2 if out_type is torch.float32 else 1, EPS[out_type], vs)
        return want, bound

    def check(self, memq, out_type=None, **kw):
        got = self.run(memq, out_type, **kw)
        assert got.dtype is (out_type or self.dtype)
        got = got.double().cpu().numpy()
        want, bound = self.reference(out_type)
        assert np.all(np.isfinite(got))
        worst = np.abs(got - want) / np.maximum(bound, 1e-300)  # the bound is 0 where the output is exactly 0
        assert worst.max() <= 1, (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
        assert memq.memq_device_fault() == 0


@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 15)], [(1, 16), (1, 17)], [(1, 33)], [(2, 2)], [(3, 64)], [(1, 1000)],
                                  [(7, 7), (1, 130), (20, 150)], [(130, 130)], [(257, 600)], [(1, 4097), (5, 31)],
                                  [(0, 40), (3, 0), (4, 2), (1, 90), (0, 0)]], ids=str)
def test_attention_lengths(memq, lens):
    Batch(lens, 8, 2, 128, 16, seed=1).check(memq)


@pytest.mark.parametrize("nh,n_kv", [(1, 1), (2, 1), (5, 5), (14, 2), (17, 1), (40, 8), (64, 8), (128, 1), (96, 32)])
def test_attention_heads(memq, nh, n_kv):
    Batch([(1, 100), (3, 45)], nh, n_kv, 64, 32, seed=nh).check(memq)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[(1, 700), (2, 90)], [(40, 300), (1, 70)]], ids=str)
def test_attention_types(memq, d, dtype, out_type, lens):
    Batch(lens, 8, 2, d, 64, dtype, seed=d).check(memq, out_type)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_attention_pages(memq, page):
    Batch([(1, 1500), (30, 200), (1, page)], 8, 2, 128, page, seed=page).check(memq)


def test_attention_many_sequences(memq):
    rng = np.random.default_rng(5)
    Batch([(int(rng.integers(0, 4)), int(rng.integers(1, 90))) for _ in range(700)], 4, 2, 64, 16, seed=6).check(memq)


def test_attention_one_long_sequence_over_all_sms(memq):
    Batch([(1, 40000)], 4, 1, 128, 64, seed=7).check(memq)


@pytest.mark.parametrize("t", [1, 40])
def test_attention_scales_far_apart(memq, t):
    """Blocks whose values are 2^-30 to 2^20 of others', and blocks of zeros."""
    b = Batch([(t, 500)], 8, 2, 64, 16, torch.float32, seed=8)
    rng = np.random.default_rng(9)
    used = ~np.isnan(b.scales[1])
    b.scales[1][used] *= np.exp2(rng.integers(-30, 20, used.sum())).astype(np.float32)
    b.check(memq)
    zero = b.table[0, 3:9]
    b.codes[1][zero], b.scales[1][zero] = 0, np.float32(2.0 ** -100)
    b.check(memq)
    b.scales[1][zero] = 0  # a scale of zero: the keys count, the values are nothing
    b.check(memq)


def test_attention_scales_that_are_no_powers_of_two(memq):
    b = Batch([(2, 200)], 8, 2, 64, 16, torch.float32, seed=10)
    rng = np.random.default_rng(11)
    for s in b.scales:
        s *= rng.uniform(0.5, 2, s.shape).astype(np.float32)
    b.check(memq)


@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t", [1, 70])
@pytest.mark.parametrize("nats", [8, 13, 18])
def test_attention_sink_and_long_tail(memq, out_type, t, nats):
    """One key far above thousands of others that together carry a part of the sum."""
    kv = 6000
    b = Batch([(t, kv)], 2, 1, 64, 64, torch.float32, seed=12, spread=0.0)
    b.q[:] = 0
    b.q[..., 0] = 8 * nats / 448.0  # scale 1/8
    first = b.table[0, 0]
    for p in b.table[0]:
        b.codes[0][p, 0, :, 0] = 0
    b.codes[0][first, 0, 0, 0] = 126  # 448
    b.scales[0][b.table[0], 0] = 1.0
    b.check(memq, out_type)


def test_attention_large_scores(memq):
    b = Batch([(2, 300), (33, 200)], 8, 2, 64, 16, seed=13)
    b.scale = 12.0
    b.check(memq)


def test_rows_outside_the_sequences_are_left_alone(memq):
    b = Batch([(2, 50), (40, 70)], 8, 2, 64, 16, seed=14)
    want, bound = b.reference()
    b.q = np.concatenate([np.full((3, 8, 64), np.nan, np.float32), b.q, np.full((2, 8, 64), np.nan, np.float32)])
    b.cu = b.cu + 3
    got = b.run(memq, fill=7.0).double().cpu().numpy()
    assert np.all(got[:3] == 7) and np.all(got[45:] == 7)
    assert np.all(np.abs(got[3:45] - want) <= bound)
    assert memq.memq_device_fault() == 0


@pytest.mark.parametrize("t", [6, 40])
def test_not_finite_rows_reach_only_who_sees_them(memq, t):
    """A new token's row that is not finite: its queries and the later ones are NaN, for its kv head alone."""
    kv, page = 90, 32
    b = Batch([(t, kv)], 8, 2, 64, page, torch.float32, seed=15)
    want, bound = b.reference()
    rng = np.random.default_rng(16)
    k, v = rows_of(rng, 2, 2, 2, 64)
    bad = kv - t + 3
    v[1, 1, 5] = np.inf
    q, kc, vc, ks, vs, table, kv_len, cu = b.device()
    s = b.slots(0, kv)
    rows = [ref.values(b.codes[i], b.scales[i], s[bad:bad + 1]).astype(np.float32) for i in range(2)]
    rows[1][0, 1, 5] = np.nan
    memq.memq_kv_cache_append(to_dev(rows[0]), to_dev(rows[1]), to_dev(s[bad:bad + 1].astype(np.int32)), kc, vc, ks, vs)
    got = memq.memq_attn_paged(q, kc, vc, ks, vs, table, kv_len, cu, b.scale).double().cpu().numpy()
    assert np.all(np.abs(got - want)[:, :4] <= bound[:, :4])
    assert np.all(np.abs(got - want)[:3, 4:] <= bound[:3, 4:])
    assert np.all(np.isnan(got[3:, 4:]))
    # a query that is not finite
    q[1, 2, 3] = float("inf")
    got = memq.memq_attn_paged(q, kc, vc, ks, vs, table, kv_len, cu, b.scale).double().cpu().numpy()
    assert np.all(np.isnan(got[1, 2]))
    assert np.all(np.abs(got - want)[1, 3] <= bound[1, 3]) and np.all(np.abs(got - want)[1, :2] <= bound[1, :2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t", [7, 60])
def test_not_finite_queries_without_keys(memq, t, dtype):
    """Tokens that see no row give zeros, whatever their queries hold."""
    b = Batch([(t, t - 5), (t, 0)], 8, 2, 64, 16, dtype, seed=23)
    want, bound = b.reference()
    b.q[:5], b.q[1, ::2], b.q[t:] = np.nan, np.inf, -np.inf
    got = b.run(memq).double().cpu().numpy()
    assert np.all(got[:5] == 0) and np.all(got[t:] == 0)
    assert np.all(np.abs(got - want)[5:t] <= bound[5:t])
    assert memq.memq_device_fault() == 0


def test_queries_that_are_parts_of_a_projection(memq):
    for dtype in (torch.float32, torch.bfloat16):
        b = Batch([(3, 40), (50, 80)], 8, 2, 128, 16, dtype, seed=17)
        dev = b.device()
        wide = torch.randn(53, 11, 128, device="cuda").to(dtype)
        wide[:, 2:10] = dev[0]
        a = memq.memq_attn_paged(wide[:, 2:10], *dev[1:], b.scale)
        assert torch.equal(a, memq.memq_attn_paged(*dev, b.scale))


def test_empty_calls(memq):
    b = Batch([(1, 40)], 8, 2, 64, 16, seed=18)
    q, kc, vc, ks, vs, table, kv, cu = b.device()
    assert memq.memq_attn_paged(q[:0], kc, vc, ks, vs, table, kv, cu, 1.0).shape == (0, 8, 64)
    out = torch.full_like(q, 3.0)
    memq.memq_attn_paged(q, kc, vc, ks, vs, table[:0], kv[:0], cu[:1], 1.0, out=out)
    assert torch.all(out == 3)
    memq.memq_kv_cache_append(q[:0, :2], q[:0, :2], kv[:0], kc, vc, ks, vs)
    assert memq.memq_kv_cache_read(kc, ks, kv[:0]).shape == (0, 2, 64)
    assert memq.memq_device_fault() == 0


def test_same_call_same_bits_and_reused_workspace(memq):
    a, b = Batch([(1, 3000), (60, 500)], 16, 4, 128, 64, seed=19), Batch([(1, 77)], 2, 1, 128, 16, seed=20)
    ws = torch.full((memq.memq_attn_paged_workspace(128),), 255, dtype=torch.uint8, device="cuda")
    first = a.run(memq, workspace=ws)
    b.check(memq, workspace=ws)
    assert torch.equal(first, a.run(memq, workspace=ws)) and torch.equal(first, a.run(memq))


def test_captured_calls_serve_other_lengths(memq):
    """Two captured graphs with a workspace each, replayed with other lengths, side by side."""
    long, short = [(1, 900), (20, 300)], [(5, 30), (16, 61)]
    a, b = Batch(long, 8, 2, 128, 32, seed=21), Batch(short, 8, 2, 128, 32, seed=21, extra=30)
    graphs = []
    for _ in range(2):
        dev = a.device()
        out = torch.zeros(a.q.shape, dtype=a.dtype, device="cuda")
        ws = torch.empty(memq.memq_attn_paged_workspace(128), dtype=torch.uint8, device="cuda")
        memq.memq_attn_paged(*dev, a.scale, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            memq.memq_attn_paged(*dev, a.scale, out=out, workspace=ws)
        graphs.append((g, dev, out, ws))  # a graph's memory is its owner's to keep
    want, bound = a.reference()
    for g, _, out, _ in graphs:
        out.zero_()
        g.replay()
    for _, _, out, _ in graphs:
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)
    _, dev, out, _ = graphs[0]
    for i in range(2):  # the other batch's rows, in this one's pool
        dev[1 + i][: b.codes[i].shape[0]] = to_dev(b.codes[i])
        dev[3 + i][: b.scales[i].shape[0]] = to_dev(b.scales[i])
    dev[5][:, : b.table.shape[1]] = to_dev(b.table)
    dev[6].copy_(to_dev(b.kv_len))
    dev[7].copy_(to_dev(b.cu))
    dev[0].copy_(to_dev(b.q))
    sts = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for st, (g, *_) in zip(sts, graphs):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    assert np.all(np.abs(graphs[1][2].double().cpu().numpy() - want) <= bound)
    want, bound = b.reference()
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)


def test_two_streams_at_once(memq):
    b = Batch([(1, 5000), (40, 700)], 8, 2, 128, 64, seed=22)
    dev = b.device()
    want = memq.memq_attn_paged(*dev, b.scale)
    sts, outs = [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for _ in range(4):
        for i, st in enumerate(sts):
            if i == 0:
                outs.append(memq.memq_attn_paged(*dev, b.scale, stream=st))
            else:
                with torch.cuda.stream(st):
                    outs.append(memq.memq_attn_paged(*dev, b.scale))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("lens", [[(2, 100), (3, 60)], [(40, 100), (50, 60)]], ids=str)
def test_input_faults_are_reported_and_contained(memq, lens):
    t0, t1 = lens[0][0], lens[0][0] + lens[1][0]

    def run(change, good):
        b = Batch(lens, 8, 2, 64, 16, seed=23)
        want, bound = b.reference()
        change(b)
        got = b.run(memq).double().cpu().numpy()
        assert memq.memq_device_fault() == 32
        assert np.all(np.abs(got - want)[good] <= bound[good])
    run(lambda b: b.kv_len.__setitem__(0, 10 ** 6), slice(t0, t1))
    run(lambda b: b.kv_len.__setitem__(1, -5), slice(0, t0))
    run(lambda b: b.table.__setitem__((0, 3), b.codes[0].shape[0]), slice(t0, t1))
    run(lambda b: b.table.__setitem__((1, 1), -1), slice(0, t0))
    run(lambda b: b.cu.__setitem__(slice(None), [0, t0, 999]), slice(0, t0))
    for cu in ([3, 2, 1], [0, 5, 4], [5, 5, -1]):
        b = Batch(lens, 8, 2, 64, 16, seed=23)
        b.cu = np.array(cu, np.int32)
        assert torch.all(b.run(memq, fill=7.0) == 7) and memq.memq_device_fault() == 32
    assert memq.memq_device_fault() == 0


def test_rows_past_four_gigabytes(memq):
    n_kv, page, pages, d = 8, 128, 64 * 1024, 128
    caches = [torch.empty(pages, n_kv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(pages, n_kv, page // 16, device="cuda") for _ in range(2)]
    b = Batch([(2, 300), (40, 300)], 16, n_kv, d, page, torch.float32, seed=24)
    far = np.array([[pages - 1, pages - 7, pages // 2 + 3], [pages - 2, pages - 5, pages // 2 + 9]], np.int32)
    for i in range(2):
        s = b.slots(i, 300)
        k, v = (to_dev(ref.values(b.codes[j], b.scales[j], s).astype(np.float32)) for j in range(2))
        slots = (far[i][:, None].astype(np.int64) * page + np.arange(page)).reshape(-1)[:300]
        assert slots.max() * n_kv * d > 1 << 32
        memq.memq_kv_cache_append(k, v, to_dev(slots.astype(np.int32)), *caches, *scales)
        back = memq.memq_kv_cache_read(caches[0], scales[0], to_dev(slots.astype(np.int32)), dtype=torch.float32)
        assert torch.equal(back, k)
    got = memq.memq_attn_paged(b.device()[0], *caches, *scales, to_dev(far), to_dev(b.kv_len), to_dev(b.cu), b.scale)
    want, bound = b.reference()
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)
    assert memq.memq_device_fault() == 0


def test_refusals_of_the_binding(memq):
    b = Batch([(2, 40)], 4, 2, 64, 16, seed=25)
    q, kc, vc, ks, vs, table, kv, cu = b.device()
    run = memq.memq_attn_paged
    for args in ((q[0], kc, vc, ks, vs, table, kv, cu), (q, kc[0], vc, ks, vs, table, kv, cu),
                 (q, kc, vc[:1], ks, vs, table, kv, cu), (q, kc, vc, ks[:1], vs, table, kv, cu),
                 (q, kc, vc, ks, vs, table[0], kv, cu), (q, kc, vc, ks, vs, table, kv, cu[:1]),
                 (q[..., :32].contiguous(), kc, vc, ks, vs, table, kv, cu), (q[..., ::2], kc, vc, ks, vs, table, kv, cu),
                 (q.cpu(), kc, vc, ks, vs, table, kv, cu), (q, kc.cpu(), vc, ks, vs, table, kv, cu)):
        with pytest.raises(ValueError):
            run(*args, 1.0)
    for args in ((q.half(), kc, vc, ks, vs, table, kv, cu), (q, kc, vc, ks.double(), vs, table, kv, cu),
                 (q, kc, vc, ks, vs, table.long(), kv, cu)):
        with pytest.raises(TypeError):
            run(*args, 1.0)
    with pytest.raises(memq.MemqError):
        run(q, kc, vc, ks, vs, table, kv, cu, 1.0, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(memq.MemqError):
        run(q, kc, vc, ks, vs, table, kv, cu, float("inf"))
    with pytest.raises(memq.MemqError):  # heads that no group divides
        run(q[:, :3].contiguous(), kc, vc, ks, vs, table, kv, cu, 1.0)
    with pytest.raises(memq.MemqError):  # rows that are not 16 bytes apart
        wide = torch.zeros(2, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")
        run(wide.as_strided((2, 4, 64), (260, 64, 1)), kc, vc, ks, vs, table, kv, cu, 1.0)
    with pytest.raises(ValueError):
        memq.memq_kv_cache_append(q, q, kv[:1].expand(2).contiguous(), kc, vc, ks, vs)  # 4 heads, the cache has 2
    with pytest.raises(TypeError):
        memq.memq_kv_cache_append(q[:, :2], q[:, :2].float(), cu, kc, vc, ks, vs)
    assert memq.memq_device_fault() == 0


# ------------------------------------------------------------------------------- the page plan
class Requests:
    def __init__(self, rng, n, page, max_pages, pages, chunk=40, used=0.6):
        cap = max_pages * page
        budget = pages * used / n * page
        self.page = page
        self.cached = np.minimum(rng.integers(0, max(2, int(2 * budget)), n), cap).astype(np.int64)
        while -(-self.cached // page).sum() > pages:
            self.cached //= 2
        kind = rng.integers(0, 6, n)
        self.keep = np.where(kind == 0, 0, np.where(kind == 1, np.maximum(0, self.cached - rng.integers(0, 9, n)), self.cached))
        self.new = np.where(kind <= 2, rng.integers(0, 4, n), np.where(kind == 3, rng.integers(0, chunk, n), 1))
        order = rng.permutation(pages)
        have = -(-self.cached // page)
        self.table = np.full((n, max_pages), -1, np.int64)
        at = 0
        for b in range(n):
            self.table[b, :have[b]] = order[at:at + have[b]]
            at += have[b]
        self.free = np.full(pages, -9, np.int64)
        self.free[:pages - at] = order[at:]
        self.n_free = pages - at

    def device(self):
        i = lambda x: to_dev(np.asarray(x, np.int32))  # noqa: E731
        return i(self.cached), i(self.new), i(self.table), i(self.free), i([self.n_free]), i(self.keep)

    def check(self, memq, n_tok=None, in_place=False):
        total = int(np.sum(self.new))
        n_tok = total if n_tok is None else n_tok
        cached, new, table, free, n_free, keep = self.device()
        kw = dict(kv_len=cached, n_free_out=n_free) if in_place else {}
        got = memq.memq_page_plan(cached, new, table, free, n_free, self.page, n_tok, keep=keep, **kw)
        if in_place:
            assert got[3] is cached and got[5] is n_free
        want = ref.plan(self.cached, self.keep, self.new, self.table, self.free, self.n_free, self.page, n_tok)
        for g, w, name in zip(got, want, ("slots", "positions", "cu_q", "kv_len", "granted", "n_free")):
            assert np.array_equal(g.cpu().numpy(), np.atleast_1d(w)), name
        assert np.array_equal(table.cpu().numpy(), self.table) and np.array_equal(free.cpu().numpy(), self.free)
        return want


@pytest.mark.parametrize("n,page,max_pages,pages", [(1, 16, 1, 1), (1, 64, 40, 50), (2, 16, 100, 64), (33, 32, 64, 400),
                                                  (1000, 16, 70, 9000), (1024, 64, 32, 4000), (1025, 16, 40, 5000),
                                                  (4096, 128, 16, 9000), (3000, 16, 30, 12000)])
def test_plan(memq, n, page, max_pages, pages):
    rng = np.random.default_rng(n + page)
    for used, in_place in ((0.5, False), (0.97, True), (0.2, True)):
        Requests(rng, n, page, max_pages, pages, used=used).check(memq, in_place=in_place)
    r = Requests(rng, n, page, max_pages, pages)
    r.check(memq, n_tok=int(r.new.sum()) + 77)
    assert memq.memq_device_fault() == 0


def test_plan_when_pages_run_out(memq):
    rng = np.random.default_rng(1)
    refused = 0
    for seed in range(12):
        r = Requests(rng, 50, 16, 40, 160, chunk=200, used=0.9)
        refused += (r.check(memq)[4] == 0).sum()
    assert refused > 0  # the case occurs
    r = Requests(rng, 20, 16, 3, 100, chunk=100)  # sequences that are full
    assert (r.check(memq)[4] == 0).sum() > 0
    assert memq.memq_device_fault() == 0


def test_plan_prompts_and_wide_batches(memq):
    rng = np.random.default_rng(2)
    r = Requests(rng, 3, 16, 9000, 20000, used=0.1)
    r.new[1] = 120000
    r.check(memq)
    r = Requests(rng, 300, 16, 400, 60000, chunk=900, used=0.1)
    r.check(memq)
    r.cached[:], r.keep[:] = 0, 0
    r = Requests(rng, 2000, 16, 30, 30000, used=0.5)
    r.keep[:] = 0  # all are finished
    r.new[:] = 0
    r.check(memq, n_tok=8)
    r = Requests(rng, 2000, 16, 30, 30000, used=0.5)
    r.new[:] = 0  # nothing happens
    r.check(memq, n_tok=0)
    assert memq.memq_device_fault() == 0


def test_plan_again_gives_the_same(memq):
    """With outputs of their own, a call's inputs are as before: a second call gives the same."""
    rng = np.random.default_rng(3)
    r = Requests(rng, 200, 16, 64, 3000)
    cached, new, table, free, n_free, keep = r.device()
    a = memq.memq_page_plan(cached, new, table, free, n_free, 16, 2000, keep=keep)
    t, f = table.clone(), free.clone()
    b = memq.memq_page_plan(cached, new, table, free, n_free, 16, 2000, keep=keep)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(t, table) and torch.equal(f, free)


def test_plan_input_faults_are_reported_and_contained(memq):
    def run(change, check):
        r = Requests(np.random.default_rng(4), 6, 16, 20, 60, used=0.5)
        r.keep[:], r.new[:] = r.cached, 2
        change(r)
        cached, new, table, free, n_free, keep = r.device()
        out = memq.memq_page_plan(cached, new, table, free, n_free, 16, 12, keep=keep)
        assert memq.memq_device_fault() == 32
        assert check(r, *(x.cpu().numpy() for x in out))
        s = out[0].cpu().numpy()
        assert np.all((s >= -1) & (s < 60 * 16))
    ok = lambda *a: True  # noqa: E731
    run(lambda r: r.cached.__setitem__(0, -3), ok)
    run(lambda r: r.cached.__setitem__(1, 10 ** 6), lambda r, s, p, cu, kv, g, n: kv[1] == r.keep[1] + 2)
    run(lambda r: r.keep.__setitem__(2, r.cached[2] + 5), ok)
    run(lambda r: r.new.__setitem__(3, -4), lambda r, s, p, cu, kv, g, n: cu[4] == cu[3] and kv[3] == r.cached[3])
    run(lambda r: r.new.__setitem__(5, 2 ** 30), lambda r, s, p, cu, kv, g, n: g[5] == 0 and cu[6] == 12)
    run(lambda r: setattr(r, "n_free", 61), ok)
    run(lambda r: setattr(r, "n_free", -1), ok)
    def bad_page(r):  # the partly filled page that the next tokens go to
        r.cached[0] = r.keep[0] = 17
        r.table[0, 1] = 60
    run(bad_page, lambda r, s, p, cu, kv, g, n: s[0] == -1)
    def too_many(r):
        r.n_free, r.keep[:], r.new[:] = 60, 0, 0
    run(too_many, lambda r, s, p, cu, kv, g, n: n[0] == 60)


def test_plan_refusals(memq):
    r = Requests(np.random.default_rng(5), 6, 16, 20, 60)
    cached, new, table, free, n_free, keep = r.device()
    run = memq.memq_page_plan
    for args in ((cached, new[:1], table, free, n_free, 16, 4), (cached, new, table[:2], free, n_free, 16, 4),
                 (cached, new, table, free, cached, 16, 4), (cached, new, table, free[:10].view(2, 5), n_free, 16, 4),
                 (cached, new, table, free, n_free, 16, -1), (cached.cpu(), new, table, free, n_free, 16, 4)):
        with pytest.raises(ValueError):
            run(*args)
    with pytest.raises(TypeError):
        run(cached.long(), new, table, free, n_free, 16, 4)
    for page in (0, 8, 24, 2048):
        with pytest.raises(memq.MemqError):
            run(cached, new, table, free, n_free, page, 4)
    assert memq.memq_device_fault() == 0


# ------------------------------------------------------------------------------- the calls together
class Model:
    """One attention layer between random projections: what a serving step computes around the calls."""

    def __init__(self, rng, nh, n_kv, d, vocab):
        self.nh, self.n_kv, self.d = nh, n_kv, d
        self.emb = to_dev(rng.normal(0, 1, (vocab, 96)).astype(np.float32))
        self.w = to_dev((rng.normal(0, 1, (96, (nh + 2 * n_kv) * d)) / 10).astype(np.float32))
        self.head = to_dev((rng.normal(0, 1, (nh * d, vocab)) / np.sqrt(d)).astype(np.float32))

    def qkv(self, tokens, positions):
        x = self.emb[tokens.long()] + torch.sin(0.3 * positions.float())[:, None]
        y = (x @ self.w).view(-1, self.nh + 2 * self.n_kv, self.d)
        return y[:, :self.nh], y[:, self.nh:self.nh + self.n_kv], y[:, self.nh + self.n_kv:]


def test_serving_steps(memq):
    """Prompts, decodes, rejected drafts, a finished and a replaced request, over a pool that is nearly full:
    plan, append, attention and sampling, each against its reference on the state as it was."""
    rng = np.random.default_rng(30)
    nh, n_kv, d, page, vocab, n = 6, 2, 64, 16, 500, 5
    model, pages, max_pages = Model(rng, nh, n_kv, d, vocab), 40, 12
    pool = Pool(rng, pages, n_kv, page, d)
    kc, vc, ks, vs = pool.device()
    table, free = np.full((n, max_pages), -1, np.int64), rng.permutation(pages).astype(np.int64)
    state = [to_dev(x.astype(np.int32)) for x in (table, free)]
    kv, n_free = torch.zeros(n, dtype=torch.int32, device="cuda"), to_dev(np.array([pages], np.int32))
    steps = [([0] * n, [37, 0, 90, 5, 16]),                    # prompts
             ([37, 0, 90, 5, 16], [1, 1, 4, 1, 1]),             # decodes, one with drafts
             ([38, 1, 92, 6, 0], [1, 1, 4, 1, 0]),              # two drafts rejected, one finished
             ([39, 2, 96, 0, 0], [1, 30, 1, 20, 150]),          # a prompt's chunk, one replaced, one new
             ([40, 32, 97, 20, 150], [1, 1, 1, 1, 1])]
    kv_host, left = np.zeros(n, np.int64), pages
    for keep, new in steps:
        n_tok = sum(new) + 3
        args = [to_dev(np.array(x, np.int32)) for x in (new, keep)]
        before = kv_host.copy()
        slots, pos, cu, kv2, ok, _ = memq.memq_page_plan(kv, args[0], state[0], state[1], n_free, page, n_tok, keep=args[1],
                                                         kv_len=kv, n_free_out=n_free)
        s, p, c, kv_host, granted, left = ref.plan(before, np.array(keep), np.array(new), table, free, left, page, n_tok)
        for got, want in ((slots, s), (pos, p), (cu, c), (kv, kv_host), (ok, granted), (state[0], table), (state[1], free),
                          (n_free, [left])):
            assert np.array_equal(got.cpu().numpy(), want)
        assert granted.all()

        tokens = to_dev(rng.integers(0, vocab, n_tok).astype(np.int32))
        q, k, v = model.qkv(tokens, pos)
        memq.memq_kv_cache_append(k, v, slots, kc, vc, ks, vs)
        ref.append(k.cpu().numpy(), v.cpu().numpy(), s, pool.codes, pool.scales, page)
        for got, want in zip((kc, vc, ks, vs), (*pool.codes, *pool.scales)):
            assert np.array_equal(got.cpu().numpy(), want)

        out = torch.zeros(n_tok, nh, d, device="cuda")
        memq.memq_attn_paged(q, kc, vc, ks, vs, state[0], kv, cu, d ** -0.5, out=out)
        qh, oh = q.cpu().numpy().astype(np.float64), out.double().cpu().numpy()
        for b in range(n):
            rows = np.arange(kv_host[b])
            at = table[b, rows // page] * page + rows % page
            kb, vb = (ref.values(pool.codes[i], pool.scales[i], at) for i in range(2))
            scales = pool.scales[1][at // page, :, at % page // 16].astype(np.float64)
            want, bound = ref.attend(qh[c[b]:c[b + 1]], kb, vb, new[b], d ** -0.5, 2, 2.0 ** -23, scales)
            assert np.all(np.abs(oh[c[b]:c[b + 1]] - want) <= bound)
        assert np.all(oh[c[-1]:] == 0)

        live = [b for b in range(n) if new[b]]
        logits = out.view(n_tok, -1)[cu[1:].long()[live] - 1] @ model.head
        u = rng.uniform(0, 1, len(live)).astype(np.float32)
        got = memq.memq_sample(logits, to_dev(u), temperature=torch.full((len(live),), 0.8, device="cuda"),
                               top_k=torch.full((len(live),), 40, dtype=torch.int32, device="cuda"),
                               top_p=torch.full((len(live),), 0.9, device="cuda"))
        for i, t in enumerate(got.tolist()):
            assert t in ref.sample(logits[i].cpu().numpy(), np.float32(0.8), 40, float(np.float32(0.9)), 0.0, float(u[i]))
    assert memq.memq_device_fault() == 0


def test_captured_decode_loop(memq):
    """A decode step captured once: lengths, block tables, slots, tokens and the draw move on with every replay;
    the same steps launched one by one give the same tokens and the same cache."""
    rng = np.random.default_rng(31)
    nh, n_kv, d, page, vocab, n, pages = 8, 2, 128, 16, 900, 7, 64
    model = Model(rng, nh, n_kv, d, vocab)
    us = to_dev(rng.uniform(0, 1, (40, n)).astype(np.float32))
    ws = torch.empty(memq.memq_attn_paged_workspace(d), dtype=torch.uint8, device="cuda")
    order = rng.permutation(pages).astype(np.int32)

    def fresh():
        kc, vc = (torch.zeros(pages, n_kv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(pages, n_kv, 1, device="cuda") for _ in range(2))
        i = dict(dtype=torch.int32, device="cuda")
        return dict(kc=kc, vc=vc, ks=ks, vs=vs, table=torch.full((n, 8), -1, **i), free=to_dev(order),
                    n_free=torch.full((1,), pages, **i), kv=torch.zeros(n, **i), new=torch.ones(n, **i),
                    slots=torch.empty(n, **i), pos=torch.empty(n, **i), cu=torch.empty(n + 1, **i),
                    ok=torch.empty(n, **i), tok=torch.arange(n, **i), u=us[0].clone(), out=torch.empty(n, nh, d, device="cuda"),
                    topp=torch.full((n,), 0.95, device="cuda"))

    def step(s):
        memq.memq_page_plan(s["kv"], s["new"], s["table"], s["free"], s["n_free"], page, n, kv_len=s["kv"],
                            n_free_out=s["n_free"], cu_q=s["cu"], slots=s["slots"], positions=s["pos"], granted=s["ok"])
        q, k, v = model.qkv(s["tok"], s["pos"])
        memq.memq_kv_cache_append(k, v, s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
        memq.memq_attn_paged(q, s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["kv"], s["cu"], d ** -0.5, out=s["out"],
                             workspace=ws)
        memq.memq_sample(s["out"].view(n, -1) @ model.head, s["u"], top_p=s["topp"], out=s["tok"])

    a, b = fresh(), fresh()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        warm = fresh()
        step(warm)
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    tokens = []
    for i in range(40):
        a["u"].copy_(us[i])
        g.replay()
        b["u"].copy_(us[i])
        step(b)
        assert torch.equal(a["tok"], b["tok"]) and torch.equal(a["out"], b["out"])
        tokens.append(a["tok"].tolist())
    assert a["kv"].tolist() == [40] * n and a["n_free"].item() == pages - 3 * n
    assert all(torch.equal(a[x], b[x]) for x in ("kc", "vc", "ks", "vs", "table", "free", "slots"))
    assert len({tuple(t) for t in tokens}) > 20
    assert memq.memq_device_fault() == 0
