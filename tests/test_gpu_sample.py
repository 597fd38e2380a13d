"""GPU parity of memq_sample: every row's token against the f64 evaluation of its definition."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from gpu_helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def memq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_decode_memq_gb300 import build
    build.build()
    import quantized_decode_memq_gb300 as m
    m.memq_device_fault()
    return m


def check(memq, logits, temperature, k, p, min_p, u):
    """All as numpy arrays; logits f32 (or a tensor)."""
    x = logits if isinstance(logits, torch.Tensor) else to_dev(logits)
    n = x.shape[0]
    full = lambda v, t: np.broadcast_to(np.asarray(v, t), (n,)).copy()  # noqa: E731
    temperature, p, min_p, u = (full(v, np.float32) for v in (temperature, p, min_p, u))
    k = full(k, np.int32)
    got = memq.memq_sample(x, to_dev(u), temperature=to_dev(temperature), top_k=to_dev(k), top_p=to_dev(p),
                           min_p=to_dev(min_p)).cpu().numpy()
    host = x.float().cpu().numpy()
    for r in range(n):
        may = ref.sample(host[r], temperature[r], int(k[r]), float(p[r]), float(min_p[r]), float(u[r]))
        assert int(got[r]) in may, (r, int(got[r]), may, temperature[r], k[r], p[r], min_p[r], u[r])
    return got


def settings(rng, n):
    return (rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.7], n), rng.choice([0, 0, 1, 2, 5, 40, 64, 300, 1500], n),
            rng.choice([1.0, 1.0, 0.0, 0.1, 0.5, 0.9, 0.95, 0.99, 0.999], n), rng.choice([0, 0, 0, 0.01, 0.1, 1], n),
            rng.uniform(0, 1, n))


def peaked(rng, n, v):
    x = (2 * rng.normal(0, 1, (n, v))).astype(np.float32)
    for r in range(n):
        at = rng.integers(0, v, min(v, 40))
        x[r, at] += rng.uniform(2, 16) * rng.uniform(0, 1, len(at))
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 2), (5, 33), (40, 1000), (9, 2049), (64, 5003), (20, 32000), (300, 4001),
                                (6, 128259), (30, 50001), (3, 360000)])
def test_rows(memq, n, v, dtype):
    rng = np.random.default_rng(n + v)
    check(memq, to_dev(peaked(rng, n, v)).to(dtype), *settings(rng, n))


@pytest.mark.parametrize("spread", [0.01, 0.5, 2.0, 6.0])
def test_flat_and_steep_rows(memq, spread):
    """Tens of thousands of tokens carry the weight, or a handful."""
    rng = np.random.default_rng(3)
    n, v = 24, 60000
    x = (spread * rng.normal(0, 1, (n, v))).astype(np.float32)
    t, k, p, m, u = settings(rng, n)
    check(memq, x, np.where(t == 0, 1, t), k, p, m, u)
    check(memq, to_dev(x).bfloat16(), 1.0, 0, np.linspace(0.01, 0.9999, n), 0.0, u)


@pytest.mark.parametrize("n", [24, 200])
def test_long_bfloat16_rows(memq, n):
    """Few values many times, of every magnitude: about zero, far below the largest, masked, all negative."""
    rng = np.random.default_rng(10)
    v = 40003
    x = peaked(rng, n, v) * rng.choice([1e-3, 0.1, 1.0, 1.0, 30.0], (n, 1)).astype(np.float32)
    x[0::6] -= 25
    x[1::6, rng.random(v) < 0.5] = -np.inf
    x[2::6] *= np.exp2(-rng.integers(0, 30, v)).astype(np.float32)
    x[3::6, 1000:] = np.where(rng.random(v - 1000) < 0.5, 0.0, -0.0)
    x[4::6, rng.random(v) < 0.3] = 1e-38
    x[5::12, rng.random(v) < 0.01] = np.nan
    t, k, p, m, u = settings(rng, n)
    x = to_dev(x).bfloat16()
    with np.errstate(invalid="ignore"):
        check(memq, x, np.where(t == 0, 1, t), k, p, m, u)
        check(memq, x, rng.choice([0.05, 1, 20, 1e4, 1e29], n), 0, rng.choice([0.3, 0.9, 1.0], n), 0.0, u)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(200, 16384), (4, 50000)])
def test_many_of_the_largest(memq, n, v, dtype):
    """top_k of hundreds to nearly all, in rows of one CTA and of several, near and far from the largest."""
    rng = np.random.default_rng(11)
    x = to_dev((rng.choice([0.1, 2.0, 8.0], (n, 1)) * rng.normal(0, 1, (n, v))).astype(np.float32)).to(dtype)
    k = rng.choice([257, 500, 1000, 1025, 3000, 12000, v - 1], n)
    for t in (rng.choice([0.05, 0.3, 1.0, 4.0], n), np.full(n, 100.0)):
        check(memq, x, t, k, rng.choice([1.0, 1.0, 0.9], n), rng.choice([0, 0, 1e-3], n), rng.choice([0.999999, 0.5, 0.99], n))


def test_equal_logits(memq):
    """Ties at every cut: all tokens alike, or one of a few values; the lowest indices are kept."""
    v = 20000
    x = np.full((12, v), 3.25, np.float32)
    x[6:] = np.random.default_rng(4).integers(0, 3, (6, v))
    u = np.linspace(0, 0.9999, 12)
    for k, p in ((0, 1.0), (0, 0.5), (7, 1.0), (5000, 1.0), (5000, 0.25), (0, 0.75), (19999, 0.999)):
        got = check(memq, x, 1.0, k, p, 0.0, u)
        assert got.min() >= 0 and got.max() < v
    assert np.all(memq.memq_sample(to_dev(x), to_dev(u.astype(np.float32)), top_k=to_dev(np.full(12, 3, np.int32)))
                  .cpu().numpy()[:6] <= 2)
    assert np.all(check(memq, x[:6], 0.0, 0, 1.0, 0.0, 0.5) == 0)


def test_masked_and_not_finite_logits(memq):
    rng = np.random.default_rng(5)
    x = peaked(rng, 10, 3000)
    x[0, 5:] = -np.inf
    x[1] = -np.inf
    x[2] = np.nan
    x[3, ::2] = np.nan
    x[4, [70, 900]] = np.inf
    x[5, :2000] = -np.inf
    x[6] = np.where(rng.random(3000) < 0.5, 0.0, -0.0)
    x[7, 10] = 3.4e38
    x[8] = -3.4e38
    x[9, :] = -np.inf
    x[9, 2999] = -5
    for k, p in ((0, 1.0), (50, 1.0), (0, 0.9), (2999, 0.6), (20, 0.5)):
        for t in (0.0, 1.0, 1e-38, 1e30):
            with np.errstate(invalid="ignore"):
                check(memq, x, t, k, p, 0.02, rng.uniform(0, 1, 10))


def test_borders_of_the_settings(memq):
    rng = np.random.default_rng(6)
    x = peaked(rng, 8, 700)
    nan, inf = np.nan, np.inf
    u = np.array([0, 1, -3, nan, inf, 0.99999994, 0.5, 1e-30], np.float32)
    n = lambda a: np.where(np.isnan(a), 0, a)  # noqa: E731
    got = memq.memq_sample(to_dev(x), to_dev(u)).cpu().numpy()
    for r in range(8):
        assert int(got[r]) in ref.sample(x[r], 1.0, 0, 1.0, 0.0, float(n(u)[r]))
    base = rng.uniform(0, 1, 8)
    for name, odd, plain in (("temperature", [nan, -1, 0, -inf], 0.0), ("top_p", [nan, 1, 7, inf], 1.0),
                             ("temperature", [inf, 1e30, 3e38, inf], 1e30), ("temperature", [1e-30, 1e-45, 1e-38, 1e-31], 1e-30),
                             ("min_p", [nan, -1, 0, -inf], 0.0), ("min_p", [1, 2, inf, 1.0000001], 1.0),
                             ("top_p", [0, -1, -inf, -0.0], 0.0), ("top_k", [0, -5, 700, 10 ** 9], 0)):
        t = np.int32 if name == "top_k" else np.float32
        a = memq.memq_sample(to_dev(x), to_dev(base.astype(np.float32)), **{name: to_dev(np.array(odd * 2, t))})
        b = memq.memq_sample(to_dev(x), to_dev(base.astype(np.float32)), **{name: to_dev(np.full(8, plain, t))})
        assert torch.equal(a, b), name


def test_frequencies(memq):
    """Evenly spaced u visit every token as often as its weight says, to one in each."""
    p = np.array([0.05, 0.3, 0.0, 0.15, 0.5])
    with np.errstate(divide="ignore"):
        x = np.log(p).astype(np.float32)
    n = 4000
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    got = memq.memq_sample(to_dev(np.tile(x, (n, 1))), to_dev(u)).cpu().numpy()
    assert np.all(np.diff(got) >= 0)
    assert np.all(np.abs(np.bincount(got, minlength=5) - n * p) <= 1.01)


def test_strided_rows_and_outputs(memq):
    rng = np.random.default_rng(7)
    for dtype in (torch.float32, torch.bfloat16):
        wide = to_dev(peaked(rng, 5, 7007)).to(dtype)
        u = to_dev(rng.uniform(0, 1, 5).astype(np.float32))
        for lo, hi in ((0, 7007), (1, 5000), (3, 7004), (7, 8)):
            out = torch.full((5,), -1, dtype=torch.int32, device="cuda")
            got = memq.memq_sample(wide[:, lo:hi], u, out=out)
            assert got is out and torch.equal(got, memq.memq_sample(wide[:, lo:hi].contiguous(), u))
        same = memq.memq_sample(wide[:1].expand(5, 7007), u)
        assert torch.equal(same, memq.memq_sample(wide[:1].repeat(5, 1), u))
    assert memq.memq_sample(wide[:0], u[:0]).shape == (0,)


def test_a_row_does_not_depend_on_the_others(memq):
    """The same row alone (a cluster of CTAs) and among hundreds (one CTA)."""
    rng = np.random.default_rng(8)
    x = to_dev(np.tile(peaked(rng, 8, 20011), (40, 1)))
    u = to_dev(np.tile(rng.uniform(0, 1, 8).astype(np.float32), 40))
    p = to_dev(np.tile(np.array([1, 0.9, 0.5, 0.99, 1, 1, 0.8, 1], np.float32), 40))
    k = to_dev(np.tile(np.array([0, 0, 0, 0, 50, 400, 30, 3000], np.int32), 40))
    many = memq.memq_sample(x, u, top_p=p, top_k=k)
    assert torch.equal(many.view(40, 8), many[:8].expand(40, 8))
    for r in range(8):
        one = slice(r, r + 1)
        assert memq.memq_sample(x[one], u[one], top_p=p[one], top_k=k[one]).item() == many[r].item()


def test_captured_call_and_two_streams(memq):
    rng = np.random.default_rng(9)
    x, u = to_dev(peaked(rng, 16, 9000)), to_dev(rng.uniform(0, 1, 16).astype(np.float32))
    p = torch.full((16,), 0.9, device="cuda")
    want = memq.memq_sample(x, u, top_p=p)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        memq.memq_sample(x, u, top_p=p, out=out)
    g.replay()
    assert torch.equal(out, want)
    p.fill_(0.3)
    u.mul_(0.5)
    g.replay()
    assert torch.equal(out, memq.memq_sample(x, u, top_p=p))
    sts, outs = [torch.cuda.Stream() for _ in range(3)], []
    want = out.clone()
    torch.cuda.synchronize()
    for _ in range(5):
        for st in sts:
            with torch.cuda.stream(st):
                outs.append(memq.memq_sample(x, u, top_p=p))
        outs.append(memq.memq_sample(x, u, top_p=p, stream=sts[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_refusals(memq):
    x, u = torch.zeros(3, 50, device="cuda"), torch.zeros(3, device="cuda")
    k = torch.zeros(3, dtype=torch.int32, device="cuda")
    run = memq.memq_sample
    for args, kw in (((x.cpu(), u), {}), ((x, u.cpu()), {}), ((x, u[:2]), {}), ((x[0], u), {}), ((x.t(), u), {}),
                     ((x, u), dict(top_k=k[:1])), ((x, u), dict(top_p=u[:1])), ((x, u), dict(out=k[:2]))):
        with pytest.raises(ValueError):
            run(*args, **kw)
    for args, kw in (((x.half(), u), {}), ((x, u.double()), {}), ((x, u), dict(top_k=u)), ((x, u), dict(top_p=k)),
                     ((x, u), dict(out=u)), ((None, u), {})):
        with pytest.raises(TypeError):
            run(*args, **kw)
    for bad in (torch.zeros(1, 360001, device="cuda"), torch.zeros(1, 0, device="cuda")):
        with pytest.raises(memq.MemqError):
            run(bad, u[:1])
    assert memq.memq_device_fault() == 0
