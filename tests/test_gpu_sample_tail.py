"""GPU parity of memq_sample where a cut falls among weights below 2^-24 of the largest, in rows of one CTA
and of several: against the f64 evaluation of its definition."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from test_gpu_sample import memq  # noqa: F401

pytestmark = pytest.mark.gpu


def may_give(x, temperature, k, p, u):
    """All tokens that the draw may give.  Every weight is within 2^-41 of the largest one's, so sums of up to n are within
    n 2^-41 of the exact ones, at the cut and at the draw: top-p may end at any place between those of the two ends, and
    for each such set of kept tokens the draw lies between the places of u's sum less and plus that."""
    w = np.exp((x.astype(np.float64) - x.max()) / float(temperature))
    order = np.lexsort((np.arange(len(x)), -x))[:k if k else len(x)]
    eps = len(order) * 2.0 ** -41
    cum = np.cumsum(w[order])
    ahead = cum - w[order]
    least, most = (max(1, int((ahead < p * cum[-1] + e).sum())) for e in (-eps, eps))
    got = set()
    for kept in range(least, most + 1):
        some = np.sort(order[:kept])
        run = np.cumsum(w[some])
        lo, hi = (min(kept - 1, int((run <= u * run[-1] + e).sum())) for e in (-eps, eps))
        got.update(some[lo:hi + 1].tolist())
    return got


def check(memq, x, temperature, k, p, u):  # noqa: F811
    dev = [to_dev(np.asarray(v, t)) for v, t in ((temperature, np.float32), (k, np.int32), (p, np.float32), (u, np.float32))]
    got = memq.memq_sample(x, dev[3], temperature=dev[0], top_k=dev[1], top_p=dev[2]).tolist()
    t, k, p, u = (v.tolist() for v in dev)
    for r, row in enumerate(x.float().cpu().numpy()):
        may = may_give(row, t[r], k[r], p[r], u[r])
        assert got[r] in may, (r, got[r], sorted(may)[:20], t[r], k[r], p[r], u[r])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(6, 30001), (3, 128259), (40, 20000)])
def test_cuts_among_the_small_weights(memq, n, v, dtype):  # noqa: F811
    """One token far above all others, which together have a hundredth to a thousandth of the weight: top-p of
    more than the first ends among them; behind a top-k too."""
    rng = np.random.default_rng(20)
    x = rng.normal(0, 0.3, (n, v)).astype(np.float32)
    top = rng.integers(0, v, n)
    x[np.arange(n), top] = 18.2 + rng.uniform(0, 0.5, n)  # 26 octaves and more
    small = np.exp(x - x.max(1, keepdims=True)).astype(np.float64).sum(1) - 1
    p = (1 - small * rng.uniform(0.2, 0.8, n)).astype(np.float32)
    assert np.all(p > 1 - small) and np.all(p < 1)
    x = to_dev(x).to(dtype)
    for k in (0, v - 7, v // 2):
        check(memq, x, np.ones(n), np.full(n, k), p, rng.choice([0.5, 1 - 2.0 ** -24, 0.9999], n))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_k_behind_all_weights_then_top_p(memq, dtype):  # noqa: F811
    """At a low temperature the k-th token has no weight left; top-p follows."""
    rng = np.random.default_rng(21)
    n, v = 12, 60000
    x = to_dev(rng.normal(0, 2, (n, v)).astype(np.float32)).to(dtype)
    for _ in range(4):
        check(memq, x, rng.choice([0.01, 0.03, 0.05], n), rng.choice([5000, 30000, v - 1], n),
              rng.choice([0.5, 0.9, 0.999], n), rng.uniform(0, 1, n))
