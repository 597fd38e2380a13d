"""GPU tests of memq_page_plan where new tokens pass n_tok, against the plan by its definition."""
import numpy as np
import pytest

from test_gpu_kv import Requests, memq  # noqa: F401

pytestmark = pytest.mark.gpu


def plan(cached, keep, new, table, free, n_free, page, n_tok):
    """The page plan by its definition: requests that get no token need no room for any."""
    pages = lambda n: -(-n // page)  # noqa: E731
    table, free, n = table.copy(), free.copy(), len(cached)
    ends = np.cumsum(new)
    room = [keep[b] + new[b] <= table.shape[1] * page and (new[b] == 0 or ends[b] <= n_tok) for b in range(n)]
    top = n_free
    for b in range(n):
        for c in range(pages(keep[b] + new[b]), pages(cached[b])):
            if room[b]:
                free[top] = table[b, c]
                top += 1
    stack, asked, kv, granted = top, 0, list(cached), [0] * n
    for b in range(n):
        take = max(0, pages(keep[b] + new[b]) - pages(cached[b])) if room[b] else 0
        asked += take
        if room[b] and (take == 0 or asked <= stack):
            granted[b], kv[b] = 1, keep[b] + new[b]
            for c in range(pages(cached[b]), pages(cached[b]) + take):
                top -= 1
                table[b, c] = free[top]
    cu = np.minimum(np.r_[0, ends], n_tok)
    slots, positions = np.full(n_tok, -1), np.full(n_tok, -1)
    for b in range(n):
        for t in range(cu[b], cu[b + 1]):
            positions[t] = i = keep[b] + t - cu[b]
            if granted[b]:
                slots[t] = table[b, i // page] * page + i % page
    return (slots, positions, cu, kv, granted, [top]), table, free


def served(memq, r, n_tok):  # noqa: F811
    cached, new, table, free, n_free, keep = r.device()
    got = memq.memq_page_plan(cached, new, table, free, n_free, r.page, n_tok, keep=keep)
    want, t, f = plan(r.cached, r.keep, r.new, r.table, r.free, r.n_free, r.page, n_tok)
    for g, w, name in zip(got, want, ("slots", "positions", "cu_q", "kv_len", "granted", "n_free")):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert np.array_equal(table.cpu().numpy(), t) and np.array_equal(free.cpu().numpy(), f)
    return want


def test_requests_without_new_tokens_are_served_behind_too_many(memq):  # noqa: F811
    """New tokens past n_tok are not served; a finished request behind them gives its pages back, a shortened one its
    last ones, an idle one stays, and pages that came back are there for requests in front."""
    r = Requests(np.random.default_rng(40), 7, 16, 20, 90, used=0.0)
    r.cached[:] = [20, 33, 48, 70, 16, 40, 17]
    r.keep[:] = [20, 33, 0, 30, 16, 40, 17]
    r.new[:] = [3, 60, 0, 0, 0, 5, 0]  # the second passes n_tok
    have = -(-r.cached // 16)
    at, pages = 0, np.random.default_rng(41).permutation(90)
    for b in range(7):
        r.table[b, :have[b]] = pages[at:at + have[b]]
        at += have[b]
    r.n_free = 90 - at
    r.free[:r.n_free] = pages[at:]
    want = served(memq, r, 12)
    assert want[4] == [1, 0, 1, 1, 1, 0, 1] and want[3] == [23, 33, 0, 30, 16, 40, 17]
    assert want[5] == [90 - at + 3 + 3] and memq.memq_device_fault() == 32


@pytest.mark.parametrize("n", [40, 1500])
def test_plans_with_room_for_some_of_the_tokens(memq, n):  # noqa: F811
    rng = np.random.default_rng(n)
    for share in (0.0, 0.3, 0.8):
        r = Requests(rng, n, 16, 40, 30 * n, chunk=60)
        served(memq, r, int(share * r.new.sum()))
        assert memq.memq_device_fault() == 32
        r = Requests(rng, n, 16, 40, 30 * n, chunk=60)
        served(memq, r, int(r.new.sum()))
        assert memq.memq_device_fault() == 0
