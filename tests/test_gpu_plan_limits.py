"""GPU tests of memq_page_plan at the numbers of requests where its shared memory passes the default limit."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from conftest import ROOT
from gpu_helpers import to_dev
from test_gpu_kv import Requests, memq  # noqa: F401

pytestmark = pytest.mark.gpu

ASCENDING = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
import numpy as np
import quantized_decode_memq_gb300 as memq
from test_gpu_kv import Requests
for n in (2036, 2037, 2038, 2042, 2047, 2048, 4096, 2038, 4095):
    Requests(np.random.default_rng(n), n, 16, 12, 8 * n, chunk=9).check(memq)
assert memq.memq_device_fault() == 0
print("served")
"""


def test_every_number_of_requests_is_served_in_a_process_of_its_own(memq):  # noqa: F811
    """The default limit holds for what the kernel declares and what a call asks for together: in ascending order no
    larger call has raised it before."""
    code = ASCENDING.format(tests=os.path.join(ROOT, "tests"), root=ROOT)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "served" in r.stdout, r.stderr[-2000:]


def test_calls_of_two_threads_do_not_lower_one_anothers_limit(memq):  # noqa: F811
    """Large and smaller plans from two host threads, each on its stream; and a large one captured around smaller ones."""
    errors = []

    def many(n, stream):
        r = Requests(np.random.default_rng(n), n, 16, 12, 8 * n, chunk=9)
        cached, new, table, free, n_free, keep = r.device()
        n_tok = int(r.new.sum())
        names = ("slots", "positions", "cu_q", "kv_len", "granted", "n_free_out")
        try:
            outs = memq.memq_page_plan(cached, new, table, free, n_free, 16, n_tok, keep=keep)
            torch.cuda.synchronize()
            for _ in range(1500):
                memq.memq_page_plan(cached, new, table, free, n_free, 16, n_tok, keep=keep, stream=stream,
                                    **dict(zip(names, outs)))
        except memq.MemqError as e:
            errors.append((n, str(e)))
        stream.synchronize()

    threads = [threading.Thread(target=many, args=(n, torch.cuda.Stream())) for n in (4096, 2100, 3000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    large, small = (Requests(np.random.default_rng(n), n, 16, 12, 8 * n, chunk=9) for n in (4096, 2100))
    args, kept = [], []
    for r in (large, small):
        cached, new, table, free, n_free, keep = r.device()
        args.append((cached, new, table, free, n_free, 16, int(r.new.sum())))
        kept.append(keep)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [memq.memq_page_plan(*a, keep=k) for a, k in zip(args, kept)]
    memq.memq_page_plan(*(x.clone() if isinstance(x, torch.Tensor) else x for x in args[1]), keep=kept[1])
    g.replay()
    torch.cuda.synchronize()
    for r, out, a in zip((large, small), outs, args):
        want = memq.memq_page_plan(*r.device()[:5], 16, a[6], keep=r.device()[5])
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    assert memq.memq_device_fault() == 0
