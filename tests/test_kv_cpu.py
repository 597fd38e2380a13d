"""The K/V cache, the attention over it, the page plan and the sampler on the CPU: the f64 reference's own
pins, and refusals before any CUDA call."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import kv_reference as ref
from paged_reference import E4M3
from quantized_decode_memq_gb300.build import CSRC


@pytest.fixture(scope="module")
def lib():
    from quantized_decode_memq_gb300 import build
    try:
        build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    import quantized_decode_memq_gb300 as m
    return m.lib()


# ------------------------------------------------------------------------------- pins of the reference
def test_scale_is_the_least_power_of_two():
    for top, want in ((448, 1), (448.0001, 2), (224, 0.5), (224.1, 1), (1, 2.0 ** -8), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7),
                      (0, 2.0 ** -100), (1e-44, 2.0 ** -100), (3e38, 2.0 ** 120)):
        assert ref.scale_of(top) == want
        assert top <= 448 * want


def test_append_fresh_grown_and_kept():
    codes, scales = [np.zeros((2, 1, 16, 4), np.uint8) for _ in range(2)], [np.zeros((2, 1, 1), np.float32) for _ in range(2)]
    put = lambda x, slots: ref.append(np.asarray(x, np.float32)[:, None], np.asarray(x, np.float32)[:, None], slots,  # noqa: E731
                                      codes, scales, 16)
    put([[1, 0.5, 0, -1]], [0])
    assert scales[0][0, 0, 0] == 2.0 ** -8
    put([[96, 0, 0, 0]], [1])  # needs 2^-2: row 0 moves along
    assert scales[0][0, 0, 0] == 0.25 and ref.values(codes[0], scales[0], [0, 1])[:, 0].tolist() == [[1, 0.5, 0, -1], [96, 0, 0, 0]]
    put([[1, 1, 1, 1]], [2])  # the scale stays
    assert scales[0][0, 0, 0] == 0.25
    put([[1, 1, 1, 1]], [0])  # afresh
    assert scales[0][0, 0, 0] == 2.0 ** -8
    put([[np.nan, 1, 1, 1], [2, 2, 2, 2]], [16, 17])
    v = [ref.values(codes[i], scales[i], [16, 17])[:, 0] for i in range(2)]
    assert np.all(np.isnan(v[0][0])) and np.all(v[1][0] == 0) and np.all(v[0][1] == 2) and np.all(v[1][1] == 2)


def test_attend_closed_forms():
    """Identical rows give that row; two keys by hand; an unseen row has no part."""
    k = np.zeros((3, 1, 4))
    v = np.arange(12.0).reshape(3, 1, 4)
    k[:, 0, 0] = [0, np.log(3), 50]
    q = np.zeros((2, 2, 4))
    q[..., 0] = 1
    out, bound = ref.attend(q, k, v, 2, 1.0, 2, 0, np.ones((3, 1)))
    np.testing.assert_allclose(out[0], np.broadcast_to((v[0, 0] + 3 * v[1, 0]) / 4, (2, 4)), rtol=1e-12)
    np.testing.assert_allclose(out[1], np.broadcast_to(v[2, 0], (2, 4)), rtol=1e-12)
    out, bound = ref.attend(np.ones((4, 2, 4)), k, v, 4, 1.0, 2, 0, np.ones((3, 1)))
    assert np.all(out[0] == 0) and np.all(bound[0] == 0) and np.all(np.isfinite(out))


def test_plan_by_hand():
    table = np.array([[4, 5, -1], [6, -1, -1], [-1, -1, -1]])
    free = np.array([0, 1, 2, 3, -1, -1, -1])
    # request 0 is replaced by one of three tokens, 1 grows over its page, 2 wants more than is left
    s, p, cu, kv, ok, left = ref.plan([20, 15, 0], [0, 15, 0], [3, 2, 48], table, free, 1, 16, 60)
    assert free[:2].tolist() == [0, 5] and left == 1 and ok.tolist() == [1, 1, 0]
    assert table.tolist() == [[4, 5, -1], [6, 5, -1], [-1, -1, -1]]
    assert cu.tolist() == [0, 3, 5, 53] and kv.tolist() == [3, 17, 0]
    assert s[:5].tolist() == [64, 65, 66, 111, 80] and np.all(s[5:] == -1)
    assert p[:6].tolist() == [0, 1, 2, 15, 16, 0] and p[52] == 47 and np.all(p[53:] == -1)


def test_sample_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3])).astype(np.float32)
    for u, want in ((0.05, 0), (0.3, 1), (0.55, 2), (0.9, 3), (0.0, 0), (1.0, 3)):
        assert ref.sample(x, 1.0, 0, 1.0, 0.0, u) == {want}
    assert ref.sample(x, 1.0, 2, 1.0, 0.0, 0.5) == {1} and ref.sample(x, 1.0, 2, 1.0, 0.0, 0.6) == {3}
    assert ref.sample(x, 1.0, 0, 0.65, 0.0, 0.99) == {3} and ref.sample(x, 1.0, 0, 0.75, 0.0, 0.5) == {2}
    assert ref.sample(x, 1.0, 0, 1.0, 0.6, 0.99) == {3} and ref.sample(x, 1.0, 0, 1.0, 0.6, 0.01) == {1}
    assert ref.sample(x, 0.0, 0, 1.0, 0.0, 0.9) == {1} and ref.sample(x, 1e-9, 0, 1.0, 0.0, 0.9) == {1}
    assert ref.sample(np.zeros(5, np.float32), 1.0, 3, 1.0, 0.0, 0.99) == {2}


def test_codes_decode_as_torch_does():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, E4M3, equal_nan=True)


# ------------------------------------------------------------------------------- refusals
def call(fn, good):
    return lambda **kw: fn(*{**good, **kw}.values())


def test_validation_rejects_before_any_cuda_call(lib):
    import quantized_decode_memq_gb300 as m
    S, P = m.Status, ctypes.c_void_p
    f, odd, odder = P(0x1000), P(0x1008), P(0x1002)  # never dereferenced

    good = dict(cached=f, keep=f, new=f, table=f, free=f, n_free=f, kv=f, n_out=f, cu=f, slots=f, pos=f, granted=f, n_seq=4,
                n_tok=8, max_pages=8, page=16, pages=64, st=None)
    plan = call(lib.memq_page_plan, good)
    for bad in (dict(n_seq=-1), dict(n_seq=4097), dict(n_tok=-1), dict(n_tok=(1 << 24) + 1), dict(page=8), dict(page=24),
                dict(page=2048), dict(pages=0), dict(pages=-1), dict(pages=1 << 27), dict(max_pages=0),
                dict(max_pages=(1 << 26) + 1), dict(n_seq=0)):
        assert plan(**bad) == S.ERR_SHAPE, bad
    for name in ("cached", "new", "table", "free", "n_free", "kv", "n_out", "cu", "slots", "pos", "granted"):
        assert plan(**{name: None}) == S.ERR_NULL, name
        assert plan(**{name: odder}) == S.ERR_ALIGN, name
    assert plan(keep=odder) == S.ERR_ALIGN
    nothing = {k: None for k in list(good)[:12]}
    assert plan(n_seq=0, n_tok=0, **nothing) == S.OK

    good = dict(dt=1, k=f, ks=512, v=f, vs=512, slots=f, kc=f, ksc=f, vc=f, vsc=f, n=4, n_kv=2, d=64, pages=16, page=32,
                st=None)
    app = call(lib.memq_kv_cache_append, good)
    for bad in (dict(dt=2), dict(dt=-1), dict(n=-1), dict(n=(1 << 24) + 1), dict(n_kv=0), dict(n_kv=1025), dict(d=96),
                dict(d=256), dict(page=8), dict(page=48), dict(page=2048), dict(pages=-1), dict(pages=1 << 25), dict(ks=-8),
                dict(vs=-8)):
        assert app(**bad) == S.ERR_SHAPE, bad
    for name in ("k", "v", "slots", "kc", "ksc", "vc", "vsc"):
        assert app(**{name: None}) == S.ERR_NULL, name
    for name in ("k", "v", "kc", "vc"):
        assert app(**{name: odd}) == S.ERR_ALIGN, name
    for name in ("slots", "ksc", "vsc"):
        assert app(**{name: odder}) == S.ERR_ALIGN, name
    for name in ("ks", "vs"):  # rows 16 bytes apart
        assert app(**{name: 516}) == S.ERR_ALIGN and app(dt=0, **{name: 514}) == S.ERR_ALIGN
    assert app(n=0, **{k: None for k in ("k", "v", "slots", "kc", "ksc", "vc", "vsc")}) == S.OK

    good = dict(dt=1, cache=f, scales=f, slots=f, out=f, n=4, n_kv=2, d=64, pages=16, page=32, st=None)
    read = call(lib.memq_kv_cache_read, good)
    for bad in (dict(dt=3), dict(n=-1), dict(n_kv=0), dict(d=32), dict(page=40), dict(pages=1 << 25)):
        assert read(**bad) == S.ERR_SHAPE, bad
    for name in ("cache", "scales", "slots", "out"):
        assert read(**{name: None}) == S.ERR_NULL and read(**{name: odder}) == S.ERR_ALIGN, name
    assert read(n=0, cache=None, scales=None, slots=None, out=None) == S.OK

    good = dict(qt=1, q=f, qs=4096, kc=f, ksc=f, vc=f, vsc=f, table=f, kv=f, cu=f, ot=1, out=f, ws=f, wsn=1 << 40, n_tok=4,
                n_seq=2, nh=64, n_kv=8, d=64, pages=16, page=64, max_pages=8, scale=0.1, st=None)
    attn = call(lib.memq_attn_paged, good)
    for bad in (dict(qt=2), dict(ot=-1), dict(n_tok=-1), dict(n_tok=(1 << 24) + 1), dict(n_seq=-1), dict(n_seq=4097),
                dict(nh=0), dict(nh=1032, n_kv=8), dict(n_kv=0), dict(n_kv=7), dict(d=96), dict(d=0), dict(page=8),
                dict(page=48), dict(page=2048), dict(pages=0), dict(pages=1 << 24), dict(max_pages=0),
                dict(max_pages=(1 << 24) + 1), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38),
                dict(qs=-8), dict(n_tok=1 << 24, nh=256)):
        assert attn(**bad) == S.ERR_SHAPE, bad
    for name in ("q", "kc", "ksc", "vc", "vsc", "table", "kv", "cu", "out", "ws"):
        assert attn(**{name: None}) == S.ERR_NULL, name
    for name in ("q", "kc", "vc", "out", "ws"):
        assert attn(**{name: odd}) == S.ERR_ALIGN, name
    for name in ("ksc", "vsc", "table", "kv", "cu"):
        assert attn(**{name: odder}) == S.ERR_ALIGN, name
    assert attn(qs=4100) == S.ERR_ALIGN
    nothing = {k: None for k in ("q", "kc", "ksc", "vc", "vsc", "table", "kv", "cu", "out", "ws")}
    assert attn(n_tok=0, **nothing) == S.OK and attn(n_seq=0, **nothing) == S.OK
    assert lib.memq_attn_paged_workspace(96) == -1

    good = dict(dt=0, x=f, stride=1000, t=f, k=f, p=f, mp=f, u=f, out=f, rows=4, vocab=1000, st=None)
    samp = call(lib.memq_sample, good)
    for bad in (dict(dt=2), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0), dict(vocab=360001), dict(stride=-1)):
        assert samp(**bad) == S.ERR_SHAPE, bad
    for name in ("x", "u", "out"):
        assert samp(**{name: None}) == S.ERR_NULL, name
    for name in ("x", "t", "k", "p", "mp", "u", "out"):
        assert samp(**{name: odder}) == S.ERR_ALIGN, name
    assert samp(dt=1, x=P(0x1001)) == S.ERR_ALIGN
    assert samp(rows=0, x=None, u=None, out=None) == S.OK


def test_binding_refuses_host_tensors_and_wrong_kinds(lib):
    import quantized_decode_memq_gb300 as m
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        m.memq_page_plan(i, i, torch.zeros(2, 3, dtype=torch.int32), i, i[:1], 16, 4)
    kc, ks = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 1)
    x = torch.zeros(2, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        m.memq_kv_cache_append(x, x, i, kc, kc, ks, ks)
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        m.memq_kv_cache_append(x.half(), x.half(), i, kc, kc, ks, ks)
    with pytest.raises(ValueError, match="CUDA"):
        m.memq_kv_cache_read(kc, ks, i)
    with pytest.raises(ValueError, match="CUDA"):
        m.memq_attn_paged(x, kc, kc, ks, ks, i.view(1, 2), i[:1], i, 1.0)
    with pytest.raises(TypeError):
        m.memq_attn_paged(None, kc, kc, ks, ks, i, i, i, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        m.memq_sample(torch.zeros(2, 5), torch.zeros(2))
    with pytest.raises(TypeError):
        m.memq_sample(torch.zeros(2, 5, dtype=torch.float16), torch.zeros(2))


def test_the_sampler_reaches_into_other_ctas_between_cluster_barriers():
    """Another CTA's shared memory is touched only behind the entry barrier's wait, and a wait stands behind the last time."""
    with open(os.path.join(CSRC, "memq_sample.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.index("sample_kernel(const SampleArgs a) {"):text.index("bool misaligned(")]
    remote = [m.start() for m in re.finditer(r"\b(?:in_cta|join_lists<T>|cluster_sum<T>)\(", body)]
    waits = [m.start() for m in re.finditer(r"\b(?:cluster_sync|cluster_wait)\(\)", body)]
    entry = [m.start() for m in re.finditer(r"\bcluster_wait_entry\(\)", body)]
    assert len(entry) == 1 and body.index("cluster_arrive_entry()") < entry[0] < remote[0]
    assert len(remote) > 10 and remote[-1] < waits[-1]
