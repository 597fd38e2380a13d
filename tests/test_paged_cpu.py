"""The paged latent cache and memq_add_rmsnorm_q8_1 on the CPU: the f64 reference's own pins, and
refusals before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import paged_reference as ref


@pytest.fixture(scope="module")
def lib():
    from quantized_decode_memq_gb300 import build
    try:
        build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    import quantized_decode_memq_gb300 as m
    return m.lib()


def test_e4m3_against_torch():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3, equal_nan=True)
    x = np.random.default_rng(1).normal(0, 60, 4000).astype(np.float32)
    x = np.r_[x, np.float32(2.0 ** -10) * np.arange(-9, 10, dtype=np.float32), np.float32([448, -448, 17, 19, 0])]
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.E4M3[ref.to_e4m3(x)], ref.E4M3[want])


def test_bf16_against_torch():
    x = np.random.default_rng(2).normal(0, 3, 1000).astype(np.float32)
    assert np.array_equal(ref.bf16(x), torch.from_numpy(x).bfloat16().float().numpy())


def test_quantise_round_trip():
    """An element is at most half an E4M3 step (2^-4 of it, or 2^-10 scaled) off, the largest none."""
    x = np.random.default_rng(3).normal(0, 1, (50, 160)).astype(np.float32)
    x[7] = 0
    codes, scales = ref.quantise(x)
    back = ref.E4M3[codes] * scales[:, None].astype(np.float64)
    off = np.abs(back - x)
    assert np.all(off <= 2.0 ** -4 * 1.0001 * np.abs(x) + 2.0 ** -10 * scales[:, None])
    assert np.all(np.abs(ref.E4M3[codes]).max(1)[np.arange(50) != 7] == 448) and np.all(codes[7] == 0)


def test_attend_closed_forms():
    """Identical rows give that row; one row gives itself; an unseen row has no part."""
    rng = np.random.default_rng(4)
    codes, scales = ref.quantise(rng.normal(0, 1, (1, 160)).astype(np.float32))
    row = ref.E4M3[codes] * scales[:, None]
    q = rng.normal(0, 1, (3, 2, 160))
    out, _ = ref.attend(q, np.repeat(codes, 9, 0), np.repeat(scales, 9), 3, 128, 0.1, 0)
    np.testing.assert_allclose(out, np.broadcast_to(row[0, :128], out.shape), rtol=1e-12)
    out, _ = ref.attend(q, codes, scales, 3, 128, 0.1, 0)  # one cached row: tokens 0 and 1 see none
    assert np.all(out[:2] == 0)
    np.testing.assert_allclose(out[2], np.broadcast_to(row[0, :128], (2, 128)), rtol=1e-12)


def test_validation_rejects_before_any_cuda_call(lib):
    import quantized_decode_memq_gb300 as m
    S, P = m.Status, ctypes.c_void_p
    f, odd = P(0x1000), P(0x1008)  # never dereferenced
    norm = lib.memq_add_rmsnorm_q8_1  # (x, res, w, h, z, qs, d, ncols, rows, eps, stream)
    assert norm(f, f, f, f, None, f, f, 48, 1, 1e-6, None) == S.ERR_SHAPE
    assert norm(f, f, f, f, None, f, f, 65536, 1, 1e-6, None) == S.ERR_SHAPE
    assert norm(f, f, f, f, None, f, f, 64, -1, 1e-6, None) == S.ERR_SHAPE
    assert norm(f, f, f, f, None, f, f, 64, 1, -1.0, None) == S.ERR_SHAPE
    assert norm(f, None, f, f, None, f, f, 64, 1, 1e-6, None) == S.ERR_NULL
    assert norm(f, f, f, None, None, f, f, 64, 1, 1e-6, None) == S.ERR_NULL
    assert norm(f, odd, f, f, None, f, f, 64, 1, 1e-6, None) == S.ERR_ALIGN
    assert norm(f, f, f, odd, None, f, f, 64, 1, 1e-6, None) == S.ERR_ALIGN
    assert norm(None, None, None, None, None, None, None, 64, 0, 1e-6, None) == S.OK

    app = lib.memq_mla_cache_append  # (dtype, latent, k_pe, slots, cache, scales, n, rank, rope, pool, stream)
    assert app(2, f, f, f, f, f, 4, 512, 64, 128, None) == S.ERR_SHAPE
    assert app(0, f, f, f, f, f, 4, 384, 64, 128, None) == S.ERR_SHAPE
    assert app(0, f, f, f, f, f, 4, 512, 16, 128, None) == S.ERR_SHAPE
    assert app(0, f, f, f, f, f, -1, 512, 64, 128, None) == S.ERR_SHAPE
    assert app(0, f, f, f, f, f, 4, 512, 64, 1 << 31, None) == S.ERR_SHAPE
    assert app(0, f, None, f, f, f, 4, 512, 64, 128, None) == S.ERR_NULL
    assert app(0, f, None, f, f, None, 4, 512, 0, 128, None) == S.ERR_NULL
    assert app(0, odd, f, f, f, f, 4, 512, 64, 128, None) == S.ERR_ALIGN
    assert app(1, P(0x1004), f, f, f, f, 4, 512, 64, 128, None) == S.ERR_ALIGN
    assert app(1, f, f, f, odd, f, 4, 512, 64, 128, None) == S.ERR_ALIGN
    assert app(0, None, None, None, None, None, 0, 512, 64, 128, None) == S.OK

    read = lib.memq_mla_cache_read  # (dtype, cache, scales, slots, out, n, rank, rope, pool, stream)
    assert read(3, f, f, f, f, 4, 512, 64, 128, None) == S.ERR_SHAPE
    assert read(1, f, f, f, f, 4, 1024, 64, 128, None) == S.ERR_SHAPE
    assert read(1, f, f, f, None, 4, 512, 64, 128, None) == S.ERR_NULL
    assert read(0, f, f, f, odd, 4, 512, 64, 128, None) == S.ERR_ALIGN
    assert read(0, None, None, None, None, 0, 512, 64, 128, None) == S.OK

    good = dict(qt=1, q=f, pe=f, cache=f, scales=f, table=f, kv=f, cu=f, ot=1, out=f, ws=f, wsn=1 << 40,
                n_tok=4, n_seq=2, nh=64, rank=512, rope=64, pages=16, page=64, max_pages=8, scale=0.1, st=None)

    def attn(**kw):
        return lib.memq_mla_attn_paged(*{**good, **kw}.values())
    for bad in (dict(qt=2), dict(ot=-1), dict(n_tok=-1), dict(n_tok=(1 << 24) + 1), dict(n_seq=-1), dict(n_seq=4097),
                dict(nh=0), dict(nh=1025), dict(rank=1024), dict(rank=64), dict(rope=96), dict(rope=-32), dict(page=8),
                dict(page=48), dict(page=2048), dict(pages=0), dict(pages=1 << 26), dict(max_pages=0),
                dict(max_pages=1 << 26), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attn(**bad) == S.ERR_SHAPE, bad
    # key indices of a sequence, rounded up to a tile, stay in 31 bits; the scale in the exponent is finite
    assert attn(max_pages=(1 << 24) + 1) == S.ERR_SHAPE and attn(max_pages=1 << 20, page=1024, q=None) == S.ERR_NULL
    assert attn(max_pages=(1 << 20) + 1, page=1024) == S.ERR_SHAPE and attn(max_pages=1 << 24, q=None) == S.ERR_NULL
    assert attn(scale=3e38) == S.ERR_SHAPE and attn(scale=2e38, q=None) == S.ERR_NULL
    for name in ("q", "pe", "cache", "scales", "table", "kv", "cu", "out", "ws"):
        assert attn(**{name: None}) == S.ERR_NULL, name
    for name in ("q", "pe", "cache", "scales", "ws"):
        assert attn(**{name: odd}) == S.ERR_ALIGN, name
    for name in ("table", "kv", "cu", "out"):
        assert attn(**{name: P(0x1002)}) == S.ERR_ALIGN, name
    assert attn(ot=0, out=odd) == S.ERR_ALIGN
    nothing = {k: None for k in ("q", "pe", "cache", "scales", "table", "kv", "cu", "out", "ws")}
    assert attn(n_tok=0, **nothing) == S.OK and attn(n_seq=0, **nothing) == S.OK
    assert lib.memq_mla_attn_paged_workspace(384) == -1


def test_binding_refuses_host_tensors(lib):
    import quantized_decode_memq_gb300 as m
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        m.memq_add_rmsnorm_q8_1(x, x, torch.ones(64))
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        m.memq_mla_cache_append(torch.zeros(2, 512, dtype=torch.float16), None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        m.memq_mla_cache_read(torch.zeros(1, 16, 512, dtype=torch.uint8), torch.zeros(1, 16), None)
    with pytest.raises(ValueError, match="CUDA"):
        m.memq_mla_attn_paged(torch.zeros(1, 1, 512), None, None, None, None, None, None, 1.0)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """With more than one GPU, a tensor that is not on the current one is refused by name."""
    import quantized_decode_memq_gb300._binding as b

    class On:
        def __init__(self, index):
            self.index, self.device = index, f"cuda:{index}"

        def get_device(self):
            return self.index
    monkeypatch.setattr(b, "_devices", 2)
    monkeypatch.setattr(b, "_cur_device", lambda: 0)
    b._here("f", On(0), None, On(0))
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        b._here("f", On(0), None, On(1))


def test_dtype_is_the_headers_enum():
    import os
    import re
    import quantized_decode_memq_gb300 as m
    from quantized_decode_memq_gb300 import _binding, build
    with open(os.path.join(build.INCLUDE, "memq.h")) as f:
        body = re.search(r"typedef enum memq_dtype \{(.*?)\}", f.read()).group(1)
    assert {k: int(v) for k, v in re.findall(r"MEMQ_(\w+) = (\d+)", body)} == {d.name: int(d) for d in m.Dtype}
    assert _binding._DTYPES == {torch.float32: m.Dtype.F32, torch.bfloat16: m.Dtype.BF16}
    assert all(isinstance(d, m.Dtype) for d in _binding._DTYPES.values())
