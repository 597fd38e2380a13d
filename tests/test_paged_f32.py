"""Paged latent attention with f32 queries and f32 outputs: operands hold the eleven bits of their f16 forms."""
import numpy as np
import pytest
import torch

import paged_reference as ref
from test_gpu_paged import Batch


def f16(bits):
    return bits.astype(np.uint16).view(np.float16)


def bits(x):
    return x.astype(np.float16).view(np.uint16).astype(np.uint32)


def test_three_terms_of_a_query_and_of_a_weight():
    """As the kernel forms them.  A query element v (the row's largest in [1/2, 1)): E4M3 codes of v and of the rest,
    bits 14..7 of their f16 forms, and the E5M2 code of 256 times what then is left; a weight p: the E4M3 code of
    p / 256 and two E5M2 codes of 256 times the rest.  Both hold the f16 form, half a step 2^-11 of the value; below
    2^-10 (2^-6 for a weight) the E4M3 steps of 2^-17 leave the E5M2 code, of three bits, 2^-18 and less: half a step
    of its upper end is 2^-21 (for a weight the two E5M2 codes have the f16 form's step, 2^-16, and half of it)."""
    v = 2.0 ** np.arange(-26, 0, 0.0007)
    x = v.astype(np.float16)
    hi = f16((bits(x) + 0x40) & 0xFF80)
    rest = (x - hi).astype(np.float16)
    mid = f16((bits(rest) + 0x40) & 0xFF80)
    lo = f16((bits((rest - mid).astype(np.float16) * np.float16(256)) + 0x80) & 0xFF00)
    got = hi.astype(np.float64) + mid.astype(np.float64) + lo.astype(np.float64) / 256
    assert np.all(np.abs(got - v) <= np.maximum(2.0 ** -11 * v, 2.0 ** -21))

    p = np.concatenate([2.0 ** np.arange(-20, 8.79, 0.0007), 2.0 ** -16 * np.arange(0, 5000)])
    x = (p / 256).astype(np.float16)
    hi = f16((bits(x) + 0x40) & 0xFF80)
    rest = ((x - hi) * np.float16(256)).astype(np.float16)
    mid = f16((bits(rest) + 0x80) & 0xFF00)
    lo = f16((bits((rest - mid).astype(np.float16)) + 0x80) & 0xFF00)
    got = 256 * hi.astype(np.float64) + mid.astype(np.float64) + lo.astype(np.float64)
    assert np.all(np.abs(got - p) <= np.maximum(2.0 ** -11 * p, 2.0 ** -17))


# Roundings of the operands are independent and within half a step of 2^-11: 2^-11 / sqrt 3 rms.  Scores of width
# 1.5 are off by 1.5 times that, weights by as much as it: together 5.1e-4 of the output, and 2^-10 is 1.9 times that
# (8-bit terms of either operand give 2^-9 and more).
RMS = 2.0 ** -10


def relative(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.fixture(scope="module")
def memq():
    import quantized_decode_memq_gb300 as m
    m.memq_device_fault()
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [128, 256, 512])
@pytest.mark.parametrize("rope", [0, 32, 64, 128])
def test_f32_in_f32_out(memq, rank, rope):
    b = Batch([(3, 700), (1, 77), (2, 0)], 20, rank, rope, 16, torch.float32, seed=rank + rope, row_scale=0.0)
    b.check(memq, torch.float32)
    got = b.run(memq, torch.float32).double().cpu().numpy()
    want, _ = b.reference(torch.float32)
    assert np.all(got[4:] == 0) and relative(got[:4], want[:4]) <= RMS


@pytest.mark.gpu
@pytest.mark.parametrize("rank,rope", [(512, 128), (512, 64), (512, 0), (128, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_runs_of_tiles(memq, rank, rope, dtype):
    """Every SM walks over many tiles: at rank 512, rope 128 the ring holds a single tile beside the terms."""
    b = Batch([(40, 1500), (2, 3000)], 64, rank, rope, 64, dtype, seed=rank, row_scale=0.0)
    got = b.run(memq, torch.float32)
    assert torch.equal(b.run(memq, torch.float32), got)
    got = got.double().cpu().numpy()
    want, bound = b.reference(torch.float32)
    assert np.all(np.abs(got - want) <= bound) and relative(got, want) <= RMS
    assert memq.memq_device_fault() == 0


@pytest.mark.gpu
def test_types_of_queries_and_outputs(memq):
    """The f32 output rounded is the bf16 output but for the third terms; a bf16 output of f32 queries is within one
    more rounding, 2^-9 / sqrt 3 rms with the weights' two terms (2^-9.6)."""
    b = Batch([(5, 900)], 24, 512, 64, 64, torch.float32, seed=41, row_scale=0.0)
    want, _ = b.reference(torch.float32)
    low = b.run(memq, torch.bfloat16).double().cpu().numpy()
    assert relative(low, want) <= np.sqrt(2.0 ** -18 / 3 + 2.0 ** -19.2 + RMS ** 2)


@pytest.mark.gpu
def test_an_element_far_above_the_others(memq):
    """Elements of an f32 query 2^-12 and less of its largest still have 2^-21 of that: the scores say so."""
    b = Batch([(2, 600)], 8, 128, 32, 16, torch.float32, seed=42, row_scale=0.0)
    b.q[..., 130] = 3000.0                                  # a position element
    b.codes[..., 130] = 0                                   # that no key answers
    got = b.run(memq, torch.float32).double().cpu().numpy()
    want, _ = b.reference(torch.float32)
    # |dq| <= 2^-20 of 3000 = 2.9e-3 per element, 2^-11 in the mean; uniform: x 1.5 / sqrt 3
    assert relative(got, want) <= RMS + 2.9e-3 * 1.5 / np.sqrt(3)
