"""Paged latent attention over many small weights beside few large ones: what the small ones carry together
must arrive in the output, however far below the largest each of them lies."""
import numpy as np
import pytest
import torch

import paged_reference as ref

T, NH, RANK, ROPE, PAGE, KV = 160, 64, 128, 32, 64, 20000
# Of the sum of |weight x value|: a weight's own error (2^-8 of it, 2^-11 more for its f16 form), the scores' f32 sums
# (2^-12), and the rows whose small weights a key on top may cost: its own tile of 128, and the next, which notices.
SHARE = 1.125 * 2.0 ** -8 + 2.0 ** -12 + 256 / KV


def single(gap):
    """One key `gap` nats above all others."""
    s = np.zeros(KV)
    s[0] = gap
    return s


def late(gap):
    s = np.zeros(KV)
    s[700] = gap
    return s


def stairs(gap):
    """One key, then 500 of them at two thirds of its height, then the rest."""
    s = np.zeros(KV)
    s[0], s[1:501] = gap, gap * 2 / 3
    return s


SHAPES = {"single": single, "late": late, "stairs": stairs}


def case(shape, gap, seed=31):
    """(q [T, NH, width], codes, scales, softmax scale): keys' scores are the shape's, spread by 0.3 nats; values of
    the key on top are near zero, all others' share a mean."""
    rng = np.random.default_rng(seed)
    target = SHAPES[shape](gap)
    scale = 1.5 / np.sqrt(RANK + ROPE)
    beta = gap / (scale * 2.0 * np.sqrt(ROPE))             # the largest rope element is 2
    q = np.empty((T, NH, RANK + ROPE))
    q[..., :RANK] = 0.1 * rng.normal(size=(T, NH, RANK))
    q[..., :RANK] -= q[..., :RANK].mean(2, keepdims=True)  # blind to the common mean
    q[..., RANK:] = beta / np.sqrt(ROPE)
    x = np.empty((KV, RANK + ROPE))
    x[:, :RANK] = 1 + 0.1 * rng.normal(size=(KV, RANK))
    x[target == target.max(), :RANK] *= 0.01
    x[:, RANK:] = 2.0 * (target / gap)[:, None] + 0.3 / (scale * beta) * rng.normal(size=(KV, ROPE)) * (target < gap)[:, None]
    codes, scales = ref.quantise(x.astype(np.float32))
    return ref.bf16(q.astype(np.float32)).astype(np.float64), codes, scales, scale


def expected(q, codes, scales, scale, tokens):
    """Per token: (output, sum of |weight x value| over the sum of weights, share of weights under 2^-17 of the top)."""
    c = ref.E4M3[codes] * scales[:, None].astype(np.float64)
    for i in tokens:
        ci = c[: KV - T + i + 1]
        s = scale * q[i] @ ci.T
        p = np.exp(s - s.max(1, keepdims=True))
        u = p * scales[: len(ci)]
        small = u < 2.0 ** -17 * u.max(1, keepdims=True)
        v, total = ci[:, :RANK], p.sum(1, keepdims=True)
        yield i, p @ v / total, p @ np.abs(v) / total, (p * small) @ v / total


GAPS = [9.0, 10.0, 11.0, 12.0, 13.0, 14.0]


def test_a_lost_tail_is_seen():
    """Dropping the weights that are far below the largest fails the check of the GPU test."""
    for gap in (13.0, 14.0):
        for _, out, mean, lost in expected(*case("single", gap), [T - 1]):
            assert np.linalg.norm(lost) > 10 * SHARE * np.linalg.norm(mean)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("gap", GAPS)
def test_small_weights_arrive(shape, gap):
    """160 new tokens over 20000 rows: every SM walks along some 160 tiles."""
    import quantized_decode_memq_gb300 as memq
    q, codes, scales, scale = case(shape, gap)
    pages = -(-KV // PAGE)
    pool = np.zeros((pages * PAGE, RANK + ROPE), np.uint8)
    pool[:KV] = codes
    sc = np.full(pages * PAGE, np.nan, np.float32)
    sc[:KV] = scales
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    qd = dev(q.astype(np.float32)).bfloat16()
    out = torch.empty(T, NH, RANK, device="cuda")
    memq.memq_mla_attn_paged(qd[..., :RANK].contiguous(), qd[..., RANK:].contiguous(), dev(pool.reshape(pages, PAGE, -1)),
                             dev(sc.reshape(pages, PAGE)), dev(np.arange(pages, dtype=np.int32)[None]),
                             dev(np.array([KV], np.int32)), dev(np.array([0, T], np.int32)), scale, out=out)
    got = out.double().cpu().numpy()
    assert memq.memq_device_fault() == 0
    for i, want, mean, _ in expected(q, codes, scales, scale, [0, T // 2, T - 1]):
        err = np.linalg.norm(got[i] - want) / np.linalg.norm(mean)
        assert err <= SHARE, f"token {i}: {err / SHARE:.2f} of the bound"


def test_the_two_terms_of_a_weight():
    """A weight p = hi + lo as the kernel forms it (bits 14..7 of f16(p / 256) and the high byte of 256 times the
    rest, both rounded) is within 1.13 x 2^-8 of p, or 1.13 x 2^-14: f16 2^-11, E4M3 2^-4, E5M2 2^-3 of the rest, half
    a step each, and steps of 2^-9, 2^-16 and 2^-16 at the lower end."""
    p = np.concatenate([2.0 ** np.arange(-20, 8.79, 0.0007), 2.0 ** -16 * np.arange(0, 5000)])
    x = (p / 256).astype(np.float16)
    hi = ((x.view(np.uint16).astype(np.uint32) + 0x40) & 0xFF80).astype(np.uint16).view(np.float16)
    lo = ((x - hi) * np.float16(256)).astype(np.float16)
    lo = ((lo.view(np.uint16).astype(np.uint32) + 0x80) & 0xFF00).astype(np.uint16).view(np.float16)
    got = 256 * hi.astype(np.float64) + lo.astype(np.float64)
    assert np.all(np.abs(got - p) <= 1.13 * np.maximum(2.0 ** -8 * p, 2.0 ** -14))
