"""GPU parity of memq_attn_paged over values whose scales are all tiny: relative precision down to scales of
2^-80, documented steps below."""
import numpy as np
import pytest
import torch

from test_gpu_kv import Batch, memq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[(1, 700)], [(3, 90), (40, 300)]], ids=str)
@pytest.mark.parametrize("lo,hi", [(-70, -60), (-80, -70), (-90, -80), (-100, -90), (-100, -60)])
def test_attention_over_tiny_values(memq, lo, hi, lens, out_type):  # noqa: F811
    """The bound of kv_reference.attend without its absolute 2^-90, and, for scales below 2^-80, the steps of 2^-33 (an
    error of 2^-34) of the largest weight times 2^-80 that each of the weights, times codes of 448 at most, may be off:
    sum_j 2^-34 2^-80 max(p) |code_j| / sum_j p_j <= 2^-114 448 n."""
    b = Batch(lens, 8, 2, 64, 16, torch.float32, seed=40)
    rng = np.random.default_rng(41)
    used = ~np.isnan(b.scales[1])
    b.scales[1][used] = np.exp2(rng.integers(lo, hi + 1, used.sum())).astype(np.float32)
    got = b.run(memq, out_type).double().cpu().numpy()
    want, bound = b.reference(out_type)
    bound = bound - 2.0 ** -90
    if lo < -80:
        at = 0
        for t, kv in lens:
            bound[at:at + t] += 2.0 ** -114 * 448 * kv * (1 + 2.0 ** -7)
            at += t
    seen = np.abs(want) > 0
    worst = np.abs(got - want)[seen] / bound[seen]
    assert worst.max() <= 1, (worst.max(), np.abs(got).max(), np.abs(want).max())
    assert memq.memq_device_fault() == 0
