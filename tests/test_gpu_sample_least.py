"""GPU test of memq_sample's least weights: whole numbers of 2^-44 of the largest one's."""
import numpy as np
import pytest
import torch

from gpu_helpers import to_dev
from test_gpu_sample import memq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("v", [900, 40000])
@pytest.mark.parametrize("how", [dict(), dict(top_k=50), dict(top_p=0.99999994)])
def test_the_last_token_that_has_a_weight(memq, v, how):  # noqa: F811
    """u = 1 draws the last token whose weight is more than 2^-45 of the largest's; the lesser ones behind it, and -infinity,
    are never drawn.  (A token at 2^-44 is beyond top-p of 1 - 2^-24.)"""
    octaves = np.array([44.2, 44.8, 45.3, 47.0, 59.0, 80.0, np.inf])
    x = np.full((7, v), -np.inf, np.float32)
    x[:, 3] = 5.0
    for r in range(7):
        x[r, v - 7:v - 7 + r + 1] = 5.0 - octaves[:r + 1] * np.log(2)
    full = {k: to_dev(np.full(7, p, np.int32 if k == "top_k" else np.float32)) for k, p in how.items()}
    got = memq.memq_sample(to_dev(x), torch.ones(7, device="cuda"), **full).tolist()
    want = [3] * 7 if "top_p" in how else [v - 7] + [v - 6] * 6
    assert got == want
