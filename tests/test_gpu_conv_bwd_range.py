"""GPU tests of the convolution's gradients where silu's argument is large."""

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
from tests.mixer_cases import BF, close, d, f64, randn

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("io", [BF, F32])
def test_slope_of_large_arguments(io):
    """The tap is 1 and alone, so c = x and dx = dy silu'(x).  silu' = p + c (1 - p): exp's argument is good to |c| 2^-23
    and exp, the reciprocal and the sums to 2^-22 each, so 1 - p is off by at most 2^-20 p, and by 0 once e^-c is
    below half a step of 1, at c = 17.4 (where p is 1); for negative c, p is off by |c| 2^-22 + 2^-20 of itself."""
    c = torch.tensor([0.0, 1, 5, 9, 12, 16, 18, 40, 100, 1e3, 1e4, 65504, 65528, 1e5, 4e6, 1e7, 2.0 ** 24, 1e8, 1e20, 1e37])
    c = torch.cat([c, -c[:12], torch.full((8,), 2.5)])
    assert c.numel() % 8 == 0
    T, D = 3, c.numel()
    x = c.expand(1, T, D).contiguous().to(io)
    w = torch.zeros(D, 2, dtype=io)
    w[:, 1] = 1
    dy = randn(1, 1, T, D, dtype=io)
    dx, dw, _ = gdn.causal_conv_bwd(d(dy), d(x), d(w))
    v = f64(x)
    e = np.exp(-np.abs(v))
    p = np.where(v >= 0, 1.0, e) / (1 + e)
    ref = f64(dy) * (p + v * e / (1 + e) ** 2)
    off = np.where(v >= 0, 2.0 ** -20 * (1 + np.minimum(v, 18)), p * (1 + np.abs(v)) * (np.abs(v) * 2.0 ** -22 + 2.0 ** -20))
    bar = np.abs(f64(dy)) * off + 2.0 ** -125
    close("dx", f64(dx), ref, bar + (2.0 ** -8 if io == BF else 2.0 ** -24) * (np.abs(ref) + bar))
