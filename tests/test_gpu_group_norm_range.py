"""GPU tests of the group norm and its gradients where fp32's range or precision
ends: groups whose sums or squares leave it; and a bias without a
weight.  Bounds: the running error analysis where values are ordinary ones, else as
derived at each test."""

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
from tests.mixer_cases import BF, close, d, f64, randn
from tests.test_gpu_group_norm import F32, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,T,G,D", [(1, 1, 16, 128), (1, 2, 16, 80), (2, 5, 3, 40), (1, 100, 16, 128), (1, 1024, 2, 520),
                                     (1, 7, 1, 2048)])
def test_a_bias_alone(B, T, G, D, shared):
    i = make(T, B, T, G, D, F32, shared=shared, gated=False)
    i["w"] = None
    check(i, G, "silu", False)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("D", [8, 80, 128, 1024, 1032, 8192])
def test_sums_past_fp32(D, io):
    # one sign, so that the sum of a group passes fp32's largest number where no element does
    i = make(D, 1, 4, 2, D, F32, gated=False, bias=False)
    i["x"] = (i["x"].abs() * 0.2 + 0.5).clamp(max=1.0) * 3e38 * torch.tensor([1.0, -1.0, 1e-3, 1.0])[None, :, None]
    i["dy"] = i["dy"] * 1e30   # dx of order 1e-8
    i["x"], i["dy"] = i["x"].to(io), i["dy"].to(io)
    for rms in (False, True):
        check(i, 2, None, rms)


@pytest.mark.parametrize("io", [BF, F32])
def test_elements_of_both_signs_at_the_end_of_the_range(io):
    # x - mean of an element may pass fp32's largest number too
    for D in (64, 8192):
        i = make(D, 1, 2, 1, D, F32, gated=False, bias=False)
        i["x"] = torch.full((1, 2, D), 3.3e38)
        i["x"][:, 0, : D // 8] = -3.3e38
        i["x"][:, 1, : 7 * D // 8] = -3.3e38
        i["x"], i["dy"] = i["x"].to(io), (i["dy"] * 1e30).to(io)
        for rms in (False, True):
            check(i, 1, None, rms)


def test_small_variance_around_a_large_mean_without_eps():
    # the deviations, 1e-18 of nothing else, are exact; their squares leave fp32's normal numbers
    dev = torch.tensor([1.0, -1.0]).repeat(32) * 2.0 ** -60
    x = torch.stack([dev, 3 * dev, 2.0 ** -40 + dev.double().float()]).reshape(1, 3, 64)
    y = gdn.group_norm_fwd(d(x), 1, activation=None, rms=False, eps=0.0)
    close("y", f64(y)[0], np.sign(f64(dev))[None].repeat(3, 0), np.full((3, 64), 2.0 ** -19))
