"""GPU tests of the group norm and its gradients where fp32's range or precision
ends: groups whose sums or squares leave it, saturated gates; and a bias without a
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


SATURATED = [0.0, 3.0, 8.0, 11.0, 12.5, 15.0, 17.0, 20.0, 30.0, 60.0, 80.0, 200.0, 1e4, 1e30]


def slope(a, act):
    """act'(a) without cancellation; e^{-|a|} underflows to 0 in 64 bits where fp32's is 0 long before"""
    e = np.exp(-np.abs(a))
    q = e / (1 + e) ** 2
    if act == "sigmoid":
        return q
    return np.where(a >= 0, 1.0, e) / (1 + e) + a * q


def slope_bound(a, act):
    """exp's argument is scaled by log2(e) first, one rounding of its size: (|a| 2^-23 + 2^-22) of e^{-a}, the
    reciprocal 2^-22 of its own, twice, the product three roundings; taken twice: 2^-19 + |a| 2^-22 of a (1 - p) p.
    Below 2^-125 nothing is asked for.  silu adds a times that, and p, which is as good."""
    e = np.exp(-np.abs(a))
    q = e / (1 + e) ** 2
    rel = 2.0 ** -19 + np.minimum(np.abs(a), 200) * 2.0 ** -22
    if act == "sigmoid":
        return rel * q + 2.0 ** -125
    return rel * (np.where(a >= 0, 1.0, e) / (1 + e) + np.abs(a) * q) + 2.0 ** -125


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("io", [BF, F32])
def test_saturated_gates(act, io):
    v = torch.tensor(SATURATED + [-s for s in SATURATED] + [0.0] * 4)
    z = v.repeat(2).reshape(1, 1, 64).to(io)
    x = torch.ones(1, 1, 64, dtype=io)
    x[..., ::3] = -1
    dy = (randn(1, 1, 1, 64).abs() + 0.5).to(io)
    _, dz, _, _ = gdn.group_norm_bwd(d(dy), d(x), 1, z=d(z), activation=act, rms=True, eps=0.0)
    zz, a = f64(z), f64(dy) * f64(x)     # n is x to 2^-21
    ref = a * slope(zz, act)
    bar = np.abs(a) * slope_bound(zz, act) + 2.0 ** -20 * np.abs(ref)
    close("dz", f64(dz), ref, bar + (2.0 ** -8 if io == BF else 2.0 ** -24) * (np.abs(ref) + bar))


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_saturated_results(act):
    # one token: dbias = dy act'(n w), with n = 1 to 2^-21, so the argument is good to 2^-21 of itself
    w = torch.tensor([s for s in SATURATED if s < 100] + [-s for s in SATURATED if s < 100] + [1.0] * 2)
    x = torch.ones(1, 1, w.numel())
    dy = randn(2, 1, 1, w.numel()).abs() + 0.5
    _, _, _, db = gdn.group_norm_bwd(d(dy), d(x), 1, d(w), d(torch.zeros_like(w)), activation=act, rms=True, eps=0.0)
    a = f64(w)
    ref = f64(dy)[0, 0] * slope(a, act)
    shift = np.abs(a) * 2.0 ** -20          # of the argument; the slopes' logarithms change by at most that ..
    size = f64(dy)[0, 0] * (slope_bound(a, act) + shift * slope_bound(a, act) / (2.0 ** -19 + np.abs(a) * 2.0 ** -22))
    close("dbias", f64(db), ref, 2 * size)


def test_forward_of_saturated_gates_is_unchanged_in_its_limits():
    z = torch.tensor([[[200.0, -200.0, 1e30, -1e30, 30.0, -30.0, float("inf"), 0.0]]])
    x = torch.ones(1, 1, 8)
    y = gdn.group_norm_fwd(d(x), 1, z=d(z), activation="sigmoid", rms=True, eps=0.0)
    ref = np.array([[[1, 0, 1, 0, 1 / (1 + np.exp(-30.0)), 1 / (1 + np.exp(30.0)), 1, 0.5]]])
    close("y", f64(y), ref, 2.0 ** -18 * ref + 2.0 ** -125)
