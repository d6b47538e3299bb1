"""GPU tests of the steps where their gates or norms leave fp32's range on the way:
thresholds past exp's largest argument, rates exp(A_log) past fp32, rows whose squares
fp32 does not hold."""

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
import oracle
from gated_delta_rule_61_amd import workloads
from tests.mixer_cases import BF, close, d, f64, randn
from tests.test_gpu_kda_decode import F32, check, make
from tests.tolerance import check as parity

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("thr", [60.0, 85.0, 1000.0, float("inf")])
def test_thresholds_past_exps_largest_argument(thr):
    i = make(1, 3, 2, 1, 2, 64, 64, F32, F32)
    i["A_log"] = torch.full((2,), -7.0)
    i["a"] = torch.linspace(-5, 400, 64).expand(3, 2, 2, 64).contiguous()
    check(i, thr=thr)
    check(i, thr=thr, sb=3.0)


@pytest.mark.parametrize("thr", [85.0, 1000.0, float("inf")])
@pytest.mark.parametrize("B", [1, 70])
def test_thresholds_of_the_scalar_step(thr, B):
    i = workloads.make_decode(B, 2, 2, 4, 128, 128, seed=3)
    i.a = torch.linspace(-5, 400, i.a.numel()).reshape(i.a.shape).to(BF)
    i.A_log = torch.full_like(i.A_log, -7.0)
    state = d(i.state).clone()
    o = gdn.gdn_decode(d(i.q), d(i.k), d(i.v), d(i.a), d(i.b), d(i.A_log), d(i.dt_bias), state, scale=i.scale,
                       softplus_threshold=thr)
    torch.cuda.synchronize()
    # at these thresholds log(1 + e^x) and x are the same number from x = 40 on, so 60 says what any of them says
    ro, rs = oracle.gdn_decode(i.q, i.k, i.v, i.a, i.b, i.A_log, i.dt_bias, i.state, scale=i.scale,
                               softplus_threshold=60.0)
    parity("o", o, ro, BF)
    parity("state", state, rs, BF)


@pytest.mark.parametrize("sb", [1.0, 0.25, 8.0])
@pytest.mark.parametrize("A", [60.0, 65.0, 88.0, 89.0, 95.0, 110.0, 143.0, 160.0, 1000.0])
def test_rates_past_fp32_times_small_steps(A, sb):
    """Keys of 0: the state only decays, by exp(-exp(A_log) softplus(a)), which is exp(-e^{A_log + sb a} / sb) for
    these a.  The exponent's sum is exact to 2^-24 of its size (at most 8 here), exp to 2^-21, so the rate to
    2^-19 of itself and the decay to that times the rate, and 2^-21."""
    K = 64
    i = make(2, 1, 1, 1, 1, K, 64, F32, F32, pool=1)
    # sums A + sb a of fp32 numbers, exact in 64 bits
    a = ((torch.linspace(-8, 4, K) - A) / sb).float()
    i["a"], i["dt_bias"], i["A_log"] = a.reshape(1, 1, 1, K), torch.zeros(1, K), torch.full((1,), A)
    i["k"].zero_()
    g = {n: d(t) for n, t in i.items()}
    gdn.kda_decode(g["q"], g["k"], g["v"], g["a"], g["b"], g["A_log"], g["dt_bias"], g["state"], softplus_beta=sb)
    bu = f64(a * torch.tensor(sb))            # in fp32, as the step forms it (powers of two: exact)
    near = np.clip(bu, -30, 30)               # below, log(1 + e^x) is e^x
    rate = np.exp(A + bu) / sb * np.where(bu < -30, 1.0, np.log1p(np.exp(near)) / np.exp(near))
    ref = f64(i["state"]) * np.exp(-rate)
    close("state", f64(g["state"]), ref, np.abs(f64(i["state"])) * np.exp(-rate) * (rate * 2.0 ** -19 + 2.0 ** -20) + 2.0 ** -125)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_rows_whose_squares_leave_fp32(K, V, io):
    i = make(4, 4, 2, 2, 2, K, V, io, F32)
    size = torch.tensor([1e25, 1e-25, 3e37, 1.0])[:, None, None, None]
    i["q"] = (i["q"].float() * size.flip(0)).to(io)
    i["k"] = (i["k"].float() * size).to(io)
    check(i, eps=0.0)
    i["k"][1:2] = i["k"][3:4]                 # with eps, 1e-25 is as good as 0
    i["q"][2:3] = i["q"][0:1]
    check(i)
