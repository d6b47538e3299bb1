"""GPU tests of the steps where their gates leave fp32's range on the way: thresholds
past exp's largest argument."""

import pytest
import torch

import gated_delta_rule_61_amd as gdn
import oracle
from gated_delta_rule_61_amd import workloads
from tests.mixer_cases import BF, d
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
