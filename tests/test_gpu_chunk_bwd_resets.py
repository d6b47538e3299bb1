"""GPU tests of log-gates that wipe the state out (a token that starts something new in
the middle of a sequence): any value whose exponential fp32 does not hold, -inf among
them, is a decay to 0, and what follows is what it is without anything before.  The
forward and its gradients against the fp64 oracle, at the bars of test_gpu_chunk_bwd."""

import pytest
import torch

import gated_delta_rule_61_amd as gdn
import oracle
from tests.mixer_cases import BF, d
from tests.test_gpu_chunk_bwd import F32, NAMES, compare, make, run, want
from tests.tolerance import check

pytestmark = pytest.mark.gpu
RESETS = [-90.0, -200.0, -1e4, -1e6, -1e30, float("-inf")]


def case(io, D, gate, lens=None):
    T = 200 if lens is None else sum(lens)
    i = make(7, 1, T, 1, 2, D, io, lens=lens)
    for t, h in ((0, 0), (5, 0), (63, 1), (64, 0), (100, 1), (101, 1), (130, 0), (190, 0), (199, 1)):
        i["g"][0, t, h] = gate
    return i


@pytest.mark.parametrize("gate", RESETS)
@pytest.mark.parametrize("lens", [None, [70, 0, 130]])
@pytest.mark.parametrize("io,D", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_gradients(io, D, lens, gate):
    i = case(io, D, gate, lens)
    compare(i, run(i))


@pytest.mark.parametrize("gate", RESETS)
@pytest.mark.parametrize("lens", [None, [70, 0, 130]])
@pytest.mark.parametrize("io,D", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_forward(io, D, lens, gate):
    i = case(io, D, gate, lens)
    o, ht = gdn.gdn_chunk_fwd(d(i["q"]), d(i["k"]), d(i["v"]), d(i["g"]), d(i["beta"]), scale=i["scale"], h0=d(i["h0"]),
                              cu_seqlens=d(i["cu"]))
    torch.cuda.synchronize()
    ro, rt = oracle.gdn_recurrent(i["q"], i["k"], i["v"], i["g"], i["beta"], i["scale"], h0=i["h0"], cu_seqlens=i["cu"])
    check("o", o.cpu(), ro, io)
    check("ht", ht.cpu(), rt, io, stored=F32)


@pytest.mark.parametrize("io", [BF, F32])
def test_every_token_resets(io):
    i = make(8, 1, 130, 1, 2, 64, io)
    i["g"].fill_(float("-inf"))
    out, ref = run(i), want(i)
    torch.cuda.synchronize()
    # dg is 0: the difference of three sums a token over 64 channels (70 u of their sizes each, all of the size of
    # q . dq here), added up over 64 tokens at most
    size = (i["q"].double().abs().numpy() * abs(ref[0])).sum(-1).max()
    assert abs(out[3].cpu().double()).max() <= 64 * 3 * 70 * 2.0 ** -24 * size
    for n in (0, 1, 2, 4):
        check(NAMES[n], out[n].cpu(), ref[n], io, stored=io)
    assert not out[5].any()


@pytest.mark.parametrize("io", [BF, F32])
def test_a_decay_that_keeps_nothing(io):
    i = make(9, 1, 130, 1, 2, 64, io, gate="gamma")
    i["gamma"][1] = float("-inf")
    compare(i, run(i))


def test_nan_gates_still_show():
    i = make(10, 1, 130, 1, 2, 64)
    i["g"][0, 70, 1] = float("nan")
    out = run(i)
    torch.cuda.synchronize()
    assert out[2][0, 70:, 1].isnan().any() and not out[2][0, :, 0].isnan().any()
