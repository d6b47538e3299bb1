"""GPU tests of the log-gates' gradient where the gate is a head's fixed decay, or
there is none: against the fp64 oracle at the bars of test_gpu_chunk_bwd, summed over
the tokens against the decay's, and against differences of the forward."""

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
from tests.mixer_cases import BF, d
from tests.test_gpu_chunk_bwd import F32, make, run, want
from tests.tolerance import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", ["gamma", "none"])
@pytest.mark.parametrize("lens,B,T", [(None, 2, 100), ([70, 0, 33, 1, 64], 1, 168)])
@pytest.mark.parametrize("Hk,HV,D", [(1, 1, 64), (2, 4, 128), (1, 3, 64)])
@pytest.mark.parametrize("io", [BF, F32])
def test_every_token(io, Hk, HV, D, lens, B, T, gate):
    i = make(T + HV, B, T, Hk, HV, D, io, lens=lens, gate=gate)
    out, ref = run(i, output_dg=True), want(i)
    torch.cuda.synchronize()
    assert out[3].shape == (B, T, HV) and out[3].dtype == io
    check("dg", out[3].cpu(), ref[3], io, stored=io)
    # the same bits as without it, and as with the decay given token by token
    plain = run(i)
    assert plain[3] is None
    for a, b in zip(out[:3] + out[4:], plain[:3] + plain[4:]):
        assert torch.equal(a, b)
    g = (torch.zeros(B, T, HV) if gate == "none" else i["gamma"].expand(B, T, HV)).contiguous()
    for a, b in zip(out, run(dict(i, g=g, gamma=None))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("io", [BF, F32])
def test_sum_over_the_tokens_is_the_decays(io):
    """A long decay.  Every token's is off by its bar, 2e-2 of the RMS and half a bf16 step (fp32: 1e-4), and so the
    sum by the sum of these at most."""
    i = make(3, 2, 1000, 2, 4, 64, io, gate="gamma")
    dg = run(i, output_dg=True)[3].cpu().double().numpy()
    ref = want(i)[3]
    bar = 2e-2 * np.sqrt((ref * ref).mean()) + 2.0 ** -8 * np.abs(ref) if io == BF else np.full(ref.shape, 1e-4)
    assert np.all(np.abs(dg.sum((0, 1)) - ref.sum((0, 1))) <= bar.sum((0, 1)))


def test_matches_differences_of_the_forward():
    # as in test_gpu_chunk_bwd the forward's error is 1e-4 of a loss of order ten, 2e-2 over a difference of 6e-3; a
    # state lasts ten tokens, so that the third derivative is a thousand times the loss: 3e-3^2 / 6 x 1e4 = 2e-2
    i = make(8, 1, 80, 1, 2, 64, F32, gate="gamma")
    dg = run(i, output_dg=True)[3].cpu().double().sum((0, 1))

    def loss(gamma):
        o, ht = gdn.gdn_chunk_fwd(d(i["q"]), d(i["k"]), d(i["v"]), None, d(i["beta"]), scale=i["scale"], h0=d(i["h0"]),
                                  g_gamma=d(gamma))
        return ((o.cpu().double() * i["dout"].double()).sum() + (ht.cpu().double() * i["dht"].double()).sum()).item()

    for h in range(2):
        step = torch.zeros(2)
        step[h] = 3e-3
        slope = (loss(i["gamma"] + step) - loss(i["gamma"] - step)) / 6e-3
        assert abs(slope - dg[h].item()) < 5e-2, (h, slope, dg[h].item())


def test_can_be_left_out():
    i = make(9, 1, 70, 1, 2, 64)
    out = run(i, output_dg=False)
    assert out[3] is None
    for a, b in zip(out[:3] + out[4:], [t for n, t in enumerate(run(i)) if n != 3]):
        assert torch.equal(a, b)
