"""GPU tests of the gradients of sequences of some dozen chunks, with a gate and without
any decay (where the roundings of a state and its gradient stay until an erase), against
the fp64 oracle.  Bars of tests/tolerance.py: a rounding to fp16, 2^-11 / sqrt(3) of the
RMS of what is rounded, is made of every chunk's share of a state and its gradient; over
n chunks these add up in squares as the shares do, so that the error of a sum keeps its
ratio to the sum, and the bound of single chunks holds."""

import pytest
import torch

from tests.mixer_cases import BF
from tests.test_gpu_chunk_bwd import F32, NAMES, make, run, want
from tests.tolerance import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", ["g", "gamma", "none"])
@pytest.mark.parametrize("lens", [[1500], [640, 0, 861]])
@pytest.mark.parametrize("io,D,Hk,HV", [(BF, 128, 1, 2), (BF, 64, 1, 1), (F32, 64, 1, 1)])
def test_some_dozen_chunks(io, D, Hk, HV, lens, gate):
    # fp32's bar is absolute: gradients of a tenth keep those without decay at order one
    i = make(sum(lens) + D, 1, sum(lens), Hk, HV, D, io, lens=lens, gate=gate, size=0.1)
    out, ref = run(i, output_dg=True, grads_in_fp32=True), want(i)
    torch.cuda.synchronize()
    for name, got, r in zip(NAMES, out, ref):
        check(name, got.cpu(), r, io, stored=got.dtype)
