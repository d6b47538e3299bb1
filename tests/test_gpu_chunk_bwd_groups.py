"""GPU tests of the delta rule's gradients where many v-heads share a key head and
their gradients differ in size: each head against the fp64 oracle at its own size,
with the bars of test_gpu_chunk_bwd (bf16 operands' scale is the largest head's, and
2^-8 of it is still 2^-14 + above fp16's smallest normal number; dg's sums are fp32,
2^-24 of the largest per addition)."""

import pytest
import torch

from tests.mixer_cases import BF
from tests.test_gpu_chunk_bwd import F32, NAMES, compare, make, run, want
from tests.tolerance import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hk,HV,D", [(1, 32, 64), (2, 32, 128), (1, 64, 64)])
@pytest.mark.parametrize("io", [BF, F32])
def test_many_heads_of_a_key_head(Hk, HV, D, io):
    # dq and dk are sums of HV / Hk heads: the square root of it brings them back to order one
    i = make(HV + D, 1, 130, Hk, HV, D, io, lens=[66, 64], size=(HV / Hk) ** -0.5)
    compare(i, run(i))


@pytest.mark.parametrize("first", [False, True])
def test_a_small_head_next_to_large_ones(first):
    i = make(7, 1, 100, 1, 4, 128)
    small = 0 if first else 3
    for n in ("dout", "dht"):
        i[n] = i[n].float()
        (i[n][:, small] if n == "dht" else i[n][:, :, small]).mul_(2.0 ** -8)
    i["dout"] = i["dout"].to(BF)
    out, ref = run(i), want(i)
    torch.cuda.synchronize()
    for name, got, r in zip(NAMES, out, ref):
        if name in ("dq", "dk"):
            check(name, got.cpu(), r, BF, stored=BF)
            continue
        at = (slice(None), small) if name == "dh0" else (slice(None), slice(None), small)
        check(name, got.cpu()[at], r[at], BF, stored=BF)
