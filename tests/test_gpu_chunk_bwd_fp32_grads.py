"""GPU tests of the delta rule's gradients of g, beta and h0 in fp32 beside bf16 io: the
numbers that the io dtype's are rounded from, at the prefill's bar without the storage
(tests/tolerance.py); and of a sequence in two segments, the second one's dh0 the first
one's dht."""

import pytest
import torch

import gated_delta_rule_61_amd as gdn
from tests.mixer_cases import BF, DEV, d
from tests.test_gpu_chunk_bwd import F32, NAMES, make, run, want
from tests.tolerance import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,B,T", [(None, 2, 100), ([70, 0, 33, 1, 64], 1, 180)])
@pytest.mark.parametrize("Hk,HV,D", [(1, 1, 64), (2, 4, 128), (1, 3, 64)])
@pytest.mark.parametrize("gate", ["g", "gamma"])
def test_what_the_io_dtypes_are_rounded_from(gate, Hk, HV, D, lens, B, T):
    i = make(T + HV, B, T, Hk, HV, D, lens=lens, gate=gate)
    end = T if lens is None else sum(lens)
    out, plain, ref = run(i, grads_in_fp32=True, output_dg=True), run(i, output_dg=True), want(i)
    torch.cuda.synchronize()
    for n in range(3):
        assert torch.equal(out[n], plain[n])
    for n in range(3, 6):
        assert out[n].dtype == F32 and torch.equal(out[n].to(BF), plain[n])
        cut = (lambda t: t) if n == 5 else lambda t: t[:, :end]
        check(NAMES[n], cut(out[n]).cpu(), cut(ref[n]), BF, stored=F32)
        if n < 5:
            assert not out[n][:, end:].any()


def test_fp32_io_has_them_anyway():
    i = make(4, 1, 90, 1, 2, 64, F32)
    for a, b in zip(run(i, grads_in_fp32=True), run(i)):
        assert a.dtype == F32 and torch.equal(a, b)


def test_two_segments():
    i = make(5, 1, 200, 2, 4, 128)
    cut = 128
    part = lambda a, b: {n: t[:, a:b].contiguous() if n in ("q", "k", "v", "g", "beta", "dout") else t  # noqa: E731
                         for n, t in i.items()}
    first, second = part(0, cut), part(cut, 200)
    _, ht = gdn.gdn_chunk_fwd(*(d(first[n]) for n in ("q", "k", "v", "g", "beta")), scale=i["scale"], h0=d(i["h0"]))
    back = run(dict(second, h0=ht), grads_in_fp32=True)
    front = run(dict(first, dht=back[5]), grads_in_fp32=True)
    torch.cuda.synchronize()
    ref = want(i)
    for n in range(5):
        got = torch.cat([front[n], back[n]], 1)
        check(NAMES[n], got.cpu(), ref[n], BF, stored=got.dtype)
    check("dh0", front[5].cpu(), ref[5], BF, stored=F32)


def test_captured():
    i = make(6, 1, 150, 1, 2, 64, lens=[60, 80])
    g = {n: d(t) if isinstance(t, torch.Tensor) else t for n, t in i.items()}
    call = lambda: gdn.gdn_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["beta"], g["dout"], g["dht"], h0=g["h0"],  # noqa: E731
                                     cu_seqlens=g["cu"], grads_in_fp32=True)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in (1, 2, 3):
        g["dout"].copy_(torch.randn(g["dout"].shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, call()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
