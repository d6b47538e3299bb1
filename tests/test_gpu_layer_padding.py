"""GPU tests of packed batches with rows behind the last sequence (a batch padded to a
fixed number of tokens): the gradients of these rows are zeros, from the binding always
and from the library where asked for, whatever the memory held, and those of the
sequences are what they are without the padding."""

import pytest
import torch

import gated_delta_rule_61_amd as gdn
from gated_delta_rule_61_amd import binding
from tests.mixer_cases import BF, DEV, d, edges, randn
from tests.test_gpu_chunk_bwd import F32, make, run
from tests.test_gpu_varlen_bounds import CU, N, SENT_BYTE, T, _guarded, _guards_ok

pytestmark = pytest.mark.gpu
NAN = float("nan")


def poison(shapes):
    """Leaves memory of these tensors' sizes behind that holds NaN."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for t in [torch.full(s, NAN, dtype=dt, device=DEV) for s, dt in shapes]:
        del t
    torch.cuda.synchronize()


@pytest.mark.parametrize("lens,T", [([70, 0, 33], 104), ([64, 64], 129), ([5], 700), ([0, 0], 65), ([1] * 20, 84),
                                    ([63] * 9 + [1], 1000), ([], 130)])
@pytest.mark.parametrize("io,Hk,HV,D", [(BF, 2, 4, 128), (F32, 1, 3, 64), (BF, 1, 1, 64), (F32, 2, 2, 128)])
def test_delta_rule(lens, T, io, Hk, HV, D):
    i = make(T + D, 1, T, Hk, HV, D, io, lens=lens or [T])
    end = sum(lens)
    if not lens:
        i.update(h0=None, dht=None)
    i["cu"] = torch.tensor(edges(lens), dtype=torch.int64)
    for n in ("q", "k", "v", "g", "beta", "dout"):   # what the padding holds reaches nothing
        i[n] = i[n].clone()
        i[n][:, end:] = NAN
    poison([((1, T, Hk, D), io), ((1, T, Hk, D), io), ((1, T, HV, D), io), ((1, T, HV), io), ((1, T, HV), io)])
    out = run(i)
    torch.cuda.synchronize()
    for t in out[:5]:
        assert not bool(t[:, end:].any()) and bool(t[:, :end].isfinite().all())
    if end:
        j = {n: t[:, :end].contiguous() if n in ("q", "k", "v", "g", "beta", "dout") else t for n, t in i.items()}
        for a, b in zip(out, run(j)):
            assert torch.equal(a[:, :end] if a.dim() < 4 or a.shape[1] == T else a, b)


def test_delta_rule_fixed_decay_with_its_gradient():
    i = make(3, 1, 200, 1, 2, 64, lens=[150], gate="gamma")
    poison([((1, 200, 2, 64), BF), ((1, 200, 2), BF), ((1, 200, 2), BF)])
    assert not bool(run(i, output_dg=True)[3][:, 150:].any())


@pytest.mark.parametrize("lens,T", [([70, 0, 33], 104), ([5], 700), ([0, 0], 65), ([], 9), ([900], 16001)])
@pytest.mark.parametrize("io,W", [(BF, 4), (F32, 3)])
@pytest.mark.parametrize("D", [64, 1032])
def test_convolution(lens, T, io, W, D):
    x, dy, w = d(randn(1, 1, T, D, dtype=io)), d(randn(2, 1, T, D, dtype=io)), d(randn(3, D, W, dtype=io))
    end = sum(lens)
    cu = torch.tensor(edges(lens), dtype=torch.int64, device=DEV)
    x[:, end:] = NAN
    dy[:, end:] = NAN
    poison([((1, T, D), io)])
    dx, dw, _ = gdn.causal_conv_bwd(dy, x, w, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert not bool(dx[:, end:].any()) and bool(dx.isfinite().all()) and bool(dw.isfinite().all())
    if end:
        want = gdn.causal_conv_bwd(dy[:, :end].contiguous(), x[:, :end].contiguous(), w, cu_seqlens=cu)
        assert torch.equal(dx[:, :end], want[0])


def test_captured_with_an_end_that_moves():
    i = make(5, 1, 300, 1, 2, 128, lens=[100, 60])
    g = {n: d(t) if isinstance(t, torch.Tensor) else t for n, t in i.items()}
    x, w = d(randn(1, 1, 300, 128, dtype=BF)), d(randn(2, 128, 4, dtype=BF))
    call = lambda: (*gdn.gdn_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["beta"], g["dout"], g["dht"],  # noqa: E731
                                       h0=g["h0"], cu_seqlens=g["cu"])[:5], gdn.causal_conv_bwd(x, x, w, cu_seqlens=g["cu"])[0])
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for cu in ([0, 10, 20], [0, 0, 300], [0, 64, 128], [0, 0, 0]):
        g["cu"].copy_(torch.tensor(cu))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, call()):
            assert torch.equal(a, b) and not bool(a[:, cu[2]:].any())
        torch.cuda.synchronize()


@pytest.mark.parametrize("io", [BF, F32])
def test_invalid_boundaries_stay_inside_the_buffers(io):
    print(f"zeros behind invalid boundaries, {io}", flush=True)
    hk, hv, D = 1, 2, 64
    q, k, v, do = (d(randn(s, 1, T, h, D, dtype=io, scale=0.1)) for s, h in ((1, hk), (2, hk), (3, hv), (4, hv)))
    g, beta = -d(randn(5, 1, T, hv)).abs() * 0.2, d(randn(6, 1, T, hv)).sigmoid()
    L, code = binding.lib(), (1 if io == BF else 0) | binding.GDN_ROWS_ZERO
    need = L.gdn_chunk_bwd_workspace_bytes(1, T, hk, hv, D, D, N, 1, code)
    assert need == binding.chunk_bwd_workspace_bytes(1, T, hk, hv, D, D, N, io, varlen=True)
    stream = torch.cuda.current_stream().cuda_stream
    for cu in (CU, CU[:-1] + [-5], CU[:-1] + [T - 1], [T] * (N + 1), [0] * (N + 1)):
        out = [_guarded(s, io) for s in ((1, T, hk, D), (1, T, hk, D), (1, T, hv, D), (1, T, hv), (1, T, hv), (1, T, 640),
                                         (640, 4))]
        ws = _guarded((need,), torch.uint8, SENT_BYTE)
        edge = torch.tensor(cu, dtype=torch.int64, device=DEV)
        assert L.gdn_chunk_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), None, beta.data_ptr(), D ** -0.5,
                               None, do.data_ptr(), None, edge.data_ptr(), N, 1, T, hk, hv, D, D, 64, code,
                               *(t.data_ptr() for _, t in out[:5]), None, ws[1].data_ptr(), need, stream) == 0
        x, w = d(randn(7, 1, T, 640, dtype=io)), d(randn(8, 640, 4, dtype=io))
        cneed = L.gdn_conv_bwd_workspace_bytes(1, T, 640, 4)
        cws = _guarded((cneed,), torch.uint8, SENT_BYTE)
        assert L.gdn_conv_bwd(x.data_ptr(), None, None, 640, 0, 0, x.data_ptr(), T * 640, 640, w.data_ptr(), None, 1, 0, 0,
                              0.0, edge.data_ptr(), N, 1, T, 640, 4, code, out[5][1].data_ptr(), out[6][1].data_ptr(),
                              None, cws[1].data_ptr(), cneed, stream) == 0
        torch.cuda.synchronize()
        assert all(_guards_ok(b) for b, _ in out) and _guards_ok(ws[0], SENT_BYTE) and _guards_ok(cws[0], SENT_BYTE)
        if not any(cu):   # valid, and everything is behind
            assert not any(bool(t.any()) for _, t in out)
