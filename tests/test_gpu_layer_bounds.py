"""GPU tests of what the gradients of packed sequences write: nothing behind the
last boundary, and with invalid boundaries (below 0, past T, backwards,
overlapping, more chunks than rows of the tables) nothing outside the caller's
buffers; an empty sequence's initial state gets its final state's gradient.
Other results of such calls are unspecified."""

import pytest
import torch

from gated_delta_rule_61_amd import binding
from tests.mixer_cases import BF, DEV, d, randn
from tests.test_gpu_varlen_bounds import CU, EMPTY, HK, HV, K, N, SENT, SENT_BYTE, T, _guarded, _guards_ok

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _delta(io, cu):
    """All outputs and the workspace between guards; returns (buffers, views, dht)."""
    n = len(cu) - 1
    D = K if io == F32 else 128
    q, k = (d(torch.nn.functional.normalize(randn(s, 1, T, HK, D), dim=-1).to(io)) for s in (1, 2))
    v, do = d(randn(3, 1, T, HV, D, dtype=io)), d(randn(4, 1, T, HV, D, dtype=io))
    g, beta = -d(randn(5, 1, T, HV)).abs() * 0.2, d(randn(6, 1, T, HV)).sigmoid()
    h0, dht = d(randn(7, n, HV, D, D)), d(randn(8, n, HV, D, D))
    out = [_guarded(s, io) for s in ((1, T, HK, D), (1, T, HK, D), (1, T, HV, D), (1, T, HV), (1, T, HV), (n, HV, D, D))]
    need = binding.chunk_bwd_workspace_bytes(1, T, HK, HV, D, D, n, io, varlen=True)
    ws = _guarded((need,), torch.uint8, SENT_BYTE)
    edges = torch.tensor(cu, dtype=torch.int64, device=DEV)
    status = binding.lib().gdn_chunk_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), None, beta.data_ptr(), D ** -0.5, h0.data_ptr(),
        do.data_ptr(), dht.data_ptr(), edges.data_ptr(), n, 1, T, HK, HV, D, D, 64, 1 if io == BF else 0,
        *(t.data_ptr() for _, t in out), ws[1].data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0
    assert all(_guards_ok(b) for b, _ in out) and _guards_ok(ws[0], SENT_BYTE)
    return [t for _, t in out], dht


@pytest.mark.parametrize("io", [BF, F32])
def test_delta_rule_invalid_boundaries(io):
    print(f"chunk gradients, invalid boundaries, {io}", flush=True)
    out, dht = _delta(io, CU)
    for n in EMPTY:
        assert torch.equal(out[5][n], dht[n].to(io))


@pytest.mark.parametrize("io", [BF, F32])
def test_delta_rule_rows_behind_the_last_boundary(io):
    print(f"chunk gradients, rows behind, {io}", flush=True)
    out, _ = _delta(io, [0, 70, 70, 150])
    for t in out[:5]:
        assert bool((t[:, 150:] == SENT).all()) and bool(t[:, :150].isfinite().all())
        assert not bool((t[:, :150] == SENT).all(-1).any()) if t.dim() == 4 else True


@pytest.mark.parametrize("io", [BF, F32])
def test_convolution_invalid_boundaries(io):
    print(f"convolution's gradients, invalid boundaries, {io}", flush=True)
    D, W = 640, 4
    x, dy, w = d(randn(11, 1, T, D, dtype=io)), d(randn(12, 1, T, D, dtype=io)), d(randn(13, D, W, dtype=io))
    out = [_guarded(s, io) for s in ((1, T, D), (D, W))]
    L = binding.lib()
    need = L.gdn_conv_bwd_workspace_bytes(1, T, D, W)
    ws = _guarded((need,), torch.uint8, SENT_BYTE)
    edges = torch.tensor(CU, dtype=torch.int64, device=DEV)
    status = L.gdn_conv_bwd(dy.data_ptr(), None, None, D, 0, 0, x.data_ptr(), T * D, D, w.data_ptr(), None, 1, 0, 0, 1e-6,
                            edges.data_ptr(), N, 1, T, D, W, 1 if io == BF else 0, out[0][1].data_ptr(),
                            out[1][1].data_ptr(), None, ws[1].data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0
    assert all(_guards_ok(b) for b, _ in out) and _guards_ok(ws[0], SENT_BYTE)


def test_an_infinite_value_stays_in_its_sequence_and_key_head():
    print("chunk gradients, an infinite value", flush=True)
    D, lens = 128, [0, 100, 200]
    i = [d(randn(s, 1, 200, h, D, dtype=BF, scale=0.1)) for s, h in ((21, 2), (22, 2), (23, 4), (24, 4))]
    g, beta = -d(randn(25, 1, 200, 4)).abs() * 0.2, d(randn(26, 1, 200, 4)).sigmoid()
    run = lambda: binding.gdn_chunk_bwd(*i[:3], g, beta, i[3], cu_seqlens=torch.tensor(lens, device=DEV))  # noqa: E731
    clean = run()
    i[2][0, 30, 1, 5] = float("inf")
    out = run()
    torch.cuda.synchronize()
    assert not bool(out[0][0, :100, 0].isfinite().all())
    for a, b, heads in zip(clean[:5], out[:5], (1, 1, 2, 2, 2)):
        assert torch.equal(a[:, 100:], b[:, 100:]) and torch.equal(a[:, :, heads:], b[:, :, heads:])
