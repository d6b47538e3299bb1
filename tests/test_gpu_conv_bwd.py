"""GPU tests of the causal convolution's gradients against the fp64 oracle, with
bounds from a running error analysis of the fp32 computation (running_error.py)
plus the storage rounding."""

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
import oracle
from tests import running_error as re
from tests.mixer_cases import BF, DEV, close, d, edges, f64, randn

pytestmark = pytest.mark.gpu
F32 = torch.float32


def case(seed, lens, sections, W=4, io=BF, act=True, norm=0, norms=2, bias=True, extra=0, B=None, tail=0, scale=1.0):
    """lens: packed sequences, or with B the length of B dense ones."""
    D = sum(sections)
    T = lens if B else sum(lens) + tail
    x = randn(seed, B or 1, T, D + extra, dtype=io, scale=scale)
    w, b = randn(seed + 1, D, W, dtype=io, scale=0.5), randn(seed + 2, D, dtype=io) if bias else None
    dy = [randn(seed + 3 + n, B or 1, T, s, dtype=io) for n, s in enumerate(sections)]
    cu = None if B else torch.tensor(edges(lens), dtype=torch.int64)
    got = gdn.causal_conv_bwd(tuple(d(t) for t in dy), d(x)[..., :D], d(w), d(b), activation="silu" if act else None,
                              sections=sections, norm_dim=norm, norm_sections=norms if norm else 0,
                              cu_seqlens=d(cu))
    torch.cuda.synchronize()
    spans = [(i, 0, T) for i in range(B)] if B else [(0, a, e) for a, e in zip(edges(lens)[:-1], edges(lens)[1:])]
    xs, dys, ws, bs = f64(x[..., :D]), f64(torch.cat(dy, -1)), f64(w), None if b is None else f64(b)
    nc = sum(sections[:norms]) if norm else 0
    dw, db, ew, eb = np.zeros((D, W)), np.zeros(D), np.zeros((D, W)), np.zeros(D)
    step = 2.0 ** -8 if io == BF else re.U
    size_w, size_b = np.zeros((D, W)), np.zeros(D)
    for n, lo, hi in spans:
        args = (dys[n, lo:hi], xs[n, lo:hi], ws, bs, act, norm, nc, 1e-6)
        ref, bar = oracle.causal_conv_bwd(*args), re.causal_conv_bwd(*args)
        close(f"dx[{lo}:{hi}]", f64(got[0])[n, lo:hi], ref[0], bar[0].round_to(step).e)
        dw, db, ew, eb = dw + ref[1], db + ref[2], ew + bar[1].e, eb + bar[2].e
        size_w, size_b = size_w + np.abs(ref[1]), size_b + np.abs(ref[2])
    # the sequences' sums added up: one more rounding each
    ew, eb = ew + 2 * len(spans) * re.U * size_w, eb + 2 * len(spans) * re.U * size_b
    close("dweight", f64(got[1]), dw, re.E(dw, ew).round_to(step).e)
    if bias:
        close("dbias", f64(got[2]), db, re.E(db, eb).round_to(step).e)
    else:
        assert got[2] is None


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("act,norm", [(True, 0), (True, 64), (False, 128), (False, 0)])
def test_packed_lengths(W, io, act, norm):
    # shorter than the taps, empty, across runs, longer than a run
    case(W, [1, 0, 2, 3, 9, 0, 0, 41, 5, 130], (128, 128, 256), W, io, act, norm)


@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (2, 2), (4, 8), (3, 17), (1, 200)])
def test_dense(B, T):
    case(T, T, (64, 64), 4, BF, True, 64, B=B)


@pytest.mark.parametrize("sections", [(8,), (520,), (16, 504), (512, 512, 8), (136, 24, 1032)])
def test_widths(sections):
    case(7, [5, 12], sections, 3, F32, bias=False)


def test_rows_of_a_wider_projection_and_all_sections_normalised():
    case(8, [30, 3], (64, 128, 64), 4, BF, norm=64, norms=3, extra=40)


def test_long_runs():
    case(9, [3000, 1, 2222], (512, 512, 512), 4, BF, norm=128)


def test_rows_behind_the_last_boundary_are_left():
    D, T = 64, 40
    x, w, dy = d(randn(1, 1, T, D, dtype=BF)), d(randn(2, D, 4, dtype=BF)), d(randn(3, 1, T, D, dtype=BF))
    cu = torch.tensor([0, 10, 25], device=DEV)
    x[:, 25:] = float("nan")
    dy[:, 25:] = float("nan")
    L = gdn.lib()
    dx = torch.full((1, T, D), 7.0, dtype=BF, device=DEV)
    dw = torch.empty(D, 4, dtype=BF, device=DEV)
    ws = torch.empty(L.gdn_conv_bwd_workspace_bytes(1, T, D, 4), dtype=torch.uint8, device=DEV)
    st = L.gdn_conv_bwd(dy.data_ptr(), None, None, D, 0, 0, x.data_ptr(), T * D, D, w.data_ptr(), None, 1, 0, 0, 0.0,
                        cu.data_ptr(), 2, 1, T, D, 4, 1, dx.data_ptr(), dw.data_ptr(), None, ws.data_ptr(), ws.numel(),
                        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want = gdn.causal_conv_bwd(dy[:, :25].contiguous(), x[:, :25].contiguous(), w, cu_seqlens=cu)
    assert torch.equal(dx[:, :25], want[0]) and (dx[:, 25:] == 7).all()
    assert torch.isfinite(dw.float()).all()
    close("dweight", f64(dw), f64(want[1]), 2.0 ** -7 * np.abs(f64(want[1])) + 1e-4)


def test_heads_whose_squares_leave_fp32():
    # u = c without an activation: gradients of n = u / |u| shrink as 1 / |u|
    D = 64
    x = torch.zeros(1, 2, D)
    x[0, 0, :] = 1e25
    w = torch.zeros(D, 2)
    w[:, 1] = 1
    dy = randn(4, 1, 2, D)
    dx, _, _ = gdn.causal_conv_bwd((d(dy),), d(x), d(w), activation=None, sections=(D,), norm_dim=64, norm_sections=1)
    ref = oracle.causal_conv_bwd(dy[0], x[0], w, None, False, 64, D, 1e-6)[0]
    close("dx", f64(dx)[0], ref, 2.0 ** -18 * np.abs(f64(dy))[0].max() * np.array([[1e-24], [1e3]]))


def test_no_tokens_and_no_sequences():
    x, w = torch.empty(1, 0, 64, dtype=BF, device=DEV), torch.ones(64, 4, dtype=BF, device=DEV)
    dx, dw, db = gdn.causal_conv_bwd(x, x, w, w[:, 0].contiguous())
    assert dx.shape == x.shape and not dw.any() and not db.any()
    x = torch.ones(1, 5, 64, dtype=BF, device=DEV)
    _, dw, _ = gdn.causal_conv_bwd(x, x, w, cu_seqlens=torch.zeros(1, dtype=torch.int64, device=DEV))
    assert not dw.any()


def test_same_bits_in_every_run_captured_and_on_another_stream():
    x, w, dy = d(randn(1, 1, 700, 256, dtype=BF)), d(randn(2, 256, 4, dtype=BF)), d(randn(3, 1, 700, 256, dtype=BF))
    cu = torch.tensor([0, 10, 10, 655, 700], device=DEV)
    run = lambda: gdn.causal_conv_bwd(dy, x, w, cu_seqlens=cu)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    side = torch.cuda.Stream()
    for seed in (5, 6, 7):
        x.copy_(d(randn(seed, 1, 700, 256, dtype=BF)))
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = run()
        side.synchronize()
        for a, b, c in zip(out[:2], want[:2], other[:2]):
            assert torch.equal(a, b) and torch.equal(b, c)
