"""GPU tests of the group norm and its gradients against the fp64 oracle, with
bounds from a running error analysis of the fp32 computation (running_error.py)
plus the storage rounding; and of strides, streams, graphs and untouched memory."""

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
import oracle
from tests import running_error as re
from tests.mixer_cases import BF, DEV, close, d, f64, randn

pytestmark = pytest.mark.gpu
F32 = torch.float32
STEP = {BF: 2.0 ** -8, F32: re.U}


def flat(t):
    return None if t is None else f64(t).reshape(-1, t.shape[-1])


def make(seed, B, T, G, D, io=BF, wdt=F32, shared=True, gated=True, bias=True):
    C = G * D
    n = D if shared else C
    return dict(x=randn(seed, B, T, C, dtype=io), z=randn(seed + 1, B, T, C, dtype=io) if gated else None,
                w=(1 + randn(seed + 2, n, scale=0.3)).to(wdt), b=randn(seed + 3, n, dtype=wdt) if bias else None,
                dy=randn(seed + 4, B, T, C, dtype=io))


def check(i, G, act, rms, eps=1e-5, wide=0):
    put = lambda t: None if t is None else d(t)  # noqa: E731
    if wide:   # x, z and dout as slices of wider rows
        def put(t):
            if t is None or t.dim() < 3:
                return None if t is None else d(t)
            room = torch.full((*t.shape[:-1], t.shape[-1] + wide), float("nan"), dtype=t.dtype, device=DEV)
            room[..., 8: 8 + t.shape[-1]] = d(t)
            return room[..., 8: 8 + t.shape[-1]]
    x, z, w, b, dy = (put(i[n]) for n in ("x", "z", "w", "b", "dy"))
    y = gdn.group_norm_fwd(x, G, w, b, z=z, activation=act, rms=rms, eps=eps)
    out = gdn.group_norm_bwd(dy, x, G, w, b, z=z, activation=act, rms=rms, eps=eps)
    torch.cuda.synchronize()
    o = [flat(i["x"]), G, None if w is None else f64(i["w"]), None if b is None else f64(i["b"]), flat(i["z"])]
    step = STEP[i["x"].dtype]
    bar = re.group_norm(*o, act, rms, eps).round_to(step)
    close("y", flat(y), oracle.group_norm(*o, act, rms, eps), bar.e)
    bars = re.group_norm(*o, act, rms, eps, dout=flat(i["dy"]))
    want = oracle.group_norm(*o, act, rms, eps, dout=flat(i["dy"]))
    for name, got, ref, e, given in zip(("dx", "dz", "dweight", "dbias"), out, want, bars, (x, z, w, b)):
        if given is None:
            assert got is None
            continue
        assert got.dtype == given.dtype and got.shape == given.shape
        close(name, f64(got).reshape(ref.shape), ref, e.round_to(STEP[got.dtype]).e)


@pytest.mark.parametrize("G,D", [(1, 8), (3, 24), (5, 40), (2, 64), (7, 72), (16, 128), (3, 200), (2, 512), (2, 520),
                                 (1, 1024), (2, 1032), (1, 2048), (1, 4096), (1, 8192)])
@pytest.mark.parametrize("io", [BF, F32])
def test_group_sizes(G, D, io):
    check(make(D, 2, 5, G, D, io, shared=D % 16 == 0), G, "silu", D % 24 == 0)


@pytest.mark.parametrize("act", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_forms(act, gated, rms, shared):
    check(make(3, 1, 9, 4, 64, gated=gated, shared=shared, wdt=BF), 4, act, rms)


@pytest.mark.parametrize("B,T", [(1, 1), (1, 2), (2, 1), (3, 7), (1, 333), (2, 1500)])
def test_token_counts(B, T):
    check(make(T, B, T, 2, 64, bias=False), 2, "silu", True)
    check(make(T + 1, B, T, 3, 40, F32, shared=False, gated=False), 3, "silu", False)


def test_many_walks_and_wide_groups_share_weights():
    # more tokens than walks run side by side, groups of a work-group each
    check(make(5, 1, 700, 2, 1536, shared=True), 2, "silu", False)


@pytest.mark.parametrize("io", [BF, F32])
def test_slices_of_wider_rows(io):
    check(make(8, 2, 6, 4, 64, io), 4, "silu", True, wide=24)


def test_without_weights():
    i = make(9, 1, 6, 4, 64, bias=False)
    i["w"] = None
    check(i, 4, "sigmoid", False)
    i = make(10, 1, 6, 4, 64)
    i["w"] = None
    check(i, 4, "silu", True)


def test_constant_and_zero_groups_and_large_values():
    i = make(11, 1, 6, 4, 64, F32)
    i["x"][0, 0] = 0
    i["x"][0, 1] = 3.0
    check(i, 4, "silu", False)
    x = torch.ones(1, 3, 128, device=DEV)
    x[0, 0, ::2] = -1
    x[0, 0] *= 3e30          # squares past fp32's largest number
    x[0, 1] *= 1e-30         # squares below its smallest
    y = gdn.group_norm_fwd(x, 2, activation=None, rms=True, eps=0.0)
    close("y", f64(y), np.sign(f64(x)), np.full(y.shape, 2.0 ** -21))
    y = gdn.group_norm_fwd(x[:, :1].contiguous(), 2, activation=None, rms=False, eps=0.0)
    close("y", f64(y), np.sign(f64(x[:, :1])), np.full(y.shape, 2.0 ** -20))


def test_infinities_and_nan_stay_in_their_group():
    i = make(12, 1, 4, 4, 64, F32)
    clean = gdn.group_norm_fwd(d(i["x"]), 4, d(i["w"]), d(i["b"]), z=d(i["z"]))
    i["x"][0, 1, 70] = float("nan")
    i["x"][0, 2, 140] = float("inf")
    y = gdn.group_norm_fwd(d(i["x"]), 4, d(i["w"]), d(i["b"]), z=d(i["z"])).cpu()
    assert y[0, 1, 64:128].isnan().all() and y[0, 2, 128:192].isnan().all()
    hit = torch.zeros(1, 4, 256, dtype=torch.bool)
    hit[0, 1, 64:128] = hit[0, 2, 128:192] = True
    assert torch.equal(y[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("shared", [False, True])
def test_no_tokens(shared):
    x = torch.empty(2, 0, 128, dtype=BF, device=DEV)
    w = torch.ones(64 if shared else 128, device=DEV)
    assert gdn.group_norm_fwd(x, 2, w).shape == x.shape
    dx, dz, dw, db = gdn.group_norm_bwd(x, x, 2, w, w, z=x)
    assert dx.shape == dz.shape == x.shape and not dw.any() and not db.any()


def test_same_bits_in_every_run_and_on_another_stream():
    i = {n: d(t) for n, t in make(13, 2, 900, 16, 128).items()}
    first = gdn.group_norm_bwd(i["dy"], i["x"], 16, i["w"], i["b"], z=i["z"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = gdn.group_norm_bwd(i["dy"], i["x"], 16, i["w"], i["b"], z=i["z"])
    side.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_captured_with_a_workspace_of_its_own():
    i = {n: d(t) for n, t in make(14, 1, 300, 4, 128).items()}
    need = gdn.lib().gdn_group_norm_bwd_workspace_bytes(1, 300, 4, 128, 1)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    run = lambda w: gdn.group_norm_bwd(i["dy"], i["x"], 4, i["w"], i["b"], z=i["z"], workspace=w)  # noqa: E731
    run(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(ws)
    for seed in (1, 2, 3):
        i["x"].copy_(d(randn(seed, 1, 300, 512, dtype=BF)))
        i["dy"].copy_(d(randn(seed + 9, 1, 300, 512, dtype=BF)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, run(None)):
            assert torch.equal(a, b)
