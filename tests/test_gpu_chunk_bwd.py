"""GPU tests of the gated delta rule's gradients against the fp64 oracle (the
token-by-token adjoint), at the parity bar of the forward (tests/tolerance.py):
bf16 io, per element 2e-2 of the RMS plus half a bf16 step, and 2e-2 of the RMS
over all; fp32 io, 1e-4 (dout and dht are drawn so that gradients are of order
one).  The bar holds for bf16 io because every operand of a product is rounded
once to fp16 (2^-11 of its size, so 2^-11 / sqrt(3) of the RMS of a sum of them)
and a gradient passes at most five such products from the inputs, plus those of
the states and state gradients, whose roundings a decay or the erase term wears
off: 5e-3 at most, where a sum's terms do not cancel below a quarter."""

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
import oracle
from gated_delta_rule_61_amd import binding, workloads
from tests.mixer_cases import BF, DEV, d, edges, randn
from tests.tolerance import check

pytestmark = pytest.mark.gpu
F32 = torch.float32
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


def make(seed, B, T, Hk, HV, D, io=BF, lens=None, gate="g", h0=True, dht=True, size=1.0):
    inp = workloads.make_prefill(B, T, Hk, HV, D, D, dtype=io, seed=seed, h0=h0)
    N = B if lens is None else len(lens)
    i = dict(q=inp.q, k=inp.k, v=inp.v, beta=inp.beta, g=inp.g if gate == "g" else None,
             gamma=-torch.rand(HV, generator=torch.Generator().manual_seed(seed)) * 0.2 if gate == "gamma" else None,
             dout=randn(seed + 1, B, T, HV, D, dtype=io, scale=size), scale=D ** -0.5,
             h0=randn(seed + 2, N, HV, D, D, scale=0.3) if h0 else None,
             dht=randn(seed + 3, N, HV, D, D, scale=0.3 * size) if dht else None,
             cu=None if lens is None else torch.tensor(edges(lens), dtype=torch.int64))
    return i


def run(i, **kw):
    g = {n: d(t) if isinstance(t, torch.Tensor) else t for n, t in i.items()}
    return gdn.gdn_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["beta"], g["dout"], g["dht"], scale=i["scale"],
                             h0=g["h0"], cu_seqlens=g["cu"], g_gamma=g["gamma"], **kw)


def want(i):
    return oracle.gdn_recurrent_bwd(i["q"], i["k"], i["v"], i["g"], i["beta"], i["dout"], i["scale"], i["h0"], i["dht"],
                                    i["cu"], i["gamma"])


def compare(i, out, size=1.0):
    torch.cuda.synchronize()
    io = i["q"].dtype
    for name, got, ref in zip(NAMES, out, want(i)):
        given = {"dg": i["g"], "dh0": i["h0"]}.get(name, i["q"])
        if given is None:
            assert got is None, name
            continue
        assert got.dtype == io, name
        check(name, got.cpu().float() / size, ref / size, io, stored=io)


@pytest.mark.parametrize("T", [1, 2, 17, 63, 64, 65, 130])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("io", [BF, F32])
def test_lengths(T, D, io):
    i = make(T, 1, T, 2, 2, D, io)
    compare(i, run(i))


@pytest.mark.parametrize("Hk,HV", [(1, 1), (1, 3), (2, 4), (3, 3)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("io", [BF, F32])
def test_heads(Hk, HV, D, io):
    i = make(Hk + 10 * HV, 2, 70, Hk, HV, D, io)
    compare(i, run(i))


@pytest.mark.parametrize("gate", ["g", "gamma", "none"])
@pytest.mark.parametrize("h0,dht", [(False, False), (True, False), (False, True)])
def test_gates_and_states(gate, h0, dht):
    for io, D in ((BF, 128), (F32, 64)):
        i = make(5, 1, 100, 1, 2, D, io, gate=gate, h0=h0, dht=dht)
        compare(i, run(i))


@pytest.mark.parametrize("lens", [[5, 0, 64, 1, 130, 63], [0, 0, 3], [200], [0], [65, 0]])
@pytest.mark.parametrize("io,D,Hk,HV", [(BF, 128, 1, 2), (F32, 64, 2, 2), (BF, 64, 1, 1)])
def test_packed(lens, io, D, Hk, HV):
    i = make(len(lens), 1, sum(lens), Hk, HV, D, io, lens=lens)
    compare(i, run(i))


@pytest.mark.parametrize("size", [1e-12, 2.0 ** -20, 3e4, 1e30])
def test_gradients_of_any_size(size):
    i = make(3, 2, 90, 1, 2, 128, size=size)
    compare(i, run(i), size)


def test_heads_and_sequences_of_different_sizes():
    # the power of two is one for each (sequence, head): a small one next to a large one keeps its precision
    i = make(4, 1, 150, 2, 2, 128, lens=[70, 80], h0=True, dht=True)
    f = torch.ones(1, 150, 2, 1)
    f[:, :70, 0], f[:, 70:, 1] = 1e-6, 1e5
    s = torch.tensor([[1e-6, 1.0], [1.0, 1e5]])
    i["dout"] = (i["dout"].float() * f).to(BF)
    i["dht"] = i["dht"] * s[:, :, None, None]
    out = [t.cpu() for t in run(i)]
    ref = want(i)
    for n, (lo, hi) in enumerate(((0, 70), (70, 150))):
        for h in range(2):
            for name, got, r in zip(NAMES[:5], out, ref):
                check(name, got[:, lo:hi, h].float() / s[n, h], r[:, lo:hi, h] / float(s[n, h]), BF, stored=BF)
            check("dh0", out[5][n, h].float() / s[n, h], ref[5][n, h] / float(s[n, h]), BF, stored=BF)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_infinities_and_nan_stay_in_their_sequence_and_head(bad):
    i = make(6, 1, 140, 2, 2, 64, lens=[66, 74])
    clean = [t.clone() for t in run(i)]
    i["dout"][0, 100, 1, 3] = bad
    out = run(i)
    torch.cuda.synchronize()
    for name, a, b in zip(NAMES[:5], out, clean):
        assert torch.equal(a[:, :66], b[:, :66]) and torch.equal(a[:, :, 0], b[:, :, 0]), name
        assert a[:, 66:, 1].isnan().all(), name
    assert torch.equal(out[5][0], clean[5][0]) and torch.equal(out[5][1, 0], clean[5][1, 0])
    assert out[5][1, 1].isnan().all()


def test_zero_gradients():
    i = make(7, 1, 70, 1, 2, 128)
    i["dout"].zero_()
    i["dht"].zero_()
    for t in run(i):
        assert not t.any()


def test_matches_differences_of_the_forward():
    """fp32 io: central differences of the forward's own outputs.  Their error is the forward's (1e-5 of a loss of
    order ten over a step of 1e-2, so 1e-2) and the third derivative's, step^2 = 1e-4 of order one."""
    i = make(8, 1, 80, 1, 2, 64, F32)
    out = dict(zip(NAMES, run(i)))

    def loss(x):
        o, ht = gdn.gdn_chunk_fwd(d(x["q"]), d(x["k"]), d(x["v"]), d(x["g"]), d(x["beta"]), scale=i["scale"], h0=d(x["h0"]))
        return ((o.cpu().double() * i["dout"].double()).sum() + (ht.cpu().double() * i["dht"].double()).sum()).item()

    gen = torch.Generator().manual_seed(1)
    for name in ("q", "k", "v", "g", "beta", "h0"):
        way = torch.randn(i[name].shape, generator=gen)
        way = way / way.norm()
        hi, lo = (dict(i, **{name: i[name] + s * way}) for s in (1e-2, -1e-2))
        slope = (loss(hi) - loss(lo)) / 2e-2
        got = (out["d" + name].cpu().double() * way.double()).sum().item()
        assert abs(slope - got) < 2e-2, (name, slope, got)


def test_long_sequence_sampled_by_state():
    """4096 tokens: the gradients of the last tokens do not depend on what was before but for the state, so a call on
    the tail alone, with the state there, gives them."""
    i = make(9, 1, 4096, 2, 4, 128, h0=False, dht=True)
    full = run(i)
    cut = 3968
    _, ht = gdn.gdn_chunk_fwd(*(d(i[n][:, :cut].contiguous()) for n in ("q", "k", "v", "g", "beta")), scale=i["scale"])
    tail = {n: (t[:, cut:].contiguous() if n in ("q", "k", "v", "g", "beta", "dout") else t) for n, t in i.items()}
    tail["h0"] = ht.cpu()
    ref = want(tail)
    torch.cuda.synchronize()
    for name, got, r in zip(NAMES[:5], full, ref):
        check(name, got[:, cut:].cpu(), r, BF)


def test_same_bits_in_every_run_and_on_another_stream():
    i = make(10, 2, 300, 2, 4, 128)
    a = run(i)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = run(i)
    side.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_captured_with_a_workspace_of_its_own():
    i = make(11, 1, 200, 1, 2, 128, lens=[90, 110])
    g = {n: d(t) if isinstance(t, torch.Tensor) else t for n, t in i.items()}
    need = binding.chunk_bwd_workspace_bytes(1, 200, 1, 2, 128, 128, 2, BF, varlen=True)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    call = lambda w: gdn.gdn_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["beta"], g["dout"], g["dht"],  # noqa: E731
                                       h0=g["h0"], cu_seqlens=g["cu"], workspace=w)
    call(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(ws)
    for seed, cut in ((1, 90), (2, 1), (3, 200)):
        j = make(seed, 1, 200, 1, 2, 128, lens=[cut, 200 - cut], size=10.0 ** -seed)
        for n in ("q", "k", "v", "g", "beta", "dout", "dht", "cu"):
            g[n].copy_(d(j[n]))
        graph.replay()
        torch.cuda.synchronize()
        other = call(None)
        torch.cuda.synchronize()
        for x, y in zip(out, other):
            assert torch.equal(x, y)


def test_a_poisoned_workspace_changes_nothing():
    i = make(12, 1, 150, 1, 2, 64, lens=[20, 0, 130])
    need = binding.chunk_bwd_workspace_bytes(1, 150, 1, 2, 64, 64, 3, BF, varlen=True)
    outs = [run(i, workspace=torch.full((need,), b, dtype=torch.uint8, device=DEV)) for b in (0, 255, 0x7F)]
    torch.cuda.synchronize()
    for o in outs[1:]:
        for x, y in zip(outs[0], o):
            assert torch.equal(x, y)


def test_no_tokens():
    i = make(13, 2, 0, 1, 2, 64)
    out = run(i)
    assert out[0].shape == (2, 0, 1, 64) and torch.equal(out[5], d(i["dht"]).to(BF))
    i = make(13, 2, 0, 1, 2, 64, F32, dht=False)
    assert not run(i)[5].any()
