"""CPU-only checks of the operators around the scans: every refusal happens on
the host before any HIP call (no GPU is touched), through the C ABI and through
the Python binding."""

import os

import pytest
import torch

from gated_delta_rule_61_amd import binding

FAKE = 1 << 20  # 16-byte aligned, never dereferenced (the checks fail first)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from gated_delta_rule_61_amd import build
        build.build()
    return binding.lib()


def _conv(L, step=False, **kw):
    a = dict(x=FAKE, xb=64 * 128, xt=128, w=FAKE, bias=None, silu=1, o0=FAKE, o1=None, o2=None, w0=128, w1=0, w2=0,
             nd=0, ns=0, eps=1e-6, st=None, idx=None, has=None, pool=0, cu=None, n=0, B=2, T=64, D=128, W=4, dt=1)
    if step:
        a.update(T=1, st=FAKE, pool=2)
    a.update(kw)
    head = (a["x"], a["xb"], a["xt"], a["w"], a["bias"], a["silu"], a["o0"], a["o1"], a["o2"], a["w0"], a["w1"], a["w2"])
    tail = (a["B"], a["T"], a["D"], a["W"], a["dt"], None)
    if step:
        return L.gdn_conv_step(*head, a["st"], a["idx"], a["pool"], *tail)
    return L.gdn_conv_fwd(*head, a["nd"], a["ns"], a["eps"], a["st"], a["idx"], a["has"], a["pool"], a["cu"], a["n"],
                          *tail)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(W=5), 2, b"taps"),
    (dict(W=1), 2, b"taps"),
    (dict(D=132, w0=132), 2, b"multiples of 8"),
    (dict(w0=64), 1, b"add up"),
    (dict(w0=64, w2=64), 1, b"add up"),
    (dict(dt=5), 1, b"dtype"),
    (dict(silu=2), 1, b"silu"),
    (dict(ns=1, nd=96), 2, b"norm_dim"),
    (dict(ns=1, nd=128, w0=64, w1=64, o1=FAKE), 1, b"divide"),
    (dict(ns=4, nd=64), 1, b"norm_sections"),
    (dict(ns=1, nd=64, eps=-1.0), 1, b"norm_eps"),
    (dict(x=None), 1, b"required"),
    (dict(o0=None), 1, b"out0"),
    (dict(w0=64, w1=64), 1, b"out1"),
    (dict(x=FAKE + 8), 1, b"aligned"),
    (dict(w=FAKE + 2), 1, b"aligned"),
    (dict(xt=130), 2, b"strides"),
    (dict(xt=-128), 1, b"strides"),
    (dict(xb=4), 2, b"strides"),
    (dict(B=-1), 1, b"sizes"),
    (dict(cu=FAKE, n=3), 1, b"B == 1"),
    (dict(cu=FAKE, n=-3, B=1), 1, b"num_seqs"),
    (dict(has=FAKE), 1, b"needs a state"),
    (dict(st=FAKE, pool=1), 1, b"pool >= N"),
    (dict(B=1 << 13, T=1 << 13), 2, b"too large"),
    (dict(B=1, T=1 << 24, D=1 << 16, w0=1 << 16, xt=1 << 16), 2, b"one launch"),
])
def test_conv_fwd_refuses(L, kw, status, msg):
    assert _conv(L, **kw) == status
    assert msg in L.gdn_last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(T=5), 1, b"1..4"),
    (dict(T=0), 1, b"1..4"),
    (dict(pool=1), 1, b"pool >= B"),
    (dict(st=None), 1, b"state"),
    (dict(W=7), 2, b"taps"),
    (dict(xb=12), 2, b"strides"),
    (dict(B=1 << 20, idx=FAKE, D=1 << 16, w0=1 << 16), 2, b"one launch"),
])
def test_conv_step_refuses(L, kw, status, msg):
    assert _conv(L, step=True, **kw) == status
    assert msg in L.gdn_last_error()


def _ssm(L, step=False, **kw):
    a = dict(x=FAKE, xb=64 * 256, xt=256, d=FAKE, db=256, dtt=4, b=FAKE, bb=64 * 64, bt=64, c=FAKE, cb=64 * 64, ct=64,
             z=None, zb=0, zt=0, al=FAKE, bias=None, D=None, sp=1, h0=None, ht=None, cu=None, n=0, B=2, T=64, Hk=1, HV=4,
             K=64, V=64, cs=64, dt=1, y=FAKE, ws=FAKE, wsb=1 << 40, st=FAKE, sdt=0, idx=None, pool=2)
    if step:
        a.update(T=1)
    a.update(kw)
    rows = (a["x"], a["xb"], a["xt"], a["d"], a["db"], a["dtt"], a["b"], a["bb"], a["bt"], a["c"], a["cb"], a["ct"],
            a["z"], a["zb"], a["zt"], a["al"], a["bias"], a["D"], a["sp"])
    dims = (a["B"], a["T"], a["Hk"], a["HV"], a["K"], a["V"])
    if step:
        return L.ssm_step(*rows, a["st"], a["sdt"], a["idx"], a["pool"], *dims, a["dt"], a["y"], None)
    return L.ssm_chunk_fwd(*rows, a["h0"], a["ht"], a["cu"], a["n"], *dims, a["cs"], a["dt"], a["y"], a["ws"], a["wsb"],
                           None)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(K=96), 2, b"head dims"),
    (dict(V=32), 2, b"head dims"),
    (dict(Hk=3), 1, b"multiple"),
    (dict(dt=9), 1, b"dtype"),
    (dict(sp=3), 1, b"dt_softplus"),
    (dict(HV=0), 1, b"sizes"),
    (dict(x=None), 1, b"required"),
    (dict(al=None), 1, b"required"),
    (dict(y=None), 1, b"required"),
    (dict(b=FAKE + 8), 1, b"aligned"),
    (dict(y=FAKE + 4), 1, b"aligned"),
    (dict(xb=-8), 1, b"strides"),
    (dict(z=FAKE, zb=12, zt=256), 2, b"z: strides"),
    (dict(cb=12), 2, b"Cm: strides"),
])
def test_ssm_refuses(L, step, kw, status, msg):
    assert _ssm(L, step, **kw) == status
    assert msg in L.gdn_last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(cs=32), 2, b"chunk_size"),
    (dict(xt=260), 2, b"x: strides"),
    (dict(xt=1 << 23), 2, b"2^23"),
    (dict(cu=FAKE, n=2), 1, b"B == 1"),
    (dict(h0=FAKE + 4), 1, b"h0"),
    (dict(ht=FAKE + 8), 1, b"ht"),
    (dict(T=8192, B=1, ws=None), 4, b"workspace"),
    (dict(T=8192, B=1, wsb=16), 4, b"workspace"),
    (dict(T=8192, B=1, ws=FAKE + 16), 1, b"256-byte"),
    (dict(B=1 << 13, T=1 << 13), 2, b"too large"),
    (dict(B=1, T=1, cu=FAKE, n=1 << 28, HV=8), 2, b"one launch"),
    (dict(B=1, T=1, cu=FAKE, n=1 << 21, HV=8), 2, b"one launch"),
])
def test_ssm_chunk_fwd_refuses(L, kw, status, msg):
    assert _ssm(L, **kw) == status
    assert msg in L.gdn_last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(T=5), 1, b"1..4"),
    (dict(pool=1), 1, b"pool >= B"),
    (dict(st=None), 1, b"state"),
    (dict(sdt=4), 1, b"state dtype"),
    (dict(st=FAKE + 8), 1, b"aligned"),
    (dict(pool=-1), 1, b"sizes"),
    (dict(B=1 << 21, HV=8, idx=FAKE), 2, b"one launch"),
])
def test_ssm_step_refuses(L, kw, status, msg):
    assert _ssm(L, True, **kw) == status
    assert msg in L.gdn_last_error()


@pytest.mark.parametrize("store", [True, False])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(K=96), 2, b"K must be"),
    (dict(sdt=3), 1, b"state dtype"),
    (dict(form=2), 1, b"8-bit format"),
    (dict(N=-1), 1, b"sizes"),
    (dict(entries=1), 1, b"entries"),
    (dict(pool=1), 1, b"entries"),
    (dict(wide=None), 1, b"required"),
    (dict(q8=FAKE + 8), 1, b"aligned"),
    (dict(scales=FAKE + 4), 1, b"aligned"),
    (dict(pool=1 << 30), 2, b"too large"),
    (dict(N=1 << 24, pool=1 << 14, entries=1 << 14, src=FAKE, dst=FAKE, HV=128, K=64), 2, b"too"),
    (dict(N=1 << 22, src=FAKE, dst=FAKE), 2, b"one launch"),
])
def test_state_q8_refuses(L, store, kw, status, msg):
    a = dict(wide=FAKE, sdt=0, entries=4, src=None, q8=FAKE, form=0, scales=FAKE, pool=4, dst=None, N=2, HV=2, K=64, V=64)
    a.update(kw)
    dims = (a["N"], a["HV"], a["K"], a["V"], None)
    if store:
        r = L.gdn_state_store_q8(a["wide"], a["sdt"], a["entries"], a["src"], a["q8"], a["form"], a["scales"], a["pool"],
                                 a["dst"], *dims)
    else:
        r = L.gdn_state_load_q8(a["q8"], a["form"], a["scales"], a["pool"], a["src"], a["wide"], a["sdt"], a["entries"],
                                a["dst"], *dims)
    assert r == status
    assert msg in L.gdn_last_error()


def test_workspace_of_the_scan():
    ws = lambda *a, **k: binding.ssm_workspace_bytes(*a, torch.bfloat16, **k)
    assert ws(16, 512, 1, 64, 128, 64, 16) == 0              # enough sequences x heads: nothing is split
    one = ws(1, 8192, 1, 64, 128, 64, 1)
    assert one >= 15 * 64 * 128 * 64 * 4 and one % 256 == 0
    assert ws(1, 8192, 1, 64, 128, 64, 3, varlen=True) >= one
    assert ws(1, 0, 1, 64, 128, 64, 1) == 0 and ws(0, 8192, 1, 64, 128, 64, 0) == 0
    assert binding.lib().ssm_chunk_fwd_workspace_bytes(1, 64, 3, 4, 64, 64, 1, 0, 1) == 0


def test_nothing_to_do_is_ok(L):
    assert _conv(L, B=0, x=None, o0=None) == 0
    assert _conv(L, T=0, x=None, o0=None) == 0
    assert _conv(L, step=True, B=0, pool=0, x=None, o0=None) == 0
    assert _ssm(L, B=0, x=None, ht=None) == 0
    assert _ssm(L, T=0, x=None, ht=None) == 0
    assert _ssm(L, True, B=0, pool=0, x=None) == 0
    assert L.gdn_state_store_q8(None, 0, 0, None, None, 0, None, 0, None, 0, 1, 64, 64, None) == 0


def test_binding_wants_gpu_tensors_and_shapes():
    x = torch.zeros(1, 4, 16)
    with pytest.raises(ValueError, match="on a GPU"):
        binding.causal_conv_fwd(x, torch.zeros(16, 4))
    with pytest.raises(ValueError, match="activation"):
        binding.causal_conv_fwd(x, torch.zeros(16, 4), activation="gelu")
    with pytest.raises(ValueError, match="must be"):
        binding.causal_conv_fwd(x[0], torch.zeros(16, 4))
    with pytest.raises(ValueError, match="on a GPU"):
        binding.ssm_chunk_fwd(torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2), torch.zeros(1, 4, 1, 64),
                              torch.zeros(1, 4, 1, 64), torch.zeros(2))
    with pytest.raises(ValueError, match="must be"):
        binding.ssm_step(torch.zeros(1, 4, 2), torch.zeros(1, 4, 2), torch.zeros(1, 4, 1, 64), torch.zeros(1, 4, 1, 64),
                         torch.zeros(2), torch.zeros(1, 2, 64, 64))
    q8, sc = torch.zeros((2, 1, 64, 64), dtype=torch.int8), torch.zeros(2, 1, 64)
    with pytest.raises(ValueError, match="on a GPU"):
        binding.state_store_q8(torch.zeros(2, 1, 64, 64), q8, sc)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        binding.state_load_q8(q8, sc, torch.zeros((2, 1, 64, 64), dtype=torch.float16))


def test_sequences_past_the_joins_launch_are_not_split(L):
    """Packed prompts of a length that is split, but too many of them to join."""
    few = L.ssm_chunk_fwd_workspace_bytes(1, 1 << 20, 8, 64, 128, 64, 1000, 1, 1)
    assert few > 0
    assert L.ssm_chunk_fwd_workspace_bytes(1, 1 << 20, 8, 64, 128, 64, 1 << 16, 1, 1) == 0


@pytest.mark.parametrize("n,length,HV,V,K", [(200, 60, 64, 64, 128), (256, 100, 64, 64, 128), (1024, 64, 64, 64, 128),
                                             (5000, 7, 32, 128, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_workspace_does_not_grow_with_the_sequences(L, n, length, HV, V, K, dtype):
    """Only sequences longer than a segment have states in the workspace: at most
    twice the segments that the tokens fill, and no more than a segment has at
    least (512 work-groups, half of them for the tails: 512 segment and head pairs
    of the bound, 8 more bytes each for the log-decays)."""
    got = binding.ssm_workspace_bytes(1, n * length, 1, HV, K, V, n, dtype, varlen=True)
    assert 0 < got <= 2 * 512 * 2 * (V * K * 4 + 8) + 512
    more = binding.ssm_workspace_bytes(1, n * length, 1, HV, K, V, 4 * n, dtype, varlen=True)
    assert more <= got


def test_workspace_of_one_packed_sequence_is_that_of_a_dense_one(L):
    dense = binding.ssm_workspace_bytes(1, 8192, 1, 64, 128, 64, 1, torch.bfloat16)
    packed = binding.ssm_workspace_bytes(1, 8192, 1, 64, 128, 64, 1, torch.bfloat16, varlen=True)
    assert 0 < dense and 0 < packed <= 2 * dense
