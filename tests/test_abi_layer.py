"""CPU-only checks of the layer operators (gradients of the convolution, norm and
its gradients, step with per-channel gates): every refusal happens on the host
before any HIP call (no GPU is touched), through the C ABI and through the
Python binding."""

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


def _conv_bwd(L, **kw):
    a = dict(o0=FAKE, o1=None, o2=None, w0=128, w1=0, w2=0, x=FAKE, xb=64 * 128, xt=128, w=FAKE, bias=None, silu=1,
             nd=0, ns=0, eps=1e-6, cu=None, n=0, B=2, T=64, D=128, W=4, dt=1, dx=FAKE, dw=FAKE, db=None, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return L.gdn_conv_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(W=5), 2, b"taps"),
    (dict(D=132, w0=132), 2, b"multiples of 8"),
    (dict(w0=64), 1, b"add up"),
    (dict(dt=5), 1, b"dtype"),
    (dict(silu=2), 1, b"silu"),
    (dict(ns=1, nd=96), 2, b"norm_dim"),
    (dict(ns=1, nd=64, eps=-1.0), 1, b"norm_eps"),
    (dict(x=None), 1, b"required"),
    (dict(o0=None), 1, b"out0"),
    (dict(dx=None), 1, b"dx"),
    (dict(x=FAKE + 8), 1, b"aligned"),
    (dict(dw=FAKE + 8), 1, b"aligned"),
    (dict(xt=130), 2, b"strides"),
    (dict(B=-1), 1, b"sizes"),
    (dict(cu=FAKE, n=3), 1, b"B == 1"),
    (dict(B=1 << 13, T=1 << 13), 2, b"too large"),
    (dict(B=1, T=1 << 24, D=1 << 16, w0=1 << 16, xt=1 << 16), 2, b"one launch"),
    (dict(ws=None), 4, b"workspace"),
    (dict(wsb=16), 4, b"workspace"),
    (dict(ws=FAKE + 16), 1, b"256-byte"),
])
def test_conv_bwd_refuses(L, kw, status, msg):
    assert _conv_bwd(L, **kw) == status
    assert msg in L.gdn_last_error()


def _norm(L, bwd=False, **kw):
    a = dict(g=FAKE, gb=64 * 256, gt=256, x=FAKE, xb=64 * 256, xt=256, w=FAKE, b=None, wdt=0, sh=1, z=None, zb=0, zt=0,
             act=1, rms=0, eps=1e-5, B=2, T=64, G=4, d=64, dt=1, y=FAKE, dz=None, dw=FAKE, db=None, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    v = list(a.values())
    if bwd:
        return L.gdn_group_norm_bwd(*v, None)
    return L.gdn_group_norm_fwd(*v[3:22], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(d=60), 2, b"multiple of 8"),
    (dict(d=8200), 2, b"up to 8192"),
    (dict(G=1 << 17), 2, b"2^23"),
    (dict(G=0), 1, b"sizes"),
    (dict(B=-1), 1, b"sizes"),
    (dict(B=1 << 13, T=1 << 13), 2, b"too large"),
    (dict(act=3), 1, b"activation"),
    (dict(rms=2), 1, b"rms"),
    (dict(sh=2), 1, b"weight_shared"),
    (dict(eps=-1.0), 1, b"eps"),
    (dict(eps=float("nan")), 1, b"eps"),
    (dict(dt=7), 1, b"dtype"),
    (dict(wdt=7), 1, b"weight dtype"),
    (dict(w=FAKE + 4), 1, b"aligned"),
    (dict(x=None), 1, b"required"),
    (dict(y=None), 1, b"required"),
    (dict(x=FAKE + 8), 1, b"aligned"),
    (dict(xt=260), 2, b"strides"),
    (dict(xb=-8), 1, b"strides"),
    (dict(z=FAKE, zt=12, dz=FAKE), 2, b"z: strides"),
])
def test_norm_refuses(L, bwd, kw, status, msg):
    assert _norm(L, bwd, **kw) == status
    assert msg in L.gdn_last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(g=None), 1, b"required"),
    (dict(z=FAKE, zt=256, zb=64 * 256), 1, b"dz"),
    (dict(gt=4), 2, b"dout: strides"),
    (dict(ws=None), 4, b"workspace"),
    (dict(wsb=64), 4, b"workspace"),
    (dict(ws=FAKE + 64), 1, b"256-byte"),
])
def test_norm_bwd_refuses(L, kw, status, msg):
    assert _norm(L, True, **kw) == status
    assert msg in L.gdn_last_error()


def _kda(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, a=FAKE, b=FAKE, al=FAKE, bias=FAKE, st=FAKE, sdt=1, idx=None, o=FAKE, B=2, T=1, H=2,
             HV=4, K=128, V=128, pool=2, scale=1.0, sb=1.0, thr=20.0, norm=1, eps=1e-6, dt=1)
    a.update(kw)
    return L.kda_decode(*a.values(), None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(T=0), 1, b"1..4"),
    (dict(T=5), 1, b"1..4"),
    (dict(H=3), 1, b"multiple"),
    (dict(HV=0), 1, b"sizes"),
    (dict(K=96), 2, b"head dims"),
    (dict(V=256), 2, b"head dims"),
    (dict(pool=1), 1, b"pool >= B"),
    (dict(pool=-1), 1, b"sizes"),
    (dict(sb=0.0), 1, b"softplus_beta"),
    (dict(eps=-1.0), 1, b"eps"),
    (dict(dt=4), 1, b"dtype"),
    (dict(sdt=4), 1, b"state dtype"),
    (dict(bias=None), 1, b"required"),
    (dict(st=None), 1, b"required"),
    (dict(q=FAKE + 8), 1, b"aligned"),
    (dict(st=FAKE + 8), 1, b"aligned"),
    (dict(pool=1 << 30, idx=FAKE), 2, b"pool too large"),
    (dict(B=1 << 24, idx=FAKE), 2, b"one launch"),
])
def test_kda_decode_refuses(L, kw, status, msg):
    assert _kda(L, **kw) == status
    assert msg in L.gdn_last_error()


def test_nothing_to_do(L):
    assert _kda(L, B=0, q=None) == 0
    assert _norm(L, B=0, x=None) == 0
    assert _norm(L, True, T=0, x=None, dw=None) == 0
    assert _conv_bwd(L, T=0, x=None, dw=None) == 0


def test_workspace_sizes(L):
    assert L.gdn_conv_bwd_workspace_bytes(1, 0, 128, 4) == 0
    assert L.gdn_conv_bwd_workspace_bytes(1, 100, 128, 5) == 0
    assert L.gdn_conv_bwd_workspace_bytes(1, 100, 128, 4) >= 5 * 128 * 4
    assert L.gdn_group_norm_bwd_workspace_bytes(1, 0, 4, 64, 1) == 0
    assert L.gdn_group_norm_bwd_workspace_bytes(1, 9, 4, 60, 1) == 0
    assert L.gdn_group_norm_bwd_workspace_bytes(1, 9, 4, 64, 0) >= 2 * 256 * 4


def test_binding_refuses():
    x, w = torch.zeros(1, 4, 128), torch.zeros(128, 4)
    with pytest.raises(ValueError, match="on a GPU"):
        binding.causal_conv_bwd(x, x, w)
    with pytest.raises(ValueError, match="activation"):
        binding.causal_conv_bwd(x, x, w, activation="relu")
    with pytest.raises(ValueError, match=r"\[B, T, D\]"):
        binding.causal_conv_bwd(x, x[0], w)
    with pytest.raises(ValueError, match="num_groups"):
        binding.group_norm_fwd(x, 3)
    with pytest.raises(ValueError, match="activation"):
        binding.group_norm_fwd(x, 2, activation="gelu")
    with pytest.raises(ValueError, match=r"\[B, T, C\]"):
        binding.group_norm_bwd(x, x[0], 2)
    with pytest.raises(ValueError, match="on a GPU"):
        binding.group_norm_bwd(x, x, 2)
    q = torch.zeros(1, 1, 2, 64)
    with pytest.raises(ValueError, match="on a GPU"):
        binding.kda_decode(q, q, q, q, q[..., 0], w[0], w, q)
    with pytest.raises(ValueError, match=r"\[B, T, H, K\]"):
        binding.kda_decode(q[0], q, q, q, q[..., 0], w[0], w, q)


def _chunk_bwd(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, gamma=None, beta=FAKE, scale=1.0, h0=None, do=FAKE, dht=None, cu=None, n=0,
             B=2, T=64, Hk=2, HV=4, K=128, V=128, cs=64, dt=1, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, db=FAKE, dh0=None,
             ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.gdn_chunk_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(K=96, V=96), 2, b"head dims"),
    (dict(K=64), 2, b"head dims"),
    (dict(Hk=3), 1, b"multiple"),
    (dict(HV=0), 1, b"sizes"),
    (dict(cs=32), 2, b"chunk_size"),
    (dict(dt=3), 1, b"dtype"),
    (dict(gamma=FAKE), 1, b"not both"),
    (dict(q=None), 1, b"required"),
    (dict(do=None), 1, b"required"),
    (dict(dq=None), 1, b"required"),
    (dict(db=None), 1, b"required"),
    (dict(do=FAKE + 8), 1, b"aligned"),
    (dict(dk=FAKE + 8), 1, b"aligned"),
    (dict(dht=FAKE + 4), 1, b"aligned"),
    (dict(cu=FAKE, n=2), 1, b"B == 1"),
    (dict(cu=FAKE, n=-2, B=1), 1, b"num_seqs"),
    (dict(B=1 << 13, T=1 << 13), 2, b"too large"),
    (dict(ws=None), 4, b"workspace"),
    (dict(wsb=1024), 4, b"workspace"),
    (dict(ws=FAKE + 128), 1, b"256-byte"),
])
def test_chunk_bwd_refuses(L, kw, status, msg):
    assert _chunk_bwd(L, **kw) == status
    assert msg in L.gdn_last_error()


def test_chunk_bwd_workspace(L):
    size = L.gdn_chunk_bwd_workspace_bytes
    assert size(1, 64, 2, 4, 128, 128, 1, 0, 9) == 0
    assert size(1, -1, 2, 4, 128, 128, 1, 0, 1) == 0
    # a chunk: two states and two [64, V] arrays of the compute type, and the prefill's arrays
    assert size(1, 64, 1, 1, 128, 128, 1, 0, 1) >= 2 * (2 * 128 * 128 + 2 * 64 * 128)
    assert size(1, 64, 1, 1, 128, 128, 1, 0, 0) >= 2 * size(1, 64, 1, 1, 128, 128, 1, 0, 1) - 4096
    assert size(1, 64, 1, 1, 128, 128, 5, 1, 1) > 4 * size(1, 64, 1, 1, 128, 128, 1, 0, 1)
    assert _chunk_bwd(L, cu=FAKE, n=0, B=1) == 0


def test_chunk_bwd_binding_refuses():
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError, match="on a GPU"):
        binding.gdn_chunk_bwd(q, q, q, q[..., 0], q[..., 0], q)
    with pytest.raises(ValueError, match=r"\[B, T, Hk, K\]"):
        binding.gdn_chunk_bwd(q[0], q, q, q[..., 0], q[..., 0], q)
