"""GPU tests of the single-token step with per-channel gates against the fp64
oracle.

Bounds: fp32 throughout.  With A the absolute values of every factor, one
token's prediction sums K products of at most six rounded factors (gate, norm,
state), so it is off by at most (K + 16) u sum|S| |e k|; the new state by that
times beta |k|, plus 16 u of its own terms; o likewise.  ``step_bound`` carries
these through the tokens.  The gate exp(-exp(A_log) sp) is off by 2^-21 plus
2^-21 of its exponent.  Then the storage of o, and of the state."""

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
import oracle
from tests.mixer_cases import BF, DEV, U, close, d, f64, randn

pytestmark = pytest.mark.gpu
F32 = torch.float32


def make(seed, B, T, H, HV, K, V, io=BF, pdt=BF, pool=None):
    g = torch.Generator().manual_seed(seed)
    pool = B + 2 if pool is None else pool
    step = torch.exp(torch.rand(HV, K, generator=g) * np.log(100.0) + np.log(1e-3))
    return dict(q=randn(seed, B, T, H, K, dtype=io), k=randn(seed + 1, B, T, H, K, dtype=io),
                v=randn(seed + 2, B, T, HV, V, dtype=io), a=randn(seed + 3, B, T, HV, K, dtype=io),
                b=randn(seed + 4, B, T, HV, dtype=io), A_log=(1 + 15 * torch.rand(HV, generator=g)).log(),
                dt_bias=torch.log(torch.expm1(step)), state=randn(seed + 5, pool, HV, V, K, dtype=pdt, scale=0.3),
                idx=torch.randperm(pool, generator=g)[:B].to(torch.int32))


def reference(i, norm=True, scale=None, eps=1e-6, sb=1.0, thr=20.0):
    """(o, state, bound of o, bound of the state) of every row, without storage."""
    q, k, v, a, b = (f64(i[n]) for n in ("q", "k", "v", "a", "b"))
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    if norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + eps) for x in (q, k))
    q = q * scale
    u = a + f64(i["dt_bias"])
    sp = np.where(sb * u <= thr, np.logaddexp(0.0, sb * u) / sb, u)
    with np.errstate(over="ignore"):
        gk = -np.exp(f64(i["A_log"]))[:, None] * sp
    beta = 1.0 / (1.0 + np.exp(-b))
    st = f64(i["state"])
    of = np.arange(HV) // (HV // H)
    o, eo = np.zeros((B, T, HV, V)), np.zeros((B, T, HV, V))
    es = np.zeros_like(st)
    for r in range(B):
        n = int(i["idx"][r])
        if not 0 <= n < st.shape[0]:
            continue
        S, e = st[n], np.zeros_like(st[n])
        for t in range(T):
            kk, qq = np.abs(k[r, t][of])[:, None, :], np.abs(q[r, t][of])[:, None, :]
            f = np.exp(gk[r, t])[:, None, :]
            # u + dt_bias rounds against its size, so sp is off by u |u|, times e^{A_log}
            fe = f * (2.0 ** -21 + np.abs(gk[r, t]) * 2.0 ** -21 + np.exp(f64(i["A_log"]))[:, None]
                      * (np.abs(u[r, t]) + 1) * 2 * U)[:, None, :]
            ed = e * f + np.abs(S) * fe
            size = (np.abs(S) * f * kk).sum(-1)
            epred = (ed * kk).sum(-1) + (K + 16) * U * size
            dd = beta[r, t][:, None] * (np.abs(v[r, t]) + size)
            edd = beta[r, t][:, None] * epred + 16 * U * dd
            e = ed + edd[:, :, None] * kk + 16 * U * (np.abs(S) * f + dd[:, :, None] * kk)
            # o = S (e q) + (k . q) d, which is off by the same terms
            osize = (np.abs(S) * f * qq).sum(-1) + (kk * qq).sum(-1) * dd
            eo[r, t] = (ed * qq).sum(-1) + (kk * qq).sum(-1) * edd + (K + 16) * U * osize
            o[r, t], S = oracle.kda_step(q[r, t], k[r, t], v[r, t], gk[r, t], beta[r, t], S)
        st[n], es[n] = S, e
    return o, st, eo, es


def check(i, **kw):
    g = {n: d(t) for n, t in i.items()}
    names = dict(use_qk_l2norm=kw.get("norm", True), softplus_beta=kw.get("sb", 1.0),
                 softplus_threshold=kw.get("thr", 20.0), eps=kw.get("eps", 1e-6), scale=kw.get("scale"))
    o = gdn.kda_decode(g["q"], g["k"], g["v"], g["a"], g["b"], g["A_log"], g["dt_bias"], g["state"], g["idx"], **names)
    torch.cuda.synchronize()
    ro, rs, eo, es = reference(i, **kw)
    io = 2.0 ** -8 if o.dtype == BF else U
    st = 2.0 ** -8 if i["state"].dtype == BF else U
    close("o", f64(o), ro, 2 * eo + io * (np.abs(ro) + 2 * eo))
    close("state", f64(g["state"]), rs, 2 * es + st * (np.abs(rs) + 2 * es))
    rest = [n for n in range(i["state"].shape[0]) if n not in i["idx"].tolist()]
    assert torch.equal(g["state"][rest].cpu(), i["state"][rest])
    return o


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io,pdt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_types_and_sizes(T, K, V, io, pdt):
    check(make(T, 3, T, 1, 2, K, V, io, pdt))


@pytest.mark.parametrize("B,H,HV", [(1, 4, 4), (64, 2, 4), (65, 1, 4), (9, 16, 32)])
def test_batches_and_heads(B, H, HV):
    # 256 (row, head) pairs and more take whole work-groups
    check(make(B, B, 2, H, HV, 128, 128))


def test_without_norm_and_with_a_threshold():
    i = make(3, 2, 3, 2, 2, 64, 64, F32, F32)
    i["q"] *= 0.1
    i["k"] *= 0.1
    check(i, norm=False, scale=0.7)
    check(make(4, 2, 3, 2, 2, 64, 64, F32, F32), sb=2.0, thr=0.5, eps=0.1)


def test_rates_past_fp32():
    i = make(5, 2, 2, 1, 2, 64, 64, F32, F32)
    i["A_log"][0] = 200.0                      # decays to nothing ..
    i["a"][0] = -300.0                         # .. but where the step is nothing too, the state stays
    i["a"][1, :, :, :32] = -300.0
    g = {n: d(t) for n, t in i.items()}
    i2 = dict(i, A_log=i["A_log"].clone())
    o = gdn.kda_decode(g["q"], g["k"], g["v"], g["a"], g["b"], g["A_log"], g["dt_bias"], g["state"], g["idx"])
    assert torch.isfinite(o).all() and torch.isfinite(g["state"]).all()
    i2["A_log"][0] = 80.0                      # softplus(-300) e^80 is nothing, softplus of the others e^80 a lot
    g2 = {n: d(t) for n, t in i2.items()}
    o2 = gdn.kda_decode(g2["q"], g2["k"], g2["v"], g2["a"], g2["b"], g2["A_log"], g2["dt_bias"], g2["state"], g2["idx"])
    assert torch.equal(o, o2) and torch.equal(g["state"], g2["state"])


def test_slots_outside_the_pool():
    i = make(6, 4, 2, 2, 4, 128, 128)
    i["idx"] = torch.tensor([2, -1, 6, 0], dtype=torch.int32)
    o = check(i)
    assert not o[1:3].any()


def test_the_same_gate_in_every_channel_is_the_scalar_step():
    i = make(7, 3, 1, 2, 4, 128, 128)
    i["a"] = i["a"][..., :1].expand(-1, -1, -1, 128).contiguous()
    i["dt_bias"] = i["dt_bias"][:, :1].expand(-1, 128).contiguous()
    g = {n: d(t) for n, t in i.items()}
    st = g["state"].clone()
    o = gdn.kda_decode(g["q"], g["k"], g["v"], g["a"], g["b"], g["A_log"], g["dt_bias"], g["state"], g["idx"])
    p = gdn.gdn_decode(g["q"], g["k"], g["v"], g["a"][..., 0].contiguous(), g["b"], g["A_log"],
                       g["dt_bias"][:, 0].contiguous(), st, g["idx"])
    # both round the same numbers, which differ by some fp32 roundings: neighbours at most
    for a, b in ((o, p), (g["state"], st)):
        close("both", f64(a), f64(b), 2.0 ** -7 * np.abs(f64(b)) + 1e-5)


def test_captured_with_slots_that_change():
    i = make(8, 3, 2, 2, 2, 64, 64)
    g = {n: d(t) for n, t in i.items()}
    run = lambda s: gdn.kda_decode(g["q"], g["k"], g["v"], g["a"], g["b"], g["A_log"], g["dt_bias"], s, g["idx"])  # noqa: E731
    run(g["state"].clone())
    torch.cuda.synchronize()
    mine = g["state"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = run(g["state"])
    for slots in ([0, 1, 2], [4, 3, 0], [2, 9, 1]):
        g["idx"].copy_(torch.tensor(slots, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = run(mine)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(g["state"], mine)
