"""Pins of the oracle's layer operators: gradients against automatic
differentiation of an independently written form in 64 bits and against
differences, the step against the recurrence, the norm against torch's."""

import numpy as np
import pytest
import torch

import oracle


def rnd(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape))


def leaf(t):
    return None if t is None else t.clone().requires_grad_()


def unit(t):
    return t / t.norm(dim=-1, keepdim=True)


def delta_rule(q, k, v, g, beta, scale, h0, edges):
    """One packed batch [T, H, .] as products of whole transition matrices (autograd's input)."""
    r = v.shape[1] // k.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    eye = torch.eye(k.shape[-1], dtype=k.dtype)
    out, last = [], []
    for n, (a, b) in enumerate(zip(edges[:-1], edges[1:])):
        S = h0[n]
        for t in range(a, b):
            kk = k[t][:, :, None] * k[t][:, None, :]
            S = torch.exp(g[t])[:, None, None] * (S @ (eye - beta[t][:, None, None] * kk)) \
                + beta[t][:, None, None] * v[t][:, :, None] * k[t][:, None, :]
            out.append(scale * (S @ q[t][:, :, None])[:, :, 0])
        last.append(S)
    return torch.stack(out), torch.stack(last)


@pytest.mark.parametrize("Hk,HV,edges", [(2, 2, [0, 9]), (1, 3, [0, 4, 4, 11]), (2, 4, [0, 1, 7])])
def test_delta_rule_gradients_match_autograd(Hk, HV, edges):
    rng = np.random.default_rng(HV)
    T, K, V, N = edges[-1], 5, 4, len(edges) - 1
    q, k, v = unit(rnd(rng, T, Hk, K)), unit(rnd(rng, T, Hk, K)), rnd(rng, T, HV, V)
    g, beta, h0 = -rnd(rng, T, HV).abs() * 0.3, torch.sigmoid(rnd(rng, T, HV)), rnd(rng, N, HV, V, K)
    do, dht = rnd(rng, T, HV, V), rnd(rng, N, HV, V, K)
    leaves = [leaf(t) for t in (q, k, v, g, beta, h0)]
    o, ht = delta_rule(*leaves[:5], 0.7, leaves[5], edges)
    want = torch.autograd.grad((o, ht), leaves, (do, dht))
    cu = torch.tensor(edges)
    b = lambda t: t[None].numpy()  # noqa: E731
    got = oracle.gdn_recurrent_bwd(b(q), b(k), b(v), b(g), b(beta), b(do), 0.7, h0.numpy(), dht.numpy(), cu)
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        np.testing.assert_allclose(x[0], y.numpy(), rtol=1e-10, atol=1e-11, err_msg=name)
    np.testing.assert_allclose(got[5], want[5].numpy(), rtol=1e-10, atol=1e-11)


def test_delta_rule_gradients_match_differences():
    rng = np.random.default_rng(3)
    T, H, K = 6, 2, 4
    x = dict(q=unit(rnd(rng, 1, T, H, K)).numpy(), k=unit(rnd(rng, 1, T, H, K)).numpy(), v=rnd(rng, 1, T, H, K).numpy(),
             g=-rnd(rng, 1, T, H).abs().numpy(), beta=torch.sigmoid(rnd(rng, 1, T, H)).numpy(),
             h0=rnd(rng, 1, H, K, K).numpy())
    do, dht = rnd(rng, 1, T, H, K).numpy(), rnd(rng, 1, H, K, K).numpy()

    def loss(**y):
        o, ht = oracle.gdn_recurrent(y["q"], y["k"], y["v"], y["g"], y["beta"], 0.5, h0=y["h0"])
        return (o * do).sum() + (ht * dht).sum()

    got = oracle.gdn_recurrent_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], do, 0.5, x["h0"], dht)
    for name, grad in zip(("q", "k", "v", "g", "beta", "h0"), got):
        for _ in range(4):
            at = tuple(rng.integers(0, s) for s in x[name].shape)
            step = 1e-5
            hi, lo = {n: a.copy() for n, a in x.items()}, {n: a.copy() for n, a in x.items()}
            hi[name][at] += step
            lo[name][at] -= step
            # central differences: error step^2 times a third derivative, and 1e-16 / step of a loss below 1e2
            assert abs((loss(**hi) - loss(**lo)) / (2 * step) - grad[at]) < 1e-7, name


def test_fixed_decay_is_the_same_gate_at_every_token():
    rng = np.random.default_rng(5)
    q, k, v = (rng.standard_normal((1, 5, 2, 4)) for _ in range(3))
    beta, do, gamma = rng.random((1, 5, 2)), rng.standard_normal((1, 5, 2, 4)), np.array([-0.1, -0.5])
    a = oracle.gdn_recurrent_bwd(q, k, v, None, beta, do, 1.0, g_gamma=gamma)
    b = oracle.gdn_recurrent_bwd(q, k, v, np.broadcast_to(gamma, (1, 5, 2)), beta, do, 1.0)
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)


def test_step_follows_the_recurrence():
    rng = np.random.default_rng(7)
    T, H, HV, K, V = 5, 2, 4, 6, 3
    q, k = rng.standard_normal((1, T, H, K)), rng.standard_normal((1, T, H, K)) * 0.4
    v, gk = rng.standard_normal((1, T, HV, V)), -rng.random((1, T, HV, K))
    beta, h0 = rng.random((1, T, HV)), rng.standard_normal((1, HV, V, K))
    want, last = oracle.kda_recurrent(q, k, v, gk, beta, 0.5, h0=h0)
    S = h0[0]
    for t in range(T):
        o, S = oracle.kda_step(0.5 * q[0, t], k[0, t], v[0, t], gk[0, t], beta[0, t], S)
        np.testing.assert_allclose(o, want[0, t], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(S, last[0], rtol=1e-12, atol=1e-13)


ACTS = {None: lambda t: t, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_matches_torch(act, gated, rms, shared):
    rng = np.random.default_rng(11)
    G, d, rows = 3, 8, 5
    x, z, dy = rnd(rng, rows, G * d), rnd(rng, rows, G * d) if gated else None, rnd(rng, rows, G * d)
    w, b = rnd(rng, d if shared else G * d), rnd(rng, d if shared else G * d)
    leaves = {n: leaf(t) for n, t in (("x", x), ("z", z), ("w", w), ("b", b)) if t is not None}
    h = leaves["x"].reshape(rows, G, d)
    if rms:
        n = torch.nn.functional.rms_norm(h, (d,), eps=1e-5)
    else:
        n = torch.nn.functional.group_norm(leaves["x"], G, eps=1e-5).reshape(h.shape)
    each = lambda t: t if shared else t.reshape(G, d)  # noqa: E731
    a = (n * each(leaves["w"]) + each(leaves["b"])).reshape(x.shape)
    y = a * ACTS[act](leaves["z"]) if gated else ACTS[act](a)
    got = oracle.group_norm(x, G, w, b, z, act, rms)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-6, atol=1e-6)
    want = torch.autograd.grad(y, list(leaves.values()), dy)
    dx, dz, dw, db = oracle.group_norm(x, G, w, b, z, act, rms, dout=dy)
    for name, grad in zip(leaves, want):
        np.testing.assert_allclose({"x": dx, "z": dz, "w": dw, "b": db}[name], grad.numpy(), rtol=1e-6, atol=1e-6,
                                   err_msg=name)


@pytest.mark.parametrize("L", [1, 2, 7])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("act,norm", [(True, 8), (True, 0), (False, 0)])
def test_conv_gradients_match_autograd(L, W, act, norm):
    rng = np.random.default_rng(L * 10 + W)
    D = 12
    x, w, b, dy = leaf(rnd(rng, L, D)), leaf(rnd(rng, D, W)), leaf(rnd(rng, D)), rnd(rng, L, D)
    y = torch.nn.functional.conv1d(torch.nn.functional.pad(x.t(), (W - 1, 0))[None], w[:, None], b, groups=D)[0].t()
    y = torch.nn.functional.silu(y) if act else y
    if norm:
        h = y[:, :norm].reshape(L, -1, 4)
        y = torch.cat([(h / (h.square().sum(-1, keepdim=True) + 1e-6).sqrt()).reshape(L, norm), y[:, norm:]], 1)
    want = torch.autograd.grad(y, (x, w, b), dy)
    got = oracle.causal_conv_bwd(dy, x.detach(), w.detach(), b.detach(), act, 4, norm, 1e-6)
    for name, p, r in zip(("dx", "dweight", "dbias"), got, want):
        np.testing.assert_allclose(p, r.numpy(), rtol=1e-6, atol=1e-6, err_msg=name)
