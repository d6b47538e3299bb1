"""The other operators of a recurrent layer, fp64 (oracle; test infrastructure
only), from their definitions: the adjoint of the scalar-gate delta rule, token
by token; the single-token step with one gate per key channel; the norm of a
token's channel groups with its activation or gate, and its gradients; the
gradients of the short convolution with silu and head norms.

* Delta rule: S' = e^{g} S, d = beta (v - S' k), S = S' + d k^T, o = scale S q.
  Its adjoint walks the tokens backwards with the gradient of S after each.
* Norm: n = (x - mean) / sqrt(var + eps) (rms: x / sqrt(mean x^2 + eps)),
  a = n w + b, y = a act(z), or act(a) without z.
* Convolution: c_t = bias + sum_j w_j x_{t-W+1+j}, u = silu(c) or c, heads of
  normalised channels u / sqrt(sum u^2 + eps).
"""

from __future__ import annotations

import numpy as np

from .recurrence import _f64, sequences


def gdn_recurrent_bwd(q, k, v, g, beta, dout, scale, h0=None, dht=None, cu_seqlens=None, g_gamma=None):
    """Gradients (dq, dk, dv, dg, dbeta, dh0) of ``gdn_recurrent``'s outputs and
    final states; arguments and layouts as there, dout [B, T, HV, V], dht [N,
    HV, V, K] or None."""
    q, k, v, g, beta, dout = _f64(q), _f64(k), _f64(v), _f64(g), _f64(beta), _f64(dout)
    h0, dht = _f64(h0), _f64(dht)
    B, T, Hk, K = q.shape
    HV, V = v.shape[2:]
    if g is None:
        g = np.zeros((B, T, HV)) if g_gamma is None else np.broadcast_to(_f64(g_gamma), (B, T, HV))
    of = np.arange(HV) // (HV // Hk)
    seqs = sequences(B, T, cu_seqlens)
    dq, dk = np.zeros_like(q), np.zeros_like(k)
    dv, dg, dbeta = np.zeros_like(v), np.zeros((B, T, HV)), np.zeros((B, T, HV))
    dh0 = np.zeros((len(seqs), HV, V, K))
    for n, (b, bos, eos) in enumerate(seqs):
        S = np.zeros((HV, V, K)) if h0 is None else h0[n].copy()
        states = []
        for t in range(bos, eos):
            states.append(S)
            kt = k[b, t, of]
            Sd = np.exp(g[b, t])[:, None, None] * S
            d = beta[b, t][:, None] * (v[b, t] - np.einsum("hvk,hk->hv", Sd, kt))
            S = Sd + d[:, :, None] * kt[:, None, :]
        dS = np.zeros((HV, V, K)) if dht is None else dht[n].copy()
        for t in reversed(range(bos, eos)):
            kt, qt, do = k[b, t, of], q[b, t, of], dout[b, t]
            a = np.exp(g[b, t])[:, None, None]
            Sd = a * states[t - bos]
            gap = v[b, t] - np.einsum("hvk,hk->hv", Sd, kt)
            d = beta[b, t][:, None] * gap
            S = Sd + d[:, :, None] * kt[:, None, :]
            np.add.at(dq[b, t], of, scale * np.einsum("hvk,hv->hk", S, do))
            dS = dS + scale * do[:, :, None] * qt[:, None, :]
            dd = np.einsum("hvk,hk->hv", dS, kt)
            dbeta[b, t] = (dd * gap).sum(-1)
            dv[b, t] = beta[b, t][:, None] * dd
            np.add.at(dk[b, t], of, np.einsum("hvk,hv->hk", dS, d) - np.einsum("hvk,hv->hk", Sd, dv[b, t]))
            dS = dS - dv[b, t][:, :, None] * kt[:, None, :]
            dg[b, t] = (dS * Sd).sum((-1, -2))
            dS = a * dS
        dh0[n] = dS
    return dq, dk, dv, dg, dbeta, dh0


def kda_step(q, k, v, gk, beta, state):
    """One token: q, k [H, K] as they enter the products, v [HV, V], gk [HV, K]
    log-gates, beta [HV], state [HV, V, K].  Returns (o [HV, V], state)."""
    q, k, v, gk, beta, S = _f64(q), _f64(k), _f64(v), _f64(gk), _f64(beta), _f64(state)
    of = np.arange(v.shape[0]) // (v.shape[0] // q.shape[0])
    S = S * np.exp(gk)[:, None, :]
    d = beta[:, None] * (v - np.einsum("hvk,hk->hv", S, k[of]))
    S = S + d[:, :, None] * k[of][:, None, :]
    return np.einsum("hvk,hk->hv", S, q[of]), S


def _sigmoid(a):
    return 1.0 / (1.0 + np.exp(-a))


def _act(a, kind):
    """(act(a), its slope)"""
    if kind is None:
        return a, np.ones_like(a)
    p = _sigmoid(a)
    if kind == "sigmoid":
        return p, p * (1 - p)
    return a * p, p * (1 + a * (1 - p))


def group_norm(x, groups, weight=None, bias=None, z=None, activation="silu", rms=False, eps=1e-5, dout=None):
    """x, z, dout [..., C]; weight, bias [C] or [C / groups].  Returns y, or with
    dout the gradients (dx, dz, dweight, dbias) (dz None without z)."""
    x = _f64(x)
    shape = x.shape
    cut = lambda a: _f64(a).reshape(-1, groups, shape[-1] // groups)  # noqa: E731
    x, d = cut(x), shape[-1] // groups
    shared = next((np.shape(a)[0] == d for a in (weight, bias) if a is not None), True)
    each = lambda a, none: np.full((1, 1, d), none) if a is None else _f64(a).reshape(1, 1 if shared else groups, d)  # noqa: E731
    w, b = each(weight, 1.0), each(bias, 0.0)
    c = x if rms else x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = c * r
    a = n * w + b
    f, df = _act(a if z is None else cut(z), activation)
    if dout is None:
        return (f if z is None else a * f).reshape(shape)
    dy = cut(dout)
    da = dy * (df if z is None else f)
    dn = da * w
    dx = dn - n * (dn * n).mean(-1, keepdims=True)
    if not rms:
        dx = dx - dn.mean(-1, keepdims=True)
    over = (0, 1) if shared else (0,)
    return ((r * dx).reshape(shape), None if z is None else (dy * a * df).reshape(shape),
            (da * n).sum(over).reshape(-1), da.sum(over).reshape(-1))


def causal_conv_bwd(dout, x, weight, bias=None, activation=True, norm_dim=0, norm_channels=0, eps=1e-6):
    """One sequence that starts from zeros: dout, x [L, D], weight [D, W]; the
    first norm_channels channels are normalised in heads of norm_dim.  Returns
    (dx, dweight, dbias)."""
    dy, x, w = _f64(dout).copy(), _f64(x), _f64(weight)
    L, D = x.shape
    W = w.shape[1]
    u = np.concatenate([np.zeros((W - 1, D)), x])
    c = np.zeros((L, D)) if bias is None else np.tile(_f64(bias), (L, 1))
    for j in range(W):
        c = c + w[:, j] * u[j: j + L]
    y, slope = _act(c, "silu" if activation else None)
    if norm_channels:
        h = y[:, :norm_channels].reshape(L, norm_channels // norm_dim, norm_dim)
        g = dy[:, :norm_channels].reshape(h.shape)
        r = 1.0 / np.sqrt((h * h).sum(-1, keepdims=True) + eps)
        dy[:, :norm_channels] = (r * (g - h * r * (h * r * g).sum(-1, keepdims=True))).reshape(L, norm_channels)
    dc = dy * slope
    dx, dw = np.zeros((L, D)), np.zeros((D, W))
    for j in range(W):
        dw[:, j] = (dc * u[j: j + L]).sum(0)
        back = W - 1 - j                       # dc of this many tokens later
        dx[: max(L - back, 0)] += w[:, j] * dc[back:]
    return dx, dw, dc.sum(0)
