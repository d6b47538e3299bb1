"""The operators around a recurrent layer's scan, fp64 (oracle; test
infrastructure only): the short causal convolution, the selective state-space
recurrence, and the 8-bit storage of states.  All from their definitions, one
token, one row at a time.

* Convolution: c_t = bias + sum_j w_j u_{t-W+1+j}, u being a sequence's rows
  behind the W - 1 rows of its state (zeros for a new sequence).
* Selective scan: D_t = softplus(dt_t + dt_bias), S <- exp(-exp(A_log) D_t) S +
  D_t x_t B_t^T, y_t = (S C_t + D x_t) silu(z_t); group of head j is
  j // (HV // Hk).
* 8-bit states: one scale per row of the last axis; int8 codes are row / scale
  rounded to nearest even, e4m3 codes row / scale rounded to the format's grid
  (three mantissa bits, spacing 2^-9 below 2^-6).
"""

from __future__ import annotations

import numpy as np

from .recurrence import _f64


def silu(a):
    a = _f64(a)
    return a / (1.0 + np.exp(-a))


def causal_conv(x, weight, bias=None, state=None, activation=True):
    """One sequence x [L, D], weight [D, W], state [W - 1, D] or None.  Returns
    (y [L, D], the last W - 1 rows, sum of |terms| [L, D])."""
    x, w = _f64(x), _f64(weight)
    L, D = x.shape
    W = w.shape[1]
    u = np.concatenate([np.zeros((W - 1, D)) if state is None else _f64(state), x])
    y = np.zeros((L, D))
    mag = np.zeros((L, D))
    for t in range(L):
        acc = np.zeros(D) if bias is None else _f64(bias).copy()
        size = np.abs(acc)
        for j in range(W):
            acc = acc + w[:, j] * u[t + j]
            size = size + np.abs(w[:, j] * u[t + j])
        y[t], mag[t] = acc, size
    return (silu(y) if activation else y), u[L:], mag


def head_norm(y, dim, eps):
    """Every head of `dim` consecutive channels of y [L, D] over its L2 norm."""
    y = _f64(y)
    h = y.reshape(y.shape[0], -1, dim)
    return (h / np.sqrt((h * h).sum(-1, keepdims=True) + eps)).reshape(y.shape)


def ssm_scan(x, dt, B, C, A_log, D=None, z=None, dt_bias=None, h0=None, softplus=True):
    """One sequence: x [L, HV, V], dt [L, HV], B, C [L, Hk, K], h0 [HV, V, K].
    Returns (y [L, HV, V], final state [HV, V, K])."""
    x, dt, B, C = _f64(x), _f64(dt), _f64(B), _f64(C)
    L, HV, V = x.shape
    Hk, K = B.shape[1:]
    rate = np.exp(_f64(A_log))
    step = dt + (0.0 if dt_bias is None else _f64(dt_bias))
    if softplus:
        step = np.logaddexp(0.0, step)
    S = np.zeros((HV, V, K)) if h0 is None else _f64(h0).copy()
    group = np.arange(HV) // (HV // Hk)
    y = np.zeros((L, HV, V))
    for t in range(L):
        S = np.exp(-rate * step[t])[:, None, None] * S + (step[t][:, None] * x[t])[:, :, None] * B[t][group][:, None, :]
        y[t] = np.einsum("hvk,hk->hv", S, C[t][group])
    if D is not None:
        y = y + _f64(D)[:, None] * x
    if z is not None:
        y = y * silu(z)
    return y, S


def quantise_state(x, form):
    """x [..., K] fp32 values; form "int8" or "e4m3".  Returns (codes as the
    numbers they are, scales [...]); a row with an infinity or NaN has codes 0
    and a NaN scale."""
    x = _f64(x)
    most = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    most = np.where(bad, 0.0, most)
    if form == "int8":
        r = np.float32(1.0) / np.float32(127.0)
        scale = np.maximum(most.astype(np.float32) * r, np.float32(2.0 ** -126)).astype(np.float64)
        codes = np.rint(np.where(bad[..., None], 0.0, x) / scale[..., None])
    else:
        with np.errstate(divide="ignore"):
            e = np.ceil(np.log2(most / 448.0))
        # log2 may be off by its rounding: settle the exponent by its definition
        e = np.where(np.isfinite(e), e, -126.0)
        e = np.where(most > 448.0 * np.exp2(e), e + 1, e)
        e = np.where((most <= 448.0 * np.exp2(e - 1)) & (most > 0), e - 1, e)
        scale = np.exp2(np.maximum(e, -126.0))
        u = np.where(bad[..., None], 0.0, x) / scale[..., None]
        unit = np.exp2(np.floor(np.log2(np.maximum(np.abs(u), 2.0 ** -6))) - 3)
        codes = np.rint(u / unit) * unit
    return codes, np.where(bad, np.nan, scale)
