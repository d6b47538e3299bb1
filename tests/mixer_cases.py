"""Inputs, oracle runs and error bounds shared by the GPU tests of the operators
around the scans.

The bounds are per element and worst-case, from the sizes of the summed terms
(the oracle on absolute values): u = 2^-24 is an fp32 rounding, a bf16 rounding
is off by at most 2^-8 of the value.

* Convolution: at most W + 1 fp32 roundings of the sum of |terms| (8 u covers
  W <= 4), silu (slope at most 1.1, relative error of exp and reciprocal below
  2^-20), then the storage.  Norm: the head's error vector over its norm, twice
  (numerator and norm), plus 2^-20.
* Scan, fp32 io: each output is a sum of K + 64 products, through at most T / 64
  rescaled states; with gates good to 2^-22 each, 512 u of the absolute sum
  covers T <= 4000.  bf16 io: x is rounded once when it enters the state, the
  state once as an operand, scores once: 2 x 2^-8 of the absolute sum, plus the
  storage.  ht (three bf16 terms, 2^-26): 512 u of the absolute state.
"""

import numpy as np
import torch

import oracle

DEV = "cuda:0"
U = 2.0 ** -24
BF = torch.bfloat16
EPS = 1e-6


def d(t):
    return None if t is None else t.to(DEV)


def randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def store(dtype, ref):
    return (2.0 ** -8 if dtype == BF else U) * np.abs(ref)


def f64(t):
    return t.detach().cpu().double().numpy()


def close(name, got, ref, bound):
    g = f64(got) if isinstance(got, torch.Tensor) else got
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{name}: non-finite values"
    if g.size:
        over = np.abs(g - ref) - bound
        i = np.unravel_index(int(np.argmax(over)), over.shape)
        assert over[i] <= 0, f"{name}{list(i)}: {g[i]:.9g} for {ref[i]:.9g}, bound {np.broadcast_to(bound, ref.shape)[i]:.3g}"


def edges(lens):
    return [0] + list(np.cumsum(lens))


def conv_ref(x, w, bias, lens, states, act, sections, norm_dim, norm_sections):
    """Packed x [R, D] (fp64-exact), states: per sequence [W - 1, D] or None.
    Returns (sections' values, their bounds without storage, the last rows)."""
    e = edges(lens)
    R, D = x.shape
    y, err = np.zeros((R, D)), np.zeros((R, D))
    last = []
    for i in range(len(lens)):
        r = slice(e[i], e[i + 1])
        yi, li, mag = oracle.causal_conv(x[r], w, bias, states[i], act)
        y[r], last = yi, last + [li]
        err[r] = 8 * U * mag * (1.1 if act else 1.0) + 2.0 ** -20 * np.abs(yi)
    outs, errs, c = [], [], 0
    for s, width in enumerate(sections):
        ys, es = y[:, c:c + width], err[:, c:c + width]
        c += width
        if s < norm_sections:
            h, eh = ys.reshape(R, -1, norm_dim), es.reshape(R, -1, norm_dim)
            n = np.sqrt((h * h).sum(-1, keepdims=True) + EPS)
            eh = eh / n + np.abs(h) / n * (np.sqrt((eh * eh).sum(-1, keepdims=True)) / n + 2.0 ** -20)
            ys, es = (h / n).reshape(R, width), eh.reshape(R, width)
        outs.append(ys)
        errs.append(es)
    return outs, errs, last


def ssm_inputs(seed, B, T, Hk, HV, K, V, dtype, N=None, z=True, D=True, h0=True, fast=0.0):
    """fast: added to dt before the softplus (strong decays)."""
    p = dict(x=randn(seed, B, T, HV, V, dtype=dtype), dt=(randn(seed + 1, B, T, HV) + fast).to(dtype),
             Bm=randn(seed + 2, B, T, Hk, K, dtype=dtype), Cm=randn(seed + 3, B, T, Hk, K, dtype=dtype, scale=K ** -0.5),
             A_log=randn(seed + 4, HV, scale=0.5), dt_bias=randn(seed + 5, HV) - 3.0,
             D=randn(seed + 6, HV) if D else None, z=randn(seed + 7, B, T, HV, V, dtype=dtype) if z else None,
             h0=randn(seed + 8, N or B, HV, V, K, scale=0.3) if h0 else None)
    return p


def ssm_ref(p, lens, softplus=True):
    """Packed rows of p (B x T flattened), sequence by sequence.  Returns (y, y's
    absolute sum times |silu z|, ht, ht's absolute sum)."""
    e = edges(lens)
    flat = lambda n: None if p[n] is None else f64(p[n]).reshape(-1, *p[n].shape[2:])
    x, dt, B, C, z = (flat(n) for n in ("x", "dt", "Bm", "Cm", "z"))
    A, bias, D = f64(p["A_log"]), f64(p["dt_bias"]), None if p["D"] is None else f64(p["D"])
    y, mag, hs, hm = np.zeros(x.shape), np.zeros(x.shape), [], []
    for i in range(len(lens)):
        r = slice(e[i], e[i + 1])
        h0 = None if p["h0"] is None else f64(p["h0"])[i]
        y[r], S = oracle.ssm_scan(x[r], dt[r], B[r], C[r], A, D, None if z is None else z[r], bias, h0, softplus)
        m, M = oracle.ssm_scan(np.abs(x[r]), dt[r], np.abs(B[r]), np.abs(C[r]), A, None, None, bias,
                               None if h0 is None else np.abs(h0), softplus)
        mag[r] = m if z is None else m * np.abs(oracle.silu(z[r]))
        hs.append(S)
        hm.append(M)
    skip = 0.0
    if D is not None:
        skip = np.abs(D[:, None] * x) * (1.0 if z is None else np.abs(oracle.silu(z)))
    return y, mag, skip, np.stack(hs), np.stack(hm)


def ssm_bound(dtype, y, mag, skip):
    b = 512 * U * mag + 2.0 ** -20 * (mag + skip)
    if dtype == BF:
        b = b + 2 * 2.0 ** -8 * mag
    return b + store(dtype, y)


def bits(t):
    t = t.contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(got, ref, what):
    for i, (x, y) in enumerate(zip(got, ref)):
        assert torch.equal(bits(x), bits(y)), f"{what}: output {i} differs"
