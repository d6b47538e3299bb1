"""Pins of the oracle of the operators around the scans (CPU): the convolution
against torch's conv1d, the selective scan against a closed form, a
degenerate case and the delta-free state scan, the 8-bit storage against
torch's e4m3 cast and exact rational arithmetic."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_is_torch_conv1d(W):
    rng = np.random.default_rng(W)
    x, w, b = rng.standard_normal((9, 5)), rng.standard_normal((5, W)), rng.standard_normal(5)
    y, last, mag = oracle.causal_conv(x, w, b, activation=False)
    ref = torch.nn.functional.conv1d(torch.from_numpy(x.T.copy())[None], torch.from_numpy(w)[:, None], torch.from_numpy(b),
                                     padding=W - 1, groups=5)[0, :, :9].numpy().T
    assert np.allclose(y, ref, rtol=0, atol=1e-13)
    assert np.array_equal(last, x[-(W - 1):])
    assert np.all(mag >= np.abs(y) - 1e-13)
    act, _, _ = oracle.causal_conv(x, w, b)
    assert np.allclose(act, torch.nn.functional.silu(torch.from_numpy(ref)).numpy(), atol=1e-13)


def test_conv_continues_from_its_state():
    rng = np.random.default_rng(7)
    x, w = rng.standard_normal((11, 3)), rng.standard_normal((3, 4))
    whole, last, _ = oracle.causal_conv(x, w)
    for cut in (0, 1, 2, 5, 10):
        a, mid, _ = oracle.causal_conv(x[:cut], w)
        b, end, _ = oracle.causal_conv(x[cut:], w, state=mid)
        assert np.allclose(np.concatenate([a, b]), whole, atol=1e-13)
        assert np.array_equal(end, last)


def test_head_norm_is_torch_normalize():
    y = np.random.default_rng(1).standard_normal((4, 32))
    ref = torch.nn.functional.normalize(torch.from_numpy(y).view(4, 4, 8), dim=-1).view(4, 32).numpy()
    assert np.allclose(oracle.head_norm(y, 8, 0.0), ref, atol=1e-14)


def _ssm(L=13, HV=4, Hk=2, V=3, K=5, seed=0):
    r = np.random.default_rng(seed)
    return dict(x=r.standard_normal((L, HV, V)), dt=r.standard_normal((L, HV)), B=r.standard_normal((L, Hk, K)),
                C=r.standard_normal((L, Hk, K)), A_log=r.standard_normal(HV) * 0.3, D=r.standard_normal(HV),
                z=r.standard_normal((L, HV, V)), dt_bias=r.standard_normal(HV), h0=r.standard_normal((HV, V, K)))


def test_ssm_closed_form():
    """y_t = sum_{s<=t} e^{-rate (cum_t - cum_s)} D_s (B_s . C_t) x_s + the decayed h0, per head."""
    p = _ssm()
    y, S = oracle.ssm_scan(**p)
    step = np.log1p(np.exp(p["dt"] + p["dt_bias"]))
    cum = np.cumsum(step, 0)
    L, HV, V = p["x"].shape
    for h in range(HV):
        g, rate = h // 2, np.exp(p["A_log"][h])
        for t in range(L):
            ref = np.exp(-rate * cum[t, h]) * p["h0"][h] @ p["C"][t, g]
            for s in range(t + 1):
                ref = ref + np.exp(-rate * (cum[t, h] - cum[s, h])) * step[s, h] * (p["B"][s, g] @ p["C"][t, g]) * p["x"][s, h]
            ref = (ref + p["D"][h] * p["x"][t, h]) * p["z"][t, h] / (1 + np.exp(-p["z"][t, h]))
            assert np.allclose(y[t, h], ref, atol=1e-12)
        end = np.exp(-rate * cum[-1, h]) * p["h0"][h]
        for s in range(L):
            end = end + np.exp(-rate * (cum[-1, h] - cum[s, h])) * step[s, h] * np.outer(p["x"][s, h], p["B"][s, g])
        assert np.allclose(S[h], end, atol=1e-12)


def test_ssm_state_is_the_decay_only_state_scan():
    p = _ssm(L=70, HV=2, Hk=1, V=4, K=4)
    step = p["dt"] ** 2
    _, S = oracle.ssm_scan(p["x"], step, p["B"], p["C"], p["A_log"], softplus=False, h0=p["h0"])
    v = (step[..., None] * p["x"])[None]
    g = (-np.exp(p["A_log"]) * step)[None]
    _, ht = oracle.state_scan(p["B"][None], v, g=g, h0=p["h0"][None], split_size=64)
    assert np.allclose(ht[0], S, atol=1e-12)


def test_ssm_empty_and_no_decay():
    p = _ssm(L=5, HV=2, Hk=2)
    y, S = oracle.ssm_scan(*(p[n][:0] for n in ("x", "dt", "B", "C")), p["A_log"], h0=p["h0"][:2])
    assert y.shape[0] == 0 and np.array_equal(S, p["h0"][:2])
    # a rate of (almost) nothing: a plain causal product
    y, _ = oracle.ssm_scan(p["x"], np.ones((5, 2)), p["B"], p["C"], np.full(2, -80.0), softplus=False)
    for h in range(2):
        full = np.tril(p["C"][:, h] @ p["B"][:, h].T) @ p["x"][:, h]
        assert np.allclose(y[:, h], full, atol=1e-12)


def _rows(seed, n=200, K=64):
    r = np.random.default_rng(seed)
    x = (r.standard_normal((n, K)) * np.exp(4 * r.standard_normal((n, 1)))).astype(np.float32)
    x[0] = 0
    x[1] = np.float32(1e-45)
    x[2, 3] = np.inf
    x[3, 5] = np.nan
    x[4] = np.linspace(-3.4e38, 3.4e38, K).astype(np.float32)
    x[5] = np.float32(2.0 ** -130)
    return x


def test_int8_storage_is_exact_rounding():
    x = _rows(3)
    codes, scale = oracle.quantise_state(x, "int8")
    assert np.isnan(scale[2]) and np.isnan(scale[3]) and not codes[2].any() and not codes[3].any()
    assert not codes[0].any() and scale[0] == 2.0 ** -126
    assert np.abs(codes).max() <= 127
    for i in (4, 5, 6, 50, 120):
        s = Fraction(float(scale[i]))
        for v, c in zip(x[i], codes[i]):
            q = Fraction(float(v)) / s
            lo = q.numerator // q.denominator
            frac = q - lo
            near = lo if frac < Fraction(1, 2) or (frac == Fraction(1, 2) and lo % 2 == 0) else lo + 1
            assert near == c


def test_e4m3_storage_is_torch_cast():
    x = _rows(4)
    codes, scale = oracle.quantise_state(x, "e4m3")
    assert np.isnan(scale[2]) and np.isnan(scale[3])
    good = np.isfinite(scale)
    m, e = np.frexp(scale[good])
    assert np.all(m == 0.5)
    most = np.abs(x[good].astype(np.float64)).max(-1)
    assert np.all(most <= 448 * scale[good])
    assert np.all((most > 224 * scale[good]) | (scale[good] == 2.0 ** -126))
    u = torch.from_numpy(x[good].astype(np.float64) / scale[good][:, None])
    assert np.array_equal(codes[good], u.to(torch.float8_e4m3fn).double().numpy())
