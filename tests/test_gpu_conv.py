"""GPU parity of the short causal convolution (prompts and single tokens)
against the fp64 oracle, at the sizes where its runs, sequences and states meet."""

import numpy as np
import pytest
import torch

from gated_delta_rule_61_amd import binding
from tests.mixer_cases import BF, DEV, EPS, bits, close, conv_ref, d, edges, f64, randn, same, store

pytestmark = pytest.mark.gpu
F32 = torch.float32

# (dtype, W, lengths or (B, T), sections, norm_dim, norm_sections, silu, bias, state, padding columns)
CASES = [
    (BF, 4, [1], (8,), 0, 0, True, False, True, 0),
    (BF, 4, [17, 0, 1, 2, 3, 40, 0], (64, 64, 128), 64, 2, True, False, True, 24),
    (F32, 4, [5, 16, 31, 0, 0, 1], (128, 128, 264), 128, 2, True, True, True, 8),
    (BF, 3, (3, 33), (520,), 0, 0, False, True, False, 0),
    (F32, 2, (2, 1), (512, 16), 0, 0, True, True, True, 0),
    (BF, 2, [100], (1024, 8, 8), 128, 1, True, True, True, 40),
    (BF, 4, [2] * 40, (72,), 0, 0, True, True, True, 0),                 # every sequence shorter than the taps
    (F32, 3, [15, 1, 1, 15, 64, 7], (24, 40), 0, 0, False, False, True, 0),
    (BF, 4, (4, 16), (256, 256, 512), 128, 3, True, False, True, 0),
    (BF, 4, [3] * 300 + [29], (16,), 0, 0, True, False, True, 0),        # more sequences than a wave has lanes
    (BF, 4, [7, 15990, 0, 1, 2, 4003], (64, 8), 64, 1, True, True, True, 0),     # enough tokens for runs of 8
    (F32, 4, [16, 33000, 15, 1, 0, 3, 7002, 1], (24,), 0, 0, True, False, True, 8),   # ... of 16
]


def _inputs(case, seed=10):
    dtype, W, lens, sections, nd, ns, act, bias, state, pad = case
    dense = isinstance(lens, tuple)
    B, T = lens if dense else (1, sum(lens))
    seqs = [T] * B if dense else lens
    D, N = sum(sections), len(seqs)
    wide = randn(seed, B, T, D + pad, dtype=dtype)
    pool = randn(seed + 1, N + 2, W - 1, D, dtype=dtype)
    slots = torch.randperm(N + 2, generator=torch.Generator().manual_seed(seed))[:N].to(torch.int32)
    has = (torch.arange(N) % 3 != 1).to(torch.int32)
    return dict(wide=wide, w=randn(seed + 2, D, W, dtype=dtype), bias=randn(seed + 3, D, dtype=dtype) if bias else None,
                pool=pool if state else None, slots=slots, has=has, seqs=seqs, dense=dense, D=D, N=N, B=B, T=T)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}-W{c[1]}-{len(c[2])}seq-{sum(c[3])}")
def test_conv_fwd(case):
    dtype, W, lens, sections, nd, ns, act, bias, state, pad = case
    print(f"conv fwd {case[:6]}", flush=True)
    p = _inputs(case)
    cu = None if p["dense"] else torch.tensor(edges(p["seqs"]), dtype=torch.int64, device=DEV)
    pool = d(p["pool"])
    kw = dict(state=pool, state_indices=d(p["slots"]), has_state=d(p["has"])) if state else {}
    got = binding.causal_conv_fwd(d(p["wide"])[..., :p["D"]], d(p["w"]), d(p["bias"]), activation="silu" if act else None,
                                  sections=sections, norm_dim=nd, norm_sections=ns, norm_eps=EPS, cu_seqlens=cu, **kw)
    torch.cuda.synchronize()
    states = [f64(p["pool"][int(s)]) if state and h else None for s, h in zip(p["slots"], p["has"])]
    x = f64(p["wide"])[..., :p["D"]].reshape(-1, p["D"])
    outs, errs, last = conv_ref(x, f64(p["w"]), None if p["bias"] is None else f64(p["bias"]), p["seqs"], states, act,
                                sections, nd, ns)
    for i, (g, r, e) in enumerate(zip(got, outs, errs)):
        close(f"section {i}", g.reshape(-1, sections[i]), r, e + store(dtype, r))
    if state:   # rows of x and of the state as they are; slots nobody names untouched
        want = f64(p["pool"]).copy()
        for s, l in zip(p["slots"], last):
            want[int(s)] = l
        assert np.array_equal(f64(pool), want)


def test_conv_fwd_without_sections_and_rows_behind_the_last_sequence():
    print("conv fwd padded batch", flush=True)
    x, w = randn(1, 1, 50, 32, dtype=BF), randn(2, 32, 4, dtype=BF)
    cu = torch.tensor([0, 7, 30], dtype=torch.int64, device=DEV)
    out = torch.full((1, 50, 32), 5.0, dtype=BF, device=DEV)
    res = binding.causal_conv_fwd(d(x), d(w), cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    assert res is out
    assert torch.all(out[:, 30:] == 5.0)
    (y,), (e,), _ = conv_ref(f64(x)[0, :30], f64(w), None, [7, 23], [None, None], True, (32,), 0, 0)
    close("y", out[0, :30], y, e + store(BF, y))


@pytest.mark.parametrize("cuts", [[20, 1, 2, 61], [3, 0, 81], [84]])
def test_a_prompt_in_parts_is_the_prompt(cuts):
    """Chunked prefill: the same rows in several calls, each from the state the
    last one left, give the same bits as one call."""
    print(f"conv parts {cuts}", flush=True)
    x, w, b = randn(3, 1, 84, 64, dtype=BF), randn(4, 64, 4, dtype=BF), randn(5, 64, dtype=BF)
    one = torch.zeros((3, 3, 64), dtype=BF, device=DEV)
    idx = torch.tensor([2], dtype=torch.int32, device=DEV)
    whole = binding.causal_conv_fwd(d(x), d(w), d(b), state=one, state_indices=idx)
    parts_state, parts, at = torch.zeros_like(one), [], 0
    for i, n in enumerate(cuts):
        has = torch.tensor([int(i > 0)], dtype=torch.int32, device=DEV)
        parts.append(binding.causal_conv_fwd(d(x[:, at:at + n].contiguous()), d(w), d(b), state=parts_state,
                                             state_indices=idx, has_state=has))
        at += n
    torch.cuda.synchronize()
    same([torch.cat(parts, 1), parts_state], [whole, one], f"parts {cuts}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 4])
def test_conv_step(dtype, W, T):
    print(f"conv step {dtype} W={W} T={T}", flush=True)
    B, sections = 5, (64, 8, 128)
    D = sum(sections)
    wide, w, bias = randn(20, B, T, D + 16, dtype=dtype), randn(21, D, W, dtype=dtype), randn(22, D, dtype=dtype)
    base = randn(23, 9, W - 1, D, dtype=dtype)
    idx = torch.tensor([7, 0, -1, 9, 3], dtype=torch.int32, device=DEV)   # two rows outside the pool
    pool = d(base).clone()
    got = binding.causal_conv_step(d(wide)[..., 8:8 + D], d(w), d(bias), pool, idx, sections=sections)
    torch.cuda.synchronize()
    want = f64(base).copy()
    for b, s in enumerate(idx.tolist()):
        if not 0 <= s < 9:
            assert all(torch.all(g[b] == 0) for g in got)
            continue
        outs, errs, last = conv_ref(f64(wide)[b, :, 8:8 + D], f64(w), f64(bias), [T], [f64(base[s])], True, sections, 0, 0)
        for g, r, e in zip(got, outs, errs):
            close(f"row {b}", g[b], r, e + store(dtype, r))
        want[s] = last[0]
    assert np.array_equal(f64(pool), want)


def test_steps_continue_a_prompt():
    """Prompt of 30 rows then 1 + 4 + 2 single tokens = a prompt of 37, bit for bit."""
    print("conv prompt then steps", flush=True)
    x, w = randn(31, 2, 37, 72, dtype=BF), randn(32, 72, 4, dtype=BF)
    a = torch.zeros((2, 3, 72), dtype=BF, device=DEV)
    whole = binding.causal_conv_fwd(d(x), d(w), state=a)
    b = torch.zeros_like(a)
    parts = [binding.causal_conv_fwd(d(x[:, :30].contiguous()), d(w), state=b)]
    for lo, hi in ((30, 31), (31, 35), (35, 37)):
        parts.append(binding.causal_conv_step(d(x)[:, lo:hi], d(w), None, b))
    torch.cuda.synchronize()
    same([torch.cat(parts, 1), b], [whole, a], "steps")


def test_conv_slots_outside_the_pool():
    print("conv slots outside", flush=True)
    x, w = randn(41, 3, 9, 16, dtype=BF), randn(42, 16, 4, dtype=BF)
    base = randn(43, 4, 3, 16, dtype=BF)
    pool = d(base).clone()
    idx = torch.tensor([-1, 2, 4], dtype=torch.int32, device=DEV)
    one = torch.ones(3, dtype=torch.int32, device=DEV)
    got = binding.causal_conv_fwd(d(x), d(w), state=pool, state_indices=idx, has_state=one)
    fresh = binding.causal_conv_fwd(d(x), d(w))
    torch.cuda.synchronize()
    same([got[0], got[2]], [fresh[0], fresh[2]], "rows whose slot is outside start from zeros")
    assert not torch.equal(got[1, 0], fresh[1, 0])
    keep = [0, 1, 3]
    assert torch.equal(bits(pool.cpu()[keep]), bits(base[keep]))
    assert torch.equal(bits(pool[2]), bits(d(x)[1, -3:]))


def test_infinities_stay_in_their_sequence_and_channel():
    print("conv infinities", flush=True)
    x, w = randn(51, 1, 24, 32, dtype=F32), randn(52, 32, 4, dtype=F32)
    cu = torch.tensor([0, 10, 24], dtype=torch.int64, device=DEV)
    clean = binding.causal_conv_fwd(d(x), d(w), cu_seqlens=cu)
    x[0, 9, 5] = float("inf")
    x[0, 8, 6] = float("nan")
    dirty = binding.causal_conv_fwd(d(x), d(w), cu_seqlens=cu)
    torch.cuda.synchronize()
    hit = torch.zeros(1, 24, 32, dtype=torch.bool)
    hit[0, 9, 5] = hit[0, 8:10, 6] = True
    assert torch.equal(bits(clean.cpu()[~hit]), bits(dirty.cpu()[~hit]))


def test_conv_offsets_past_32_bits():
    """x and out of 4.6 GB each: the last sequence of a packed batch lies past 4 GiB."""
    print("conv offsets past 4 GiB", flush=True)
    D, T = 8192, 280000
    x = torch.zeros((1, T, D), dtype=BF, device=DEV)
    tail, w = randn(61, 1, 50, D, dtype=BF), randn(62, D, 4, dtype=BF)
    x[:, -50:] = d(tail)
    cu = torch.tensor([0, T - 50, T], dtype=torch.int64, device=DEV)
    y = binding.causal_conv_fwd(x, d(w), cu_seqlens=cu)
    alone = binding.causal_conv_fwd(d(tail), d(w))
    torch.cuda.synchronize()
    assert torch.equal(bits(y[:, -50:]), bits(alone))
    assert not y[:, :-50].any()
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm_dim", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_heads_whose_squares_leave_fp32(dtype, norm_dim, eps):
    """Heads of 1e-30 to 1e37: the squares under- or overflow, the norms do not."""
    print(f"conv norm of tiny and huge heads {dtype} {norm_dim} eps={eps}", flush=True)
    size = [1e-30, 1e-21, 1e-19, 1.0, 1e18, 1e20, 1e30, 1e37]
    B, T, sec = len(size), 3, (2 * norm_dim, norm_dim, 40)
    x = (randn(1500, B, T, sum(sec)) * torch.tensor(size)[:, None, None]).to(dtype)
    w = randn(1501, sum(sec), 2, dtype=dtype, scale=0.5)
    outs = binding.causal_conv_fwd(d(x), d(w), activation=None, sections=sec, norm_dim=norm_dim, norm_sections=2,
                                   norm_eps=eps)
    torch.cuda.synchronize()
    x64, w64 = f64(x), f64(w)
    past = np.concatenate([np.zeros((B, 1, sum(sec))), x64[:, :-1]], 1)
    y = w64[:, 0] * past + w64[:, 1] * x64
    err = 3 * 2.0 ** -24 * (np.abs(w64[:, 0] * past) + np.abs(w64[:, 1] * x64))     # two products and their sum
    at = 0
    for i, (got, width) in enumerate(zip(outs, sec)):
        r, e = y[..., at:at + width], err[..., at:at + width]
        at += width
        if i < 2:   # as conv_ref: the head's error over its norm, twice, and 2^-20
            h, eh = (a.reshape(B, T, -1, norm_dim) for a in (r, e))
            n = np.sqrt((h * h).sum(-1, keepdims=True) + eps)
            e = (eh / n + np.abs(h) / n * (np.sqrt((eh * eh).sum(-1, keepdims=True)) / n + 2.0 ** -20)).reshape(r.shape)
            r = (h / n).reshape(r.shape)
        close(f"out{i}", got, r, e + store(dtype, r))
