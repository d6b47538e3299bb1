"""GPU parity of the selective state-space scan (prompts) and step (single
tokens) against the fp64 oracle."""

import numpy as np
import pytest
import torch

from gated_delta_rule_61_amd import binding
from tests.mixer_cases import BF, DEV, U, bits, close, d, edges, f64, randn, same, ssm_bound, ssm_inputs, ssm_ref, store

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _run(p, **kw):
    return binding.ssm_chunk_fwd(*(d(p[n]) for n in ("x", "dt", "Bm", "Cm", "A_log")), D=d(p["D"]), z=d(p["z"]),
                                 dt_bias=d(p["dt_bias"]), h0=d(p["h0"]), **kw)


def _check(p, lens, dtype, softplus=True, **kw):
    y, ht = _run(p, dt_softplus=softplus, **kw)
    torch.cuda.synchronize()
    ry, mag, skip, rh, hm = ssm_ref(p, lens, softplus)
    close("y", y.reshape(-1, *y.shape[2:]), ry, ssm_bound(dtype, ry, mag, skip))
    close("ht", ht, rh, 512 * U * hm + 2.0 ** -20 * hm)


# (dtype, lengths or (B, T), Hk, HV, K, V, z, D, h0)
CASES = [
    (BF, [64, 1, 63, 0, 65, 130, 2], 1, 4, 128, 64, True, True, True),
    (F32, [64, 1, 63, 0, 65, 130, 2], 1, 4, 128, 64, True, True, True),
    (BF, (2, 100), 3, 3, 64, 64, False, True, False),       # odd number of heads a group: one head a work-group
    (F32, (2, 100), 3, 3, 64, 64, False, True, False),
    (BF, (1, 200), 2, 4, 64, 128, True, False, True),
    (F32, (1, 129), 2, 4, 128, 128, False, False, True),
    (BF, (3, 70), 2, 2, 128, 128, True, True, False),
    (F32, (3, 1), 1, 2, 64, 64, True, True, True),
    (BF, (5, 1), 1, 6, 128, 64, True, True, True),
    (BF, [3] * 150, 1, 2, 64, 64, False, False, True),      # more sequences than a wave has lanes
    (F32, [0, 0], 1, 2, 64, 128, False, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}-{len(c[1])}seq-{c[2]}x{c[3]}-K{c[4]}V{c[5]}")
def test_scan(case):
    dtype, lens, Hk, HV, K, V, z, D, h0 = case
    print(f"scan {case}", flush=True)
    dense = isinstance(lens, tuple)
    B, T = lens if dense else (1, sum(lens))
    seqs = [T] * B if dense else lens
    p = ssm_inputs(100, B, T, Hk, HV, K, V, dtype, N=len(seqs), z=z, D=D, h0=h0)
    cu = None if dense else torch.tensor(edges(seqs), dtype=torch.int64, device=DEV)
    _check(p, seqs, dtype, cu_seqlens=cu)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [(1, 2200), [1500, 0, 40, 700, 1], (2, 1025)])
def test_scan_split_into_segments(dtype, lens):
    """Few sequences and heads: short segments and their join."""
    dense = isinstance(lens, tuple)
    B, T = lens if dense else (1, sum(lens))
    seqs = [T] * B if dense else lens
    print(f"scan split {dtype} {lens}", flush=True)
    assert binding.ssm_workspace_bytes(B, T, 1, 2, 64, 64, len(seqs), dtype, varlen=not dense) > 0
    p = ssm_inputs(200, B, T, 1, 2, 64, 64, dtype, N=len(seqs))
    cu = None if dense else torch.tensor(edges(seqs), dtype=torch.int64, device=DEV)
    _check(p, seqs, dtype, cu_seqlens=cu)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_split_scan_reads_no_workspace_it_has_not_written(dtype):
    """Long sequences among more short ones than a wave has lanes, over a
    workspace of NaN; without ht the last segments' states are nobody's."""
    print(f"scan split over a poisoned workspace {dtype}", flush=True)
    seqs = [3] * 70 + [300] + [5, 0] * 35 + [200, 0, 129, 64]
    T, Hk, HV, K, V = sum(seqs), 1, 2, 128, 64
    p = ssm_inputs(140, 1, T, Hk, HV, K, V, dtype, N=len(seqs))
    cu = torch.tensor(edges(seqs), dtype=torch.int64, device=DEV)
    nbytes = binding.ssm_workspace_bytes(1, T, Hk, HV, K, V, len(seqs), dtype, varlen=True)
    assert nbytes > 0
    ry, mag, skip, rh, hm = ssm_ref(p, seqs, True)
    bound = ssm_bound(dtype, ry, mag, skip)
    runs = []
    for fill, ht_too in ((0xFF, True), (0, True), (0xFF, False)):
        ws = torch.full((nbytes + 64,), fill, dtype=torch.uint8, device=DEV)
        y, ht = _run(p, cu_seqlens=cu, workspace=ws[:nbytes], output_final_state=ht_too)
        torch.cuda.synchronize()
        close("y", y.reshape(-1, *y.shape[2:]), ry, bound)
        assert torch.all(ws[nbytes:] == fill)
        if ht_too:
            close("ht", ht, rh, 512 * U * hm + 2.0 ** -20 * hm)
            runs.append([y, ht])
        else:
            assert ht is None
    same(*runs, "0xFF against zeroed workspace")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fast", [6.0, 25.0, -12.0])
def test_scan_strong_and_weak_decays(dtype, fast):
    """Step sizes of several units (every factor underflows within a chunk or a
    segment), past the softplus threshold, and of 1e-7 (nothing decays)."""
    print(f"scan decays {dtype} {fast}", flush=True)
    p = ssm_inputs(300, 1, 700, 1, 2, 64, 64, dtype, fast=fast)
    _check(p, [700], dtype)


def test_scan_without_softplus_and_final_state():
    print("scan plain dt", flush=True)
    p = ssm_inputs(400, 2, 90, 1, 2, 128, 64, F32)
    p["dt"], p["dt_bias"] = p["dt"].abs() * 0.1, torch.zeros(2)
    p["dt"][0, 5] = 0.0           # a token that leaves the state alone and adds nothing
    _check(p, [90, 90], F32, softplus=False)
    y, ht = _run(p, dt_softplus=False, output_final_state=False)
    assert ht is None
    same([y], [_run(p, dt_softplus=False)[0]], "without the final state")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_takes_slices(dtype):
    """x, B, C side by side in one tensor, z and dt in another, as a layer has them."""
    print(f"scan slices {dtype}", flush=True)
    B, T, Hk, HV, K, V = 2, 77, 2, 4, 64, 64
    xbc, zdt = randn(1, B, T, HV * V + 2 * Hk * K + 32, dtype=dtype), randn(2, B, T, HV * V + 16, dtype=dtype)
    p = ssm_inputs(500, B, T, Hk, HV, K, V, dtype)
    p["x"] = xbc[..., :HV * V].unflatten(-1, (HV, V))
    p["Bm"] = xbc[..., HV * V:HV * V + Hk * K].unflatten(-1, (Hk, K))
    p["Cm"] = xbc[..., HV * V + Hk * K:HV * V + 2 * Hk * K].unflatten(-1, (Hk, K))
    p["z"], p["dt"] = zdt[..., :HV * V].unflatten(-1, (HV, V)), zdt[..., HV * V:HV * V + HV]
    gx, gz = d(xbc), d(zdt)
    args = (gx[..., :HV * V].unflatten(-1, (HV, V)), gz[..., HV * V:HV * V + HV],
            gx[..., HV * V:HV * V + Hk * K].unflatten(-1, (Hk, K)),
            gx[..., HV * V + Hk * K:HV * V + 2 * Hk * K].unflatten(-1, (Hk, K)))
    kw = dict(D=d(p["D"]), z=gz[..., :HV * V].unflatten(-1, (HV, V)), dt_bias=d(p["dt_bias"]), h0=d(p["h0"]))
    got = binding.ssm_chunk_fwd(*args, d(p["A_log"]), **kw)
    kw["z"] = kw["z"].contiguous()
    packed = binding.ssm_chunk_fwd(*(a.contiguous() for a in args), d(p["A_log"]), **kw)
    torch.cuda.synchronize()
    same(got, packed, "slices")
    ry, mag, skip, _, _ = ssm_ref(p, [T] * B)
    close("y", got[0].reshape(-1, HV, V), ry, ssm_bound(dtype, ry, mag, skip))


def test_scan_leaves_rows_behind_the_last_sequence():
    print("scan padded batch", flush=True)
    p = ssm_inputs(600, 1, 150, 1, 2, 64, 64, BF, N=2)
    for n in ("x", "Bm", "Cm", "z"):
        p[n][:, 100:] = float("nan")
    cu = torch.tensor([0, 31, 100], dtype=torch.int64, device=DEV)
    out = torch.full((1, 150, 2, 64), 5.0, dtype=BF, device=DEV)
    y, ht = _run(p, cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    assert y is out and torch.all(out[:, 100:] == 5.0)
    q = {n: (v[:, :100] if n in ("x", "dt", "Bm", "Cm", "z") else v) for n, v in p.items()}
    ry, mag, skip, rh, hm = ssm_ref(q, [31, 69])
    close("y", out[0, :100], ry, ssm_bound(BF, ry, mag, skip))
    close("ht", ht, rh, 512 * U * hm + 2.0 ** -20 * hm)


def test_nan_stays_in_its_sequence_and_heads():
    print("scan nan", flush=True)
    p = ssm_inputs(700, 1, 200, 2, 4, 64, 64, BF, N=2)
    cu = torch.tensor([0, 90, 200], dtype=torch.int64, device=DEV)
    clean = _run(p, cu_seqlens=cu)
    p["x"][0, 70, 1, 3] = float("nan")       # sequence 0, head 1, one channel
    p["Bm"][0, 150, 1, 5] = float("inf")     # sequence 1, group 1 (heads 2 and 3)
    dirty = _run(p, cu_seqlens=cu)
    torch.cuda.synchronize()
    y0, y1 = clean[0].cpu(), dirty[0].cpu()
    assert torch.equal(bits(y0[0, :90, [0, 2, 3]]), bits(y1[0, :90, [0, 2, 3]]))
    assert torch.equal(bits(y0[0, :64, 1]), bits(y1[0, :64, 1]))          # the chunk before it
    assert torch.all(torch.isnan(y1[0, 70:90, 1, 3]))
    assert torch.equal(bits(y0[0, 90:, :2]), bits(y1[0, 90:, :2]))
    assert torch.equal(bits(y0[0, 90:150, 2:]), bits(y1[0, 90:150, 2:]))   # token 150 is the first that reads it
    other = [c for c in range(64) if c != 3]
    assert torch.equal(bits(y0[0, :90, 1][:, other]), bits(y1[0, :90, 1][:, other]))
    assert torch.equal(bits(clean[1].cpu()[0, [0, 2, 3]]), bits(dirty[1].cpu()[0, [0, 2, 3]]))


def test_boundaries_out_of_order_stay_in_the_buffers():
    """Nonsense boundaries: results unspecified, nothing outside the buffers is touched."""
    print("scan / conv bad boundaries", flush=True)
    p = ssm_inputs(800, 1, 300, 1, 2, 64, 64, BF, N=5)
    cu = torch.tensor([-40, 280, 20, 700, 3, 300], dtype=torch.int64, device=DEV)
    guard = torch.full((3, 1, 300, 2, 64), 3.0, dtype=BF, device=DEV)
    nbytes = binding.ssm_workspace_bytes(1, 300, 1, 2, 64, 64, 5, BF, varlen=True)
    ws = torch.zeros(nbytes + 4096, dtype=torch.uint8, device=DEV)
    _run(p, cu_seqlens=cu, out=guard[1], workspace=ws[:max(nbytes, 256)] if nbytes else None)
    out = torch.full((3, 1, 300, 128), 3.0, dtype=BF, device=DEV)
    x, w = d(p["x"]).flatten(2), d(randn(801, 128, 4, dtype=BF))
    state = torch.full((3, 5, 3, 128), 3.0, dtype=BF, device=DEV)
    binding.causal_conv_fwd(x, w, cu_seqlens=cu, out=out[1], state=state[1])
    torch.cuda.synchronize()
    assert torch.all(guard[0] == 3) and torch.all(guard[2] == 3) and not ws[nbytes:].any()
    assert torch.all(out[0] == 3) and torch.all(out[2] == 3)
    assert torch.all(state[0] == 3) and torch.all(state[2] == 3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sdt", [BF, F32])
@pytest.mark.parametrize("K,V,T,B", [(64, 64, 1, 5), (128, 64, 4, 3), (64, 128, 2, 4), (128, 128, 3, 3), (128, 128, 1, 300)])
def test_step(dtype, sdt, K, V, T, B):
    print(f"step {dtype} pool {sdt} K={K} V={V} T={T} B={B}", flush=True)
    Hk, HV, n = 1, 2, min(B, 5)
    p = ssm_inputs(900, B, T, Hk, HV, K, V, dtype, h0=False, z=T != 2, D=T != 3)
    base = randn(901, B + 2, HV, V, K, dtype=sdt, scale=0.3)
    idx = torch.randperm(B + 2, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    idx[1] = -1
    idx[2] = B + 2
    pool = d(base).clone()
    y = binding.ssm_step(*(d(p[k]) for k in ("x", "dt", "Bm", "Cm", "A_log")), pool, state_indices=d(idx), D=d(p["D"]),
                         z=d(p["z"]), dt_bias=d(p["dt_bias"]))
    torch.cuda.synchronize()
    assert not y[1].any() and not y[2].any()
    named = {int(i) for i in idx if 0 <= i < B + 2}
    for s in range(B + 2):
        if s not in named:
            assert torch.equal(bits(pool[s]), bits(d(base[s])))
    for b in sorted({*range(n), B - 1} - {1, 2}):
        one = {k: (v[b:b + 1] if v is not None and k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in p.items()}
        one["h0"] = base[int(idx[b])][None].float()
        ry, mag, skip, rh, hm = ssm_ref(one, [T])
        # no operand is rounded here: fp32 throughout, then the storage
        close(f"y[{b}]", y[b], ry, 512 * U * mag + 2.0 ** -20 * (mag + skip) + store(dtype, ry))
        close(f"state[{b}]", pool[int(idx[b])], rh[0], 2.0 ** -20 * hm[0] + store(sdt, rh[0]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_steps_continue_a_prompt(dtype):
    print(f"prompt then steps {dtype}", flush=True)
    p = ssm_inputs(1000, 2, 107, 1, 2, 128, 64, dtype)
    cut = {n: (v[:, :100].contiguous() if v is not None and n in ("x", "dt", "Bm", "Cm", "z") else v) for n, v in p.items()}
    _, ht = _run(cut)
    pool = ht.clone()
    ys = []
    for lo, hi in ((100, 101), (101, 105), (105, 107)):
        a = [d(p[n])[:, lo:hi] for n in ("x", "dt", "Bm", "Cm")]
        ys.append(binding.ssm_step(*a, d(p["A_log"]), pool, D=d(p["D"]), z=d(p["z"])[:, lo:hi], dt_bias=d(p["dt_bias"])))
    torch.cuda.synchronize()
    ry, mag, skip, rh, hm = ssm_ref(p, [107, 107])
    pick = lambda a: a.reshape(2, 107, *a.shape[1:])[:, 100:]
    close("y", torch.cat(ys, 1), pick(ry), 512 * U * pick(mag) + 2.0 ** -20 * (pick(mag) + pick(skip)) + store(dtype, pick(ry)))
    close("state", pool, rh, 512 * U * hm + 2.0 ** -19 * hm)


def test_scan_offsets_past_32_bits():
    """x, z and y of 4.6 GB each; the last sequence lies past 4 GiB and equals the
    same sequence alone."""
    print("scan offsets past 4 GiB", flush=True)
    HV, V, K, T = 64, 64, 64, 560128
    p = ssm_inputs(1100, 1, 130, 1, HV, K, V, BF, h0=False)
    big = {n: torch.zeros((1, T, *p[n].shape[2:]), dtype=BF, device=DEV) for n in ("x", "dt", "Bm", "Cm", "z")}
    for n in big:
        big[n][:, -130:] = d(p[n])
    cu = torch.tensor([0, T - 130, T], dtype=torch.int64, device=DEV)
    y, ht = binding.ssm_chunk_fwd(big["x"], big["dt"], big["Bm"], big["Cm"], d(p["A_log"]), D=d(p["D"]), z=big["z"],
                                  dt_bias=d(p["dt_bias"]), cu_seqlens=cu)
    torch.cuda.synchronize()
    assert big["x"].numel() * 2 > 1 << 32
    ry, mag, skip, rh, hm = ssm_ref(p, [130])
    close("y", y[0, -130:], ry, ssm_bound(BF, ry, mag, skip))
    close("ht", ht[1:], rh, 512 * U * hm + 2.0 ** -20 * hm)
    assert not y[:, :-130].any() and not ht[0].any()
    del big, y
    torch.cuda.empty_cache()


def _fast_rates(seed, B, T, HV, K, V, dtype, N=None):
    """Heads whose rate exp(A_log) passes fp32's largest number, with steps that
    underflow to 0 (dt = -200) or are 2e-35 (-80) among ordinary ones.  (No fp32
    subnormal steps: their own rounding, times such a rate, is no small error.)"""
    p = ssm_inputs(seed, B, T, 1, HV, K, V, dtype, N=N)
    p["A_log"] = torch.tensor([90.0, 0.3, 200.0, 89.0, 64.5, 95.0])[:HV]
    p["dt_bias"] = torch.zeros(HV)
    p["dt"][:, 3::7] = -200.0
    p["dt"][:, 5::11] = -80.0
    p["dt"][:, 20:45] = -200.0     # the state of a long run of such tokens
    return p


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,HV,V", [([100, 1, 64, 70], 4, 64), ([100, 3], 3, 64), ([1000, 0, 40], 1, 64),
                                       ([900], 2, 128), ([700, 33], 2, 64)])
def test_scan_at_rates_past_fp32(dtype, lens, HV, V):
    """A decay of 0, and 1 where the step is 0: also behind the end of a sequence,
    within a chunk and in the chunks that fill up a group of gates."""
    print(f"scan rates past fp32 {dtype} {lens} HV={HV} V={V}", flush=True)
    T = sum(lens)
    p = _fast_rates(1200, 1, T, HV, 64, V, dtype, N=len(lens))
    y, ht = _run(p, cu_seqlens=torch.tensor(edges(lens), dtype=torch.int64, device=DEV))
    torch.cuda.synchronize()
    ry, mag, skip, rh, hm = ssm_ref(p, lens)
    close("y", y[0], ry, ssm_bound(dtype, ry, mag, skip))
    # bf16 io: a step of 2e-35 makes state elements of 1e-36.  Of the three bf16 terms
    # whose products with B form them the second and third are then below 2^-126, where
    # the matrix cores take a bf16 operand as 0: at most 2^-126 |B_s| a term is lost, and
    # decays after it are at most 1.  2^-125 sum_s |B_s| is below 1e-34 here.
    lost = np.zeros_like(hm)
    if dtype == BF:
        e, B = edges(lens), np.abs(f64(p["Bm"])[0, :, 0])
        lost += 2.0 ** -125 * np.stack([B[lo:hi].sum(0) for lo, hi in zip(e, e[1:])])[:, None, None, :]
    close("ht", ht, rh, 512 * U * hm + 2.0 ** -20 * hm + lost)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_step_at_rates_past_fp32(dtype):
    print(f"step rates past fp32 {dtype}", flush=True)
    for row, dt in enumerate((-200.0, -80.0, 0.5)):
        p = _fast_rates(1300 + row, 1, 2, 6, 64, 64, dtype)
        p["dt"][:] = dt
        pool = d(p["h0"]).clone()
        y = binding.ssm_step(*(d(p[k]) for k in ("x", "dt", "Bm", "Cm", "A_log")), pool, D=d(p["D"]), z=d(p["z"]),
                             dt_bias=d(p["dt_bias"]))
        torch.cuda.synchronize()
        ry, mag, skip, rh, hm = ssm_ref(p, [2])
        close(f"y {dt}", y[0], ry, 512 * U * mag + 2.0 ** -20 * (mag + skip) + store(dtype, ry))
        # elements below 2^-126 are 2^-149 apart: three roundings a token (D x, its product
        # with B, the sum), two tokens, half a step each
        close(f"state {dt}", pool, rh, 2.0 ** -20 * hm + store(F32, rh) + 6 * 2.0 ** -150)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_split_sequences_than_a_wave_has_lanes(dtype):
    """70 sequences of two segments among short and empty ones: their states are
    numbered over 64 sequences at a time; the workspace is as large as asked for."""
    print(f"scan many split sequences {dtype}", flush=True)
    seqs = [0, 5, 330] * 20 + [335, 1] * 30 + [3] * 70 + [322] * 20
    T, Hk, HV, K, V = sum(seqs), 1, 1, 64, 64
    p = ssm_inputs(1400, 1, T, Hk, HV, K, V, dtype, N=len(seqs))
    p["dt_bias"] -= 3.0     # slow decays: the first segment's state matters in the second
    nbytes = binding.ssm_workspace_bytes(1, T, Hk, HV, K, V, len(seqs), dtype, varlen=True)
    seg = 320               # 2 sqrt(T) tokens, in chunks of 64
    assert (seg - 64) ** 2 < 4 * T <= seg ** 2 and sum(n > seg for n in seqs) == 70
    assert nbytes <= 2 * (T // seg) * (V * K * 4 + 8) + 512
    ws = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    y, ht = _run(p, cu_seqlens=torch.tensor(edges(seqs), dtype=torch.int64, device=DEV), workspace=ws[:nbytes])
    torch.cuda.synchronize()
    assert torch.all(ws[nbytes:] == 0xFF)
    ry, mag, skip, rh, hm = ssm_ref(p, seqs)
    close("y", y[0], ry, ssm_bound(dtype, ry, mag, skip))
    close("ht", ht, rh, 512 * U * hm + 2.0 ** -20 * hm)


def _part(p, lens, seqs, heads):
    """Sequences and heads of p (packed rows), each head with a group of its own; their lengths."""
    e, per = edges(lens), p["x"].shape[2] // p["Bm"].shape[2]
    rows = np.concatenate([np.arange(e[i], e[i + 1]) for i in seqs])
    groups = [h // per for h in heads]
    flat = lambda n: p[n].reshape(1, -1, *p[n].shape[2:])[:, rows]
    q = {n: flat(n)[:, :, heads] for n in ("x", "dt", "z")} | {n: flat(n)[:, :, groups] for n in ("Bm", "Cm")}
    q |= {n: p[n][heads] for n in ("A_log", "dt_bias", "D")} | {"h0": p["h0"][seqs][:, heads]}
    return q, rows, [lens[i] for i in seqs]


def _check_part(p, lens, dtype, y, ht, seqs, heads):
    q, rows, ql = _part(p, lens, seqs, heads)
    ry, mag, skip, rh, hm = ssm_ref(q, ql)
    close("y", y.reshape(-1, *y.shape[2:])[rows][:, heads], ry, ssm_bound(dtype, ry, mag, skip))
    if ht is not None:
        close("ht", ht[seqs][:, heads], rh, 512 * U * hm + 2.0 ** -20 * hm)


# (lengths or (B, T), Hk, HV, K, V, sequences and heads that are compared)
LONG = [
    ((8, 2100), 2, 8, 128, 64, [0, 7], [1, 6]),                      # two 64-wide heads a work-group
    ((12, 2800), 2, 4, 128, 128, [0, 11], [0, 3]),                   # a 128-wide one
    ((12, 3700), 1, 3, 64, 64, [3, 11], [0, 2]),                     # a 64-wide one (odd group)
    ((12, 2800), 1, 4, 64, 128, [5], [1, 2]),
    ((12, 3700), 3, 3, 128, 64, [11], [1]),
    ([3900] * 7 + [3000, 0, 1, 64, 769, 384, 385, 0, 2000], 2, 4, 128, 128, [6, 7, 8, 9, 10, 11, 12, 13, 14, 15], [0, 2]),
    ([3900] * 7 + [3000, 0, 1, 64, 769, 384, 385, 0, 2000], 2, 4, 64, 64, [6, 7, 8, 9, 10, 11, 12, 13, 14, 15], [1, 3]),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", LONG, ids=lambda c: f"{len(c[0])}seq-{c[1]}x{c[2]}-K{c[3]}V{c[4]}")
def test_split_scan_of_long_segments(case, dtype):
    """Segments of more chunks than a group of gates has (2 for two heads a
    work-group, 4 for one), and slow decays: a token of the first chunk of a
    segment still shows in the state behind it."""
    lens, Hk, HV, K, V, seqs, heads = case
    print(f"scan long segments {dtype} {Hk}x{HV} K={K} V={V}", flush=True)
    dense = isinstance(lens, tuple)
    B, T = lens if dense else (1, sum(lens))
    lens = [T] * B if dense else lens
    group = 2 if V == 64 and HV // Hk % 2 == 0 else 4
    nbytes = binding.ssm_workspace_bytes(B, T, Hk, HV, K, V, len(lens), dtype, varlen=not dense)
    states = nbytes // (HV * (V * K * 4 + 8))
    if dense:   # B ceil(T / segment) states: no shorter segment makes so few
        assert 2 <= states // B < T / (64 * group)
    else:       # floor(T / segment) and that once more, or the number of sequences
        full = states // 2 if states < 2 * len(lens) else states - len(lens)
        assert 2 <= full and T / (full + 1) > 64 * group
    p = ssm_inputs(1600, B, T, Hk, HV, K, V, dtype, N=len(lens))
    p["dt_bias"] -= 3.0
    y, ht = _run(p, cu_seqlens=None if dense else torch.tensor(edges(lens), dtype=torch.int64, device=DEV))
    torch.cuda.synchronize()
    _check_part(p, lens, dtype, y, ht, seqs, heads)


@pytest.mark.parametrize("B,T,HV", [(64, 640, 16), (2, 1100, 4)])
def test_bf16_y_with_and_without_the_final_state(B, T, HV):
    """Not split (ten chunks) and split: within the bound both times, whatever the
    number of terms that the state takes."""
    print(f"scan bf16 without ht B={B} T={T}", flush=True)
    p = ssm_inputs(1700, B, T, 1, HV, 128, 64, BF)
    p["dt_bias"] -= 3.0
    assert (binding.ssm_workspace_bytes(B, T, 1, HV, 128, 64, B, BF) == 0) == (B == 64)
    y, ht = _run(p)
    bare, none = _run(p, output_final_state=False)
    torch.cuda.synchronize()
    assert none is None
    _check_part(p, [T] * B, BF, y, ht, [0, B - 1], [0, HV - 1])
    _check_part(p, [T] * B, BF, bare, None, [0, B - 1], [0, HV - 1])


def test_time_does_not_grow_with_the_square_of_the_sequences():
    """Eight times the packed sequences take about eight times as long (not 64)."""
    print("scan of 2048 and 16384 sequences", flush=True)
    best = []
    for n in (2048, 16384):
        p = {k: d(v) for k, v in ssm_inputs(1800, 1, 8 * n, 1, 4, 128, 64, BF, N=1, h0=False).items()}
        cu = torch.arange(0, 8 * n + 1, 8, dtype=torch.int64, device=DEV)
        run = lambda: _run(p, cu_seqlens=cu, output_final_state=False)
        run()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        times = []
        for _ in range(5):
            a.record()
            run()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        best.append(min(times))
    print(f"{best[0]:.3f} and {best[1]:.3f} ms", flush=True)
    assert best[1] < 20 * best[0]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_prompts_among_thousands_of_short_ones(dtype):
    """Split sequences first, last and among 5000 of 8 tokens, whose bits are those
    of a dense batch of them; the long ones against the oracle."""
    print(f"scan of thousands of sequences {dtype}", flush=True)
    long = {0: 1500, 1: 700, 2600: 2000, 5003: 1200}
    lens = [long.get(i, 8) for i in range(5004)]
    T, HV, K, V = sum(lens), 4, 64, 64
    p = ssm_inputs(1900, 1, T, 1, HV, K, V, dtype, N=len(lens))
    e = edges(lens)
    assert binding.ssm_workspace_bytes(1, T, 1, HV, K, V, len(lens), dtype, varlen=True) > 0
    y, ht = _run(p, cu_seqlens=torch.tensor(e, dtype=torch.int64, device=DEV))
    short = [i for i in range(len(lens)) if i not in long]
    rows = torch.tensor([list(range(e[i], e[i + 1])) for i in short])
    q = {n: (p[n][0, rows] if n in ("x", "dt", "Bm", "Cm", "z") else p[n][short] if n == "h0" else p[n]) for n in p}
    ys, hs = _run(q)
    torch.cuda.synchronize()
    same([y[0, d(rows)], ht[short]], [ys, hs], "short sequences")
    for i in long:
        if i == 2600:
            _check_part(p, lens, dtype, y, ht, [i], [0, 1, 2, 3])
        else:
            _check_part(p, lens, dtype, y, ht, [i], [2])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_and_step_of_rows_far_apart(dtype):
    """Token strides just below the largest: 32-bit offsets within a chunk."""
    print(f"scan of rows far apart {dtype}", flush=True)
    T, Hk, HV, K, V = 66, 1, 2, 64, 64
    p = ssm_inputs(2000, 1, T, Hk, HV, K, V, dtype)
    names, at = ("x", "Bm", "Cm", "z", "dt"), 0
    wide = torch.empty((1, T, (1 << 23) - 8), dtype=dtype, device=DEV)
    far = {}
    for n in names:
        t = d(p[n]).flatten(2)
        wide[..., at:at + t.shape[-1]] = t
        far[n] = wide[..., at:at + t.shape[-1]].view(1, T, *p[n].shape[2:])
        assert far[n].stride(1) == (1 << 23) - 8
        at += t.shape[-1]
    kw = dict(D=d(p["D"]), dt_bias=d(p["dt_bias"]))
    got = binding.ssm_chunk_fwd(*(far[n] for n in ("x", "dt", "Bm", "Cm")), d(p["A_log"]), z=far["z"], h0=d(p["h0"]), **kw)
    want = _run(p)
    pools = [d(p["h0"]).clone() for _ in range(2)]
    got += (binding.ssm_step(*(far[n][:, :4] for n in ("x", "dt", "Bm", "Cm")), d(p["A_log"]), pools[0],
                             z=far["z"][:, :4], **kw), pools[0])
    want += (binding.ssm_step(*(d(p[n])[:, :4] for n in ("x", "dt", "Bm", "Cm")), d(p["A_log"]), pools[1],
                              z=d(p["z"])[:, :4], **kw), pools[1])
    torch.cuda.synchronize()
    same(got, want, "rows far apart")
    del wide, far, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rates_past_fp32_without_softplus(dtype):
    """Steps of 0, 2^-100 and ordinary ones, as they are given."""
    print(f"scan and step, rates past fp32, plain dt {dtype}", flush=True)
    B, T, HV = 2, 150, 5
    p = ssm_inputs(2100, B, T, 1, HV, 64, 64, dtype)
    p["A_log"], p["dt_bias"] = torch.tensor([90.0, 200.0, 0.3, 63.0, 70.0]), torch.zeros(HV)
    p["dt"] = (p["dt"].float().abs() * 0.1).to(dtype)
    p["dt"][:, 2::5], p["dt"][:, 4::9], p["dt"][:, 30:60] = 0.0, 2.0 ** -100, 0.0
    y, ht = _run(p, dt_softplus=False)
    pool = ht.clone()
    q = {n: (p[n][:, 100:104] if n in ("x", "dt", "Bm", "Cm", "z") else p[n]) for n in p}
    ys = binding.ssm_step(*(d(q[n]) for n in ("x", "dt", "Bm", "Cm", "A_log")), pool, D=d(q["D"]), z=d(q["z"]),
                          dt_bias=d(q["dt_bias"]), dt_softplus=False)
    torch.cuda.synchronize()
    ry, mag, skip, rh, hm = ssm_ref(p, [T] * B, softplus=False)
    close("y", y.reshape(-1, HV, 64), ry, ssm_bound(dtype, ry, mag, skip))
    # the bf16 terms of steps of 2^-100 that the matrix cores take as 0, as above
    lost = 2.0 ** -125 * np.abs(f64(p["Bm"])[:, :, 0]).sum(1)[:, None, None] if dtype == BF else 0.0
    close("ht", ht, rh, 512 * U * hm + 2.0 ** -20 * hm + lost)
    q["h0"] = ht.cpu()
    ry, mag, skip, rh, hm = ssm_ref(q, [4] * B, softplus=False)
    close("step y", ys.reshape(-1, HV, 64), ry, 512 * U * mag + 2.0 ** -20 * (mag + skip) + store(dtype, ry))
    close("step state", pool, rh, 2.0 ** -20 * hm + store(F32, rh) + 12 * 2.0 ** -150)   # four tokens, as above
