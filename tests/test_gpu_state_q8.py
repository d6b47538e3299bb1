"""GPU tests of the 8-bit state cache: codes and scales bit for bit against the
oracle, and everything the indices may name."""

import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_61_amd import binding
from tests.mixer_cases import BF, DEV, bits, d, f64, randn

pytestmark = pytest.mark.gpu
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _states(seed, n, HV, V, K, dtype):
    x = randn(seed, n, HV, V, K) * torch.exp(3 * randn(seed + 1, n, HV, V, 1))
    f = x.view(-1, K)
    f[0] = 0
    f[1] = 1e-45
    f[2] = 2.0 ** -130
    f[3] = torch.linspace(-3.3e38, 3.3e38, K)
    f[4] = torch.arange(K) - 0.5          # ties: max 127 - 0.5 or 63 - 0.5
    f[5] = (torch.arange(K) % 16 + 0.5) * 2
    f[5, 0] = 127.0                       # scale close to 1: ties of the code itself
    f[6] = 448.0
    f[7, 1:] = 0
    f[7, 0] = 449.0
    return x.to(dtype)


def _store(x, form, pool, src=None, dst=None):
    n, HV, V, K = x.shape
    q8 = torch.full((pool, HV, V, K), 3, device=DEV).to(CODE[form])
    sc = torch.full((pool, HV, V), 7.0, device=DEV)
    binding.state_store_q8(d(x), q8, sc, src, dst)
    torch.cuda.synchronize()
    return q8, sc


def _num(q8):
    return q8.cpu().float().double().numpy()


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("HV,V,K", [(1, 16, 64), (3, 128, 128), (2, 5, 128), (1, 9, 64)])
def test_store_bit_exact(form, dtype, HV, V, K):
    print(f"q8 store {form} {dtype} HV={HV} V={V} K={K}", flush=True)
    x = _states(HV * K, 4, HV, V, K, dtype)
    q8, sc = _store(x, form, 4)
    codes, scale = oracle.quantise_state(f64(x), form)
    assert np.array_equal(sc.cpu().double().numpy(), scale, equal_nan=True)   # row 3 overflows in its making
    assert np.array_equal(_num(q8), codes)


@pytest.mark.parametrize("form,dtype,K", [("int8", BF, 64), ("int8", torch.float32, 128), ("e4m3", torch.float32, 64),
                                          ("e4m3", BF, 128)])
def test_store_of_many_rows(form, dtype, K):
    """Over 2^17 rows, the last work-group's half empty; read back."""
    print(f"q8 store many {form} {dtype} K={K}", flush=True)
    x = _states(K, 1, 3, 43693, K, dtype)
    q8, sc = _store(x, form, 2, dst=torch.tensor([1], dtype=torch.int32, device=DEV))
    codes, scale = oracle.quantise_state(f64(x), form)
    assert np.array_equal(sc[1:].cpu().double().numpy(), scale, equal_nan=True)
    assert np.array_equal(_num(q8[1:]), codes)
    assert torch.all(q8[0].float() == 3) and torch.all(sc[0] == 7)
    out = binding.state_load_q8(q8, sc, torch.zeros(x.shape, dtype=dtype, device=DEV),
                                torch.tensor([1], dtype=torch.int32, device=DEV))
    want = (q8[1:].float() * sc[1:, ..., None]).to(dtype)
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want))


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_load_is_code_times_scale(form, dtype):
    print(f"q8 load {form} {dtype}", flush=True)
    x = _states(9, 3, 2, 128, 64, torch.float32)
    q8, sc = _store(x, form, 3)
    out = binding.state_load_q8(q8, sc, torch.full(x.shape, 9.0, dtype=dtype, device=DEV))
    want = (q8.float() * sc[..., None]).to(dtype)
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want))
    # and near the state: half a step of the row's scale, or of e4m3's grid
    err = np.abs(f64(out) - f64(x))
    s = sc.cpu().double().numpy()[..., None]
    step = 0.5 * s if form == "int8" else np.maximum(2.0 ** -4 * np.abs(f64(x)), 2.0 ** -10 * s)
    ok = np.broadcast_to(np.isfinite(s), err.shape)
    step = np.broadcast_to(step, err.shape)[ok]
    assert np.all(err[ok] <= step * (1 + 2.0 ** -20) + (2.0 ** -8 if dtype == BF else 2.0 ** -24) * (np.abs(f64(x))[ok] + step))


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_broken_rows_read_back_as_nan(form):
    print(f"q8 broken rows {form}", flush=True)
    x = randn(3, 1, 1, 8, 64)
    x[0, 0, 2, 5] = float("inf")
    x[0, 0, 4, 0] = float("nan")
    x[0, 0, 6, 63] = float("-inf")
    q8, sc = _store(x, form, 1)
    out = binding.state_load_q8(q8, sc, torch.zeros(x.shape, device=DEV)).cpu()
    bad = torch.tensor([i in (2, 4, 6) for i in range(8)])
    assert torch.all(torch.isnan(out[0, 0, bad])) and torch.all(torch.isfinite(out[0, 0, ~bad]))
    assert torch.equal(torch.isnan(sc.cpu()[0, 0]), bad)


@pytest.mark.parametrize("src,dst,pool", [
    ([2, 0, 2, 1], [5, 1, 0, 3], 6),        # one state into two slots, any order
    ([0, -1, 3, 1], [0, 1, 2, 6], 6),       # a source below, one past the entries, a target past the pool
    (None, [4, 2, 0], 5),
    ([1, 1, 2], None, 3),
])
def test_indices(src, dst, pool):
    print(f"q8 indices {src} {dst}", flush=True)
    x = randn(5, 3, 2, 64, 128)
    t = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)
    q8, sc = _store(x, "int8", pool, t(src), t(dst))
    codes, scale = oracle.quantise_state(f64(x), "int8")
    want, ws = np.full((pool, 2, 64, 128), 3.0), np.full((pool, 2, 64), 7.0)
    n = len(src or dst)
    for s, e in zip(src or range(n), dst or range(n)):
        if 0 <= s < 3 and 0 <= e < pool:
            want[e], ws[e] = codes[s], scale[s]
    assert np.array_equal(_num(q8), want) and np.array_equal(sc.cpu().double().numpy(), ws)
    # the way back, the same pairs: entries nobody names stay
    back = torch.full(x.shape, 11.0, device=DEV)
    binding.state_load_q8(q8, sc, back, t(dst), t(src) if src is None or len(set(src)) == len(src) else t(range(n)))
    torch.cuda.synchronize()
    if src is None:
        for s, e in zip(range(n), dst):
            assert torch.equal(back[s], q8[e].float() * sc[e][..., None])


def test_cache_offsets_past_32_bits():
    """A cache of 4.6 GB of codes: the last slot lies past 4 GiB."""
    print("q8 offsets past 4 GiB", flush=True)
    pool, HV = 8800, 32
    q8 = torch.zeros((pool, HV, 128, 128), dtype=torch.int8, device=DEV)
    sc = torch.zeros((pool, HV, 128), device=DEV)
    x = randn(8, 2, HV, 128, 128)
    idx = torch.tensor([pool - 1, 17], dtype=torch.int32, device=DEV)
    binding.state_store_q8(d(x), q8, sc, dst_indices=idx)
    out = binding.state_load_q8(q8, sc, torch.zeros((2, HV, 128, 128), device=DEV), src_indices=idx)
    torch.cuda.synchronize()
    codes, scale = oracle.quantise_state(f64(x), "int8")
    assert np.array_equal(_num(q8[pool - 1]), codes[0]) and np.array_equal(_num(q8[17]), codes[1])
    assert torch.equal(out[0], q8[pool - 1].float() * sc[pool - 1][..., None])
    named = torch.zeros(pool, dtype=torch.bool, device=DEV)
    named[idx.long()] = True
    assert not sc[~named].any()
    del q8
    torch.cuda.empty_cache()


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("src,dst,pool,entries", [
    ([2, 0, 2, 1], [5, 1, 0, 3], 3, 6),           # one slot into two entries, any order
    ([0, -1, 3, 1, 2], [0, 1, 2, 6, -2], 3, 6),   # slots and entries outside their arrays, on either side
    ([2, 0, -7], None, 3, 5),                     # targets 0, 1, 2 of 5
    (None, [4, 2, 0], 3, 5),
    (None, [1, 9], 3, 2),
    (None, None, 4, 3),
    ([0, 2147483647, -2147483648], [2, 0, 1], 3, 3),
])
def test_load_indices(form, dtype, src, dst, pool, entries):
    """Slot src[i] into entry dst[i] where both exist, every other entry as it was."""
    print(f"q8 load indices {form} {dtype} {src} {dst}", flush=True)
    x = randn(6, pool, 2, 64, 128)
    t = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)
    q8, sc = _store(x, form, pool)
    out = torch.full((entries, 2, 64, 128), 11.0, dtype=dtype, device=DEV)
    want = out.clone()
    value = (q8.float() * sc[..., None]).to(dtype)
    n = len(src if src is not None else dst if dst is not None else range(entries))
    for s, e in zip(src or range(n), dst or range(n)):
        if 0 <= s < pool and 0 <= e < entries:
            want[e] = value[s]
    got = binding.state_load_q8(q8, sc, out, t(src), t(dst))
    torch.cuda.synchronize()
    assert got is out and torch.equal(bits(out), bits(want))
