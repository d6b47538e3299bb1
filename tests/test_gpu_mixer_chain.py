"""The operators around the scans as a server runs them: together, twice the
same, in captured graphs, and on other streams."""

import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_61_amd import binding, workloads
from tests.mixer_cases import (BF, DEV, EPS, bits, close, conv_ref, d, f64, randn, same, ssm_bound, ssm_inputs, ssm_ref,
                               store)
from tests.test_gpu_graphs import _capture, _other_work
from tests.tolerance import check

pytestmark = pytest.mark.gpu


def test_convolution_in_front_of_the_delta_rule():
    """Projection -> convolution, silu and norms -> delta-rule prefill -> handoff;
    then single tokens: convolution step -> decode.  Against the oracle's chain on
    the convolution's own (bf16) outputs."""
    print("conv -> gdn prefill -> handoff -> conv step -> gdn decode", flush=True)
    Hk, HV, K, lens = 2, 4, 128, [70, 0, 33]
    sec = (Hk * K, Hk * K, HV * K)
    D, T, N = sum(sec), sum(lens), len(lens)
    proj, w = randn(1, 1, T, D + 64, dtype=BF), randn(2, D, 4, dtype=BF, scale=0.5)
    gen = torch.Generator().manual_seed(3)
    g, beta = -torch.rand(1, T, HV, generator=gen) * 0.2, torch.rand(1, T, HV, generator=gen)
    cu = torch.tensor([0, 70, 70, 103], dtype=torch.int64)
    conv_pool, slots = torch.zeros((5, 3, D), dtype=BF, device=DEV), torch.tensor([4, 1, 2], dtype=torch.int32, device=DEV)
    q, k, v = binding.causal_conv_fwd(d(proj)[..., :D], d(w), sections=sec, norm_dim=K, norm_sections=2, norm_eps=EPS,
                                      state=conv_pool, state_indices=slots, cu_seqlens=d(cu))
    h = lambda t, n: t.unflatten(-1, (n, K))
    o, ht = binding.gdn_chunk_fwd(h(q, Hk), h(k, Hk), h(v, HV), d(g), d(beta), cu_seqlens=d(cu))
    pool = torch.zeros((5, HV, K, K), dtype=BF, device=DEV)
    binding.state_to_pool(ht, pool, slots)
    torch.cuda.synchronize()
    outs, errs, last = conv_ref(f64(proj)[0, :, :D], f64(w), None, lens, [None] * 3, True, sec, K, 2)
    for got, r, e in zip((q, k, v), outs, errs):
        close("conv", got[0], r, e + store(BF, r))
    norms = np.sqrt((f64(k).reshape(-1, K) ** 2).sum(-1))
    assert np.all(np.abs(norms - 1) < 2.0 ** -8)
    o_ref, ht_ref = oracle.gdn_recurrent(h(q, Hk).cpu(), h(k, Hk).cpu(), h(v, HV).cpu(), g, beta, K ** -0.5, cu_seqlens=cu)
    check("o", o.cpu(), o_ref, BF)
    check("ht", ht.cpu(), ht_ref, BF)
    # one token each
    x1 = randn(5, N, 1, D + 64, dtype=BF)
    a, b, A_log, bias = randn(6, N, 1, HV, dtype=BF), randn(7, N, 1, HV, dtype=BF), randn(8, HV), randn(9, HV)
    before = pool.clone()
    q1, k1, v1 = binding.causal_conv_step(d(x1)[..., :D], d(w), None, conv_pool, slots, sections=sec)
    o1 = binding.gdn_decode(h(q1, Hk), h(k1, Hk), h(v1, HV), d(a), d(b), d(A_log), d(bias), pool, slots)
    torch.cuda.synchronize()
    for n in range(N):
        r, e, _ = conv_ref(f64(x1)[n, :, :D], f64(w), None, [1], [last[n]], True, sec, 0, 0)
        for got, rr, ee in zip((q1, k1, v1), r, e):
            close("conv step", got[n], rr, ee + store(BF, rr))
    o1_ref, s_ref = oracle.gdn_decode(h(q1, Hk).cpu(), h(k1, Hk).cpu(), h(v1, HV).cpu(), a, b, A_log, bias, before.cpu(),
                                      indices=slots.tolist(), scale=K ** -0.5)
    check("decode o", o1.cpu(), o1_ref, BF)
    check("decode state", pool.cpu(), s_ref, BF)


def _layer_inputs(seed, N, T, Hk, HV, K, V):
    c = HV * V + 2 * Hk * K
    p = ssm_inputs(seed, N, T, Hk, HV, K, V, BF, h0=False)
    return dict(xbc=randn(seed + 20, N, T, c, dtype=BF), z=p["z"], dt=p["dt"], A_log=p["A_log"], D=p["D"],
                dt_bias=p["dt_bias"], w=randn(seed + 21, c, 4, dtype=BF, scale=0.5), bias=randn(seed + 22, c, dtype=BF))


def _layer(s, q, Hk, HV, K, V, conv, pool=None, h0=None, has=None):
    """One selective-scan layer over the device tensors s: prompts (pool None) or single tokens."""
    sec = (HV * V, Hk * K, Hk * K)
    if pool is None:
        x, B, C = binding.causal_conv_fwd(s["xbc"], q["w"], q["bias"], sections=sec, state=conv, has_state=has)
    else:
        x, B, C = binding.causal_conv_step(s["xbc"], q["w"], q["bias"], conv, sections=sec)
    a = (x.unflatten(-1, (HV, V)), s["dt"], B.unflatten(-1, (Hk, K)), C.unflatten(-1, (Hk, K)), q["A_log"])
    kw = dict(D=q["D"], z=s["z"], dt_bias=q["dt_bias"])
    if pool is None:
        return binding.ssm_chunk_fwd(*a, h0=h0, **kw)
    return binding.ssm_step(*a, pool, **kw)


def test_prefix_from_the_cache_goes_on_like_the_prompt():
    """A prompt's first part is run, its states go into the 8-bit cache (int8) and
    come back as the initial state of the second part, then single tokens.  The
    state differs by at most half an int8 step a value; with y linear in it, the
    outputs stay within that step's reach of the uninterrupted run's."""
    print("prefix cache chain", flush=True)
    N, Hk, HV, K, V = 2, 1, 4, 128, 64
    p = _layer_inputs(50, N, 170, Hk, HV, K, V)
    q = {n: d(p[n]) for n in ("w", "bias", "A_log", "D", "dt_bias")}
    part = lambda lo, hi: {n: d(p[n][:, lo:hi].contiguous()) for n in ("xbc", "z", "dt")}
    dims = (Hk, HV, K, V)
    conv = torch.zeros((N, 3, HV * V + 2 * Hk * K), dtype=BF, device=DEV)
    y_all, h_all = _layer(part(0, 170), q, *dims, conv.clone())
    _, h1 = _layer(part(0, 100), q, *dims, conv)
    q8 = torch.zeros((6, HV, V, K), dtype=torch.int8, device=DEV)
    sc = torch.zeros((6, HV, V), device=DEV)
    slots = torch.tensor([5, 2], dtype=torch.int32, device=DEV)
    binding.state_store_q8(h1, q8, sc, dst_indices=slots)
    back = binding.state_load_q8(q8, sc, torch.empty_like(h1), src_indices=slots)
    one = torch.ones(N, dtype=torch.int32, device=DEV)
    y2, h2 = _layer(part(100, 166), q, *dims, conv, h0=back, has=one)
    pool = h2.clone()
    y3 = _layer(part(166, 170), q, *dims, conv, pool=pool)
    torch.cuda.synchronize()
    step = (sc[slots.long()] * 0.5)[..., None]
    assert torch.all((back - h1).abs() <= step * (1 + 2.0 ** -20))
    # |y - y'| <= |silu z| (half a step) sum |C| + the bf16 roundings of both runs
    diff = (torch.cat([y2, y3], 1).float() - y_all[:, 100:].float()).abs()
    cmax = 16.0 * K ** 0.5   # |C| after silu: sum over K of values below 16 / sqrt(K) on average
    lim = torch.nn.functional.silu(d(p["z"])[:, 100:].float()).abs() * step.amax(-1)[:, None] * cmax
    assert torch.all(diff <= lim + 2.0 ** -5 * (1 + y_all[:, 100:].float().abs().amax()))
    assert torch.all((pool - h_all).abs() <= step + 2.0 ** -7 * h_all.abs().amax())


def _all_ops(seed):
    """A step of every entry point on fixed buffers; returns (call, buffers to reset)."""
    N, T, Hk, HV, K, V = 3, 300, 1, 4, 128, 64
    p = _layer_inputs(seed, N, T, Hk, HV, K, V)
    s1, s2 = {n: d(p[n]) for n in ("xbc", "z", "dt")}, {n: d(p[n][:, :2].contiguous()) for n in ("xbc", "z", "dt")}
    q = {n: d(p[n]) for n in ("w", "bias", "A_log", "D", "dt_bias")}
    conv0 = d(randn(seed + 30, N, 3, HV * V + 2 * Hk * K, dtype=BF))
    conv, has = conv0.clone(), torch.tensor([1, 0, 1], dtype=torch.int32, device=DEV)
    q8, sc = torch.zeros((N, HV, V, K), dtype=torch.float8_e4m3fn, device=DEV), torch.zeros((N, HV, V), device=DEV)
    pool = torch.zeros((N, HV, V, K), device=DEV)

    def call():
        y, ht = _layer(s1, q, Hk, HV, K, V, conv, has=has)
        binding.state_store_q8(ht, q8, sc)
        binding.state_load_q8(q8, sc, pool)
        y2 = _layer(s2, q, Hk, HV, K, V, conv, pool=pool)
        return y, ht, y2

    def reset():
        conv.copy_(conv0)

    return call, reset, (conv, q8, sc, pool)


def test_bitwise_repeatable():
    print("mixer repeatable", flush=True)
    call, reset, bufs = _all_ops(70)
    runs = []
    for _ in range(3):
        reset()
        outs = call()
        torch.cuda.synchronize()
        runs.append([t.clone() for t in (*outs, *bufs)])
    same(runs[0], runs[1], "second run")
    same(runs[0], runs[2], "third run")


def test_graph_replays():
    print("mixer graph", flush=True)
    call, reset, bufs = _all_ops(80)
    reset()
    outs = call()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (*outs, *bufs)]
    g, outs = _capture(call)
    for rep in range(4):
        reset()
        for t in outs:
            t.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        same([*outs, *bufs], ref, f"replay {rep}")
        _other_work()


def test_two_graphs_and_two_streams():
    """Two captured calls replayed in turn (each with its own workspace), and the
    same calls on two streams at once."""
    print("mixer graphs and streams", flush=True)
    a, b = _all_ops(90), _all_ops(91)
    refs = []
    for call, reset, bufs in (a, b):
        reset()
        outs = call()
        torch.cuda.synchronize()
        refs.append([t.clone() for t in (*outs, *bufs)])
    graphs = [_capture(x[0]) for x in (a, b)]
    for rep in range(3):
        for (g, outs), (_, reset, bufs), ref in zip(graphs, (a, b), refs):
            reset()
            g.replay()
        torch.cuda.synchronize()
        for (g, outs), (_, _, bufs), ref in zip(graphs, (a, b), refs):
            same([*outs, *bufs], ref, f"graph replay {rep}")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for st, (call, reset, bufs) in zip(streams, (a, b)):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            reset()
            got.append((call(), bufs))
    torch.cuda.synchronize()
    for (outs, bufs), ref in zip(got, refs):
        same([*outs, *bufs], ref, "two streams")


def test_profile_stages():
    print("mixer profile stages", flush=True)
    call, _, _ = _all_ops(95)
    call()
    torch.cuda.synchronize()
    binding.profile_read()
    binding.profile_enable(True)
    call()
    binding.profile_enable(False)
    torch.cuda.synchronize()
    prof = binding.profile_read()
    assert prof["conv"][1] == 2 and prof["ssm_scan"][1] == 1 and prof["ssm_step"][1] == 1 and prof["state_q8"][1] == 2
    assert all(prof[s][0] > 0 for s in ("conv", "ssm_scan", "ssm_step", "state_q8"))


def test_a_prompt_that_goes_on_from_the_cache_element_by_element():
    """The second part of a prompt and its single tokens, from a state that was read
    back from the cache: every y and state against the oracle on the convolution's
    own outputs and that state, with the element-wise bounds of the scan and step."""
    print("prefix cache chain, element by element", flush=True)
    N, Hk, HV, K, V = 3, 2, 4, 64, 64
    p = _layer_inputs(60, N, 250, Hk, HV, K, V)
    q = {n: d(p[n]) for n in ("w", "bias", "A_log", "D", "dt_bias")}
    part = lambda lo, hi: {n: d(p[n][:, lo:hi].contiguous()) for n in ("xbc", "z", "dt")}
    dims, sec = (Hk, HV, K, V), (HV * V, Hk * K, Hk * K)
    conv = torch.zeros((N, 3, sum(sec)), dtype=BF, device=DEV)
    _, h1 = _layer(part(0, 90), q, *dims, conv)
    slots = torch.tensor([4, 0, 3], dtype=torch.int32, device=DEV)
    for form in (torch.int8, torch.float8_e4m3fn):
        q8, sc = torch.zeros((5, HV, V, K), device=DEV).to(form), torch.zeros((5, HV, V), device=DEV)
        binding.state_store_q8(h1, q8, sc, dst_indices=slots)
        back = binding.state_load_q8(q8, sc, torch.empty_like(h1), src_indices=slots)
        c, one = conv.clone(), torch.ones(N, dtype=torch.int32, device=DEV)
        mid = binding.causal_conv_fwd(part(90, 247)["xbc"], q["w"], q["bias"], sections=sec, state=c.clone(), has_state=one)
        y2, h2 = _layer(part(90, 247), q, *dims, c, h0=back, has=one)
        pool = h2.clone()
        end = binding.causal_conv_step(part(247, 250)["xbc"], q["w"], q["bias"], c.clone(), sections=sec)
        y3 = _layer(part(247, 250), q, *dims, c, pool=pool)
        torch.cuda.synchronize()

        def ref(xbc, lo, hi, h0):
            x, B, C = (t.cpu() for t in xbc)
            r = dict(x=x.unflatten(-1, (HV, V)), Bm=B.unflatten(-1, (Hk, K)), Cm=C.unflatten(-1, (Hk, K)),
                     z=p["z"][:, lo:hi], dt=p["dt"][:, lo:hi], h0=h0.cpu(), **{n: p[n] for n in ("A_log", "D", "dt_bias")})
            return ssm_ref(r, [hi - lo] * N)

        ry, mag, skip, rh, hm = ref(mid, 90, 247, back)
        close("y of the second part", y2.reshape(-1, HV, V), ry, ssm_bound(BF, ry, mag, skip))
        close("its state", h2, rh, 512 * 2.0 ** -24 * hm + 2.0 ** -20 * hm)
        ry, mag, skip, rh, hm = ref(end, 247, 250, h2)
        close("y of the single tokens", y3.reshape(-1, HV, V), ry,
              512 * 2.0 ** -24 * mag + 2.0 ** -20 * (mag + skip) + store(BF, ry))
        close("the pool", pool, rh, 2.0 ** -20 * hm + store(torch.float32, rh))


def test_graph_replays_with_other_boundaries():
    """A captured packed call (the host never reads the boundaries): replayed with
    other sequences, more, fewer or none of them split, and with none at all."""
    print("mixer graph, other boundaries", flush=True)
    T, N, Hk, HV, K, V = 1700, 7, 1, 2, 64, 64
    p = _layer_inputs(110, 1, T, Hk, HV, K, V)
    s, q = {n: d(p[n]) for n in ("xbc", "z", "dt")}, {n: d(p[n]) for n in ("w", "bias", "A_log", "D", "dt_bias")}
    sec = (HV * V, Hk * K, Hk * K)
    h0, conv0 = d(randn(111, N, HV, V, K)), d(randn(112, N, 3, sum(sec), dtype=BF))
    has = torch.tensor([1, 0, 1, 1, 0, 1, 0], dtype=torch.int32, device=DEV)
    cu, conv = torch.zeros(N + 1, dtype=torch.int64, device=DEV), conv0.clone()
    outs = tuple(torch.zeros((1, T, w), dtype=BF, device=DEV) for w in sec)
    y = torch.zeros((1, T, HV, V), dtype=BF, device=DEV)

    def call():
        x, B, C = binding.causal_conv_fwd(s["xbc"], q["w"], q["bias"], sections=sec, state=conv, has_state=has,
                                          cu_seqlens=cu, out=outs)
        return binding.ssm_chunk_fwd(x.unflatten(-1, (HV, V)), s["dt"], B.unflatten(-1, (Hk, K)),
                                     C.unflatten(-1, (Hk, K)), q["A_log"], D=q["D"], z=s["z"], dt_bias=q["dt_bias"],
                                     h0=h0, cu_seqlens=cu, out=y)[1]

    edges = [[0, 200, 200, 900, 901, 1500, 1600, 1700], [0, 100, 220, 340, 400, 500, 600, 700], [0, 0, 0, 0, 0, 0, 0, 1700],
             [0] * 8, [0, 1700] + [1700] * 6, [0, 200, 200, 900, 901, 1500, 1600, 1700]]
    assert binding.ssm_workspace_bytes(1, T, Hk, HV, K, V, N, BF, varlen=True) > 0
    fresh = lambda: (conv.copy_(conv0), y.fill_(7.0), [o.fill_(7.0) for o in outs])

    def set_cu(e):
        cu.copy_(torch.tensor(e))
        fresh()

    want = []
    for e in edges:
        set_cu(e)
        ht = call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (ht, y, conv, *outs)])
    set_cu(edges[0])
    g, ht = _capture(call)
    for e, ref in zip(edges, want):
        set_cu(e)
        ht.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        same([ht, y, conv, *outs], ref, f"replay with {e}")
        _other_work()


def test_steps_over_pools_past_4_gib():
    print("steps over pools of 4.6 GB", flush=True)
    N, HV, K, V = 3, 32, 128, 128
    p = _layer_inputs(120, N, 2, 1, HV, K, V)
    s, q = {n: d(p[n]) for n in ("xbc", "z", "dt")}, {n: d(p[n]) for n in ("w", "bias", "A_log", "D", "dt_bias")}
    D, sec = p["xbc"].shape[-1], (HV * V, K, K)
    st, cv = d(randn(121, N, HV, V, K)), d(randn(122, N, 3, D, dtype=BF))
    small, conv = st.clone(), cv.clone()
    ref = _layer(s, q, 1, HV, K, V, conv, pool=small)
    for state, slots in ((st, 2200), (cv, 4600 * 1000 * 1000 // (6 * D))):
        pool = torch.zeros((slots, *state.shape[1:]), dtype=state.dtype, device=DEV)
        idx = torch.tensor([slots - 1, 5, slots - 2], dtype=torch.int32, device=DEV)
        assert pool.numel() * pool.element_size() > 1 << 32
        pool[idx.long()] = state
        if state is st:
            x, B, C = binding.causal_conv_step(s["xbc"], q["w"], q["bias"], cv.clone(), sections=sec)
            y = binding.ssm_step(x.unflatten(-1, (HV, V)), s["dt"], B.unflatten(-1, (1, K)), C.unflatten(-1, (1, K)),
                                 q["A_log"], pool, state_indices=idx, D=q["D"], z=s["z"], dt_bias=q["dt_bias"])
            got = [y, pool[idx.long()]]
            want = [ref, small]
        else:
            out = binding.causal_conv_step(s["xbc"], q["w"], q["bias"], pool, idx, sections=sec)
            got = [*out, pool[idx.long()]]
            want = [*binding.causal_conv_step(s["xbc"], q["w"], q["bias"], cv.clone(), sections=sec), conv]
        torch.cuda.synchronize()
        same(got, want, "large pool")
        del pool
        torch.cuda.empty_cache()
