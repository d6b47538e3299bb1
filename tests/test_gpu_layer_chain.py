"""The operators of a recurrent layer together, as training and serving use them:
convolution, delta rule and gated norm with their gradients; the prompt, then
single tokens with per-channel gates; captured and on two streams; at sizes past
32-bit offsets."""

import gc

import numpy as np
import pytest
import torch

import gated_delta_rule_61_amd as gdn
import oracle
from tests import running_error as re
from tests.mixer_cases import BF, DEV, EPS, close, conv_ref, d, edges, f64, randn, same, store
from tests.test_gpu_graphs import _capture, _other_work
from tests.test_gpu_kda_decode import reference
from tests.tolerance import check

pytestmark = pytest.mark.gpu
F32 = torch.float32
LENS = [70, 0, 33, 1, 64]
HK, HV, K = 2, 4, 64
SEC = (HK * K, HK * K, HV * K)
CU = torch.tensor(edges(LENS), dtype=torch.int64)


def layer(seed, io, extra=0):
    T, N = sum(LENS), len(LENS)
    gen = torch.Generator().manual_seed(seed)
    return dict(x=randn(seed, 1, T, sum(SEC) + extra, dtype=io), w=randn(seed + 1, sum(SEC), 4, dtype=io, scale=0.5),
                g=-torch.rand(1, T, HV, generator=gen) * 0.2, beta=torch.rand(1, T, HV, generator=gen),
                h0=randn(seed + 2, N, HV, K, K, scale=0.3), z=randn(seed + 3, 1, T, HV * K, dtype=io),
                nw=1 + randn(seed + 4, K, scale=0.3), dy=randn(seed + 5, 1, T, HV * K, dtype=io),
                dht=randn(seed + 6, N, HV, K, K, scale=0.3))


def heads(t, n):
    return t.unflatten(-1, (n, K))


def forward(i, cu):
    q, k, v = gdn.causal_conv_fwd(i["x"][..., :sum(SEC)], i["w"], sections=SEC, norm_dim=K, norm_sections=2,
                                  norm_eps=EPS, cu_seqlens=cu)
    q, k, v = heads(q, HK), heads(k, HK), heads(v, HV)
    o, ht = gdn.gdn_chunk_fwd(q, k, v, i["g"], i["beta"], h0=i["h0"], cu_seqlens=cu)
    y = gdn.group_norm_fwd(o.flatten(2), HV, i["nw"], z=i["z"], activation="silu", rms=True)
    return dict(q=q, k=k, v=v, o=o, ht=ht, y=y)


def backward(i, f, cu):
    do, dz, dnw, _ = gdn.group_norm_bwd(i["dy"], f["o"].flatten(2), HV, i["nw"], z=i["z"], activation="silu", rms=True)
    dq, dk, dv, dg, dbeta, dh0 = gdn.gdn_chunk_bwd(f["q"], f["k"], f["v"], i["g"], i["beta"], heads(do, HV), i["dht"],
                                                   h0=i["h0"], cu_seqlens=cu)
    dx, dw, _ = gdn.causal_conv_bwd((dq.flatten(2), dk.flatten(2), dv.flatten(2)), i["x"][..., :sum(SEC)], i["w"],
                                    sections=SEC, norm_dim=K, norm_sections=2, norm_eps=EPS, cu_seqlens=cu)
    return dict(do=do, dz=dz, dnw=dnw, dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta, dh0=dh0, dx=dx, dw=dw)


@pytest.mark.parametrize("io", [BF, F32])
def test_a_layer_and_its_gradients_step_by_step(io):
    """Every operator's result against the oracle on what it was given (its inputs as stored), with its own bounds."""
    print(f"layer chain {io}", flush=True)
    i = layer(1, io, extra=64)
    c, cu = {n: d(t) for n, t in i.items()}, d(CU)
    f = forward(c, cu)
    b = backward(c, f, cu)
    torch.cuda.synchronize()
    x, w, step = f64(i["x"])[0, :, :sum(SEC)], f64(i["w"]), 2.0 ** -8 if io == BF else re.U
    outs, errs, _ = conv_ref(x, w, None, LENS, [None] * len(LENS), True, SEC, K, 2)
    for n, r, e in zip("qkv", outs, errs):
        close(n, f[n].flatten(2)[0], r, e + store(io, r))
    f, b = ({n: t.cpu() for n, t in m.items()} for m in (f, b))
    o, ht = oracle.gdn_recurrent(f["q"], f["k"], f["v"], i["g"], i["beta"], K ** -0.5, h0=i["h0"], cu_seqlens=CU)
    check("o", f["o"], o, io)
    check("ht", f["ht"], ht, io)
    rows = lambda t: f64(t).reshape(-1, HV * K)  # noqa: E731
    norm = (rows(f["o"]), HV, f64(i["nw"]), None, rows(i["z"]), "silu", True, 1e-5)
    close("y", rows(f["y"]), oracle.group_norm(*norm), re.group_norm(*norm).round_to(step).e)
    want, bars = oracle.group_norm(*norm, dout=rows(i["dy"])), re.group_norm(*norm, dout=rows(i["dy"]))
    for n, r, e in zip(("do", "dz", "dnw"), want, bars):
        close(n, f64(b[n]).reshape(r.shape), r, e.round_to(re.U if n == "dnw" else step).e)
    ref = oracle.gdn_recurrent_bwd(f["q"], f["k"], f["v"], i["g"], i["beta"], heads(b["do"], HV), K ** -0.5, i["h0"],
                                   i["dht"], CU)
    for n, r in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), ref):
        check(n, b[n], r, io, stored=io)
    dy = f64(torch.cat([b[n].flatten(2) for n in ("dq", "dk", "dv")], -1))[0]
    dw, ew, size = np.zeros(w.shape), np.zeros(w.shape), np.zeros(w.shape)
    for lo, hi in zip(edges(LENS)[:-1], edges(LENS)[1:]):
        args = (dy[lo:hi], x[lo:hi], w, None, True, K, sum(SEC[:2]), EPS)
        r, e = oracle.causal_conv_bwd(*args), re.causal_conv_bwd(*args)
        close("dx", f64(b["dx"])[0, lo:hi], r[0], e[0].round_to(step).e)
        dw, ew, size = dw + r[1], ew + e[1].e, size + np.abs(r[1])
    close("dw", f64(b["dw"]), dw, re.E(dw, ew + 2 * len(LENS) * re.U * size).round_to(step).e)


def _oracle_layer(i, x, w, h0, z, nw, dy, dht):
    """The loss sum(y dy) + sum(ht dht) and its gradients, all in 64 bits."""
    seqs = list(zip(edges(LENS)[:-1], edges(LENS)[1:]))
    nc = sum(SEC[:2])
    c = np.concatenate([oracle.causal_conv(x[lo:hi], w, None, None, True)[0] for lo, hi in seqs])
    h = c[:, :nc].reshape(-1, nc // K, K)
    c[:, :nc] = (h / np.sqrt((h * h).sum(-1, keepdims=True) + EPS)).reshape(-1, nc)
    cut = lambda lo, n: c[:, lo: lo + n * K].reshape(1, -1, n, K)  # noqa: E731
    q, k, v = cut(0, HK), cut(SEC[0], HK), cut(nc, HV)
    o, ht = oracle.gdn_recurrent(q, k, v, i["g"], i["beta"], K ** -0.5, h0=h0, cu_seqlens=CU)
    o = o.reshape(-1, HV * K)
    norm = (o, HV, nw, None, z, "silu", True, 1e-5)
    loss = (oracle.group_norm(*norm) * dy).sum() + (ht * dht).sum()
    do, dz, dnw, _ = oracle.group_norm(*norm, dout=dy)
    dq, dk, dv, _, _, dh0 = oracle.gdn_recurrent_bwd(q, k, v, i["g"], i["beta"], do.reshape(1, -1, HV, K), K ** -0.5, h0,
                                                     dht, CU)
    dc = np.concatenate([t.reshape(-1, s) for t, s in zip((dq, dk, dv), SEC)], -1)
    back = [oracle.causal_conv_bwd(dc[lo:hi], x[lo:hi], w, None, True, K, nc, EPS)[:2] for lo, hi in seqs]
    return loss, dict(x=np.concatenate([r[0] for r in back]), w=sum(r[1] for r in back), h0=dh0, z=dz, nw=dnw)


def test_gradients_through_the_layer_in_fp32():
    """fp32 from end to end against the formula in 64 bits and against differences of the loss.  A value of any of
    the three operators is a sum of at most 2^11 rounded terms, each off by 2^-24 of its size: 2^-13 of the gradient's
    norm for each operator on the way forth and back, six at most.  A difference over 2e-5 of the leaves' norms is
    off by its square times the third derivatives, below 2^-20 of the loss's slope."""
    print("layer chain, end to end", flush=True)
    i = layer(9, F32)
    c, cu = {n: d(t) for n, t in i.items()}, d(CU)
    b = backward(c, forward(c, cu), cu)
    torch.cuda.synchronize()
    rows = lambda t: f64(t).reshape(-1, t.shape[-1])  # noqa: E731
    leaf = dict(x=rows(i["x"]), w=f64(i["w"]), h0=f64(i["h0"]), z=rows(i["z"]), nw=f64(i["nw"]))
    fixed = (rows(i["dy"]), f64(i["dht"]))
    _, ref = _oracle_layer(i, *leaf.values(), *fixed)
    for n in leaf:
        got = f64(b["d" + n]).reshape(ref[n].shape)
        size = np.linalg.norm(ref[n])
        assert np.linalg.norm(got - ref[n]) <= 6 * 2.0 ** -13 * size, n
        to = got / np.linalg.norm(got) + 0.5 * np.sign(np.cos(np.arange(got.size))).reshape(got.shape) / got.size ** 0.5
        h = 2e-5 * np.linalg.norm(leaf[n])
        far = [_oracle_layer(i, *dict(leaf, **{n: leaf[n] + s * h * to}).values(), *fixed)[0] for s in (1, -1)]
        slope = (far[0] - far[1]) / (2 * h)
        assert abs(slope - (got * to).sum()) <= (6 * 2.0 ** -13 + 2.0 ** -20) * size * np.linalg.norm(to), n


def test_the_prompt_then_single_tokens_with_channel_gates():
    """Convolution -> per-channel-gated prefill -> pool; then convolution step -> step -> gated norm, twice: against
    the oracle step by step, each on the stored inputs.  The first step's outputs also go on from the prompt: one
    prefill over the prompt and the tokens gives them, up to the state's and the inputs' storage."""
    print("conv -> kda prefill -> pool -> conv step -> kda step -> norm", flush=True)
    T, N, D = sum(LENS), len(LENS), sum(SEC)
    x, w = randn(21, 1, T, D, dtype=BF), randn(22, D, 4, dtype=BF, scale=0.5)
    A_log, dt_bias = randn(23, HV, scale=0.3), randn(24, HV, K) - 3
    gate = lambda a: -torch.exp(A_log.double())[:, None] * torch.nn.functional.softplus(a.double() + dt_bias)  # noqa: E731
    a, bl = randn(25, 1, T, HV, K, dtype=BF), randn(26, 1, T, HV, dtype=BF)
    slots = torch.tensor([6, 0, 3, 5, 1], dtype=torch.int32, device=DEV)
    conv_pool, cu = torch.zeros((7, 3, D), dtype=BF, device=DEV), d(CU)
    q, k, v = gdn.causal_conv_fwd(d(x), d(w), sections=SEC, norm_dim=K, norm_sections=2, norm_eps=EPS, state=conv_pool,
                                  state_indices=slots, cu_seqlens=cu)
    q, k, v = heads(q, HK), heads(k, HK), heads(v, HV)
    gk, beta = gate(a).float(), bl.float().sigmoid()
    o, ht, _, _ = gdn.kda_chunk_fwd(q, k, v, d(gk), d(beta), cu_seqlens=cu, return_intra=False)
    pool = torch.zeros((7, HV, K, K), device=DEV)
    pool[slots.long()] = ht
    torch.cuda.synchronize()
    ro, rh = oracle.kda_recurrent(q.cpu(), k.cpu(), v.cpu(), gk, beta, K ** -0.5, cu_seqlens=CU)
    check("o", o.cpu(), ro, BF)
    check("ht", ht.cpu(), rh, BF)
    for tokens in (3, 1):
        s = 30 + tokens
        x1, a1, b1 = randn(s, N, tokens, D, dtype=BF), randn(s + 1, N, tokens, HV, K, dtype=BF), randn(s + 2, N, tokens, HV, dtype=BF)
        z1, nw = randn(s + 3, N, tokens, HV * K, dtype=BF), 1 + randn(s + 4, K, scale=0.3)
        q1, k1, v1 = gdn.causal_conv_step(d(x1), d(w), None, conv_pool, slots, sections=SEC)
        q1, k1, v1 = heads(q1, HK), heads(k1, HK), heads(v1, HV)
        before = pool.clone()
        o1 = gdn.kda_decode(q1, k1, v1, d(a1), d(b1), d(A_log), d(dt_bias), pool, slots)
        y1 = gdn.group_norm_fwd(o1.flatten(2), HV, d(nw), z=d(z1), activation="sigmoid", rms=True)
        torch.cuda.synchronize()
        r = reference(dict(q=q1, k=k1, v=v1, a=a1, b=b1, A_log=A_log, dt_bias=dt_bias, state=before, idx=slots))
        close("o1", f64(o1), r[0], 2 * r[2] + 2.0 ** -8 * (np.abs(r[0]) + 2 * r[2]))
        close("pool", f64(pool), r[1], 2 * r[3] + re.U * (np.abs(r[1]) + 2 * r[3]))
        norm = (f64(o1).reshape(-1, HV * K), HV, f64(nw), None, f64(z1).reshape(-1, HV * K), "sigmoid", True, 1e-5)
        close("y1", f64(y1).reshape(-1, HV * K), oracle.group_norm(*norm), re.group_norm(*norm).round_to(2.0 ** -8).e)
        if tokens == 3:   # the longest sequence in one prefill, q and k normalised (and stored) as the step takes them
            unit = lambda t: (t / ((t * t).sum(-1, keepdim=True) + 1e-6).sqrt())  # noqa: E731
            join = lambda p, t: torch.cat([p[:, :LENS[0]], t[:1].to(p.dtype)], 1)  # noqa: E731
            whole, _ = oracle.kda_recurrent(join(q.cpu().float(), unit(q1.cpu().float())), join(k.cpu().float(), unit(k1.cpu().float())),
                                            join(v.cpu(), v1.cpu()), join(gk, gate(a1).float()), join(beta, b1.float().sigmoid()), K ** -0.5)
            check("goes on", o1[:1].cpu(), whole[:, LENS[0]:], BF)


def test_captured_and_on_two_streams():
    """Two captured training steps replayed in turn, each with its own memory, eager work between them; then both on
    two streams at once.  Always the eager call's bits."""
    print("layer chain graphs and streams", flush=True)
    sides = [{n: d(t) for n, t in layer(s, BF).items()} for s in (41, 51)]
    cu = d(CU)

    def step(i):
        f = forward(i, cu)
        return [*f.values(), *backward(i, f, cu).values()]

    refs = [[t.clone() for t in step(i)] for i in sides]
    torch.cuda.synchronize()
    graphs = [_capture(lambda i=i: step(i)) for i in sides]
    for rep in range(3):
        for g, outs in graphs:
            for t in outs:
                t.fill_(7.0)
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, outs), ref in zip(graphs, refs):
            same(outs, ref, f"replay {rep}")
        _other_work()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s, i in zip(streams, sides):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(step(i))
    torch.cuda.synchronize()
    for outs, ref in zip(got, refs):
        same(outs, ref, "two streams")


def _release():
    gc.collect()
    torch.cuda.empty_cache()


def test_delta_rule_gradients_past_4_gib():
    """q, k, v, dout of 4.3 GB and 17 GB of states: two (sequence, head) pairs carry data, the last among them; all
    other gradients are exactly zero."""
    B, T, H, D = 2048, 64, 128, 128
    print("chunk gradients past 4 GiB", flush=True)
    big = [torch.zeros(B, T, H, D, dtype=BF, device=DEV) for _ in range(4)]
    gates = [torch.zeros(B, T, H, device=DEV) for _ in range(2)]
    assert big[0].numel() * 2 >= 1 << 32
    gen = torch.Generator().manual_seed(3)
    small = {}
    for s, (n, h) in enumerate(((5, 0), (B - 1, H - 1))):
        i = dict(q=randn(70 + s, 1, T, 1, D), k=torch.nn.functional.normalize(randn(72 + s, 1, T, 1, D), dim=-1),
                 v=randn(74 + s, 1, T, 1, D), do=randn(76 + s, 1, T, 1, D))
        i = {name: t.to(BF) for name, t in i.items()}
        i.update(g=-torch.rand(1, T, 1, generator=gen) * 0.2, beta=torch.rand(1, T, 1, generator=gen))
        for dst, name in zip(big, ("q", "k", "v", "do")):
            dst[n, :, h] = d(i[name][0, :, 0])
        for dst, name in zip(gates, ("g", "beta")):
            dst[n, :, h] = d(i[name][0, :, 0])
        small[n, h] = i
    out = gdn.gdn_chunk_bwd(*big[:3], *gates, big[3])
    torch.cuda.synchronize()
    for (n, h), i in small.items():
        ref = oracle.gdn_recurrent_bwd(i["q"], i["k"], i["v"], i["g"], i["beta"], i["do"], D ** -0.5)
        for name, got, r in zip(("dq", "dk", "dv", "dg", "dbeta"), out, ref):
            check(name, got[n: n + 1, :, h: h + 1].cpu(), r, BF, stored=BF)
            got[n, :, h] = 0
    for got in out[:5]:
        assert not bool(got.any())
    del big, gates, out, got
    _release()


def test_rows_past_4_gib():
    """The norm, its gradients and the convolution's on tensors of 4.3 GB: the last rows as in a call on them alone."""
    print("rows past 4 GiB", flush=True)
    C, T, G, n = 16384, 131200, 128, 40
    x, z, dy = (torch.zeros(1, T, C, dtype=BF, device=DEV) for _ in range(3))
    assert x.numel() * 2 > 1 << 32
    for s, t in enumerate((x, z, dy)):
        t[0, -n:] = d(randn(80 + s, n, C, dtype=BF))
    tail = [t[:, -n:].contiguous() for t in (x, z, dy)]
    w = d(1 + randn(83, C // G, scale=0.3))
    y = gdn.group_norm_fwd(x, G, w, z=z, rms=True)
    same([y[:, -n:]], [gdn.group_norm_fwd(tail[0], G, w, z=tail[1], rms=True)], "norm")
    assert not bool(y[:, :-n].any())
    del y
    a, b = gdn.group_norm_bwd(dy, x, G, w, z=z, rms=True), gdn.group_norm_bwd(tail[2], tail[0], G, w, z=tail[1], rms=True)
    same([a[0][:, -n:], a[1][:, -n:]], b[:2], "norm's gradients")
    assert not bool(a[0][:, :-n].any()) and not bool(a[1][:, :-n].any())
    bars = re.group_norm(f64(tail[0])[0], G, f64(w), None, f64(tail[1])[0], "silu", True, 1e-5, f64(tail[2])[0])
    close("dweight", f64(a[2]), bars[2].v, bars[2].round_to(re.U).e)
    del a
    _release()
    cw = d(randn(84, C, 4, dtype=BF, scale=0.5))
    cu = torch.tensor([0, T - n, T], device=DEV)
    a = gdn.causal_conv_bwd(dy, x, cw, cu_seqlens=cu)
    b = gdn.causal_conv_bwd(tail[2], tail[0], cw)
    same([a[0][:, -n:]], [b[0]], "convolution's dx")
    assert not bool(a[0][:, :-n].any())
    bar = re.causal_conv_bwd(f64(tail[2])[0], f64(tail[0])[0], f64(cw), None, True, 0, 0, 1e-6)[1]
    close("dw", f64(a[1]), bar.v, bar.round_to(2.0 ** -8).e)
    del a, x, z, dy
    _release()


def test_a_step_over_a_pool_past_4_gib():
    print("step over a pool of 8.6 GB", flush=True)
    B, H, D, slots = 3, 32, 128, 8200
    pool = torch.zeros(slots, H, D, D, dtype=BF, device=DEV)
    idx = torch.tensor([slots - 1, 4, slots - 2], dtype=torch.int32, device=DEV)
    small = d(randn(90, B, H, D, D, dtype=BF, scale=0.3))
    pool[idx.long()] = small
    i = [d(t) for t in (randn(91, B, 2, H, D, dtype=BF), randn(92, B, 2, H, D, dtype=BF), randn(93, B, 2, H, D, dtype=BF),
                        randn(94, B, 2, H, D, dtype=BF), randn(95, B, 2, H, dtype=BF), randn(96, H, scale=0.3),
                        randn(97, H, D) - 3)]
    o = gdn.kda_decode(*i, pool, idx)
    ref = gdn.kda_decode(*i, small)
    torch.cuda.synchronize()
    same([o, pool[idx.long()]], [ref, small], "large pool")
    pool[idx.long()] = 0
    assert not bool(pool.any())
    del pool
    _release()
