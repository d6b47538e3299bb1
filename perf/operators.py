"""The operators around a recurrent mixer, as workloads: the short causal
convolution in front of the scan (prompts and single tokens), the selective
state-space scan (prompts and single tokens) and the 8-bit cache of recurrent
states (written and read back).

``listed()`` gives the fixed workloads, ``draw(rng)`` more of the same ranges.
``prepare`` makes what a serving process holds before the call, ``run`` makes
one pass: the framework's operators where ``own`` is true, elementary torch
operations in 32 bits (64 for running sums and for values next to a rounding
border) where it is false.  ``exact`` computes the same outputs in 64 bits,
token by token, from the operators' definitions.

Formulas (per sequence; silu(a) = a / (1 + e^-a)):

  convolution   c_t = bias + sum_j w_j * u_{t-W+1+j}, u_{<0} = the W - 1 rows
                of the sequence's state slot; optionally silu; optionally each
                head of the leading sections divided by
                sqrt(sum of squares + eps).  The slot then holds the last
                W - 1 rows of the sequence.
  scan          D_t = softplus(dt_t + dt_bias), a_t = e^{-e^{A_log} D_t},
                S_t = a_t S_{t-1} + D_t x_t B_t^T,
                y_t = (S_t C_t + D x_t) silu(z_t)
  state cache   int8: s = max|row| / 127 (in 32 bits, at least 2^-126),
                code = round(row / s), ties to even; e4m3: s = the smallest
                power of two (at least 2^-126) with max|row| / s <= 448,
                code = row / s rounded to e4m3; read back as code * s.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _conv(name, dtype="bf16", seqs=1, tokens=1, ragged=False, hk=16, hv=32, k=128, v=128, width=4, act=True,
          norm=True, state=True, bias=False, extra=0):
    return {"name": name, "op": "conv_fwd", "dtype": dtype, "seqs": seqs, "tokens": tokens, "ragged": ragged,
            "hk": hk, "hv": hv, "k": k, "v": v, "width": width, "act": act, "norm": norm, "state": state,
            "bias": bias, "extra": extra}


def _conv_step(name, dtype="bf16", seqs=1, t=1, hk=16, hv=32, k=128, v=128, width=4, act=True, bias=False, extra=0):
    return {"name": name, "op": "conv_step", "dtype": dtype, "seqs": seqs, "t": t, "hk": hk, "hv": hv, "k": k,
            "v": v, "width": width, "act": act, "bias": bias, "extra": extra}


def _ssm(name, dtype="bf16", seqs=1, tokens=1, ragged=False, hk=1, hv=64, k=128, v=64, z=True, h0=False):
    return {"name": name, "op": "ssm_fwd", "dtype": dtype, "seqs": seqs, "tokens": tokens, "ragged": ragged,
            "hk": hk, "hv": hv, "k": k, "v": v, "z": z, "h0": h0}


def _ssm_step(name, dtype="bf16", pool="f32", seqs=1, t=1, hk=1, hv=64, k=128, v=64, z=True):
    return {"name": name, "op": "ssm_step", "dtype": dtype, "pool": pool, "seqs": seqs, "t": t, "hk": hk, "hv": hv,
            "k": k, "v": v, "z": z}


def _q8(name, op, form="int8", dtype="f32", states=1, hv=32, k=128, v=128):
    return {"name": name, "op": op, "form": form, "dtype": dtype, "states": states, "hv": hv, "k": k, "v": v}


def listed():
    return [
        # the q, k, v projections of a packed batch of eight ragged prompts (grouped heads, 16 x 32): convolution,
        # silu and the norms of q and k in front of a gated-delta-rule prefill
        _conv("conv prompts packed", seqs=8, tokens=16001, ragged=True),
        # a short prompt in fp32, three taps, no norm, taken from a wider projection
        _conv("conv prompt short f32", dtype="f32", tokens=100, hk=2, hv=4, k=64, v=64, width=3, norm=False,
              state=False, bias=True, extra=64),
        # one request decoding: the launch is what counts
        _conv_step("conv step B1"),
        # 256 requests, four speculated tokens each
        _conv_step("conv step B256 T4", seqs=256, t=4),
        # one long prompt: 64 heads of 64 channels that share one B and C
        _ssm("scan prompt long", tokens=8192),
        # a packed ragged batch that continues from earlier states, heads of 128 channels
        _ssm("scan prompts packed", seqs=8, tokens=5003, ragged=True, hk=8, hv=32, v=128, z=False, h0=True),
        # one request decoding over a bf16 pool
        _ssm_step("scan step B1", pool="bf16"),
        # a full decode batch over an fp32 pool
        _ssm_step("scan step B256", seqs=256, hv=32, v=128),
        # the final state of one prompt into the prefix cache
        _q8("cache store one", "q8_store"),
        # a snapshot of every request of a batch, kept as e4m3
        _q8("cache store many e4m3", "q8_store", form="e4m3", dtype="f32", states=128),
        # one cached prefix becomes the initial state of a prompt
        _q8("cache load one", "q8_load"),
        # cached states of a batch straight into the bf16 decode pool
        _q8("cache load many bf16", "q8_load", dtype="bf16", states=256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_step", "ssm_fwd", "ssm_fwd", "ssm_step", "q8_store", "q8_load"])
    k, v = rng.choice([64, 128]), rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv_fwd", "conv_step"):
        hk = rng.choice([1, 2, 4, 8, 16])
        c = dict(dtype=dtype, hk=hk, hv=hk * rng.choice([1, 2]), k=k, v=v, width=rng.choice([2, 3, 4, 4]),
                 act=rng.random() < 0.8, bias=rng.random() < 0.5, extra=rng.choice([0, 64, 200]))
        if op == "conv_step":
            c = _conv_step("", seqs=_log_int(rng, 1, 256), t=rng.randint(1, 4), **c)
        else:
            seqs = _log_int(rng, 1, 32)
            tokens = _log_int(rng, 1, 6000)
            ragged = rng.random() < 0.6
            c = _conv("", seqs=seqs, ragged=ragged, norm=rng.random() < 0.5 and k == v, state=rng.random() < 0.7,
                      tokens=tokens if ragged else max(1, tokens // seqs) * seqs, **c)
    elif op in ("ssm_fwd", "ssm_step"):
        hk = rng.choice([1, 1, 2, 4, 8])
        c = dict(dtype=dtype, hk=hk, hv=hk * rng.choice([1, 2, 5, 8] if hk > 2 else [4, 16, 20, 32]), k=k, v=v,
                 z=rng.random() < 0.5)
        c["hv"] = min(c["hv"], 32)
        c["hv"] -= c["hv"] % hk
        if op == "ssm_step":
            c = _ssm_step("", pool=rng.choice(["bf16", "f32"]), seqs=_log_int(rng, 1, 128), t=rng.randint(1, 4), **c)
        else:
            seqs = _log_int(rng, 1, 16)
            tokens = _log_int(rng, 1, 4000)
            ragged = rng.random() < 0.6
            c = _ssm("", seqs=seqs, ragged=ragged, h0=rng.random() < 0.5,
                     tokens=tokens if ragged else max(1, tokens // seqs) * seqs, **c)
    else:
        c = _q8("", op, form=rng.choice(["int8", "e4m3"]), dtype=rng.choice(["f32", "bf16"]),
                states=_log_int(rng, 1, 100), hv=rng.choice([1, 3, 8, 16, 32]), k=k, v=v)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
def _bounds(c):
    """Sequence boundaries of a case on packed tokens (ragged ones may be empty)."""
    n, t = c["seqs"], c["tokens"]
    if not c["ragged"]:
        return [i * (t // n) for i in range(n + 1)]
    r = random.Random(n * 1000003 + t)
    return [0] + sorted(r.randint(0, t) for _ in range(n - 1)) + [t]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _slots(g, n):
    """Pool size and the slot of each of n rows, in no order."""
    pool = n + 3
    return pool, torch.randperm(pool, generator=g, device=DEV)[:n].to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    op = c["op"]
    if op in ("conv_fwd", "conv_step"):
        io = DT[c["dtype"]]
        s["sections"] = (c["hk"] * c["k"], c["hk"] * c["k"], c["hv"] * c["v"])
        d = sum(s["sections"])
        if op == "conv_step":
            shape = (c["seqs"], c["t"])
        else:
            shape = (1, c["tokens"]) if c["ragged"] else (c["seqs"], c["tokens"] // c["seqs"])
        # the projection's output row holds the convolved channels, then what other parts of the layer take
        s["x"] = _randn(g, *shape, d + c["extra"], dtype=io)[..., :d]
        s["weight"] = _randn(g, d, c["width"], scale=c["width"] ** -0.5, dtype=io)
        s["bias"] = _randn(g, d, scale=0.1, dtype=io) if c["bias"] else None
        if op == "conv_step" or c["state"]:
            pool, s["slots"] = _slots(g, c["seqs"])
            s["state"] = _randn(g, pool, c["width"] - 1, d, dtype=io)
        if op == "conv_fwd":
            s["cu"] = torch.tensor(_bounds(c), dtype=torch.int64, device=DEV)
            if c["state"]:  # some of the prompts go on from an earlier part, the others are new
                s["has"] = (torch.rand(c["seqs"], generator=g, device=DEV) < 0.5).to(torch.int32)
    elif op in ("ssm_fwd", "ssm_step"):
        io = DT[c["dtype"]]
        hk, hv, k, v = c["hk"], c["hv"], c["k"], c["v"]
        if op == "ssm_step":
            shape = (c["seqs"], c["t"])
        else:
            shape = (1, c["tokens"]) if c["ragged"] else (c["seqs"], c["tokens"] // c["seqs"])
        # x, B and C lie side by side in the convolution's output, z and dt in the projection's
        xbc = torch.nn.functional.silu(_randn(g, *shape, hv * v + 2 * hk * k)).to(io)
        s["x"] = xbc[..., : hv * v].unflatten(-1, (hv, v))
        s["B"] = xbc[..., hv * v: hv * v + hk * k].unflatten(-1, (hk, k))
        s["C"] = xbc[..., hv * v + hk * k:].unflatten(-1, (hk, k))
        zdt = _randn(g, *shape, hv * v + (hv + 7) // 8 * 8, dtype=io)
        s["z"] = zdt[..., : hv * v].unflatten(-1, (hv, v)) if c["z"] else None
        s["dt"] = zdt[..., hv * v: hv * v + hv]
        # decays 1 .. 16 and step sizes 0.001 .. 0.1 (log-uniform), as such layers are initialised
        s["A_log"] = (1 + 15 * torch.rand(hv, generator=g, device=DEV)).log()
        step = torch.exp(torch.rand(hv, generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["D"] = _randn(g, hv) * 0.1 + 1
        if op == "ssm_step":
            pool, s["slots"] = _slots(g, c["seqs"])
            s["state"] = _randn(g, pool, hv, v, k, scale=0.3, dtype=DT[c["pool"]])
        else:
            s["cu"] = torch.tensor(_bounds(c), dtype=torch.int64, device=DEV)
            s["h0"] = _randn(g, c["seqs"], hv, v, k, scale=0.3) if c["h0"] else None
    else:
        n, shape = c["states"], (c["hv"], c["v"], c["k"])
        pool, s["slots"] = _slots(g, n)
        code = torch.int8 if c["form"] == "int8" else torch.float8_e4m3fn
        # rows of a recurrent state differ in size by orders of magnitude; a few are still zero
        size = torch.exp(_randn(g, *shape[:2], 1)) * (torch.rand((*shape[:2], 1), generator=g, device=DEV) > 0.02)
        if op == "q8_store":
            s["src"] = (_randn(g, n, *shape) * size).to(DT[c["dtype"]])
            s["q8"] = torch.zeros((pool, *shape), dtype=code, device=DEV)
            s["scales"] = torch.zeros((pool, *shape[:2]), device=DEV)
        else:
            codes = torch.randint(-127, 128, (pool, *shape), generator=g, device=DEV, dtype=torch.int32)
            s["q8"] = codes.to(torch.int8) if c["form"] == "int8" else (codes.float() * 3.5).to(code)
            s["scales"] = (size[..., 0] / 127 + torch.rand((pool, *shape[:2]), generator=g, device=DEV) * 1e-3)
            if c["form"] == "e4m3":
                s["scales"] = torch.exp2(torch.floor(torch.log2(s["scales"])))
            s["dst"] = torch.zeros((n, *shape), dtype=DT[c["dtype"]], device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import gated_delta_rule_61_amd as gdn
    c = s["case"]
    op = c["op"]
    act = "silu" if c.get("act") else None
    if op == "conv_fwd":
        out = gdn.causal_conv_fwd(s["x"], s["weight"], s["bias"], activation=act, sections=s["sections"],
                                  norm_dim=c["k"] if c["norm"] else 0, norm_sections=2 if c["norm"] else 0,
                                  norm_eps=EPS, state=s.get("state"), state_indices=s.get("slots"),
                                  has_state=s.get("has"), cu_seqlens=s["cu"] if c["ragged"] else None)
        return [*out, s["state"]] if c["state"] else list(out)
    if op == "conv_step":
        out = gdn.causal_conv_step(s["x"], s["weight"], s["bias"], s["state"], s["slots"], activation=act,
                                   sections=s["sections"])
        return [*out, s["state"]]
    if op == "ssm_fwd":
        y, ht = gdn.ssm_chunk_fwd(s["x"], s["dt"], s["B"], s["C"], s["A_log"], D=s["D"], z=s["z"],
                                  dt_bias=s["dt_bias"], h0=s["h0"], cu_seqlens=s["cu"] if c["ragged"] else None)
        return [y, ht]
    if op == "ssm_step":
        y = gdn.ssm_step(s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["state"], state_indices=s["slots"], D=s["D"],
                         z=s["z"], dt_bias=s["dt_bias"])
        return [y, s["state"]]
    if op == "q8_store":
        gdn.state_store_q8(s["src"], s["q8"], s["scales"], dst_indices=s["slots"])
        return _stored(s)
    gdn.state_load_q8(s["q8"], s["scales"], s["dst"], src_indices=s["slots"])
    return s["dst"]


def _stored(s):
    """The cache as it was left, as the values that it stands for (e4m3: in units of the row's scale)."""
    if s["q8"].dtype == torch.int8:
        return [s["q8"] * s["scales"][..., None], s["scales"]]
    return [s["q8"], s["scales"]]


# --------------------------------------------------- the plain forms (32 bits)
def _silu(a):
    return a / (1 + torch.exp(-a))


def _rows(s):
    """Packed tokens of a prompt: sequence of each, its place in it, and the boundaries."""
    cu = s["cu"]
    t = torch.arange(s["case"]["tokens"], device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return cu, seq, t - cu[seq]


def _plain_conv_out(y, s, norm):
    c = s["case"]
    if c["act"]:
        y = _silu(y)
    parts = torch.split(y, s["sections"], dim=-1)
    if norm:
        heads = [p.unflatten(-1, (-1, c["k"])) for p in parts[:2]]
        heads = [(h / torch.sqrt((h * h).sum(-1, keepdim=True) + EPS)).flatten(-2) for h in heads]
        parts = [*heads, parts[2]]
    return [p.to(s["x"].dtype).contiguous() for p in parts]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "conv_fwd":
        cu, seq, at = _rows(s)
        w, d = c["width"], s["x"].shape[-1]
        x = s["x"].flatten(0, 1).float()
        before = torch.zeros((c["seqs"], w - 1, d), device=x.device)
        if c["state"]:
            slots = s["slots"].long()
            before = s["state"][slots].float() * s["has"][:, None, None]
        tap = at[:, None] + torch.arange(1 - w, 1, device=x.device)
        rows = torch.where((tap >= 0)[..., None], x[(cu[seq][:, None] + tap).clamp(min=0)],
                           before[seq[:, None], (tap + w - 1).clamp(max=w - 2)])
        y = (rows * s["weight"].float().t()).sum(1)
        y = y + s["bias"].float() if c["bias"] else y
        out = _plain_conv_out(y.unflatten(0, s["x"].shape[:2]), s, c["norm"])
        if not c["state"]:
            return out
        tap = (cu[1:] - cu[:-1])[:, None] + torch.arange(1 - w, 0, device=x.device)
        one = torch.arange(c["seqs"], device=x.device)[:, None]
        last = torch.where((tap >= 0)[..., None], x[(cu[:-1, None] + tap).clamp(0, x.shape[0] - 1)],
                           before[one, (tap + w - 1).clamp(max=w - 2)])
        s["state"][slots] = last.to(s["state"].dtype)
        return [*out, s["state"]]
    if op == "conv_step":
        slots, w = s["slots"].long(), c["width"]
        rows = torch.cat([s["state"][slots].float(), s["x"].float()], 1)
        y = (rows.unfold(1, w, 1) * s["weight"].float()).sum(-1)
        y = y + s["bias"].float() if c["bias"] else y
        s["state"][slots] = rows[:, 1 - w:].to(s["state"].dtype)
        return [*_plain_conv_out(y, s, False), s["state"]]
    if op == "ssm_fwd":
        cu, seq, at = _rows(s)
        longest = max(b - a for a, b in zip(_bounds(c)[:-1], _bounds(c)[1:]))
        spread = lambda a: _spread(a.flatten(0, 1).float(), seq, at, c["seqs"], longest)  # noqa: E731
        y, ht = _plain_scan(*(spread(s[n]) for n in ("x", "B", "C")), _plain_dt(s, spread, seq, at, longest), s, s["h0"])
        y = y[seq, at].unflatten(0, s["x"].shape[:2])
        return [_plain_gate(y, s), ht]
    if op == "ssm_step":
        slots = s["slots"].long()
        dt = _softplus(s["dt"].float() + s["dt_bias"])
        y, st = _plain_scan(s["x"].float(), s["B"].float(), s["C"].float(), dt, s, s["state"][slots].float(), c["t"])
        s["state"][slots] = st.to(s["state"].dtype)
        return [_plain_gate(y, s), s["state"]]
    slots = s["slots"].long()
    if op == "q8_store":
        x = s["src"].float()
        most = x.abs().amax(-1, keepdim=True)
        if c["form"] == "int8":
            scale = (most / 127).clamp(min=2.0 ** -126)
            code = torch.round(x.double() / scale.double()).to(torch.int8)
        else:
            frac, e = torch.frexp(most)
            e = torch.where(most > 0, torch.where(frac <= 0.875, e - 9, e - 8), -126).clamp(min=-126)
            scale = torch.ldexp(torch.ones_like(most), e)
            code = torch.ldexp(x, -e).to(torch.float8_e4m3fn)
        s["q8"].view(torch.uint8)[slots] = code.view(torch.uint8)
        s["scales"][slots] = scale[..., 0]
        return _stored(s)
    q8 = s["q8"].view(torch.uint8)[slots].view(s["q8"].dtype)
    s["dst"].copy_(q8.float() * s["scales"][slots][..., None])
    return s["dst"]


def _softplus(a):
    return torch.where(a > 20, a, torch.log1p(torch.exp(a.clamp(max=20))))


def _spread(a, seq, at, n, longest):
    """Packed rows as [sequence, token], zeros behind each sequence's end."""
    out = torch.zeros((n, longest, *a.shape[1:]), dtype=a.dtype, device=a.device)
    out[seq, at] = a
    return out


def _plain_dt(s, spread, seq, at, longest):
    """Step sizes as [sequence, token, head]; 0 behind a sequence's end, which leaves the state as it is."""
    dt = _softplus(s["dt"].flatten(0, 1).float() + s["dt_bias"])
    return _spread(dt, seq, at, s["case"]["seqs"], longest)


def _plain_scan(x, b, c, dt, s, first, block=64):
    """The recurrence over blocks of tokens as products: within a block the masked, decayed C B^T, across blocks
    the decayed sum of the blocks' states.  x [n, t, hv, v], b / c [n, t, hk, k], dt [n, t, hv]."""
    n, t, hv, v = x.shape
    hk, k = b.shape[2:]
    blocks = -(-t // block)
    pad = blocks * block - t
    cut = lambda a: torch.cat([a, a.new_zeros((n, pad, *a.shape[2:]))], 1).unflatten(1, (blocks, block))  # noqa: E731
    x, b, c, dt = (cut(a) for a in (x, b, c, dt))
    # log-decays summed in 64 bits; [n, hv, blocks, block]
    run = (dt.double() * -torch.exp(s["A_log"].double())).permute(0, 3, 1, 2).cumsum(-1)
    x = (x * dt[..., None]).permute(0, 3, 1, 2, 4)                                     # [n, hv, blocks, block, v]
    b, c = (a.permute(0, 3, 1, 2, 4).repeat_interleave(hv // hk, 1) for a in (b, c))   # [n, hv, blocks, block, k]
    keep = torch.ones((block, block), dtype=torch.bool, device=x.device).tril()
    gap = (run[..., :, None] - run[..., None, :]).masked_fill(~keep, -math.inf).float()
    y = ((c @ b.transpose(-1, -2)) * torch.exp(gap)) @ x
    left = torch.exp((run[..., -1:] - run).float())
    states = (x * left[..., None]).transpose(-1, -2) @ b                               # [n, hv, blocks, v, k]
    if first is None:
        first = torch.zeros((n, hv, v, k), device=x.device)
    states = torch.cat([first[:, :, None], states], 2)
    total = torch.nn.functional.pad(run[..., -1].cumsum(-1), (1, 0))                   # [n, hv, blocks + 1]
    keep = torch.ones((blocks + 1, blocks + 1), dtype=torch.bool, device=x.device).tril()
    gap = (total[..., :, None] - total[..., None, :]).masked_fill(~keep, -math.inf).float()
    states = (torch.exp(gap) @ states.flatten(-2)).unflatten(-1, (v, k))
    y = y + (c @ states[:, :, :-1].transpose(-1, -2)) * torch.exp(run.float())[..., None]
    y = y.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :t]
    return y, states[:, :, -1].contiguous()


def _plain_gate(y, s):
    y = y + s["D"][:, None] * s["x"].float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["x"].dtype)


# ---------------------------------------------------------------- what it takes
def work(case):
    c = case
    e = 4 if c.get("dtype") == "f32" else 2
    op = c["op"]
    if op in ("conv_fwd", "conv_step"):
        d = 2 * c["hk"] * c["k"] + c["hv"] * c["v"]
        rows = c["tokens"] if op == "conv_fwd" else c["seqs"] * c["t"]
        held = c["seqs"] * (c["width"] - 1) * d * e if op == "conv_step" or c["state"] else 0
        return {"bytes": 2 * rows * d * e + 2 * held + d * (c["width"] + c["bias"]) * e,
                "flops": rows * d * (2 * c["width"] + 5 * c["act"])}
    if op in ("ssm_fwd", "ssm_step"):
        rows = c["tokens"] if op == "ssm_fwd" else c["seqs"] * c["t"]
        per = c["hv"] * c["v"] * (3 if c["z"] else 2) + 2 * c["hk"] * c["k"] + c["hv"]
        state = c["seqs"] * c["hv"] * c["v"] * c["k"]
        if op == "ssm_fwd":
            held = state * 4 * (2 if c["h0"] else 1)
        else:
            held = state * 2 * (4 if c["pool"] == "f32" else 2)
        return {"bytes": rows * per * e + held, "flops": rows * c["hv"] * c["v"] * (5 * c["k"] + 4)}
    n = c["states"] * c["hv"] * c["v"]
    return {"bytes": n * c["k"] * (e + 1) + 4 * n, "flops": 2 * n * c["k"]}


# ------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("conv_fwd", "conv_step"):
        w, d = c["width"], s["x"].shape[-1]
        edge = _bounds(c) if op == "conv_fwd" else [i * c["t"] for i in range(c["seqs"] + 1)]
        x = s["x"].reshape(-1, d).double()
        state = s["state"].double() if "state" in s else None
        y = torch.empty_like(x)
        for i in range(c["seqs"]):
            u = torch.zeros((w - 1, d), dtype=torch.float64, device=x.device)
            if state is not None and (op == "conv_step" or int(s["has"][i])):
                u = state[int(s["slots"][i])].clone()
            u = torch.cat([u, x[edge[i]: edge[i + 1]]])
            n = edge[i + 1] - edge[i]
            acc = s["bias"].double().expand(n, d).clone() if c["bias"] else torch.zeros((n, d), dtype=torch.float64,
                                                                                       device=x.device)
            for j in range(w):
                acc += s["weight"][:, j].double() * u[j: j + n]
            y[edge[i]: edge[i + 1]] = acc
            if state is not None:
                state[int(s["slots"][i])] = u[u.shape[0] - (w - 1):]
        if c["act"]:
            y = y * torch.sigmoid(y)
        out, at = [], 0
        for i, width in enumerate(s["sections"]):
            part = y[:, at: at + width]
            at += width
            if op == "conv_fwd" and c["norm"] and i < 2:
                heads = part.reshape(part.shape[0], -1, c["k"])
                part = (heads / heads.square().sum(-1, keepdim=True).add(EPS).sqrt()).reshape(part.shape)
            out.append(part.reshape(*s["x"].shape[:2], width))
        return out if state is None else [*out, state]
    if op in ("ssm_fwd", "ssm_step"):
        hk, hv, k, v = c["hk"], c["hv"], c["k"], c["v"]
        edge = _bounds(c) if op == "ssm_fwd" else [i * c["t"] for i in range(c["seqs"] + 1)]
        if (edge[-1] + max(b - a for a, b in zip(edge, edge[1:])) * 40) * hv * v * k > 6e11:
            return None
        flat = lambda a: a.reshape(-1, *a.shape[2:]).double()  # noqa: E731
        x, b, cc, dt = flat(s["x"]), flat(s["B"]), flat(s["C"]), flat(s["dt"])
        dt = torch.logaddexp(dt + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device=x.device))
        a = torch.exp(-torch.exp(s["A_log"].double()) * dt)
        pool = s["state"].double() if op == "ssm_step" else None
        if op == "ssm_step":
            h = pool[s["slots"].long()]
        else:
            h = s["h0"].double() if s["h0"] is not None else x.new_zeros((c["seqs"], hv, v, k))
        y = torch.empty_like(x)
        first = torch.tensor(edge[:-1], device=x.device)
        length = torch.tensor([q - p for p, q in zip(edge, edge[1:])], device=x.device)
        order = torch.argsort(length, descending=True)     # the sequences still running come first
        h, first = h[order], first[order]
        lengths = sorted((q - p for p, q in zip(edge, edge[1:])), reverse=True)
        live = len(lengths)
        for t in range(lengths[0]):
            while lengths[live - 1] <= t:
                live -= 1
            r = first[:live] + t
            bt = b[r].repeat_interleave(hv // hk, 1)
            ct = cc[r].repeat_interleave(hv // hk, 1)
            h[:live].mul_(a[r][..., None, None]).add_((dt[r][..., None] * x[r])[..., None] * bt[..., None, :])
            y[r] = (h[:live] @ ct[..., None])[..., 0]
        h = torch.empty_like(h).index_copy_(0, order, h)
        y = y + s["D"].double()[:, None] * x
        if s["z"] is not None:
            zz = flat(s["z"])
            y = y * zz * torch.sigmoid(zz)
        y = y.reshape(s["x"].shape)
        if op == "ssm_step":
            pool[s["slots"].long()] = h
            return [y, pool]
        return [y, h]
    slots = s["slots"].long()
    if op == "q8_load":
        code = s["q8"].to(torch.float32).double()[slots]
        return code * s["scales"].double()[slots].unsqueeze(-1)
    x = s["src"].double()
    most = x.abs().max(-1).values
    codes = torch.zeros(s["q8"].shape, dtype=torch.float64, device=x.device)
    scales = s["scales"].double()
    if c["form"] == "int8":
        step = (most.float() / 127).clamp(min=2.0 ** -126).double()
        codes[slots] = torch.round(x / step[..., None])
    else:
        step = torch.full_like(most, 2.0 ** -126)
        for e in range(-126, 121):                          # the smallest power of two that is enough
            step = torch.where(most > 448 * step, torch.full_like(step, 2.0 ** (e + 1)), step)
        u = x / step[..., None]
        unit = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)   # e4m3's spacing at u
        codes[slots] = torch.round(u / unit) * unit
    scales[slots] = step
    return [codes * scales[..., None] if c["form"] == "int8" else codes, scales]
