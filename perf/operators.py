"""Cases of the query / key preparation and of the gated linear recurrence, with their plain forms.

``qk``    per-head norm of q and k with the position rotation in the same pass, alone
          (prefill, decode) or with its backward pass (training).
``scan``  the per-channel recurrence h_t = a_t h_{t-1} + b_t x_t over dense batches and over
          packed sequences, alone or with its backward pass; ``step`` its single-token form.

``run`` computes a case in plain torch operations, or with ``own`` through the package.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def _qk(name, B, T, Hq, Hk, d, *, io="bf16", norm="rms", weight=True, layout="half", rot=None, far=0, fused=True, train=False):
    return dict(name=name, op="qk", B=B, T=T, Hq=Hq, Hk=Hk, d=d, io=io, norm=norm, weight=weight, layout=layout,
                rot=d if rot is None else rot, far=far, fused=fused, train=train)


def _scan(name, B, T, H, dv, *, io="bf16", gate="f32", form="value", beta="one", seqs=0, fused=False, train=False):
    return dict(name=name, op="scan", B=B, T=T, H=H, dv=dv, io=io, gate=gate, form=form, beta=beta, seqs=seqs,
                fused=fused, train=train)


def _step(name, B, H, dv, *, io="bf16", gate="f32", form="value", beta="one"):
    return dict(name=name, op="step", B=B, H=H, dv=dv, io=io, gate=gate, form=form, beta=beta)


def listed():
    return [
        # one token of a few requests, out of the fused projection: a decode step's latency
        _qk("qk_decode_8x16x128", 8, 1, 16, 16, 128, far=60000),
        # the headline prefill batch: keys normalised as the delta rule wants them, no positions
        _qk("qk_prefill_l2_4x4096x16x128", 4, 4096, 16, 16, 128, norm="l2", weight=False, rot=0, fused=False),
        # one long prompt at far positions, shared key heads, queries and keys out of the fused projection
        _qk("qk_prefill_65536x32+8x128", 1, 65536, 32, 8, 128, far=1 << 20),
        # training with a part of each head rotated, fp32, odd lengths and head sizes
        _qk("qk_train_f32_3x777x12+4x80", 3, 777, 12, 4, 80, io="f32", rot=40, layout="interleaved", train=True),
        # training at the headline batch
        _qk("qk_train_4x4096x16x128", 4, 4096, 16, 16, 128, train=True),
        # decode of a large batch
        _step("step_512x16x128", 512, 16, 128),
        # a small fp32 layer: an odd number of channels, one block of tokens
        _scan("scan_f32_2x300x5x77", 2, 300, 5, 77, io="f32"),
        # the headline prefill batch: bf16 stream, fp32 log gates
        _scan("scan_prefill_4x4096x16x128", 4, 4096, 16, 128, form="log", beta="coupled"),
        # one long prompt, everything in bf16, stream and gates out of one projection
        _scan("scan_prefill_65536x32x128", 1, 65536, 32, 128, gate="bf16", fused=True),
        # packed prompts of many requests, an input gate of its own
        _scan("scan_packed_f32_37x20000x1000", 1, 20000, 8, 125, io="f32", beta="given", seqs=37),
        # training at the headline batch
        _scan("scan_train_4x4096x16x128", 4, 4096, 16, 128, form="log", beta="coupled", train=True),
        # training in fp32 with an input gate, a ragged last block
        _scan("scan_train_f32_2x5000x16x64", 2, 5000, 16, 64, io="f32", beta="given", train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "qk", "scan", "scan", "scan", "step"])
    io = rng.choice(["bf16", "bf16", "f32"])
    gate = rng.choice(["bf16", "f32"])
    form, beta = rng.choice(["value", "log"]), rng.choice(["one", "given", "coupled"])
    if op == "qk":
        d = 8 * rng.randint(2, 32)
        Hq = rng.randint(1, 40)
        Hk = rng.choice([Hq, max(1, Hq // 4), 1])
        train = rng.random() < 0.5
        most = (1 << 27) // (2 if io == "f32" else 1) // (3 if train else 1)
        tokens = _log(rng, 1, max(1, most // ((Hq + Hk) * d)))
        B = min(tokens, _log(rng, 1, 64))
        return {k: v for k, v in _qk("", B, tokens // B, Hq, Hk, d, io=io, norm=rng.choice(["rms", "rms", "l2", "none"]),
                                     weight=rng.random() < 0.7, layout=rng.choice(["half", "interleaved"]),
                                     rot=2 * rng.randint(0, d // 2) if rng.random() < 0.5 else d,
                                     far=rng.choice([0, 0, 1000, 1 << 20]), fused=rng.random() < 0.5,
                                     train=train).items() if k != "name"}
    H, dv = _log(rng, 1, 40), rng.randint(1, 256)
    if op == "step":
        return {k: v for k, v in _step("", _log(rng, 1, 1024), H, dv, io=io, gate=gate, form=form, beta=beta).items() if k != "name"}
    train = rng.random() < 0.5
    most = (1 << 26) // (2 if io == "f32" else 1) // (3 if train else 1)
    tokens = _log(rng, 2, max(2, min(65536, most // (H * dv))))
    packed = rng.random() < 0.3
    B = 1 if packed else min(tokens, _log(rng, 1, 16))
    return {k: v for k, v in _scan("", B, tokens // B, H, dv, io=io, gate=gate, form=form, beta=beta,
                                   seqs=_log(rng, 1, min(tokens, 200)) if packed else 0,
                                   fused=gate == io and rng.random() < 0.5, train=train).items() if k != "name"}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape, dtype=torch.float32):
    """Normal values, drawn in slices of the leading axis so that no large fp32 copy of a bf16 tensor is made."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 26):
        part = flat[at:at + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda"))
    return out


def _gate(gen, shape, form, dtype):
    """Decays mostly between 0.9 and 0.999, as values or as their logarithms."""
    x = _randn(gen, *shape) - 4.0
    return (-torch.nn.functional.softplus(x) if form == "log" else torch.sigmoid(-x)).to(dtype)


def _rows(T):
    """The rows that belong to packed sequences: a few at either end belong to none."""
    return min(3, T // 8), T - min(7, T // 8)


def _offsets(gen, T, n):
    """Borders of n packed sequences over the rows of `_rows`; sequences may be empty."""
    lo, hi = _rows(T)
    cuts = torch.randint(lo, hi + 1, (n - 1,), generator=gen, device="cuda", dtype=torch.int32)
    ends = torch.tensor([lo, hi], dtype=torch.int32, device="cuda")
    return torch.cat([ends, cuts]).sort().values.to(torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    io = DTYPE[c["io"]]
    s = {"case": c}
    if c["op"] == "qk":
        B, T, Hq, Hk, d = c["B"], c["T"], c["Hq"], c["Hk"], c["d"]
        if c["fused"]:  # q | k | v of one projection's output
            width = (Hq + 2 * Hk) * d
            x = _randn(gen, B, T, width, dtype=io)
            s["q"] = x[..., :Hq * d].unflatten(-1, (Hq, d))
            s["k"] = x[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
        else:
            s["q"], s["k"] = _randn(gen, B, T, Hq, d, dtype=io), _randn(gen, B, T, Hk, d, dtype=io)
        s["wq"] = s["wk"] = None
        if c["weight"] and c["norm"] != "none":
            s["wq"], s["wk"] = (1 + 0.2 * _randn(gen, d) for _ in range(2))
        if c["rot"]:
            pos = torch.arange(T, device="cuda", dtype=torch.int32).expand(B, T)
            start = torch.randint(0, c["far"] + 1, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
            s["pos"] = (pos + start).contiguous()
            i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda")
            s["inv_freq"] = 10000.0 ** (-i / c["rot"])
        else:
            s["pos"] = s["inv_freq"] = None
        s["eps"], s["q_scale"] = (1e-6 if c["norm"] != "none" else 0.0), d ** -0.5
        if c["train"]:
            s["gq"], s["gk"] = _randn(gen, B, T, Hq, d, dtype=io), _randn(gen, B, T, Hk, d, dtype=io)
        return s
    gate = DTYPE[c["gate"]]
    B, H, dv = c["B"], c["H"], c["dv"]
    if c["op"] == "step":
        s["x"] = _randn(gen, B, H, dv, dtype=io)
        s["alpha"] = _gate(gen, (B, H, dv), c["form"], gate)
        s["beta"] = torch.sigmoid(_randn(gen, B, H, dv)).to(gate) if c["beta"] == "given" else None
        s["S"] = _randn(gen, B, H, dv)
        return s
    T = c["T"]
    if c["fused"]:  # stream | gate of one projection's output
        both = torch.empty(B, T, 2, H, dv, dtype=io, device="cuda")
        both[:, :, 0] = _randn(gen, B, T, H, dv, dtype=io)
        both[:, :, 1] = _gate(gen, (B, T, H, dv), c["form"], gate)
        s["x"], s["alpha"] = both[:, :, 0], both[:, :, 1]
    else:
        s["x"] = _randn(gen, B, T, H, dv, dtype=io)
        s["alpha"] = _gate(gen, (B, T, H, dv), c["form"], gate)
    s["beta"] = torch.sigmoid(_randn(gen, B, T, H, dv)).to(gate) if c["beta"] == "given" else None
    n = c["seqs"] or B
    s["S0"] = _randn(gen, n, H, dv)
    s["offsets"] = _offsets(gen, T, c["seqs"]) if c["seqs"] else None
    if c["train"]:
        s["dy"], s["dST"] = _randn(gen, B, T, H, dv, dtype=io), _randn(gen, n, H, dv)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _angles(s):
    """cos, sin [B, T, 1, rot / 2] in fp32 of angles formed in 64 bits."""
    a = s["pos"].double()[..., None] * s["inv_freq"]
    return torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]


def _pairs(x, rot, layout):
    """The two members of each rotated pair, and the channels that are not rotated."""
    r = x[..., :rot]
    e, o = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else (r[..., :rot // 2], r[..., rot // 2:])
    return e, o, x[..., rot:]


def _join(e, o, rest, layout):
    r = torch.stack([e, o], -1).flatten(-2) if layout == "interleaved" else torch.cat([e, o], -1)
    return torch.cat([r, rest], -1)


def _inverse_norm(x, norm, eps):
    if norm == "none":
        return None
    ss = (x * x).mean(-1, keepdim=True) if norm == "rms" else (x * x).sum(-1, keepdim=True)
    return torch.rsqrt(ss + eps)


def _prep(x, w, cs, scale, c, eps):
    x = x.float()
    r = _inverse_norm(x, c["norm"], eps)
    n = x if r is None else x * r
    n = n if w is None else n * w
    if cs is not None:
        e, o, rest = _pairs(n, c["rot"], c["layout"])
        n = _join(cs[0] * e - cs[1] * o, cs[1] * e + cs[0] * o, rest, c["layout"])
    return n * scale


def _prep_back(x, w, grad, cs, scale, c, eps):
    x, grad = x.float(), grad.float() * scale
    if cs is not None:
        e, o, rest = _pairs(grad, c["rot"], c["layout"])
        grad = _join(cs[0] * e + cs[1] * o, cs[0] * o - cs[1] * e, rest, c["layout"])
    r = _inverse_norm(x, c["norm"], eps)
    if r is None:
        return grad, None
    hat = x * r
    dw = None if w is None else (grad * hat).sum((0, 1, 2))
    t = grad if w is None else grad * w
    dot = (t * hat).mean(-1, keepdim=True) if c["norm"] == "rms" else (t * hat).sum(-1, keepdim=True)
    return r * (t - hat * dot), dw


def _coefficients(s, c):
    """a and b of h_t = a h_{t-1} + b x_t in fp32."""
    raw = s["alpha"].float()
    a = torch.exp(raw) if c["form"] == "log" else raw
    if c["beta"] == "given":
        return a, s["beta"].float()
    if c["beta"] == "one":
        return a, None
    return a, (-torch.expm1(raw) if c["form"] == "log" else 1 - a)


def _doubling(a, u, axis=1):
    """All h_t = a_t h_{t-1} + u_t from h_{-1} = 0: maps of 1, 2, 4, ... tokens are joined until they reach the start."""
    T, n = a.shape[axis], 1
    while n < T:
        late, early = [z.narrow(axis, n, T - n) for z in (a, u)], [z.narrow(axis, 0, T - n) for z in (a, u)]
        joined = torch.addcmul(late[1], late[0], early[1])
        u = torch.cat([u.narrow(axis, 0, n), joined], axis)
        if 2 * n < T:
            a = torch.cat([a.narrow(axis, 0, n), late[0] * early[0]], axis)
        n *= 2
    return u


def _borders(s):
    """Of packed sequences: which rows open and close a sequence, and the sequences that have rows."""
    off = s["offsets"].long()
    some = off[1:] > off[:-1]
    return off[:-1][some], off[1:][some] - 1, some.nonzero()[:, 0]


def _scan_plain(s, c):
    x = s["x"].float()
    a, b = _coefficients(s, c)
    u = x if b is None else b * x
    S0, dims = s["S0"], u.shape
    if s["offsets"] is None:
        u = u.clone()
        u[:, 0] += a[:, 0] * S0
        h = _doubling(a, u)
        ST = h[:, -1].clone()
        before = torch.cat([S0[:, None], h[:, :-1]], 1)
        inside = None
    else:
        first, last, ids = _borders(s)
        u, linked = u.clone(), a.clone()
        u[0, first] += a[0, first] * S0[ids]
        linked[0, first] = 0
        h = _doubling(linked, u)
        ST = S0.clone()
        ST[ids] = h[0, last]
        before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
        before[0, first] = S0[ids]
        inside = _rows(c["T"])
    y = h.to(s["x"].dtype)
    if inside is not None:
        y = y[:, inside[0]:inside[1]]
    out = {"y": y, "ST": ST}
    if not c["train"]:
        return out
    dy, dST = s["dy"].float(), s["dST"]
    gate = s["alpha"].dtype
    v, linked = a * dy, a
    if inside is None:
        v[:, -1] += a[:, -1] * dST
    else:
        v[0, last] += a[0, last] * dST[ids]
        linked = a.clone()
        linked[0, last] = 0
    G = _doubling(linked.flip(1), v.flip(1)).flip(1)
    after = torch.cat([G[:, 1:], torch.zeros_like(G[:, :1])], 1)
    if inside is None:
        after[:, -1] = dST
        out["dS0"] = G[:, 0].clone()
    else:
        after[0, last] = dST[ids]
        out["dS0"] = dST.clone()
        out["dS0"][ids] = G[0, first]
    g = dy + after
    da = g * (before - x) if c["beta"] == "coupled" else g * before
    grads = {"dx": (g if b is None else b * g).to(s["x"].dtype), "dalpha": (da * a if c["form"] == "log" else da).to(gate)}
    if c["beta"] == "given":
        grads["dbeta"] = (g * x).to(gate)
    out.update(grads if inside is None else {k: z[:, inside[0]:inside[1]] for k, z in grads.items()})
    return out


def _run_plain(s, c):
    if c["op"] == "qk":
        cs = _angles(s) if c["rot"] else None
        out = {}
        for n, scale in (("q", s["q_scale"]), ("k", 1.0)):
            out[n] = _prep(s[n], s["w" + n], cs, scale, c, s["eps"]).to(s[n].dtype)
            if c["train"]:
                d, dw = _prep_back(s[n], s["w" + n], s["g" + n], cs, scale, c, s["eps"])
                out["d" + n], out["dw" + n] = d.to(s[n].dtype), dw
        return out
    if c["op"] == "step":
        a, b = _coefficients(s, c)
        x = s["x"].float()
        s["S"].mul_(a).add_(x if b is None else b * x)
        return {"y": s["S"].to(s["x"].dtype), "S": s["S"]}
    return _scan_plain(s, c)


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _run_own(s, c):
    import gated_delta_rule_84_amd as g

    if c["op"] == "qk":
        how = dict(norm=c["norm"], wq=s["wq"], wk=s["wk"], eps=s["eps"], positions=s["pos"], inv_freq=s["inv_freq"],
                   layout=c["layout"], q_scale=s["q_scale"])
        q, k = g.qk_prep(s["q"], s["k"], **how)
        out = {"q": q, "k": k}
        if c["train"]:
            out["dq"], out["dk"], out["dwq"], out["dwk"] = g.qk_prep_bwd(s["q"], s["k"], s["gq"], s["gk"], **how)
        return out
    how = dict(beta=s["beta"], log_gate=c["form"] == "log", coupled=c["beta"] == "coupled")
    if c["op"] == "step":
        return {"y": g.scan_step(s["S"], s["x"], s["alpha"], **how), "S": s["S"]}
    how.update(S0=s["S0"], seq_offsets=s["offsets"])
    y, ST, ckpt = g.scan_fwd(s["x"], s["alpha"], want_ckpt=c["train"], **how)
    out = {"y": y, "ST": ST}
    if c["train"]:
        out["dx"], out["dalpha"], dbeta, out["dS0"] = g.scan_bwd(s["x"], s["alpha"], s["dy"], ckpt, dST=s["dST"], **how)
        if dbeta is not None:
            out["dbeta"] = dbeta
    if s["offsets"] is not None:  # rows that belong to no sequence are not written
        lo, hi = _rows(c["T"])
        out.update({k: out[k][:, lo:hi] for k in ("y", "dx", "dalpha", "dbeta") if k in out})
    return out


def run(state):
    c = state["case"]
    return _run_own(state, c) if own else _run_plain(state, c)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    es = SIZE[c["io"]]
    if c["op"] == "qk":
        rows = c["B"] * c["T"] * (c["Hq"] + c["Hk"])
        n = rows * c["d"]
        return {"bytes": n * es * (4 if c["train"] else 2) + 4 * c["B"] * c["T"] * bool(c["rot"]),
                "flops": n * (20 if c["train"] else 7)}
    gs = SIZE[c["gate"]]
    given = c["beta"] == "given"
    n = c["B"] * c.get("T", 1) * c["H"] * c["dv"]
    state = (c.get("seqs") or c["B"]) * c["H"] * c["dv"] * 4
    moved = n * (2 * es + gs * (2 if given else 1)) + 2 * state
    if c.get("train"):
        moved += n * (2 * es + gs * (3 if given else 1)) + 2 * state  # x and the gates once in all: each input is read once
    return {"bytes": moved, "flops": n * (12 if c.get("train") else 4)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_head(x, w, g, pos, f, scale, c, eps):
    """One tensor of heads, by 2 x 2 rotation matrices and the norm's Jacobian applied term by term."""
    x = x.double()
    d = x.shape[-1]
    if c["norm"] == "none":
        r, kappa = torch.ones_like(x[..., :1]), 0.0
    else:
        kappa = 1.0 if c["norm"] == "l2" else 1.0 / d
        r = (kappa * x.pow(2).sum(-1, keepdim=True) + eps).pow(-0.5)
    wd = torch.ones(d, dtype=torch.float64, device=x.device) if w is None else w.double()
    half = c["rot"] // 2
    i = torch.arange(half, device=x.device)
    ie, io_ = (2 * i, 2 * i + 1) if c["layout"] == "interleaved" else (i, i + half)
    y = x * r * wd
    if half:
        th = pos.double()[:, :, None, None] * f
        z = torch.polar(torch.ones_like(th), th)
        zz = torch.complex(y[..., ie], y[..., io_]) * z
        y[..., ie], y[..., io_] = zz.real, zz.imag
    y *= scale
    if g is None:
        return y, None, None
    gn = g.double() * scale
    if half:
        zz = torch.complex(gn[..., ie], gn[..., io_]) * z.conj()
        gn[..., ie], gn[..., io_] = zz.real, zz.imag
    dw = None if w is None else (gn * x * r).sum((0, 1, 2))
    t = gn * wd
    dx = r * t - kappa * r.pow(3) * (t * x).sum(-1, keepdim=True) * x
    return y, dx, dw


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "qk":
        if c["B"] * c["T"] * (c["Hq"] + c["Hk"]) * c["d"] > 1e9:
            return None
        out = {}
        for n, scale in (("q", s["q_scale"]), ("k", 1.0)):
            y, dx, dw = _exact_head(s[n], s["w" + n], s.get("g" + n), s["pos"], s["inv_freq"], scale, c, s["eps"])
            out[n] = y
            if c["train"]:
                out["d" + n], out["dw" + n] = dx, dw
        return out
    raw, x = s["alpha"].double(), s["x"].double()
    a = raw.exp() if c["form"] == "log" else raw
    b = s["beta"].double() if c["beta"] == "given" else (1 - a if c["beta"] == "coupled" else torch.ones_like(a))
    if c["op"] == "step":
        h = a * s["S"].double() + b * x
        return {"y": h, "S": h}
    T = x.shape[1]
    u = b * x
    h, before = torch.empty_like(u), torch.empty_like(u)
    S0 = s["S0"].double()
    off = None if s["offsets"] is None else s["offsets"].tolist()
    lo, hi = (0, T) if off is None else (off[0], off[-1])
    runs = [(0, T, slice(None))] if off is None else [(p, q, slice(i, i + 1)) for i, (p, q) in enumerate(zip(off, off[1:]))]
    ST = S0.clone()
    for p, q, who in runs:
        state = S0[who]
        for t in range(p, q):
            before[:, t] = state
            state = torch.addcmul(u[:, t], a[:, t], state, out=h[:, t])
        ST[who] = state
    out = {"y": h[:, lo:hi], "ST": ST}
    if not c["train"]:
        return out
    dST, g = s["dST"].double(), s["dy"].double()
    dS0 = dST.clone()
    for p, q, who in runs:
        down = dST[who]
        for t in reversed(range(p, q)):
            g[:, t] += down
            down = a[:, t] * g[:, t]
        dS0[who] = down
    da = g * (before - x) if c["beta"] == "coupled" else g * before
    out["dS0"] = dS0
    grads = {"dx": b * g, "dalpha": da * a if c["form"] == "log" else da}
    if c["beta"] == "given":
        grads["dbeta"] = g * x
    out.update({k: z[:, lo:hi] for k, z in grads.items()})
    return out
