"""The trainable delta rule on the GPU against its fp64 reference: forward, backward and single tokens.

Tolerances, relative to the norm of the exact result.  An fp32 product or sum is off by at most U = 2^-24 of its value; a
result is reached through at most four products one behind the other (pairs, their inverse, what the tokens write, state
or output), of at most dk + 128 terms together; the errors of n terms, up or down alike, come to sqrt(n) of one: 4
sqrt(dk + 128) U forward, twice that backward, which passes them again.  Gradients of log_gate and beta are dot
products: their errors go with the norms of the factors.  A result that is stored as bf16 is off by half a step, 2^-8 of
it, and what only such results read keeps two bf16 terms: 2^-16 a product, and eight of them with their sums stay below
2^-13."""
import numpy as np
import pytest

from oracle import delta as ref
from tests.gpu_util import gpu, log, to_np

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8


def _tol(dk, stored, io, backward=False, own=True):
    """Of a result stored as `stored`; own: it keeps fp32's precision with bf16 inputs too."""
    t = 4 * np.sqrt(dk + 128) * U * (2 if backward else 1)
    if io == "bf16" and not own:
        t = 2.0 ** -13
    return t + (HALF if stored == "bf16" else 0.0)


def _types(torch):
    return {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    def __init__(self, B, T, Hk, Hv, dk, dv, io="bf16", gate="f32", off=None, lay="dense", resets=False, decay=1.0, states=True,
                 seed=7):
        torch, _ = gpu()
        self.B, self.T, self.Hk, self.Hv, self.dk, self.dv, self.io, self.gate, self.off = B, T, Hk, Hv, dk, dv, io, gate, off
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        it, gt = _types(torch)[io], _types(torch)[gate]
        n = B if off is None else len(off) - 1
        k = r(B, T, Hk, dk)
        q, k, v = r(B, T, Hk, dk) / dk ** 0.5, k / k.norm(dim=-1, keepdim=True), r(B, T, Hv, dv)
        g, b = -decay * torch.nn.functional.softplus(r(B, T, Hv) - 2), torch.sigmoid(r(B, T, Hv))
        if resets:
            g[torch.rand(B, T, Hv, generator=gen) < 0.03] = -float("inf")
            g[torch.rand(B, T, Hv, generator=gen) < 0.05] = -25.0
        if off is not None:  # rows of no sequence hold anything
            out = torch.ones(T, dtype=torch.bool)
            out[off[0]:off[-1]] = False
            for x in (q, k, v, g, b):
                x[0, out] = float("nan")
        S0, dST = (0.3 * r(n, Hv, dk, dv), r(n, Hv, dk, dv)) if states else (None, None)
        do = r(B, T, Hv, dv).to(it)
        if lay == "dense":
            place = lambda xs: [x.cuda() for x in xs]  # noqa: E731
        else:  # slices of one projection's output; "odd": at addresses and strides of single elements
            shift = 1 if lay == "odd" else 8

            def place(xs):
                width = sum(x.shape[2:].numel() for x in xs) + 2 * shift
                whole = torch.full((B, T, width), float("nan"), dtype=xs[0].dtype, device="cuda")
                at, got = shift, []
                for x in xs:
                    m = x.shape[2:].numel()
                    to = whole[:, :, at:at + m].unflatten(2, x.shape[2:])
                    to.copy_(x)
                    got.append(to)
                    at += m
                return got
        self.q, self.k, self.v = place([x.to(it) for x in (q, k, v)])
        self.g, self.b = place([x.to(gt) for x in (g, b)])
        self.do = do.cuda()
        self.S0, self.dST = (None if x is None else x.cuda() for x in (S0, dST))
        self.seq = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
        if off is not None and n and off[0] == off[-1]:
            self.do.zero_()

    @property
    def inputs(self):
        return self.q, self.k, self.v, self.g, self.b

    def runs(self):
        return [(b, 0, self.T, b) for b in range(self.B)] if self.off is None else \
            [(0, p, e, i) for i, (p, e) in enumerate(zip(self.off, self.off[1:]))]

    def forward(self, **kw):
        _, g = gpu()
        return g.delta_fwd(*self.inputs, S0=self.S0, seq_offsets=self.seq, **kw)

    def backward(self, ckpt, **kw):
        _, g = gpu()
        return g.delta_bwd(*self.inputs, self.do, ckpt, dST=self.dST, seq_offsets=self.seq, **kw)


def _close(name, got, want, tol, size=None):
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want if size is None else size)
    log(f"  {name}: {err / max(norm, 1e-300):.2e} (bound {tol:.2e})")
    assert np.isfinite(got).all(), name
    assert err <= tol * norm, (name, err / max(norm, 1e-300), tol)


def _check(c, backward=True):
    x = [to_np(t) for t in c.inputs]
    do, S0, dST = to_np(c.do), None if c.S0 is None else to_np(c.S0), None if c.dST is None else to_np(c.dST)
    o, ST, ckpt = c.forward(want_ckpt=backward)
    got = [to_np(o), to_np(ST)]
    if backward:
        got += [to_np(t) for t in c.backward(ckpt)]
    parts = [[] for _ in range(10)]
    rows, seqs = [], []
    for b, p, e, i in c.runs():
        s = [t[b, p:e] for t in x]
        start = None if S0 is None else S0[i]
        ow, Sw, _ = ref.forward(*s, start)
        gw = ref.backward(*s, do[b, p:e], None if dST is None else dST[i], start) if backward else ()
        for to, val in zip(parts, (ow, Sw) + tuple(gw)):
            to.append(val)
        rows.append((b, p, e))
        seqs.append(i)
    take = lambda t: np.concatenate([t[b, p:e] for b, p, e in rows])  # noqa: E731
    cat, dk = np.concatenate, c.dk
    _close("o", take(got[0]), cat(parts[0]), _tol(dk, c.io, c.io, own=False))
    _close("ST", got[1][seqs], np.stack(parts[1]), _tol(dk, "f32", c.io))
    if backward:
        for j, name in enumerate(("dq", "dk", "dv")):
            _close(name, take(got[2 + j]), cat(parts[2 + j]), _tol(dk, c.io, c.io, True, own=False))
        _close("dlog_gate", take(got[5]), cat(parts[5]), _tol(dk, c.gate, c.io, True), cat(parts[8]))
        _close("dbeta", take(got[6]), cat(parts[6]), _tol(dk, c.gate, c.io, True), cat(parts[9]))
        _close("dS0", got[7][seqs], np.stack(parts[7]), _tol(dk, "f32", c.io, True))


SHAPES = [
    dict(B=1, T=1, Hk=1, Hv=1, dk=8, dv=8),
    dict(B=3, T=1, Hk=2, Hv=4, dk=128, dv=128),
    dict(B=2, T=63, Hk=1, Hv=2, dk=16, dv=24, lay="fused"),
    dict(B=1, T=64, Hk=2, Hv=2, dk=64, dv=64, states=False),
    dict(B=2, T=65, Hk=2, Hv=4, dk=72, dv=40, resets=True, lay="odd"),
    dict(B=1, T=200, Hk=1, Hv=3, dk=128, dv=128, lay="fused"),
    dict(B=2, T=130, Hk=2, Hv=2, dk=104, dv=8, resets=True),
    dict(B=1, T=129, Hk=1, Hv=1, dk=40, dv=120, lay="odd"),
    dict(B=1, T=210, Hk=2, Hv=4, dk=64, dv=56, off=[3, 3, 4, 67, 131, 196, 196, 203], lay="fused"),
    dict(B=1, T=190, Hk=1, Hv=2, dk=120, dv=128, off=[0, 65, 65, 190], resets=True, lay="odd"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, (s[k] for k in ("B", "T", "Hk", "Hv", "dk", "dv")))))
@pytest.mark.parametrize("io,gate", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_against_reference(io, gate, shape):
    _check(Case(io=io, gate=gate, **shape))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (48, 104)])
def test_many_heads(io, dk, dv):
    """So many columns of states that a workgroup of the recurrence takes two tiles a wave pair more."""
    _check(Case(B=36, T=70, Hk=1, Hv=2, dk=dk, dv=dv, io=io, lay="fused" if dk == 64 else "dense"))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [1e-4, 30.0, 400.0])
def test_weak_and_strong_decay(io, decay):
    _check(Case(B=1, T=150, Hk=1, Hv=2, dk=32, dv=32, io=io, decay=decay))


def test_growing_states():
    """Gates above 0: e^0.02 a token."""
    torch, _ = gpu()
    c = Case(B=1, T=150, Hk=1, Hv=2, dk=32, dv=32, io="f32")
    c.g.copy_(torch.rand(c.g.shape, generator=torch.Generator().manual_seed(3)) * 0.04)
    _check(c)


def test_no_tokens_and_empty_sequences():
    """ST = S0 and dS0 = dST where there is no token."""
    torch, g = gpu()
    for kw in (dict(B=2, T=0), dict(B=1, T=5, off=[2, 2, 2, 2])):
        c = Case(Hk=1, Hv=2, dk=16, dv=16, **kw)
        o, ST, ck = c.forward(want_ckpt=True)
        assert torch.equal(ST, c.S0)
        grads = c.backward(ck)
        assert torch.equal(grads[5], c.dST)
        c.S0 = c.dST = None
        assert (c.forward()[1] == 0).all()
        assert (c.backward(ck)[5] == 0).all()
    c = Case(B=1, T=5, Hk=1, Hv=1, dk=8, dv=8, off=[0])
    assert c.forward()[1].shape[0] == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_of_no_sequence(io):
    """They hold NaN, nothing of them reaches a result, and theirs stay as they were; guards around outputs stay too."""
    torch, g = gpu()
    c = Case(B=1, T=150, Hk=1, Hv=2, dk=24, dv=40, off=[10, 80, 80, 121], io=io)
    it, n = _types(torch)[io], 3
    desc = g.DeltaDesc(1, 150, 1, 2, 24, 40, g.GDR_BF16 if io == "bf16" else g.GDR_F32, g.GDR_F32, 0, 0, 0, 0, 0)
    guard = 64

    def room(shape, dtype):
        m = int(np.prod(shape))
        whole = torch.full((m + 2 * guard,), 7.0, dtype=dtype, device="cuda")
        return whole, whole[guard:guard + m].view(shape)
    f32 = torch.float32
    o, ST = room((1, 150, 2, 40), it), room((n, 2, 24, 40), f32)
    ck = room((g.gdr_delta_ckpt_size(desc, n) // 4,), f32)
    need = g.gdr_delta_workspace_size(desc, n, True)
    ws = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")  # NaN as any type
    rc = g.gdr_delta_fwd(desc, *c.inputs, c.seq, n, c.S0, o[1], ST[1], ck[1], ws, need)
    assert rc == g.GDR_OK
    outs = [room((1, 150, 1, 24), it), room((1, 150, 1, 24), it), room((1, 150, 2, 40), it), room((1, 150, 2), f32),
            room((1, 150, 2), f32), room((n, 2, 24, 40), f32)]
    c.do[0, :10] = float("nan")
    c.do[0, 121:] = float("nan")
    ws.fill_(255)
    rc = g.gdr_delta_bwd(desc, *c.inputs, c.seq, n, ck[1], c.do, c.dST, *(x[1] for x in outs), ws, need)
    assert rc == g.GDR_OK
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all()
    for whole, t in [o, ST, ck] + outs:
        assert (whole[:guard] == 7).all() and (whole[-guard:] == 7).all()
        if t.dim() > 1 and t.shape[1] == 150:
            assert (t[0, :10] == 7).all() and (t[0, 121:] == 7).all()
            assert torch.isfinite(t[0, 10:121].float()).all()
    plain = Case(B=1, T=150, Hk=1, Hv=2, dk=24, dv=40, off=[10, 80, 80, 121], io=io)
    o2, S2, ck2 = plain.forward(want_ckpt=True)
    assert torch.equal(o2[0, 10:121], o[1][0, 10:121]) and torch.equal(S2, ST[1])


def test_state_in_place_and_resumed():
    """Two halves, the second from the first one's state in place, give the whole; a half ends inside a chunk."""
    torch, g = gpu()
    c = Case(B=2, T=150, Hk=1, Hv=2, dk=64, dv=64, io="f32")
    o, ST, _ = c.forward()
    S, parts = c.S0.clone(), []
    for p, e in ((0, 91), (91, 150)):
        cut = [x[:, p:e].contiguous() for x in c.inputs]
        desc = g.DeltaDesc(2, e - p, 1, 2, 64, 64, g.GDR_F32, g.GDR_F32, 0, 0, 0, 0, 0)
        out = torch.empty_like(cut[2])
        need = g.gdr_delta_workspace_size(desc)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert g.gdr_delta_fwd(desc, *cut, None, 0, S, out, S, None, ws, need) == g.GDR_OK
        parts.append(out)
    tol = 2 * _tol(64, "f32", "f32")  # each side its own
    _close("o", to_np(torch.cat(parts, 1)), to_np(o), tol)
    _close("ST", to_np(S), to_np(ST), tol)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_reset_forgets_exactly(io):
    """Behind a gate of -inf the results are those of a start there; the gate's gradient is 0."""
    torch, g = gpu()
    c = Case(B=1, T=140, Hk=1, Hv=2, dk=64, dv=64, io=io)
    c.g[:, 128] = -float("inf")
    o, ST, ck = c.forward(want_ckpt=True)
    grads = c.backward(ck)
    assert (grads[3][:, 128] == 0).all() and (grads[5].abs().sum() > 0)
    tail = [x[:, 128:].contiguous() for x in c.inputs]
    o2, S2, _ = g.delta_fwd(*tail)
    assert torch.equal(o[:, 128:], o2) and torch.equal(ST, S2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hk,Hv,dk,dv,lay", [(1, 1, 1, 8, 8, "dense"), (5, 2, 6, 72, 104, "odd"), (3, 4, 4, 128, 128, "fused"),
                                                (600, 1, 2, 16, 64, "dense")])
def test_step(io, B, Hk, Hv, dk, dv, lay):
    torch, g = gpu()
    c = Case(B=B, T=3, Hk=Hk, Hv=Hv, dk=dk, dv=dv, io=io, lay=lay)
    c.g[0, 1, 0] = -float("inf")
    S = c.S0.clone()
    outs = [g.delta_step(S, *(x[:, t] for x in c.inputs)) for t in range(3)]  # strides of a whole stream
    want = [ref.forward(*(to_np(x)[b] for x in c.inputs), to_np(c.S0)[b]) for b in range(B)]
    # a step keeps fp32 throughout: two contractions and an update
    _close("o", to_np(torch.stack(outs, 1)), np.stack([w[0] for w in want]), _tol(dk, io, "f32"))
    _close("S", to_np(S), np.stack([w[1] for w in want]), _tol(dk, "f32", "f32"))


def test_step_follows_forward():
    torch, g = gpu()
    c = Case(B=2, T=70, Hk=1, Hv=2, dk=64, dv=128, io="f32")
    o, ST, _ = c.forward()
    S = c.S0.clone()
    out = torch.stack([g.delta_step(S, *(x[:, t].contiguous() for x in c.inputs)) for t in range(70)], 1)
    tol = _tol(64, "f32", "f32") * 2  # each side its own
    _close("o", to_np(out), to_np(o), tol)
    _close("S", to_np(S), to_np(ST), tol)


def test_gradients_against_differences():
    """(f(x + h d) - f(x - h d)) / 2 h of the GPU's own forward pass.  f is linear in q, v and S0: only f's rounding over h is
    left, 4 sqrt(dk + 128) U |f|, |f| at most the norms' products.  In k, log_gate and beta h^2 / 6 of the third derivative is left as
    well: d moves a product of up to T factors by h sqrt(T) <= 0.03, so below 0.03^2 / 6 < 2e-4 of the products' size."""
    torch, g = gpu()
    c = Case(B=1, T=70, Hk=1, Hv=2, dk=32, dv=32, io="f32")
    ck = c.forward(want_ckpt=True)[2]
    grads = c.backward(ck)
    gen = torch.Generator().manual_seed(9)
    for name, x, grad in zip(("q", "k", "v", "log_gate", "beta", "S0"), c.inputs + (c.S0,), grads):
        linear = name in ("q", "v", "S0")
        h = 0.5 if linear else 2.0 ** -8
        d = torch.randn(x.shape, generator=gen).cuda()
        keep, sides = x.clone(), []
        size = 0.0
        for sign in (1, -1):
            x.copy_(keep + sign * h * d)
            o, ST, _ = c.forward()
            terms = (o.double() * c.do.double()).sum() + (ST.double() * c.dST.double()).sum()
            size = max(size, float(o.double().norm() * c.do.double().norm() + ST.double().norm() * c.dST.double().norm()))
            sides.append(float(terms))
        moved = ((keep + h * d) - (keep - h * d)).double() / (2 * h)  # the step that fp32 took
        x.copy_(keep)
        want, got = float((grad.double() * moved).sum()), (sides[0] - sides[1]) / (2 * h)
        bound = 4 * np.sqrt(160) * U * size / h + (0 if linear else 2e-4 * size) + 8 * np.sqrt(160) * U * float(
            grad.double().norm() * moved.norm())
        log(f"  {name}: {got:.6f} against {want:.6f}, bound {bound:.1e}")
        assert abs(got - want) <= bound


def test_deterministic_and_whatever_the_workspace_held():
    torch, g = gpu()
    c = Case(B=1, T=300, Hk=2, Hv=4, dk=128, dv=64, off=[0, 100, 101, 300])
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((1 << 25,), fill, dtype=torch.uint8, device="cuda")
        o, ST, ck = c.forward(want_ckpt=True, workspace=ws)
        ws.fill_(fill)
        now = [o, ST] + list(c.backward(ck, workspace=ws))
        if first:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_two_streams_at_once():
    torch, g = gpu()
    cases = [Case(B=1, T=700, Hk=2, Hv=4, dk=64, dv=64, seed=s) for s in (1, 2)]
    want = []
    for c in cases:
        o, ST, ck = c.forward(want_ckpt=True)
        want.append([o, ST, *c.backward(ck)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        got = []
        for c, s in zip(cases, streams):
            o, ST, ck = c.forward(want_ckpt=True, stream=s)
            got.append([o, ST, *c.backward(ck, stream=s)])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed():
    """Forward, backward and a step in one graph, replayed on other inputs with eager work between the replays."""
    torch, g = gpu()
    c = Case(B=2, T=100, Hk=1, Hv=2, dk=64, dv=64)
    state = c.S0.clone()

    def run():
        o, ST, ck = c.forward(want_ckpt=True)
        state.copy_(ST)
        y = g.delta_step(state, *(x[:, 0] for x in c.inputs))
        return [o, ST, *c.backward(ck), y, state]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for seed in (11, 12, 13):
        new = Case(B=2, T=100, Hk=1, Hv=2, dk=64, dv=64, seed=seed)
        for to, x in zip(c.inputs + (c.do, c.S0, c.dST), new.inputs + (new.do, new.S0, new.dST)):
            to.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    """Rows of a wide projection whose elements lie past 2^32, and kept states past 4 GiB."""
    torch, g = gpu()
    T, ld = 70000, 65536
    whole = torch.empty(1, T, ld, dtype=torch.bfloat16, device="cuda")
    c = Case(B=1, T=130, Hk=1, Hv=1, dk=64, dv=64, io="bf16", off=[0, 130])
    at = 0
    wide = []
    for x in (c.q, c.k, c.v):
        to = whole[:, :, at:at + 64].unflatten(2, (1, 64))
        to[:, T - 130:] = x
        wide.append(to)
        at += 64
    pad = lambda x: torch.cat([x.new_full((1, T - 130) + x.shape[2:], float("nan")), x], 1)  # noqa: E731
    seq = torch.tensor([T - 130, T], dtype=torch.int32, device="cuda")
    how = dict(seq_offsets=seq)
    o, ST, ck = g.delta_fwd(*wide, pad(c.g), pad(c.b), S0=c.S0, want_ckpt=True, **how)
    grads = g.delta_bwd(*wide, pad(c.g), pad(c.b), pad(c.do), ck, dST=c.dST, **how)
    o2, S2, ck2 = c.forward(want_ckpt=True)
    grads2 = c.backward(ck2)
    assert torch.equal(o[:, T - 130:], o2) and torch.equal(ST, S2) and torch.equal(grads[5], grads2[5])
    for a, b in zip(grads[:5], grads2[:5]):
        assert torch.equal(a[:, T - 130:], b)
    del whole, wide, o, ck, grads
    T, H, tail = 66000, 48, 200
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, do = (r(1, T, H, 128) * f for f in (0.09, 0.09, 1, 1))
    a, b = -torch.rand(1, T, H, generator=gen, device="cuda"), torch.rand(1, T, H, generator=gen, device="cuda")
    off = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    o, ST, ck = g.delta_fwd(q, k, v, a, b, seq_offsets=off, want_ckpt=True)
    assert ck.numel() * 4 > 1 << 32
    grads = g.delta_bwd(q, k, v, a, b, do, ck, seq_offsets=off)
    # A call with other numbers of sequences and heads may sum in another order (a state's columns on one wave or on two), so
    # the last sequence alone need not give the same bits: some of its heads are held to the reference, with the bounds above.
    heads = [0, 17, 31, 47]
    end = [to_np(x[0, T - tail:, heads]) for x in (q, k, v, a, b, do)]
    ow, Sw, _ = ref.forward(*end[:5])
    want = ref.backward(*end)
    _close("o", to_np(o[0, T - tail:, heads]), ow, _tol(128, "bf16", "bf16", own=False))
    _close("ST", to_np(ST[1, heads]), Sw, _tol(128, "f32", "bf16"))
    for name, got, exact in zip(("dq", "dk", "dv"), grads, want):
        _close(name, to_np(got[0, T - tail:, heads]), exact, _tol(128, "bf16", "bf16", True, own=False))
    _close("dlog_gate", to_np(grads[3][0, T - tail:, heads]), want[3], _tol(128, "f32", "bf16", True), want[6])
    _close("dbeta", to_np(grads[4][0, T - tail:, heads]), want[4], _tol(128, "f32", "bf16", True), want[7])
    _close("dS0", to_np(grads[5][1, heads]), want[5], _tol(128, "f32", "bf16", True))
