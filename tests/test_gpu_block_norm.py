"""The block norm on the GPU against its fp64 reference, and the layer that it, the preparation and the trainable delta
rule are: forward, backward, prefill and then token by token.

Tolerances.  U = 2^-24 is what one fp32 operation is off by, of its value.  y: the sum of squares has at most 32 terms a
lane and 9 levels above them, halved by the root: 21 U; the gate's factor |z| 1.45 U + 4 U for |z| up to 12: 22 U; the
products and the sum 8 U: below 64 U of |scale act u| + |res_scale residual|, each element.  n: the same again through
the second sum, 128 U.  Gradients of x, gate and residual pass both norms forward and back, on dot products whose errors
go with the rows' norms: 256 U of the tensor's norm.  Weights' gradients: their terms are off by 256 U, and the sum of N
rows, up or down alike, by sqrt(N) U.  A value stored as bf16 is off by half a step, 2^-8 of it, more."""
import numpy as np
import pytest

from oracle import block_norm as ref
from oracle import delta as delta_ref
from tests.gpu_util import gpu, log, to_np

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8


def _norm_close(name, got, want, tol):
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    log(f"  {name}: {err / max(norm, 1e-300):.2e} (bound {tol:.2e})")
    assert np.isfinite(got).all(), name
    assert err <= tol * norm, (name, err / max(norm, 1e-300), tol)


def _inputs(B, T, H, d, io, wt, lay, seed=3, clip=12.0):
    torch, _ = gpu()
    types = {"bf16": torch.bfloat16, "f32": torch.float32}
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, z, res = r(B, T, H, d), (2 * r(B, T, H, d)).clamp(-clip, clip), r(B, T, H, d)
    w, w2 = 1 + 0.3 * r(d), 1 + 0.3 * r(d)
    dy, dn = r(B, T, H, d), r(B, T, H, d)

    def place(t):
        t = t.to(types[io])
        if lay == "dense":
            return t.cuda()
        shift = 1 if lay == "odd" else 16
        whole = torch.full((B, T, H * d + 2 * shift), float("nan"), dtype=t.dtype, device="cuda")
        to = whole[:, :, shift:shift + H * d].unflatten(2, (H, d))
        to.copy_(t)
        return to
    return [place(t) for t in (x, z, res)] + [t.to(types[wt]).cuda() for t in (w, w2)] + [t.to(types[io]).cuda() for t in (dy, dn)]


def _check(B, T, H, d, *, io="bf16", wt="f32", lay="dense", norm="rms", act="silu", weight=True, residual=True, next_norm="rms",
           next_weight=True, eps=1e-6, scale=0.7, res_scale=1.3):
    torch, g = gpu()
    x, z, res, w, w2, dy, dn = _inputs(B, T, H, d, io, wt, lay)
    next_norm = None if next_norm == "none" else next_norm
    how = dict(norm=norm, weight=w if weight else None, gate=z if act else None, act=act, scale=scale,
               residual=res if residual else None, res_scale=res_scale, eps=eps, next_norm=next_norm,
               next_weight=w2 if next_norm and next_weight else None)
    y, n = g.block_norm(x, **how)
    grads = g.block_norm_bwd(x, dy, dn=dn if next_norm else None, **how)
    f32 = np.float32
    how64 = {k: (to_np(v).reshape(-1, d) if v.dim() > 1 else to_np(v)) if isinstance(v, torch.Tensor) else v for k, v in how.items()}
    # the scalars as the fp32 values they are handed over as
    how64.update(eps=float(f32(eps)), scale=float(f32(scale)), res_scale=float(f32(res_scale)))
    flat = lambda t: to_np(t).reshape(-1, d)  # noqa: E731
    X = flat(x)
    yw, nw = ref.forward(X, **how64)
    inner = ref.forward(X, **dict(how64, residual=None, next_norm=None, next_weight=None))[0]
    size = np.abs(inner) + (np.abs(how64["res_scale"] * how64["residual"]) if residual else 0)
    half = HALF if io == "bf16" else 0.0
    err = np.abs(flat(y) - yw) - half * np.abs(yw) - 64 * U * size
    log(f"  y: {np.max(np.abs(flat(y) - yw) / np.maximum(size, 1e-300)):.2e}")
    assert np.isfinite(flat(y)).all() and (err <= 0).all(), err.max()
    if next_norm:
        m = (yw * yw).sum(-1, keepdims=True) / (d if next_norm == "rms" else 1) + how64["eps"]
        scale_n = size / np.sqrt(m) * (np.abs(how64["next_weight"]) if next_weight else 1)
        # the sum's own share goes with |n| of a row's worst element relative to its root
        grow = np.linalg.norm(size, axis=-1, keepdims=True) / np.maximum(np.linalg.norm(yw, axis=-1, keepdims=True), 1e-300)
        err = np.abs(flat(n) - nw) - half * np.abs(nw) - 128 * U * grow * scale_n
        assert np.isfinite(flat(n)).all() and (err <= 0).all(), err.max()
    want = ref.backward(X, flat(dy), dn=flat(dn) if next_norm else None, **how64)
    N = B * T * H
    for name, got, exact in zip(("dx", "dgate", "dresidual", "dweight", "dnext_weight"), grads, want):
        assert (got is None) == (exact is None), name
        if got is not None:
            sums = name.endswith("weight")
            _norm_close(name, to_np(got).reshape(exact.shape), exact, (256 + (np.sqrt(N) if sums else 0)) * U + (0 if sums else half))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("act", [None, "linear", "sigmoid", "silu"])
@pytest.mark.parametrize("next_norm", ["none", "l2", "rms"])
def test_forms(io, norm, act, next_norm):
    _check(2, 7, 3, 40, io=io, norm=norm, act=act, next_norm=next_norm, residual=act != "linear", weight=norm != "l2")


@pytest.mark.parametrize("io,wt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,T,H,d,lay", [
    (1, 1, 1, 8, "dense"), (3, 5, 2, 64, "odd"), (2, 33, 4, 128, "fused"), (1, 300, 3, 72, "odd"), (2, 9, 1, 264, "fused"),
    (1, 70, 1, 1000, "odd"), (1, 40, 1, 2048, "dense"), (1, 9, 1, 2056, "fused"), (1, 7, 1, 4104, "odd"), (1, 6, 1, 8192, "fused")])
def test_widths(io, wt, B, T, H, d, lay):
    _check(B, T, H, d, io=io, wt=wt, lay=lay)


@pytest.mark.parametrize("d", [64, 128, 1024])
def test_many_rows(d):
    """More rows than workgroups hold at once: each takes several."""
    _check(2, 20000 // (d // 64), 2, d, residual=False, next_norm="none")
    _check(1, 9001, 1, d, io="f32", next_weight=False)


def test_rows_of_zeros():
    """Without eps a norm of 0 gives 0, forward and backward."""
    torch, g = gpu()
    x = torch.zeros(1, 3, 2, 16, device="cuda")
    x[0, 1] = 1
    w, dy = torch.ones(16, device="cuda"), torch.ones_like(x)
    for norm in ("rms", "l2"):
        y, n = g.block_norm(x, norm=norm, weight=w, eps=0.0, next_norm=norm, next_weight=w)
        grads = g.block_norm_bwd(x, dy, dn=dy, norm=norm, weight=w, eps=0.0, next_norm=norm, next_weight=w)
        for t in (y, n, grads[0]):
            assert torch.isfinite(t).all() and (t[0, 0] == 0).all() and (t[0, 2] == 0).all()
        assert torch.isfinite(grads[3]).all() and torch.isfinite(grads[4]).all()


def test_gates_far_out():
    """Factors of gates from -100 to 100: sigmoid to 0 and 1, silu to 0 and the gate, with finite gradients."""
    torch, g = gpu()
    z = torch.linspace(-100, 100, 64, device="cuda").reshape(1, 1, 1, 64)
    x, one = torch.ones_like(z), torch.ones_like(z)
    for act in ("sigmoid", "silu"):
        how = dict(norm="none", gate=z, act=act)
        y, _ = g.block_norm(x, **how)
        grads = g.block_norm_bwd(x, one, **how)
        z64 = to_np(z)[0, 0]
        want = ref.forward(np.ones((1, 64)), norm="none", gate=z64, act=act)[0]
        # |z| 1.45 U of the factor through the exponent, and what is below fp32's smallest normal number
        assert (np.abs(to_np(y)[0, 0] - want) <= 256 * U * np.abs(want) + 2.0 ** -125 * 100).all()
        back = ref.backward(np.ones((1, 64)), np.ones((1, 64)), norm="none", gate=z64, act=act)
        for a, b in zip(grads[:2], back[:2]):
            assert (np.abs(to_np(a)[0, 0] - b) <= 256 * U * (np.abs(b) + np.abs(z64) * np.exp(-np.abs(z64))) + 2.0 ** -125 * 1e4).all()


def test_nan_stays_in_its_row():
    torch, g = gpu()
    x, z, res, w, w2, dy, dn = _inputs(1, 50, 2, 128, "f32", "f32", "dense")
    how = dict(weight=w, gate=z, act="silu", residual=res, next_norm="rms", next_weight=w2)
    y, n = g.block_norm(x, **how)
    dx = g.block_norm_bwd(x, dy, dn=dn, **how)[0]
    x[0, 17, 1, 5] = float("nan")
    y2, n2 = g.block_norm(x, **how)
    dx2 = g.block_norm_bwd(x, dy, dn=dn, **how)[0]
    keep = torch.ones(50, 2, dtype=torch.bool, device="cuda")
    keep[17, 1] = False
    for a, b in ((y, y2), (n, n2), (dx, dx2)):
        assert torch.equal(a[0][keep], b[0][keep]) and torch.isnan(b[0, 17, 1]).all()


def test_residual_in_place_and_no_rows():
    torch, g = gpu()
    x, z, res, w, w2, dy, dn = _inputs(2, 30, 1, 512, "bf16", "f32", "dense")
    how = dict(weight=w, residual=res, next_norm="rms", next_weight=w2)
    y, n = g.block_norm(x, **how)
    stream = res.clone()
    y2, n2 = g.block_norm(x, **dict(how, residual=stream), out=stream)
    assert y2.data_ptr() == stream.data_ptr() and torch.equal(y2, y) and torch.equal(n2, n)
    none = x[:, :0].contiguous()
    grads = g.block_norm_bwd(none, none, dn=none, **dict(how, residual=none))
    assert (grads[3] == 0).all() and (grads[4] == 0).all() and g.block_norm(none, **dict(how, residual=none))[0].numel() == 0


def test_guards_and_workspace():
    """Nothing is written around outputs; what the workspace held does not matter; the same results each time."""
    torch, g = gpu()
    x, z, res, w, w2, dy, dn = _inputs(1, 77, 3, 72, "bf16", "f32", "odd")
    desc = g.BlockNormDesc(1, 77, 3, 72, g.GDR_BF16, g.GDR_F32, g.GDR_NORM_RMS, g.GDR_NORM_L2, g.GDR_ACT_SIGMOID, 1e-6, 1.0, 1.0,
                           x.stride(1), z.stride(1), res.stride(1))
    m, pad = x.numel(), 64
    room = lambda k, t: torch.full((k + 2 * pad,), 7.0, dtype=t, device="cuda")  # noqa: E731
    need = g.gdr_block_norm_bwd_workspace_size(desc)
    first = None
    for fill in (0, 255):
        outs = [room(m, x.dtype) for _ in range(5)] + [room(72, torch.float32) for _ in range(2)]
        inner = [t[pad:-pad] for t in outs]
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        assert g.gdr_block_norm_fwd(desc, x, z, res, w, w2, inner[0], inner[1]) == g.GDR_OK
        assert g.gdr_block_norm_bwd(desc, x, z, res, w, w2, dy, dn, *inner[2:], ws, need) == g.GDR_OK
        torch.cuda.synchronize()
        for t in outs:
            assert (t[:pad] == 7).all() and (t[-pad:] == 7).all()
        assert (ws[need:] == fill).all()
        if first:
            assert all(torch.equal(a, b) for a, b in zip(first, outs))
        first = outs


def test_captured_and_on_another_stream():
    torch, g = gpu()
    x, z, res, w, w2, dy, dn = _inputs(2, 40, 2, 128, "bf16", "f32", "dense")
    how = dict(weight=w, gate=z, act="silu", residual=res, next_norm="rms", next_weight=w2)
    run = lambda **kw: [*g.block_norm(x, **how, **kw), *g.block_norm_bwd(x, dy, dn=dn, **how, **kw)]  # noqa: E731
    side = torch.cuda.Stream()
    want = run()
    torch.cuda.synchronize()
    got = run(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for seed in (21, 22, 23):
        for to, t in zip((x, z, res, w, w2, dy, dn), _inputs(2, 40, 2, 128, "bf16", "f32", "dense", seed=seed)):
            to.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in outs]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_rows_past_32_bits():
    """Rows of a strided input whose elements lie past 2^32, and more than 2^32 bytes of output."""
    torch, g = gpu()
    T, ld = 70000, 65536
    whole = torch.empty(1, T, ld, dtype=torch.bfloat16, device="cuda")
    x = whole[:, :, 64:64 + 256].unflatten(2, (2, 128))
    new = torch.randn(1, 40, 2, 128, device="cuda").bfloat16()
    x[:, T - 40:] = new
    y, _ = g.block_norm(x)
    assert torch.equal(y[:, T - 40:], g.block_norm(new)[0])
    del whole, x, y
    big = torch.randn(1, 300000, 1, 8192, device="cuda", dtype=torch.bfloat16)
    y, _ = g.block_norm(big)
    tail = big[:, -9:].contiguous()
    assert torch.equal(y[:, -9:], g.block_norm(tail)[0])


# ---------------------------------------------------------------------------
# a layer: fused projection -> qk_prep -> delta rule -> gated norm of its heads -> join with the residual and the
# next layer's norm
# ---------------------------------------------------------------------------
H, D = 4, 64
PREP, HEADS, JOIN = dict(norm="l2", eps=1e-6, q_scale=D ** -0.5), dict(norm="rms", act="silu"), dict(norm="none", next_norm="rms")


def _layer_inputs(B, T):
    torch, _ = gpu()
    gen = torch.Generator().manual_seed(41)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    proj = r(B, T, 4 * H * D)  # q, k, v, gate
    gates = torch.cat([-torch.nn.functional.softplus(r(B, T, H) - 2), torch.sigmoid(r(B, T, H))], -1)
    return proj, gates, r(B, T, 1, H * D), 1 + 0.2 * r(D), 1 + 0.2 * r(H * D)


def _cut(proj, gates):
    q, k, v, z = (proj[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(4))
    return q, k, v, z, gates[..., :H], gates[..., H:]


def test_layer_forward_and_backward():
    torch, g = gpu()
    B, T = 2, 150
    proj, gates, res, w, w2 = _layer_inputs(B, T)
    q, k, v, z, a, b = _cut(proj, gates)
    qq, kk = g.qk_prep(q, k, **PREP)
    o, ST, ck = g.delta_fwd(qq, kk, v, a, b, want_ckpt=True)
    y, _ = g.block_norm(o, weight=w, gate=z, **HEADS)
    flat = y.view(B, T, 1, H * D)
    h, n = g.block_norm(flat, residual=res, next_weight=w2, **JOIN)
    gen = torch.Generator().manual_seed(43)
    dh, dn = (torch.randn(B, T, 1, H * D, generator=gen).cuda() for _ in range(2))
    dflat, _, dres, _, dw2 = g.block_norm_bwd(flat, dh, dn=dn, residual=res, next_weight=w2, **JOIN)
    do, dz, _, dw, _ = g.block_norm_bwd(o, dflat.view(B, T, H, D), weight=w, gate=z, **HEADS)
    dqq, dkk, dv, dg, db, _ = g.delta_bwd(qq, kk, v, a, b, do, ck)
    dq, dk = g.qk_prep_bwd(q, k, dqq, dkk, **PREP)[:2]

    f = lambda t: to_np(t)  # noqa: E731
    eps = float(np.float32(1e-6))
    scale = float(np.float32(D ** -0.5))
    q64, k64 = f(q), f(k)
    unit = lambda x: x / np.sqrt((x * x).sum(-1, keepdims=True) + eps)  # noqa: E731
    qn, kn = unit(q64) * scale, unit(k64)
    seqs = [delta_ref.forward(qn[i], kn[i], f(v)[i], f(a)[i], f(b)[i]) for i in range(B)]
    o64 = np.stack([s[0] for s in seqs])
    heads = dict(norm="rms", weight=f(w), gate=f(z).reshape(-1, D), act="silu", eps=eps)
    join = dict(norm="none", residual=f(res).reshape(-1, H * D), next_norm="rms", next_weight=f(w2), eps=eps)
    y64, _ = ref.forward(o64.reshape(-1, D), **heads)
    h64, n64 = ref.forward(y64.reshape(-1, H * D), **join)
    back = ref.backward(y64.reshape(-1, H * D), f(dh).reshape(-1, H * D), dn=f(dn).reshape(-1, H * D), **join)
    inner = ref.backward(o64.reshape(-1, D), back[0].reshape(-1, D), **heads)
    do64 = inner[0].reshape(B, T, H, D)
    grads = [np.stack(x) for x in zip(*(delta_ref.backward(qn[i], kn[i], f(v)[i], f(a)[i], f(b)[i], do64[i])[:5] for i in range(B)))]

    def through_unit(x, gr):
        r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) + eps)
        return r * gr - r ** 3 * (gr * x).sum(-1, keepdims=True) * x
    # the stages' bounds added: preparation 64 U, delta rule 4 sqrt(dk + 128) U < 64 U, norms 64 and 128 U; a row norm turns the
    # errors of small heads' outputs up by at most their share, a factor of 4 here
    fwd = 4 * (64 + 64 + 64 + 128) * U
    _norm_close("h", f(h).reshape(-1, H * D), h64, fwd)
    _norm_close("n", f(n).reshape(-1, H * D), n64, fwd)
    bwd = fwd + 4 * (256 + 256 + 128 + 64) * U
    _norm_close("dresidual", f(dres).reshape(-1, H * D), back[2], bwd)
    _norm_close("dw2", f(dw2), back[4], bwd)
    _norm_close("dw", f(dw), inner[3], bwd)
    _norm_close("dz", f(dz).reshape(-1, D), inner[1], bwd)
    _norm_close("dv", f(dv), grads[2], bwd)
    _norm_close("dq", f(dq), through_unit(q64, grads[0] * scale), bwd)
    _norm_close("dk", f(dk), through_unit(k64, grads[1]), bwd)
    _norm_close("dlog_gate", f(dg), grads[3], 4 * bwd)  # dot products: their factors' norms are larger than the sums
    _norm_close("dbeta", f(db), grads[4], 4 * bwd)


def test_layer_prefill_then_tokens():
    """A prompt in one call and then token by token: the same as the whole in one call."""
    torch, g = gpu()
    B, T, more = 2, 130, 6
    proj, gates, res, w, w2 = _layer_inputs(B, T + more)

    def layer(p, e, S):
        cut = lambda t: t[:, p:e].contiguous()  # noqa: E731
        q, k, v, z, a, b = _cut(cut(proj), cut(gates))
        qq, kk = g.qk_prep(q, k, **PREP)
        if e - p == 1:
            o = g.delta_step(S, qq[:, 0], kk[:, 0], v[:, 0], a[:, 0], b[:, 0])[:, None]
        else:
            o, S, _ = g.delta_fwd(qq, kk, v, a, b, S0=S)
        y, _ = g.block_norm(o, weight=w, gate=z, **HEADS)
        h, n = g.block_norm(y.view(B, e - p, 1, H * D), residual=cut(res), next_weight=w2, **JOIN)
        return torch.stack([h, n]), S
    whole, S1 = layer(0, T + more, None)
    parts = []
    out, S = layer(0, T, None)
    parts.append(out)
    for t in range(T, T + more):
        out, S = layer(t, t + 1, S)
        parts.append(out)
    tol = 2 * 4 * (64 + 64 + 128) * U  # each side its own, as above
    _norm_close("outputs", to_np(torch.cat(parts, 2)), to_np(whole), tol)
    _norm_close("state", to_np(S), to_np(S1), tol)
