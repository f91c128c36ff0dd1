"""Query / key preparation against its fp64 reference.

Tolerances (u = 2^-24, one fp32 rounding; step = half a step of the stored type).  The sum of
squares of d <= 256 channels is at most 2 VP + log2 P <= 13 additions deep, so r is within
about 10 u; cosine and sine are within 4 u of an angle reduced in 64 bits; each member of a
rotated pair adds the errors of 5 products and a sum.  40 u of the row's largest normalised
value, rotated (a factor sqrt 2), covers it; the backward pass has twice the chain, and a sum
over the row.  A weight gradient's sum runs over at most 8 rows per item and item loop, 6
steps over a wave, 4 waves, and up to 768 / 64 + 6 sums of workgroups."""
import numpy as np
import pytest

from oracle import qk_prep as ref
from tests.gpu_util import gpu, log, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
STEP = {"bf16": 2.0 ** -8, "f32": U}


def _case(torch, seed, B, T, Hq, Hk, d, io, wt, norm, rot, layout, far, fused):
    gen = torch.Generator().manual_seed(seed)
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    if fused:
        x = torch.randn(B, T, (Hq + 2 * Hk) * d + 3, generator=gen).to(t[io]).cuda()
        q = x[..., :Hq * d].unflatten(-1, (Hq, d))
        k = x[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    else:
        q, k = (torch.randn(B, T, h, d, generator=gen).to(t[io]).cuda() for h in (Hq, Hk))
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=gen)).to(t[wt]).cuda() if wt and norm != "none" else None for _ in range(2))
    pos = torch.randint(-5, far, (B, T), generator=gen, dtype=torch.int32).cuda() if far else None
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda() if rot else None
    gq, gk = (torch.randn(B, T, h, d, generator=gen).to(t[io]).cuda() for h in (Hq, Hk))
    return q, k, gq, gk, dict(norm=norm, wq=wq, wk=wk, eps=1e-5, positions=pos, inv_freq=f, layout=layout, rot_scale=1.25,
                              q_scale=0.125)


def _check(name, got, want, step, err):
    got = to_np(got)
    assert got.shape == want.shape
    bound = step * np.abs(want) + err
    worst = float(np.max(np.abs(got - want) / np.maximum(bound, 1e-300))) if got.size else 0.0
    log(f"[qk_prep] {name}: error / bound {worst:.3f}")
    assert worst <= 1.0, name


CASES = [
    # B, T, Hq, Hk, d, io, weight, norm, rot, layout, far, fused
    (1, 1, 1, 1, 8, "bf16", "f32", "rms", 8, "half", 100, False),
    (1, 1, 16, 16, 128, "bf16", "bf16", "rms", 128, "half", 100000, True),
    (3, 5, 6, 2, 64, "bf16", "f32", "l2", 64, "interleaved", 0, True),
    (2, 33, 4, 4, 128, "bf16", None, "l2", 0, "half", 0, False),
    (2, 17, 3, 1, 96, "f32", "f32", "rms", 24, "half", 1 << 20, True),
    (1, 40, 9, 3, 80, "f32", "bf16", "rms", 40, "interleaved", 1000, False),
    (1, 19, 5, 7, 256, "bf16", "f32", "rms", 256, "half", 1 << 20, False),
    (1, 21, 2, 2, 256, "f32", "f32", "l2", 130, "half", 50, True),      # pairs at unaligned places
    (2, 9, 17, 1, 40, "bf16", "f32", "rms", 10, "half", 50, True),      # five pairs
    (1, 13, 1, 1, 72, "bf16", "f32", "none", 72, "half", 50, False),
    (2, 8, 2, 2, 24, "f32", None, "none", 6, "interleaved", 50, True),
    (1, 7, 3, 0, 64, "bf16", "f32", "rms", 32, "half", 50, False),      # queries alone
    (1, 2000, 10, 2, 16, "bf16", "f32", "rms", 16, "interleaved", 0, True),
    (1, 1700, 16, 2, 128, "bf16", "f32", "rms", 64, "half", 5000, True),   # workgroups that come round again
    (2, 450, 9, 3, 256, "f32", "bf16", "l2", 256, "interleaved", 0, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_backward(case):
    torch, g = gpu()
    B, T, Hq, Hk, d, io, wt, norm, rot, layout, far, fused = case
    log(f"[qk_prep] {case}")
    q, k, gq, gk, how = _case(torch, 11, *case)
    outs = g.qk_prep(q, k, **how)
    grads = g.qk_prep_bwd(q, k, gq, gk, **how)
    torch.cuda.synchronize()
    pos = None if how["positions"] is None else how["positions"].cpu().numpy()
    f = None if how["inv_freq"] is None else how["inv_freq"].cpu().numpy()
    for i, (x, go, w, scale) in enumerate(((q, gq, how["wq"], 0.125), (k, gk, how["wk"], 1.0))):
        if x.numel() == 0:
            continue
        x64, g64, w64 = to_np(x), to_np(go), None if w is None else to_np(w)
        kw = dict(norm=norm, eps=float(np.float32(1e-5)), pos=pos, inv_freq=f, layout=layout, rot_scale=1.25, scale=scale)
        want = ref.forward(x64, w64, **kw)
        flat = ref.forward(x64, w64, norm=norm, eps=kw["eps"], scale=scale)
        top = 1.25 * 1.5 * np.abs(flat).max(-1, keepdims=True)
        _check("qk"[i], outs[i], want, STEP[io], 40 * U * top)
        dx, dw = ref.backward(x64, g64, w64, **kw)
        r = ref._r(x64, norm, kw["eps"])
        t = 1.25 * 1.5 * scale * np.abs(g64).max(-1, keepdims=True) * (1.0 if w64 is None else np.abs(w64).max())
        hat = np.abs(r * x64)
        kappa = {"none": 0.0, "l2": 1.0, "rms": 1.0 / d}[norm]
        _check("d" + "qk"[i], grads[i], dx, STEP[io], 80 * U * r * (t + kappa * hat * (t * hat).sum(-1, keepdims=True)))
        if w is None:
            assert grads[2 + i] is None
        else:
            terms = (t / np.abs(w64).max() * hat).sum((0, 1, 2))
            _check("dw" + "qk"[i], grads[2 + i], dw, U, (60 + 140) * U * terms)


def test_zero_rows_and_special_values():
    """A row of zeros gives zeros and zero gradients with eps = 0; NaN and infinities stay in their row."""
    torch, g = gpu()
    q = torch.randn(1, 6, 2, 64, dtype=torch.float32, device="cuda")
    q[0, 1, 0] = 0
    q[0, 2, 1, 5] = float("nan")
    q[0, 3, 0, 7] = float("inf")
    clean = q.clone()
    clean[0, 2, 1], clean[0, 3, 0] = 1, 1
    f, _ = g.rope_inv_freq(32)
    for norm in ("l2", "rms"):
        how = dict(norm=norm, eps=0.0, inv_freq=f)
        out, _ = g.qk_prep(q, q.clone(), **how)
        want, _ = g.qk_prep(clean, clean.clone(), **how)
        go = torch.randn_like(q)
        dq = g.qk_prep_bwd(q, q.clone(), go, go, **how)[0]
        assert not out[0, 1, 0].any() and not dq[0, 1, 0].any()
        assert out[0, 2, 1].isnan().all() and out[0, 3, 0, 7].isnan()
        rows = torch.ones(1, 6, 2, dtype=torch.bool, device="cuda")
        rows[0, 2, 1] = rows[0, 3, 0] = False
        assert torch.equal(out[rows], want[rows]) and dq[rows].isfinite().all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [0, 12, 64])
def test_backward_without_a_norm_does_not_look_at_the_inputs(layout, rot):
    """dx = scale Rot^T(g) whatever x holds: infinities, NaN, and rows whose sum of squares passes fp32's range."""
    torch, g = gpu()
    q, k, gq, gk, how = _case(torch, 12, 2, 37, 3, 2, 64, "f32", None, "none", rot, layout, 5000, True)
    want = g.qk_prep_bwd(q, k, gq, gk, **how)
    q, k = torch.randn_like(q) * 3e38, k.clone()
    q[0, 1, 0], q[0, 2, 1, 5], k[1, 3] = float("nan"), float("inf"), float("-inf")
    got = g.qk_prep_bwd(q, k, gq, gk, **how)
    assert all(torch.equal(a, b) for a, b in zip(got[:2], want[:2])) and got[2] is None and got[3] is None
    f = None if how["inv_freq"] is None else how["inv_freq"].cpu().numpy()
    pos = how["positions"].cpu().numpy()
    for i, (x, go, scale) in enumerate(((q, gq, 0.125), (k, gk, 1.0))):
        g64 = to_np(go)
        dx, _ = ref.backward(np.zeros_like(g64), g64, norm="none", pos=pos, inv_freq=f, layout=layout, rot_scale=1.25, scale=scale)
        _check("d" + "qk"[i], got[i], dx, U, 40 * U * 1.25 * 1.5 * scale * np.abs(g64).max(-1, keepdims=True))
    # each gradient written over, as with a norm
    desc = g._qk_desc(q, k, "none", None, None, 1e-5, how["inv_freq"], layout, 1.25, 0.125)
    oq, ok = gq.clone(), gk.clone()
    assert g.gdr_qk_prep_bwd(desc, q, k, None, None, how["positions"], how["inv_freq"], oq, ok, oq, ok, None, None, None, 0) == g.GDR_OK
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])


def test_in_place_and_empty():
    torch, g = gpu()
    q, k = (torch.randn(2, 70, h, 128, device="cuda").bfloat16() for h in (4, 2))
    f, _ = g.rope_inv_freq(64)
    w = torch.rand(128, device="cuda")
    want = g.qk_prep(q, k, wq=w, inv_freq=f)
    q2, k2 = q.clone(), k.clone()
    got = g.qk_prep(q2, k2, wq=w, inv_freq=f, out=(q2, k2))
    assert got[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    dq, dk, dwq, dwk = g.qk_prep_bwd(q, k, gq, gk, wq=w, inv_freq=f)
    assert dwk is None
    desc = g._qk_desc(q, k, "rms", w, None, 1e-6, f, "half", 1.0, 1.0)
    need = g.gdr_qk_prep_bwd_workspace_size(desc)
    ws, dw = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty_like(w)
    assert g.gdr_qk_prep_bwd(desc, q, k, w, None, None, f, gq, gk, gq, gk, dw, None, ws, need) == g.GDR_OK
    assert torch.equal(gq, dq) and torch.equal(gk, dk) and torch.equal(dw, dwq)
    # no tokens: nothing to write but the weights' gradients
    e = torch.empty(0, 5, 4, 128, device="cuda")
    out = g.qk_prep_bwd(e, e, e, e, wq=w, wk=w)
    assert out[0].shape == e.shape and not out[2].any() and not out[3].any()
    # queries alone: the absent keys' weight gets a gradient of zero
    none = torch.empty(2, 70, 0, 128, device="cuda", dtype=torch.bfloat16)
    assert not g.qk_prep_bwd(q, none, torch.randn_like(q), none, wq=w, wk=w)[3].any()


def test_deterministic_and_captured():
    """Twice the same bits, and a captured forward and backward replay equal to the eager calls,
    with other work on the workspace's stream between the replays."""
    torch, g = gpu()
    q, k = (torch.randn(2, 700, h, 64, device="cuda") for h in (8, 2))
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    how = dict(wq=torch.rand(64, device="cuda"), wk=torch.rand(64, device="cuda"), inv_freq=g.rope_inv_freq(64)[0])
    step = lambda: g.qk_prep(q, k, **how) + g.qk_prep_bwd(q, k, gq, gk, **how)  # noqa: E731
    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in range(3):
        q.copy_(torch.randn_like(q))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed


def test_many_tokens_split_like_few():
    """Rows of a long batch equal the rows of short calls, bit for bit: the split of the work does not enter."""
    torch, g = gpu()
    x = torch.randn(1, 40000, 3 * 4 * 128, device="cuda").bfloat16()
    q, k = x[..., :512].unflatten(-1, (4, 128)), x[..., 512:1024].unflatten(-1, (4, 128))
    pos = torch.randint(0, 1 << 20, (1, 40000), dtype=torch.int32, device="cuda")
    how = dict(wq=torch.rand(128, device="cuda"), inv_freq=g.rope_inv_freq(128)[0])
    a = g.qk_prep(q, k, positions=pos, **how)
    for t in (0, 1, 12345, 39998):
        b = g.qk_prep(q[:, t:t + 2], k[:, t:t + 2], positions=pos[:, t:t + 2].contiguous(), **how)
        assert torch.equal(a[0][:, t:t + 2], b[0]) and torch.equal(a[1][:, t:t + 2], b[1])


def test_more_rows_than_a_launch_has_groups_for():
    """2^27 + 77 tokens of one head of 256, in place (69 GB): the workgroups come round again, and every row is done once."""
    torch, g = gpu()
    n, T = 131071, (1 << 27) + 77
    base = torch.randn(1, n, 1, 256, device="cuda").bfloat16()
    none = torch.empty(1, n, 0, 256, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(256, device="cuda")
    want, _ = g.qk_prep(base, none, norm="l2", wq=w)
    q, k = torch.empty(1, T, 1, 256, device="cuda", dtype=torch.bfloat16), none.new_empty(1, T, 0, 256)
    for t in range(0, T, n):
        q[:, t:t + n] = base[:, :T - t]
    log(f"[qk_prep] {T} tokens")
    g.qk_prep(q, k, norm="l2", wq=w, out=(q, k))
    assert all(torch.equal(q[:, t:t + n], want[:, :T - t]) for t in range(0, T, n))
