"""The preparation, the delta rule and the gated recurrence run together, as a stack of two
token-mixing layers does: one fused projection's output -> qk_prep -> chunk_fwd -> scan_fwd,
then token by token through qk_prep, decode_step and scan_step; and the recurrence's
gradient handed back through the preparation."""
import numpy as np
import pytest

import oracle
from oracle import qk_prep as qk_ref
from oracle import scan as scan_ref
from tests.gpu_util import gpu, log, to_np

pytestmark = pytest.mark.gpu


def _inputs(torch, B, T, H, d):
    gen = torch.Generator().manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return (r(B, T, 3, H, d).bfloat16().cuda(), torch.sigmoid(r(B, T, H) + 4).cuda(), torch.sigmoid(r(B, T, H)).cuda(),
            (-torch.nn.functional.softplus(r(B, T, H, d) - 4)).cuda())


def test_prefill_then_decode():
    torch, g = gpu()
    B, T, H, d, more = 2, 600, 3, 128, 5
    qkv, alpha, beta, gate = _inputs(torch, B, T + more, H, d)
    f, scale = g.rope_inv_freq(64, scaling="yarn", factor=4, original_len=256)
    how = dict(norm="l2", eps=1e-6, inv_freq=f, rot_scale=scale, q_scale=d ** -0.5)
    cut = lambda t, p, q: t[:, p:q].contiguous()  # noqa: E731

    def layers(p, q, S, h):
        x = cut(qkv, p, q)
        pos = torch.arange(p, q, dtype=torch.int32, device="cuda").expand(B, q - p).contiguous()
        qq, kk = g.qk_prep(x[:, :, 0], x[:, :, 1], positions=pos, **how)
        v = x[:, :, 2].contiguous()
        if q - p == 1:
            o = g.decode_step(S, qq[:, 0], kk[:, 0], v[:, 0], alpha[:, p].contiguous(), beta[:, p].contiguous())
            return g.scan_step(h, o, gate[:, p].contiguous(), log_gate=True, coupled=True)[:, None], o[:, None], S, h
        o, S = g.chunk_fwd(qq, kk, v, cut(alpha, p, q), cut(beta, p, q), S0=S)
        y, h, _ = g.scan_fwd(o, cut(gate, p, q), log_gate=True, coupled=True, S0=h)
        return y, o, S, h

    y, o, S, h = layers(0, T, None, None)
    ys, os_ = [y], [o]
    for t in range(T, T + more):
        y, o, S, h = layers(t, t + 1, S, h)
        ys.append(y)
        os_.append(o)
    torch.cuda.synchronize()
    y, o = torch.cat(ys, 1), torch.cat(os_, 1)
    # the fp64 references, chained; the delta rule's inputs are bf16 heads
    x64 = to_np(qkv)
    f64 = f.cpu().numpy()
    kw = dict(norm="l2", eps=1e-6, inv_freq=f64, rot_scale=scale)
    heads = [torch.from_numpy(qk_ref.forward(x64[:, :, i], scale=s, **kw)).bfloat16().double().numpy()
             for i, s in ((0, d ** -0.5), (1, 1.0))]
    o_ref, S_ref = oracle.forward(heads[0], heads[1], x64[:, :, 2], to_np(alpha), to_np(beta))
    h_all, h_ref = scan_ref.forward(o_ref.reshape(B, T + more, -1), to_np(gate).reshape(B, T + more, -1), log=True, coupled=True)
    # heads rounded on either side of a tie, an output stored in bf16 (2e-3 for the delta rule alone), and a mean of it
    eo, ey = oracle.rel_l2(to_np(o), o_ref), oracle.rel_l2(to_np(y).reshape(h_all.shape), h_all)
    es, eh = oracle.rel_l2(to_np(S), S_ref), oracle.rel_l2(to_np(h).reshape(h_ref.shape), h_ref)
    log(f"[stack] rel-L2 o={eo:.2e} y={ey:.2e} S={es:.2e} h={eh:.2e}")
    assert max(eo, ey) <= 3e-3 and max(es, eh) <= 2e-3


def test_gradients_through_both():
    """Keys prepared and then smoothed over time: the recurrence's dx is the preparation's output gradient."""
    torch, g = gpu()
    B, T, H, d = 1, 700, 2, 64
    qkv, _, _, gate = _inputs(torch, B, T, H, d)
    qkv = qkv.float()
    f, _ = g.rope_inv_freq(d)
    w = 1 + 0.2 * torch.randn(d, device="cuda")
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    dy = torch.randn(B, T, H, d, device="cuda")
    how = dict(wq=w, wk=w, inv_freq=f, eps=1e-6)
    qq, kk = g.qk_prep(q, k, **how)
    _, _, ck = g.scan_fwd(kk, gate, log_gate=True, coupled=True, want_ckpt=True)
    dk_out, dgate, _, _ = g.scan_bwd(kk, gate, dy, ck, log_gate=True, coupled=True)
    _, dk, _, dw = g.qk_prep_bwd(q, k, torch.zeros_like(qq), dk_out, **how)
    torch.cuda.synchronize()
    k64, w64, kw = to_np(k), to_np(w), dict(norm="rms", eps=1e-6, inv_freq=f.cpu().numpy())
    flat = lambda a: a.reshape(B, T, H * d)  # noqa: E731
    kk64 = qk_ref.forward(k64, w64, **kw)
    dx, da, _, _ = scan_ref.backward(flat(kk64), flat(to_np(gate)), flat(to_np(dy)), log=True, coupled=True)
    dk64, dw64 = qk_ref.backward(k64, dx.reshape(kk64.shape), w64, **kw)
    for name, a, b in (("dgate", flat(to_np(dgate)), da), ("dk", to_np(dk), dk64), ("dw", to_np(dw), dw64)):
        e = oracle.rel_l2(a, b)
        log(f"[stack] {name} rel-L2 {e:.2e}")
        assert e <= 1e-5
