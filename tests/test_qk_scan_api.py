"""Host-side checks of the query / key preparation and of the gated linear recurrence:
every refusal, with nothing launched (these calls never reach the GPU)."""
import pytest
import torch

from tests.test_abi import FakePtr, _ptrs


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_84_amd as g

    return g


def _qk(g, **kw):
    base = dict(B=2, T=100, Hq=4, Hk=2, d=64, io_dtype=g.GDR_BF16, weight_dtype=g.GDR_F32, norm=g.GDR_NORM_RMS,
                rot_layout=g.GDR_ROT_HALF, rot_dim=32, eps=1e-6, q_scale=1.0, rot_scale=1.0, ldq=0, ldk=0)
    base.update(kw)
    return g.QkDesc(**base)


NAN = float("nan")


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, -1), ("T", -1, -1), ("Hq", -1, -1), ("Hk", -2, -1), ("io_dtype", 2, -1), ("weight_dtype", 9, -1),
    ("norm", 3, -1), ("norm", -1, -1), ("rot_layout", 2, -1), ("rot_dim", 3, -1), ("rot_dim", -2, -1), ("rot_dim", 66, -1),
    ("eps", -1e-6, -1), ("eps", NAN, -1), ("q_scale", NAN, -1), ("rot_scale", NAN, -1), ("ldq", 255, -1), ("ldk", -128, -1),
    ("ldq", 1 << 62, -1), ("d", 0, -1), ("d", 4, -1), ("d", 36, -2), ("d", 264, -2), ("Hq", 65537, -2), ("B", 1 << 30, -2),
])
def test_qk_descriptor(g, field, value, status):
    d = _qk(g, **{field: value})
    q, k, wq, wk, pos, f, qo, ko, dq, dk = _ptrs(n=10, step=0x10000000)
    assert g.gdr_qk_prep_fwd(d, q, k, wq, wk, pos, f, qo, ko, 0) == status
    assert g.gdr_qk_prep_bwd(d, q, k, wq, wk, pos, f, qo, ko, dq, dk, None, None, None, 0, 0) == status


def test_qk_pointers(g):
    d = _qk(g)
    q, k, wq, wk, pos, f, qo, ko = _ptrs(n=8, step=0x10000000)
    call = lambda desc=d, **a: g.gdr_qk_prep_fwd(  # noqa: E731
        desc, a.get("q", q), a.get("k", k), a.get("wq", wq), wk, a.get("pos", pos), a.get("f", f), a.get("qo", qo),
        a.get("ko", ko), 0)
    for name in ("q", "k", "f", "qo", "ko"):
        assert call(**{name: None}) == g.GDR_EINVAL
    assert call(q=FakePtr(q.addr + 1)) == g.GDR_EINVAL                      # element alignment
    assert call(pos=FakePtr(pos.addr + 2)) == g.GDR_EINVAL
    assert call(f=FakePtr(f.addr + 4)) == g.GDR_EINVAL
    assert call(qo=FakePtr(q.addr + 128)) == g.GDR_EINVAL                   # inside the input
    assert call(_qk(g, ldq=512), qo=q) == g.GDR_EINVAL                      # in place needs a dense input
    assert call(qo=k) == g.GDR_EINVAL                                       # the other tensor's input
    assert call(qo=ko) == g.GDR_EINVAL
    assert call(qo=wq) == g.GDR_EINVAL
    assert call(_qk(g, norm=g.GDR_NORM_NONE)) == g.GDR_EINVAL               # weights without a norm
    assert call(_qk(g, B=0), q=None, qo=None) == g.GDR_OK                   # nothing to do


def test_qk_backward_pointers(g):
    d = _qk(g)
    q, k, wq, wk, pos, f, gq, gk, dq, dk, dwq, dwk, ws = _ptrs(n=13, step=0x10000000)
    need = g.gdr_qk_prep_bwd_workspace_size(d)
    assert need > 0 and need % (64 * 4) == 0
    assert g.gdr_qk_prep_bwd_workspace_size(_qk(g, norm=g.GDR_NORM_NONE)) == 0
    assert g.gdr_qk_prep_bwd_workspace_size(_qk(g, d=20)) == 0
    call = lambda desc=d, **a: g.gdr_qk_prep_bwd(  # noqa: E731
        desc, q, k, a.get("wq", wq), wk, pos, f, a.get("gq", gq), gk, a.get("dq", dq), a.get("dk", dk), a.get("dwq", dwq), dwk,
        a.get("ws", ws), a.get("wb", need), 0)
    assert call(gq=None) == g.GDR_EINVAL
    assert call(dk=None) == g.GDR_EINVAL
    assert call(wq=None) == g.GDR_EINVAL                                    # its gradient without the weight
    assert call(dwq=FakePtr(dwq.addr + 2)) == g.GDR_EINVAL
    assert call(ws=None) == g.GDR_EWORKSPACE
    assert call(wb=need - 4) == g.GDR_EWORKSPACE
    assert call(ws=FakePtr(ws.addr + 8)) == g.GDR_EWORKSPACE
    assert call(dq=q) == g.GDR_EINVAL                                       # the input is read for the norm
    assert call(dq=gk) == g.GDR_EINVAL
    assert call(dq=FakePtr(gq.addr + 64)) == g.GDR_EINVAL
    assert call(ws=gq) == g.GDR_EINVAL
    assert call(dwq=dk) == g.GDR_EINVAL


def test_qk_binding(g):
    bf = torch.bfloat16
    q, k = torch.zeros(2, 5, 4, 16, dtype=bf), torch.zeros(2, 5, 2, 16, dtype=bf)
    f = torch.ones(8, dtype=torch.float64)
    with pytest.raises(ValueError, match="device tensor"):
        g.qk_prep(q, k, inv_freq=f)
    with pytest.raises(ValueError, match="positions"):                      # int64 positions
        g.qk_prep(q, k, inv_freq=f, positions=torch.zeros(2, 5, dtype=torch.int64))
    with pytest.raises(ValueError, match="inv_freq"):
        g.qk_prep(q, k, inv_freq=f.float())
    with pytest.raises(ValueError, match="wq"):
        g.qk_prep(q, k, wq=torch.zeros(8))
    with pytest.raises(ValueError, match="norm"):
        g.qk_prep(q, k, norm="l1")
    with pytest.raises(ValueError, match="layout"):
        g.qk_prep(q, k, layout="quarter")
    with pytest.raises(ValueError, match="expected q"):
        g.qk_prep(q, k[:, :4])
    with pytest.raises(ValueError, match="expected q"):
        g.qk_prep(q, k.float())
    with pytest.raises(ValueError, match="one type"):
        g.qk_prep(q, k, wq=torch.zeros(16), wk=torch.zeros(16, dtype=bf))
    with pytest.raises(TypeError):
        g.qk_prep(q.half(), k.half())
    with pytest.raises(ValueError, match="dense"):                          # heads transposed
        g.qk_prep(torch.zeros(2, 4, 5, 16, dtype=bf).transpose(1, 2), k)
    with pytest.raises(ValueError, match="evenly"):                         # a cut of the tokens of a batch
        g.qk_prep(torch.zeros(2, 7, 4, 16, dtype=bf)[:, :5], k)
    with pytest.raises(ValueError, match="evenly|overlapping"):             # one row for every sequence
        g.qk_prep(torch.zeros(1, 5, 4, 16, dtype=bf).expand(2, 5, 4, 16), k)
    with pytest.raises(ValueError, match="contiguous|device"):
        g.qk_prep_bwd(q, k, torch.zeros(2, 4, 5, 16, dtype=bf).transpose(1, 2), k)


def _scan(g, **kw):
    base = dict(B=2, T=1100, H=3, dk=1, dv=20, chunk=64, io_dtype=g.GDR_BF16, gate_dtype=g.GDR_F32,
                alpha_mode=g.GDR_ALPHA_CHANNEL, beta_mode=0, flags=0)
    base.update(kw)
    return g.Desc(**base)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, -1), ("T", -1, -1), ("H", -1, -1), ("dv", 0, -1), ("io_dtype", 5, -1), ("gate_dtype", 2, -1),
    ("alpha_mode", 2, -1), ("alpha_mode", 0, -2), ("flags", 0x10, -1), ("flags", 0x1, -1), ("H", 1 << 28, -2),
    ("T", 1 << 29, -2),
])
def test_scan_descriptor(g, field, value, status):
    d = _scan(g, **{field: value})
    x, a, S, y, ck, dx, da, ws = _ptrs(n=8, step=0x10000000)
    assert g.gdr_scan_fwd(d, x, 0, a, 0, None, 0, None, 0, None, y, None, None, ws, 1 << 40, 0) == status
    assert g.gdr_scan_bwd(d, x, 0, a, 0, None, 0, None, 0, None, ck, y, None, dx, da, None, None, ws, 1 << 40, 0) == status
    assert g.gdr_scan_workspace_size(d) == 0
    if field != "T":
        assert g.gdr_scan_step(d, x, 0, a, 0, None, 0, S, y, 0) == status


@pytest.mark.parametrize("B,T,dv", [(1 << 26, 1, 1), (1 << 26, 15, 4), (1 << 27, 7, 2), (1 << 28, 3, 1), (1, (1 << 30) - 1, 65),
                                    (3, (1 << 28) + 1, 64 * 9)])
def test_scan_launches_that_are_too_large(g, B, T, dv):
    """A launch has fewer than 2^32 threads: refused before any."""
    x, a, y, ck, dx, da, ws = _ptrs(n=7, step=1 << 50)
    d = _scan(g, B=B, T=T, H=1, dv=dv)
    wb = g.gdr_scan_workspace_size(d)
    assert g.gdr_scan_fwd(d, x, 0, a, 0, None, 0, None, 0, None, y, None, None, ws, wb, 0) == g.GDR_EUNSUPPORTED
    assert g.gdr_scan_bwd(d, x, 0, a, 0, None, 0, None, 0, None, ck, y, None, dx, da, None, None, ws, wb, 0) == g.GDR_EUNSUPPORTED


def test_scan_pointers(g):
    d = _scan(g)
    x, a, b, off, S0, y, ST, ck, ws = _ptrs(n=9, step=0x10000000)
    need = g.gdr_scan_workspace_size(d)
    call = lambda desc=d, **v: g.gdr_scan_fwd(  # noqa: E731
        desc, v.get("x", x), v.get("ldx", 0), v.get("a", a), v.get("lda", 0), v.get("b", b), v.get("ldb", 0),
        v.get("off", None), v.get("n", 0), v.get("S0", S0), v.get("y", y), v.get("ST", ST), v.get("ck", ck),
        v.get("ws", ws), v.get("wb", need), 0)
    for name in ("x", "a", "y"):
        assert call(**{name: None}) == g.GDR_EINVAL
    assert call(_scan(g, flags=g.GDR_FLAG_COUPLED)) == g.GDR_EINVAL          # coupled leaves no room for beta
    assert call(ldx=59) == g.GDR_EINVAL
    assert call(lda=-60) == g.GDR_EINVAL
    assert call(ldb=1 << 60) == g.GDR_EINVAL
    assert call(ldx=(1 << 20) + 1) == g.GDR_EUNSUPPORTED
    assert call(x=FakePtr(x.addr + 1)) == g.GDR_EINVAL
    assert call(a=FakePtr(a.addr + 2)) == g.GDR_EINVAL                       # fp32 gates
    assert call(ST=FakePtr(ST.addr + 2)) == g.GDR_EINVAL
    assert call(n=1) == g.GDR_EINVAL                                         # a count without offsets
    assert call(off=off, n=1) == g.GDR_EINVAL                                # packed rows are a batch of one
    one = _scan(g, B=1)
    assert call(one, off=off, n=-1) == g.GDR_EINVAL
    assert call(one, off=FakePtr(off.addr + 2), n=1) == g.GDR_EINVAL
    assert call(one, off=off, n=2, ST=S0) == g.GDR_EINVAL                    # no in-place resume when packed
    assert call(one, off=off, n=2, y=FakePtr(off.addr - 64)) == g.GDR_EINVAL
    assert call(y=x) == g.GDR_EINVAL
    assert call(ST=FakePtr(S0.addr + 4)) == g.GDR_EINVAL
    assert call(ck=FakePtr(y.addr + 64)) == g.GDR_EINVAL
    assert call(x=x, ldx=1000, ST=FakePtr(x.addr + 2 * 2199 * 1000 + 100)) == g.GDR_EINVAL  # the strided extent's end
    if need:
        assert call(ws=None) == g.GDR_EWORKSPACE
        assert call(wb=need - 1) == g.GDR_EWORKSPACE
        assert call(ws=FakePtr(ws.addr + 4)) == g.GDR_EWORKSPACE
        assert call(ws=y) == g.GDR_EINVAL
    assert call(_scan(g, B=0), x=None, a=None, y=None) == g.GDR_OK
    assert call(_scan(g, H=0), x=None, a=None, b=None, y=None) == g.GDR_OK


def test_scan_backward_pointers(g):
    d = _scan(g)
    x, a, b, S0, ck, dy, dST, dx, da, db, dS0, ws = _ptrs(n=12, step=0x10000000)
    need = g.gdr_scan_workspace_size(d)
    call = lambda desc=d, **v: g.gdr_scan_bwd(  # noqa: E731
        desc, x, 0, a, 0, v.get("b", b), 0, v.get("off", None), v.get("n", 0), S0, v.get("ck", ck), v.get("dy", dy), dST,
        v.get("dx", dx), v.get("da", da), v.get("db", db), v.get("dS0", dS0), ws, need, 0)
    for name in ("ck", "dy", "dx", "da", "db", "b"):                         # db without b and b without db
        assert call(**{name: None}) == g.GDR_EINVAL
    assert call(dx=dy) == g.GDR_EINVAL
    assert call(da=a) == g.GDR_EINVAL
    assert call(dS0=dST) == g.GDR_EINVAL
    assert call(dS0=ck) == g.GDR_EINVAL
    assert call(db=da) == g.GDR_EINVAL
    assert call(da=FakePtr(da.addr + 2)) == g.GDR_EINVAL


def test_scan_step_pointers(g):
    d = _scan(g, T=-5)                                                       # the step does not look at T
    x, a, S, y = _ptrs(n=4, step=0x10000000)
    call = lambda desc=d, **v: g.gdr_scan_step(desc, v.get("x", x), v.get("ldx", 0), v.get("a", a), 0, None, 0,  # noqa: E731
                                              v.get("S", S), v.get("y", y), 0)
    for name in ("x", "a", "S", "y"):
        assert call(**{name: None}) == g.GDR_EINVAL
    assert call(y=S) == g.GDR_EINVAL
    assert call(y=x) == g.GDR_EINVAL
    assert call(S=FakePtr(S.addr + 2)) == g.GDR_EINVAL
    assert call(ldx=59) == g.GDR_EINVAL
    assert call(_scan(g, B=0), x=None) == g.GDR_OK
    assert g._lib.gdr_scan_step(None, None, 0, None, 0, None, 0, None, None, None) == g.GDR_EINVAL


def test_scan_step_strides(g):
    """A stride over 2^20 elements is no reason to refuse; here the NULL output is, or what cannot be addressed."""
    d = _scan(g)
    x, a, S, y = _ptrs(n=4, step=0x10000000)
    for ld in ((1 << 20) + 1, 1 << 40):
        assert g.gdr_scan_step(d, x, ld, a, 0, None, 0, S, None, 0) == g.GDR_EINVAL
        assert g.gdr_scan_step(d, x, 0, a, ld, None, 0, S, None, 0) == g.GDR_EINVAL
        assert g.gdr_scan_step(d, x, 0, a, 0, a, ld, S, None, 0) == g.GDR_EINVAL
    assert g.gdr_scan_step(d, x, 1 << 60, a, 0, None, 0, S, y, 0) == g.GDR_EINVAL


def test_scan_binding(g):
    bf = torch.bfloat16
    x, a = torch.zeros(1, 6, 2, 8, dtype=bf), torch.zeros(1, 6, 2, 8)
    S = torch.zeros(1, 2, 8)
    with pytest.raises(ValueError, match="device tensor"):
        g.scan_fwd(x, a)
    with pytest.raises(ValueError, match="beta"):
        g.scan_fwd(x, a, beta=torch.zeros(1, 6, 2, 8, dtype=bf))             # gates of two types
    with pytest.raises(ValueError, match="expected x and alpha"):
        g.scan_fwd(x, torch.zeros(1, 6, 2))                                  # one gate per head
    with pytest.raises(ValueError, match="seq_off"):
        g.scan_fwd(x, a, seq_offsets=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="S0"):
        g.scan_fwd(x, a, seq_offsets=torch.zeros(3, dtype=torch.int32), S0=S)  # two sequences, one state
    with pytest.raises(ValueError, match="dy"):
        g.scan_bwd(x, a, a, None)
    with pytest.raises(ValueError, match="ckpt"):
        g.scan_bwd(x, a, x, torch.zeros(1, 2, 2, 8))
    with pytest.raises(ValueError, match="evenly"):
        g.scan_fwd(torch.zeros(2, 9, 2, 8, dtype=bf)[:, :6], torch.zeros(2, 6, 2, 8))
    with pytest.raises(ValueError, match="S: expected dtype"):
        g.scan_step(S.to(bf), x[:, 0], a[:, 0])
    with pytest.raises(ValueError, match="expected x and alpha"):
        g.scan_step(S, x, a)
