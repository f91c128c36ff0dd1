"""Host-side checks of the trainable delta rule and of the block norm: every refusal, with nothing launched (these
calls never reach the GPU), and the chunks that packed sequences are cut into, whatever their offsets are."""
import os
import subprocess

import numpy as np
import pytest
import torch

from tests.test_abi import FakePtr, _ptrs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang++"
NAN = float("nan")


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_84_amd as g

    return g


def _delta(g, **kw):
    base = dict(B=2, T=100, Hk=2, Hv=4, dk=64, dv=48, io_dtype=g.GDR_BF16, gate_dtype=g.GDR_F32, ldq=0, ldk=0, ldv=0, ldg=0,
                ldb=0)
    base.update(kw)
    return g.DeltaDesc(**base)


FAR = 0x10000000


def _fwd(g, d, n=0, need=1 << 40, **a):
    q, k, v, gate, beta, S0, o, ST, ck, ws = _ptrs(n=10, step=FAR)
    have = dict(q=q, k=k, v=v, gate=gate, beta=beta, off=None, S0=S0, o=o, ST=ST, ck=ck, ws=ws)
    have.update(a)
    return g.gdr_delta_fwd(d, have["q"], have["k"], have["v"], have["gate"], have["beta"], have["off"], n, have["S0"], have["o"],
                           have["ST"], have["ck"], have["ws"], need, 0)


def _bwd(g, d, n=0, need=1 << 40, **a):
    names = "q k v gate beta ck do dST dq dk dv dg db dS0 ws".split()
    have = dict(zip(names, _ptrs(n=len(names), step=FAR)), off=None)
    have.update(a)
    return g.gdr_delta_bwd(d, *(have[x] for x in "q k v gate beta off".split()), n,
                           *(have[x] for x in "ck do dST dq dk dv dg db dS0 ws".split()), need, 0)


def _step(g, d, **a):
    names = "q k v gate beta S o".split()
    have = dict(zip(names, _ptrs(n=7, step=FAR)))
    have.update(a)
    return g.gdr_delta_step(d, *(have[x] for x in names), 0)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, -1), ("T", -1, -1), ("Hk", -1, -1), ("Hv", -4, -1), ("Hv", 3, -1), ("Hk", 0, -1), ("io_dtype", 2, -1),
    ("gate_dtype", -1, -1), ("dk", 0, -2), ("dk", 12, -2), ("dk", 136, -2), ("dv", 4, -2), ("dv", 256, -2), ("dv", -8, -2),
    ("ldq", 127, -1), ("ldk", -128, -1), ("ldv", 191, -1), ("ldg", 3, -1), ("ldb", 1, -1), ("ldq", 1 << 62, -1),
    ("Hv", 65538, -2), ("B", 1 << 30, -2), ("ldq", (1 << 20) + 1, -2), ("ldv", 1 << 30, -2), ("ldg", (1 << 20) + 1, -2),
    ("B", 1 << 23, -2),
])
def test_delta_descriptor(g, field, value, status):
    d = _delta(g, **{field: value})
    assert _fwd(g, d) == status
    assert _bwd(g, d) == status
    assert g.gdr_delta_workspace_size(d) == 0
    assert g.gdr_delta_ckpt_size(d) == 0
    if field not in ("T", "ldq", "ldv", "ldg", "B") or status == -1 and field != "T":
        assert _step(g, d) == status


def test_delta_heads_of_a_row(g):
    assert _fwd(g, _delta(g, Hk=16384, Hv=16384, dk=128)) == g.GDR_EUNSUPPORTED       # 2^21 elements
    assert _step(g, _delta(g, Hk=1, Hv=65536, dv=128)) == g.GDR_EUNSUPPORTED


@pytest.mark.parametrize("name,shift", [("q", 1), ("k", 1), ("v", 1), ("gate", 2), ("beta", 1), ("S0", 4), ("o", 1), ("ST", 8), ("ck", 4)])
def test_delta_forward_pointers(g, name, shift):
    d = _delta(g)
    at = dict(zip("q k v gate beta S0 o ST ck".split(), _ptrs(n=9, step=FAR)))
    assert _fwd(g, d, **{name: FakePtr(at[name].addr + shift)}) == g.GDR_EINVAL
    if name not in ("S0", "ST", "ck"):
        assert _fwd(g, d, **{name: None}) == g.GDR_EINVAL


def test_delta_forward_sequences_and_overlaps(g):
    d, one = _delta(g), _delta(g, B=1)
    off = FakePtr(0x7000000)
    assert _fwd(g, d, off=off, n=2) == g.GDR_EINVAL                     # packed rows are one batch row
    assert _fwd(g, d, n=1) == g.GDR_EINVAL                              # sequences without offsets
    assert _fwd(g, one, off=off, n=-1) == g.GDR_EINVAL
    assert _fwd(g, one, off=FakePtr(off.addr + 2), n=2) == g.GDR_EINVAL
    q, k, v, gate, beta, S0, o, ST, ck, ws = _ptrs(n=10, step=FAR)
    for inside in (q, k, v, gate, beta, S0):
        assert _fwd(g, d, o=FakePtr(inside.addr + 16)) == g.GDR_EINVAL
        assert _fwd(g, d, ck=FakePtr(inside.addr + 16)) == g.GDR_EINVAL
    assert _fwd(g, d, o=ST) == g.GDR_EINVAL
    assert _fwd(g, d, ws=o) == g.GDR_EINVAL
    assert _fwd(g, d, ST=FakePtr(S0.addr + 16)) == g.GDR_EINVAL
    assert _fwd(g, one, off=off, n=2, ST=S0) == g.GDR_EINVAL            # in place is for dense batches
    assert _fwd(g, one, off=off, n=2, o=off) == g.GDR_EINVAL
    need = g.gdr_delta_workspace_size(d)
    assert need > 0
    assert _fwd(g, d, need=need - 1) == g.GDR_EWORKSPACE
    assert _fwd(g, d, ws=None) == g.GDR_EWORKSPACE
    assert _fwd(g, d, ws=FakePtr(ws.addr + 8)) == g.GDR_EWORKSPACE
    assert _fwd(g, _delta(g, B=0), q=None, o=None, ws=None, ck=None) == g.GDR_OK      # nothing to do
    assert _fwd(g, _delta(g, Hk=0, Hv=0), q=None, o=None, ws=None) == g.GDR_OK
    assert _fwd(g, one, off=off, n=0, q=None, ws=None) == g.GDR_OK


def test_delta_sizes(g):
    """Chunks B ceil(T / 64), or floor(T / 64) + n packed; state and written tokens as 1 KiB tiles."""
    d = _delta(g, B=1, T=130)
    assert g.gdr_delta_ckpt_size(d) == 3 * 4 * 3 * (4 + 4) * 1024
    assert g.gdr_delta_ckpt_size(d, 5) == (2 + 5) * 4 * 3 * (4 + 4) * 1024
    assert g.gdr_delta_ckpt_size(_delta(g, T=0)) == 0
    assert g.gdr_delta_workspace_size(_delta(g, T=0)) == 0
    assert g.gdr_delta_workspace_size(d, 5, True) > g.gdr_delta_workspace_size(d, 5)
    assert g.gdr_delta_workspace_size(d, -1) == 0
    assert g.gdr_delta_workspace_size(_delta(g), 2) == 0                # packed with two batch rows


@pytest.mark.parametrize("name,shift", [("q", 1), ("beta", 2), ("ck", 4), ("do", 1), ("dST", 8), ("dq", 1), ("dk", 1), ("dv", 1),
                                        ("dg", 2), ("db", 1), ("dS0", 4)])
def test_delta_backward_pointers(g, name, shift):
    d = _delta(g)
    names = "q k v gate beta ck do dST dq dk dv dg db dS0 ws".split()
    at = dict(zip(names, _ptrs(n=len(names), step=FAR)))
    assert _bwd(g, d, **{name: FakePtr(at[name].addr + shift)}) == g.GDR_EINVAL
    if name not in ("dST", "dS0"):
        assert _bwd(g, d, **{name: None}) == g.GDR_EINVAL
    if name.startswith("d") and name not in ("do", "dST"):
        for other in "q v ck do dST".split():
            assert _bwd(g, d, **{name: at[other]}) == g.GDR_EINVAL
        assert _bwd(g, d, **{name: at["ws"]}) == g.GDR_EINVAL


def test_delta_backward_workspace(g):
    d = _delta(g)
    need = g.gdr_delta_workspace_size(d, 0, True)
    assert _bwd(g, d, need=need - 1) == g.GDR_EWORKSPACE
    assert _bwd(g, d, ws=None) == g.GDR_EWORKSPACE
    assert _bwd(g, _delta(g, B=0), q=None, ck=None, ws=None, dq=None) == g.GDR_OK
    assert _bwd(g, d, n=3) == g.GDR_EINVAL


def test_delta_step_pointers(g):
    d = _delta(g, T=0)                                                  # T does not matter
    q, k, v, gate, beta, S, o = _ptrs(n=7, step=FAR)
    for name in "q k v gate beta S o".split():
        assert _step(g, d, **{name: None}) == g.GDR_EINVAL
    assert _step(g, d, S=FakePtr(S.addr + 4)) == g.GDR_EINVAL
    assert _step(g, d, o=v) == g.GDR_EINVAL
    assert _step(g, d, S=FakePtr(q.addr + 16)) == g.GDR_EINVAL
    assert _step(g, d, o=S) == g.GDR_EINVAL
    assert g.gdr_delta_step(None or _delta(g, B=0), None, None, None, None, None, None, None, 0) == g.GDR_OK


def test_null_descriptors(g):
    """A C caller's NULL descriptor."""
    import ctypes
    null = ctypes.POINTER(g.DeltaDesc)()
    lib = ctypes.CDLL(g.LIB_PATH)
    z = [None] * 20
    assert lib.gdr_delta_step(null, *z[:8]) == g.GDR_EINVAL
    assert lib.gdr_delta_fwd(null, *z[:6], 0, *z[:6]) == g.GDR_EINVAL
    assert lib.gdr_delta_bwd(null, *z[:6], 0, *z[:13]) == g.GDR_EINVAL
    assert lib.gdr_delta_workspace_size(null, 0, 0) == 0
    assert lib.gdr_block_norm_fwd(null, *z[:8]) == g.GDR_EINVAL
    assert lib.gdr_block_norm_bwd(null, *z[:15]) == g.GDR_EINVAL
    assert lib.gdr_block_norm_bwd_workspace_size(null) == 0


def test_delta_binding(g):
    bf = torch.bfloat16
    q, v = torch.zeros(2, 5, 2, 16, dtype=bf), torch.zeros(2, 5, 4, 24, dtype=bf)
    a = torch.zeros(2, 5, 4)
    with pytest.raises(ValueError, match="device tensor"):
        g.delta_fwd(q, q, v, a, a)
    with pytest.raises(ValueError, match="expected q, k"):
        g.delta_fwd(q, q[:, :4], v, a, a)
    with pytest.raises(ValueError, match="expected q, k"):
        g.delta_fwd(q, q, v, a[..., :2], a)
    with pytest.raises(ValueError, match="expected q, k"):
        g.delta_fwd(q[0], q[0], v[0], a[0], a[0])
    with pytest.raises(ValueError, match="one type"):
        g.delta_fwd(q, q.float(), v, a, a)
    with pytest.raises(ValueError, match="one type"):
        g.delta_fwd(q, q, v, a, a.to(bf))
    with pytest.raises(TypeError):
        g.delta_fwd(q.half(), q.half(), v.half(), a, a)
    with pytest.raises(TypeError):
        g.delta_fwd(q, q, v, a.double(), a.double())
    with pytest.raises(ValueError, match="S0"):
        g.delta_fwd(q, q, v, a, a, S0=torch.zeros(2, 4, 24, 16))
    with pytest.raises(ValueError, match="S0"):
        g.delta_fwd(q, q, v, a, a, S0=torch.zeros(2, 4, 24, 16).transpose(2, 3))
    with pytest.raises(ValueError, match="seq_offsets"):
        g.delta_fwd(q[:1], q[:1], v[:1], a[:1], a[:1], seq_offsets=torch.tensor([0, 5]))
    with pytest.raises(ValueError, match="seq_offsets"):
        g.delta_fwd(q[:1], q[:1], v[:1], a[:1], a[:1], seq_offsets=torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="dense"):                      # heads behind tokens
        g.delta_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), q, v, a, a)
    with pytest.raises(ValueError, match="evenly|overlapping"):         # one row for every sequence
        g.delta_fwd(q[:1].expand(2, 5, 2, 16), q, v, a, a)
    with pytest.raises(ValueError, match="dense|evenly|overlapping"):   # one gate for every head
        g.delta_fwd(q, q, v, a[..., :1].expand(2, 5, 4), a)
    with pytest.raises(ValueError, match="d_o"):
        g.delta_bwd(q, q, v, a, a, v.float(), torch.zeros(1))
    with pytest.raises(ValueError, match="ckpt"):
        g.delta_bwd(q, q, v, a, a, v, torch.zeros(1))
    with pytest.raises(ValueError, match="expected q, k"):
        g.delta_step(torch.zeros(2, 4, 16, 24), q, q, v, a, a)
    with pytest.raises(ValueError, match="S: expected"):
        g.delta_step(torch.zeros(2, 4, 16, 24, dtype=bf), q[:, 0], q[:, 0], v[:, 0], a[:, 0], a[:, 0])
    with pytest.raises(ValueError, match="workspace"):
        g.delta_fwd(q, q, v, a, a, workspace=torch.zeros(1 << 20, dtype=torch.uint8)[::2])
    d = g.DeltaDesc(2, 5, 2, 4, 16, 24, g.GDR_BF16, g.GDR_F32, 0, 0, 0, 0, 0)
    with pytest.raises(ValueError):                                     # the thin binding checks its tensors too
        g.gdr_delta_fwd(d, q, q, v.float(), a, a, None, 0, None, v, None, None, None, 0)


def _norm(g, **kw):
    base = dict(B=2, T=9, H=3, d=64, io_dtype=g.GDR_BF16, weight_dtype=g.GDR_F32, norm=g.GDR_NORM_RMS, next_norm=g.GDR_NORM_RMS,
                act=g.GDR_ACT_SILU, eps=1e-6, scale=1.0, res_scale=1.0, ldx=0, ldg=0, ldr=0)
    base.update(kw)
    return g.BlockNormDesc(**base)


NORM_FWD = "x gate res w w2 y n".split()
NORM_BWD = "x gate res w w2 dy dn dx dgate dres dw dw2 ws".split()


def _nf(g, d, **a):
    have = dict(zip(NORM_FWD, _ptrs(n=7, step=FAR)))
    have.update(a)
    return g.gdr_block_norm_fwd(d, *(have[x] for x in NORM_FWD), 0)


def _nb(g, d, need=1 << 40, **a):
    have = dict(zip(NORM_BWD, _ptrs(n=13, step=FAR)))
    have.update(a)
    return g.gdr_block_norm_bwd(d, *(have[x] for x in NORM_BWD), need, 0)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, -1), ("T", -1, -1), ("H", -1, -1), ("io_dtype", 3, -1), ("weight_dtype", 2, -1), ("norm", 3, -1), ("norm", -1, -1),
    ("next_norm", 3, -1), ("next_norm", -1, -1), ("act", 3, -1), ("act", -1, -1), ("eps", -1e-6, -1), ("eps", NAN, -1),
    ("scale", NAN, -1), ("res_scale", NAN, -1), ("ldx", 191, -1), ("ldg", -192, -1), ("ldr", 100, -1), ("ldx", 1 << 60, -1),
    ("d", 0, -2), ("d", 12, -2), ("d", 8200, -2), ("B", 1 << 30, -2), ("H", 1 << 28, -2),
])
def test_norm_descriptor(g, field, value, status):
    d = _norm(g, **{field: value})
    assert _nf(g, d) == status
    assert _nb(g, d) == status
    if not field.startswith("ld"):
        assert g.gdr_block_norm_bwd_workspace_size(d) == 0


def test_norm_forward_pointers(g):
    d = _norm(g)
    at = dict(zip(NORM_FWD, _ptrs(n=7, step=FAR)))
    for name in ("x", "y", "n"):
        assert _nf(g, d, **{name: None}) == g.GDR_EINVAL
    for name, shift in (("x", 1), ("gate", 1), ("res", 1), ("w", 2), ("w2", 2), ("y", 1), ("n", 1)):
        assert _nf(g, d, **{name: FakePtr(at[name].addr + shift)}) == g.GDR_EINVAL
    for name in ("y", "n"):
        for other in ("x", "gate", "w", "w2"):
            assert _nf(g, d, **{name: at[other]}) == g.GDR_EINVAL
    assert _nf(g, d, n=at["res"]) == g.GDR_EINVAL
    assert _nf(g, d, y=at["n"]) == g.GDR_EINVAL
    assert _nf(g, _norm(g, ldr=256), y=at["res"]) == g.GDR_EINVAL       # in place needs a dense residual
    assert _nf(g, d, y=FakePtr(at["res"].addr + 64)) == g.GDR_EINVAL
    off = _norm(g, next_norm=g.GDR_NORM_NONE)
    assert _nf(g, off, w2=None) == g.GDR_EINVAL                         # n without a next norm
    assert _nf(g, off, n=None) == g.GDR_EINVAL                          # its weight without one
    assert _nf(g, _norm(g, T=0), x=None, y=None, n=None) == g.GDR_OK


def test_norm_backward_pointers(g):
    d = _norm(g)
    at = dict(zip(NORM_BWD, _ptrs(n=13, step=FAR)))
    need = g.gdr_block_norm_bwd_workspace_size(d)
    assert need > 0
    for name in ("x", "dy", "dn", "dx", "dgate", "dres"):
        assert _nb(g, d, **{name: None}) == g.GDR_EINVAL
    for name in ("gate", "res", "w", "w2"):                             # a gradient without its input
        assert _nb(g, d, **{name: None}) == g.GDR_EINVAL
    for name, shift in (("x", 1), ("dy", 1), ("dn", 1), ("dx", 1), ("dgate", 1), ("dres", 1), ("dw", 2), ("dw2", 2)):
        assert _nb(g, d, **{name: FakePtr(at[name].addr + shift)}) == g.GDR_EINVAL
    for name in ("dx", "dgate", "dres", "dw", "dw2"):
        for other in ("x", "gate", "res", "w", "w2", "dy", "dn", "ws"):
            assert _nb(g, d, **{name: at[other]}) == g.GDR_EINVAL
    assert _nb(g, d, dx=at["dres"]) == g.GDR_EINVAL
    assert _nb(g, d, ws=None) == g.GDR_EWORKSPACE
    assert _nb(g, d, need=need - 1) == g.GDR_EWORKSPACE
    assert _nb(g, d, ws=FakePtr(at["ws"].addr + 4)) == g.GDR_EWORKSPACE
    off = _norm(g, next_norm=g.GDR_NORM_NONE)
    assert _nb(g, off, w2=None, dw2=None) == g.GDR_EINVAL               # dn without a next norm


def test_norm_binding(g):
    x = torch.zeros(2, 5, 3, 16)
    w = torch.ones(16)
    with pytest.raises(ValueError, match="device tensor"):
        g.block_norm(x)
    with pytest.raises(ValueError, match="norm"):
        g.block_norm(x, norm="l1")
    with pytest.raises(ValueError, match="act"):
        g.block_norm(x, gate=x, act="tanh")
    with pytest.raises(ValueError, match="gate"):
        g.block_norm(x, gate=x)
    with pytest.raises(ValueError, match="gate"):
        g.block_norm(x, act="silu")
    with pytest.raises(ValueError, match="residual"):
        g.block_norm(x, residual=x.bfloat16())
    with pytest.raises(ValueError, match="residual"):
        g.block_norm(x, residual=x[:, :4])
    with pytest.raises(ValueError, match="weight"):
        g.block_norm(x, weight=w[:8])
    with pytest.raises(ValueError, match="one type"):
        g.block_norm(x, weight=w, next_norm="rms", next_weight=w.bfloat16())
    with pytest.raises(ValueError, match="expected x"):
        g.block_norm(x[0])
    with pytest.raises(TypeError):
        g.block_norm(x.half())
    with pytest.raises(ValueError, match="out"):
        g.block_norm(x, out=torch.zeros(2, 5, 3, 8))
    with pytest.raises(ValueError, match="dense"):
        g.block_norm(torch.zeros(2, 3, 5, 16).transpose(1, 2))
    with pytest.raises(ValueError, match="dy"):
        g.block_norm_bwd(x, x.bfloat16())
    with pytest.raises(ValueError, match="dn"):
        g.block_norm_bwd(x, x, next_norm="rms", dn=x[:, :2])


PLACES = r'''
#include <stdio.h>
#include <stdlib.h>
#include "delta_place.hpp"
using namespace gdr;
// T, nseq, the offsets: every slot's sequence, first row and rows, and every sequence's slots
int main(int argc, char **argv) {
    DeltaParams p{};
    p.B = 1;
    p.T = atoi(argv[1]);
    p.nseq = atoi(argv[2]);
    int32_t *off = static_cast<int32_t *>(malloc(4 * (p.nseq + 1)));
    for (int i = 0; i <= p.nseq; ++i) off[i] = atoi(argv[3 + i]);
    p.off = off;
    p.nslot = p.T / kDeltaC + p.nseq;
    for (int s = 0; s < p.nslot; ++s) {
        const Place at = place_of(p, s);
        printf("%d %d %ld\n", at.seq, at.n, at.row0);
    }
    for (int i = 0; i < p.nseq; ++i) {
        long row0;
        const int n = tokens_of(p, i, row0);
        printf("%d %d %ld\n", first_slot(p, i), n, row0);
    }
    free(off);
}
'''


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("needs ROCm's clang++")
    at = tmp_path_factory.mktemp("places")
    (at / "places.cpp").write_text(PLACES)
    subprocess.run([CLANG, "-O1", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "tests", "host_gpu"), "-I", os.path.join(ROOT, "gated_delta_rule_84_amd", "csrc"),
                    str(at / "places.cpp"), "-c", "-o", str(at / "places.o")], check=True)
    # sanitizers need their runtime at the link; where it is not there the program runs without
    out = str(at / "places")
    if subprocess.run([CLANG, "-fsanitize=address,undefined", str(at / "places.o"), "-o", out], capture_output=True).returncode:
        subprocess.run([CLANG, "-O1", "-std=c++17", "-I", os.path.join(ROOT, "tests", "host_gpu"), "-I",
                        os.path.join(ROOT, "gated_delta_rule_84_amd", "csrc"), str(at / "places.cpp"), "-o", out], check=True)

    def run(T, off):
        n = len(off) - 1
        text = subprocess.run([out, str(T), str(n), *map(str, off)], check=True, capture_output=True, text=True).stdout
        rows = np.array(text.split(), np.int64).reshape(-1, 3)
        return rows[:-n], rows[-n:]
    return run


@pytest.mark.parametrize("T,off", [
    (1, [0, 1]), (200, [0, 200]), (200, [0, 64, 128, 200]), (200, [0, 0, 63, 63, 128, 193, 193]), (200, [5, 70, 70, 135, 190]),
    (130, [130, 130, 130]), (64, [0] * 9 + [64]), (300, [0, 1, 2, 3, 67, 68, 300])])
def test_places_of_sequences(places, T, off):
    """Every row of a sequence lies in one slot, at its place, and a sequence's slots follow each other."""
    slots, seqs = places(T, off)
    for i, (first, n, row0) in enumerate(seqs):
        assert n == off[i + 1] - off[i] and row0 == off[i]
        for c in range((n + 63) // 64):
            assert tuple(slots[first + c]) == (i, min(64, n - 64 * c), off[i] + 64 * c)
    assert sum(max(n, 0) for _, n, _ in slots) == off[-1] - off[0]


def test_places_of_any_offsets(places):
    """Whatever the offsets are, no slot and no sequence's chunk passes the rows, the slots or the states."""
    rng = np.random.default_rng(5)
    for _ in range(300):
        T, n = int(rng.integers(1, 400)), int(rng.integers(1, 12))
        kind = rng.integers(3)
        off = (rng.integers(-100, 600, n + 1) if kind == 0 else rng.integers(-2 ** 31, 2 ** 31, n + 1) if kind == 1 else
               np.sort(rng.integers(0, T + 1, n + 1))[::-1])
        slots, seqs = places(T, off.tolist())
        for seq, rows, row0 in slots:
            assert 0 <= seq < n and rows <= 64
            assert rows <= 0 or (row0 >= 0 and row0 + rows <= T)
        for first, rows, row0 in seqs:
            assert rows >= 0 and row0 >= 0 and row0 + rows <= T
            assert first >= 0 and first + (rows + 63) // 64 <= len(slots)
