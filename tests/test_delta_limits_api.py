"""Host-side checks of the trainable delta rule and of the bindings beside it, with nothing launched: limits that are those of
the launches, tensors that are checked whatever the descriptor's ignored fields hold."""
import pytest
import torch

from tests.test_abi import FakePtr
from tests.test_delta_norm_api import _bwd, _delta, _fwd, _step


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_84_amd as g

    return g


def _far(*names):
    """Addresses that no tensor of these calls reaches from one to the next."""
    return {n: FakePtr((i + 1) << 44) for i, n in enumerate(names)}


@pytest.mark.parametrize("dv,most", [(128, (2 ** 32 - 1) // 768 // 8 * 8), (72, (2 ** 32 - 1) // 768 // 8 * 8), (64, 2 ** 23 - 9)])
def test_chains_of_a_launch(g, dv, most):
    """The recurrence has 384 threads to four column tiles of a value head of a sequence, heads rounded up to 8: a launch of 2^32
    threads or more is refused before anything is launched, also without tokens, where it only copies states."""
    for T in (0, 1):
        over = _delta(g, B=most + 1, T=T, Hk=1, Hv=1, dk=8, dv=dv)
        assert _fwd(g, over, **_far("q", "k", "v", "gate", "beta", "S0", "o", "ST", "ck", "ws")) == g.GDR_EUNSUPPORTED
        assert _bwd(g, over, **_far(*"q k v gate beta ck do dST dq dk dv dg db dS0 ws".split())) == g.GDR_EUNSUPPORTED
        off = FakePtr(0x7000000)
        packed = _delta(g, B=1, T=T, Hk=1, Hv=1, dk=8, dv=dv)
        assert _fwd(g, packed, n=most + 1, off=off, **_far("q", "k", "v", "gate", "beta", "S0", "o", "ST", "ck", "ws")) == \
            g.GDR_EUNSUPPORTED
    assert g.gdr_delta_workspace_size(over) == 0 and g.gdr_delta_ckpt_size(over) == 0
    fits = _delta(g, B=most, T=1, Hk=1, Hv=1, dk=8, dv=dv)
    assert g.gdr_delta_workspace_size(fits) > 0 and g.gdr_delta_ckpt_size(fits) > 0


@pytest.mark.parametrize("T", [-1, -(2 ** 31), 0, 1, 2 ** 31 - 1])
def test_step_checks_its_tensors_whatever_T_is(g, T):
    """A step ignores the descriptor's T, and the binding's checks of its tensors do too."""
    B, Hk, Hv, dk, dv = 2, 2, 4, 16, 24
    d = _delta(g, B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv)
    bf = torch.bfloat16
    have = dict(q=torch.zeros(B, Hk, dk, dtype=bf), k=torch.zeros(B, Hk, dk, dtype=bf), v=torch.zeros(B, Hv, dv, dtype=bf),
                gate=torch.zeros(B, Hv), beta=torch.zeros(B, Hv), S=torch.zeros(B, Hv, dk, dv), o=torch.zeros(B, Hv, dv, dtype=bf))
    names = dict(gate="log_gate")
    for name, t in have.items():
        with pytest.raises(ValueError, match=f"{names.get(name, name)}: expected .* elements"):
            _step(g, d, **dict(have, **{name: t[:1]}))
        with pytest.raises(ValueError, match=f"{names.get(name, name)}: expected dtype"):
            _step(g, d, **dict(have, **{name: t.double()}))


def test_key_heads_without_value_heads(g):
    """Nothing would be computed, and the gradients of q and k of these heads, which are 0, would be left unwritten."""
    d = _delta(g, Hk=2, Hv=0)
    assert _fwd(g, d) == g.GDR_EINVAL and _bwd(g, d) == g.GDR_EINVAL and _step(g, d) == g.GDR_EINVAL
    assert g.gdr_delta_workspace_size(d) == 0 and g.gdr_delta_ckpt_size(d) == 0


def test_workspace_that_is_not_used(g):
    """A workspace that is too small is replaced, whatever its strides are; one that is used is dense."""
    every_other = torch.zeros(64, dtype=torch.uint8)[::2]
    new = g._room(every_other, 33, "cpu")
    assert new.numel() == 33 and new.is_contiguous()
    with pytest.raises(ValueError, match="workspace"):
        g._room(every_other, 32, "cpu")
    dense = torch.zeros(64, dtype=torch.uint8)
    assert g._room(dense, 64, "cpu") is dense and g._room(dense, 0, "cpu") is dense and g._room(None, 0, "cpu") is None


@pytest.mark.gpu
def test_small_strided_workspace_is_replaced(g):
    """As scan_fwd, scan_bwd and qk_prep_bwd always did."""
    x, a = torch.rand(1, 600, 2, 64, device="cuda"), torch.rand(1, 600, 2, 64, device="cuda")
    small = torch.zeros(16, dtype=torch.uint8, device="cuda")[::2]
    y, ST, ck = g.scan_fwd(x, a, want_ckpt=True)
    y2, S2, ck2 = g.scan_fwd(x, a, want_ckpt=True, workspace=small)
    assert torch.equal(y, y2) and torch.equal(ST, S2) and torch.equal(ck, ck2)
    assert all(torch.equal(p, r) for p, r in zip([t for t in g.scan_bwd(x, a, x, ck) if t is not None],
                                                 [t for t in g.scan_bwd(x, a, x, ck, workspace=small) if t is not None]))
    w = torch.rand(64, device="cuda")
    assert all(torch.equal(p, r) for p, r in zip(g.qk_prep_bwd(x, a, x, a, wq=w, wk=w),
                                                 g.qk_prep_bwd(x, a, x, a, wq=w, wk=w, workspace=small)))
