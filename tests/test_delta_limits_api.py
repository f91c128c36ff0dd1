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
