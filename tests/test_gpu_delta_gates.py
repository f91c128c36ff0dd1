"""The trainable delta rule with single log gates so low that nothing passes them: whatever their size, the gates behind
them count in full.  Tolerances as in test_gpu_delta.py: a gate's e^g is 0 in the reference and in fp32 alike."""
import numpy as np
import pytest

from tests.gpu_util import gpu, to_np
from tests.test_gpu_delta import Case, _check, _close, _tol

pytestmark = pytest.mark.gpu

LOWEST = {"f32": -3.4028234663852886e38, "bf16": -3.3895313892515355e38}


def _cut(c, value):
    """One such gate in the middle of the first chunk, two in the second, one at the border of the third, in a head each."""
    value = LOWEST[c.gate] if value == "lowest" else value
    for head in range(c.Hv):
        for t in (20 + head, 90, 101 + head, 128):
            c.g[:, t, head] = value
    return c


@pytest.mark.parametrize("io,gate", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("value", [-120.0, -255.0, -257.0, -1e4, -1e12, -1e30, "lowest"])
def test_gates_behind_a_low_one(io, gate, value):
    _check(_cut(Case(B=2, T=150, Hk=1, Hv=2, dk=32, dv=32, io=io, gate=gate), value))


@pytest.mark.parametrize("value", [-1e4, -1e30, "lowest"])
def test_low_gate_in_packed_rows_and_wide_heads(value):
    _check(_cut(Case(B=1, T=190, Hk=1, Hv=2, dk=128, dv=128, off=[0, 65, 65, 190], lay="fused"), value))


@pytest.mark.parametrize("value", [-300.0, -1e12, "lowest", -float("inf")])
def test_low_gate_forgets_exactly(value):
    """Behind it, results are those of a start there, bit for bit, and its gradient is 0."""
    torch, g = gpu()
    c = Case(B=1, T=140, Hk=1, Hv=2, dk=64, dv=64, io="f32")
    c.g[:, 128] = LOWEST["f32"] if value == "lowest" else value
    o, ST, ck = c.forward(want_ckpt=True)
    assert (c.backward(ck)[3][:, 128] == 0).all()
    o2, S2, _ = g.delta_fwd(*(x[:, 128:].contiguous() for x in c.inputs))
    assert torch.equal(o[:, 128:], o2) and torch.equal(ST, S2)


@pytest.mark.parametrize("value", [-1e4, -1e12, -1e30, "lowest"])
def test_low_gate_step_follows_forward(value):
    torch, g = gpu()
    c = _cut(Case(B=2, T=140, Hk=1, Hv=2, dk=64, dv=64, io="f32"), value)
    o, ST, _ = c.forward()
    S = c.S0.clone()
    out = torch.stack([g.delta_step(S, *(x[:, t].contiguous() for x in c.inputs)) for t in range(140)], 1)
    tol = 2 * _tol(64, "f32", "f32")  # each side its own
    _close("o", to_np(out), to_np(o), tol)
    _close("S", to_np(S), to_np(ST), tol)


def test_growth_behind_a_low_gate():
    """Gates above 0 behind the cut: e^0.02 a token."""
    torch, _ = gpu()
    c = Case(B=1, T=150, Hk=1, Hv=2, dk=32, dv=32, io="f32")
    c.g.copy_(torch.rand(c.g.shape, generator=torch.Generator().manual_seed(3)) * 0.04)
    _check(_cut(c, -1e30))


def test_lowest_values_are_the_types():
    torch, _ = gpu()
    assert np.float32(LOWEST["f32"]) == torch.finfo(torch.float32).min and LOWEST["bf16"] == torch.finfo(torch.bfloat16).min
