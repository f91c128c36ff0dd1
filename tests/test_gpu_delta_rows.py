"""Gradients of rows that belong to no packed sequence, as the binding returns them."""
import pytest

from tests.gpu_util import gpu
from tests.test_gpu_delta import Case

pytestmark = pytest.mark.gpu


def _poison(torch, shapes):
    """Memory that the next allocations of these shapes are likely to get, filled with NaN."""
    held = [torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in shapes]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("io,gate", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("off", [[10, 80, 80, 121], [0, 150], [150, 150], [0, 0, 64], [5]])
def test_gradients_of_rows_of_no_sequence_are_zero(io, gate, off):
    """They do not enter the loss, so their gradients are 0 even where the rows hold NaN."""
    torch, g = gpu()
    c = Case(B=1, T=150, Hk=1, Hv=2, dk=24, dv=40, off=off, io=io, gate=gate)
    ck = c.forward(want_ckpt=True)[2]
    _poison(torch, [(x.shape, x.dtype) for x in c.inputs])
    grads = c.backward(ck)
    for x, grad in zip(c.inputs, grads):
        assert grad.shape == x.shape and grad.dtype == x.dtype
        assert (grad[0, :off[0]] == 0).all() and (grad[0, off[-1]:] == 0).all()
        assert torch.isfinite(grad.float()).all()
    if off[-1] - off[0] > 1:
        assert all((grad[0, off[0]:off[-1]] != 0).any() for grad in grads[:5])


def test_zeroed_rows_in_a_graph():
    """Captured and replayed: the rows are zeros after each replay, whatever was written there between."""
    torch, g = gpu()
    c = Case(B=1, T=150, Hk=1, Hv=2, dk=24, dv=40, off=[10, 80, 121])
    ck = c.forward(want_ckpt=True)[2]
    want = [x.clone() for x in c.backward(ck)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = c.backward(ck)
    for _ in range(3):
        for x in grads:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, grads))
        torch.ones(1000, device="cuda").sum().item()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_packed_sequences_without_any_row(io):
    """T = 0: states pass through, forward and backward, and the gradients have no rows."""
    torch, g = gpu()
    c = Case(B=1, T=0, Hk=1, Hv=2, dk=128, dv=72, off=[0, 0, 0, 0], io=io)
    o, ST, ck = c.forward(want_ckpt=True)
    grads = c.backward(ck)
    assert o.numel() == 0 and torch.equal(ST, c.S0) and torch.equal(grads[5], c.dST)
    assert all(x.shape == y.shape for x, y in zip(grads, c.inputs))
