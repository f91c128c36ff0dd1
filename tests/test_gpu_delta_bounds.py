"""What the trainable delta rule promises of single elements of a bf16 o, and of results beside inputs that are not finite.

o's bound, element by element (include/gdr.h): its rounding to bf16, half a step; 2^-15 of sum |q| |front S|, whose state is cut to
16 bits; 2^-13 of sum |Q| |D|, both cut; and what reaches it in fp32: D, each of whose elements is off by its share of 2^-21 of
the products it comes from, at most 64 + dk terms one behind another, taken as (64 + dk) 2^-21 of the largest |D| a token can
have, and sums of as many terms, (64 + dk) 2^-24 of the sizes above."""
import numpy as np
import pytest

from oracle import delta as ref
from tests.gpu_util import gpu, log, to_np
from tests.test_gpu_delta import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cancels", [False, True])
@pytest.mark.parametrize("dk,dv,T", [(64, 64, 64), (128, 40, 37), (128, 128, 1)])
def test_elements_of_o(cancels, dk, dv, T):
    torch, _ = gpu()
    c = Case(B=1, T=T, Hk=1, Hv=2, dk=dk, dv=dv, io="bf16")
    if cancels:  # large states whose rows nearly agree, read with weights that sum to nothing: o is 1 in a thousand of its terms
        c.S0.copy_(100 + 0.1 * c.S0)
        c.q[..., 1::2] = -c.q[..., 0::2]
    o = to_np(c.forward()[0])[0]
    q, k, v, g, b = (to_np(x)[0] for x in c.inputs)
    want = ref.forward(q, k, v, g, b, to_np(c.S0)[0])
    S0, worst = to_np(c.S0)[0], 0.0
    for h in range(2):
        P = np.cumsum(g[:, h])
        before = np.concatenate([S0[None, h], want[2][:-1, h]])
        D = v[:, h] - np.exp(g[:, h])[:, None] * np.einsum("tij,ti->tj", before, k[:, 0])
        e = np.tril(np.exp(np.minimum(P[:, None] - P[None], 0.0))) * b[None, :, h]
        Q = np.abs(e * (q[:, 0] @ k[:, 0].T))
        read = np.exp(P)[:, None] * (np.abs(q[:, 0]) @ np.abs(S0[h]))
        wrote = Q @ np.abs(D)
        first = np.abs(v[:, h]) + np.exp(P)[:, None] * (np.abs(k[:, 0]) @ np.abs(S0[h]))  # what D is solved from
        n = T + dk
        bound = 2.0 ** -8 * np.abs(want[0][:, h]) + 2.0 ** -15 * read + 2.0 ** -13 * wrote + n * 2.0 ** -24 * (read + wrote) + \
            n * 2.0 ** -21 * Q.sum(-1, keepdims=True) * first.max()
        worst = max(worst, float((np.abs(o[:, h] - want[0][:, h]) / bound).max()))
    log(f"  o: {worst:.3f} of the bound")
    assert worst <= 1


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["q", "k", "v", "g", "b"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_inside_a_sequence(io, what, value):
    """At token 100 of the second of three sequences: the chunks before it, other heads and other sequences keep their bits,
    forward and backward."""
    torch, g = gpu()
    off = [0, 70, 270, 331]
    make = lambda: Case(B=1, T=331, Hk=2, Hv=4, dk=64, dv=48, io=io, off=off)  # noqa: E731
    c, bad = make(), make()
    at, head = 70 + 100, 1            # chunk 1 of its sequence; a key head, and its value heads 2 and 3
    x = getattr(bad, what)
    x[0, at, head if what in "qk" else 2 * head] = value
    touched = [2, 3] if what in "qk" else [2]
    rest = [h for h in range(4) if h not in touched]
    o, ST, ck = c.forward(want_ckpt=True)
    o2, ST2, ck2 = bad.forward(want_ckpt=True)
    assert torch.equal(o[:, :, rest], o2[:, :, rest]) and torch.equal(ST[:, rest], ST2[:, rest])
    first = 70 + 64                   # of the chunk
    assert torch.equal(o[:, :first], o2[:, :first]) and torch.equal(o[:, 270:], o2[:, 270:])
    assert torch.equal(ST[[0, 2]], ST2[[0, 2]])
    assert not torch.isfinite(o2[0, at, 2].float()).any()
    grads, grads2 = c.backward(ck), bad.backward(ck2)
    for j, (a, b) in enumerate(zip(grads[:5], grads2[:5])):
        others = [0] if j < 2 else rest
        assert torch.equal(a[:, :, others], b[:, :, others])
        assert torch.equal(a[:, :70], b[:, :70]) and torch.equal(a[:, 270:], b[:, 270:])
    assert torch.equal(grads[5][:, rest], grads2[5][:, rest]) and torch.equal(grads[5][[0, 2]], grads2[5][[0, 2]])
