"""Block norm: rows of zeros with an eps of almost nothing, and workgroups that stay for several rows, in the forms that
test_gpu_block_norm.py gives one row each.  Tolerances as derived there."""
import numpy as np
import pytest

from oracle import block_norm as ref
from tests.gpu_util import gpu, to_np
from tests.test_gpu_block_norm import U, _check, _norm_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [16, 72, 1000, 4104])
@pytest.mark.parametrize("eps", [1e-40, 1e-38, 1e-30])
def test_rows_of_zeros_with_a_tiny_eps(d, eps):
    """The factor r' = eps^(-1/2) is up to 1e20 and its square passes fp32's range: gradients are r' w_next dn."""
    torch, g = gpu()
    x = torch.zeros(1, 5, 3, d, device="cuda")
    x[0, 1] = 1
    gen = torch.Generator().manual_seed(5)
    dn, w2 = torch.randn(x.shape, generator=gen).cuda(), torch.ones(d, device="cuda")
    dy = torch.zeros_like(x)
    for norm in ("rms", "l2"):
        how = dict(norm="none", eps=eps, next_norm=norm)
        y, n = g.block_norm(x, next_weight=w2, **how)
        dx, _, _, _, dw2 = g.block_norm_bwd(x, dy, dn=dn, next_weight=w2, **how)
        flat = lambda t: to_np(t).reshape(-1, d)  # noqa: E731
        how["eps"] = float(np.float32(eps))
        want = ref.backward(flat(x), flat(dy), dn=flat(dn), next_weight=np.ones(d), **how)
        for row in range(15):  # each by itself: rows of zeros have gradients 1e20 times those of the others
            _norm_close(f"dx {row}", flat(dx)[row], want[0][row], 256 * U)
        _norm_close("dw_next", to_np(dw2), want[4], (256 + 4) * U)
        assert (n[0, 0] == 0).all() and torch.isfinite(n).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,rows", [(4104, 2000), (8192, 1700)])
def test_many_wide_rows(io, d, rows):
    """Two pieces a lane, without the next row's loads ahead: at most 910 workgroups backward, two or three rows each."""
    _check(1, rows, 1, d, io=io, act="sigmoid")


@pytest.mark.parametrize("d,rows", [(64, 70001), (128, 40001), (40, 70001)])
def test_many_narrow_rows_in_fp32(d, rows):
    """Workgroups take at most 65,536 rows of 64 channels, or 32,768 of 128, at once: the rest is their second round."""
    _check(1, rows, 1, d, io="f32", wt="bf16", residual=False, next_norm="none")
    _check(1, rows, 1, d, io="f32", act=None)
