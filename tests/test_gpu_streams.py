"""Calls of the wrappers with a `stream` that is not torch's current one.  What they allocate, what
they return and what they are given must not share memory with other work that is still pending:
the stream that the call runs on, or the current one, is held up by long work while the other one
goes on, and every result has to be that of the same call made alone."""
import pytest

from tests.gpu_util import gpu, log

pytestmark = pytest.mark.gpu


def _calls(torch, g):
    """name -> (call(inputs, **kw) returning a tuple of tensors and None, its inputs)"""
    gen = torch.Generator().manual_seed(61)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    x, dy, gate = r(1, 3000, 2, 64), r(1, 3000, 2, 64), torch.sigmoid(r(1, 3000, 2, 64))
    dST, w, f = r(1, 2, 64), r(64), g.rope_inv_freq(64)[0]
    q, k = r(1, 3000, 4, 64), r(1, 3000, 2, 64)
    ckpt = g.scan_fwd(x, gate, want_ckpt=True)[2]
    S = r(512, 2, 64)
    bf, sig, unit = torch.bfloat16, torch.sigmoid, torch.nn.functional.normalize
    heads = [unit(r(1, 1024, 2, 128), dim=-1).to(bf) for _ in range(3)]
    alpha, beta = sig(r(1, 1024, 2) + 4), sig(r(1, 1024, 2))
    states = g.chunk_fwd_ckpt(*heads, alpha, beta, 256)[2]
    n, few = 32, [unit(r(64, 50, 2, 8), dim=-1) for _ in range(3)]
    return {
        "chunk_fwd": (g.chunk_fwd, (*heads, alpha, beta)),
        "chunk_fwd_ckpt": (lambda *t, **kw: g.chunk_fwd_ckpt(*t, 256, **kw), (*heads, alpha, beta)),
        "mc_readout": (lambda q, c, **kw: (g.mc_readout(q, c, 256, **kw),), (heads[0], states)),
        "osdn_precond": (lambda k, b, **kw: g.osdn_precond(k, b, 0.5, **kw), (heads[1], beta)),
        "sdm_fwd": (lambda *t, **kw: g.sdm_fwd(*t, 8, 8, want_slots=True, **kw),
                    (r(1, 2, n * n, 128), r(1, 1024, 2, 2, n), r(1, 1024, 2, 2, n), r(1, 1024, 2, 128).to(bf), alpha, beta)),
        "dmem_fwd": (lambda *t, **kw: (g.dmem_fwd(*t, **kw),),
                     (r(64, 2, 8, 8), *few, sig(r(64, 50, 2)), sig(r(64, 50, 2)))),
        "decode_step": (lambda *t, **kw: (g.decode_step(*t, **kw),),
                        (r(64, 2, 64, 64), *(unit(r(64, 2, 64), dim=-1) for _ in range(3)), sig(r(64, 2)), sig(r(64, 2)))),
        "scan_fwd": (lambda x, a, **kw: g.scan_fwd(x, a, want_ckpt=True, **kw), (x, gate)),
        "scan_bwd": (lambda x, a, dy, ck, d, **kw: g.scan_bwd(x, a, dy, ck, dST=d, **kw), (x, gate, dy, ckpt, dST)),
        "scan_step": (lambda S, x, a, **kw: (g.scan_step(S, x, a, **kw),), (S, r(512, 2, 64), torch.sigmoid(r(512, 2, 64)))),
        "qk_prep": (lambda q, k, w, f, **kw: g.qk_prep(q, k, wq=w, wk=w, inv_freq=f, **kw), (q, k, w, f)),
        "qk_prep_bwd": (lambda q, k, gq, gk, w, f, **kw: g.qk_prep_bwd(q, k, gq, gk, wq=w, wk=w, inv_freq=f, **kw),
                        (q, k, r(1, 3000, 4, 64), r(1, 3000, 2, 64), w, f)),
    }


NAMES = ["chunk_fwd", "chunk_fwd_ckpt", "mc_readout", "osdn_precond", "sdm_fwd", "dmem_fwd", "decode_step",
         "scan_fwd", "scan_bwd", "scan_step", "qk_prep", "qk_prep_bwd"]


def _busy(torch, stream):
    """Some tens of milliseconds of work on `stream`."""
    with torch.cuda.stream(stream):
        big = torch.zeros(1 << 28, device="cuda")
        for _ in range(60):
            big.add_(1.0)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_dropped_results_and_inputs(name, raw):
    """Results and inputs dropped right after the call are not handed to the current stream's work meanwhile."""
    torch, g = gpu()
    log(f"[streams] dropped, {name}")
    call, inputs = _calls(torch, g)[name]
    want = call(*[t.clone() for t in inputs])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for keep in range(len(want)):
        given = [t.clone() for t in inputs]
        side.wait_stream(torch.cuda.current_stream())
        _busy(torch, side)
        got = call(*given, stream=side.cuda_stream if raw else side)
        sizes = [(t.shape, t.dtype) for t in got + tuple(given) if t is not None]
        got = got[keep]  # the other results and the inputs are gone
        del given
        fills = [torch.zeros(s, dtype=d, device="cuda") for s, d in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert not any(t.any() for t in fills)
        assert got is None or torch.equal(got, want[keep])


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_pending_work_still_uses(name):
    """A block dropped on the current stream, with work pending there that still writes to it, is not what a call on
    another stream works in."""
    torch, g = gpu()
    log(f"[streams] pending, {name}")
    call, inputs = _calls(torch, g)[name]
    want = call(*[t.clone() for t in inputs])
    sizes = [(t.shape, t.dtype) for t in want if t is not None] + [((1 << 16,), torch.uint8)]  # and a workspace's
    given = [t.clone() for t in inputs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy(torch, torch.cuda.current_stream())
    blocks = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes for _ in range(3)]
    for t in blocks:
        t.fill_(77)
    del blocks, t
    got = call(*given, stream=side)
    torch.cuda.synchronize()
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))
