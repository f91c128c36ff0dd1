"""The gated linear recurrence's entry points and kernels on the CPU.

The library's own sources are compiled for the CPU (tests/host_gpu): a workgroup is a thread, its
lanes are fibers, workgroups run side by side, and every tensor lies between pages that cannot be
accessed, at their start and at their end.  An access out of range ends the program, which
fails the case.  Results are held to the bounds of tests/test_gpu_scan.py.  The offsets are
any whole numbers in some cases: then only the accesses count."""
import os
import shutil
import struct
import subprocess

import numpy as np
import pytest
import torch

from tests.test_gpu_scan import STEP, U, _bounds

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_84_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
LOG, COUPLED = 0x40, 0x80

pytestmark = pytest.mark.skipif(not os.path.exists(CLANG), reason="needs ROCm's clang++")


def _build(out, csrc):
    subprocess.run([CLANG, "-O1", "-std=c++17", "-mfma", "-pthread", "-I", os.path.join(ROOT, "tests", "host_gpu"), "-I",
                    os.path.join(ROOT, "include"), "-I", csrc, "-x", "c++",
                    os.path.join(ROOT, "tests", "host_gpu", "scan_host.cpp"), "-o", str(out)], check=True)
    return str(out)


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return _build(tmp_path_factory.mktemp("scan") / "scan_host", CSRC)


def _raw(t):
    return (t.contiguous().view(torch.int16) if t.dtype == torch.bfloat16 else t.contiguous()).numpy().tobytes()


def _run(program, B, T, D, io, gate, form, kind, offsets=None, gap=0, states=True, at_end=True, resident=16, skip_first=False):
    """Inputs and, where the program ends well, its outputs as fp64 arrays with the raw bytes of y, dx and dalpha."""
    gen = torch.Generator().manual_seed(51)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n = B if offsets is None else len(offsets) - 1
    ld = D + gap
    rows = lambda v, t: torch.cat([v, r(B * T, gap)], -1).to(TYPE[t]) if gap else v.to(TYPE[t])  # noqa: E731
    raw = -torch.nn.functional.softplus(r(B * T, D) * 2 - 2)
    x, alpha = rows(r(B * T, D), io), rows(raw if form == "log" else raw.exp(), gate)
    beta = rows(torch.sigmoid(r(B * T, D)), gate) if kind == "beta" else None
    dy, S0, dST = r(B * T, D).to(TYPE[io]), r(n, D), r(n, D)
    flags = (LOG if form == "log" else 0) | (COUPLED if kind == "coupled" else 0)
    head = struct.pack("<16q", B, T, 1, D, io == "f32", gate == "f32", flags, ld, ld, ld, beta is not None,
                       -1 if offsets is None else n, states, at_end, resident, skip_first)
    cut = lambda t: None if t is None else _raw(t)[:max(0, (B * T - 1) * ld + D) * t.element_size()]  # noqa: E731
    parts = [cut(x), cut(alpha), cut(beta), None if offsets is None else np.array(offsets, np.int32).tobytes(),
             _raw(S0) if states else None, _raw(dy), _raw(dST) if states else None]
    done = subprocess.run([program], input=head + b"".join(p for p in parts if p is not None), capture_output=True, timeout=110)
    assert done.returncode == 0, f"ended with {done.returncode}: {done.stderr[-500:]!r}"
    blocks = -(-T // 256)
    shapes = [("y", (B, T, D), io), ("ST", (n, D), "f32"), ("ckpt", (B, blocks, D), "f32"), ("dx", (B, T, D), io),
              ("dalpha", (B, T, D), gate)] + ([("dbeta", (B, T, D), gate)] if beta is not None else []) + [("dS0", (n, D), "f32")]
    out, bits, at = {}, {}, 0
    for name, shape, t in shapes:
        size = int(np.prod(shape)) * (2 if t == "bf16" else 4)
        piece = np.frombuffer(done.stdout, np.uint8, size, at).copy()
        at += size
        bits[name] = piece.reshape(shape[:-1] + (-1,)) if size else piece
        out[name] = torch.from_numpy(piece).view(TYPE[t]).double().numpy().reshape(shape)
    assert at == len(done.stdout)
    f64 = lambda t: t[:, :D].double().numpy().reshape(B, T, D)  # noqa: E731
    state = lambda t: t.numpy().astype(np.float64) * states  # noqa: E731
    how = dict(beta=None if beta is None else beta[:, None, :D].reshape(B, T, 1, D), S0=torch.from_numpy(state(S0)).reshape(n, 1, D),
               log_gate=form == "log", coupled=kind == "coupled")
    return out, bits, lambda: _bounds(f64(x), f64(alpha), how, f64(dy), state(dST), offsets)


def _check(out, bits, want, io, gate, offsets):
    for name, (value, err) in want.items():
        step = {"y": STEP[io], "dx": STEP[io], "dalpha": STEP[gate], "dbeta": STEP[gate]}.get(name, U)
        there = ~np.isnan(value)
        over = np.abs(out[name] - value)[there] / np.maximum(step * np.abs(value) + err, 1e-300)[there]
        assert over.size == 0 or np.max(over) <= 1.0, (name, np.max(over))
    if offsets is not None:  # rows of no sequence are left as they were
        inside = np.zeros(out["y"].shape[1], bool)
        for p, q in zip(offsets, offsets[1:]):
            inside[p:q] = True
        for name in ("y", "dx", "dalpha", "dbeta"):
            assert name not in bits or (bits[name][:, ~inside] == 0x5a).all(), name


DENSE = [
    # B, T, channels, io, gate, form, kind, gap
    (1, 1, 1, "f32", "f32", "value", "one", 0),
    (2, 7, 3, "bf16", "f32", "value", "beta", 5),
    (2, 513, 65, "bf16", "bf16", "value", "one", 3),
    (1, 257, 129, "bf16", "bf16", "log", "beta", 0),
    (3, 256, 32, "f32", "f32", "log", "coupled", 0),
    (1, 5300, 3, "f32", "bf16", "log", "coupled", 1),
    (1, 2600, 12, "f32", "f32", "log", "beta", 0),
]


@pytest.mark.parametrize("at_end", [False, True], ids=["start", "end"])
@pytest.mark.parametrize("case", DENSE, ids=lambda c: "-".join(map(str, c)))
def test_dense(program, case, at_end):
    B, T, D, io, gate, form, kind, gap = case
    out, bits, want = _run(program, B, T, D, io, gate, form, kind, gap=gap, at_end=at_end)
    _check(out, bits, want(), io, gate, None)


PACKED = [
    # rows, borders, channels, io, gate, form, kind
    (2600, [1030, 1040], 12, "f32", "f32", "log", "beta"),        # the case that tests/test_gpu_scan.py leaves out
    (2600, [1030, 1040], 12, "f32", "f32", "value", "beta"),
    (2600, [1030, 1040], 12, "f32", "f32", "log", "one"),
    (2600, [1030, 1040], 13, "bf16", "bf16", "log", "beta"),
    (2600, [1030, 1040], 70, "f32", "bf16", "log", "coupled"),
    (2599, [1023, 1024], 11, "f32", "f32", "log", "beta"),
    (2600, [0, 1], 12, "f32", "f32", "log", "beta"),
    (2600, [2599, 2600], 12, "f32", "f32", "log", "beta"),
    (2600, [1030, 1030, 1040, 1040], 12, "f32", "f32", "log", "beta"),
    (9, [0, 0, 9, 9], 5, "f32", "bf16", "log", "coupled"),
    (1500, [0, 0, 0, 0], 12, "bf16", "f32", "log", "beta"),
    (4700, [7, 7, 2050, 4500], 5, "bf16", "f32", "value", "beta"),
    (700, [3, 3, 4, 12, 250, 256, 257, 600, 600, 690], 11, "bf16", "bf16", "value", "coupled"),
]


@pytest.mark.parametrize("at_end", [False, True], ids=["start", "end"])
@pytest.mark.parametrize("states", [True, False], ids=["states", "none"])
@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"{c[0]}x{c[2]}-{len(c[1]) - 1}seqs-{'-'.join(c[3:])}")
def test_packed(program, case, states, at_end):
    T, offsets, D, io, gate, form, kind = case
    out, bits, want = _run(program, 1, T, D, io, gate, form, kind, offsets=offsets, states=states, at_end=at_end)
    _check(out, bits, want(), io, gate, offsets)


@pytest.mark.parametrize("resident", [1, 3, 40])
def test_results_do_not_depend_on_how_many_blocks_run_at_once(program, resident):
    for offsets in (None, [1030, 1040], [5, 300, 300, 4700, 4990]):
        args = (program, 1, 5000, 12, "f32", "f32", "log", "beta")
        _, one, _ = _run(*args, offsets=offsets)
        _, many, _ = _run(*args, offsets=offsets, resident=resident)
        assert all(np.array_equal(one[k], many[k]) for k in one)


BAD = [[40, 10], [-5, 2600], [0, 1 << 30], [2 ** 31 - 1, -2 ** 31], [0, 900, 300, 2600], [-1, -1, 700, 3000, 5, 2600],
       [2 ** 31 - 1] * 4, [-2 ** 31] * 4, [500, 400, 300, 200, 100]]


@pytest.mark.parametrize("at_end", [False, True], ids=["start", "end"])
@pytest.mark.parametrize("offsets", BAD, ids=str)
def test_offsets_that_break_the_rules_reach_nothing_outside(program, offsets, at_end):
    _run(program, 1, 2600, 12, "f32", "f32", "log", "beta", offsets=offsets, at_end=at_end)
    _run(program, 1, 300, 70, "bf16", "bf16", "value", "one", offsets=offsets, at_end=at_end)


def test_a_wait_in_vain_ends_and_shows(tmp_path):
    """The first block is never run and the bound is small: every block behind it ends, with NaN and not with numbers."""
    csrc = tmp_path / "csrc"
    shutil.copytree(CSRC, csrc)
    header = csrc / "scan_impl.hpp"
    text = header.read_text()
    assert text.count("kMaxPolls = 1 << 22") == 1
    header.write_text(text.replace("kMaxPolls = 1 << 22", "kMaxPolls = 20"))
    program = _build(tmp_path / "scan_host", str(csrc))
    for T, offsets in ((3000, None), (700, None), (3000, [0, 3000]), (3000, [100, 2500])):
        out, bits, _ = _run(program, 1, T, 12, "f32", "f32", "value", "one", offsets=offsets, skip_first=True)
        end = T if offsets is None else offsets[-1]
        assert (bits["y"][:, :256] == 0x5a).all()
        assert np.isnan(out["y"][:, 256:end]).all() and np.isnan(out["ST"]).all()
        assert np.isnan(out["ckpt"][:, 1:end // 256]).all()
