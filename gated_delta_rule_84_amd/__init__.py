"""Python binding of the gated delta-rule HIP library (libgdr.so, include/gdr.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C-ABI.  PyTorch supplies device memory and the current
stream.  The functions with the C names (``gdr_chunk_fwd``, ``gdr_decode_step``,
``gdr_chunk_fwd_workspace_size``, ``gdr_chunk_fwd_path``, ``gdr_status_string``)
take a ``Desc`` and tensors (or None) and return the C status code;
``chunk_fwd`` and ``decode_step`` allocate outputs and raise on a non-OK
status.

The library must have been built (``python gated_delta_rule_84_amd/build.py``);
importing this package without it raises ImportError.  There is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch  # loads the HIP runtime the library binds to

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")

GDR_OK, GDR_EINVAL, GDR_EUNSUPPORTED, GDR_EWORKSPACE, GDR_EHIP, GDR_ETOOLARGE = 0, -1, -2, -3, -4, -5
GDR_NOALLOC_SCRATCH_BYTES = 128 << 20
GDR_BF16, GDR_F32 = 0, 1
GDR_ALPHA_SCALAR, GDR_ALPHA_CHANNEL = 0, 1
GDR_BETA_SCALAR, GDR_BETA_SHARED, GDR_BETA_KV = 0, 1, 2
GDR_FLAG_READ_BEFORE_WRITE = 0x10
GDR_FLAG_UNDECAYED_PREDICTION = 0x20
GDR_FLAG_LOG_GATE, GDR_FLAG_COUPLED = 0x40, 0x80
GDR_NORM_NONE, GDR_NORM_L2, GDR_NORM_RMS = 0, 1, 2
GDR_ROT_HALF, GDR_ROT_INTERLEAVED = 0, 1
GDR_SCAN_BLOCK = 256
GDR_DELTA_CHUNK = 64
GDR_ACT_LINEAR, GDR_ACT_SIGMOID, GDR_ACT_SILU = 0, 1, 2
PATH_MFMA, PATH_VALU = 1, 2


class Desc(ctypes.Structure):
    """Mirror of ``gdr_desc``."""

    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "T", "H", "dk", "dv", "chunk", "io_dtype", "gate_dtype", "alpha_mode",
                 "beta_mode", "flags")]


class QkDesc(ctypes.Structure):
    """Mirror of ``gdr_qk_desc``."""

    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "T", "Hq", "Hk", "d", "io_dtype", "weight_dtype", "norm", "rot_layout",
                                               "rot_dim")]
                + [(n, ctypes.c_float) for n in ("eps", "q_scale", "rot_scale")]
                + [(n, ctypes.c_int64) for n in ("ldq", "ldk")])


class DeltaDesc(ctypes.Structure):
    """Mirror of ``gdr_delta_desc``."""

    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "T", "Hk", "Hv", "dk", "dv", "io_dtype", "gate_dtype")]
                + [(n, ctypes.c_int64) for n in ("ldq", "ldk", "ldv", "ldg", "ldb")])


class BlockNormDesc(ctypes.Structure):
    """Mirror of ``gdr_block_norm_desc``."""

    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "T", "H", "d", "io_dtype", "weight_dtype", "norm", "next_norm", "act")]
                + [(n, ctypes.c_float) for n in ("eps", "scale", "res_scale")]
                + [(n, ctypes.c_int64) for n in ("ldx", "ldg", "ldr")])


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python gated_delta_rule_84_amd/build.py`")
_lib = ctypes.CDLL(LIB_PATH)
_vp = ctypes.c_void_p
_dp = ctypes.POINTER(Desc)
_lib.gdr_chunk_fwd_workspace_size.argtypes = [_dp]
_lib.gdr_chunk_fwd_workspace_size.restype = ctypes.c_size_t
_lib.gdr_chunk_fwd.argtypes = [_dp] + [_vp] * 10 + [_vp, ctypes.c_size_t, _vp]
_lib.gdr_chunk_fwd.restype = ctypes.c_int
_lib.gdr_chunk_fwd_ctx.argtypes = [_dp] + [_vp] * 10 + [_vp, ctypes.c_size_t, _vp, _vp]
_lib.gdr_chunk_fwd_ctx.restype = ctypes.c_int
_lib.gdr_chunk_fwd_noalloc.argtypes = [_dp] + [_vp] * 10 + [_vp]
_lib.gdr_chunk_fwd_noalloc.restype = ctypes.c_int
_lib.gdr_decode_step.argtypes = [_dp] + [_vp] * 9 + [_vp]
_lib.gdr_decode_step.restype = ctypes.c_int
_lib.gdr_chunk_fwd_path.argtypes = [_dp]
_lib.gdr_chunk_fwd_path.restype = ctypes.c_int
_lib.gdr_status_string.argtypes = [ctypes.c_int]
_lib.gdr_status_string.restype = ctypes.c_char_p
_lib.gdr_version.argtypes = []
_lib.gdr_version.restype = ctypes.c_int
_lib.gdr_chunk_fwd_ckpt.argtypes = [_dp] + [_vp] * 10 + [ctypes.c_int32, _vp, _vp, ctypes.c_size_t, _vp]
_lib.gdr_chunk_fwd_ckpt.restype = ctypes.c_int
_lib.gdr_mc_readout_workspace_size.argtypes = [_dp, ctypes.c_int32]
_lib.gdr_mc_readout_workspace_size.restype = ctypes.c_size_t
_lib.gdr_mc_readout.argtypes = [_dp, _vp, _vp, ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp, _vp,
                                ctypes.c_size_t, _vp]
_lib.gdr_mc_readout.restype = ctypes.c_int
_lib.gdr_osdn_precond_workspace_size.argtypes = [_dp]
_lib.gdr_osdn_precond_workspace_size.restype = ctypes.c_size_t
_lib.gdr_osdn_precond.argtypes = [_dp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp,
                                  _vp]
_lib.gdr_osdn_precond.restype = ctypes.c_int
_lib.gdr_sdm_workspace_size.argtypes = [_dp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
_lib.gdr_sdm_workspace_size.restype = ctypes.c_size_t
_lib.gdr_sdm_fwd.argtypes = [_dp] + [ctypes.c_int32] * 3 + [_vp] * 10 + [ctypes.c_size_t, _vp, _vp]
_lib.gdr_sdm_fwd.restype = ctypes.c_int
_lib.gdr_dmem_fwd.argtypes = [_dp, ctypes.c_int32] + [_vp] * 8 + [_vp]
_lib.gdr_dmem_fwd.restype = ctypes.c_int
_lib.gdr_context_create.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
_lib.gdr_context_create.restype = ctypes.c_int
_lib.gdr_context_destroy.argtypes = [_vp]
_lib.gdr_context_destroy.restype = ctypes.c_int
_qp = ctypes.POINTER(QkDesc)
_i64 = ctypes.c_int64
_lib.gdr_qk_prep_fwd.argtypes = [_qp] + [_vp] * 8 + [_vp]
_lib.gdr_qk_prep_fwd.restype = ctypes.c_int
_lib.gdr_qk_prep_bwd_workspace_size.argtypes = [_qp]
_lib.gdr_qk_prep_bwd_workspace_size.restype = ctypes.c_size_t
_lib.gdr_qk_prep_bwd.argtypes = [_qp] + [_vp] * 12 + [_vp, ctypes.c_size_t, _vp]
_lib.gdr_qk_prep_bwd.restype = ctypes.c_int
_lib.gdr_scan_workspace_size.argtypes = [_dp]
_lib.gdr_scan_workspace_size.restype = ctypes.c_size_t
_rows = [_vp, _i64] * 3  # x, alpha, beta with their strides
_lib.gdr_scan_fwd.argtypes = [_dp] + _rows + [_vp, ctypes.c_int32] + [_vp] * 4 + [_vp, ctypes.c_size_t, _vp]
_lib.gdr_scan_fwd.restype = ctypes.c_int
_lib.gdr_scan_bwd.argtypes = [_dp] + _rows + [_vp, ctypes.c_int32] + [_vp] * 8 + [_vp, ctypes.c_size_t, _vp]
_lib.gdr_scan_bwd.restype = ctypes.c_int
_lib.gdr_scan_step.argtypes = [_dp] + _rows + [_vp] * 2 + [_vp]
_lib.gdr_scan_step.restype = ctypes.c_int
_ddp = ctypes.POINTER(DeltaDesc)
_lib.gdr_delta_workspace_size.argtypes = [_ddp, ctypes.c_int32, ctypes.c_int32]
_lib.gdr_delta_workspace_size.restype = ctypes.c_size_t
_lib.gdr_delta_ckpt_size.argtypes = [_ddp, ctypes.c_int32]
_lib.gdr_delta_ckpt_size.restype = ctypes.c_size_t
_lib.gdr_delta_fwd.argtypes = [_ddp] + [_vp] * 6 + [ctypes.c_int32] + [_vp] * 4 + [_vp, ctypes.c_size_t, _vp]
_lib.gdr_delta_fwd.restype = ctypes.c_int
_lib.gdr_delta_bwd.argtypes = [_ddp] + [_vp] * 6 + [ctypes.c_int32] + [_vp] * 9 + [_vp, ctypes.c_size_t, _vp]
_lib.gdr_delta_bwd.restype = ctypes.c_int
_lib.gdr_delta_step.argtypes = [_ddp] + [_vp] * 7 + [_vp]
_lib.gdr_delta_step.restype = ctypes.c_int
_np = ctypes.POINTER(BlockNormDesc)
_lib.gdr_block_norm_fwd.argtypes = [_np] + [_vp] * 7 + [_vp]
_lib.gdr_block_norm_fwd.restype = ctypes.c_int
_lib.gdr_block_norm_bwd_workspace_size.argtypes = [_np]
_lib.gdr_block_norm_bwd_workspace_size.restype = ctypes.c_size_t
_lib.gdr_block_norm_bwd.argtypes = [_np] + [_vp] * 12 + [_vp, ctypes.c_size_t, _vp]
_lib.gdr_block_norm_bwd.restype = ctypes.c_int

EXPORTED = ("gdr_chunk_fwd_workspace_size", "gdr_chunk_fwd", "gdr_decode_step", "gdr_chunk_fwd_path",
            "gdr_status_string", "gdr_version", "gdr_chunk_fwd_ckpt", "gdr_mc_readout_workspace_size",
            "gdr_mc_readout", "gdr_osdn_precond_workspace_size", "gdr_osdn_precond",
            "gdr_sdm_workspace_size", "gdr_sdm_fwd", "gdr_context_create", "gdr_context_destroy",
            "gdr_chunk_fwd_noalloc", "gdr_dmem_fwd", "gdr_chunk_fwd_ctx", "gdr_qk_prep_fwd",
            "gdr_qk_prep_bwd_workspace_size", "gdr_qk_prep_bwd", "gdr_scan_workspace_size", "gdr_scan_fwd", "gdr_scan_bwd",
            "gdr_scan_step", "gdr_delta_workspace_size", "gdr_delta_ckpt_size", "gdr_delta_fwd", "gdr_delta_bwd", "gdr_delta_step",
            "gdr_block_norm_fwd", "gdr_block_norm_bwd_workspace_size", "gdr_block_norm_bwd")


class GdrError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {gdr_status_string(status)} ({status})")
        self.status = status


def _ptr(t: Optional[torch.Tensor]):
    """Device address of a tensor for the library, which reads every tensor as dense
    row-major device memory: a view with other strides or a host tensor is refused
    here (ValueError) instead of being read wrongly or faulting on the device."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("expected a contiguous (dense row-major) tensor")
        if not t.is_cuda:
            raise ValueError(f"expected a device tensor, got one on {t.device}")
    return t.data_ptr()


_TORCH_DTYPE = {GDR_BF16: torch.bfloat16, GDR_F32: torch.float32}


def _check_all(specs) -> None:
    """The library trusts the descriptor: every tensor handed to it must hold exactly
    the element count and dtype the descriptor implies, on the current device, else
    ValueError before the call (a short or mistyped buffer would be read or written
    past its end on the device).  `specs` is a list of (name, tensor or None, count,
    dtype); sizes and dtypes are checked for all before devices.  An object that is not
    a tensor but has data_ptr() is a raw device address: it is passed as it is, and
    the caller answers for its size."""
    here = wrong = None
    for name, t, count, dtype in specs:
        if t is None or not isinstance(t, torch.Tensor):
            continue
        if t.dtype != dtype:
            raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
        if t.numel() != count:
            raise ValueError(f"{name}: expected {count} elements for this descriptor, got {t.numel()} "
                             f"(shape {tuple(t.shape)})")
        if here is None:
            here = torch._C._cuda_getDevice() if t.is_cuda else -2  # what current_device() asks, once there is a device
        if wrong is None and t.get_device() != here:
            wrong = name, t
    if wrong is not None:
        name, t = wrong
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a device tensor, got one on {t.device}")
        raise ValueError(f"{name}: tensor on {t.device}, current device is cuda:{torch.cuda.current_device()}")


def _check_workspace(workspace, workspace_bytes: int) -> None:
    if workspace is None or not isinstance(workspace, torch.Tensor):
        return
    have = workspace.numel() * workspace.element_size()
    if int(workspace_bytes) > have:
        raise ValueError(f"workspace_bytes = {int(workspace_bytes)} exceeds the workspace tensor ({have} bytes)")


def _io(desc: Desc):
    if desc.io_dtype not in _TORCH_DTYPE or desc.gate_dtype not in _TORCH_DTYPE:
        return None, None
    return _TORCH_DTYPE[desc.io_dtype], _TORCH_DTYPE[desc.gate_dtype]


def _prefill_specs(desc: Desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST) -> list:
    io, gt = _io(desc)
    if io is None or min(desc.B, desc.T, desc.H, desc.dk, desc.dv) < 0:
        return []  # the library rejects the descriptor itself
    n = desc.B * desc.T * desc.H
    st = desc.B * desc.H * desc.dk * desc.dv
    return [("q", q, n * desc.dk, io), ("k", k, n * desc.dk, io), ("k_w", k_w, n * desc.dk, io),
            ("v", v, n * desc.dv, io), ("o", o, n * desc.dv, io),
            ("alpha", alpha, n * (desc.dk if desc.alpha_mode == GDR_ALPHA_CHANNEL else 1), gt),
            ("beta_k", beta_k, n * (desc.dk if desc.beta_mode in (GDR_BETA_SHARED, GDR_BETA_KV) else 1), gt),
            ("beta_v", beta_v, n * desc.dv, gt), ("S0", S0, st, torch.float32), ("ST", ST, st, torch.float32)]


def _stream(stream) -> int:
    if stream is None:  # the current stream's handle without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return _handle(stream)


def _handle(stream) -> int:
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ---------------------------------------------------------------------------
# the C entry points, one to one
# ---------------------------------------------------------------------------

def gdr_context_create() -> ctypes.c_void_p:
    """A caller-owned execution context (a second stream and events) on the current
    device; raises on failure.  Release it with gdr_context_destroy."""
    h = ctypes.c_void_p()
    rc = int(_lib.gdr_context_create(ctypes.byref(h)))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_context_create")
    return h


def gdr_context_destroy(ctx) -> int:
    return int(_lib.gdr_context_destroy(ctx))


class Context:
    """Owns one gdr_context; usable as a context manager.  Pass it (or its `handle`)
    as `ctx` to osdn_precond / sdm_fwd to overlap their parallel passes on the
    context's second stream."""

    def __init__(self):
        self.handle = gdr_context_create()

    def close(self):
        if self.handle is not None:
            rc = gdr_context_destroy(self.handle)
            self.handle = None
            if rc != GDR_OK:
                raise GdrError(rc, "gdr_context_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _ctx(ctx):
    if ctx is None:
        return None
    return ctx.handle if isinstance(ctx, Context) else ctx


def gdr_version() -> int:
    return int(_lib.gdr_version())


def gdr_status_string(status: int) -> str:
    return _lib.gdr_status_string(int(status)).decode()


def gdr_chunk_fwd_workspace_size(desc: Desc) -> int:
    return int(_lib.gdr_chunk_fwd_workspace_size(ctypes.byref(desc)))


def gdr_chunk_fwd_path(desc: Desc) -> int:
    return int(_lib.gdr_chunk_fwd_path(ctypes.byref(desc)))


def gdr_chunk_fwd(desc: Desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST, workspace,
                  workspace_bytes: int, stream=None) -> int:
    _check_all(_prefill_specs(desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST))
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_chunk_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(k_w), _ptr(v), _ptr(alpha),
                                  _ptr(beta_k), _ptr(beta_v), _ptr(S0), _ptr(o), _ptr(ST),
                                  _ptr(workspace), int(workspace_bytes), _stream(stream)))


def gdr_chunk_fwd_ctx(desc: Desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST, workspace,
                      workspace_bytes: int, ctx, stream=None) -> int:
    _check_all(_prefill_specs(desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST))
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_chunk_fwd_ctx(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(k_w), _ptr(v), _ptr(alpha),
                                      _ptr(beta_k), _ptr(beta_v), _ptr(S0), _ptr(o), _ptr(ST),
                                      _ptr(workspace), int(workspace_bytes), _ctx(ctx), _stream(stream)))


def gdr_chunk_fwd_noalloc(desc: Desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST, stream=None) -> int:
    _check_all(_prefill_specs(desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST))
    return int(_lib.gdr_chunk_fwd_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(k_w), _ptr(v), _ptr(alpha),
                                          _ptr(beta_k), _ptr(beta_v), _ptr(S0), _ptr(o), _ptr(ST), _stream(stream)))


def gdr_chunk_fwd_ckpt(desc: Desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST, seg_len: int, ckpt,
                       workspace, workspace_bytes: int, stream=None) -> int:
    specs = _prefill_specs(desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST)
    if specs and int(seg_len) > 0:
        specs.append(("ckpt", ckpt, desc.B * desc.H * (desc.T // int(seg_len)) * desc.dk * desc.dv, torch.float32))
    _check_all(specs)
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_chunk_fwd_ckpt(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(k_w), _ptr(v), _ptr(alpha),
                                       _ptr(beta_k), _ptr(beta_v), _ptr(S0), _ptr(o), _ptr(ST), int(seg_len),
                                       _ptr(ckpt), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def gdr_mc_readout_workspace_size(desc: Desc, n_ckpt: int) -> int:
    return int(_lib.gdr_mc_readout_workspace_size(ctypes.byref(desc), int(n_ckpt)))


def gdr_mc_readout(desc: Desc, q, ckpt, n_ckpt: int, seg_len: int, gates, o_in, o_out, workspace,
                   workspace_bytes: int, stream=None) -> int:
    io, _ = _io(desc)
    if io is not None and min(desc.B, desc.T, desc.H, desc.dk, desc.dv, int(n_ckpt)) >= 0:
        n = desc.B * desc.T * desc.H
        _check_all([("q", q, n * desc.dk, io),
                    ("ckpt", ckpt, desc.B * desc.H * int(n_ckpt) * desc.dk * desc.dv, torch.float32),
                    ("gates", gates, n * int(n_ckpt), torch.float32), ("o_in", o_in, n * desc.dv, io),
                    ("o_out", o_out, n * desc.dv, io)])
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_mc_readout(ctypes.byref(desc), _ptr(q), _ptr(ckpt), int(n_ckpt), int(seg_len),
                                   _ptr(gates), _ptr(o_in), _ptr(o_out), _ptr(workspace), int(workspace_bytes),
                                   _stream(stream)))


def gdr_osdn_precond_workspace_size(desc: Desc) -> int:
    return int(_lib.gdr_osdn_precond_workspace_size(ctypes.byref(desc)))


def gdr_osdn_precond(desc: Desc, k, beta, r, eta: float, d0, k_w, dT, qgeo, workspace, workspace_bytes: int,
                     ctx=None, stream=None) -> int:
    io, gt = _io(desc)
    if io is not None and min(desc.B, desc.T, desc.H, desc.dk) >= 0:
        n = desc.B * desc.T * desc.H
        _check_all([("k", k, n * desc.dk, io), ("k_w", k_w, n * desc.dk, io), ("beta", beta, n, gt),
                    ("r", r, n, gt), ("d0", d0, desc.B * desc.H * desc.dk, torch.float32),
                    ("dT", dT, desc.B * desc.H * desc.dk, torch.float32),
                    ("qgeo", qgeo, desc.B * desc.H, torch.float32)])
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_osdn_precond(ctypes.byref(desc), _ptr(k), _ptr(beta), _ptr(r), float(eta), _ptr(d0), _ptr(k_w),
                                     _ptr(dT), _ptr(qgeo), _ptr(workspace), int(workspace_bytes), _ctx(ctx),
                                     _stream(stream)))


def gdr_sdm_workspace_size(desc: Desc, n: int, W: int, R: int) -> int:
    return int(_lib.gdr_sdm_workspace_size(ctypes.byref(desc), int(n), int(W), int(R)))


def gdr_sdm_fwd(desc: Desc, n: int, W: int, R: int, ks, qs, v, alpha, beta, M, o, w_slots, r_slots, workspace,
                workspace_bytes: int, ctx=None, stream=None) -> int:
    io, gt = _io(desc)
    if io is not None and min(desc.B, desc.T, desc.H, desc.dv, int(n), int(W), int(R)) >= 0:
        nt = desc.B * desc.T * desc.H
        _check_all([("ks", ks, nt * 2 * int(n), torch.float32), ("qs", qs, nt * 2 * int(n), torch.float32),
                    ("v", v, nt * desc.dv, io), ("o", o, nt * desc.dv, io), ("alpha", alpha, nt, gt),
                    ("beta", beta, nt, gt), ("M", M, desc.B * desc.H * int(n) * int(n) * desc.dv, torch.float32),
                    ("w_slots", w_slots, nt * int(W), torch.int32), ("r_slots", r_slots, nt * int(R), torch.int32)])
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_sdm_fwd(ctypes.byref(desc), int(n), int(W), int(R), _ptr(ks), _ptr(qs), _ptr(v), _ptr(alpha),
                                _ptr(beta), _ptr(M), _ptr(o), _ptr(w_slots), _ptr(r_slots), _ptr(workspace),
                                int(workspace_bytes), _ctx(ctx), _stream(stream)))


def gdr_dmem_fwd(desc: Desc, J: int, q, k, v, lam, beta, seg_end, M, out, stream=None) -> int:
    io, gt = _io(desc)
    if io is not None and min(desc.B, desc.T, desc.H, desc.dk) >= 0 and int(J) >= 1 and desc.H % int(J) == 0:
        nt = desc.B * desc.T * desc.H
        _check_all([("q", q, nt * desc.dk, io), ("k", k, nt * desc.dk, io), ("v", v, nt * desc.dk, io),
                    ("lam", lam, nt, gt), ("beta", beta, nt, gt), ("seg_end", seg_end, desc.B * desc.T, torch.uint8),
                    ("M", M, desc.B * desc.H * desc.dk * desc.dk, torch.float32),
                    ("out", out, nt // int(J) * desc.dk, io)])
    return int(_lib.gdr_dmem_fwd(ctypes.byref(desc), int(J), _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(beta),
                                 _ptr(seg_end), _ptr(M), _ptr(out), _stream(stream)))


def gdr_decode_step(desc: Desc, q, k, k_w, v, alpha, beta_k, beta_v, S, o, stream=None) -> int:
    io, gt = _io(desc)
    if io is not None and min(desc.B, desc.H, desc.dk, desc.dv) >= 0:
        n = desc.B * desc.H
        _check_all([("q", q, n * desc.dk, io), ("k", k, n * desc.dk, io), ("k_w", k_w, n * desc.dk, io),
                    ("v", v, n * desc.dv, io), ("o", o, n * desc.dv, io),
                    ("alpha", alpha, n * (desc.dk if desc.alpha_mode == GDR_ALPHA_CHANNEL else 1), gt),
                    ("beta_k", beta_k, n * (desc.dk if desc.beta_mode in (GDR_BETA_SHARED, GDR_BETA_KV) else 1), gt),
                    ("beta_v", beta_v, n * desc.dv, gt), ("S", S, n * desc.dk * desc.dv, torch.float32)])
    return int(_lib.gdr_decode_step(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(k_w), _ptr(v), _ptr(alpha),
                                    _ptr(beta_k), _ptr(beta_v), _ptr(S), _ptr(o), _stream(stream)))


def _row_stride(name: str, t: torch.Tensor, inner: int) -> int:
    """Elements between successive tokens of a tensor [..., heads, channels] whose last two
    axes are dense and whose leading axes step evenly (a dense tensor, or a slice of a fused
    projection's output); ValueError for any other strides, which the library cannot read."""
    if t.is_contiguous():
        return inner
    size, stride = t.shape, t.stride()
    if size[-1] > 1 and stride[-1] != 1 or size[-2] > 1 and stride[-2] != size[-1]:
        raise ValueError(f"{name}: heads and channels must be dense, got strides {stride}")
    ld, rows = 0, 1  # rows walked so far, from the last leading axis out
    for n, s in zip(reversed(size[:-2]), reversed(stride[:-2])):
        if n > 1:
            if rows == 1:
                ld = s
            elif s != rows * ld:
                raise ValueError(f"{name}: batch and token axes must step evenly, got strides {stride}")
            rows *= n
    if rows > 1 and ld < inner:
        raise ValueError(f"{name}: overlapping tokens, got strides {stride}")
    return ld if rows > 1 else inner


def _addr(name: str, t, ld: int, inner: int):
    """Device address of a tensor of rows `ld` elements apart (0: dense)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and not (t.is_contiguous() and ld in (0, inner)) and t.numel():
        if t.dim() < 3:
            raise ValueError(f"{name}: expected heads and channels as the last two axes, got shape {tuple(t.shape)}")
        have = _row_stride(name, t, inner)
        if t.numel() > inner and have != (int(ld) or inner):
            raise ValueError(f"{name}: tokens are {have} elements apart, not {int(ld) or inner}")
    return t.data_ptr()


def _qk_kinds(desc: QkDesc):
    """(count, dtype) of q, k, the weights, positions and inv_freq; None for a descriptor that the library rejects."""
    io, wt = _TORCH_DTYPE.get(desc.io_dtype), _TORCH_DTYPE.get(desc.weight_dtype)
    B, T, Hq, Hk, d, rot = desc.B, desc.T, desc.Hq, desc.Hk, desc.d, desc.rot_dim
    if io is None or wt is None or min(B, T, Hq, Hk, d, rot) < 0:
        return None
    n = B * T
    return (n * Hq * d, io), (n * Hk * d, io), (d, wt), (n, torch.int32), (rot // 2, torch.float64)


def gdr_qk_prep_fwd(desc: QkDesc, q, k, wq, wk, positions, inv_freq, q_out, k_out, stream=None) -> int:
    kinds = _qk_kinds(desc)
    if kinds is not None:
        nq, nk, nw, npos, nf = kinds
        _check_all((("q", q) + nq, ("k", k) + nk, ("wq", wq) + nw, ("wk", wk) + nw, ("positions", positions) + npos,
                    ("inv_freq", inv_freq) + nf, ("q_out", q_out) + nq, ("k_out", k_out) + nk))
    return int(_lib.gdr_qk_prep_fwd(ctypes.byref(desc), _addr("q", q, desc.ldq, desc.Hq * desc.d),
                                    _addr("k", k, desc.ldk, desc.Hk * desc.d), _ptr(wq), _ptr(wk), _ptr(positions),
                                    _ptr(inv_freq), _ptr(q_out), _ptr(k_out), _stream(stream)))


def gdr_qk_prep_bwd_workspace_size(desc: QkDesc) -> int:
    return int(_lib.gdr_qk_prep_bwd_workspace_size(ctypes.byref(desc)))


def gdr_qk_prep_bwd(desc: QkDesc, q, k, wq, wk, positions, inv_freq, dq_out, dk_out, dq, dk, dwq, dwk, workspace,
                    workspace_bytes: int, stream=None) -> int:
    kinds = _qk_kinds(desc)
    if kinds is not None:
        nq, nk, nw, npos, nf = kinds
        dw = desc.d, torch.float32
        _check_all((("q", q) + nq, ("k", k) + nk, ("wq", wq) + nw, ("wk", wk) + nw, ("positions", positions) + npos,
                    ("inv_freq", inv_freq) + nf, ("dq_out", dq_out) + nq, ("dk_out", dk_out) + nk, ("dq", dq) + nq,
                    ("dk", dk) + nk, ("dwq", dwq) + dw, ("dwk", dwk) + dw))
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_qk_prep_bwd(ctypes.byref(desc), _addr("q", q, desc.ldq, desc.Hq * desc.d),
                                    _addr("k", k, desc.ldk, desc.Hk * desc.d), _ptr(wq), _ptr(wk), _ptr(positions),
                                    _ptr(inv_freq), _ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk),
                                    _ptr(workspace), int(workspace_bytes), _stream(stream)))


def gdr_scan_workspace_size(desc: Desc) -> int:
    return int(_lib.gdr_scan_workspace_size(ctypes.byref(desc)))


def _scan_kinds(desc: Desc, rows: int, n_seq):
    """(count, dtype) of the streams, gates, states, ckpt and offsets; n_seq None where the rows are not packed.
    None for a descriptor that the library rejects."""
    io, gt = _TORCH_DTYPE.get(desc.io_dtype), _TORCH_DTYPE.get(desc.gate_dtype)
    B, T, H, dv, n = desc.B, desc.T, desc.H, desc.dv, 0 if n_seq is None else int(n_seq)
    if io is None or gt is None or min(B, T, H, dv, n) < 0:
        return None
    D, f32 = H * dv, torch.float32
    return ((rows * D, io), (rows * D, gt), ((B if n_seq is None else n) * D, f32),
            (B * ((T + GDR_SCAN_BLOCK - 1) // GDR_SCAN_BLOCK) * D, f32), (n + 1, torch.int32))


def _scan_rows(desc: Desc, x, ldx, alpha, lda, beta, ldb):
    D = desc.H * desc.dv
    return (_addr("x", x, ldx, D), int(ldx), _addr("alpha", alpha, lda, D), int(lda), _addr("beta", beta, ldb, D), int(ldb))


def gdr_scan_fwd(desc: Desc, x, ldx: int, alpha, lda: int, beta, ldb: int, seq_off, n_seq: int, S0, y, ST, ckpt, workspace,
                 workspace_bytes: int, stream=None) -> int:
    kinds = _scan_kinds(desc, desc.B * desc.T, None if seq_off is None else n_seq)
    if kinds is not None:
        io, gate, state, blocks, offsets = kinds
        _check_all((("x", x) + io, ("alpha", alpha) + gate, ("beta", beta) + gate, ("y", y) + io, ("S0", S0) + state,
                    ("ST", ST) + state, ("ckpt", ckpt) + blocks, ("seq_off", seq_off) + offsets))
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_scan_fwd(ctypes.byref(desc), *_scan_rows(desc, x, ldx, alpha, lda, beta, ldb), _ptr(seq_off),
                                 int(n_seq), _ptr(S0), _ptr(y), _ptr(ST), _ptr(ckpt), _ptr(workspace), int(workspace_bytes),
                                 _stream(stream)))


def gdr_scan_bwd(desc: Desc, x, ldx: int, alpha, lda: int, beta, ldb: int, seq_off, n_seq: int, S0, ckpt, dy, dST, dx,
                 dalpha, dbeta, dS0, workspace, workspace_bytes: int, stream=None) -> int:
    kinds = _scan_kinds(desc, desc.B * desc.T, None if seq_off is None else n_seq)
    if kinds is not None:
        io, gate, state, blocks, offsets = kinds
        _check_all((("x", x) + io, ("alpha", alpha) + gate, ("beta", beta) + gate, ("dy", dy) + io, ("dx", dx) + io,
                    ("dalpha", dalpha) + gate, ("dbeta", dbeta) + gate, ("S0", S0) + state, ("dST", dST) + state,
                    ("dS0", dS0) + state, ("ckpt", ckpt) + blocks, ("seq_off", seq_off) + offsets))
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_scan_bwd(ctypes.byref(desc), *_scan_rows(desc, x, ldx, alpha, lda, beta, ldb), _ptr(seq_off),
                                 int(n_seq), _ptr(S0), _ptr(ckpt), _ptr(dy), _ptr(dST), _ptr(dx), _ptr(dalpha), _ptr(dbeta),
                                 _ptr(dS0), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def gdr_scan_step(desc: Desc, x, ldx: int, alpha, lda: int, beta, ldb: int, S, y, stream=None) -> int:
    kinds = _scan_kinds(desc, desc.B, None)
    if kinds is not None:
        io, gate, state = kinds[:3]
        _check_all((("x", x) + io, ("alpha", alpha) + gate, ("beta", beta) + gate, ("y", y) + io, ("S", S) + state))
    return int(_lib.gdr_scan_step(ctypes.byref(desc), *_scan_rows(desc, x, ldx, alpha, lda, beta, ldb), _ptr(S), _ptr(y),
                                  _stream(stream)))


def gdr_delta_workspace_size(desc: DeltaDesc, n_seq: int = 0, backward: bool = False) -> int:
    return int(_lib.gdr_delta_workspace_size(ctypes.byref(desc), int(n_seq), int(backward)))


def gdr_delta_ckpt_size(desc: DeltaDesc, n_seq: int = 0) -> int:
    return int(_lib.gdr_delta_ckpt_size(ctypes.byref(desc), int(n_seq)))


def _delta_kinds(desc: DeltaDesc, rows: int, n_seq, step=False):
    """(count, dtype) of q and k, v, the gates, the states, ckpt and offsets; None for a descriptor that the library
    rejects (a step ignores T)."""
    io, gt = _TORCH_DTYPE.get(desc.io_dtype), _TORCH_DTYPE.get(desc.gate_dtype)
    n = 0 if n_seq is None else int(n_seq)
    if io is None or gt is None or min(desc.B, 0 if step else desc.T, desc.Hk, desc.Hv, desc.dk, desc.dv, n) < 0:
        return None
    f32, square = torch.float32, desc.dk * desc.dv
    return ((rows * desc.Hk * desc.dk, io), (rows * desc.Hv * desc.dv, io), (rows * desc.Hv, gt),
            ((desc.B if n_seq is None else n) * desc.Hv * square, f32),
            (gdr_delta_ckpt_size(desc, n) // 4, f32), (n + 1, torch.int32))


def _addr_flat(name: str, t, ld: int, inner: int):
    """_addr of a tensor whose last axis alone is a row (gates [.., H])."""
    return _addr(name, t.unsqueeze(-1) if isinstance(t, torch.Tensor) else t, ld, inner)


def _delta_rows(desc: DeltaDesc, q, k, v, log_gate, beta):
    key, value = desc.Hk * desc.dk, desc.Hv * desc.dv
    return (_addr("q", q, desc.ldq, key), _addr("k", k, desc.ldk, key), _addr("v", v, desc.ldv, value),
            _addr_flat("log_gate", log_gate, desc.ldg, desc.Hv), _addr_flat("beta", beta, desc.ldb, desc.Hv))


def gdr_delta_fwd(desc: DeltaDesc, q, k, v, log_gate, beta, seq_off, n_seq: int, S0, o, ST, ckpt, workspace,
                  workspace_bytes: int, stream=None) -> int:
    kinds = _delta_kinds(desc, desc.B * desc.T, None if seq_off is None else n_seq)
    if kinds is not None:
        key, value, gate, state, blocks, offsets = kinds
        _check_all((("q", q) + key, ("k", k) + key, ("v", v) + value, ("log_gate", log_gate) + gate, ("beta", beta) + gate,
                    ("o", o) + value, ("S0", S0) + state, ("ST", ST) + state, ("ckpt", ckpt) + blocks,
                    ("seq_off", seq_off) + offsets))
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_delta_fwd(ctypes.byref(desc), *_delta_rows(desc, q, k, v, log_gate, beta), _ptr(seq_off), int(n_seq),
                                  _ptr(S0), _ptr(o), _ptr(ST), _ptr(ckpt), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream)))


def gdr_delta_bwd(desc: DeltaDesc, q, k, v, log_gate, beta, seq_off, n_seq: int, ckpt, d_o, dST, dq, dk, dv, dlog_gate, dbeta,
                  dS0, workspace, workspace_bytes: int, stream=None) -> int:
    kinds = _delta_kinds(desc, desc.B * desc.T, None if seq_off is None else n_seq)
    if kinds is not None:
        key, value, gate, state, blocks, offsets = kinds
        _check_all((("q", q) + key, ("k", k) + key, ("v", v) + value, ("log_gate", log_gate) + gate, ("beta", beta) + gate,
                    ("d_o", d_o) + value, ("dq", dq) + key, ("dk", dk) + key, ("dv", dv) + value,
                    ("dlog_gate", dlog_gate) + gate, ("dbeta", dbeta) + gate, ("dST", dST) + state, ("dS0", dS0) + state,
                    ("ckpt", ckpt) + blocks, ("seq_off", seq_off) + offsets))
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_delta_bwd(ctypes.byref(desc), *_delta_rows(desc, q, k, v, log_gate, beta), _ptr(seq_off), int(n_seq),
                                  _ptr(ckpt), _ptr(d_o), _ptr(dST), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlog_gate), _ptr(dbeta),
                                  _ptr(dS0), _ptr(workspace), int(workspace_bytes), _stream(stream)))


def gdr_delta_step(desc: DeltaDesc, q, k, v, log_gate, beta, S, o, stream=None) -> int:
    kinds = _delta_kinds(desc, desc.B, None, step=True)
    if kinds is not None:
        key, value, gate, state = kinds[:4]
        _check_all((("q", q) + key, ("k", k) + key, ("v", v) + value, ("log_gate", log_gate) + gate, ("beta", beta) + gate,
                    ("S", S) + state, ("o", o) + value))
    return int(_lib.gdr_delta_step(ctypes.byref(desc), *_delta_rows(desc, q, k, v, log_gate, beta), _ptr(S), _ptr(o),
                                   _stream(stream)))


def _norm_kinds(desc: BlockNormDesc):
    """(count, dtype) of the rows, the weights and their gradients; None for a descriptor that the library rejects."""
    io, wt = _TORCH_DTYPE.get(desc.io_dtype), _TORCH_DTYPE.get(desc.weight_dtype)
    if io is None or wt is None or min(desc.B, desc.T, desc.H, desc.d) < 0:
        return None
    return (desc.B * desc.T * desc.H * desc.d, io), (desc.d, wt), (desc.d, torch.float32)


def _norm_rows(desc: BlockNormDesc, x, gate, residual):
    D = desc.H * desc.d
    return _addr("x", x, desc.ldx, D), _addr("gate", gate, desc.ldg, D), _addr("residual", residual, desc.ldr, D)


def gdr_block_norm_fwd(desc: BlockNormDesc, x, gate, residual, w, w_next, y, n, stream=None) -> int:
    kinds = _norm_kinds(desc)
    if kinds is not None:
        io, wt, _ = kinds
        _check_all((("x", x) + io, ("gate", gate) + io, ("residual", residual) + io, ("w", w) + wt, ("w_next", w_next) + wt,
                    ("y", y) + io, ("n", n) + io))
    return int(_lib.gdr_block_norm_fwd(ctypes.byref(desc), *_norm_rows(desc, x, gate, residual), _ptr(w), _ptr(w_next), _ptr(y),
                                       _ptr(n), _stream(stream)))


def gdr_block_norm_bwd_workspace_size(desc: BlockNormDesc) -> int:
    return int(_lib.gdr_block_norm_bwd_workspace_size(ctypes.byref(desc)))


def gdr_block_norm_bwd(desc: BlockNormDesc, x, gate, residual, w, w_next, dy, dn, dx, dgate, dresidual, dw, dw_next, workspace,
                       workspace_bytes: int, stream=None) -> int:
    kinds = _norm_kinds(desc)
    if kinds is not None:
        io, wt, sums = kinds
        _check_all((("x", x) + io, ("gate", gate) + io, ("residual", residual) + io, ("w", w) + wt, ("w_next", w_next) + wt,
                    ("dy", dy) + io, ("dn", dn) + io, ("dx", dx) + io, ("dgate", dgate) + io, ("dresidual", dresidual) + io,
                    ("dw", dw) + sums, ("dw_next", dw_next) + sums))
    _check_workspace(workspace, workspace_bytes)
    return int(_lib.gdr_block_norm_bwd(ctypes.byref(desc), *_norm_rows(desc, x, gate, residual), _ptr(w), _ptr(w_next), _ptr(dy),
                                       _ptr(dn), _ptr(dx), _ptr(dgate), _ptr(dresidual), _ptr(dw), _ptr(dw_next),
                                       _ptr(workspace), int(workspace_bytes), _stream(stream)))


# ---------------------------------------------------------------------------
# convenience wrappers (allocate outputs, raise on error)
# ---------------------------------------------------------------------------

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDR_BF16
    if t.dtype == torch.float32:
        return GDR_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _tensors(values):
    for t in values:
        if isinstance(t, torch.Tensor):
            if t.is_cuda:
                yield t
        elif isinstance(t, (tuple, list)):
            yield from _tensors(t)


def _on_its_stream(call):
    """A wrapper called with a `stream` that is not torch's current one runs with it as the current one.  What
    it allocates then comes from that stream's memory (a block of the current stream's may still be in use by
    work pending there), and neither what it returns nor what it was given is handed to other work, once
    dropped, before both streams are done with it.  Waiting for the inputs, and for the results, is the caller's."""
    @functools.wraps(call)
    def run(*args, **kw):
        stream = kw.get("stream")
        if stream is None or not torch.cuda.is_initialized():  # without a device the call refuses its tensors
            return call(*args, **kw)
        handle = _handle(stream)
        if handle == torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()):
            return call(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
        here = torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            out = call(*args, **dict(kw, stream=stream))
        for t in _tensors((args, tuple(kw.values()))):
            t.record_stream(stream)
        for t in _tensors((out,)):
            t.record_stream(here)
        return out
    return run


def make_desc(q, v, alpha, beta_k, beta_v=None, *, chunk=64, decode=False, flags=0) -> Desc:
    """Descriptor from tensor shapes: prefill q [B, T, H, dk], decode q [B, H, dk]."""
    if decode:
        B, H, dk = q.shape
        T = 1
        alpha_ch = alpha.dim() == 3
        beta_vec = beta_k.dim() == 3
    else:
        B, T, H, dk = q.shape
        alpha_ch = alpha.dim() == 4
        beta_vec = beta_k.dim() == 4
    beta_mode = GDR_BETA_KV if beta_v is not None else (GDR_BETA_SHARED if beta_vec else GDR_BETA_SCALAR)
    return Desc(B=B, T=T, H=H, dk=dk, dv=v.shape[-1], chunk=chunk, io_dtype=_dtype_code(q),
                gate_dtype=_dtype_code(alpha), alpha_mode=GDR_ALPHA_CHANNEL if alpha_ch else GDR_ALPHA_SCALAR,
                beta_mode=beta_mode, flags=flags)


@_on_its_stream
def chunk_fwd(q, k, v, alpha, beta_k, *, k_w=None, beta_v=None, S0=None, chunk=64, want_state=True,
              out=None, final_state=None, workspace=None, ctx=None, stream=None):
    """Prefill.  Returns (o [B, T, H, dv] in q's dtype, ST [B, H, dk, dv] fp32 or None).
    With an execution context `ctx` the call goes through gdr_chunk_fwd_ctx."""
    desc = make_desc(q, v, alpha, beta_k, beta_v, chunk=chunk)
    o = out if out is not None else torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    ST = final_state
    if ST is None and want_state:
        ST = torch.empty((desc.B, desc.H, desc.dk, desc.dv), dtype=torch.float32, device=q.device)
    need = gdr_chunk_fwd_workspace_size(desc)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if ctx is None:
        rc = gdr_chunk_fwd(desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST, workspace, wbytes, stream)
    else:
        rc = gdr_chunk_fwd_ctx(desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST, workspace, wbytes, ctx, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_chunk_fwd" if ctx is None else "gdr_chunk_fwd_ctx")
    return o, ST


@_on_its_stream
def chunk_fwd_ckpt(q, k, v, alpha, beta_k, seg_len, *, k_w=None, beta_v=None, S0=None, chunk=64,
                   want_state=True, workspace=None, stream=None):
    """Prefill that also keeps the state after every complete segment of seg_len tokens.
    Returns (o, ST or None, ckpt [B, H, floor(T / seg_len), dk, dv] fp32)."""
    desc = make_desc(q, v, alpha, beta_k, beta_v, chunk=chunk)
    o = torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    ST = torch.empty((desc.B, desc.H, desc.dk, desc.dv), dtype=torch.float32, device=q.device) if want_state else None
    n = desc.T // int(seg_len) if seg_len > 0 else 0
    ckpt = torch.empty((desc.B, desc.H, n, desc.dk, desc.dv), dtype=torch.float32, device=q.device)
    need = gdr_chunk_fwd_workspace_size(desc)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = gdr_chunk_fwd_ckpt(desc, q, k, k_w, v, alpha, beta_k, beta_v, S0, o, ST, seg_len,
                            ckpt if n > 0 else None, workspace, wbytes, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_chunk_fwd_ckpt")
    return o, ST, ckpt


@_on_its_stream
def mc_readout(q, ckpt, seg_len, *, gates=None, o_in=None, out=None, workspace=None, stream=None):
    """o_out[t] = o_in[t] + sum_{s < min(t // seg_len, N)} g[t, s] M_s^T q[t] (g = 1 without gates).
    q [B, T, H, 128] bf16, ckpt [B, H, N, 128, 128] fp32, gates [B, T, H, N] fp32 or None."""
    B, T, H, dk = q.shape
    n = ckpt.shape[2]
    desc = Desc(B=B, T=T, H=H, dk=dk, dv=ckpt.shape[-1], chunk=64, io_dtype=_dtype_code(q), gate_dtype=GDR_F32,
                alpha_mode=0, beta_mode=0, flags=0)
    o = out if out is not None else torch.empty(q.shape[:-1] + (ckpt.shape[-1],), dtype=q.dtype, device=q.device)
    need = gdr_mc_readout_workspace_size(desc, n)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = gdr_mc_readout(desc, q, ckpt, n, seg_len, gates, o_in, o, workspace, wbytes, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_mc_readout")
    return o


@_on_its_stream
def osdn_precond(k, beta, eta, *, r=None, d0=None, workspace=None, ctx=None, stream=None):
    """OSDN phase 1.  k [B, T, H, dk] (bf16 or fp32), beta and r [B, T, H].
    Returns (k_w like k, dT [B, H, dk] fp32, qgeo [B, H] fp32)."""
    B, T, H, dk = k.shape
    desc = Desc(B=B, T=T, H=H, dk=dk, dv=dk, chunk=64, io_dtype=_dtype_code(k), gate_dtype=_dtype_code(beta),
                alpha_mode=0, beta_mode=0, flags=0)
    kw = torch.empty_like(k)
    dT = torch.empty((B, H, dk), dtype=torch.float32, device=k.device)
    qg = torch.empty((B, H), dtype=torch.float32, device=k.device)
    need = gdr_osdn_precond_workspace_size(desc)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=k.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = gdr_osdn_precond(desc, k, beta, r, eta, d0, kw, dT, qg, workspace, wbytes, ctx, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_osdn_precond")
    return kw, dT, qg


@_on_its_stream
def sdm_fwd(M, ks, qs, v, alpha, beta, W, R, *, want_slots=False, workspace=None, ctx=None, stream=None):
    """Sparse Delta Memory over T tokens.  M [B, H, n * n, dv] fp32 is updated in place;
    ks, qs [B, T, H, 2, n] fp32; v [B, T, H, dv].  Returns o (and the selected write /
    read slots when want_slots)."""
    B, T, H, _, n = ks.shape
    dv = v.shape[-1]
    desc = Desc(B=B, T=T, H=H, dk=dv, dv=dv, chunk=64, io_dtype=_dtype_code(v), gate_dtype=_dtype_code(alpha),
                alpha_mode=0, beta_mode=0, flags=0)
    o = torch.empty_like(v)
    ws_ = ((torch.empty((B, T, H, W), dtype=torch.int32, device=v.device),
            torch.empty((B, T, H, R), dtype=torch.int32, device=v.device)) if want_slots else (None, None))
    need = gdr_sdm_workspace_size(desc, n, W, R)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=v.device)
    rc = gdr_sdm_fwd(desc, n, W, R, ks, qs, v, alpha, beta, M, o, ws_[0], ws_[1], workspace,
                     workspace.numel() * workspace.element_size(), ctx, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_sdm_fwd")
    return (o, ws_[0], ws_[1]) if want_slots else o


@_on_its_stream
def dmem_fwd(M, q, k, v, lam, beta, *, seg_end=None, J=1, out=None, stream=None):
    """delta-mem context pass: M [B, H, r, r] fp32 is updated in place; q, k, v
    [B, T, H, r]; lam, beta [B, T, H]; seg_end [B, T] uint8 or None (one write per
    token).  Returns the reads [B, T, H // J, r] (J sub-states per group, reads summed)."""
    B, T, H, r = q.shape
    desc = Desc(B=B, T=T, H=H, dk=r, dv=r, chunk=64, io_dtype=_dtype_code(q), gate_dtype=_dtype_code(lam),
                alpha_mode=0, beta_mode=0, flags=0)
    o = out if out is not None else torch.empty((B, T, H // J, r), dtype=q.dtype, device=q.device)
    rc = gdr_dmem_fwd(desc, J, q, k, v, lam, beta, seg_end, M, o, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_dmem_fwd")
    return o


@_on_its_stream
def decode_step(S, q, k, v, alpha, beta_k, *, k_w=None, beta_v=None, out=None, flags=0, stream=None):
    """One token for every (b, h); S [B, H, dk, dv] fp32 is updated in place.  Returns o [B, H, dv].
    `flags`: GDR_FLAG_READ_BEFORE_WRITE and / or GDR_FLAG_UNDECAYED_PREDICTION."""
    desc = make_desc(q, v, alpha, beta_k, beta_v, decode=True, flags=flags)
    o = out if out is not None else torch.empty(q.shape[:-1] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    rc = gdr_decode_step(desc, q, k, k_w, v, alpha, beta_k, beta_v, S, o, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_decode_step")
    return o


def rope_inv_freq(rot_dim, *, base=10000.0, scaling=None, factor=1.0, original_len=None, fast=32.0, slow=1.0, device="cuda"):
    """Frequencies of the rotation, ``inv_freq`` [rot_dim / 2] fp64, and ``rot_scale``, for qk_prep.

    Plain: f_i = base^(-2 i / rot_dim), scale 1.  For contexts `factor` times longer than the
    `original_len` tokens that a model was trained on, `scaling`:
      "linear"  every frequency divided by the factor (positions interpolated);
      "ntk"     the base raised by factor^(rot_dim / (rot_dim - 2)), which divides the lowest frequency by the
                factor and leaves the highest as it is;
      "yarn"    by wavelength (the YaRN paper, Peng et al., 2023): frequencies that turn more than `fast` times
                over original_len stay, those that turn less than `slow` times are divided by the factor, those
                between are mixed linearly in the channel's index; scale 0.1 ln(factor) + 1.
    """
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and not negative, got {rot_dim}")
    if not base > 0 or not factor >= 1:
        raise ValueError(f"base must be positive and factor at least 1, got {base} and {factor}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f, scale = base ** (-2.0 * i / max(rot_dim, 1)), 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if original_len is None or not original_len > 0 or not fast > slow > 0 or not base > 1:
            raise ValueError("yarn needs original_len > 0, fast > slow > 0 and base > 1")
        # the (real) channel index whose frequency turns n times over original_len
        at = lambda n: rot_dim * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot_dim - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1) if hi > 0 else torch.ones_like(i)
        f, scale = f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f.to(device), scale


_NORMS = {None: GDR_NORM_NONE, "none": GDR_NORM_NONE, "l2": GDR_NORM_L2, "rms": GDR_NORM_RMS}
_LAYOUTS = {"half": GDR_ROT_HALF, "interleaved": GDR_ROT_INTERLEAVED}


def _qk_desc(q, k, norm, wq, wk, eps, inv_freq, layout, rot_scale, q_scale) -> QkDesc:
    if norm not in _NORMS:
        raise ValueError(f"norm must be None, 'none', 'l2' or 'rms', got {norm!r}")
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    qs, ks = tuple(q.shape), tuple(k.shape)
    if len(qs) != 4 or len(ks) != 4 or qs[:2] != ks[:2] or qs[3] != ks[3] or q.dtype != k.dtype:
        raise ValueError(f"expected q [B, T, Hq, d] and k [B, T, Hk, d] of one type, got {tuple(q.shape)} {q.dtype} and "
                         f"{tuple(k.shape)} {k.dtype}")
    if wq is not None and wk is not None and wq.dtype != wk.dtype:
        raise ValueError(f"wq and wk must have one type, got {wq.dtype} and {wk.dtype}")
    (B, T, Hq, d), Hk = qs, ks[2]
    w = wq if wq is not None else wk
    return QkDesc(B, T, Hq, Hk, d, _dtype_code(q), GDR_F32 if w is None else _dtype_code(w), _NORMS[norm], _LAYOUTS[layout],
                  0 if inv_freq is None else 2 * inv_freq.numel(), eps, q_scale, rot_scale,
                  0 if q.is_contiguous() else _row_stride("q", q, Hq * d), 0 if k.is_contiguous() else _row_stride("k", k, Hk * d))


@_on_its_stream
def qk_prep(q, k, *, norm="rms", wq=None, wk=None, eps=1e-6, positions=None, inv_freq=None, layout="half", rot_scale=1.0,
            q_scale=1.0, out=None, stream=None):
    """Norm of every head of q [B, T, Hq, d] and k [B, T, Hk, d] and the rotation by position, in one pass.

    norm None, "l2" or "rms" with optional weights wq, wk [d]; inv_freq [rot_dim / 2] fp64 (rope_inv_freq) rotates the
    first rot_dim channels by positions [B, T] int32 (default 0 .. T - 1), in the "half" or "interleaved" layout, times
    rot_scale; q is multiplied by q_scale.  q and k may be slices of a fused projection's output.  Returns (q, k), dense;
    `out` a pair of tensors to write instead (q, k themselves where dense)."""
    desc = _qk_desc(q, k, norm, wq, wk, eps, inv_freq, layout, rot_scale, q_scale)
    qo, ko = out if out is not None else (q.new_empty(q.shape), k.new_empty(k.shape))
    rc = gdr_qk_prep_fwd(desc, q, k, wq, wk, positions, inv_freq, qo, ko, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_qk_prep_fwd")
    return qo, ko


@_on_its_stream
def qk_prep_bwd(q, k, dq_out, dk_out, *, norm="rms", wq=None, wk=None, eps=1e-6, positions=None, inv_freq=None,
                layout="half", rot_scale=1.0, q_scale=1.0, workspace=None, stream=None):
    """Backward pass of qk_prep, from its inputs and the (dense) gradients of its outputs.
    Returns (dq, dk, dwq, dwk): dense gradients in q's type, weight gradients [d] in fp32 or None."""
    desc = _qk_desc(q, k, norm, wq, wk, eps, inv_freq, layout, rot_scale, q_scale)
    dq, dk = q.new_empty(q.shape), k.new_empty(k.shape)
    dwq, dwk = (None if w is None else w.new_empty(w.shape, dtype=torch.float32) for w in (wq, wk))
    if dwq is not None or dwk is not None:
        workspace = _room(workspace, gdr_qk_prep_bwd_workspace_size(desc), q.device)
    rc = gdr_qk_prep_bwd(desc, q, k, wq, wk, positions, inv_freq, dq_out, dk_out, dq, dk, dwq, dwk, workspace,
                         _nbytes(workspace), stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_qk_prep_bwd")
    return dq, dk, dwq, dwk


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _room(workspace, need: int, device):
    """`workspace` where it holds `need` bytes, else a new one (None for 0)."""
    if need and _nbytes(workspace) < need:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    return workspace


def _scan_desc(x, alpha, log_gate, coupled, step=False) -> Desc:
    shape = tuple(x.shape)
    if len(shape) != (3 if step else 4) or tuple(alpha.shape) != shape:
        raise ValueError(f"expected x and alpha [B, {'' if step else 'T, '}H, dv], got {tuple(x.shape)} and {tuple(alpha.shape)}")
    H, dv = shape[-2:]
    flags = (GDR_FLAG_LOG_GATE if log_gate else 0) | (GDR_FLAG_COUPLED if coupled else 0)
    return Desc(shape[0], 1 if step else shape[1], H, 1, dv, 64, _dtype_code(x), _dtype_code(alpha), GDR_ALPHA_CHANNEL, 0,
                flags)


def _strides(desc: Desc, x, alpha, beta):
    D = desc.H * desc.dv
    return (0 if x.is_contiguous() else _row_stride("x", x, D), 0 if alpha.is_contiguous() else _row_stride("alpha", alpha, D),
            0 if beta is None or beta.is_contiguous() else _row_stride("beta", beta, D))


@_on_its_stream
def scan_fwd(x, alpha, *, beta=None, log_gate=False, coupled=False, S0=None, seq_offsets=None, want_state=True,
             want_ckpt=False, workspace=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + b_t x_t over x [B, T, H, dv], y = h.

    a = alpha [B, T, H, dv] (or exp(alpha) with log_gate); b = beta where given, 1 - a with coupled, else 1.
    seq_offsets [n + 1] int32 cuts the T rows of a B = 1 batch into packed sequences; S0 [B or n, H, dv] fp32.
    Returns (y like x, ST like S0 or None, ckpt [B, ceil(T / 256), H, dv] fp32 for scan_bwd or None).  Rows of y that
    belong to no packed sequence are left unwritten."""
    desc = _scan_desc(x, alpha, log_gate, coupled)
    n_seq = 0 if seq_offsets is None else max(seq_offsets.numel() - 1, 0)
    H, dv, dev = desc.H, desc.dv, x.device
    y = x.new_empty(x.shape)
    ST = x.new_empty((desc.B if seq_offsets is None else n_seq, H, dv), dtype=torch.float32) if want_state else None
    ckpt = (x.new_empty((desc.B, (desc.T + GDR_SCAN_BLOCK - 1) // GDR_SCAN_BLOCK, H, dv), dtype=torch.float32)
            if want_ckpt else None)
    workspace = _room(workspace, gdr_scan_workspace_size(desc), dev)
    ldx, lda, ldb = _strides(desc, x, alpha, beta)
    rc = gdr_scan_fwd(desc, x, ldx, alpha, lda, beta, ldb, seq_offsets, n_seq, S0, y, ST, ckpt, workspace, _nbytes(workspace),
                      stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_scan_fwd")
    return y, ST, ckpt


@_on_its_stream
def scan_bwd(x, alpha, dy, ckpt, *, beta=None, log_gate=False, coupled=False, S0=None, dST=None, seq_offsets=None,
             workspace=None, stream=None):
    """Backward pass of scan_fwd with its inputs and its ckpt (None where T <= 256): gradients dy of y (dense) and
    dST of ST.  Returns (dx, dalpha, dbeta or None, dS0): dalpha is the gradient of alpha as stored.  Rows that belong to no
    packed sequence are left unwritten."""
    desc = _scan_desc(x, alpha, log_gate, coupled)
    n_seq = 0 if seq_offsets is None else max(seq_offsets.numel() - 1, 0)
    dev = x.device
    dx, dalpha = x.new_empty(x.shape), alpha.new_empty(x.shape)
    dbeta = None if beta is None else alpha.new_empty(x.shape)
    dS0 = x.new_empty((desc.B if seq_offsets is None else n_seq, desc.H, desc.dv), dtype=torch.float32)
    workspace = _room(workspace, gdr_scan_workspace_size(desc), dev)
    ldx, lda, ldb = _strides(desc, x, alpha, beta)
    rc = gdr_scan_bwd(desc, x, ldx, alpha, lda, beta, ldb, seq_offsets, n_seq, S0, ckpt, dy, dST, dx, dalpha, dbeta, dS0,
                      workspace, _nbytes(workspace), stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_scan_bwd")
    return dx, dalpha, dbeta, dS0


@_on_its_stream
def scan_step(S, x, alpha, *, beta=None, log_gate=False, coupled=False, out=None, stream=None):
    """One token of the recurrence for every sequence: x, alpha, beta [B, H, dv]; S [B, H, dv] fp32 is updated in
    place.  Returns y [B, H, dv]."""
    desc = _scan_desc(x, alpha, log_gate, coupled, step=True)
    y = out if out is not None else x.new_empty(x.shape)
    ldx, lda, ldb = _strides(desc, x, alpha, beta)
    rc = gdr_scan_step(desc, x, ldx, alpha, lda, beta, ldb, S, y, stream)
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_scan_step")
    return y


def _ld(name, t, inner) -> int:
    return 0 if t is None or t.is_contiguous() else _row_stride(name, t, inner)


def _ld_flat(name, t) -> int:
    """_ld of a tensor [.., heads] whose last axis alone is a row."""
    return 0 if t.is_contiguous() else _row_stride(name, t.unsqueeze(-1), t.shape[-1])


def _addresses(**tensors):
    """Device addresses of tensors whose types, shapes and strides the caller has checked; ValueError for one that is
    not on the current device."""
    found = []
    here = None
    for name, t in tensors.items():
        if t is None:
            found.append(None)
            continue
        at = t.get_device()
        if at != here:
            if at < 0:
                raise ValueError(f"{name}: expected a device tensor, got one on {t.device}")
            if here is None:
                here = torch._C._cuda_getDevice()
            if at != here:
                raise ValueError(f"{name}: tensor on {t.device}, current device is cuda:{here}")
        found.append(t.data_ptr())
    return found


def _dense(name, t, shape, dtype):
    """ValueError unless t, where there is one, is a dense tensor of that shape and type."""
    if t is not None and (t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous tensor {shape} of {dtype}, got {tuple(t.shape)} of {t.dtype}")


def _delta_desc(q, k, v, log_gate, beta, step=False) -> DeltaDesc:
    lead = 1 if step else 2
    qs, vs, gs = q.shape, v.shape, log_gate.shape
    if (len(qs) != lead + 2 or k.shape != qs or len(vs) != lead + 2 or vs[:lead] != qs[:lead] or gs != vs[:-1]
            or beta.shape != gs):
        T = "" if step else "T, "
        raise ValueError(f"expected q, k [B, {T}Hk, dk], v [B, {T}Hv, dv] and log_gate, beta [B, {T}Hv], got {tuple(qs)}, "
                         f"{tuple(k.shape)}, {tuple(vs)}, {tuple(gs)} and {tuple(beta.shape)}")
    if k.dtype != q.dtype or v.dtype != q.dtype or log_gate.dtype != beta.dtype:
        raise ValueError(f"q, k and v must have one type, and log_gate and beta, got {q.dtype}, {k.dtype}, {v.dtype}, "
                         f"{log_gate.dtype} and {beta.dtype}")
    Hk, dk, Hv, dv = qs[-2], qs[-1], vs[-2], vs[-1]
    return DeltaDesc(qs[0], 1 if step else qs[1], Hk, Hv, dk, dv, _dtype_code(q), _dtype_code(log_gate), _ld("q", q, Hk * dk),
                     _ld("k", k, Hk * dk), _ld("v", v, Hv * dv), _ld_flat("log_gate", log_gate), _ld_flat("beta", beta))


def _packed(seq_offsets, desc):
    """Sequences of a call (None where its rows are not packed) and the shape of its states."""
    if seq_offsets is None:
        return None, (desc.B, desc.Hv, desc.dk, desc.dv)
    n = seq_offsets.numel() - 1
    if n < 0 or seq_offsets.dtype != torch.int32 or not seq_offsets.is_contiguous():
        raise ValueError(f"seq_offsets: expected a contiguous tensor [n + 1] of int32, got {tuple(seq_offsets.shape)} of "
                         f"{seq_offsets.dtype}")
    return n, (n, desc.Hv, desc.dk, desc.dv)


@_on_its_stream
def delta_fwd(q, k, v, log_gate, beta, *, S0=None, seq_offsets=None, want_state=True, want_ckpt=False, workspace=None,
              stream=None):
    """Trainable delta rule S = a S + beta k (v - a S^T k)^T, o = S^T q with a = exp(log_gate).  States have fp32's
    precision whatever the types; factors that only a bf16 o reads are cut to 16 bits.

    q, k [B, T, Hk, dk], v [B, T, Hv, dv], log_gate, beta [B, T, Hv], Hv a multiple of Hk; all may be slices of a fused
    projection's output.  seq_offsets [n + 1] int32 cuts the T rows of a B = 1 batch into packed sequences; S0
    [B or n, Hv, dk, dv] fp32.  Returns (o like v, ST like S0 or None, ckpt, a flat fp32 tensor for delta_bwd, or None).
    Rows of o that belong to no packed sequence are left unwritten."""
    desc = _delta_desc(q, k, v, log_gate, beta)
    n, states = _packed(seq_offsets, desc)
    f32 = torch.float32
    _dense("S0", S0, states, f32)
    o = v.new_empty(v.shape)
    ST = v.new_empty(states, dtype=f32) if want_state else None
    ckpt = v.new_empty(gdr_delta_ckpt_size(desc, n or 0) // 4, dtype=f32) if want_ckpt else None
    workspace = _room(workspace, gdr_delta_workspace_size(desc, n or 0), v.device)
    a = _addresses(q=q, k=k, v=v, log_gate=log_gate, beta=beta, seq_offsets=seq_offsets, S0=S0, o=o, ST=ST, ckpt=ckpt,
                   workspace=workspace)
    rc = _lib.gdr_delta_fwd(ctypes.byref(desc), *a[:6], n or 0, *a[6:], _nbytes(workspace), _stream(stream))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_delta_fwd")
    return o, ST, ckpt


@_on_its_stream
def delta_bwd(q, k, v, log_gate, beta, d_o, ckpt, *, dST=None, seq_offsets=None, want_dS0=True, workspace=None, stream=None):
    """Backward pass of delta_fwd with its inputs and its ckpt: gradients d_o of o (dense) and dST of ST.
    Returns (dq, dk, dv, dlog_gate, dbeta, dS0 or None), dense, in their inputs' types; dS0 fp32.  Gradients of rows that
    belong to no packed sequence are 0."""
    desc = _delta_desc(q, k, v, log_gate, beta)
    n, states = _packed(seq_offsets, desc)
    f32 = torch.float32
    _dense("d_o", d_o, tuple(v.shape), v.dtype)
    _dense("dST", dST, states, f32)
    _dense("ckpt", ckpt, (gdr_delta_ckpt_size(desc, n or 0) // 4,), f32)
    # the library leaves rows of no packed sequence as they are; which ones there are only the device knows
    dq, dk, dv, dg, db = (t.new_empty(t.shape) if n is None else t.new_zeros(t.shape) for t in (q, k, v, log_gate, beta))
    dS0 = v.new_empty(states, dtype=f32) if want_dS0 else None
    workspace = _room(workspace, gdr_delta_workspace_size(desc, n or 0, True), v.device)
    a = _addresses(q=q, k=k, v=v, log_gate=log_gate, beta=beta, seq_offsets=seq_offsets, ckpt=ckpt, d_o=d_o, dST=dST, dq=dq, dk=dk,
                   dv=dv, dlog_gate=dg, dbeta=db, dS0=dS0, workspace=workspace)
    rc = _lib.gdr_delta_bwd(ctypes.byref(desc), *a[:6], n or 0, *a[6:], _nbytes(workspace), _stream(stream))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_delta_bwd")
    return dq, dk, dv, dg, db, dS0


@_on_its_stream
def delta_step(S, q, k, v, log_gate, beta, *, out=None, stream=None):
    """One token of the delta rule for every sequence: q, k [B, Hk, dk], v [B, Hv, dv], log_gate, beta [B, Hv]; S
    [B, Hv, dk, dv] fp32 is updated in place.  Returns o [B, Hv, dv]."""
    desc = _delta_desc(q, k, v, log_gate, beta, step=True)
    _dense("S", S, (desc.B, desc.Hv, desc.dk, desc.dv), torch.float32)
    _dense("out", out, tuple(v.shape), v.dtype)
    o = out if out is not None else v.new_empty(v.shape)
    a = _addresses(q=q, k=k, v=v, log_gate=log_gate, beta=beta, S=S, o=o)
    rc = _lib.gdr_delta_step(ctypes.byref(desc), *a, _stream(stream))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_delta_step")
    return o


_ACTS = {"none": None, None: None, "linear": GDR_ACT_LINEAR, "sigmoid": GDR_ACT_SIGMOID, "silu": GDR_ACT_SILU}


def _norm_desc(x, norm, weight, gate, act, scale, residual, res_scale, eps, next_norm, next_weight) -> BlockNormDesc:
    if norm not in _NORMS or next_norm not in _NORMS:
        raise ValueError(f"norm and next_norm must be None, 'none', 'l2' or 'rms', got {norm!r} and {next_norm!r}")
    if act not in _ACTS:
        raise ValueError(f"act must be None, 'none', 'linear', 'sigmoid' or 'silu', got {act!r}")
    if (gate is None) != (_ACTS[act] is None):
        raise ValueError(f"a gate needs an act, and an act a gate, got act {act!r}")
    shape = x.shape
    if len(shape) != 4:
        raise ValueError(f"expected x [B, T, H, d], got {tuple(shape)}")
    for name, t in (("gate", gate), ("residual", residual)):
        if t is not None and (t.shape != shape or t.dtype != x.dtype):
            raise ValueError(f"{name}: expected {tuple(shape)} {x.dtype} like x, got {tuple(t.shape)} {t.dtype}")
    for name, t in (("weight", weight), ("next_weight", next_weight)):
        if t is not None and (t.numel() != shape[-1] or not t.is_contiguous()):
            raise ValueError(f"{name}: expected a contiguous tensor [{shape[-1]}], got {tuple(t.shape)}")
    if weight is not None and next_weight is not None and weight.dtype != next_weight.dtype:
        raise ValueError(f"weight and next_weight must have one type, got {weight.dtype} and {next_weight.dtype}")
    B, T, H, d = shape
    w = weight if weight is not None else next_weight
    return BlockNormDesc(B, T, H, d, _dtype_code(x), GDR_F32 if w is None else _dtype_code(w), _NORMS[norm], _NORMS[next_norm],
                         _ACTS[act] or 0, eps, scale, res_scale, _ld("x", x, H * d), _ld("gate", gate, H * d),
                         _ld("residual", residual, H * d))


@_on_its_stream
def block_norm(x, *, norm="rms", weight=None, gate=None, act=None, scale=1.0, residual=None, res_scale=1.0, eps=1e-6,
               next_norm=None, next_weight=None, out=None, stream=None):
    """Norm behind a block with its gate and the scaled residual, and the norm in front of the next block, in one pass:

        y = res_scale * residual + scale * act(gate) * weight * norm(x),   n = next_weight * next_norm(y)

    over the d channels of every row of x [B, T, H, d] (the heads of the delta rule's output, or H = 1 for whole rows).
    norm and next_norm None, "l2" or "rms"; act of the gate "linear", "sigmoid" or "silu"; gate and residual like x, slices of
    a fused projection's output allowed; weights [d].  Returns (y, n or None), dense; `out` a tensor to write y to (the
    residual itself where dense)."""
    desc = _norm_desc(x, norm, weight, gate, act, scale, residual, res_scale, eps, next_norm, next_weight)
    y = out if out is not None else x.new_empty(x.shape)
    n = x.new_empty(x.shape) if desc.next_norm else None
    _dense("out", out, tuple(x.shape), x.dtype)
    a = _addresses(x=x, gate=gate, residual=residual, weight=weight, next_weight=next_weight, y=y, n=n)
    rc = _lib.gdr_block_norm_fwd(ctypes.byref(desc), *a, _stream(stream))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_block_norm_fwd")
    return y, n


@_on_its_stream
def block_norm_bwd(x, dy, *, dn=None, norm="rms", weight=None, gate=None, act=None, scale=1.0, residual=None, res_scale=1.0,
                   eps=1e-6, next_norm=None, next_weight=None, workspace=None, stream=None):
    """Backward pass of block_norm, from its inputs and the (dense) gradients dy of y and dn of n.
    Returns (dx, dgate, dresidual, dweight, dnext_weight): dense gradients in x's type, weight gradients [d] in fp32,
    None for what was not given."""
    desc = _norm_desc(x, norm, weight, gate, act, scale, residual, res_scale, eps, next_norm, next_weight)
    dx = x.new_empty(x.shape)
    dgate, dres = (None if t is None else x.new_empty(x.shape) for t in (gate, residual))
    dw, dw_next = (None if w is None else w.new_empty(w.shape, dtype=torch.float32) for w in (weight, next_weight))
    if dw is not None or dw_next is not None:
        workspace = _room(workspace, gdr_block_norm_bwd_workspace_size(desc), x.device)
    _dense("dy", dy, tuple(x.shape), x.dtype)
    _dense("dn", dn, tuple(x.shape), x.dtype)
    a = _addresses(x=x, gate=gate, residual=residual, weight=weight, next_weight=next_weight, dy=dy, dn=dn, dx=dx, dgate=dgate,
                   dresidual=dres, dweight=dw, dnext_weight=dw_next, workspace=workspace)
    rc = _lib.gdr_block_norm_bwd(ctypes.byref(desc), *a, _nbytes(workspace), _stream(stream))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_block_norm_bwd")
    return dx, dgate, dres, dw, dw_next


def loaded_library_path() -> str:
    return LIB_PATH
