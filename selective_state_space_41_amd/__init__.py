"""vmscan: MI355X (gfx950) Vision Mamba bidirectional selective scan and VMamba SS2D cross-scan.

Thin ctypes binding over ``libvmscan.so`` (C ABI in ``include/vmscan.h``).  The functions below
only check and marshal arguments (torch tensors -> device pointers, the current HIP stream, a
workspace from torch's allocator); every step of the scan runs in the library's HIP kernels.
There is no fallback: the library is loaded on first use (``load()``), and if it is missing or
cannot be loaded that raises.
"""
import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvmscan.so")

VMSCAN_F32 = 0
VMSCAN_BF16 = 1
CHUNK_LANE_SCAN = -1  # VMSCAN_CHUNK_LANE_SCAN: chunk_len that selects the lane-scan path (seqlen <= 8192)
D_STATE = 16          # the usual state size; the forward entry points also take 32
D_STATES_FWD = (16, 32)

_c_void_p = ctypes.c_void_p
_i64 = ctypes.c_int64


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m selective_state_space_41_amd.build` "
                          "(or __graft_entry__.build()) first")
    lib = ctypes.CDLL(LIB_PATH)
    lib.vmscan_status_string.restype = ctypes.c_char_p
    lib.vmscan_status_string.argtypes = [ctypes.c_int]
    lib.vmscan_last_hip_error.restype = ctypes.c_int
    lib.vmscan_last_hip_error.argtypes = []
    lib.vmscan_fwd_bidir_chunk_len.restype = _i64
    lib.vmscan_fwd_bidir_chunk_len.argtypes = [_i64, _i64, _i64, ctypes.c_int]
    lib.vmscan_fwd_bidir_workspace_bytes.restype = ctypes.c_size_t
    lib.vmscan_fwd_bidir_workspace_bytes.argtypes = [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int]
    lib.vmscan_fwd_bidir_workspace_bytes_ex.restype = ctypes.c_size_t
    lib.vmscan_fwd_bidir_workspace_bytes_ex.argtypes = [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _i64]
    fwd_args = [_c_void_p] * 13 + [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _c_void_p, ctypes.c_size_t]
    lib.vmscan_fwd_bidir.restype = ctypes.c_int
    lib.vmscan_fwd_bidir.argtypes = fwd_args + [_c_void_p]
    lib.vmscan_fwd_bidir_ex.restype = ctypes.c_int
    lib.vmscan_fwd_bidir_ex.argtypes = fwd_args + [_i64, _c_void_p]
    lib.vmscan_fwd_bidir_stage.restype = ctypes.c_int
    lib.vmscan_fwd_bidir_stage.argtypes = fwd_args + [_i64, ctypes.c_int, _c_void_p]
    lib.vmscan_fwd_bidir_noalloc.restype = ctypes.c_int
    lib.vmscan_fwd_bidir_noalloc.argtypes = [_c_void_p] * 13 + [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                                                 _c_void_p]
    v2_args = [_c_void_p] * 16 + [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _c_void_p, ctypes.c_size_t, _i64]
    lib.vmscan_fwd_bidir_v2.restype = ctypes.c_int
    lib.vmscan_fwd_bidir_v2.argtypes = v2_args + [_c_void_p]
    lib.vmscan_fwd_bidir_v2_stage.restype = ctypes.c_int
    lib.vmscan_fwd_bidir_v2_stage.argtypes = v2_args + [ctypes.c_int, _c_void_p]
    lib.vmscan_bwd_bidir_v2_workspace_bytes.restype = ctypes.c_size_t
    lib.vmscan_bwd_bidir_v2_workspace_bytes.argtypes = [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int]
    lib.vmscan_bwd_bidir_v2.restype = ctypes.c_int
    lib.vmscan_bwd_bidir_v2.argtypes = ([_c_void_p] * 31 + [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _c_void_p,
                                                           ctypes.c_size_t, _c_void_p])
    lib.ss2d_cross_scan_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.ss2d_cross_scan_bwd_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int]
    lib.ss2d_cross_scan_bwd.restype = ctypes.c_int
    lib.ss2d_cross_scan_bwd.argtypes = ([_c_void_p] * 17 + [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                                           _c_void_p, ctypes.c_size_t, _c_void_p])
    lib.ss2d_cross_scan_workspace_bytes.restype = ctypes.c_size_t
    lib.ss2d_cross_scan_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int]
    lib.ss2d_cross_scan_workspace_bytes_ex.restype = ctypes.c_size_t
    lib.ss2d_cross_scan_workspace_bytes_ex.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _i64]
    ss_args = [_c_void_p] * 9 + [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _c_void_p, ctypes.c_size_t]
    lib.ss2d_cross_scan_fwd.restype = ctypes.c_int
    lib.ss2d_cross_scan_fwd.argtypes = ss_args + [_c_void_p]
    lib.ss2d_cross_scan_fwd_ex.restype = ctypes.c_int
    lib.ss2d_cross_scan_fwd_ex.argtypes = ss_args + [_i64, _c_void_p]
    lib.ss2d_cross_scan_fwd_xt.restype = ctypes.c_int
    lib.ss2d_cross_scan_fwd_xt.argtypes = [_c_void_p] + ss_args + [_i64, _c_void_p]
    lib.vmscan_conv1d_silu_fwd.restype = ctypes.c_int
    lib.vmscan_conv1d_silu_fwd.argtypes = [_c_void_p] * 7 + [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _c_void_p]
    lib.ss2d_conv2d_silu_fwd.restype = ctypes.c_int
    lib.ss2d_conv2d_silu_fwd.argtypes = ([_c_void_p] * 3 + [ctypes.c_int] + [_c_void_p] * 2 +
                                         [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _c_void_p])
    lib.vmscan_rmsnorm_fwd.restype = ctypes.c_int
    lib.vmscan_rmsnorm_fwd.argtypes = ([_c_void_p, _i64] + [_c_void_p] * 6 + [_i64, _i64, ctypes.c_float] +
                                       [ctypes.c_int] * 4 + [_c_void_p])
    lib.vmscan_rmsnorm_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.vmscan_rmsnorm_bwd_workspace_bytes.argtypes = [_i64, _i64]
    bwd_args = [_c_void_p] * 6 + [_i64, _i64, ctypes.c_int, ctypes.c_int, _c_void_p, ctypes.c_size_t, _c_void_p]
    lib.vmscan_rmsnorm_bwd.restype = ctypes.c_int
    lib.vmscan_rmsnorm_bwd.argtypes = [_c_void_p] * 2 + bwd_args
    lib.vmscan_rmsnorm_bwd_ex.restype = ctypes.c_int
    lib.vmscan_rmsnorm_bwd_ex.argtypes = [_c_void_p] * 2 + [_i64] + bwd_args
    lib.vmscan_rope_axes.restype = ctypes.c_int
    lib.vmscan_rope_axes.argtypes = ([_c_void_p] * 9 + [_i64, _c_void_p, _c_void_p, _i64, _i64] + [ctypes.c_int] * 8 +
                                     [_c_void_p])
    sizes = [_i64, _i64] + [ctypes.c_int] * 4
    lib.vmscan_linattn_plan.restype = ctypes.c_int
    lib.vmscan_linattn_plan.argtypes = [_i64, _i64] + [ctypes.c_int] * 5 + [_c_void_p]
    lib.vmscan_linattn_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.vmscan_linattn_fwd_workspace_bytes.argtypes = [_i64, _i64] + [ctypes.c_int] * 4
    lib.vmscan_linattn_fwd.restype = ctypes.c_int
    lib.vmscan_linattn_fwd.argtypes = ([_c_void_p] * 12 + sizes + [ctypes.c_float, ctypes.c_int, _c_void_p,
                                                                   ctypes.c_size_t, _c_void_p])
    lib.vmscan_linattn_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.vmscan_linattn_bwd_workspace_bytes.argtypes = [_i64, _i64] + [ctypes.c_int] * 6
    lib.vmscan_linattn_bwd.restype = ctypes.c_int
    lib.vmscan_linattn_bwd.argtypes = ([_c_void_p] * 18 + sizes + [ctypes.c_float, ctypes.c_int, _c_void_p,
                                                                   ctypes.c_size_t, _c_void_p])
    lib.vmscan_linattn_step.restype = ctypes.c_int
    lib.vmscan_linattn_step.argtypes = [_c_void_p] * 11 + sizes + [ctypes.c_float, ctypes.c_int, _c_void_p]
    return lib


_LIB = None


def load():
    """Load libvmscan.so (once) and return the ctypes handle; raises if it is not built."""
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return load()
    raise AttributeError(name)


def status_string(code):
    return load().vmscan_status_string(int(code)).decode()


def _check(code):
    if code != 0:
        msg = status_string(code)
        if code == 6:
            msg += f" (hipError_t {load().vmscan_last_hip_error()})"
        raise RuntimeError(msg)


def _call(fn, args, prepare, keep):
    """Make the C call now, or with ``prepare`` return a callable that makes it again with the same
    validated and marshalled arguments (no per-call checks: for timing and serving loops that
    repeat one call on the same tensors, which ``keep`` holds alive)."""
    if prepare:
        def run(_keep=keep):
            _check(fn(*args))
        return run
    _check(fn(*args))
    return None


def _act_dtype(t):
    if t.dtype == torch.float32:
        return VMSCAN_F32
    if t.dtype == torch.bfloat16:
        return VMSCAN_BF16
    raise TypeError(f"activation dtype must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _workspace(ws, nbytes, dev):
    """The caller's workspace if it is a large enough uint8 device tensor; a new one when none
    was given and the call needs one (None when it needs none).  A workspace that is given but
    too small is an error, not silently replaced: the stages of one call must see the same
    buffer."""
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes > 0 else None
    if ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    if ws.numel() < nbytes:
        raise ValueError(f"workspace holds {ws.numel()} bytes, {nbytes} needed")
    return ws


def _nbytes(t):
    return t.numel() if t is not None else 0


def _d_state(A_log):
    """d_state from the last dimension of A_log (the library rejects sizes it does not take)."""
    if A_log.dim() < 1:
        raise ValueError("A_log must have a state dimension")
    return int(A_log.shape[-1])


def vmscan_fwd_bidir(u, delta_raw, z, A_log, A_b_log, B, C, B_b, C_b, D, D_b, delta_bias,
                     out=None, chunk_len=0, workspace=None, stream=None, stage=3, prepare=False):
    """Bidirectional selective scan with the silu(z) gate; returns ``out`` [batch, dim, L].

    u, delta_raw, z: [batch, dim, L]; A_log, A_b_log: [dim, N] float32 (d_state N = 16 or 32,
    taken from A_log); B, C, B_b, C_b: [batch, N, L] (original token order); D, D_b, delta_bias:
    [dim] float32.  Activations are
    float32 or bfloat16 (all the same).  ``chunk_len`` 0 lets the library choose;
    ``CHUNK_LANE_SCAN`` selects the lane-scan path (no chunks, seqlen <= 8192).  ``stage``
    1 / 2 runs only the preparation (B/C copy, chunk carries) / the fused scan
    (vmscan_fwd_bidir_stage); 3 runs both.  ``prepare=True`` validates once and returns a callable
    that repeats the call on the same tensors and stream."""
    if u.dim() != 3:
        raise ValueError("u must be [batch, dim, L]")
    nb, nd, L = u.shape
    ns = _d_state(A_log)
    dev = u.device
    adt = u.dtype
    dt = _act_dtype(u)
    for name, t in (("u", u), ("delta_raw", delta_raw), ("z", z)):
        _need(t, name, (nb, nd, L), adt, dev)
    for name, t in (("B", B), ("C", C), ("B_b", B_b), ("C_b", C_b)):
        _need(t, name, (nb, ns, L), adt, dev)
    for name, t in (("A_log", A_log), ("A_b_log", A_b_log)):
        _need(t, name, (nd, ns), torch.float32, dev)
    for name, t in (("D", D), ("D_b", D_b), ("delta_bias", delta_bias)):
        _need(t, name, (nd,), torch.float32, dev)
    if out is None:
        out = torch.empty_like(u)
    else:
        _need(out, "out", (nb, nd, L), adt, dev)
    lib = load()
    wsb = lib.vmscan_fwd_bidir_workspace_bytes_ex(nb, nd, L, ns, dt, int(chunk_len))
    workspace = _workspace(workspace, wsb, dev)
    args = (_ptr(u), _ptr(delta_raw), _ptr(z), _ptr(A_log), _ptr(A_b_log), _ptr(B), _ptr(C), _ptr(B_b), _ptr(C_b),
            _ptr(D), _ptr(D_b), _ptr(delta_bias), _ptr(out), nb, nd, L, ns, dt,
            _ptr(workspace), _nbytes(workspace), int(chunk_len), int(stage), _stream(stream, dev))
    run = _call(lib.vmscan_fwd_bidir_stage, args, prepare, (u, delta_raw, z, A_log, A_b_log, B, C, B_b, C_b, D, D_b,
                                                            delta_bias, out, workspace))
    return run if prepare else out


SCRATCH_BYTES = 64 << 20  # VMSCAN_SCRATCH_BYTES: the no-allocation entry point's fixed scratch


def vmscan_fwd_bidir_noalloc(u, delta_raw, z, A_log, A_b_log, B, C, B_b, C_b, D, D_b, delta_bias, out,
                             stream=None):
    """vmscan_fwd_bidir without any device allocation: the library's fixed per-GPU scratch buffer
    stands in for the workspace, and the caller passes ``out``.  Same arguments and result as
    ``vmscan_fwd_bidir`` (bit for bit); raises for shapes whose workspace would exceed
    ``SCRATCH_BYTES``.  Calls that overlap on one GPU share that buffer and race."""
    if u.dim() != 3:
        raise ValueError("u must be [batch, dim, L]")
    nb, nd, L = u.shape
    ns = _d_state(A_log)
    dev = u.device
    adt = u.dtype
    dt = _act_dtype(u)
    for name, t in (("u", u), ("delta_raw", delta_raw), ("z", z), ("out", out)):
        _need(t, name, (nb, nd, L), adt, dev)
    for name, t in (("B", B), ("C", C), ("B_b", B_b), ("C_b", C_b)):
        _need(t, name, (nb, ns, L), adt, dev)
    for name, t in (("A_log", A_log), ("A_b_log", A_b_log)):
        _need(t, name, (nd, ns), torch.float32, dev)
    for name, t in (("D", D), ("D_b", D_b), ("delta_bias", delta_bias)):
        _need(t, name, (nd,), torch.float32, dev)
    _check(load().vmscan_fwd_bidir_noalloc(
        _ptr(u), _ptr(delta_raw), _ptr(z), _ptr(A_log), _ptr(A_b_log), _ptr(B), _ptr(C), _ptr(B_b), _ptr(C_b),
        _ptr(D), _ptr(D_b), _ptr(delta_bias), _ptr(out), nb, nd, L, ns, dt, _stream(stream, dev)))
    return out


def vmscan_fwd_bidir_v2(u, delta_raw, delta_bias, u_b, delta_raw_b, delta_bias_b, z, A_log, A_b_log, B, C, B_b,
                        C_b, D, D_b, out=None, chunk_len=0, workspace=None, stream=None, stage=3, prepare=False):
    """Bidirectional scan whose backward branch has its own u_b, delta_raw_b and delta_bias_b
    (vmscan_fwd_bidir_v2_stage); the other arguments as for ``vmscan_fwd_bidir``.  u_b and
    delta_raw_b are [batch, dim, L] in original token order, delta_bias_b is [dim] float32; any
    of them may be the forward branch's tensor.  ``prepare`` as for ``vmscan_fwd_bidir``."""
    if u.dim() != 3:
        raise ValueError("u must be [batch, dim, L]")
    nb, nd, L = u.shape
    ns = _d_state(A_log)
    dev = u.device
    adt = u.dtype
    dt = _act_dtype(u)
    for name, t in (("u", u), ("delta_raw", delta_raw), ("u_b", u_b), ("delta_raw_b", delta_raw_b), ("z", z)):
        _need(t, name, (nb, nd, L), adt, dev)
    for name, t in (("B", B), ("C", C), ("B_b", B_b), ("C_b", C_b)):
        _need(t, name, (nb, ns, L), adt, dev)
    for name, t in (("A_log", A_log), ("A_b_log", A_b_log)):
        _need(t, name, (nd, ns), torch.float32, dev)
    for name, t in (("D", D), ("D_b", D_b), ("delta_bias", delta_bias), ("delta_bias_b", delta_bias_b)):
        _need(t, name, (nd,), torch.float32, dev)
    if out is None:
        out = torch.empty_like(u)
    else:
        _need(out, "out", (nb, nd, L), adt, dev)
    lib = load()
    wsb = lib.vmscan_fwd_bidir_workspace_bytes_ex(nb, nd, L, ns, dt, int(chunk_len))
    workspace = _workspace(workspace, wsb, dev)
    args = (_ptr(u), _ptr(delta_raw), _ptr(delta_bias), _ptr(u_b), _ptr(delta_raw_b), _ptr(delta_bias_b), _ptr(z),
            _ptr(A_log), _ptr(A_b_log), _ptr(B), _ptr(C), _ptr(B_b), _ptr(C_b), _ptr(D), _ptr(D_b), _ptr(out),
            nb, nd, L, ns, dt, _ptr(workspace), _nbytes(workspace), int(chunk_len), int(stage),
            _stream(stream, dev))
    run = _call(lib.vmscan_fwd_bidir_v2_stage, args, prepare, (u, delta_raw, delta_bias, u_b, delta_raw_b,
                                                               delta_bias_b, z, A_log, A_b_log, B, C, B_b, C_b, D,
                                                               D_b, out, workspace))
    return run if prepare else out


def vmscan_bwd_bidir_v2(u, delta_raw, delta_bias, u_b, delta_raw_b, delta_bias_b, z, A_log, A_b_log, B, C, B_b, C_b,
                        D, D_b, dout, shared=False, workspace=None, stream=None, prepare=False):
    """Gradients of ``vmscan_fwd_bidir_v2`` for ``dout`` (vmscan_bwd_bidir_v2); returns a dict with
    du, ddelta_raw, ddelta_bias, du_b, ddelta_raw_b, ddelta_bias_b, dz, dA_log, dA_b_log, dB, dC,
    dB_b, dC_b, dD, dD_b.  With ``shared=True`` (u_b is u, delta_raw_b is delta_raw, delta_bias_b
    is delta_bias, i.e. ``vmscan_fwd_bidir``) the backward branch's du, ddelta_raw and ddelta_bias
    are added into the forward ones and the ``_b`` entries are None.  d_state 16 or 32.  With
    ``prepare`` it returns (callable, gradient dict): each call rewrites the same gradient tensors."""
    if u.dim() != 3:
        raise ValueError("u must be [batch, dim, L]")
    nb, nd, L = u.shape
    ns = _d_state(A_log)
    dev = u.device
    adt = u.dtype
    dt = _act_dtype(u)
    for name, t in (("u", u), ("delta_raw", delta_raw), ("u_b", u_b), ("delta_raw_b", delta_raw_b), ("z", z),
                    ("dout", dout)):
        _need(t, name, (nb, nd, L), adt, dev)
    for name, t in (("B", B), ("C", C), ("B_b", B_b), ("C_b", C_b)):
        _need(t, name, (nb, ns, L), adt, dev)
    for name, t in (("A_log", A_log), ("A_b_log", A_b_log)):
        _need(t, name, (nd, ns), torch.float32, dev)
    for name, t in (("D", D), ("D_b", D_b), ("delta_bias", delta_bias), ("delta_bias_b", delta_bias_b)):
        _need(t, name, (nd,), torch.float32, dev)
    act = lambda: torch.empty_like(u)
    bcs = lambda: torch.empty_like(B)
    par = lambda *s: torch.empty(*s, dtype=torch.float32, device=dev)
    g = dict(du=act(), ddelta_raw=act(), ddelta_bias=par(nd), dz=act(), dA_log=par(nd, ns),
             dA_b_log=par(nd, ns), dB=bcs(), dC=bcs(), dB_b=bcs(), dC_b=bcs(), dD=par(nd), dD_b=par(nd))
    g["du_b"], g["ddelta_raw_b"], g["ddelta_bias_b"] = (None, None, None) if shared else (act(), act(), par(nd))
    lib = load()
    wsb = lib.vmscan_bwd_bidir_v2_workspace_bytes(nb, nd, L, ns, dt)
    workspace = _workspace(workspace, wsb, dev)
    args = (_ptr(u), _ptr(delta_raw), _ptr(delta_bias), _ptr(u_b), _ptr(delta_raw_b), _ptr(delta_bias_b), _ptr(z),
            _ptr(A_log), _ptr(A_b_log), _ptr(B), _ptr(C), _ptr(B_b), _ptr(C_b), _ptr(D), _ptr(D_b), _ptr(dout),
            *[_ptr(g[k]) for k in ("du", "ddelta_raw", "ddelta_bias", "du_b", "ddelta_raw_b", "ddelta_bias_b", "dz",
                                   "dA_log", "dA_b_log", "dB", "dC", "dB_b", "dC_b", "dD", "dD_b")],
            nb, nd, L, ns, dt, _ptr(workspace), _nbytes(workspace), _stream(stream, dev))
    run = _call(lib.vmscan_bwd_bidir_v2, args, prepare, (u, delta_raw, delta_bias, u_b, delta_raw_b, delta_bias_b, z,
                                                         A_log, A_b_log, B, C, B_b, C_b, D, D_b, dout, g, workspace))
    return (run, g) if prepare else g


def ss2d_cross_scan_fwd(x, delta_raw, A_log, B, C, D, delta_bias, z=None, out=None, chunk_len=0,
                        workspace=None, stream=None, xT=None, prepare=False):
    """SS2D four-direction cross-scan with cross-merge; returns ``out`` [batch, dim, H, W].

    x: [batch, dim, H, W]; delta_raw: [batch, 4, dim, H*W]; A_log: [4, dim, N] float32 (d_state
    N = 16 or 32); B, C: [batch, 4, N, H*W] (each direction's scan order); D, delta_bias: [4, dim]
    float32; z: optional [batch, dim, H, W] gate; xT: optional [batch, dim, W, H], x transposed
    (as written by ``ss2d_conv2d_silu_fwd``), read instead of a copy made by the call
    (ss2d_cross_scan_fwd_xt).  ``prepare`` as for ``vmscan_fwd_bidir``."""
    if x.dim() != 4:
        raise ValueError("x must be [batch, dim, H, W]")
    nb, nd, H, W = x.shape
    L = H * W
    ns = _d_state(A_log)
    dev = x.device
    adt = x.dtype
    dt = _act_dtype(x)
    _need(x, "x", (nb, nd, H, W), adt, dev)
    _need(delta_raw, "delta_raw", (nb, 4, nd, L), adt, dev)
    _need(B, "B", (nb, 4, ns, L), adt, dev)
    _need(C, "C", (nb, 4, ns, L), adt, dev)
    _need(A_log, "A_log", (4, nd, ns), torch.float32, dev)
    _need(D, "D", (4, nd), torch.float32, dev)
    _need(delta_bias, "delta_bias", (4, nd), torch.float32, dev)
    if z is not None:
        _need(z, "z", (nb, nd, H, W), adt, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", (nb, nd, H, W), adt, dev)
    lib = load()
    wsb = lib.ss2d_cross_scan_workspace_bytes_ex(nb, nd, H, W, ns, dt, int(chunk_len))
    workspace = _workspace(workspace, wsb, dev)
    args = (_ptr(delta_raw), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(delta_bias), _ptr(z), _ptr(out),
            nb, nd, H, W, ns, dt, _ptr(workspace), _nbytes(workspace), int(chunk_len), _stream(stream, dev))
    keep = (x, xT, delta_raw, A_log, B, C, D, delta_bias, z, out, workspace)
    if xT is None:
        run = _call(lib.ss2d_cross_scan_fwd_ex, (_ptr(x),) + args, prepare, keep)
    else:
        _need(xT, "xT", (nb, nd, W, H), adt, dev)
        run = _call(lib.ss2d_cross_scan_fwd_xt, (_ptr(x), _ptr(xT)) + args, prepare, keep)
    return run if prepare else out


def ss2d_cross_scan_bwd(x, delta_raw, A_log, B, C, D, delta_bias, z, dout, workspace=None, stream=None,
                        prepare=False):
    """Gradients of ``ss2d_cross_scan_fwd`` for ``dout`` (ss2d_cross_scan_bwd); returns a dict with
    dx, ddelta_raw, dA_log, dB, dC, dD, ddelta_bias and dz (None when z is None).  d_state 16 or 32.
    ``prepare`` as for ``vmscan_bwd_bidir_v2``."""
    if x.dim() != 4:
        raise ValueError("x must be [batch, dim, H, W]")
    nb, nd, H, W = x.shape
    L = H * W
    ns = _d_state(A_log)
    dev = x.device
    adt = x.dtype
    dt = _act_dtype(x)
    _need(x, "x", (nb, nd, H, W), adt, dev)
    _need(dout, "dout", (nb, nd, H, W), adt, dev)
    _need(delta_raw, "delta_raw", (nb, 4, nd, L), adt, dev)
    _need(B, "B", (nb, 4, ns, L), adt, dev)
    _need(C, "C", (nb, 4, ns, L), adt, dev)
    _need(A_log, "A_log", (4, nd, ns), torch.float32, dev)
    _need(D, "D", (4, nd), torch.float32, dev)
    _need(delta_bias, "delta_bias", (4, nd), torch.float32, dev)
    if z is not None:
        _need(z, "z", (nb, nd, H, W), adt, dev)
    g = dict(dx=torch.empty_like(x), ddelta_raw=torch.empty_like(delta_raw), dA_log=torch.empty_like(A_log),
             dB=torch.empty_like(B), dC=torch.empty_like(C), dD=torch.empty_like(D),
             ddelta_bias=torch.empty_like(delta_bias), dz=torch.empty_like(x) if z is not None else None)
    lib = load()
    wsb = lib.ss2d_cross_scan_bwd_workspace_bytes(nb, nd, H, W, ns, dt)
    workspace = _workspace(workspace, wsb, dev)
    args = (_ptr(x), _ptr(delta_raw), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(delta_bias), _ptr(z), _ptr(dout),
            *[_ptr(g[k]) for k in ("dx", "ddelta_raw", "dA_log", "dB", "dC", "dD", "ddelta_bias", "dz")],
            nb, nd, H, W, ns, dt, _ptr(workspace), _nbytes(workspace), _stream(stream, dev))
    run = _call(lib.ss2d_cross_scan_bwd, args, prepare, (x, delta_raw, A_log, B, C, D, delta_bias, z, dout, g,
                                                         workspace))
    return (run, g) if prepare else g


def conv1d_silu_fwd(x, conv_w, conv_b, conv_w_b=None, conv_b_b=None, u=None, u_b=None, stream=None):
    """Front of the Vim scan (vmscan_conv1d_silu_fwd): u = silu(causal depthwise conv1d(x) + conv_b)
    and, when conv_w_b / conv_b_b are given, u_b = the flipped branch's convolution in original
    token order.  x: [batch, dim, L] float32 or bfloat16; conv_w(_b): [dim, d_conv] float32
    (d_conv 1..4); conv_b(_b): [dim] float32.  Returns (u, u_b), u_b None for one branch."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, dim, L]")
    nb, nd, L = x.shape
    dev, adt, dt = x.device, x.dtype, _act_dtype(x)
    if conv_w.dim() != 2:
        raise ValueError("conv_w must be [dim, d_conv]")
    K = int(conv_w.shape[1])
    _need(conv_w, "conv_w", (nd, K), torch.float32, dev)
    _need(conv_b, "conv_b", (nd,), torch.float32, dev)
    two = conv_w_b is not None or conv_b_b is not None
    if two:
        _need(conv_w_b, "conv_w_b", (nd, K), torch.float32, dev)
        _need(conv_b_b, "conv_b_b", (nd,), torch.float32, dev)
    if u is None:
        u = torch.empty_like(x)
    _need(u, "u", (nb, nd, L), adt, dev)
    if two:
        if u_b is None:
            u_b = torch.empty_like(x)
        _need(u_b, "u_b", (nb, nd, L), adt, dev)
    else:
        u_b = None
    _check(load().vmscan_conv1d_silu_fwd(_ptr(x), _ptr(conv_w), _ptr(conv_b), _ptr(conv_w_b), _ptr(conv_b_b),
                                         _ptr(u), _ptr(u_b), nb, nd, L, K, dt, _stream(stream, dev)))
    return u, u_b


def ss2d_conv2d_silu_fwd(x, conv_w, conv_b, act=True, transposed=True, x_out=None, xT_out=None, stream=None):
    """Front of SS2D (ss2d_conv2d_silu_fwd): depthwise 3 x 3 convolution (+ SiLU when ``act``) of
    x [batch, dim, H, W]; conv_w [dim, 3, 3], conv_b [dim] float32.  Returns (x_out, xT_out):
    the result row-major and, when ``transposed``, also as [batch, dim, W, H]."""
    if x.dim() != 4:
        raise ValueError("x must be [batch, dim, H, W]")
    nb, nd, H, W = x.shape
    dev, adt, dt = x.device, x.dtype, _act_dtype(x)
    if conv_w.dim() != 3:
        raise ValueError("conv_w must be [dim, K, K]")
    K = int(conv_w.shape[1])
    _need(conv_w, "conv_w", (nd, K, K), torch.float32, dev)
    _need(conv_b, "conv_b", (nd,), torch.float32, dev)
    if x_out is None:
        x_out = torch.empty_like(x)
    _need(x_out, "x_out", (nb, nd, H, W), adt, dev)
    if transposed:
        if xT_out is None:
            xT_out = torch.empty((nb, nd, W, H), dtype=adt, device=dev)
        _need(xT_out, "xT_out", (nb, nd, W, H), adt, dev)
    else:
        xT_out = None
    _check(load().ss2d_conv2d_silu_fwd(_ptr(x), _ptr(conv_w), _ptr(conv_b), int(bool(act)), _ptr(x_out),
                                       _ptr(xT_out), nb, nd, H, W, K, dt, _stream(stream, dev)))
    return x_out, xT_out


def fwd_bidir_chunk_len(batch, dim, seqlen, d_state=D_STATE):
    return int(load().vmscan_fwd_bidir_chunk_len(batch, dim, seqlen, d_state))


# ------------------------------------------------------------------------------------------------
# Operators of a linear-attention block: norm with residual, rotary positions, decayed attention.
#
# ``stream``: the stream that a call works on, the current one by default.  Ordering it after what makes the inputs, and
# the current one after it, is the caller's; memory that the call allocates is safe on both.

_DTYPES = {torch.float32: VMSCAN_F32, torch.bfloat16: VMSCAN_BF16}
_FP8 = torch.float8_e4m3fn


def _is_act(t, name, ndim):
    """The activation dtype code of a [..., channels] device tensor whose channels are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return dt


_pack2, _pack3 = struct.Struct("=2q").pack, struct.Struct("=3q").pack


def _strided(t, name, shape, dtype, device):
    """A tensor [batch, (token,) head, channel] of any strides but contiguous channels; its leading
    strides as the library's int64 array, 0 where the dimension has one element (whose stride says
    nothing)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name} must have contiguous channels")
    if len(st) == 4:
        a, b, c, _ = st
        n, m, k, _ = shape
        return _pack3(a if n != 1 else 0, b if m != 1 else 0, c if k != 1 else 0)
    a, b, _ = st
    n, m, _ = shape
    return _pack2(a if n != 1 else 0, b if m != 1 else 0)


def _on_stream(stream, fn, *args):
    """The call on another stream: what it allocates is that stream's memory (a block of the current one's could still
    be written by work that waits there), and stays reserved while the current one uses it."""
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        got = fn(*args)
    for t in got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,):
        for x in t.values() if isinstance(t, dict) else (t,):
            if isinstance(x, torch.Tensor):
                x.record_stream(here)
    return got


def _enqueue(fn, args, dev, prepare=False, keep=None):
    """The C call with the tensors' device current (a stream belongs to a device)."""
    if prepare:
        return _call(fn, args, True, keep)
    if dev.index == torch.cuda.current_device():
        code = fn(*args)
    else:
        with torch.cuda.device(dev):
            code = fn(*args)
    if code:
        _check(code)
    return None


# The current stream's handle without making a Stream object (a tenth of the time, and these calls
# may be as short as a few microseconds), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(dev):
    return _raw_stream(dev.index) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _p(t):
    return t.data_ptr() if t is not None else None


def _row_stride(t, name):
    """The row stride of a contiguous [..., dim] tensor, or of a [rows, dim] one whose rows are apart."""
    if t.is_contiguous():
        return t.shape[-1]
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
        return t.stride(0)
    raise ValueError(f"{name} must be contiguous, or [rows, dim] with contiguous channels and rows that do not overlap")


def rmsnorm_fwd(x, weight, residual=None, eps=1e-5, out_dtype=None, group=0, y=None, residual_out=None, stream=None):
    """Residual addition and root-mean-square norm (vmscan_rmsnorm_fwd): r = x + residual, y = r *
    rsqrt(mean(r^2) + eps) * weight.  Returns (y, scale, residual_out, rstd).

    x: [..., dim] float32 or bfloat16 (rows may be apart: [rows, dim] with any row stride); weight: [dim]
    float32; residual: like x, dtype x's or float32, or None (then residual_out is x itself).
    out_dtype None: y in x's dtype, scale None; torch.float8_e4m3fn: y holds 8-bit codes and scale
    [..., 1] float32 (group 0, one per row) or [..., ceil(dim / 128)] (group 128): y * scale is the
    norm.  ``residual_out`` may be ``residual`` (in place).  rstd [...] float32 is for ``rmsnorm_bwd``."""
    if stream is not None:
        return _on_stream(stream, rmsnorm_fwd, x, weight, residual, eps, out_dtype, group, y, residual_out)
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a torch.Tensor with a channel dimension")
    dt = _is_act(x, "x", x.dim())
    dev, shape = x.device, tuple(x.shape)
    dim, lead = shape[-1], shape[:-1]
    rows = x.numel() // dim if dim else 0
    row_stride = _row_stride(x, "x")
    _need(weight, "weight", (dim,), torch.float32, dev)
    rdt = dt
    if residual is not None:
        rdt = _is_act(residual, "residual", x.dim())
        _need(residual, "residual", shape, residual.dtype, dev)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        else:
            _need(residual_out, "residual_out", shape, residual.dtype, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    fp8 = out_dtype == _FP8
    if out_dtype is not None and not fp8 and out_dtype != x.dtype:
        raise TypeError(f"out_dtype must be {x.dtype} or {_FP8}, got {out_dtype}")
    ydt = _FP8 if fp8 else x.dtype
    if y is None:
        y = torch.empty(shape, dtype=ydt, device=dev) if fp8 or row_stride != dim else torch.empty_like(x)
    else:
        _need(y, "y", shape, ydt, dev)
    scale = None
    if fp8:
        scale = torch.empty(lead + (-(-dim // group) if group else 1,), dtype=torch.float32, device=dev)
    rstd = torch.empty(lead, dtype=torch.float32, device=dev)
    _enqueue(load().vmscan_rmsnorm_fwd,
             (x.data_ptr(), row_stride, _p(residual), weight.data_ptr(), y.data_ptr(), _p(scale), _p(residual_out),
              rstd.data_ptr(), rows, dim, eps, dt, rdt, int(fp8), int(group), _current(dev)), dev)
    return y, scale, residual_out if residual is not None else x, rstd


def rmsnorm_bwd(dy, r, weight, rstd, dresidual_out=None, workspace=None, stream=None):
    """Gradient of ``rmsnorm_fwd`` (vmscan_rmsnorm_bwd); returns a dict with dx (dy's dtype), dresidual
    (r's dtype; dx itself when the two are the same) and dweight [dim] float32.

    dy: [..., dim] contiguous gradient of y; r: the forward's residual_out (without a residual its x, rows apart
    or not); rstd: the forward's; dresidual_out: the gradient that reaches residual_out on its other way, or None."""
    if stream is not None:
        return _on_stream(stream, rmsnorm_bwd, dy, r, weight, rstd, dresidual_out, workspace)
    dt = _is_act(dy, "dy", dy.dim() if isinstance(dy, torch.Tensor) else 0)
    dev, shape, dim = dy.device, dy.shape, dy.shape[-1]
    rdt = _is_act(r, "r", dy.dim())
    _need(dy, "dy", shape, dy.dtype, dev)
    if r.shape != shape or r.device != dev:
        raise ValueError(f"r is {tuple(r.shape)} on {r.device}, expected {tuple(shape)} on {dev}")
    r_stride = _row_stride(r, "r")
    _need(weight, "weight", (dim,), torch.float32, dev)
    _need(rstd, "rstd", shape[:-1], torch.float32, dev)
    if dresidual_out is not None:
        _need(dresidual_out, "dresidual_out", shape, r.dtype, dev)
    rows = dy.numel() // dim if dim else 0
    lib = load()
    workspace = _workspace(workspace, lib.vmscan_rmsnorm_bwd_workspace_bytes(rows, dim), dev)
    dx, dw = torch.empty_like(dy), torch.empty(dim, dtype=torch.float32, device=dev)
    dres = torch.empty(shape, dtype=r.dtype, device=dev) if r.dtype != dy.dtype else None
    _enqueue(lib.vmscan_rmsnorm_bwd_ex,
             (dy.data_ptr(), r.data_ptr(), r_stride, weight.data_ptr(), rstd.data_ptr(), _p(dresidual_out), dx.data_ptr(),
              _p(dres), dw.data_ptr(), rows, dim, dt, rdt, _p(workspace), _nbytes(workspace), _current(dev)), dev)
    return dict(dx=dx, dresidual=dx if dres is None else dres, dweight=dw)


def rope_axes(q, k, positions, inv_freq, axis, interleaved=False, inverse=False, q_out=None, k_out=None, stream=None):
    """Rotary positions with several axes (vmscan_rope_axes); returns (q_out, k_out).

    q: [batch, L, heads, dim], k: [batch, L, kheads, dim] or None, float32 or bfloat16, any strides with
    contiguous channels; positions: [L, axes] or [batch, L, axes] float32; inv_freq: [pairs] float32 and
    axis: [pairs] int32 give pair p the angle positions[..., axis[p]] * inv_freq[p].  The pairs are the
    channels (p, p + pairs), or (2p, 2p + 1) when ``interleaved``; channels from 2 * pairs on pass
    through.  ``inverse`` turns back: the gradient of the forward turn.  Outputs are contiguous unless
    given; an output may be its own input, unless that is expanded (its elements overlap)."""
    if stream is not None:
        return _on_stream(stream, rope_axes, q, k, positions, inv_freq, axis, interleaved, inverse, q_out, k_out)
    dt = _is_act(q, "q", 4)
    dev, (nb, L, H, dim) = q.device, q.shape
    qs = _strided(q, "q", q.shape, q.dtype, dev)
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a [pairs] tensor")
    pairs = inv_freq.shape[0]
    _need(inv_freq, "inv_freq", (pairs,), torch.float32, dev)
    _need(axis, "axis", (pairs,), torch.int32, dev)
    if not isinstance(positions, torch.Tensor) or positions.dim() not in (2, 3):
        raise ValueError("positions must be [L, axes] or [batch, L, axes]")
    axes = positions.shape[-1]
    _need(positions, "positions", (L, axes) if positions.dim() == 2 else (nb, L, axes), torch.float32, dev)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    qos = _strided(q_out, "q_out", q.shape, q.dtype, dev)
    Hk, ks, kos = 0, None, None
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be [batch, L, kheads, dim]")
        Hk = k.shape[2]
        if Hk < 1:
            raise ValueError("k has no heads")
        ks = _strided(k, "k", (nb, L, Hk, dim), q.dtype, dev)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=dev)
        kos = _strided(k_out, "k_out", k.shape, q.dtype, dev)
    elif k_out is not None:
        raise ValueError("k_out needs a k")
    _enqueue(load().vmscan_rope_axes,
             (q.data_ptr(), qs, q_out.data_ptr(), qos, _p(k), ks, _p(k_out), kos, positions.data_ptr(),
              L * axes if positions.dim() == 3 else 0, inv_freq.data_ptr(), axis.data_ptr(), nb, L, H, Hk, dim,
              2 * pairs, axes, int(bool(interleaved)), int(bool(inverse)), dt, _current(dev)), dev)
    return q_out, k_out


def _linattn_args(q, k, v, log_decay, ndim):
    """Checks what every linear-attention call takes; returns (dtype code, batch and token sizes, heads,
    kheads, dk, dv, strides of q, k, v and of the decay, None for one decay per head)."""
    dt = _is_act(q, "q", ndim)
    dev, adt, shape = q.device, q.dtype, tuple(q.shape)
    lead, Hk, dk = shape[:-2], shape[-2], shape[-1]
    if not isinstance(v, torch.Tensor) or v.dim() != ndim:
        raise ValueError(f"v must have {ndim} dimensions")
    vshape = tuple(v.shape)
    H, dv = vshape[-2], vshape[-1]
    if Hk < 1 or H % Hk:
        raise ValueError(f"{H} heads of v cannot share {Hk} heads of q and k")
    qs = _strided(q, "q", shape, adt, dev)
    ks = _strided(k, "k", shape, adt, dev)
    vs = _strided(v, "v", lead + (H, dv), adt, dev)
    if not isinstance(log_decay, torch.Tensor):
        raise TypeError("log_decay must be a torch.Tensor")
    if log_decay.dtype != torch.float32 or log_decay.device != dev:
        raise TypeError(f"log_decay must be float32 on {dev}, got {log_decay.dtype} on {log_decay.device}")
    gs = None
    if log_decay.dim() == 1:
        _need(log_decay, "log_decay", (H,), torch.float32, dev)
    elif log_decay.shape == lead + (H,):
        gs = (_pack3 if ndim == 4 else _pack2)(*[s if d != 1 else 0 for s, d in zip(log_decay.stride(), log_decay.shape)])
    else:
        raise ValueError(f"log_decay has shape {tuple(log_decay.shape)}, expected {(H,)} or {lead + (H,)}")
    return dt, lead, H, Hk, dk, dv, qs, ks, vs, gs


def linattn_plan(batch, seqlen, heads, dk, dv, dtype=torch.bfloat16, gradient=False):
    """How ``linattn_fwd`` (or, with ``gradient``, ``linattn_bwd``) cuts up a call (vmscan_linattn_plan): a dict with the
    tokens of a block, the value channels of a workgroup (width), segments of a sequence, parts of a segment and how their
    states are joined (None, "walk" or "launch")."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    cut = (ctypes.c_int32 * 5)()
    _check(load().vmscan_linattn_plan(batch, seqlen, heads, dk, dv, _DTYPES[dtype], int(bool(gradient)), cut))
    return dict(block=cut[0], width=cut[1], segments=cut[2], parts=cut[3], join=(None, "walk", "launch")[cut[4]])


def linattn_fwd(q, k, v, log_decay, scale=None, initial_state=None, lengths=None, out=None, final_state=None,
                workspace=None, stream=None, prepare=False):
    """Linear attention with a decay for each head (vmscan_linattn_fwd); returns (out, final_state).

    Per head S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T and out_t = scale * S_t^T q_t.  q, k: [batch, L,
    kheads, dk]; v: [batch, L, heads, dv], heads a multiple of kheads (a q/k head serves neighbouring
    heads); float32 or bfloat16, contiguous channels, other strides multiples of 16 bytes; dk and dv
    multiples of 8 up to 128.  log_decay: float32 [batch, L, heads] (any strides) or [heads].  scale
    defaults to dk ** -0.5.  initial_state / final_state: [batch, heads, dk, dv] float32; the same tensor for
    both is updated in place (they must not overlap otherwise).  lengths: [batch]
    int32, the tokens of each row; out is 0 past them.  ``prepare`` as for ``vmscan_fwd_bidir`` (the
    callable then rewrites the same out and final_state): returns (callable, out, final_state)."""
    if stream is not None:
        return _on_stream(stream, linattn_fwd, q, k, v, log_decay, scale, initial_state, lengths, out, final_state,
                          workspace, None, prepare)
    dt, (nb, L), H, Hk, dk, dv, qs, ks, vs, gs = _linattn_args(q, k, v, log_decay, 4)
    dev = q.device
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None:
            _need(t, name, (nb, H, dk, dv), torch.float32, dev)
    if lengths is not None:
        _need(lengths, "lengths", (nb,), torch.int32, dev)
    if out is None:
        out = torch.empty(nb, L, H, dv, dtype=q.dtype, device=dev)
    else:
        _need(out, "out", (nb, L, H, dv), q.dtype, dev)
    if final_state is None:
        final_state = torch.empty(nb, H, dk, dv, dtype=torch.float32, device=dev)
    lib = load()
    workspace = _workspace(workspace, lib.vmscan_linattn_fwd_workspace_bytes(nb, L, H, dk, dv, dt), dev)
    args = (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, log_decay.data_ptr(), gs, _p(initial_state),
            _p(lengths), out.data_ptr(), final_state.data_ptr(), nb, L, H, Hk, dk, dv,
            float(dk ** -0.5 if scale is None else scale), dt, _p(workspace), _nbytes(workspace), _current(dev))
    run = _enqueue(lib.vmscan_linattn_fwd, args, dev, prepare,
                   (q, k, v, log_decay, initial_state, lengths, out, final_state, workspace))
    return (run, out, final_state) if prepare else (out, final_state)


def linattn_bwd(q, k, v, log_decay, dout, scale=None, initial_state=None, lengths=None, dfinal_state=None,
                workspace=None, stream=None, prepare=False):
    """Gradients of ``linattn_fwd`` for ``dout`` [batch, L, heads, dv] and, optionally, ``dfinal_state``
    [batch, heads, dk, dv] (vmscan_linattn_bwd); returns a dict with dq, dk, dv, dlog_decay (of log_decay's
    shape) and dinitial_state (None without an initial_state).  Deterministic.  ``prepare`` as for
    ``vmscan_bwd_bidir_v2``."""
    if stream is not None:
        return _on_stream(stream, linattn_bwd, q, k, v, log_decay, dout, scale, initial_state, lengths, dfinal_state,
                          workspace, None, prepare)
    dt, (nb, L), H, Hk, dk, dv, qs, ks, vs, gs = _linattn_args(q, k, v, log_decay, 4)
    dev = q.device
    os_ = _strided(dout, "dout", (nb, L, H, dv), q.dtype, dev)
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _need(t, name, (nb, H, dk, dv), torch.float32, dev)
    if lengths is not None:
        _need(lengths, "lengths", (nb,), torch.int32, dev)
    f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device=dev)
    act = lambda *s: torch.empty(*s, dtype=q.dtype, device=dev)
    g = dict(dq=act(nb, L, Hk, dk), dk=act(nb, L, Hk, dk), dv=act(nb, L, H, dv), dlog_decay=f32(*log_decay.shape),
             dinitial_state=f32(nb, H, dk, dv) if initial_state is not None else None)
    lib = load()
    workspace = _workspace(workspace, lib.vmscan_linattn_bwd_workspace_bytes(nb, L, H, Hk, dk, dv, int(gs is None), dt),
                           dev)
    args = (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, log_decay.data_ptr(), gs, _p(initial_state),
            _p(lengths), dout.data_ptr(), os_, _p(dfinal_state), g["dq"].data_ptr(), g["dk"].data_ptr(),
            g["dv"].data_ptr(), g["dlog_decay"].data_ptr(), _p(g["dinitial_state"]), nb, L, H, Hk, dk, dv,
            float(dk ** -0.5 if scale is None else scale), dt, _p(workspace), _nbytes(workspace), _current(dev))
    run = _enqueue(lib.vmscan_linattn_bwd, args, dev, prepare,
                   (q, k, v, log_decay, initial_state, lengths, dout, dfinal_state, g, workspace))
    return (run, g) if prepare else g


def linattn_step(q, k, v, log_decay, state, scale=None, slots=None, out=None, stream=None, prepare=False):
    """One token of each of ``batch`` sequences (vmscan_linattn_step): updates ``state`` in place and
    returns out [batch, heads, dv].

    q, k: [batch, kheads, dk]; v: [batch, heads, dv]; log_decay: float32 [batch, heads] or [heads]; state:
    [pool, heads, dk, dv] float32; slots: [batch] int32, the state of each sequence (all different; one
    outside 0 .. pool - 1 skips the row, whose out is 0), or None with pool = batch.  ``prepare`` as for
    ``linattn_fwd``: returns (callable, out)."""
    if stream is not None:
        return _on_stream(stream, linattn_step, q, k, v, log_decay, state, scale, slots, out, None, prepare)
    dt, (nb,), H, Hk, dk, dv, qs, ks, vs, gs = _linattn_args(q, k, v, log_decay, 3)
    dev = q.device
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be [pool, heads, dk, dv]")
    pool = state.shape[0]
    _need(state, "state", (pool, H, dk, dv), torch.float32, dev)
    if slots is not None:
        _need(slots, "slots", (nb,), torch.int32, dev)
    elif pool != nb:
        raise ValueError(f"without slots the pool holds one state per sequence: {pool} for {nb}")
    if out is None:
        out = torch.empty(nb, H, dv, dtype=q.dtype, device=dev)
    else:
        _need(out, "out", (nb, H, dv), q.dtype, dev)
    args = (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, log_decay.data_ptr(), gs, state.data_ptr(),
            _p(slots), out.data_ptr(), nb, pool, H, Hk, dk, dv, float(dk ** -0.5 if scale is None else scale), dt,
            _current(dev))
    run = _enqueue(load().vmscan_linattn_step, args, dev, prepare, (q, k, v, log_decay, state, slots, out))
    return (run, out) if prepare else out
