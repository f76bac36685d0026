"""Python binding of the MI355X selective-scan (S6) library (include/ss.h).

Argument marshalling only: torch supplies device memory and the current stream,
every step of the scan runs in the library's HIP kernels.  There is no CPU or
PyTorch fallback: if the compiled library is missing, ``load()`` raises.

    y = ss_fwd(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, z=None, h0=None)
    y, h_final = ss_fwd(..., return_final=True)
    y, h_final, h_ckpt = ss_fwd(..., return_final=True, return_ckpt=True)
    grads = ss_bwd(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, dy, z=None, h0=None, dh_final=None,
                   h_ckpt=None)
    y_t = ss_step(x_t, dt_raw_t, dt_bias, A, B_t, C_t, Dskip, h, z_t=None)   # h updated in place
    o = ss_la_fwd(q, k, v, g=None, s0=None, scale=1.0)      # linear attention, decay per head
    grads = ss_la_bwd(q, k, v, do, g=None, s0=None, ds_final=None, scale=1.0)
    o_t = ss_la_step(q_t, k_t, v_t, s, g_t=None, scale=1.0)                  # s updated in place
    y, r = ss_rms_fwd(x, w, res)                 # RMS norm after the residual's addition
    y8, y_scale, r = ss_rms_fwd(x, w, res, q8=SS_Q8_FP8)                     # ... in 8 bits
    dx, dw = ss_rms_bwd(dy, r, w, dr=None)
    y = ss_q4_mv(x, wq, scales, zeros=None, x_scale=None)                    # 4-bit weights
    y = ss_gr_fwd(x, r, i, lam, h0=None)         # gated recurrence of one number a channel
    y, h_ckpt = ss_gr_fwd(..., return_ckpt=True)
    grads = ss_gr_bwd(x, r, i, lam, dy, h0=None, dh_final=None, h_ckpt=None)
    y_t = ss_gr_step(x_t, r_t, i_t, lam, h)                                  # h updated in place
    y, r = ss_ln_fwd(x, w, b, res)               # layer norm after the residual's addition
    dx, dw, db = ss_ln_bwd(dy, r, w, dr=None)
    codes, exps = ss_mx4_quant(x)                # 4-bit values, 32 to a power of two
    y = ss_mx4_mm(codes, exps, wq, w_exps)       # their products, for one row or for many

Layouts: x, dt_raw, z, y [B, D, L]; Bm, Cm [B, N, L]; A [D, N]; dt_bias, Dskip [D];
h0, h_final [B, D, N]; h_ckpt [B, D, ceil(L/16), N] (state entering every 16th step).  x, dt_raw, z, Bm, Cm are float32 or bfloat16 (all the same);
everything else is float32.
"""
import contextlib
import ctypes
import functools
import os

from ._build import LIB, build, stale, tree_id  # noqa: F401

SS_F32, SS_BF16 = 0, 1
SS_PLAN_AUTO, SS_PLAN_SINGLE, SS_PLAN_CHUNKED = 0, 1, 2
SS_LAYOUT_AUTO, SS_LAYOUT_QUAD, SS_LAYOUT_LANE, SS_LAYOUT_OCT = 0, 1, 2, 3
SS_DISC_EULER, SS_DISC_ZOH = 0, 1
SS_ORDER_BDL, SS_ORDER_BLD = 0, 1
SS_DT_FULL, SS_DT_SHARED = 0, 1
SS_LA_DECAY_NONE, SS_LA_DECAY_HEAD, SS_LA_DECAY_TOKEN = 0, 1, 2
SS_Q8_NONE, SS_Q8_FP8, SS_Q8_INT8 = 0, 1, 2
SS_Q4_MX = 3
SS_GR_CKPT = 64

ERRORS = {0: "SS_OK", -1: "SS_ERR_NULL", -2: "SS_ERR_DIMS", -3: "SS_ERR_DTYPE", -4: "SS_ERR_ALIGN",
          -5: "SS_ERR_WORKSPACE", -6: "SS_ERR_HIP", -7: "SS_ERR_UNSUPPORTED", -8: "SS_ERR_SCRATCH"}

EXPORTS = ("ss_fwd", "ss_bwd", "ss_step", "ss_fwd_workspace_size", "ss_bwd_workspace_size",
           "ss_block_fwd", "ss_block_fwd_workspace_size", "ss_in_proj", "ss_strerror",
           "ss_last_hip_error", "ss_version", "ss_build_id", "ss_fwd_noalloc",
           "ss_la_fwd", "ss_la_bwd", "ss_la_step", "ss_la_fwd_workspace_size",
           "ss_la_bwd_workspace_size", "ss_rms_fwd", "ss_rms_bwd", "ss_rms_bwd_workspace_size",
           "ss_q4_mv", "ss_gr_fwd", "ss_gr_bwd", "ss_gr_step", "ss_gr_fwd_workspace_size",
           "ss_gr_bwd_workspace_size", "ss_ln_fwd", "ss_ln_bwd", "ss_ln_bwd_workspace_size",
           "ss_mx4_quant", "ss_mx4_mm")


class ss_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("in_dtype", ctypes.c_int32), ("plan", ctypes.c_int32),
                ("chunk", ctypes.c_int64), ("layout", ctypes.c_int32), ("disc", ctypes.c_int32),
                ("order", ctypes.c_int32), ("dt_layout", ctypes.c_int32)]


class ss_block_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("d_in", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("plan", ctypes.c_int32),
                ("layout", ctypes.c_int32)]


class ss_la_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("kheads", ctypes.c_int64), ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("q_stride", ctypes.c_int64 * 3), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3), ("in_dtype", ctypes.c_int32),
                ("decay", ctypes.c_int32), ("scale", ctypes.c_float)]


class ss_rms_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("q8", ctypes.c_int32), ("eps", ctypes.c_float)]


class ss_q4_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("group", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("x_q8", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32)]


class ss_gr_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("x_stride", ctypes.c_int64 * 2), ("r_stride", ctypes.c_int64 * 2),
                ("i_stride", ctypes.c_int64 * 2), ("in_dtype", ctypes.c_int32),
                ("c", ctypes.c_float)]


class ss_ln_dims(ctypes.Structure):
    _fields_ = list(ss_rms_dims._fields_)


class ss_mx4_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("x_q8", ctypes.c_int32), ("y_dtype", ctypes.c_int32)]


class SSError(RuntimeError):
    def __init__(self, code, lib=None):
        msg = ERRORS.get(code, str(code))
        if lib is not None:
            msg += ": " + lib.ss_strerror(code).decode()
            if code == -6:
                msg += f" (hipError {lib.ss_last_hip_error()})"
        super().__init__(msg)
        self.code = code


_lib = None


def load(path: str = LIB, expect: str = None):
    """Load libss.so (built in-tree by ``build()``).  Raises if it is missing, or if its build
    identity (ss_build_id) differs from ``expect`` (default: the digest of the sources in this
    tree, ``tree_id()``): a library built from other sources is never used."""
    global _lib
    if _lib is not None and expect is None and path == LIB:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"HIP library not built: {path} (run selective_state_space_34_amd.build())")
    lib = ctypes.CDLL(path)
    lib.ss_build_id.restype = ctypes.c_char_p
    got = lib.ss_build_id().decode()
    want = tree_id() if expect is None else expect
    if got != want:
        raise RuntimeError(f"{path} was built from other sources (library id {got[:16]}..., "
                           f"expected {want[:16]}...): rebuild it with build()")
    P = ctypes.c_void_p
    D = ctypes.POINTER(ss_dims)
    lib.ss_fwd.argtypes = [D] + [P] * 12 + [P, ctypes.c_size_t, P]
    lib.ss_fwd.restype = ctypes.c_int
    lib.ss_bwd.argtypes = [D] + [P] * 9 + [P, P, P] + [P] * 9 + [P, ctypes.c_size_t, P]
    lib.ss_bwd.restype = ctypes.c_int
    lib.ss_fwd_noalloc.argtypes = [D] + [P] * 12 + [P]
    lib.ss_fwd_noalloc.restype = ctypes.c_int
    lib.ss_step.argtypes = [D] + [P] * 12
    lib.ss_step.restype = ctypes.c_int
    for f in ("ss_fwd_workspace_size", "ss_bwd_workspace_size"):
        getattr(lib, f).argtypes = [D, ctypes.POINTER(ctypes.c_size_t)]
        getattr(lib, f).restype = ctypes.c_int
    BD = ctypes.POINTER(ss_block_dims)
    lib.ss_block_fwd.argtypes = [BD] + [P] * 14 + [P, ctypes.c_size_t, P]
    lib.ss_block_fwd.restype = ctypes.c_int
    lib.ss_block_fwd_workspace_size.argtypes = [BD, ctypes.POINTER(ctypes.c_size_t)]
    lib.ss_block_fwd_workspace_size.restype = ctypes.c_int
    lib.ss_in_proj.argtypes = [BD] + [P] * 5
    lib.ss_in_proj.restype = ctypes.c_int
    LD = ctypes.POINTER(ss_la_dims)
    lib.ss_la_fwd.argtypes = [LD] + [P] * 9 + [ctypes.c_size_t, P]
    lib.ss_la_fwd.restype = ctypes.c_int
    lib.ss_la_bwd.argtypes = [LD] + [P] * 14 + [ctypes.c_size_t, P]
    lib.ss_la_bwd.restype = ctypes.c_int
    lib.ss_la_step.argtypes = [LD] + [P] * 8
    lib.ss_la_step.restype = ctypes.c_int
    for f in ("ss_la_fwd_workspace_size", "ss_la_bwd_workspace_size"):
        getattr(lib, f).argtypes = [LD, ctypes.POINTER(ctypes.c_size_t)]
        getattr(lib, f).restype = ctypes.c_int
    RD = ctypes.POINTER(ss_rms_dims)
    lib.ss_rms_fwd.argtypes = [RD] + [P] * 7
    lib.ss_rms_fwd.restype = ctypes.c_int
    lib.ss_rms_bwd.argtypes = [RD] + [P] * 7 + [ctypes.c_size_t, P]
    lib.ss_rms_bwd.restype = ctypes.c_int
    lib.ss_rms_bwd_workspace_size.argtypes = [RD, ctypes.POINTER(ctypes.c_size_t)]
    lib.ss_rms_bwd_workspace_size.restype = ctypes.c_int
    lib.ss_q4_mv.argtypes = [ctypes.POINTER(ss_q4_dims)] + [P] * 7
    lib.ss_q4_mv.restype = ctypes.c_int
    GD = ctypes.POINTER(ss_gr_dims)
    lib.ss_gr_fwd.argtypes = [GD] + [P] * 11 + [ctypes.c_size_t, P]
    lib.ss_gr_fwd.restype = ctypes.c_int
    lib.ss_gr_bwd.argtypes = [GD] + [P] * 16 + [ctypes.c_size_t, P]
    lib.ss_gr_bwd.restype = ctypes.c_int
    lib.ss_gr_step.argtypes = [GD] + [P] * 8
    lib.ss_gr_step.restype = ctypes.c_int
    lib.ss_gr_fwd_workspace_size.argtypes = [GD, ctypes.POINTER(ctypes.c_size_t)]
    lib.ss_gr_fwd_workspace_size.restype = ctypes.c_int
    lib.ss_gr_bwd_workspace_size.argtypes = [GD, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
    lib.ss_gr_bwd_workspace_size.restype = ctypes.c_int
    ND = ctypes.POINTER(ss_ln_dims)
    lib.ss_ln_fwd.argtypes = [ND] + [P] * 8
    lib.ss_ln_fwd.restype = ctypes.c_int
    lib.ss_ln_bwd.argtypes = [ND] + [P] * 8 + [ctypes.c_size_t, P]
    lib.ss_ln_bwd.restype = ctypes.c_int
    lib.ss_ln_bwd_workspace_size.argtypes = [ND, ctypes.POINTER(ctypes.c_size_t)]
    lib.ss_ln_bwd_workspace_size.restype = ctypes.c_int
    MD = ctypes.POINTER(ss_mx4_dims)
    lib.ss_mx4_quant.argtypes = [MD] + [P] * 4
    lib.ss_mx4_quant.restype = ctypes.c_int
    lib.ss_mx4_mm.argtypes = [MD] + [P] * 6
    lib.ss_mx4_mm.restype = ctypes.c_int
    lib.ss_strerror.argtypes = [ctypes.c_int]
    lib.ss_strerror.restype = ctypes.c_char_p
    lib.ss_last_hip_error.restype = ctypes.c_int
    lib.ss_version.restype = ctypes.c_int
    if expect is None and path == LIB:
        _lib = lib
    return lib


def make_dims(batch, seqlen, dim, dstate, in_dtype=SS_F32, plan=SS_PLAN_AUTO, chunk=0,
              layout=SS_LAYOUT_AUTO, disc=SS_DISC_EULER, order=SS_ORDER_BDL, dt_layout=SS_DT_FULL):
    return ss_dims(batch, seqlen, dim, dstate, in_dtype, plan, chunk, layout, disc, order,
                   dt_layout)


def workspace_size(dims, backward=False) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    fn = lib.ss_bwd_workspace_size if backward else lib.ss_fwd_workspace_size
    rc = fn(ctypes.byref(dims), ctypes.byref(n))
    if rc != 0:
        raise SSError(rc, lib)
    return n.value


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, shape, dtype, device):
    if t is None:
        return
    try:  # what is right passes with the fewest steps: a call's checks are most of its host time
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _seq_shape(x, order):
    """(B, D, L) of a sequence tensor in the given order."""
    if x.dim() != 3:
        raise ValueError(f"x must be 3-D, got shape {tuple(x.shape)}")
    if order == SS_ORDER_BDL:
        return tuple(x.shape)
    if order == SS_ORDER_BLD:
        Bn, L, D = x.shape
        return Bn, D, L
    raise ValueError(f"order must be SS_ORDER_BDL or SS_ORDER_BLD, got {order}")


def _dims_of(x, A, dt_raw, plan, chunk, layout=SS_LAYOUT_AUTO, disc=SS_DISC_EULER,
             order=SS_ORDER_BDL):
    import torch
    Bn, D, L = _seq_shape(x, order)
    N = A.shape[1]
    if x.dtype == torch.float32:
        dt = SS_F32
    elif x.dtype == torch.bfloat16:
        dt = SS_BF16
    else:
        raise ValueError(f"x dtype must be float32 or bfloat16, got {x.dtype}")
    dtl = SS_DT_SHARED if dt_raw.dim() == 2 else SS_DT_FULL
    return make_dims(Bn, L, D, N, dt, plan, chunk, layout, disc, order, dtl)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _seq(Bn, D, L, order):
    return (Bn, D, L) if order == SS_ORDER_BDL else (Bn, L, D)


def _check_inputs(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, z, h0, order=SS_ORDER_BDL):
    """Shapes: x, z [B, D, L] ([B, L, D] token-major); dt_raw as x, or [B, L] (one value
    per token); Bm, Cm [B, N, L] ([B, L, N]); A [D, N]; dt_bias, Dskip [D]; h0 [B, D, N]."""
    import torch
    Bn, D, L = _seq_shape(x, order)
    N = A.shape[1]
    dev = x.device
    f32 = torch.float32
    _check(dt_raw, "dt_raw", (Bn, L) if dt_raw.dim() == 2 else _seq(Bn, D, L, order), x.dtype, dev)
    _check(z, "z", _seq(Bn, D, L, order), x.dtype, dev)
    _check(Bm, "Bm", _seq(Bn, N, L, order), x.dtype, dev)
    _check(Cm, "Cm", _seq(Bn, N, L, order), x.dtype, dev)
    _check(A, "A", (D, N), f32, dev)
    _check(dt_bias, "dt_bias", (D,), f32, dev)
    _check(Dskip, "Dskip", (D,), f32, dev)
    _check(h0, "h0", (Bn, D, N), f32, dev)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")


CKPT_STEPS = 16


def ss_fwd(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, z=None, h0=None, *, return_final=False,
           return_ckpt=False, y=None, h_final=None, h_ckpt=None, workspace=None,
           plan=SS_PLAN_AUTO, chunk=0, layout=SS_LAYOUT_AUTO, disc=SS_DISC_EULER,
           order=SS_ORDER_BDL, stream=None):
    """Forward scan through the C ABI.  Returns y, (y, h_final) with return_final, and
    the checkpoints last with return_ckpt (or when h_ckpt is passed).  disc: SS_DISC_EULER
    (input term δ·B·x) or SS_DISC_ZOH (exact zero-order hold).  order: SS_ORDER_BDL or
    SS_ORDER_BLD (token-major x, z, y, Bm, Cm); a 2-D dt_raw [B, L] is one value per token."""
    import torch
    lib = load()
    _check_inputs(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, z, h0, order)
    dims = _dims_of(x, A, dt_raw, plan, chunk, layout, disc, order)
    Bn, D, L = _seq_shape(x, order)
    N = A.shape[1]
    if y is None:
        y = torch.empty(_seq(Bn, D, L, order), dtype=torch.float32, device=x.device)
    _check(y, "y", _seq(Bn, D, L, order), torch.float32, x.device)
    if return_final and h_final is None:
        h_final = torch.empty((Bn, D, N), dtype=torch.float32, device=x.device)
    _check(h_final, "h_final", (Bn, D, N), torch.float32, x.device)
    nck = (L + CKPT_STEPS - 1) // CKPT_STEPS
    if return_ckpt and h_ckpt is None:
        h_ckpt = torch.empty((Bn, D, nck, N), dtype=torch.float32, device=x.device)
    _check(h_ckpt, "h_ckpt", (Bn, D, nck, N), torch.float32, x.device)
    need = workspace_size(dims)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.ss_fwd(ctypes.byref(dims), _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(Bm),
                    _ptr(Cm), _ptr(Dskip), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_final), _ptr(h_ckpt),
                    _ptr(workspace), wbytes, _stream(stream))
    if rc != 0:
        raise SSError(rc, lib)
    out = (y,)
    if return_final or h_final is not None:
        out += (h_final,)
    if h_ckpt is not None:
        out += (h_ckpt,)
    return out if len(out) > 1 else y


def ss_fwd_noalloc(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, y, z=None, h0=None, *, h_final=None,
                   h_ckpt=None, plan=SS_PLAN_AUTO, chunk=0, layout=SS_LAYOUT_AUTO,
                   disc=SS_DISC_EULER, order=SS_ORDER_BDL, stream=None):
    """ss_fwd without a workspace: the library's static scratch (SS_NOALLOC_SCRATCH_MIB MiB per
    GPU) serves the chunked and one-lane plans, and nothing is allocated, here or in the
    library.  The caller passes every output (y, and h_final / h_ckpt if wanted).  Calls that
    overlap on one GPU share that scratch and race; calls ordered on one stream do not."""
    import torch
    lib = load()
    _check_inputs(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, z, h0, order)
    dims = _dims_of(x, A, dt_raw, plan, chunk, layout, disc, order)
    Bn, D, L = _seq_shape(x, order)
    N = A.shape[1]
    if y is None:
        raise ValueError("y is required")
    _check(y, "y", _seq(Bn, D, L, order), torch.float32, x.device)
    _check(h_final, "h_final", (Bn, D, N), torch.float32, x.device)
    nck = (L + CKPT_STEPS - 1) // CKPT_STEPS
    _check(h_ckpt, "h_ckpt", (Bn, D, nck, N), torch.float32, x.device)
    rc = lib.ss_fwd_noalloc(ctypes.byref(dims), _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A),
                            _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z), _ptr(h0), _ptr(y),
                            _ptr(h_final), _ptr(h_ckpt), _stream(stream))
    if rc != 0:
        raise SSError(rc, lib)
    return y


def ss_bwd(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, dy, z=None, h0=None, dh_final=None, *,
           h_ckpt=None, workspace=None, chunk=0, order=SS_ORDER_BDL, disc=SS_DISC_EULER,
           out=None, stream=None):
    """Backward through the C ABI.  Returns a dict dx, ddt_raw, ddt_bias, dA, dB, dC, dD,
    dz (None without gate), dh0 (None without h0); all float32, each shaped like its input
    (order as in ss_fwd).  h_ckpt: the checkpoints of an ss_fwd call on the same inputs
    (optional; made with the same disc).  disc: the discretisation the forward used."""
    import torch
    lib = load()
    _check_inputs(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, z, h0, order)
    dims = _dims_of(x, A, dt_raw, SS_PLAN_CHUNKED, chunk, disc=disc, order=order)
    Bn, D, L = _seq_shape(x, order)
    N = A.shape[1]
    dev = x.device
    f32 = torch.float32
    sq = _seq(Bn, D, L, order)
    _check(dy, "dy", sq, f32, dev)
    _check(dh_final, "dh_final", (Bn, D, N), f32, dev)
    _check(h_ckpt, "h_ckpt", (Bn, D, (L + CKPT_STEPS - 1) // CKPT_STEPS, N), f32, dev)
    shapes = dict(dx=sq, ddt_raw=tuple(dt_raw.shape), ddt_bias=(D,), dA=(D, N),
                  dB=_seq(Bn, N, L, order), dC=_seq(Bn, N, L, order), dD=(D,), dz=sq,
                  dh0=(Bn, D, N))
    g = {} if out is None else dict(out)
    for k, shp in shapes.items():
        if (k == "dz" and z is None) or (k == "dh0" and h0 is None):
            g[k] = None
            continue
        if g.get(k) is None:
            g[k] = torch.empty(shp, dtype=f32, device=dev)
        _check(g[k], k, shp, f32, dev)
    need = workspace_size(dims, backward=True)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.ss_bwd(ctypes.byref(dims), _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(Bm),
                    _ptr(Cm), _ptr(Dskip), _ptr(z), _ptr(h0), _ptr(dy), _ptr(dh_final), _ptr(h_ckpt),
                    _ptr(g["dx"]), _ptr(g["ddt_raw"]), _ptr(g["ddt_bias"]), _ptr(g["dA"]),
                    _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["dz"]), _ptr(g["dh0"]),
                    _ptr(workspace), wbytes, _stream(stream))
    if rc != 0:
        raise SSError(rc, lib)
    return g


def ss_step(x, dt_raw, dt_bias, A, Bm, Cm, Dskip, h, z=None, *, h_out=None, y=None,
            disc=SS_DISC_EULER, stream=None):
    """One decode step through the C ABI: x, z [B, D]; dt_raw [B, D] or [B] (one value per
    token); Bm, Cm [B, N]; h [B, D, N]
    float32, the state before the token.  The state after it goes to h_out (default: h
    itself, updated in place).  Returns y [B, D] float32."""
    import torch
    lib = load()
    if x.dim() != 2:
        raise ValueError(f"x must be [B, D], got shape {tuple(x.shape)}")
    Bn, D = x.shape
    N = A.shape[1]
    dev = x.device
    f32 = torch.float32
    if x.dtype == torch.float32:
        dt = SS_F32
    elif x.dtype == torch.bfloat16:
        dt = SS_BF16
    else:
        raise ValueError(f"x dtype must be float32 or bfloat16, got {x.dtype}")
    _check(x, "x", (Bn, D), x.dtype, dev)
    _check(dt_raw, "dt_raw", (Bn,) if dt_raw.dim() == 1 else (Bn, D), x.dtype, dev)
    _check(z, "z", (Bn, D), x.dtype, dev)
    _check(Bm, "Bm", (Bn, N), x.dtype, dev)
    _check(Cm, "Cm", (Bn, N), x.dtype, dev)
    _check(A, "A", (D, N), f32, dev)
    _check(dt_bias, "dt_bias", (D,), f32, dev)
    _check(Dskip, "Dskip", (D,), f32, dev)
    _check(h, "h", (Bn, D, N), f32, dev)
    if h_out is None:
        h_out = h
    _check(h_out, "h_out", (Bn, D, N), f32, dev)
    if y is None:
        y = torch.empty((Bn, D), dtype=f32, device=dev)
    _check(y, "y", (Bn, D), f32, dev)
    dims = make_dims(Bn, 1, D, N, dt, disc=disc,
                     dt_layout=SS_DT_SHARED if dt_raw.dim() == 1 else SS_DT_FULL)
    rc = lib.ss_step(ctypes.byref(dims), _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(Bm),
                     _ptr(Cm), _ptr(Dskip), _ptr(z), _ptr(h), _ptr(h_out), _ptr(y), _stream(stream))
    if rc != 0:
        raise SSError(rc, lib)
    return y


def make_block_dims(batch, seqlen, d_in, dim, dstate, plan=SS_PLAN_AUTO, layout=SS_LAYOUT_AUTO):
    return ss_block_dims(batch, seqlen, d_in, dim, dstate, plan, layout)


def block_workspace_size(dims) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    rc = lib.ss_block_fwd_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != 0:
        raise SSError(rc, lib)
    return n.value


def ss_block_fwd(u, W_in, W_x, dt_bias, A, Dskip, h0=None, *, return_final=False,
                 return_proj=False, y=None, workspace=None, plan=SS_PLAN_AUTO,
                 layout=SS_LAYOUT_AUTO, stream=None):
    """Projections and gated scan through the C ABI: u [B, L, d_in] bf16, W_in [2D, d_in]
    bf16, W_x [1 + 2N, D] float32, dt_bias, Dskip [D], A [D, N], h0 [B, D, N] float32.
    Returns y [B, L, D] float32; with return_final also h_final [B, D, N]; with return_proj
    also a dict of the projections x, z [B, L, D], dt [B, L], B, C [B, L, N] (float32)."""
    import torch
    lib = load()
    if u.dim() != 3:
        raise ValueError(f"u must be [B, L, d_in], got shape {tuple(u.shape)}")
    Bn, L, Din = u.shape
    D, N = A.shape
    dev = u.device
    f32, bf = torch.float32, torch.bfloat16
    _check(u, "u", (Bn, L, Din), bf, dev)
    _check(W_in, "W_in", (2 * D, Din), bf, dev)
    _check(W_x, "W_x", (1 + 2 * N, D), f32, dev)
    _check(dt_bias, "dt_bias", (D,), f32, dev)
    _check(A, "A", (D, N), f32, dev)
    _check(Dskip, "Dskip", (D,), f32, dev)
    _check(h0, "h0", (Bn, D, N), f32, dev)
    dims = make_block_dims(Bn, L, Din, D, N, plan, layout)
    if y is None:
        y = torch.empty((Bn, L, D), dtype=f32, device=dev)
    _check(y, "y", (Bn, L, D), f32, dev)
    hf = torch.empty((Bn, D, N), dtype=f32, device=dev) if return_final else None
    proj = None
    if return_proj:
        proj = dict(x=torch.empty((Bn, L, D), dtype=f32, device=dev),
                    z=torch.empty((Bn, L, D), dtype=f32, device=dev),
                    dt=torch.empty((Bn, L), dtype=f32, device=dev),
                    B=torch.empty((Bn, L, N), dtype=f32, device=dev),
                    C=torch.empty((Bn, L, N), dtype=f32, device=dev))
    need = block_workspace_size(dims)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wbytes = workspace.numel() * workspace.element_size()
    g = (lambda k: None) if proj is None else (lambda k: _ptr(proj[k]))
    rc = lib.ss_block_fwd(ctypes.byref(dims), _ptr(u), _ptr(W_in), _ptr(W_x), _ptr(dt_bias),
                          _ptr(A), _ptr(Dskip), _ptr(h0), _ptr(y), _ptr(hf), g("x"), g("z"),
                          g("dt"), g("B"), g("C"), _ptr(workspace), wbytes, _stream(stream))
    if rc != 0:
        raise SSError(rc, lib)
    out = (y,)
    if return_final:
        out += (hf,)
    if return_proj:
        out += (proj,)
    return out if len(out) > 1 else y


def ss_in_proj(u, W_in, *, x=None, z=None, stream=None):
    """[x | z] = u · W_inᵀ through the C ABI: u [B, L, d_in] bf16, W_in [2D, d_in] bf16;
    returns x, z [B, L, D] float32."""
    import torch
    lib = load()
    Bn, L, Din = u.shape
    D = W_in.shape[0] // 2
    dev = u.device
    _check(u, "u", (Bn, L, Din), torch.bfloat16, dev)
    _check(W_in, "W_in", (2 * D, Din), torch.bfloat16, dev)
    if x is None:
        x = torch.empty((Bn, L, D), dtype=torch.float32, device=dev)
    if z is None:
        z = torch.empty((Bn, L, D), dtype=torch.float32, device=dev)
    _check(x, "x", (Bn, L, D), torch.float32, dev)
    _check(z, "z", (Bn, L, D), torch.float32, dev)
    dims = make_block_dims(Bn, L, Din, D, 1)
    rc = lib.ss_in_proj(ctypes.byref(dims), _ptr(u), _ptr(W_in), _ptr(x), _ptr(z), _stream(stream))
    if rc != 0:
        raise SSError(rc, lib)
    return x, z


# ---- linear attention with a decay for each head --------------------------------------------

_HERE = contextlib.nullcontext()


def _on(device, stream, used):
    """Context in which a call allocates and launches: the given stream (else the current one of
    the tensors' device).  Memory made inside belongs to that stream, and the tensors that come
    from elsewhere are recorded on it, so neither is handed out again while the call runs."""
    import torch
    if stream is None and device.index == torch.cuda.current_device():
        return _HERE
    s = torch.cuda.current_stream(device) if stream is None else stream
    if stream is not None:
        for t in used:
            if t is not None and t.is_cuda:
                t.record_stream(s)
    return torch.cuda.stream(s)


def _bytes(n, device):
    import torch
    return torch.empty(n, dtype=torch.uint8, device=device)


def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(device):
    """Handle of the device's current stream (without the Stream object where torch gives it)."""
    import torch
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(device).cuda_stream if get is None else get(device.index)


def _in_dtype(x, name):
    import torch
    if x.dtype == torch.bfloat16:
        return SS_BF16
    if x.dtype == torch.float32:
        return SS_F32
    raise ValueError(f"{name} dtype must be float32 or bfloat16, got {x.dtype}")


def make_la_dims(batch, seqlen, heads, kheads, dk, dv, in_dtype=SS_BF16,
                 decay=SS_LA_DECAY_TOKEN, scale=1.0, q_stride=(0, 0, 0), k_stride=(0, 0, 0),
                 v_stride=(0, 0, 0)):
    T3 = ctypes.c_int64 * 3
    return ss_la_dims(batch, seqlen, heads, kheads, dk, dv, T3(*q_stride), T3(*k_stride),
                      T3(*v_stride), in_dtype, decay, scale)


def la_workspace_size(dims, backward=False) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    fn = lib.ss_la_bwd_workspace_size if backward else lib.ss_la_fwd_workspace_size
    rc = fn(ctypes.byref(dims), ctypes.byref(n))
    if rc != 0:
        raise SSError(rc, lib)
    return n.value


@functools.lru_cache(maxsize=512)
def _la_plan(key, backward):
    """The dims structure of a call's shapes and strides, and the workspace they need."""
    dims = make_la_dims(*key)
    return dims, la_workspace_size(dims, backward)


def _la_rows(t, name, shape, dtype, device):
    """Checks a [.., head, width] input that may be strided; its element strides."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device or t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected {dtype} "
                         f"{shape} on {device}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: the last axis must be contiguous, got strides {st}")
    if not any(st[:-1]) and t.numel() > shape[-1]:
        raise ValueError(f"{name}: one row broadcast over every axis is not taken")
    return st[:-1]


def _la_key(q, k, v, g, s0, scale, lengths, step):
    """Checks the inputs that the three calls share; the key of their dims, and (B, T, H, dk, dv)."""
    import torch
    nd = 3 if step else 4
    if not isinstance(v, torch.Tensor) or not isinstance(q, torch.Tensor):
        raise TypeError("q, k, v must be torch.Tensors")
    if v.dim() != nd or q.dim() != nd:
        raise ValueError(f"q, k, v must be {nd}-D, got shapes {tuple(q.shape)}, {tuple(v.shape)}")
    dev, dt = v.device, v.dtype
    lead = tuple(v.shape[:-2])
    H, dv = v.shape[-2:]
    Hk, dk = q.shape[-2:]
    qs = _la_rows(q, "q", lead + (Hk, dk), dt, dev)
    ks = _la_rows(k, "k", lead + (Hk, dk), dt, dev)
    vs = _la_rows(v, "v", lead + (H, dv), dt, dev)
    B, T = (lead[0], 1) if step else lead
    if step:
        qs, ks, vs = ((s[0], s[0], s[1]) for s in (qs, ks, vs))
    f32 = torch.float32
    decay = SS_LA_DECAY_NONE
    if g is not None:
        decay = SS_LA_DECAY_HEAD if g.dim() == 1 else SS_LA_DECAY_TOKEN
        _check(g, "g", (H,) if g.dim() == 1 else lead + (H,), f32, dev)
    _check(s0, "s" if step else "s0", (B, H, dk, dv), f32, dev)
    _check(lengths, "lengths", (B,), torch.int32, dev)
    key = (B, T, H, Hk, dk, dv, _in_dtype(v, "v"), decay, float(scale), qs, ks, vs)
    return key, (B, T, H, dk, dv)


def ss_la_fwd(q, k, v, g=None, s0=None, *, scale=1.0, lengths=None, return_final=False, o=None,
              s_final=None, workspace=None, stream=None):
    """Linear attention over T tokens through the C ABI: S_t = e^{g_t} S_{t-1} + k_t v_tᵀ,
    o_t = scale · S_tᵀ q_t.  q, k [B, T, Hk, dk], v [B, T, H, dv] (float32 or bfloat16, may be
    strided slices with a contiguous last axis; H % Hk == 0), g None, [H] or [B, T, H] float32
    (natural log of the decay), s0 [B, H, dk, dv] float32, lengths [B] int32.  Returns o
    [B, T, H, dv] in v's type, or (o, s_final) with return_final (or when s_final is passed; it
    may be s0, updated in place)."""
    import torch
    lib = load()
    key, (B, T, H, dk, dv) = _la_key(q, k, v, g, s0, scale, lengths, False)
    dims, need = _la_plan(key, False)
    dev = v.device
    with _on(dev, stream, (q, k, v, g, s0, lengths, o, s_final, workspace)):
        if o is None:
            o = torch.empty((B, T, H, dv), dtype=v.dtype, device=dev)
        _check(o, "o", (B, T, H, dv), v.dtype, dev)
        if return_final and s_final is None:
            s_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
        _check(s_final, "s_final", (B, H, dk, dv), torch.float32, dev)
        if workspace is None and need > 0:
            workspace = _bytes(need, dev)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib.ss_la_fwd(dims, _addr(q), _addr(k), _addr(v), _addr(g), _addr(s0),
                           _addr(lengths), _addr(o), _addr(s_final), _addr(workspace), wbytes,
                           _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return o if s_final is None else (o, s_final)


def ss_la_bwd(q, k, v, do, g=None, s0=None, ds_final=None, *, scale=1.0, lengths=None,
              workspace=None, out=None, stream=None):
    """Gradients of ss_la_fwd through the C ABI: do [B, T, H, dv] in v's type, ds_final
    [B, H, dk, dv] float32.  Returns a dict dq, dk, dv (the inputs' type), dg (float32, shaped
    like g; None without decay), ds0 (None without s0).  out: a dict of tensors to take them; its
    ds0 may be ds_final."""
    import torch
    lib = load()
    key, (B, T, H, dk, dv) = _la_key(q, k, v, g, s0, scale, lengths, False)
    dims, need = _la_plan(key, True)
    dev, dt, f32 = v.device, v.dtype, torch.float32
    _check(do, "do", (B, T, H, dv), dt, dev)
    _check(ds_final, "ds_final", (B, H, dk, dv), f32, dev)
    shapes = dict(dq=(tuple(q.shape), dt), dk=(tuple(q.shape), dt), dv=(tuple(v.shape), dt),
                  dg=None if g is None else (tuple(g.shape), f32),
                  ds0=None if s0 is None else ((B, H, dk, dv), f32))
    r = {} if out is None else dict(out)
    with _on(dev, stream, (q, k, v, do, g, s0, ds_final, lengths, workspace, *r.values())):
        for name, want in shapes.items():
            if want is None:
                r[name] = None
                continue
            if r.get(name) is None:
                r[name] = torch.empty(want[0], dtype=want[1], device=dev)
            _check(r[name], name, want[0], want[1], dev)
        if workspace is None and need > 0:
            workspace = _bytes(need, dev)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib.ss_la_bwd(dims, _addr(q), _addr(k), _addr(v), _addr(g), _addr(s0),
                           _addr(lengths), _addr(do), _addr(ds_final), _addr(r["dq"]),
                           _addr(r["dk"]), _addr(r["dv"]), _addr(r["dg"]), _addr(r["ds0"]),
                           _addr(workspace), wbytes, _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return r


def ss_la_step(q, k, v, s, g=None, *, scale=1.0, s_out=None, o=None, stream=None):
    """One token through the C ABI: q, k [B, Hk, dk], v [B, H, dv], g None, [H] or [B, H], s
    [B, H, dk, dv] float32, the state before the token.  The state after it goes to s_out
    (default: s itself, updated in place).  Returns o [B, H, dv] in v's type."""
    import torch
    lib = load()
    key, (B, _, H, dk, dv) = _la_key(q, k, v, g, s, scale, None, True)
    dims, _ = _la_plan(key, False)
    dev = v.device
    with _on(dev, stream, (q, k, v, g, s, s_out, o)):
        if s_out is None:
            s_out = s
        else:
            _check(s_out, "s_out", (B, H, dk, dv), torch.float32, dev)
        if o is None:
            o = torch.empty((B, H, dv), dtype=v.dtype, device=dev)
        else:
            _check(o, "o", (B, H, dv), v.dtype, dev)
        rc = lib.ss_la_step(dims, _addr(q), _addr(k), _addr(v), _addr(g), _addr(s), _addr(s_out),
                            _addr(o), _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return o


# ---- root-mean-square norm with the residual's addition, in 8 bits where asked -----------------

def make_rms_dims(rows, dim, in_dtype=SS_BF16, res_dtype=SS_BF16, q8=SS_Q8_NONE, eps=1e-5):
    return ss_rms_dims(rows, dim, in_dtype, res_dtype, q8, eps)


def rms_workspace_size(dims) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    rc = lib.ss_rms_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != 0:
        raise SSError(rc, lib)
    return n.value


@functools.lru_cache(maxsize=512)
def _rms_plan(key, backward):
    dims = make_rms_dims(*key)
    return dims, rms_workspace_size(dims) if backward else 0


def _rows_of(x, name):
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError(f"{name} must have rows and a width, got shape {tuple(x.shape)}")
    D = x.shape[-1]
    return x.numel() // D, D


def ss_rms_fwd(x, w, res=None, *, eps=1e-5, q8=SS_Q8_NONE, y=None, y_scale=None, r=None,
               stream=None):
    """y = r / sqrt(mean(r²) + eps) · w with r = x + res, over the last axis, through the C ABI.
    x [..., D] float32 or bfloat16; res like x, or float32; w [D] float32.  y has x's type, or
    with q8 = SS_Q8_FP8 / SS_Q8_INT8 it holds float8_e4m3fn / int8 codes with y_scale [...]
    float32, y ≈ code · y_scale.  r (default new; may be res) takes the sum, in res's type.
    Returns y, followed by y_scale with q8 and by r with res."""
    import torch
    lib = load()
    M, D = _rows_of(x, "x")
    dev, shape, f32 = x.device, tuple(x.shape), torch.float32
    dt = _in_dtype(x, "x")
    _check(x, "x", shape, x.dtype, dev)
    _check(w, "w", (D,), f32, dev)
    rdt = x.dtype if res is None else res.dtype
    _check(res, "res", shape, rdt, dev)
    dims, _ = _rms_plan((M, D, dt, dt if res is None else _in_dtype(res, "res"), q8, float(eps)), False)
    with _on(dev, stream, (x, w, res, y, y_scale, r)):
        yt = {SS_Q8_FP8: torch.float8_e4m3fn, SS_Q8_INT8: torch.int8}.get(q8, x.dtype)
        if y is None:
            y = torch.empty(shape, dtype=yt, device=dev)
        else:
            _check(y, "y", shape, yt, dev)
        if q8 != SS_Q8_NONE:
            if y_scale is None:
                y_scale = torch.empty(shape[:-1], dtype=f32, device=dev)
            else:
                _check(y_scale, "y_scale", shape[:-1], f32, dev)
        if res is not None:
            if r is None:
                r = torch.empty(shape, dtype=rdt, device=dev)
            else:
                _check(r, "r", shape, rdt, dev)
        rc = lib.ss_rms_fwd(dims, _addr(x), _addr(res), _addr(w), _addr(r), _addr(y),
                            _addr(y_scale), _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    out = (y,) if q8 == SS_Q8_NONE else (y, y_scale)
    if res is not None:
        out += (r,)
    return out if len(out) > 1 else y


def ss_rms_bwd(dy, r, w, dr=None, *, eps=1e-5, dx=None, dw=None, workspace=None, stream=None):
    """Gradients of ss_rms_fwd through the C ABI: dy [..., D] (the forward's x's type), r [..., D]
    the sum the forward returned (its x without a residual), dr like r, the gradient of r where
    it goes on beside the norm.  Returns dx (like r: the gradient of x and of res) and dw [D]
    float32."""
    import torch
    lib = load()
    M, D = _rows_of(r, "r")
    dev, shape, f32 = r.device, tuple(r.shape), torch.float32
    _check(r, "r", shape, r.dtype, dev)
    _check(dy, "dy", shape, dy.dtype, dev)
    _check(w, "w", (D,), f32, dev)
    _check(dr, "dr", shape, r.dtype, dev)
    dims, need = _rms_plan((M, D, _in_dtype(dy, "dy"), _in_dtype(r, "r"), SS_Q8_NONE, float(eps)), True)
    with _on(dev, stream, (dy, r, w, dr, dx, dw, workspace)):
        if dx is None:
            dx = torch.empty(shape, dtype=r.dtype, device=dev)
        else:
            _check(dx, "dx", shape, r.dtype, dev)
        if dw is None:
            dw = torch.empty((D,), dtype=f32, device=dev)
        else:
            _check(dw, "dw", (D,), f32, dev)
        if workspace is None:
            workspace = _bytes(need, dev)
        wbytes = workspace.numel() * workspace.element_size()
        rc = lib.ss_rms_bwd(dims, _addr(dy), _addr(r), _addr(w), _addr(dr), _addr(dx), _addr(dw),
                            _addr(workspace), wbytes, _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return dx, dw


# ---- products with 4-bit weights ---------------------------------------------------------------

def make_q4_dims(rows, n, k, group=128, in_dtype=SS_BF16, x_q8=SS_Q8_NONE, y_dtype=SS_BF16):
    return ss_q4_dims(rows, n, k, group, in_dtype, x_q8, y_dtype)


@functools.lru_cache(maxsize=512)
def _q4_plan(key):
    return make_q4_dims(*key)


def ss_q4_mv(x, wq, scales, zeros=None, *, group=128, x_scale=None, y=None, y_dtype=None,
             stream=None):
    """y = x · Wᵀ with W[i, j] = scales[i, j // group] · (u[i, j] - zeros[i, j // group]) through
    the C ABI.  x [..., K] float32 or bfloat16, or float8_e4m3fn or int8 with x_scale [...]
    float32; wq [N, K / 2] uint8, two codes a byte, the first in the low half; scales
    [N, ceil(K / group)] bfloat16; zeros the same in uint8 (None: 8).  Returns y [..., N], in
    y_dtype (default: float32 for float32 x, else bfloat16)."""
    import torch
    lib = load()
    M, K = _rows_of(x, "x")
    dev, lead = x.device, tuple(x.shape[:-1])
    q8 = {torch.float8_e4m3fn: SS_Q8_FP8, torch.int8: SS_Q8_INT8}.get(x.dtype, SS_Q8_NONE)
    dt = SS_BF16 if q8 else _in_dtype(x, "x")
    if (x_scale is not None) != (q8 != SS_Q8_NONE):
        raise ValueError("x_scale goes with 8-bit x, and only with it")
    if y is not None:
        y_dtype = y.dtype
    elif y_dtype is None:
        y_dtype = torch.float32 if x.dtype == torch.float32 else torch.bfloat16
    if wq.dim() != 2 or group <= 0:
        raise ValueError(f"wq must be [N, K / 2] and group positive, got {tuple(wq.shape)}, {group}")
    N, ng = wq.shape[0], -(-K // group)
    _check(x, "x", (*lead, K), x.dtype, dev)
    _check(wq, "wq", (N, K // 2), torch.uint8, dev)
    _check(scales, "scales", (N, ng), torch.bfloat16, dev)
    _check(zeros, "zeros", (N, ng), torch.uint8, dev)
    _check(x_scale, "x_scale", lead, torch.float32, dev)
    if y_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"y dtype must be float32 or bfloat16, got {y_dtype}")
    dims = _q4_plan((M, N, K, group, dt, q8, SS_F32 if y_dtype == torch.float32 else SS_BF16))
    with _on(dev, stream, (x, wq, scales, zeros, x_scale, y)):
        if y is None:
            y = torch.empty((*lead, N), dtype=y_dtype, device=dev)
        else:
            _check(y, "y", (*lead, N), y_dtype, dev)
        rc = lib.ss_q4_mv(dims, _addr(x), _addr(x_scale), _addr(wq), _addr(scales), _addr(zeros),
                          _addr(y), _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return y


# ---- gated linear recurrence -------------------------------------------------------------------

def make_gr_dims(batch, seqlen, dim, in_dtype=SS_BF16, c=8.0, x_stride=(0, 0), r_stride=(0, 0),
                 i_stride=(0, 0)):
    T2 = ctypes.c_int64 * 2
    return ss_gr_dims(batch, seqlen, dim, T2(*x_stride), T2(*r_stride), T2(*i_stride), in_dtype, c)


def gr_workspace_size(dims, backward=False, given_ckpt=False) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    if backward:
        rc = lib.ss_gr_bwd_workspace_size(ctypes.byref(dims), int(given_ckpt), ctypes.byref(n))
    else:
        rc = lib.ss_gr_fwd_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != 0:
        raise SSError(rc, lib)
    return n.value


@functools.lru_cache(maxsize=512)
def _gr_plan(key, backward, given_ckpt):
    """The dims structure of a call's shapes and strides, and the workspace they need."""
    dims = make_gr_dims(*key)
    return dims, gr_workspace_size(dims, backward, given_ckpt)


def _gr_rows(t, name, shape, dtype, device):
    """Checks an operand [B, T, D] (the step's [B, D]) that may be strided; its strides of batch
    row and token."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device or t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected {dtype} "
                         f"{tuple(shape)} on {device}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}: the last axis must be contiguous, got strides {st}")
    if not any(st[:-1]) and t.numel() > shape[-1]:
        raise ValueError(f"{name}: one row broadcast over every axis is not taken")
    return st[:2] if len(st) == 3 else (st[0], st[0])


def _gr_key(x, r, i, lam, c, step):
    """Checks the inputs that the three calls share; the key of their dims, and (B, T, D)."""
    import torch
    nd = 2 if step else 3
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() != nd or x.numel() == 0:
        raise ValueError(f"x must be {nd}-D and hold something, got shape {tuple(x.shape)}")
    dev, dt, shape = x.device, x.dtype, x.shape
    B, T, D = (shape[0], 1, shape[1]) if step else shape
    _check(lam, "lam", (D,), torch.float32, dev)
    sx = x.stride()
    try:  # operands laid out alike pass with the fewest steps, as in _check
        if (sx[-1] == 1 and sx[0] and sx[-2] and r.stride() == sx and i.stride() == sx and r.shape == shape
                and i.shape == shape and r.dtype is dt and i.dtype is dt and r.device == dev and i.device == dev):
            sx = sx[:2] if nd == 3 else (sx[0], sx[0])
            return (B, T, D, _in_dtype(x, "x"), float(c), sx, sx, sx), (B, T, D)
    except AttributeError:
        pass
    return (B, T, D, _in_dtype(x, "x"), float(c), _gr_rows(x, "x", shape, dt, dev),
            _gr_rows(r, "r", shape, dt, dev), _gr_rows(i, "i", shape, dt, dev)), (B, T, D)


def _gr_marks(lengths, reset, B, T, device):
    import torch
    _check(lengths, "lengths", (B,), torch.int32, device)
    if reset is not None:
        if getattr(reset, "dtype", None) not in (torch.bool, torch.uint8):
            raise ValueError("reset must be a bool or uint8 tensor")
        _check(reset, "reset", (B, T), reset.dtype, device)


def _check_workspace(t, device):
    """A workspace's size is taken from its elements, so they have to be memory of the call's own device and
    all there."""
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"workspace is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")


def ss_gr_fwd(x, r, i, lam, h0=None, *, c=8.0, lengths=None, reset=None, return_final=False,
              return_ckpt=False, y=None, h_final=None, h_ckpt=None, workspace=None, stream=None):
    """Gated linear recurrence through the C ABI: a_t = exp(-c softplus(lam) sigmoid(r_t)),
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, y_t = h_t.  x, r, i [B, T, D] (float32 or
    bfloat16, may be strided slices with a contiguous last axis), lam [D], h0 [B, D] float32,
    lengths [B] int32, reset [B, T] bool or uint8 (tokens that begin a document).  Returns y
    [B, T, D] in x's type, followed by h_final [B, D] with return_final (or when h_final is passed;
    it may be h0, updated in place) and by h_ckpt [B, ceil(T / 64), D], the states that enter every
    64th token, with return_ckpt (or when h_ckpt is passed)."""
    import torch
    lib = load()
    key, (B, T, D) = _gr_key(x, r, i, lam, c, False)
    dims, need = _gr_plan(key, False, False)
    dev, f32 = x.device, torch.float32
    _check(h0, "h0", (B, D), f32, dev)
    _gr_marks(lengths, reset, B, T, dev)
    _check_workspace(workspace, dev)
    with _on(dev, stream, (x, r, i, lam, h0, lengths, reset, y, h_final, h_ckpt, workspace)):
        if y is None:
            y = x.new_empty((B, T, D))
        else:
            _check(y, "y", (B, T, D), x.dtype, dev)
        if return_final and h_final is None:
            h_final = lam.new_empty((B, D))
        else:
            _check(h_final, "h_final", (B, D), f32, dev)
        nc = -(-T // SS_GR_CKPT)
        if return_ckpt and h_ckpt is None:
            h_ckpt = lam.new_empty((B, nc, D))
        else:
            _check(h_ckpt, "h_ckpt", (B, nc, D), f32, dev)
        if workspace is None and need > 0:
            workspace = _bytes(need, dev)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        rc = lib.ss_gr_fwd(dims, _addr(x), _addr(r), _addr(i), _addr(lam), _addr(h0),
                           _addr(lengths), _addr(reset), _addr(y), _addr(h_final), _addr(h_ckpt),
                           _addr(workspace), wbytes, _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    out = (y,) + ((h_final,) if h_final is not None else ()) + ((h_ckpt,) if h_ckpt is not None else ())
    return out if len(out) > 1 else y


def ss_gr_bwd(x, r, i, lam, dy, h0=None, dh_final=None, *, c=8.0, lengths=None, reset=None,
              h_ckpt=None, workspace=None, out=None, stream=None):
    """Gradients of ss_gr_fwd through the C ABI: dy [B, T, D] in x's type, dh_final [B, D] float32;
    h_ckpt as the forward gave it for the same inputs (None: the states are formed once more).
    Returns a dict dx, dr, di (x's type, dense), dlam [D], dh0 [B, D] (None without h0), float32.
    out: a dict of tensors to take them; its dh0 may be dh_final."""
    import torch
    lib = load()
    key, (B, T, D) = _gr_key(x, r, i, lam, c, False)
    dims, need = _gr_plan(key, True, h_ckpt is not None)
    dev, dt, f32 = x.device, x.dtype, torch.float32
    _check(dy, "dy", (B, T, D), dt, dev)
    _check(h0, "h0", (B, D), f32, dev)
    _check(dh_final, "dh_final", (B, D), f32, dev)
    _check(h_ckpt, "h_ckpt", (B, -(-T // SS_GR_CKPT), D), f32, dev)
    _gr_marks(lengths, reset, B, T, dev)
    _check_workspace(workspace, dev)
    g = {} if out is None else dict(out)
    with _on(dev, stream, (x, r, i, lam, dy, h0, dh_final, lengths, reset, h_ckpt, workspace,
                           *g.values())):
        for name, like in (("dx", dy), ("dr", dy), ("di", dy), ("dlam", lam), ("dh0", h0)):
            if like is None:
                g[name] = None
            elif g.get(name) is None:
                g[name] = torch.empty_like(like)
            else:
                _check(g[name], name, like.shape, like.dtype, dev)
        if workspace is None:
            workspace = _bytes(need, dev)
        wbytes = workspace.numel() * workspace.element_size()
        rc = lib.ss_gr_bwd(dims, _addr(x), _addr(r), _addr(i), _addr(lam), _addr(h0),
                           _addr(lengths), _addr(reset), _addr(dy), _addr(dh_final),
                           _addr(h_ckpt), _addr(g["dx"]), _addr(g["dr"]), _addr(g["di"]),
                           _addr(g["dlam"]), _addr(g["dh0"]), _addr(workspace), wbytes,
                           _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return g


def ss_gr_step(x, r, i, lam, h, *, c=8.0, h_out=None, y=None, stream=None):
    """One token through the C ABI: x, r, i [B, D], h [B, D] float32, the state before the token.
    The state after it goes to h_out (default: h itself, updated in place).  Returns y [B, D] in
    x's type."""
    import torch
    lib = load()
    key, (B, _, D) = _gr_key(x, r, i, lam, c, True)
    dims, _ = _gr_plan(key, False, False)
    dev = x.device
    if h is None:
        raise TypeError("h must be a torch.Tensor")
    _check(h, "h", (B, D), torch.float32, dev)
    with _on(dev, stream, (x, r, i, lam, h, h_out, y)):
        if h_out is None:
            h_out = h
        else:
            _check(h_out, "h_out", (B, D), torch.float32, dev)
        if y is None:
            y = torch.empty_like(h, dtype=x.dtype)
        else:
            _check(y, "y", (B, D), x.dtype, dev)
        rc = lib.ss_gr_step(dims, _addr(x), _addr(r), _addr(i), _addr(lam), _addr(h), _addr(h_out),
                            _addr(y), _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return y


# ---- layer norm with the residual's addition -----------------------------------------------------

def make_ln_dims(rows, dim, in_dtype=SS_BF16, res_dtype=SS_BF16, q8=SS_Q8_NONE, eps=1e-5):
    return ss_ln_dims(rows, dim, in_dtype, res_dtype, q8, eps)


def ln_workspace_size(dims) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    rc = lib.ss_ln_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != 0:
        raise SSError(rc, lib)
    return n.value


@functools.lru_cache(maxsize=512)
def _ln_plan(key, backward):
    dims = make_ln_dims(*key)
    return dims, ln_workspace_size(dims) if backward else 0


def ss_ln_fwd(x, w, b=None, res=None, *, eps=1e-5, q8=SS_Q8_NONE, y=None, y_scale=None, r=None,
              stream=None):
    """y = (r - mean(r)) / sqrt(var(r) + eps) · w + b with r = x + res, over the last axis, through
    the C ABI; types and returns as for ss_rms_fwd.  With q8 = SS_Q4_MX (D a multiple of 32) y holds
    codes [..., D / 2] and y_scale exponents [..., D / 32], both uint8, as ss_mx4_quant gives
    them."""
    import torch
    lib = load()
    M, D = _rows_of(x, "x")
    dev, shape, f32, u8 = x.device, x.shape, torch.float32, torch.uint8
    dt = _in_dtype(x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    _check(w, "w", (D,), f32, dev)
    _check(b, "b", (D,), f32, dev)
    rdt = x.dtype if res is None else res.dtype
    _check(res, "res", shape, rdt, dev)
    dims, _ = _ln_plan((M, D, dt, dt if res is None else _in_dtype(res, "res"), q8, float(eps)), False)
    with _on(dev, stream, (x, w, b, res, y, y_scale, r)):
        if q8 == SS_Q4_MX:
            if D % 32 != 0:
                raise ValueError(f"blocks of 32 need a width that is a multiple of 32, got {D}")
            ys, yt, ss, st = (*shape[:-1], D // 2), u8, (*shape[:-1], D // 32), u8
        else:
            yt = (x.dtype if q8 == SS_Q8_NONE else torch.float8_e4m3fn if q8 == SS_Q8_FP8 else torch.int8)
            ys, ss, st = shape, shape[:-1], f32
        if y is None:
            y = x.new_empty(ys, dtype=yt) if q8 == SS_Q4_MX else torch.empty_like(x, dtype=yt)
        else:
            _check(y, "y", ys, yt, dev)
        if q8 != SS_Q8_NONE:
            if y_scale is None:
                y_scale = x.new_empty(ss, dtype=st)
            else:
                _check(y_scale, "y_scale", ss, st, dev)
        if res is not None:
            if r is None:
                r = torch.empty_like(res)
            else:
                _check(r, "r", shape, rdt, dev)
        rc = lib.ss_ln_fwd(dims, _addr(x), _addr(res), _addr(w), _addr(b), _addr(r), _addr(y),
                           _addr(y_scale), _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    out = (y,) if q8 == SS_Q8_NONE else (y, y_scale)
    if res is not None:
        out += (r,)
    return out if len(out) > 1 else y


def ss_ln_bwd(dy, r, w, dr=None, *, eps=1e-5, bias=True, dx=None, dw=None, db=None,
              workspace=None, stream=None):
    """Gradients of ss_ln_fwd through the C ABI, as ss_rms_bwd's.  Returns dx (like r: the gradient
    of x and of res), dw [D] and db [D] float32 (None where bias is false)."""
    import torch
    lib = load()
    M, D = _rows_of(r, "r")
    dev, shape, f32 = r.device, r.shape, torch.float32
    if not r.is_contiguous():
        raise ValueError("r must be contiguous")
    _check(dy, "dy", shape, dy.dtype, dev)
    _check(w, "w", (D,), f32, dev)
    _check(dr, "dr", shape, r.dtype, dev)
    dims, need = _ln_plan((M, D, _in_dtype(dy, "dy"), _in_dtype(r, "r"), SS_Q8_NONE, float(eps)), True)
    if db is not None and not bias:
        raise ValueError("db goes with bias=True")
    _check_workspace(workspace, dev)
    with _on(dev, stream, (dy, r, w, dr, dx, dw, db, workspace)):
        if dx is None:
            dx = torch.empty_like(r)
        else:
            _check(dx, "dx", shape, r.dtype, dev)
        if dw is None:
            dw = torch.empty_like(w)
        else:
            _check(dw, "dw", (D,), f32, dev)
        if db is None and bias:
            db = torch.empty_like(w)
        else:
            _check(db, "db", (D,), f32, dev)
        if workspace is None:
            workspace = _bytes(need, dev)
        wbytes = workspace.numel() * workspace.element_size()
        rc = lib.ss_ln_bwd(dims, _addr(dy), _addr(r), _addr(w), _addr(dr), _addr(dx), _addr(dw),
                           _addr(db), _addr(workspace), wbytes, _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return dx, dw, db


# ---- microscaled 4-bit values and their products ---------------------------------------------------

def make_mx4_dims(rows, n, k, in_dtype=SS_BF16, x_q8=SS_Q4_MX, y_dtype=SS_BF16):
    return ss_mx4_dims(rows, n, k, in_dtype, x_q8, y_dtype)


@functools.lru_cache(maxsize=512)
def _mx4_plan(key):
    return make_mx4_dims(*key)


def ss_mx4_quant(x, *, codes=None, exps=None, stream=None):
    """x [..., K] (float32 or bfloat16, K a multiple of 32) in 4 bits with a power of two for every
    32 columns, through the C ABI: codes [..., K / 2] uint8, two e2m1 codes a byte, the first in the
    low half, and exponents exps [..., K / 32] uint8."""
    import torch
    lib = load()
    M, K = _rows_of(x, "x")
    dev, lead, u8 = x.device, x.shape[:-1], torch.uint8
    dt = _in_dtype(x, "x")
    if K % 32 != 0:
        raise ValueError(f"blocks of 32 need a width that is a multiple of 32, got {K}")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    dims = _mx4_plan((M, 1, K, dt))
    with _on(dev, stream, (x, codes, exps)):
        if codes is None:
            codes = x.new_empty((*lead, K // 2), dtype=u8)
        else:
            _check(codes, "codes", (*lead, K // 2), u8, dev)
        if exps is None:
            exps = x.new_empty((*lead, K // 32), dtype=u8)
        else:
            _check(exps, "exps", (*lead, K // 32), u8, dev)
        rc = lib.ss_mx4_quant(dims, _addr(x), _addr(codes), _addr(exps), _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return codes, exps


def ss_mx4_mm(x, x_scale, wq, w_exps, *, y=None, y_dtype=None, stream=None):
    """y = x · Wᵀ through the C ABI, W in ss_mx4_quant's format: wq [N, K / 2], w_exps [N, K / 32]
    uint8.  x is in it too (codes [..., K / 2], x_scale its exponents [..., K / 32]), or
    float8_e4m3fn [..., K] with x_scale [...] float32 as the norms give it.  Returns y [..., N] in
    y_dtype (default bfloat16)."""
    import torch
    lib = load()
    dev, u8 = x.device, torch.uint8
    lead = x.shape[:-1]
    M, K = _rows_of(x, "x")
    if x.dtype == u8:
        K *= 2
        q8 = SS_Q4_MX
        _check(x_scale, "x_scale", (*lead, K // 32), u8, dev)
    elif x.dtype == torch.float8_e4m3fn:
        q8 = SS_Q8_FP8
        _check(x_scale, "x_scale", lead, torch.float32, dev)
    else:
        raise ValueError(f"x must be uint8 codes or float8_e4m3fn, got {x.dtype}")
    if x_scale is None:
        raise TypeError("x_scale must be a torch.Tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if wq.dim() != 2:
        raise ValueError(f"wq must be [N, K / 2], got {tuple(wq.shape)}")
    N = wq.shape[0]
    _check(wq, "wq", (N, K // 2), u8, dev)
    _check(w_exps, "w_exps", (N, K // 32), u8, dev)
    if y is not None:
        y_dtype = y.dtype
    elif y_dtype is None:
        y_dtype = torch.bfloat16
    if y_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"y dtype must be float32 or bfloat16, got {y_dtype}")
    dims = _mx4_plan((M, N, K, SS_BF16, q8, SS_F32 if y_dtype == torch.float32 else SS_BF16))
    with _on(dev, stream, (x, x_scale, wq, w_exps, y)):
        if y is None:
            y = x.new_empty((*lead, N), dtype=y_dtype)
        else:
            _check(y, "y", (*lead, N), y_dtype, dev)
        rc = lib.ss_mx4_mm(dims, _addr(x), _addr(x_scale), _addr(wq), _addr(w_exps), _addr(y),
                           _raw_stream(dev))
    if rc != 0:
        raise SSError(rc, lib)
    return y
