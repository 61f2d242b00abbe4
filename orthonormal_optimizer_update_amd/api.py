"""Python binding of libortho.so (argument marshalling only).

Every step of the computation runs in the library's HIP kernels; this module
only turns torch tensors into ``ortho_mat`` descriptors (device pointer, rows,
cols, leading dimension, dtype), sizes the workspace, and passes torch's
current HIP stream.  It raises if the library has not been built -- there is no
fallback path.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libortho.so")

ORTHO_F32, ORTHO_BF16, ORTHO_E4M3, ORTHO_E8M0 = 0, 1, 2, 3
FP8_BLOCK = 128
ORTHO_E_SCRATCH = 9
NOALLOC_SCRATCH_BYTES = 64 << 20
DEV_CHOL_SHIFT, DEV_ZERO_COLUMN = 1, 2
MUON_ABC = (3.4445, -4.7750, 2.0315)


class OrthoMat(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class OrthoError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed with status {status}: {text}")
        self.status = status


_lib = None

_SIGS = {
    "ortho_dion_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]),
    "ortho_ns_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]),
    "dion_step": (ctypes.c_int, [OrthoMat, OrthoMat, OrthoMat, OrthoMat, ctypes.c_int32, ctypes.c_float,
                                 ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "dion_step_ex": (ctypes.c_int, [OrthoMat, OrthoMat, OrthoMat, OrthoMat, ctypes.c_int32, ctypes.c_float,
                                    ctypes.c_float, ctypes.c_float, ctypes.POINTER(OrthoMat),
                                    ctypes.POINTER(OrthoMat), ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]),
    "dion_step_batched": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(OrthoMat), ctypes.POINTER(OrthoMat),
                                         ctypes.POINTER(OrthoMat), ctypes.POINTER(OrthoMat), ctypes.c_int32,
                                         ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "newton_schulz": (ctypes.c_int, [OrthoMat, OrthoMat, ctypes.c_int32, ctypes.POINTER(ctypes.c_float),
                                     ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "newton_schulz_batched": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(OrthoMat), ctypes.POINTER(OrthoMat),
                                             ctypes.c_int32, ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                             ctypes.c_size_t, ctypes.c_void_p]),
    "ortho_muon_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]),
    "muon_step": (ctypes.c_int, [OrthoMat, OrthoMat, OrthoMat, ctypes.c_int32, ctypes.POINTER(ctypes.c_float),
                                 ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
                                 ctypes.c_size_t, ctypes.c_void_p]),
    "muon_step_batched": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(OrthoMat), ctypes.POINTER(OrthoMat),
                                         ctypes.POINTER(OrthoMat), ctypes.c_int32,
                                         ctypes.POINTER(ctypes.c_float), ctypes.c_float, ctypes.c_float,
                                         ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "ortho_normuon_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]),
    "normuon_step": (ctypes.c_int, [OrthoMat, OrthoMat, OrthoMat, ctypes.c_int32, ctypes.POINTER(ctypes.c_float),
                                    ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]),
    "normuon_step_batched": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(OrthoMat), ctypes.POINTER(OrthoMat),
                                            ctypes.POINTER(OrthoMat), ctypes.c_int32,
                                            ctypes.POINTER(ctypes.c_float), ctypes.c_float, ctypes.c_float,
                                            ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "dion_step_noalloc": (ctypes.c_int, [OrthoMat, OrthoMat, OrthoMat, OrthoMat, ctypes.c_int32,
                                         ctypes.c_float, ctypes.c_float, ctypes.c_void_p]),
    "ortho_dion2_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]),
    "dion2_step": (ctypes.c_int, [OrthoMat, OrthoMat, OrthoMat, ctypes.c_int32, ctypes.c_int32,
                                  ctypes.POINTER(ctypes.c_float), ctypes.c_float, ctypes.c_float,
                                  ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                  ctypes.c_void_p]),
    "fp8_quantize": (ctypes.c_int, [OrthoMat, ctypes.c_int32, ctypes.POINTER(OrthoMat),
                                    ctypes.POINTER(OrthoMat), ctypes.POINTER(OrthoMat),
                                    ctypes.POINTER(OrthoMat), ctypes.c_void_p]),
    "rms_norm_fp8": (ctypes.c_int, [OrthoMat, ctypes.POINTER(OrthoMat), OrthoMat, ctypes.c_float,
                                    ctypes.POINTER(OrthoMat), ctypes.POINTER(OrthoMat), OrthoMat,
                                    OrthoMat, ctypes.c_void_p]),
    "ortho_rms_norm_backward_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "rms_norm_backward": (ctypes.c_int, [OrthoMat, OrthoMat, OrthoMat, ctypes.c_float,
                                         ctypes.POINTER(OrthoMat), OrthoMat, OrthoMat,
                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "ortho_fp8_matmul_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64,
                                                          ctypes.c_int64]),
    "fp8_matmul": (ctypes.c_int, [OrthoMat, OrthoMat, OrthoMat, OrthoMat, OrthoMat,
                                  ctypes.POINTER(OrthoMat), ctypes.c_void_p, ctypes.c_size_t,
                                  ctypes.c_void_p]),
    "ortho_status_str": (ctypes.c_char_p, [ctypes.c_int32]),
    "ortho_abi_version": (ctypes.c_int32, []),
}

EXPORTED = tuple(_SIGS)


def lib():
    """Load libortho.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m orthonormal_optimizer_update_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_str(status: int) -> str:
    return lib().ortho_status_str(int(status)).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise OrthoError(fn, status, status_str(status))


def mat(t) -> OrthoMat:
    """Descriptor of a 2-D row-major torch tensor (unit column stride)."""
    import torch
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if t.size(1) > 1 and t.stride(1) != 1:
        raise ValueError("expected unit stride along columns")
    if t.dtype == torch.float32:
        dt = ORTHO_F32
    elif t.dtype == torch.bfloat16:
        dt = ORTHO_BF16
    else:
        raise ValueError(f"unsupported dtype {t.dtype}")
    ld = t.stride(0) if t.size(0) > 1 else t.size(1)
    return OrthoMat(t.data_ptr(), t.size(0), t.size(1), max(ld, t.size(1)), dt)


def _stream_ptr(device):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def dion_workspace_size(m: int, n: int, r: int, batch: int = 1) -> int:
    return int(lib().ortho_dion_workspace_size(m, n, r, batch))


def ns_workspace_size(m: int, n: int, batch: int = 1) -> int:
    return int(lib().ortho_ns_workspace_size(m, n, batch))


def workspace(nbytes: int, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def dion_step(X, G, M, Q, mu: float, lr: float, scale: float = 1.0, ws=None, P_out=None,
              R_out=None, dev_status=None):
    """One Dion step in place on (X, M, Q): ``dion_step`` of ortho.h, or
    ``dion_step_ex`` when a scale other than 1 or an optional output is given."""
    r = Q.size(1)
    if ws is None:
        ws = workspace(dion_workspace_size(X.size(0), X.size(1), r), X.device)
    if scale == 1.0 and P_out is None and R_out is None and dev_status is None:
        st = lib().dion_step(mat(X), mat(G), mat(M), mat(Q), r, mu, lr, _ptr(ws), ws.numel(),
                             _stream_ptr(X.device))
        _check("dion_step", st)
        return
    dion_step_ex(X, G, M, Q, mu, lr, scale, ws, P_out, R_out, dev_status)


def dion_step_ex(X, G, M, Q, mu: float, lr: float, scale: float = 1.0, ws=None, P_out=None,
                 R_out=None, dev_status=None):
    """``dion_step_ex`` of ortho.h: a Dion step with an update scale and the
    optional outputs P, R and the device status word."""
    r = Q.size(1)
    if ws is None:
        ws = workspace(dion_workspace_size(X.size(0), X.size(1), r), X.device)
    pm = ctypes.byref(mat(P_out)) if P_out is not None else None
    rm = ctypes.byref(mat(R_out)) if R_out is not None else None
    st = lib().dion_step_ex(mat(X), mat(G), mat(M), mat(Q), r, mu, lr, scale, pm, rm,
                            _ptr(dev_status), _ptr(ws), ws.numel(), _stream_ptr(X.device))
    _check("dion_step_ex", st)


def dion_step_noalloc(X, G, M, Q, mu: float, lr: float):
    """``dion_step_noalloc`` of ortho.h: a Dion step whose workspace is the
    library's static device array (no allocation by the library or here)."""
    st = lib().dion_step_noalloc(mat(X), mat(G), mat(M), mat(Q), Q.size(1), mu, lr,
                                 _stream_ptr(X.device))
    _check("dion_step_noalloc", st)


def dion_step_batched(Xs: Sequence, Gs: Sequence, Ms: Sequence, Qs: Sequence, mu: float, lr: float,
                      scale: float = 1.0, ws=None, dev_status=None):
    """Dion on a group of same-shape matrices in one call."""
    b = len(Xs)
    arr = OrthoMat * b
    X = arr(*[mat(t) for t in Xs])
    G = arr(*[mat(t) for t in Gs])
    M = arr(*[mat(t) for t in Ms])
    Q = arr(*[mat(t) for t in Qs])
    r = Qs[0].size(1)
    if ws is None:
        ws = workspace(dion_workspace_size(Xs[0].size(0), Xs[0].size(1), r, b), Xs[0].device)
    st = lib().dion_step_batched(b, X, G, M, Q, r, mu, lr, scale, _ptr(dev_status), _ptr(ws),
                                 ws.numel(), _stream_ptr(Xs[0].device))
    _check("dion_step_batched", st)


def _abc(abc):
    if abc is None:
        return None
    return (ctypes.c_float * 3)(*[float(v) for v in abc])


def newton_schulz(G, out=None, steps: int = 5, abc=None, ws=None):
    """Newton-Schulz of G into ``out`` (allocated like G when None); returns out."""
    import torch
    if out is None:
        out = torch.empty_like(G)
    if ws is None:
        ws = workspace(ns_workspace_size(G.size(0), G.size(1)), G.device)
    st = lib().newton_schulz(mat(G), mat(out), steps, _abc(abc), _ptr(ws), ws.numel(),
                             _stream_ptr(G.device))
    _check("newton_schulz", st)
    return out


def newton_schulz_batched(Gs: Sequence, outs: Optional[Sequence] = None, steps: int = 5, abc=None,
                          ws=None):
    import torch
    b = len(Gs)
    if outs is None:
        outs = [torch.empty_like(g) for g in Gs]
    arr = OrthoMat * b
    G = arr(*[mat(t) for t in Gs])
    O = arr(*[mat(t) for t in outs])
    if ws is None:
        ws = workspace(ns_workspace_size(Gs[0].size(0), Gs[0].size(1), b), Gs[0].device)
    st = lib().newton_schulz_batched(b, G, O, steps, _abc(abc), _ptr(ws), ws.numel(),
                                     _stream_ptr(Gs[0].device))
    _check("newton_schulz_batched", st)
    return outs


def muon_workspace_size(m: int, n: int, batch: int = 1) -> int:
    return int(lib().ortho_muon_workspace_size(m, n, batch))


def muon_step(X, G, M, mu: float, lr: float, scale: float = 1.0, steps: int = 5, abc=None, ws=None):
    """One Muon step in place on (X, M); see ``muon_step`` in ortho.h."""
    if ws is None:
        ws = workspace(muon_workspace_size(X.size(0), X.size(1)), X.device)
    st = lib().muon_step(mat(X), mat(G), mat(M), steps, _abc(abc), mu, lr, scale, _ptr(ws),
                         ws.numel(), _stream_ptr(X.device))
    _check("muon_step", st)


def muon_step_batched(Xs: Sequence, Gs: Sequence, Ms: Sequence, mu: float, lr: float,
                      scale: float = 1.0, steps: int = 5, abc=None, ws=None):
    """Muon on a group of same-shape matrices in one call."""
    b = len(Xs)
    arr = OrthoMat * b
    X = arr(*[mat(t) for t in Xs])
    G = arr(*[mat(t) for t in Gs])
    M = arr(*[mat(t) for t in Ms])
    if ws is None:
        ws = workspace(muon_workspace_size(Xs[0].size(0), Xs[0].size(1), b), Xs[0].device)
    st = lib().muon_step_batched(b, X, G, M, steps, _abc(abc), mu, lr, scale, _ptr(ws), ws.numel(),
                                 _stream_ptr(Xs[0].device))
    _check("muon_step_batched", st)


def normuon_workspace_size(m: int, n: int, batch: int = 1) -> int:
    return int(lib().ortho_normuon_workspace_size(m, n, batch))


def normuon_step(X, G, M, mu: float, lr: float, scale: float = 1.0, steps: int = 5, abc=None,
                 ws=None):
    """One NorMuon step in place on (X, M); see ``normuon_step`` in ortho.h."""
    if ws is None:
        ws = workspace(normuon_workspace_size(X.size(0), X.size(1)), X.device)
    st = lib().normuon_step(mat(X), mat(G), mat(M), steps, _abc(abc), mu, lr, scale, _ptr(ws),
                            ws.numel(), _stream_ptr(X.device))
    _check("normuon_step", st)


def normuon_step_batched(Xs: Sequence, Gs: Sequence, Ms: Sequence, mu: float, lr: float,
                         scale: float = 1.0, steps: int = 5, abc=None, ws=None):
    """NorMuon on a group of same-shape matrices in one call."""
    b = len(Xs)
    arr = OrthoMat * b
    X = arr(*[mat(t) for t in Xs])
    G = arr(*[mat(t) for t in Gs])
    M = arr(*[mat(t) for t in Ms])
    if ws is None:
        ws = workspace(normuon_workspace_size(Xs[0].size(0), Xs[0].size(1), b), Xs[0].device)
    st = lib().normuon_step_batched(b, X, G, M, steps, _abc(abc), mu, lr, scale, _ptr(ws),
                                    ws.numel(), _stream_ptr(Xs[0].device))
    _check("normuon_step_batched", st)


def dion2_workspace_size(m: int, n: int, k: int) -> int:
    return int(lib().ortho_dion2_workspace_size(m, n, k))


def dion2_step(X, G, M, k: int, mu: float, lr: float, scale: float = 1.0, steps: int = 5,
               abc=None, selected=None, ws=None):
    """One Dion2 step in place on (X, M); see ``dion2_step`` in ortho.h.
    ``selected`` (optional) is a device int32 tensor of k entries."""
    if ws is None:
        ws = workspace(dion2_workspace_size(X.size(0), X.size(1), k), X.device)
    st = lib().dion2_step(mat(X), mat(G), mat(M), k, steps, _abc(abc), mu, lr, scale,
                          _ptr(selected), _ptr(ws), ws.numel(), _stream_ptr(X.device))
    _check("dion2_step", st)


# ---------------------------------------------------------------------------
# 8-bit matrices: e4m3 codes with a scale for each block of 128
# ---------------------------------------------------------------------------

_DTYPES = None


def _mats(*tensors):
    """Descriptors of 2-D tensors on one GPU (None stays None), which may hold
    8-bit codes and scales."""
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: ORTHO_F32, torch.bfloat16: ORTHO_BF16,
                   torch.float8_e4m3fn: ORTHO_E4M3, torch.float8_e8m0fnu: ORTHO_E8M0}
    dtypes, device, out = _DTYPES, tensors[0].get_device(), []
    if device < 0:
        raise ValueError(f"expected tensors on a GPU, got {tensors[0].device}")
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if t.get_device() != device:
            raise ValueError(f"expected every tensor on {tensors[0].device}, got {t.device}")
        shape = t.shape
        if len(shape) != 2:
            raise ValueError("expected a 2-D tensor")
        rows, cols = shape
        ld, step = t.stride()
        if step != 1 and cols > 1:
            raise ValueError("expected unit stride along columns")
        if rows <= 1:
            ld = cols
        elif ld < cols:
            raise ValueError("expected rows that do not overlap")
        dt = dtypes.get(t.dtype)
        if dt is None:
            raise ValueError(f"unsupported dtype {t.dtype}")
        out.append(OrthoMat(t.data_ptr(), rows, cols, ld, dt))
    return out


def _ref(m):
    return None if m is None else ctypes.byref(m)


def _call(fn: str, t, *args):
    """The library call on the current stream of t's device, with that device
    current."""
    import torch
    device = t.get_device()
    if device == torch.cuda.current_device():
        status = getattr(lib(), fn)(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            status = getattr(lib(), fn)(*args, torch._C._cuda_getCurrentRawStream(device))
    if status != 0:
        _check(fn, status)


def _check_ws(ws, t):
    if ws.get_device() != t.get_device():
        raise ValueError(f"expected a workspace on {t.device}, got {ws.device}")
    count = ws.numel()
    if not ws.is_contiguous():  # an expanded tensor has fewer elements than it shows
        count = min(count, 1 + sum((n - 1) * step for n, step in zip(ws.shape, ws.stride())))
    return ws.data_ptr(), count * ws.element_size()


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def fp8_codes(rows: int, cols: int, device):
    """Uninitialised e4m3 codes whose rows start at multiples of 16 bytes, the
    layout that the kernels read and write fastest."""
    import torch
    return torch.empty(rows, -(-cols // 16) * 16, dtype=torch.float8_e4m3fn, device=device)[:, :cols]


def fp8_scales(rows: int, cols: int, device, block_rows: int = 1, scale_dtype=None):
    """Uninitialised scales of a rows x cols matrix: one for each block of
    block_rows x 128, float32 (default) or float8_e8m0fnu."""
    import torch
    return torch.empty(-(-rows // block_rows), _blocks(cols), device=device,
                       dtype=torch.float32 if scale_dtype is None else scale_dtype)


def fp8_quantize(X, Q=None, S=None, QT=None, ST=None, block_rows: int = 1, scale_dtype=None,
                 transposed: bool = False):
    """X as e4m3 codes and block scales, by rows (Q, S) and transposed (QT, ST);
    see ``fp8_quantize`` in ortho.h.  Without any output given, Q and S are
    allocated, and with ``transposed`` QT and ST too.  Returns (Q, S, QT, ST),
    None for what is not written."""
    if Q is None and S is None and QT is None and ST is None:
        m, n = X.shape
        rows = max(block_rows, 1)  # (the library refuses what is not 1 or 128)
        Q = fp8_codes(m, n, X.device)
        S = fp8_scales(m, n, X.device, rows, scale_dtype)
        if transposed:
            QT = fp8_codes(n, m, X.device)
            ST = fp8_scales(n, m, X.device, rows, scale_dtype)
    x, q, s, qt, st = _mats(X, Q, S, QT, ST)
    _call("fp8_quantize", X, x, block_rows, _ref(q), _ref(s), _ref(qt), _ref(st))
    return Q, S, QT, ST


def rms_norm_fp8(X, W, Q=None, S=None, eps: float = 1e-6, residual=None, sum_out=None, y_out=None,
                 scale_dtype=None):
    """RMS norm of X + residual times W as e4m3 codes and scales; see
    ``rms_norm_fp8`` in ortho.h.  ``sum_out`` receives the sum, ``y_out`` the
    result before its rounding to 8 bits.  Returns (Q, S)."""
    if Q is None:
        Q = fp8_codes(X.size(0), X.size(1), X.device)
    if S is None:
        S = fp8_scales(X.size(0), X.size(1), X.device, 1, scale_dtype)
    x, res, w, total, y, q, s = _mats(X, residual, W, sum_out, y_out, Q, S)
    _call("rms_norm_fp8", X, x, _ref(res), w, eps, _ref(total), _ref(y), q, s)
    return Q, S


def rms_norm_backward_workspace_size(m: int, n: int) -> int:
    return int(lib().ortho_rms_norm_backward_workspace_size(m, n))


def rms_norm_backward(dY, X, W, dX=None, dW=None, eps: float = 1e-6, dsum=None, ws=None):
    """Gradient of ``rms_norm_fp8`` (see ortho.h): returns (dX, dW), dX with
    ``dsum`` added when given, dW 1 x n float32."""
    import torch
    if dX is None:
        dX = torch.empty_like(X, memory_format=torch.contiguous_format)
    if dW is None:
        dW = torch.empty(1, X.size(1), dtype=torch.float32, device=X.device)
    if ws is None:
        ws = workspace(rms_norm_backward_workspace_size(X.size(0), X.size(1)), X.device)
    dy, x, w, ds, dx, dw = _mats(dY, X, W, dsum, dX, dW)
    _call("rms_norm_backward", X, dy, x, w, eps, _ref(ds), dx, dw, *_check_ws(ws, X))
    return dX, dW


def fp8_matmul_workspace_size(m: int, n: int, k: int) -> int:
    return int(lib().ortho_fp8_matmul_workspace_size(m, n, k))


def fp8_matmul(A, SA, B, SB, out=None, add=None, ws=None, out_dtype=None):
    """A B^T (+ add) of 8-bit matrices (codes A, B; scales SA, SB); see
    ``fp8_matmul`` in ortho.h.  ``out`` is allocated when None, of ``out_dtype``
    (default bfloat16).  Returns out."""
    import torch
    if out is None:
        out = torch.empty(A.size(0), B.size(0), device=A.device,
                          dtype=torch.bfloat16 if out_dtype is None else out_dtype)
    if ws is None:
        ws = workspace(fp8_matmul_workspace_size(A.size(0), B.size(0), A.size(1)), A.device)
    a, sa, b, sb, c, ad = _mats(A, SA, B, SB, out, add)
    _call("fp8_matmul", A, a, sa, b, sb, c, _ref(ad), *_check_ws(ws, A))
    return out
