"""ctypes binding of libdsrows.so (include/ds_rows.h, include/ds_token_rows.h):
argument marshalling only.

Every computation runs in the library's HIP kernels.  The functions take
torch tensors on a HIP device, check dtype/shape/contiguity/device, pass raw
pointers and the current stream, and raise ``RuntimeError`` with the
library's status string on a nonzero status.  Loading fails loudly if the
library has not been built (``python -m scale_invariant_row_amd.build``).

bf16 tensors may be ``torch.bfloat16`` or ``torch.int16``/``torch.uint16``
holding the bit patterns.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
from typing import List, NamedTuple, Optional, Sequence, Tuple

PKG = os.path.dirname(os.path.abspath(__file__))
# DS_ROWS_LIB may name another build of the same library (the tests'
# AddressSanitizer build of the host code); there is no fallback either way
LIB_PATH = os.environ.get("DS_ROWS_LIB") or os.path.join(PKG, "_lib", "libdsrows.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "ds_rows.h")
TOKEN_HEADER = os.path.join(os.path.dirname(PKG), "include", "ds_token_rows.h")

DS_OK = 0
DS_ERR_NULL = -1
DS_ERR_SHAPE = -2
DS_ERR_ALIGN = -3
DS_ERR_ARG = -4
DS_ERR_ALLOC = -5
DS_ERR_LAUNCH = -6
DS_ERR_DEVICE = -7
DS_ERR_CAPTURE = -8
DS_ERR_SCRATCH = -9
DS_ERR_WORKSPACE = -10
DS_SCRATCH_FLOATS = 1 << 20
DS_MAX_TOP = 32
DS_TYPE_BF16, DS_TYPE_F32 = 0, 1


class RownormDesc(ctypes.Structure):
    """ds_rownorm_desc."""
    _fields_ = [
        ("w", ctypes.c_void_p),
        ("gain", ctypes.c_void_p),
        ("radius", ctypes.c_float),
        ("norm_out", ctypes.c_void_p),
        ("w_eff", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("gain_mode", ctypes.c_int32),
        ("seg", ctypes.c_int32),
        ("ld", ctypes.c_int64),
    ]


class RownormGradDesc(ctypes.Structure):
    """ds_rownorm_grad_desc."""
    _fields_ = [
        ("w", ctypes.c_void_p),
        ("gain", ctypes.c_void_p),
        ("radius", ctypes.c_float),
        ("dw_eff", ctypes.c_void_p),
        ("dw", ctypes.c_void_p),
        ("dgain", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("gain_mode", ctypes.c_int32),
        ("dgain_total", ctypes.c_void_p),
        ("seg", ctypes.c_int32),
        ("ld", ctypes.c_int64),
    ]


class RescaleDesc(ctypes.Structure):
    """ds_rescale_desc."""
    _fields_ = [
        ("w", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("radius", ctypes.c_float),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("seg", ctypes.c_int32),
        ("ld", ctypes.c_int64),
    ]


_lib = None
_token = None          # the library once ds_token_rows.h's entry points are declared
_raw_stream = None     # torch's own look-up of a device's current stream, where it has one


def lib() -> ctypes.CDLL:
    """The loaded library (loaded once); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m scale_invariant_row_amd.build` (there is no fallback)")
        # torch first: it maps its own HIP runtime (same soname), and the
        # library then binds to that one, so the kernels, the tensors' memory
        # and the streams all live in one HIP runtime.  Loaded the other way
        # round, the process would hold two runtimes and the library's own
        # would not share torch's device state.
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
        for name in ("ds_l2_rows", "ds_rms_rows"):
            getattr(L, name).argtypes = [vp, vp, vp, i64, i64, f32, vp]
            getattr(L, name).restype = ctypes.c_int
        L.ds_slerp_rows.argtypes = [vp, vp, vp, vp, i64, i64, f32, vp]
        L.ds_slerp_rows.restype = ctypes.c_int
        L.ds_weight_rownorm_gain.argtypes = [ctypes.POINTER(RownormDesc), ctypes.c_int32, vp]
        L.ds_weight_rownorm_gain.restype = ctypes.c_int
        L.ds_gate_l2_rows.argtypes = [vp, vp, vp, vp, i64, i64, f32, vp]
        L.ds_gate_l2_rows.restype = ctypes.c_int
        L.ds_swiglu_l2_rows.argtypes = [vp, vp, vp, vp, vp, i64, i64, f32, vp]
        L.ds_swiglu_l2_rows.restype = ctypes.c_int
        i32 = ctypes.c_int32
        L.ds_qk_rows_l2.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, i64,
                                    i32, i32, i32, f32, vp]
        L.ds_qk_rows_l2.restype = ctypes.c_int
        for name in ("ds_rescale_project", "ds_rescale_after_step"):
            getattr(L, name).argtypes = [ctypes.POINTER(RescaleDesc), ctypes.c_int32, vp]
            getattr(L, name).restype = ctypes.c_int
        for name in ("ds_l2_rows_backward", "ds_rms_rows_backward"):
            getattr(L, name).argtypes = [vp, vp, vp, vp, i64, i64, f32, vp]
            getattr(L, name).restype = ctypes.c_int
        for name in ("ds_weight_rownorm_gain_backward", "ds_weight_rownorm_gain_backward_noalloc"):
            getattr(L, name).argtypes = [ctypes.POINTER(RownormGradDesc), ctypes.c_int32, vp]
            getattr(L, name).restype = ctypes.c_int
        L.ds_status_string.argtypes = [ctypes.c_int]
        L.ds_status_string.restype = ctypes.c_char_p
        L.ds_version.argtypes = []
        L.ds_version.restype = ctypes.c_int
        _lib = L
    return _lib


def _token_lib() -> ctypes.CDLL:
    """The library with ds_token_rows.h's entry points declared; raises if the
    loaded build does not hold them."""
    global _token, _raw_stream
    if _token is None:
        L = lib()
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        sig = {
            "ds_embed_rows": [vp, i32, i64, vp, i32, f32, vp, i64, i64, vp],
            "ds_embed_rows_backward": [vp, vp, i32, f32, vp, i32, i32, i64, i64, i64, vp, i64, vp],
            "ds_qk_rows_rms": [vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, i64, i64, i32, i32,
                               i32, f32, vp],
            "ds_qk_rows_rms_backward": [vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, i64, vp, i64,
                                        vp, i64, vp, vp, i64, i32, i32, i32, f32, vp, i64, vp],
            "ds_logprob_rows": [vp, i32, i64, vp, f32, vp, i32, vp, vp, vp, vp, vp, i32, i64, i64,
                                vp, i64, vp],
            "ds_logprob_rows_backward": [vp, i32, i64, vp, f32, vp, i32, vp, vp, vp, vp, vp, i64, vp,
                                         i64, i64, vp, i64, vp],
        }
        sizes = {
            "ds_embed_rows_backward_workspace": [i64, i64, i64],
            "ds_qk_rows_rms_backward_workspace": [i64, i32, i32, i32],
            "ds_logprob_rows_workspace": [i64, i64, i32],
            "ds_logprob_rows_backward_workspace": [i64, i64],
        }
        for table, res in ((sig, ctypes.c_int), (sizes, i64)):
            for name, args in table.items():
                try:
                    f = getattr(L, name)
                except AttributeError:
                    raise RuntimeError(f"{LIB_PATH} does not hold {name}: build the library again "
                                       "with `python -m scale_invariant_row_amd.build`") from None
                f.argtypes, f.restype = args, res
        _raw_stream = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
        _token = L
    return _token


def header_functions(header: str = HEADER) -> List[str]:
    """Names of the functions a header (include/ds_rows.h) declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(ds_\w+)\s*\(", text, re.M)))


def ds_status_string(status: int) -> str:
    return lib().ds_status_string(int(status)).decode()


def ds_version() -> int:
    return lib().ds_version()


def _check(status: int, what: str) -> None:
    if status != DS_OK:
        raise RuntimeError(f"{what}: {ds_status_string(status)}")


# --------------------------------------------------------------- tensors

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _bf16_2d(t, name, device: bool = True):
    """A bf16 [rows, cols] contiguous tensor (and, unless the caller checks
    devices itself afterwards, on a HIP device)."""
    torch = _torch()
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{name}: expected bf16 data (bfloat16 or 16-bit int bits), got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D [rows, cols] tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if device and t.device.type != "cuda":
        raise ValueError(f"{name}: must be on a HIP device")


def _same(a, b, name):
    if b.shape != a.shape or b.device != a.device:
        raise ValueError(f"{name}: shape/device mismatch {tuple(b.shape)} vs {tuple(a.shape)}")


def _stream_of(t, stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _torch_stream(t, stream):
    """The torch stream object for ``stream`` (None: t's current stream; a raw
    handle is wrapped without taking ownership)."""
    torch = _torch()
    if t is None:
        return None
    if stream is None:
        return torch.cuda.current_stream(t.device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.ExternalStream(handle, device=t.device)


def _norm_rows(name, x, r, eps, out, stream):
    torch = _torch()
    _bf16_2d(x, "x")
    if r is not None:
        _bf16_2d(r, "r")
        _same(x, r, "r")
    if out is None:
        out = torch.empty_like(x)
    _bf16_2d(out, "out")
    _same(x, out, "out")
    with torch.cuda.device(x.device):
        st = getattr(lib(), name)(x.data_ptr(), None if r is None else r.data_ptr(),
                                  out.data_ptr(), x.shape[0], x.shape[1], float(eps),
                                  _stream_of(x, stream))
    _check(st, name)
    return out


def ds_rms_rows(x, r=None, eps: float = 1e-6, out=None, stream=None):
    """y = bf16(s / sqrt(sum(s^2) / cols + eps)) per row, s = x or bf16(x + r).

    Returns ``out`` (allocated like ``x`` when not given; may be ``x`` or ``r``).
    """
    return _norm_rows("ds_rms_rows", x, r, eps, out, stream)


def ds_rms_rows_backward(x, r, dy, eps: float = 1e-6, out=None, stream=None):
    """dx = bf16((dy - s <s,dy>/(cols D^2)) / D), D^2 = sum(s^2)/cols + eps: the
    gradient of ds_rms_rows(x, r, eps) with respect to x (and r).  Returns
    ``out`` (allocated like ``dy`` when not given; may be ``x``, ``r`` or ``dy``)."""
    return _norm_rows_backward("ds_rms_rows_backward", x, r, dy, eps, out, stream)


def ds_l2_rows(x, r=None, eps: float = 1e-6, out=None, stream=None):
    """y = bf16(s / sqrt(sum(s^2) + eps)) per row, s = x or bf16(x + r).

    Returns ``out`` (allocated like ``x`` when not given; may be ``x`` or ``r``).
    """
    return _norm_rows("ds_l2_rows", x, r, eps, out, stream)


def ds_slerp_rows(res, out_rows, alpha, eps: float = 1e-6, h=None, stream=None):
    """h = bf16(l2(a + |alpha| (b - a))), a = bf16(l2(res)), b = bf16(l2(out_rows))."""
    torch = _torch()
    _bf16_2d(res, "res")
    _bf16_2d(out_rows, "out")
    _same(res, out_rows, "out")
    if alpha.dtype != torch.float32 or alpha.dim() != 1 or alpha.shape[0] != res.shape[1] \
            or not alpha.is_contiguous() or alpha.device != res.device:
        raise ValueError("alpha: expected a contiguous fp32 [cols] tensor on the rows' device")
    if h is None:
        h = torch.empty_like(res)
    _bf16_2d(h, "h")
    _same(res, h, "h")
    with torch.cuda.device(res.device):
        st = lib().ds_slerp_rows(res.data_ptr(), out_rows.data_ptr(), alpha.data_ptr(),
                                 h.data_ptr(), res.shape[0], res.shape[1], float(eps),
                                 _stream_of(res, stream))
    _check(st, "ds_slerp_rows")
    return h


DS_GAIN_ROW, DS_GAIN_SCALAR, DS_GAIN_NONE = 0, 1, 2


def _layout(w, seg):
    """(rows, cols, seg, ld) of a stored 2-D weight.  seg None or 0: its rows
    are the unit rows.  seg > 0: a column block (GPT-2's Conv1D [in, out] with
    seg 1; one ConvTranspose group [in, out * k] with seg k): unit u owns the
    seg values at u * seg of every stored row."""
    if not seg:
        return w.shape[0], w.shape[1], 0, 0
    if w.shape[1] % seg != 0:
        raise ValueError(f"a column block of seg {seg} needs a multiple of {seg} stored columns")
    return w.shape[1] // seg, w.shape[0] * seg, int(seg), w.shape[1]


def _gain_mode(g, rows: int, name: str) -> int:
    """A gain tensor's mode: None (no gain), a 0-dim or one-element tensor for
    rows != 1 (one gain for the matrix), or a [rows] tensor (a gain per row)."""
    torch = _torch()
    if g is None:
        return DS_GAIN_NONE
    if g.dtype != torch.float32 or not g.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous fp32 tensor")
    if g.dim() == 0 or (g.numel() == 1 and rows != 1):
        return DS_GAIN_SCALAR
    if g.shape != (rows,):
        raise ValueError(f"{name}: expected fp32 [rows], one value, or None")
    return DS_GAIN_ROW


def ds_weight_rownorm_gain(ws: Sequence, gains: Sequence, radius: Optional[Sequence[float]] = None,
                           norm_out: Optional[Sequence] = None, w_eff: Optional[Sequence] = None,
                           stream=None, segs: Optional[Sequence] = None) -> Tuple[list, list]:
    """Per matrix: ||W_i|| (fp32) and bf16(W_i * g_i * radius / ||W_i||), in one call.

    ``ws``: fp32 2-D tensors; ``gains``: per matrix an fp32 [rows] tensor (a
    gain per row), a single value (one gain for the matrix) or None (no gain);
    ``segs``: per matrix None (the stored rows are the unit rows) or the seg
    of a column block (see ``_layout``).  Returns (norms, w_effs); w_effs are
    bfloat16 tensors shaped like ws unless given.
    """
    torch = _torch()
    n = len(ws)
    if len(gains) != n:
        raise ValueError("one gain entry per matrix")
    radius = [1.0] * n if radius is None else list(radius)
    lay = [_layout(w, None if segs is None else segs[i]) for i, w in enumerate(ws)]
    if norm_out is None:
        norm_out = [torch.empty(lay[i][0], dtype=torch.float32, device=w.device)
                    for i, w in enumerate(ws)]
    if w_eff is None:
        w_eff = [torch.empty(w.shape, dtype=torch.bfloat16, device=w.device) for w in ws]
    descs = (RownormDesc * max(n, 1))()
    dev = None
    for i, (w, g) in enumerate(zip(ws, gains)):
        if w.dtype != torch.float32 or w.dim() != 2 or not w.is_contiguous():
            raise ValueError(f"ws[{i}]: expected a contiguous fp32 [rows, cols] tensor")
        rows, cols, seg, ld = lay[i]
        mode = _gain_mode(g, rows, f"gains[{i}]")
        _bf16_2d(w_eff[i], f"w_eff[{i}]", device=False)
        if tuple(w_eff[i].shape) != tuple(w.shape):
            raise ValueError(f"w_eff[{i}]: shape mismatch")
        if norm_out[i] is not None and (norm_out[i].dtype != torch.float32
                                        or norm_out[i].shape != (rows,)
                                        or not norm_out[i].is_contiguous()):
            raise ValueError(f"norm_out[{i}]: expected a contiguous fp32 [rows] tensor")
        for t in (w, g, w_eff[i], norm_out[i]):
            if t is None:
                continue
            if t.device.type != "cuda" or (dev is not None and t.device != dev):
                raise ValueError("all tensors must be on one HIP device")
            dev = t.device
        descs[i] = RownormDesc(w.data_ptr(), None if g is None else g.data_ptr(), float(radius[i]),
                               None if norm_out[i] is None else norm_out[i].data_ptr(),
                               w_eff[i].data_ptr(), rows, cols, mode, seg, ld)
    if n == 0:
        return [], []
    with torch.cuda.device(dev):
        st = lib().ds_weight_rownorm_gain(descs, n, _stream_of(ws[0], stream))
    _check(st, "ds_weight_rownorm_gain")
    return list(norm_out), list(w_eff)


def _norm_rows_backward(name, x, r, dy, eps, out, stream):
    torch = _torch()
    _bf16_2d(x, "x")
    _bf16_2d(dy, "dy")
    _same(x, dy, "dy")
    if r is not None:
        _bf16_2d(r, "r")
        _same(x, r, "r")
    if out is None:
        out = torch.empty_like(dy)
    _bf16_2d(out, "out")
    _same(x, out, "out")
    with torch.cuda.device(x.device):
        st = getattr(lib(), name)(x.data_ptr(), None if r is None else r.data_ptr(),
                                  dy.data_ptr(), out.data_ptr(), x.shape[0], x.shape[1],
                                  float(eps), _stream_of(x, stream))
    _check(st, name)
    return out


def ds_l2_rows_backward(x, r, dy, eps: float = 1e-6, out=None, stream=None):
    """dx = bf16((dy - s <s,dy>/D^2) / D), the gradient of ds_l2_rows(x, r, eps)
    with respect to x (and to r when given).  Returns ``out`` (allocated like
    ``dy`` when not given; may be ``x``, ``r`` or ``dy``)."""
    return _norm_rows_backward("ds_l2_rows_backward", x, r, dy, eps, out, stream)


def ds_weight_rownorm_gain_backward(ws: Sequence, gains: Sequence, dw_effs: Sequence,
                                    radius: Optional[Sequence[float]] = None,
                                    dw: Optional[Sequence] = None,
                                    dgain: Optional[Sequence] = None,
                                    want_dgain: bool = True, stream=None,
                                    segs: Optional[Sequence] = None,
                                    _noalloc: bool = False) -> Tuple[list, list]:
    """Per matrix: dL/dW (fp32) and dL/dg (fp32) from dL/dW_eff (bf16), in one call.

    ``gains`` and ``segs`` as for ds_weight_rownorm_gain.  Returns (dws, dgains): dL/dg is
    an fp32 [rows] tensor for a gain per row, a 0-dim fp32 tensor for one gain
    per matrix (the library sums the rows' shares, kept in a [rows] buffer),
    and None with no gain or when ``want_dgain`` is false and none was given.
    """
    torch = _torch()
    n = len(ws)
    if len(gains) != n or len(dw_effs) != n:
        raise ValueError("one gain entry and one dW_eff per matrix")
    radius = [1.0] * n if radius is None else list(radius)
    if dw is None:
        dw = [torch.empty(w.shape, dtype=torch.float32, device=w.device) for w in ws]
    lay = [_layout(w, None if segs is None else segs[i]) for i, w in enumerate(ws)]
    modes = [_gain_mode(g, lay[i][0], f"gains[{i}]") for i, g in enumerate(gains)]
    if dgain is None:
        dgain = [torch.empty(lay[i][0] if m == DS_GAIN_ROW else (), dtype=torch.float32,
                             device=w.device) if want_dgain and m != DS_GAIN_NONE else None
                 for i, (w, m) in enumerate(zip(ws, modes))]
    dev = None
    for i, (w, g, de) in enumerate(zip(ws, gains, dw_effs)):
        if w.dtype != torch.float32 or w.dim() != 2 or not w.is_contiguous():
            raise ValueError(f"ws[{i}]: expected a contiguous fp32 [rows, cols] tensor")
        _bf16_2d(de, f"dw_effs[{i}]", device=False)
        if tuple(de.shape) != tuple(w.shape):
            raise ValueError(f"dw_effs[{i}]: shape mismatch")
        if dw[i].dtype != torch.float32 or tuple(dw[i].shape) != tuple(w.shape) \
                or not dw[i].is_contiguous():
            raise ValueError(f"dw[{i}]: expected a contiguous fp32 tensor shaped like ws[{i}]")
        want = (lay[i][0],) if modes[i] == DS_GAIN_ROW else ()
        if dgain[i] is not None and (dgain[i].dtype != torch.float32 or dgain[i].shape != want
                                     or not dgain[i].is_contiguous()):
            raise ValueError(f"dgain[{i}]: expected a contiguous fp32 tensor of shape {want}")
        for t in (w, g, de, dw[i], dgain[i]):
            if t is None:
                continue
            if t.device.type != "cuda" or (dev is not None and t.device != dev):
                raise ValueError("all tensors must be on one HIP device")
            dev = t.device
    if n == 0:
        return [], []
    # A scalar gain's per-row shares: a temporary the kernels write and read
    # on the launch stream.  It is allocated on that stream, so when it is
    # dropped below, the caching allocator hands its block only to work
    # ordered after those kernels.  (The allocation-free entry point keeps
    # them in the library's own scratch instead.)
    with torch.cuda.device(dev), torch.cuda.stream(_torch_stream(ws[0], stream)):
        shares = [torch.empty(lay[i][0], dtype=torch.float32, device=dev)
                  if m == DS_GAIN_SCALAR and dgain[i] is not None and not _noalloc else None
                  for i, m in enumerate(modes)]
    descs = (RownormGradDesc * n)()
    for i, (w, g, de) in enumerate(zip(ws, gains, dw_effs)):
        rows, cols, seg, ld = lay[i]
        per_row = dgain[i] if modes[i] == DS_GAIN_ROW else shares[i]
        total = dgain[i] if modes[i] == DS_GAIN_SCALAR else None
        descs[i] = RownormGradDesc(w.data_ptr(), None if g is None else g.data_ptr(),
                                   float(radius[i]), de.data_ptr(), dw[i].data_ptr(),
                                   None if per_row is None else per_row.data_ptr(),
                                   rows, cols, modes[i],
                                   None if total is None else total.data_ptr(), seg, ld)
    name = "ds_weight_rownorm_gain_backward" + ("_noalloc" if _noalloc else "")
    with torch.cuda.device(dev):
        st = getattr(lib(), name)(descs, n, _stream_of(ws[0], stream))
    _check(st, name)
    return list(dw), list(dgain)


def ds_weight_rownorm_gain_backward_noalloc(ws: Sequence, gains: Sequence, dw_effs: Sequence,
                                            radius: Optional[Sequence[float]] = None,
                                            dw: Optional[Sequence] = None,
                                            dgain: Optional[Sequence] = None,
                                            want_dgain: bool = True, stream=None,
                                            segs: Optional[Sequence] = None
                                            ) -> Tuple[list, list]:
    """ds_weight_rownorm_gain_backward through the allocation-free entry point:
    the library allocates nothing (a scalar gain's row shares live in its fixed
    per-GPU scratch).  Pass ``dw`` and ``dgain`` to keep this wrapper from
    allocating its outputs through torch."""
    return ds_weight_rownorm_gain_backward(ws, gains, dw_effs, radius, dw, dgain, want_dgain,
                                           stream, segs, _noalloc=True)


def _col_vector(v, cols, like, name):
    torch = _torch()
    if v.dtype != torch.float32 or v.dim() != 1 or v.shape[0] != cols \
            or not v.is_contiguous() or v.device != like.device:
        raise ValueError(f"{name}: expected a contiguous fp32 [cols] tensor on the rows' device")


def ds_gate_l2_rows(o, g, sg, eps: float = 1e-6, out=None, stream=None):
    """y = bf16(l2(bf16(o * sigmoid(g * sg)))) per row (sg: fp32 [cols])."""
    torch = _torch()
    _bf16_2d(o, "o")
    _bf16_2d(g, "g")
    _same(o, g, "g")
    _col_vector(sg, o.shape[1], o, "sg")
    if out is None:
        out = torch.empty_like(o)
    _bf16_2d(out, "out")
    _same(o, out, "out")
    with torch.cuda.device(o.device):
        st = lib().ds_gate_l2_rows(o.data_ptr(), g.data_ptr(), sg.data_ptr(), out.data_ptr(),
                                   o.shape[0], o.shape[1], float(eps), _stream_of(o, stream))
    _check(st, "ds_gate_l2_rows")
    return out


def ds_swiglu_l2_rows(g, u, sug, suu, eps: float = 1e-6, out=None, stream=None):
    """y = bf16(l2(bf16(silu(bf16(g * sug)) * bf16(u * suu)))) per row."""
    torch = _torch()
    _bf16_2d(g, "g")
    _bf16_2d(u, "u")
    _same(g, u, "u")
    _col_vector(sug, g.shape[1], g, "sug")
    _col_vector(suu, g.shape[1], g, "suu")
    if out is None:
        out = torch.empty_like(g)
    _bf16_2d(out, "out")
    _same(g, out, "out")
    with torch.cuda.device(g.device):
        st = lib().ds_swiglu_l2_rows(g.data_ptr(), u.data_ptr(), sug.data_ptr(), suu.data_ptr(),
                                     out.data_ptr(), g.shape[0], g.shape[1], float(eps),
                                     _stream_of(g, stream))
    _check(st, "ds_swiglu_l2_rows")
    return out


def ds_qk_rows_l2(q, k, positions, inv_freq, q_scale, head_dim: int, eps: float = 1e-6,
                  q_out=None, k_out=None, stream=None):
    """RoPE, per-head L2 and q's scale on q [rows, >= nq*hd] and k [rows, >= nk*hd].

    ``q``/``k`` may be strided row views (a fused projection's slices); the
    number of heads is the used width / head_dim, given by ``q_scale``'s
    length for q and by k's width for k.  Returns (q_out, k_out).

    Every argument is checked (dtype, shape, row count, unit column stride,
    contiguity of the vectors, one HIP device for all) before anything is
    launched; a bad one raises ValueError naming it.
    """
    torch = _torch()
    bf16 = (torch.bfloat16, torch.int16, torch.uint16)
    head_dim = int(head_dim)
    if head_dim <= 0:
        raise ValueError("head_dim: must be positive")

    def rows_tensor(t, name):
        if t.dtype not in bf16 or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name}: expected a bf16 [rows, cols] tensor with unit column stride")

    def vector(t, name, dtype, n=None):
        if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous() \
                or (n is not None and t.shape[0] != n):
            want = f"[{n}]" if n is not None else "[n]"
            raise ValueError(f"{name}: expected a contiguous {dtype} {want} tensor")

    rows_tensor(q, "q")
    rows = q.shape[0]
    vector(q_scale, "q_scale", torch.float32)
    if q_scale.shape[0] == 0 or q_scale.shape[0] % head_dim:
        raise ValueError("q_scale: its length must be n_q_heads * head_dim")
    nq = q_scale.shape[0] // head_dim
    if q.shape[1] < nq * head_dim:
        raise ValueError("q: must hold n_q_heads * head_dim columns")
    nk = 0
    if k is not None:
        rows_tensor(k, "k")
        if k.shape[0] != rows:
            raise ValueError(f"k: expected {rows} rows like q, got {k.shape[0]}")
        if k.shape[1] % head_dim:
            raise ValueError("k: its width must be a whole number of heads")
        nk = k.shape[1] // head_dim
    elif k_out is not None:
        raise ValueError("k_out: given without k")
    vector(positions, "positions", torch.int32, rows)
    vector(inv_freq, "inv_freq", torch.float32, head_dim // 2)
    if q_out is not None:
        rows_tensor(q_out, "q_out")
        if q_out.shape[0] != rows or q_out.shape[1] < nq * head_dim:
            raise ValueError(f"q_out: expected [{rows}, >= {nq * head_dim}]")
    if k_out is not None:
        rows_tensor(k_out, "k_out")
        if k_out.shape[0] != rows or k_out.shape[1] < nk * head_dim:
            raise ValueError(f"k_out: expected [{rows}, >= {nk * head_dim}]")
    tensors = [("q", q), ("k", k), ("positions", positions), ("inv_freq", inv_freq),
               ("q_scale", q_scale), ("q_out", q_out), ("k_out", k_out)]
    for name, t in tensors:
        if t is not None and (t.device.type != "cuda" or t.device != q.device):
            raise ValueError(f"{name}: must be on the HIP device of q")
    if q_out is None:
        q_out = torch.empty(rows, nq * head_dim, dtype=q.dtype, device=q.device)
    if k is not None and k_out is None:
        k_out = torch.empty(rows, nk * head_dim, dtype=k.dtype, device=k.device)
    with torch.cuda.device(q.device):
        st = lib().ds_qk_rows_l2(
            q.data_ptr(), q.stride(0), None if k is None else k.data_ptr(),
            0 if k is None else k.stride(0), positions.data_ptr(), inv_freq.data_ptr(),
            q_scale.data_ptr(), q_out.data_ptr(), q_out.stride(0),
            None if k_out is None else k_out.data_ptr(), 0 if k_out is None else k_out.stride(0),
            rows, nq, nk, head_dim, float(eps), _stream_of(q, stream))
    _check(st, "ds_qk_rows_l2")
    return q_out, k_out


def _rescale(ws, vs, radius, after_step, stream, segs=None):
    torch = _torch()
    n = len(ws)
    vs = [None] * n if vs is None else list(vs)
    radius = [1.0] * n if radius is None else list(radius)
    descs = (RescaleDesc * max(n, 1))()
    dev = None
    for i, w in enumerate(ws):
        for t, name in ((w, "w"), (vs[i], "v")):
            if t is None:
                continue
            if t.dtype != torch.float32 or t.dim() != 2 or not t.is_contiguous() \
                    or t.shape != w.shape or t.device.type != "cuda" \
                    or (dev is not None and t.device != dev):
                raise ValueError(f"{name}[{i}]: expected a contiguous fp32 HIP tensor shaped like w")
            dev = t.device
        rows, cols, seg, ld = _layout(w, None if segs is None else segs[i])
        descs[i] = RescaleDesc(w.data_ptr(), None if vs[i] is None else vs[i].data_ptr(),
                               float(radius[i]), rows, cols, seg, ld)
    if n == 0:
        return
    with torch.cuda.device(dev):
        fn = lib().ds_rescale_after_step if after_step else lib().ds_rescale_project
        st = fn(descs, n, _stream_of(ws[0], stream))
    _check(st, "ds_rescale_after_step" if after_step else "ds_rescale_project")


def ds_rescale_project(ws: Sequence, grads: Sequence, stream=None,
                       segs: Optional[Sequence] = None) -> None:
    """In place, per matrix: grad <- grad - w <w, grad> / ||w||^2 per unit row
    (``segs`` as for ds_weight_rownorm_gain)."""
    if len(grads) != len(ws):
        raise ValueError("one gradient per matrix")
    _rescale(ws, grads, None, False, stream, segs)


def ds_rescale_after_step(ws: Sequence, moms: Optional[Sequence] = None,
                          radius: Optional[Sequence[float]] = None, stream=None,
                          segs: Optional[Sequence] = None) -> None:
    """In place, per matrix: project the momentum (if given), then w <- radius w/||w||."""
    _rescale(ws, moms, radius, True, stream, segs)


# ------------------------------------------------------------- token rows

# Calls of a few rows take less time on the GPU than in here, so the common
# case (the tensors' device is the current one, its current stream) enters no
# context, and sizes are asked for once.

_SAME = contextlib.nullcontext()


def _launch_on(t, stream):
    """(context, raw stream) of a call on tensor t: inside the context t's
    device is the current one and the launch stream torch's current one, so
    what is allocated there belongs to that stream."""
    torch = _torch()
    if stream is None:
        index = t.get_device()
        raw = torch.cuda.current_stream(index).cuda_stream if _raw_stream is None \
            else _raw_stream(index)
        return (_SAME if torch.cuda.current_device() == index else torch.cuda.device(index)), raw
    s = _torch_stream(t, stream)
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(t.device))
    ctx.enter_context(torch.cuda.stream(s))
    return ctx, s.cuda_stream


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(call: str, *sizes) -> int:
    n = getattr(_token_lib(), call + "_workspace")(*sizes)
    if n < 0:
        _check(n, call)
    return n


def _workspace(nbytes: int, like):
    """Scratch memory of a call, on the launch stream: dropped after the call,
    its block is handed only to work ordered after the call's kernels."""
    return like.new_empty(nbytes, dtype=_torch().uint8) if nbytes else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _value_type(t, name: str) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return DS_TYPE_F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return DS_TYPE_BF16
    raise TypeError(f"{name}: expected fp32 or bf16 data, got {t.dtype}")


def _ids(t, name: str, rows: Optional[int] = None) -> int:
    torch = _torch()
    wide = t.dtype == torch.int64
    if not (wide or t.dtype == torch.int32) or t.dim() != 1 or not t.is_contiguous() \
            or (rows is not None and t.shape[0] != rows):
        want = "[rows]" if rows is None else f"[{rows}]"
        raise ValueError(f"{name}: expected a contiguous int32 or int64 {want} tensor")
    return 8 if wide else 4


def _vec(t, name: str, n: int, dtype):
    if t is not None and (t.dtype != dtype or t.dim() != 1 or t.shape[0] != n
                          or not t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {dtype} [{n}] tensor")


def _on_device_of(first, name: str, **others):
    if not first.is_cuda:
        raise ValueError(f"{name}: must be on a HIP device")
    index = first.get_device()
    for n, t in others.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{n}: must be on the HIP device of {name}")


def ds_embed_rows(table, ids, scale: float = 1.0, out=None, stream=None):
    """out_i = bf16(scale * table[ids_i]) (bf16 [rows, cols]).

    ``table``: fp32 or bf16 [vocab, cols]; ``ids``: int32 or int64 [rows].  An
    id outside the table gives a row of zeros.
    """
    torch = _torch()
    kind = _value_type(table, "table")
    if table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table: expected a contiguous [vocab, cols] tensor")
    id_bytes = _ids(ids, "ids")
    rows, (vocab, cols) = ids.shape[0], table.shape
    if out is not None:
        _bf16_2d(out, "out", device=False)
        if tuple(out.shape) != (rows, cols):
            raise ValueError(f"out: expected [{rows}, {cols}]")
    _on_device_of(table, "table", ids=ids, out=out)
    L = _token_lib()
    ctx, raw = _launch_on(table, stream)
    with ctx:
        if out is None:
            out = table.new_empty((rows, cols), dtype=torch.bfloat16)
        st = L.ds_embed_rows(table.data_ptr(), kind, vocab, ids.data_ptr(), id_bytes, scale,
                             out.data_ptr(), rows, cols, raw)
    _check(st, "ds_embed_rows")
    return out


def ds_embed_rows_backward(dy, ids, vocab: int, scale: float = 1.0, dtable=None, dtype=None,
                           accumulate: bool = False, stream=None):
    """dtable[t] = scale * sum of dy_i over the rows with ids_i == t.

    ``dtable`` ([vocab, cols], fp32 or bf16) is allocated as ``dtype`` (fp32
    when not given) and written whole; with ``accumulate`` the sums are added
    to a given ``dtable`` and the rows of absent tokens stay as they are.
    Returns ``dtable``.
    """
    torch = _torch()
    _bf16_2d(dy, "dy", device=False)
    rows, cols = dy.shape
    id_bytes = _ids(ids, "ids", rows)
    vocab = int(vocab)
    if vocab < 0:
        raise ValueError("vocab: must not be negative")
    if dtable is not None:
        if dtype is not None and dtable.dtype != dtype:
            raise ValueError("dtable: has another dtype than the one asked for")
        if tuple(dtable.shape) != (vocab, cols) or not dtable.is_contiguous():
            raise ValueError(f"dtable: expected a contiguous [{vocab}, {cols}] tensor")
        _value_type(dtable, "dtable")
    elif accumulate:
        raise ValueError("dtable: accumulate needs one")
    elif dtype not in (None, torch.float32, torch.bfloat16):
        raise TypeError(f"dtype: expected fp32 or bf16, got {dtype}")
    _on_device_of(dy, "dy", ids=ids, dtable=dtable)
    L = _token_lib()
    nbytes = _workspace_bytes("ds_embed_rows_backward", vocab, rows, cols)
    ctx, raw = _launch_on(dy, stream)
    with ctx:
        if dtable is None:
            dtable = dy.new_empty((vocab, cols), dtype=dtype or torch.float32)
        ws = _workspace(nbytes, dy)
        st = L.ds_embed_rows_backward(dy.data_ptr(), ids.data_ptr(), id_bytes, scale,
                                      dtable.data_ptr(), _value_type(dtable, "dtable"),
                                      int(bool(accumulate)), vocab, rows, cols, _ptr(ws), nbytes,
                                      raw)
    _check(st, "ds_embed_rows_backward")
    return dtable


def _heads(t, name: str, head_dim: int, rows: Optional[int] = None) -> int:
    """Number of heads of a bf16 [rows, heads * head_dim] view (rows may be strided)."""
    torch = _torch()
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or t.dim() != 2 \
            or (t.numel() > 0 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a bf16 [rows, cols] tensor with unit column stride")
    if rows is not None and t.shape[0] != rows:
        raise ValueError(f"{name}: expected {rows} rows like q, got {t.shape[0]}")
    if t.shape[1] % head_dim:
        raise ValueError(f"{name}: its width must be a whole number of heads")
    return t.shape[1] // head_dim


def _row_stride(t) -> int:
    """A view's row stride (0 for None); a lone row's may be anything, and is
    not read."""
    if t is None:
        return 0
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


def _qk_rms_checks(q, k, positions, inv_freq, q_weight, k_weight, head_dim):
    torch = _torch()
    if head_dim <= 0:
        raise ValueError("head_dim: must be positive")
    nq = _heads(q, "q", head_dim)
    nk = _heads(k, "k", head_dim, q.shape[0]) if k is not None else 0
    _vec(positions, "positions", q.shape[0], torch.int32)
    _vec(inv_freq, "inv_freq", head_dim // 2, torch.float32)
    _vec(q_weight, "q_weight", head_dim, torch.float32)
    _vec(k_weight, "k_weight", head_dim, torch.float32)
    return nq, nk


def _like_heads(t, like, name: str, head_dim: int, rows: int, heads: int):
    """A given output or gradient must hold exactly the heads of ``like``."""
    if t is None:
        return
    if like is None:
        raise ValueError(f"{name}: given without k")
    if _heads(t, name, head_dim, rows) != heads:
        raise ValueError(f"{name}: expected [{rows}, {heads * head_dim}]")


def ds_qk_rows_rms(q, k, positions, inv_freq, q_weight, k_weight, head_dim: int,
                   eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Each head's RMS norm times a learned weight, then rotate-half RoPE, on
    q [rows, nq * head_dim] and k [rows, nk * head_dim] (k may be None).

    ``q``/``k`` may be strided row views (a fused projection's slices);
    ``positions``: int32 [rows]; ``inv_freq``: fp32 [head_dim / 2]; weights:
    fp32 [head_dim] or None (1).  Returns (q_out, k_out); the outputs may be
    the inputs themselves.
    """
    torch = _torch()
    head_dim = int(head_dim)
    nq, nk = _qk_rms_checks(q, k, positions, inv_freq, q_weight, k_weight, head_dim)
    rows = q.shape[0]
    _like_heads(q_out, q, "q_out", head_dim, rows, nq)
    _like_heads(k_out, k, "k_out", head_dim, rows, nk)
    _on_device_of(q, "q", k=k, positions=positions, inv_freq=inv_freq, q_weight=q_weight,
                  k_weight=k_weight, q_out=q_out, k_out=k_out)
    L = _token_lib()
    ctx, raw = _launch_on(q, stream)
    with ctx:
        if q_out is None:
            q_out = q.new_empty((rows, nq * head_dim))
        if k is not None and k_out is None:
            k_out = k.new_empty((rows, nk * head_dim))
        st = L.ds_qk_rows_rms(
            q.data_ptr(), _row_stride(q), _ptr(k), _row_stride(k), positions.data_ptr(),
            inv_freq.data_ptr(), _ptr(q_weight), _ptr(k_weight), q_out.data_ptr(),
            _row_stride(q_out), _ptr(k_out), _row_stride(k_out), rows, nq, nk, head_dim, eps, raw)
    _check(st, "ds_qk_rows_rms")
    return q_out, k_out


def ds_qk_rows_rms_backward(q, k, positions, inv_freq, q_weight, k_weight, dq_out, dk_out,
                            head_dim: int, eps: float = 1e-6, dq=None, dk=None,
                            want_dweights: bool = True, stream=None):
    """The gradient of ds_qk_rows_rms(q, k, ...) from the gradients reaching
    its outputs.  Returns (dq, dk, dq_weight, dk_weight): bf16 like q and k
    (``dq`` may be ``dq_out`` or ``q``, ``dk`` likewise), the weights' fp32
    [head_dim], or None without ``want_dweights`` (and for k without k).
    """
    torch = _torch()
    head_dim = int(head_dim)
    nq, nk = _qk_rms_checks(q, k, positions, inv_freq, q_weight, k_weight, head_dim)
    rows = q.shape[0]
    _like_heads(dq_out, q, "dq_out", head_dim, rows, nq)
    if k is not None and dk_out is None:
        raise ValueError("dk_out: missing")
    _like_heads(dk_out, k, "dk_out", head_dim, rows, nk)
    _like_heads(dq, q, "dq", head_dim, rows, nq)
    _like_heads(dk, k, "dk", head_dim, rows, nk)
    _on_device_of(q, "q", k=k, positions=positions, inv_freq=inv_freq, q_weight=q_weight,
                  k_weight=k_weight, dq_out=dq_out, dk_out=dk_out, dq=dq, dk=dk)
    L = _token_lib()
    nbytes = _workspace_bytes("ds_qk_rows_rms_backward", rows, nq, nk, head_dim) \
        if want_dweights else 0
    ctx, raw = _launch_on(q, stream)
    with ctx:
        if dq is None:
            dq = q.new_empty((rows, nq * head_dim))
        if k is not None and dk is None:
            dk = k.new_empty((rows, nk * head_dim))
        dqw = dkw = None
        if want_dweights:
            dqw = q.new_empty(head_dim, dtype=torch.float32)
            dkw = q.new_empty(head_dim, dtype=torch.float32) if k is not None else None
        ws = _workspace(nbytes, q)
        st = L.ds_qk_rows_rms_backward(
            q.data_ptr(), _row_stride(q), _ptr(k), _row_stride(k), positions.data_ptr(),
            inv_freq.data_ptr(), _ptr(q_weight), _ptr(k_weight), dq_out.data_ptr(),
            _row_stride(dq_out), _ptr(dk_out), _row_stride(dk_out), dq.data_ptr(), _row_stride(dq),
            _ptr(dk), _row_stride(dk), _ptr(dqw), _ptr(dkw), rows, nq, nk, head_dim, eps, _ptr(ws),
            nbytes, raw)
    _check(st, "ds_qk_rows_rms_backward")
    return dq, dk, dqw, dkw


class LogprobRows(NamedTuple):
    """What ds_logprob_rows returns: fp32 [rows] each; the top alternatives'
    int32 ids and fp32 log probabilities, [rows, top_k]."""
    logp: object
    entropy: object
    lse: object
    top_ids: object
    top_logp: object


def _logits(t, name: str):
    kind = _value_type(t, name)
    if t.dim() != 2 or (t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a [rows, vocab] tensor with unit column stride")
    rows, vocab = t.shape
    return kind, rows, vocab, (t.stride(0) if rows > 1 else vocab)


def ds_logprob_rows(logits, labels=None, scale=None, inv_temp: float = 1.0, top_k: int = 0,
                    stream=None) -> LogprobRows:
    """Per row of logits [rows, vocab] (fp32 or bf16; rows may be strided): the
    log probability of its label, the entropy, log sum exp, and the ``top_k``
    largest tokens, of z = logits * scale * inv_temp.

    ``labels``: int32 or int64 [rows], one outside the vocabulary marks a row
    to ignore (logp 0); without labels logp is None.  ``scale``: fp32 [vocab]
    or None.  top_ids and top_logp are None for top_k 0.
    """
    torch = _torch()
    kind, rows, vocab, ld = _logits(logits, "logits")
    label_bytes = 8 if labels is None else _ids(labels, "labels", rows)
    _vec(scale, "scale", vocab, torch.float32)
    top_k = int(top_k)
    if not 0 <= top_k <= min(DS_MAX_TOP, vocab):
        raise ValueError(f"top_k: expected 0 to {min(DS_MAX_TOP, vocab)}")
    _on_device_of(logits, "logits", labels=labels, scale=scale)
    L = _token_lib()
    nbytes = _workspace_bytes("ds_logprob_rows", rows, vocab, top_k)
    ctx, raw = _launch_on(logits, stream)
    with ctx:
        lse, entropy, logp = logits.new_empty((3, rows), dtype=torch.float32).unbind()
        if labels is None:
            logp = None
        ids = top = None
        if top_k:
            ids = logits.new_empty((rows, top_k), dtype=torch.int32)
            top = logits.new_empty((rows, top_k), dtype=torch.float32)
        ws = _workspace(nbytes, logits)
        st = L.ds_logprob_rows(logits.data_ptr(), kind, ld, _ptr(scale), inv_temp, _ptr(labels),
                               label_bytes, _ptr(logp), entropy.data_ptr(), lse.data_ptr(),
                               _ptr(ids), _ptr(top), top_k, rows, vocab, _ptr(ws), nbytes, raw)
    _check(st, "ds_logprob_rows")
    return LogprobRows(logp, entropy, lse, ids, top)


def ds_logprob_rows_backward(logits, labels, lse, entropy, dlogp, dentropy=None, scale=None,
                             inv_temp: float = 1.0, dlogits=None, want_dscale: bool = True,
                             stream=None):
    """The gradient of ds_logprob_rows' logp and entropy: (dlogits, dscale).

    ``lse`` and ``entropy`` are the forward call's (entropy may be None
    without ``dentropy``; a row with ``|lse| >= 2**24`` then gets no gradient,
    and with it only if one token holds its maximum alone);
    ``dlogp``/``dentropy``: fp32 [rows] or None.
    ``dlogits`` (like logits; may be logits itself) is allocated contiguous
    when not given; dscale is None without ``scale`` or ``want_dscale``.
    """
    torch = _torch()
    kind, rows, vocab, ld = _logits(logits, "logits")
    label_bytes = 8 if labels is None else _ids(labels, "labels", rows)
    if dlogp is not None and labels is None:
        raise ValueError("labels: dlogp needs them")
    if dentropy is not None and entropy is None:
        raise ValueError("entropy: dentropy needs the forward call's")
    if lse is None:
        raise ValueError("lse: the forward call's is needed")
    for t, n in ((lse, "lse"), (entropy, "entropy"), (dlogp, "dlogp"), (dentropy, "dentropy")):
        _vec(t, n, rows, torch.float32)
    _vec(scale, "scale", vocab, torch.float32)
    ldo = vocab
    if dlogits is not None:
        if dlogits.dtype != logits.dtype or tuple(dlogits.shape) != (rows, vocab):
            raise ValueError(f"dlogits: expected a [{rows}, {vocab}] tensor like logits")
        ldo = _logits(dlogits, "dlogits")[3]
    _on_device_of(logits, "logits", labels=labels, lse=lse, entropy=entropy, dlogp=dlogp,
                  dentropy=dentropy, scale=scale, dlogits=dlogits)
    L = _token_lib()
    want_dscale = scale is not None and want_dscale
    nbytes = _workspace_bytes("ds_logprob_rows_backward", rows, vocab) if want_dscale else 0
    ctx, raw = _launch_on(logits, stream)
    with ctx:
        if dlogits is None:
            dlogits = logits.new_empty((rows, vocab))
        dscale = logits.new_empty(vocab, dtype=torch.float32) if want_dscale else None
        ws = _workspace(nbytes, logits)
        st = L.ds_logprob_rows_backward(
            logits.data_ptr(), kind, ld, _ptr(scale), inv_temp, _ptr(labels), label_bytes,
            lse.data_ptr(), _ptr(entropy), _ptr(dlogp), _ptr(dentropy), dlogits.data_ptr(), ldo,
            _ptr(dscale), rows, vocab, _ptr(ws), nbytes, raw)
    _check(st, "ds_logprob_rows_backward")
    return dlogits, dscale
