"""ctypes binding of the low-precision operators (include/distgemm_mx.h):
microscaled (MX) tensors, their products, and the RMS norm that feeds them.

Every function mirrors a C entry point; GPU tensors are checked for type,
shape and layout before their addresses are passed.  Nothing is allocated: the
caller owns every output.  There is no fallback.

An MX tensor is a pair of GPU tensors, codes and scales: codes are rows x cols
(``E4M3``, torch.float8_e4m3fn or uint8) or rows x cols / 2 (``E2M1``, uint8,
two per byte, the even element low), scales rows x
``dist_gemm_mx_scale_pitch(cols)`` uint8 or torch.float8_e8m0fnu.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import _enum, DistGemmError, lib

ELEMS = {"F32": 0, "BF16": 1}
MX_FORMATS = {"E2M1": 0, "E4M3": 1}
NORM_OUTPUTS = {"SAME": 0, "E4M3": 1, "MX_E2M1": 2, "MX_E4M3": 3}

# C functions declared in include/distgemm_mx.h (checked by the CPU tests)
MX_C_FUNCTIONS = ("dist_gemm_mx_scale_pitch", "dist_gemm_mx_quantize", "dist_gemm_mx_dequantize",
                  "dist_gemm_rms_norm", "dist_gemm_rms_norm_workspace", "dist_gemm_rms_norm_backward",
                  "dist_gemm_mx_plan", "dist_gemm_mx_run", "dist_gemm_mx_destroy", "dist_gemm_mx_last_error")

_i64, _i32, _f32, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
lib.dist_gemm_mx_scale_pitch.argtypes = [_i64]
lib.dist_gemm_mx_scale_pitch.restype = _i64
lib.dist_gemm_mx_quantize.argtypes = [_vp, _i64, _i32, _i64, _i64, _i32, _vp, _vp, _vp]
lib.dist_gemm_mx_dequantize.argtypes = [_vp, _vp, _i32, _i64, _i64, _vp, _i64, _i32, _vp]
lib.dist_gemm_rms_norm.argtypes = [_vp, _i64, _vp, _i64, _vp, _i32, _i64, _i64, _f32, _i32, _f32, _vp, _i64, _vp,
                                   _vp, _i64, _vp, _vp]
lib.dist_gemm_rms_norm_workspace.argtypes = [_i64, _i64]
lib.dist_gemm_rms_norm_workspace.restype = _i64
lib.dist_gemm_rms_norm_backward.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _i64, _i64, _vp, _i64,
                                            _vp, _vp, _i64, _vp]
lib.dist_gemm_mx_plan.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32, ctypes.POINTER(_vp)]
lib.dist_gemm_mx_run.argtypes = [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _f32, _f32, _vp]
lib.dist_gemm_mx_destroy.argtypes = [_vp]
lib.dist_gemm_mx_last_error.argtypes = [_vp]
lib.dist_gemm_mx_last_error.restype = ctypes.c_char_p
for _name in ("dist_gemm_mx_quantize", "dist_gemm_mx_dequantize", "dist_gemm_rms_norm", "dist_gemm_rms_norm_backward",
              "dist_gemm_mx_plan", "dist_gemm_mx_run", "dist_gemm_mx_destroy"):
    getattr(lib, _name).restype = _i32

_ELEM_OF = {torch.float32: 0, torch.bfloat16: 1}
_DTYPE_OF = {0: torch.float32, 1: torch.bfloat16}
_BYTES = (torch.uint8, torch.float8_e4m3fn)
_SCALES = (torch.uint8, torch.float8_e8m0fnu)


def _raise(rc: int, plan=None):
    msg = lib.dist_gemm_mx_last_error(plan)
    raise DistGemmError(rc, msg.decode() if msg else "")


_raw_stream, _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _stream_of(stream, device: int) -> Optional[int]:
    if stream is None:
        return _raw_stream(device) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


# A call of a few microseconds is mostly these checks and the launch: each is
# one comparison where the argument is right, and the message is made where not.

def _device(t, name) -> int:
    """The device of an operator's first tensor, which has to be the current one."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    if d != _current():
        raise ValueError(f"{name} is on GPU {d}, which is not the current device")
    return d


def _rows(t, name, dtype, shape, device) -> int:
    """Checks a matrix whose rows are contiguous; its leading dimension."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _wrong(t, name, (dtype,), tuple(shape), device)
    s0, s1 = t.stride()
    rows, cols = shape
    if s1 != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if s0 < cols:
        if rows > 1:
            raise ValueError(f"the rows of {name} overlap")
        return cols
    return s0


def _flat(t, name, dtypes, count, device):
    """Checks a tensor of `count` elements without gaps."""
    if t.dtype not in dtypes or t.numel() != count or not t.is_contiguous() or t.get_device() != device:
        _wrong(t, name, dtypes, count, device)


def _wrong(t, name, dtypes, size, device):
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, is {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on GPU {device}")
    if isinstance(size, tuple):
        raise ValueError(f"{name} must be {' x '.join(map(str, size))}, is {tuple(t.shape)}")
    if t.numel() != size:
        raise ValueError(f"{name} must have {size} elements, has {t.numel()}")
    raise ValueError(f"{name} must be contiguous")


def _matrix(t, name):
    """(device, element type, shape) of an operator's first tensor."""
    d = _device(t, name)
    e = _ELEM_OF.get(t.dtype)
    if e is None:
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, is {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix")
    return d, e, shape


def _format(f) -> int:
    v = MX_FORMATS.get(f, f)
    if v not in (0, 1):
        raise ValueError(f"unknown MX format {f!r}")
    return v


def dist_gemm_mx_scale_pitch(cols: int) -> int:
    """Bytes of one row of scales: cols / 32 rounded up to a multiple of 16."""
    return lib.dist_gemm_mx_scale_pitch(cols)


def _mx_pair(codes, scales, fmt, rows, cols, device, name=""):
    _flat(codes, f"{name}codes", _BYTES if fmt else (torch.uint8,), rows * cols // (1 if fmt else 2), device)
    _flat(scales, f"{name}scales", _SCALES, rows * ((cols // 32 + 15) // 16 * 16), device)


def dist_gemm_mx_quantize(x, format, codes, scales, stream=None):
    """Quantise x (rows x cols, f32 or bf16, rows at any pitch) to the MX tensor (codes, scales)."""
    d, e, shape = _matrix(x, "x")
    fmt = _format(format)
    rows, cols = shape
    ld = _rows(x, "x", x.dtype, shape, d)
    _mx_pair(codes, scales, fmt, rows, cols, d)
    rc = lib.dist_gemm_mx_quantize(x.data_ptr(), ld, e, rows, cols, fmt, codes.data_ptr(), scales.data_ptr(),
                                   _stream_of(stream, d))
    if rc:
        _raise(rc)


def dist_gemm_mx_dequantize(codes, scales, format, y, stream=None):
    """The values of the MX tensor (codes, scales) into y (rows x cols, f32 or bf16, rows at any pitch)."""
    d, e, shape = _matrix(y, "y")
    fmt = _format(format)
    rows, cols = shape
    ld = _rows(y, "y", y.dtype, shape, d)
    _mx_pair(codes, scales, fmt, rows, cols, d)
    rc = lib.dist_gemm_mx_dequantize(codes.data_ptr(), scales.data_ptr(), fmt, rows, cols, y.data_ptr(), ld, e,
                                     _stream_of(stream, d))
    if rc:
        _raise(rc)


def dist_gemm_rms_norm(x, weight, y, eps=1e-6, output="SAME", residual=None, h=None, rstd=None, scales=None,
                       scale=1.0, stream=None):
    """RMS norm of x's rows (of h = x + residual, which is kept, if there is a residual).

    output: "SAME" (y of x's type), "E4M3" (y holds e4m3 of the result over
    `scale`, the operand of an E4M3 plan with that scale), "MX_E4M3" or
    "MX_E2M1" (y the codes and `scales` the scales of an MX tensor)."""
    d, e, shape = _matrix(x, "x")
    out = NORM_OUTPUTS.get(output, -1)
    t = x.dtype
    rows, cols = shape
    ldx = _rows(x, "x", t, shape, d)
    _flat(weight, "weight", (t,), cols, d)
    ldr = ldh = ldy = 0
    pr = ph = ps = pt = None
    if residual is not None and h is not None:
        ldr, ldh = _rows(residual, "residual", t, shape, d), _rows(h, "h", t, shape, d)
        pr, ph = residual.data_ptr(), h.data_ptr()
    elif residual is not None or h is not None:
        raise ValueError("residual and h go together")
    if rstd is not None:
        _flat(rstd, "rstd", (torch.float32,), rows, d)
        pt = rstd.data_ptr()
    if out == 0:
        ldy = _rows(y, "y", t, shape, d)
    elif out == 1:
        if y.dtype not in _BYTES:
            _wrong(y, "y", _BYTES, tuple(shape), d)
        ldy = _rows(y, "y", y.dtype, shape, d)
    elif out > 1:
        if scales is None:
            raise ValueError("an MX output needs scales")
        _mx_pair(y, scales, out - 2, rows, cols, d)
        ps = scales.data_ptr()
    else:
        raise ValueError(f"unknown output {output!r}")
    rc = lib.dist_gemm_rms_norm(x.data_ptr(), ldx, pr, ldr, weight.data_ptr(), e, rows, cols, eps, out, scale,
                                y.data_ptr(), ldy, ps, ph, ldh, pt, _stream_of(stream, d))
    if rc:
        _raise(rc)


def dist_gemm_rms_norm_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace that dist_gemm_rms_norm_backward needs."""
    return lib.dist_gemm_rms_norm_workspace(rows, cols)


def dist_gemm_rms_norm_backward(dy, h, rstd, weight, dx, dweight, workspace, dh=None, stream=None):
    """Gradient of dist_gemm_rms_norm: dx (+ dh, the residual stream's own gradient) and dweight (fp32)."""
    d, e, shape = _matrix(h, "h")
    t = h.dtype
    rows, cols = shape
    ldh, lddy, lddx = _rows(h, "h", t, shape, d), _rows(dy, "dy", t, shape, d), _rows(dx, "dx", t, shape, d)
    lddh = 0 if dh is None else _rows(dh, "dh", t, shape, d)
    _flat(weight, "weight", (t,), cols, d)
    _flat(rstd, "rstd", (torch.float32,), rows, d)
    _flat(dweight, "dweight", (torch.float32,), cols, d)
    if workspace.get_device() != d or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous, on GPU {d}")
    rc = lib.dist_gemm_rms_norm_backward(dy.data_ptr(), lddy, h.data_ptr(), ldh, None if dh is None else dh.data_ptr(),
                                         lddh, rstd.data_ptr(), weight.data_ptr(), e, rows, cols, dx.data_ptr(), lddx,
                                         dweight.data_ptr(), workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), _stream_of(stream, d))
    if rc:
        _raise(rc)


class MxPlan:
    """Products of MX tensors with up to M rows: D = alpha * A * B^T + beta * C (+ bias).

    groups = 0: B is N x K.  groups > 0: B is groups x N x K (and a bias groups
    x N), and `offsets` (groups + 1 int32 on the GPU) says which rows of A each
    group has.  A is in `a_format`, B in E2M1, C, D and bias in `out_dtype`."""

    def __init__(self, M, N, K, groups=0, a_format="E2M1", out_dtype="BF16"):
        self.M, self.N, self.K, self.groups = M, N, K, groups
        self.a_format = _format(a_format)
        self.out = _enum(ELEMS, out_dtype)
        self.handle = None
        h = ctypes.c_void_p()
        rc = lib.dist_gemm_mx_plan(M, N, K, groups, self.a_format, self.out, ctypes.byref(h))
        if rc:
            _raise(rc)
        self.handle = h
        self._dtype = _DTYPE_OF[self.out]
        self.device = torch._C._cuda_getDevice()
        # elements per row of A, and of B with its scales
        self._ka, self._pitch = K // (1 if self.a_format else 2), (K // 32 + 15) // 16 * 16
        self._nb, self._ns = max(groups, 1) * N * (K // 2), max(groups, 1) * N * self._pitch

    def run(self, A, A_scales, B, B_scales, D, bias=None, C=None, alpha=1.0, beta=0.0, offsets=None, stream=None):
        """One product of D's rows (at most M)."""
        if self.handle is None:
            raise ValueError("the plan is closed")
        d, N = self.device, self.N
        shape = D.shape
        rows = shape[0]
        if len(shape) != 2 or shape[1] != N:
            raise ValueError(f"D must be rows x {N}, is {tuple(shape)}")
        ldd = _rows(D, "D", self._dtype, shape, d)
        _flat(A, "A", _BYTES if self.a_format else (torch.uint8,), rows * self._ka, d)
        _flat(A_scales, "A_scales", _SCALES, rows * self._pitch, d)
        _flat(B, "B", (torch.uint8,), self._nb, d)
        _flat(B_scales, "B_scales", _SCALES, self._ns, d)
        ldc, pc, pb, po = 0, None, None, None
        if C is not None:
            ldc, pc = _rows(C, "C", self._dtype, shape, d), C.data_ptr()
        if bias is not None:
            _flat(bias, "bias", (self._dtype,), max(self.groups, 1) * N, d)
            pb = bias.data_ptr()
        if offsets is not None:
            _flat(offsets, "offsets", (torch.int32,), self.groups + 1, d)
            po = offsets.data_ptr()
        rc = lib.dist_gemm_mx_run(self.handle, rows, A.data_ptr(), A_scales.data_ptr(), B.data_ptr(),
                                  B_scales.data_ptr(), pc, ldc, D.data_ptr(), ldd, pb, po, alpha, beta,
                                  _stream_of(stream, d))
        if rc:
            _raise(rc, self.handle)

    def close(self):
        if self.handle is not None:
            lib.dist_gemm_mx_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
