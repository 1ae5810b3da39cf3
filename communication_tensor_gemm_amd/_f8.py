"""ctypes binding of the 8-bit training operators (include/distgemm_f8.h):
tensors of E4M3 elements with a scale per block of 128 (F8 tensors), their
transposition and products, and the layer norm with its gradient.

Every function mirrors a C entry point; GPU tensors are checked for type,
shape and layout before their addresses are passed.  Nothing is allocated: the
caller owns every output.  There is no fallback.

An F8 tensor of rows x cols values is a pair of GPU tensors: codes, rows x
``dist_gemm_f8_pitch(cols)`` torch.float8_e4m3fn or uint8 (zero past cols), and
scales, rows x ``dist_gemm_f8_scale_pitch(cols)`` uint8 or
torch.float8_e8m0fnu.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import DistGemmError, lib
from ._mx import _BYTES, _ELEM_OF, _SCALES, _current, _device, _flat, _matrix, _rows, _stream_of, _wrong

LAYER_NORM_OUTPUTS = {"SAME": 0, "E4M3": 1, "F8": 2}

# C functions declared in include/distgemm_f8.h (checked by the CPU tests)
F8_C_FUNCTIONS = ("dist_gemm_f8_pitch", "dist_gemm_f8_scale_pitch", "dist_gemm_f8_quantize", "dist_gemm_f8_dequantize",
                  "dist_gemm_f8_transpose", "dist_gemm_f8_product_workspace", "dist_gemm_f8_product",
                  "dist_gemm_layer_norm", "dist_gemm_layer_norm_workspace", "dist_gemm_layer_norm_backward",
                  "dist_gemm_f8_last_error")

_i64, _i32, _f32, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
lib.dist_gemm_f8_pitch.argtypes = lib.dist_gemm_f8_scale_pitch.argtypes = [_i64]
lib.dist_gemm_f8_quantize.argtypes = [_vp, _i64, _i32, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp]
lib.dist_gemm_f8_dequantize.argtypes = [_vp, _vp, _i64, _i64, _vp, _i64, _i32, _vp]
lib.dist_gemm_f8_transpose.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp]
lib.dist_gemm_f8_product_workspace.argtypes = [_i64, _i64, _i64]
lib.dist_gemm_f8_product.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _f32, _f32,
                                     _vp, _i64, _vp]
lib.dist_gemm_layer_norm.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _i32, _i64, _i64, _f32, _i32, _f32, _vp, _i64, _vp,
                                     _vp, _i64, _vp, _vp, _vp, _vp, _vp]
lib.dist_gemm_layer_norm_workspace.argtypes = [_i64, _i64]
lib.dist_gemm_layer_norm_backward.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i32, _i64, _i64, _vp,
                                              _i64, _vp, _vp, _vp, _i64, _vp]
lib.dist_gemm_f8_last_error.argtypes = []
lib.dist_gemm_f8_last_error.restype = ctypes.c_char_p
for _name in ("dist_gemm_f8_pitch", "dist_gemm_f8_scale_pitch", "dist_gemm_f8_product_workspace",
              "dist_gemm_layer_norm_workspace"):
    getattr(lib, _name).restype = _i64
for _name in ("dist_gemm_f8_quantize", "dist_gemm_f8_dequantize", "dist_gemm_f8_transpose", "dist_gemm_f8_product",
              "dist_gemm_layer_norm", "dist_gemm_layer_norm_backward"):
    getattr(lib, _name).restype = _i32


def _raise(rc: int):
    msg = lib.dist_gemm_f8_last_error()
    raise DistGemmError(rc, msg.decode() if msg else "")


def dist_gemm_f8_pitch(cols: int) -> int:
    """Bytes of one row of codes: cols rounded up to a multiple of 128."""
    return lib.dist_gemm_f8_pitch(cols)


def dist_gemm_f8_scale_pitch(cols: int) -> int:
    """Bytes of one row of scales: the blocks of 128 rounded up to a multiple of 16."""
    return lib.dist_gemm_f8_scale_pitch(cols)


# As in _mx.py: each check is one comparison where the argument is right, and
# the functions that take the argument apart make the message where it is not.

def _first(t, name):
    """(device, element type, rows, cols, leading dimension) of an operator's first matrix."""
    d, e = t.get_device(), _ELEM_OF.get(t.dtype)
    if d < 0 or d != _current() or e is None or t.dim() != 2:
        _matrix(t, name)
    rows, cols = t.shape
    s0, s1 = t.stride()
    if s0 < cols or s1 != 1:
        s0 = _rows(t, name, t.dtype, t.shape, d)
    return d, e, rows, cols, s0


def _f8_pair(codes, scales, rows, blocks, device, name="codes", scales_name="scales"):
    """Checks an F8 tensor of `rows` rows of `blocks` blocks of 128; its two addresses."""
    if (codes.dtype not in _BYTES or codes.numel() != rows * blocks * 128 or not codes.is_contiguous()
            or codes.get_device() != device):
        _wrong(codes, name, _BYTES, rows * blocks * 128, device)
    if (scales.dtype not in _SCALES or scales.numel() != rows * ((blocks + 15) // 16 * 16) or not scales.is_contiguous()
            or scales.get_device() != device):
        _wrong(scales, scales_name, _SCALES, rows * ((blocks + 15) // 16 * 16), device)
    return codes.data_ptr(), scales.data_ptr()


def _pair_or_none(codes, scales, rows, blocks, device, name, scales_name):
    if codes is not None and scales is not None:
        return _f8_pair(codes, scales, rows, blocks, device, name, scales_name)
    if codes is not None or scales is not None:
        raise ValueError(f"{name} and {scales_name} go together")
    return None, None


def _workspace(t, device):
    """(address, bytes) of a workspace, or of none."""
    if t is None:
        return None, 0
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"the workspace must be contiguous, on GPU {device}")
    return t.data_ptr(), t.numel() * t.element_size()


def dist_gemm_f8_quantize(x, codes=None, scales=None, codes_t=None, scales_t=None, block_rows=1, stream=None):
    """Quantise x (rows x cols, f32 or bf16, rows at any pitch) to the F8 tensor
    (codes, scales) and / or that of its transpose (codes_t, scales_t).

    block_rows = 128: blocks of 128 x 128 share a scale (weights)."""
    d, e, rows, cols, ld = _first(x, "x")
    pc, ps = _pair_or_none(codes, scales, rows, (cols + 127) // 128, d, "codes", "scales")
    pct, pst = _pair_or_none(codes_t, scales_t, cols, (rows + 127) // 128, d, "codes_t", "scales_t")
    rc = lib.dist_gemm_f8_quantize(x.data_ptr(), ld, e, rows, cols, block_rows, pc, ps, pct, pst, _stream_of(stream, d))
    if rc:
        _raise(rc)


def dist_gemm_f8_dequantize(codes, scales, y, stream=None):
    """The values of the F8 tensor (codes, scales) into y (rows x cols, f32 or bf16, rows at any pitch)."""
    d, e, rows, cols, ld = _first(y, "y")
    pc, ps = _f8_pair(codes, scales, rows, (cols + 127) // 128, d)
    rc = lib.dist_gemm_f8_dequantize(pc, ps, rows, cols, y.data_ptr(), ld, e, _stream_of(stream, d))
    if rc:
        _raise(rc)


def _codes(t, name):
    if len(t.shape) != 2:
        raise ValueError(f"{name} must be a matrix: rows x dist_gemm_f8_pitch(cols)")
    return t.shape


def dist_gemm_f8_transpose(codes, scales, codes_t, scales_t, stream=None):
    """The F8 tensor (codes_t, scales_t) of the transpose of the F8 tensor (codes, scales).

    The sizes are the two tensors' rows: codes is rows x pitch(cols), codes_t cols x pitch(rows)."""
    d = _device(codes, "codes")
    rows, cols = _codes(codes, "codes")[0], _codes(codes_t, "codes_t")[0]
    pc, ps = _f8_pair(codes, scales, rows, (cols + 127) // 128, d)
    pct, pst = _f8_pair(codes_t, scales_t, cols, (rows + 127) // 128, d, "codes_t", "scales_t")
    rc = lib.dist_gemm_f8_transpose(pc, ps, rows, cols, pct, pst, _stream_of(stream, d))
    if rc:
        _raise(rc)


def dist_gemm_f8_product_workspace(M: int, N: int, K: int) -> int:
    """Bytes of workspace that dist_gemm_f8_product needs on the current device (K: the operands' pitch)."""
    return lib.dist_gemm_f8_product_workspace(M, N, K)


def dist_gemm_f8_product(A, A_scales, B, B_scales, D, bias=None, C=None, alpha=1.0, beta=0.0, workspace=None, stream=None):
    """D = alpha * A * B^T + beta * C (+ bias) of the F8 tensors A (M x K) and B (N x K); D, C and bias f32 or bf16.

    K is the operands' pitch (their codes' second size); workspace: any GPU
    tensor of at least dist_gemm_f8_product_workspace(M, N, K) bytes."""
    d, e, M, N, ldd = _first(D, "D")
    K = _codes(A, "A")[1]
    if K % 128 or _codes(B, "B")[1] != K:
        raise ValueError(f"A and B must have rows of one pitch (a multiple of 128), have {K} and {B.shape[1]}")
    pa, pas = _f8_pair(A, A_scales, M, K // 128, d, "A", "A_scales")
    pb, pbs = _f8_pair(B, B_scales, N, K // 128, d, "B", "B_scales")
    ldc, pc, pbias = 0, None, None
    if C is not None:
        ldc, pc = _rows(C, "C", D.dtype, D.shape, d), C.data_ptr()
    if bias is not None:
        _flat(bias, "bias", (D.dtype,), N, d)
        pbias = bias.data_ptr()
    pw, wb = _workspace(workspace, d)
    rc = lib.dist_gemm_f8_product(pa, pas, pb, pbs, M, N, K, pc, ldc, D.data_ptr(), ldd, e, pbias, alpha, beta, pw, wb,
                                  _stream_of(stream, d))
    if rc:
        _raise(rc)


def dist_gemm_layer_norm(x, weight, bias, y, eps=1e-5, output="SAME", residual=None, h=None, mean=None, rstd=None,
                         scales=None, scale=1.0, kept=None, kept_scales=None, stream=None):
    """Layer norm of x's rows (of h = x + residual, which is kept, if there is a residual); bias may be None.

    output: "SAME" (y of x's type), "E4M3" (y holds e4m3 of the result over
    `scale`) or "F8" (y the codes and `scales` the scales of an F8 tensor).
    kept, kept_scales: room for the normalised rows as an F8 tensor, the 8-bit
    checkpoint for the gradient."""
    d, e, rows, cols, ldx = _first(x, "x")
    out = LAYER_NORM_OUTPUTS.get(output, -1)
    t, blocks = x.dtype, (cols + 127) // 128
    _flat(weight, "weight", (t,), cols, d)
    ldr = ldh = ldy = 0
    pr = ph = ps = pm = pt = pbias = None
    if bias is not None:
        _flat(bias, "bias", (t,), cols, d)
        pbias = bias.data_ptr()
    if residual is not None and h is not None:
        shape = x.shape
        ldr, ldh = _rows(residual, "residual", t, shape, d), _rows(h, "h", t, shape, d)
        pr, ph = residual.data_ptr(), h.data_ptr()
    elif residual is not None or h is not None:
        raise ValueError("residual and h go together")
    if mean is not None:
        _flat(mean, "mean", (torch.float32,), rows, d)
        pm = mean.data_ptr()
    if rstd is not None:
        _flat(rstd, "rstd", (torch.float32,), rows, d)
        pt = rstd.data_ptr()
    if out == 0:
        ldy = _rows(y, "y", t, x.shape, d)
    elif out == 1:
        if y.dtype not in _BYTES:
            _wrong(y, "y", _BYTES, tuple(x.shape), d)
        ldy = _rows(y, "y", y.dtype, x.shape, d)
    elif out == 2:
        if scales is None:
            raise ValueError("an F8 output needs scales")
        _, ps = _f8_pair(y, scales, rows, blocks, d, "y")
    else:
        raise ValueError(f"unknown output {output!r}")
    pk, pks = _pair_or_none(kept, kept_scales, rows, blocks, d, "kept", "kept_scales")
    rc = lib.dist_gemm_layer_norm(x.data_ptr(), ldx, pr, ldr, weight.data_ptr(), pbias, e, rows, cols, eps, out, scale,
                                  y.data_ptr(), ldy, ps, ph, ldh, pm, pt, pk, pks, _stream_of(stream, d))
    if rc:
        _raise(rc)


def dist_gemm_layer_norm_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace that dist_gemm_layer_norm_backward needs."""
    return lib.dist_gemm_layer_norm_workspace(rows, cols)


def dist_gemm_layer_norm_backward(dy, h, mean, rstd, weight, dx, dweight, dbias, workspace, dh=None, h_scales=None,
                                  stream=None):
    """Gradient of dist_gemm_layer_norm: dx (+ dh, the residual stream's own gradient), dweight and dbias (fp32; dbias
    may be None).

    h is the normalised stream itself (dy's type, with mean), or with h_scales
    the F8 tensor of the normalised rows that the forward pass kept (mean is
    not used and may be None)."""
    d, e, rows, cols, lddy = _first(dy, "dy")
    t, shape = dy.dtype, dy.shape
    lddx = _rows(dx, "dx", t, shape, d)
    lddh = 0 if dh is None else _rows(dh, "dh", t, shape, d)
    ldh, phs, pm, pdb = 0, None, None, None
    if h_scales is not None:
        ph, phs = _f8_pair(h, h_scales, rows, (cols + 127) // 128, d, "h", "h_scales")
    else:
        ldh, ph = _rows(h, "h", t, shape, d), h.data_ptr()
        if mean is None:
            raise ValueError("mean is needed with h in its own type")
        _flat(mean, "mean", (torch.float32,), rows, d)
        pm = mean.data_ptr()
    _flat(weight, "weight", (t,), cols, d)
    _flat(rstd, "rstd", (torch.float32,), rows, d)
    _flat(dweight, "dweight", (torch.float32,), cols, d)
    if dbias is not None:
        _flat(dbias, "dbias", (torch.float32,), cols, d)
        pdb = dbias.data_ptr()
    pw, wb = _workspace(workspace, d)
    rc = lib.dist_gemm_layer_norm_backward(dy.data_ptr(), lddy, ph, ldh, phs, None if dh is None else dh.data_ptr(), lddh,
                                           pm, rstd.data_ptr(), weight.data_ptr(), e, rows, cols, dx.data_ptr(), lddx,
                                           dweight.data_ptr(), pdb, pw, wb, _stream_of(stream, d))
    if rc:
        _raise(rc)
