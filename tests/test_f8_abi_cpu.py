"""CPU checks of the 8-bit training operators' C ABI: every function that
include/distgemm_f8.h declares is exported, and wrong arguments are refused on
the host, before any GPU work."""
import ctypes
import os
import re

import pytest

import communication_tensor_gemm_amd as dg
from oracle import f8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # an aligned address that is never read: the calls below are refused first
INVALID, SHAPE = -1, -2
BIG = 1 << 31


def test_header_declarations_are_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "distgemm_f8.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(dist_gemm_\w+)\s*\(", text)))
    lib = ctypes.CDLL(dg.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name), name
    assert sorted(dg.F8_C_FUNCTIONS) == declared


def test_enum_matches_the_header():
    text = open(os.path.join(ROOT, "include", "distgemm_f8.h")).read()
    for name, v in dg.LAYER_NORM_OUTPUTS.items():
        assert re.search(rf"DIST_GEMM_LAYER_NORM_{name} = {v}\b", text), name


@pytest.mark.parametrize("cols", [1, 127, 128, 129, 2048, 2049, 5123, 16384, (1 << 31) - 128])
def test_pitches(cols):
    assert dg.dist_gemm_f8_pitch(cols) == f8.pitch(cols)
    assert dg.dist_gemm_f8_scale_pitch(cols) == f8.scale_pitch(cols)


@pytest.mark.parametrize("cols", [0, -1, (1 << 31) - 127, 1 << 40])
def test_pitches_of_no_width(cols):
    assert dg.dist_gemm_f8_pitch(cols) == 0 and dg.dist_gemm_f8_scale_pitch(cols) == 0


def call(fn, good, change):
    """The status of `fn` with the arguments of `good` changed; a refusal leaves a message."""
    rc = getattr(dg.lib, fn)(*{**good, **change}.values(), None)
    if rc:
        assert dg.lib.dist_gemm_f8_last_error().decode().split(":")[0]
    return rc


QUANTIZE = dict(x=P, ldx=64, elem=1, rows=4, cols=64, block_rows=1, codes=2 * P, scales=3 * P, codes_t=4 * P, scales_t=5 * P)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(codes_t=None), INVALID),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), INVALID), (dict(elem=2), INVALID),
    (dict(block_rows=2), INVALID), (dict(rows=-1), INVALID), (dict(cols=0, ldx=0), INVALID), (dict(codes=2 * P + 8), INVALID),
    (dict(scales_t=P + 1), INVALID), (dict(x=P + 1), INVALID), (dict(ldx=63), SHAPE), (dict(rows=BIG), SHAPE),
    (dict(cols=BIG - 127, ldx=BIG), SHAPE), (dict(rows=BIG - 128, cols=BIG - 128, ldx=BIG), SHAPE),
])
def test_quantize_refuses(change, status):
    assert call("dist_gemm_f8_quantize", QUANTIZE, change) == status


@pytest.mark.parametrize("one,other", [(a, b) for i, a in enumerate(("x", "codes", "scales", "codes_t", "scales_t"))
                                       for b in ("x", "codes", "scales", "codes_t", "scales_t")[i + 1:]])
def test_quantize_refuses_shared_memory(one, other):
    assert call("dist_gemm_f8_quantize", QUANTIZE, {other: QUANTIZE[one]}) == INVALID
    assert b"alias" in dg.lib.dist_gemm_f8_last_error()


DEQUANTIZE = dict(codes=P, scales=2 * P, rows=4, cols=64, y=3 * P, ldy=64, elem=0)
TRANSPOSE = dict(codes=P, scales=2 * P, rows=4, cols=64, codes_t=3 * P, scales_t=4 * P)


@pytest.mark.parametrize("change,status", [
    (dict(codes=None), INVALID), (dict(y=None), INVALID), (dict(elem=-1), INVALID), (dict(ldy=63), SHAPE),
    (dict(codes=P + 4), INVALID), (dict(y=3 * P + 2), INVALID), (dict(y=P), INVALID), (dict(y=2 * P), INVALID),
    (dict(rows=BIG), SHAPE), (dict(rows=-1), INVALID)])
def test_dequantize_refuses(change, status):
    assert call("dist_gemm_f8_dequantize", DEQUANTIZE, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(codes=None), INVALID), (dict(scales_t=None), INVALID), (dict(codes_t=3 * P + 1), INVALID), (dict(codes_t=P), INVALID),
    (dict(scales_t=2 * P), INVALID), (dict(scales_t=3 * P), INVALID), (dict(rows=BIG), SHAPE), (dict(cols=0), INVALID)])
def test_transpose_refuses(change, status):
    assert call("dist_gemm_f8_transpose", TRANSPOSE, change) == status


PRODUCT = dict(A=P, As=2 * P, B=3 * P, Bs=4 * P, M=4, N=64, K=256, C=5 * P, ldc=64, D=6 * P, ldd=64, out=0, bias=7 * P,
               alpha=1.0, beta=1.0, workspace=8 * P, bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(A=None), INVALID), (dict(Bs=None), INVALID), (dict(D=None), INVALID), (dict(C=None), INVALID), (dict(out=2), INVALID),
    (dict(M=-1), INVALID), (dict(M=BIG), SHAPE), (dict(N=0), SHAPE), (dict(N=BIG, ldd=BIG, ldc=BIG), SHAPE), (dict(K=0), SHAPE),
    (dict(K=192), SHAPE), (dict(K=(1 << 22) + 128), SHAPE), (dict(ldd=63), SHAPE), (dict(ldc=63), SHAPE),
    (dict(alpha=float("nan")), INVALID), (dict(beta=float("inf")), INVALID), (dict(A=P + 8), INVALID), (dict(D=6 * P + 2), INVALID),
    (dict(bias=7 * P + 1), INVALID), (dict(D=5 * P, ldd=65), INVALID)] + [(dict(D=PRODUCT[k]), INVALID) for k in ("A", "As", "B", "Bs", "bias")])
def test_product_refuses(change, status):
    assert call("dist_gemm_f8_product", PRODUCT, change) == status


NORM = dict(x=P, ldx=64, residual=None, ldr=0, weight=2 * P, bias=3 * P, elem=1, rows=4, cols=64, eps=1e-6, out=0, scale=1.0,
            y=4 * P, ldy=64, scales=None, h=None, ldh=0, mean=None, rstd=None, kept=None, kept_scales=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID), (dict(elem=-1), INVALID),
    (dict(out=3), INVALID), (dict(out=-1), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(residual=5 * P, ldr=64), INVALID), (dict(h=5 * P, ldh=64), INVALID),
    (dict(out=1, scale=0.0), INVALID), (dict(out=1, scale=float("inf")), INVALID), (dict(out=1, scale=1e-45), INVALID),
    (dict(out=2), INVALID), (dict(out=2, scales=5 * P + 1), INVALID), (dict(out=2, scales=5 * P, y=4 * P + 8), INVALID),
    (dict(kept=5 * P), INVALID), (dict(kept_scales=5 * P), INVALID), (dict(kept=5 * P + 8, kept_scales=6 * P), INVALID),
    (dict(x=P + 1), INVALID), (dict(bias=P + 1), INVALID), (dict(mean=P + 2), INVALID), (dict(y=2 * P), INVALID),
    (dict(y=3 * P), INVALID), (dict(out=1, y=P), INVALID), (dict(cols=32769, ldx=32769, ldy=32769), SHAPE),
    (dict(rows=BIG), SHAPE), (dict(ldx=63), SHAPE), (dict(ldy=63), SHAPE), (dict(y=P, ldy=65), INVALID),
    (dict(residual=5 * P, ldr=63, h=6 * P, ldh=64), SHAPE), (dict(residual=5 * P, ldr=64, h=P, ldh=65), INVALID),
    (dict(residual=5 * P, ldr=64, h=4 * P, ldh=64), INVALID), (dict(residual=5 * P, ldr=64, h=3 * P, ldh=64), INVALID),
])
def test_layer_norm_refuses(change, status):
    assert call("dist_gemm_layer_norm", NORM, change) == status


ALL = {**NORM, "out": 2, "residual": 5 * P, "ldr": 64, "h": 6 * P, "ldh": 64, "scales": 7 * P, "mean": 8 * P, "rstd": 9 * P,
       "kept": 10 * P, "kept_scales": 11 * P}


@pytest.mark.parametrize("what", ["mean", "rstd", "scales", "kept", "kept_scales"])
@pytest.mark.parametrize("where", ["x", "residual", "weight", "bias", "y", "h", "mean", "rstd", "scales", "kept", "kept_scales"])
def test_layer_norm_refuses_shared_memory(what, where):
    if what == where:
        return
    assert call("dist_gemm_layer_norm", ALL, {what: ALL[where]}) == INVALID
    assert b"alias" in dg.lib.dist_gemm_f8_last_error()


BACKWARD = dict(dy=P, lddy=64, h=2 * P, ldh=64, h_scales=None, dh=None, lddh=0, mean=3 * P, rstd=4 * P, weight=5 * P, elem=0,
                rows=4, cols=64, dx=6 * P, lddx=64, dweight=7 * P, dbias=8 * P, workspace=9 * P, bytes=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(weight=None), INVALID), (dict(dx=None), INVALID), (dict(dweight=None), INVALID), (dict(workspace=None), INVALID),
    (dict(workspace=9 * P + 8), INVALID), (dict(bytes=64 * 8 - 1), INVALID), (dict(elem=2), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=40000, lddy=40000, ldh=40000, lddx=40000), SHAPE), (dict(lddy=63), SHAPE), (dict(ldh=63), SHAPE),
    (dict(lddx=63), SHAPE), (dict(dh=10 * P, lddh=63), SHAPE), (dict(dx=P, lddx=65), INVALID), (dict(dx=2 * P, lddx=65), INVALID),
    (dict(dx=5 * P), INVALID), (dict(dx=3 * P), INVALID), (dict(dx=4 * P), INVALID), (dict(dweight=8 * P), INVALID),
    (dict(dbias=P), INVALID), (dict(dweight=5 * P), INVALID), (dict(dbias=8 * P + 2), INVALID),
    (dict(h_scales=10 * P + 4), INVALID), (dict(h_scales=10 * P, h=2 * P + 8), INVALID), (dict(h_scales=10 * P, dx=2 * P), INVALID),
    (dict(h_scales=10 * P, dx=10 * P), INVALID),
])
def test_layer_norm_backward_refuses(change, status):
    assert call("dist_gemm_layer_norm_backward", BACKWARD, change) == status


@pytest.mark.parametrize("where", ["dy", "h", "h_scales", "dh", "rstd", "weight", "dx", "dweight", "dbias"])
def test_layer_norm_backward_refuses_a_workspace_on_an_operand(where):
    a = {**BACKWARD, "dh": 11 * P, "lddh": 64, "h_scales": 10 * P}
    assert call("dist_gemm_layer_norm_backward", a, dict(workspace=a[where])) == INVALID
    assert b"alias" in dg.lib.dist_gemm_f8_last_error()


def test_nothing_to_do_is_no_error():
    assert call("dist_gemm_f8_quantize", QUANTIZE, dict(rows=0, x=None)) == 0
    assert call("dist_gemm_f8_dequantize", DEQUANTIZE, dict(rows=0, y=None)) == 0
    assert call("dist_gemm_f8_transpose", TRANSPOSE, dict(rows=0, codes=None)) == 0
    assert call("dist_gemm_f8_product", PRODUCT, dict(M=0, A=None, D=None)) == 0
    assert call("dist_gemm_layer_norm", NORM, dict(rows=0, x=None, y=None)) == 0


@pytest.mark.parametrize("rows,cols", [(0, 64), (1, 1), (4, 64), (5000, 512), (5000, 520), (5000, 8192), (5000, 16384),
                                       (5000, 16385), (3, 32768), (5000, 32768)])
def test_workspace_holds_every_partial_sum(rows, cols):
    n = dg.dist_gemm_layer_norm_workspace(rows, cols)
    assert n >= 8 * cols and n % (8 * cols) == 0 and n <= 8 * cols * max(1, min(rows, 2048))


def test_workspace_of_refused_sizes():
    for rows, cols in ((-1, 64), (4, 0), (4, 32769), (BIG, 64)):
        assert dg.dist_gemm_layer_norm_workspace(rows, cols) == 0
