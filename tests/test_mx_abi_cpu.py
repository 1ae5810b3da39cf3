"""CPU checks of the low-precision operators' C ABI: every function that
include/distgemm_mx.h declares is exported, and wrong arguments are refused
on the host, before any GPU work."""
import ctypes
import os
import re

import pytest

import communication_tensor_gemm_amd as dg
from oracle import mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # an aligned address that is never read: the calls below are refused first
INVALID, SHAPE = -1, -2
BIG = 1 << 31


def test_header_declarations_are_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "distgemm_mx.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(dist_gemm_\w+)\s*\(", text)))
    lib = ctypes.CDLL(dg.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name), name
    assert sorted(dg.MX_C_FUNCTIONS) == declared


def test_enums_match_the_header():
    text = open(os.path.join(ROOT, "include", "distgemm_mx.h")).read()
    for prefix, table in (("ELEM_", dg.ELEMS), ("MX_", dg.MX_FORMATS), ("NORM_", dg.NORM_OUTPUTS)):
        for name, v in table.items():
            assert re.search(rf"DIST_GEMM_{prefix}{name} = {v}\b", text), name


@pytest.mark.parametrize("cols", [32, 480, 512, 544, 3584, 16384, 1 << 22])
def test_scale_pitch(cols):
    assert dg.dist_gemm_mx_scale_pitch(cols) == mx.scale_pitch(cols)


@pytest.mark.parametrize("cols", [0, -32, 31, 33])
def test_scale_pitch_of_no_mx_width(cols):
    assert dg.dist_gemm_mx_scale_pitch(cols) == 0


QUANTIZE = dict(x=P, ldx=64, elem=1, rows=4, cols=64, format=0, codes=P, scales=P)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(elem=2), INVALID), (dict(format=2), INVALID), (dict(rows=-1), INVALID), (dict(cols=0, ldx=0), INVALID),
    (dict(codes=P + 8), INVALID), (dict(scales=P + 1), INVALID), (dict(x=P + 1), INVALID),
    (dict(cols=48), SHAPE), (dict(ldx=63), SHAPE), (dict(rows=BIG), SHAPE), (dict(cols=BIG, ldx=BIG), SHAPE),
])
def test_quantize_refuses(change, status):
    a = {**QUANTIZE, **change}
    assert dg.lib.dist_gemm_mx_quantize(a["x"], a["ldx"], a["elem"], a["rows"], a["cols"], a["format"], a["codes"],
                                        a["scales"], None) == status
    assert dg.lib.dist_gemm_mx_dequantize(a["codes"], a["scales"], a["format"], a["rows"], a["cols"], a["x"],
                                          a["ldx"], a["elem"], None) == status
    assert dg.lib.dist_gemm_mx_last_error(None)


def test_nothing_to_do_is_no_error():
    assert dg.lib.dist_gemm_mx_quantize(None, 64, 1, 0, 64, 0, None, None, None) == 0
    assert dg.lib.dist_gemm_mx_dequantize(None, None, 0, 0, 64, None, 64, 1, None) == 0
    assert dg.lib.dist_gemm_rms_norm(None, 64, None, 0, None, 1, 0, 64, 1e-6, 0, 1.0, None, 64, None, None, 0, None,
                                     None) == 0


NORM = dict(x=P, ldx=64, residual=None, ldr=0, weight=2 * P, elem=1, rows=4, cols=64, eps=1e-6, out=0, scale=1.0,
            y=3 * P, ldy=64, scales=None, h=None, ldh=0, rstd=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID), (dict(elem=-1), INVALID),
    (dict(out=4), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(residual=4 * P, ldr=64), INVALID), (dict(h=4 * P, ldh=64), INVALID),
    (dict(out=1, scale=0.0), INVALID), (dict(out=1, scale=float("inf")), INVALID), (dict(out=1, scale=1e-45), INVALID),
    (dict(out=3), INVALID), (dict(out=3, scales=4 * P + 1), INVALID), (dict(out=2, scales=4 * P, y=3 * P + 8), INVALID),
    (dict(x=P + 1), INVALID), (dict(rstd=P + 2), INVALID), (dict(y=2 * P), INVALID), (dict(out=1, y=P), INVALID),
    (dict(y=P, ldy=65), INVALID), (dict(residual=4 * P, ldr=64, h=P, ldh=65), INVALID),
    (dict(ldx=63), SHAPE), (dict(ldy=63), SHAPE), (dict(cols=32769, ldx=32769, ldy=32769), SHAPE),
    (dict(out=3, scales=4 * P, cols=48), SHAPE), (dict(rows=BIG), SHAPE),
    (dict(residual=4 * P, ldr=63, h=5 * P, ldh=64), SHAPE),
])
def test_rms_norm_refuses(change, status):
    a = {**NORM, **change}
    assert dg.lib.dist_gemm_rms_norm(*(a[k] for k in NORM), None) == status


BACKWARD = dict(dy=P, lddy=64, h=2 * P, ldh=64, dh=None, lddh=0, rstd=3 * P, weight=4 * P, elem=0, rows=4, cols=64,
                dx=5 * P, lddx=64, dweight=6 * P, workspace=7 * P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(rstd=None), INVALID), (dict(weight=None), INVALID),
    (dict(dx=None), INVALID), (dict(dweight=None), INVALID), (dict(workspace=None), INVALID), (dict(elem=5), INVALID),
    (dict(workspace=7 * P + 4), INVALID), (dict(workspace_bytes=64), INVALID), (dict(rows=-1), INVALID),
    (dict(dx=4 * P), INVALID), (dict(dx=P, lddx=65), INVALID), (dict(dweight=P), INVALID), (dict(dh=8 * P + 2, lddh=64), INVALID),
    (dict(lddy=63), SHAPE), (dict(ldh=63), SHAPE), (dict(lddx=63), SHAPE), (dict(dh=8 * P, lddh=63), SHAPE),
    (dict(cols=32769, lddy=32769, ldh=32769, lddx=32769), SHAPE),
])
def test_rms_norm_backward_refuses(change, status):
    a = {**BACKWARD, **change}
    assert dg.lib.dist_gemm_rms_norm_backward(*(a[k] for k in BACKWARD), None) == status


def test_workspace_of_refused_sizes_is_zero():
    assert dg.dist_gemm_rms_norm_workspace(8, 32769) == 0 and dg.dist_gemm_rms_norm_workspace(-1, 8) == 0
    assert dg.dist_gemm_rms_norm_workspace(0, 8) > 0


@pytest.mark.parametrize("args,status", [
    ((0, 64, 64, 0, 0, 1), INVALID), ((8, 0, 64, 0, 0, 1), INVALID), ((8, 64, 0, 0, 0, 1), INVALID),
    ((8, 64, 64, -1, 0, 1), INVALID), ((8, 64, 64, 0, 2, 1), INVALID), ((8, 64, 64, 0, 0, 7), INVALID),
    ((8, 64, 48, 0, 0, 1), SHAPE), ((BIG, 64, 64, 0, 0, 1), SHAPE), ((8, BIG, 64, 0, 0, 1), SHAPE),
    ((8, 64, (1 << 22) + 32, 0, 0, 1), SHAPE), ((8, 64, 64, 65536, 0, 1), SHAPE),
])
def test_plan_refuses(args, status):
    h = ctypes.c_void_p(1)
    assert dg.lib.dist_gemm_mx_plan(*args, ctypes.byref(h)) == status
    assert not h.value
    assert dg.lib.dist_gemm_mx_last_error(None)


def test_null_plans():
    assert dg.lib.dist_gemm_mx_plan(8, 64, 64, 0, 0, 1, None) == INVALID
    assert dg.lib.dist_gemm_mx_run(None, 8, P, P, P, P, None, 0, P, 64, None, None, 1.0, 0.0, None) == INVALID
    assert dg.lib.dist_gemm_mx_destroy(None) == 0


def test_cpu_tensors_are_refused():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        dg.dist_gemm_mx_quantize(x, "E2M1", torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU"):
        dg.dist_gemm_rms_norm(x, torch.ones(64), x)
