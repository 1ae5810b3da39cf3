"""CPU checks that the low-precision operators refuse outputs which start at the
address of another argument (test_mx_abi_cpu.py has the arguments and the
other refusals)."""
import pytest

import communication_tensor_gemm_amd as dg
from test_mx_abi_cpu import BACKWARD, INVALID, NORM, QUANTIZE, P


# one address for two arguments, at least one of them written
@pytest.mark.parametrize("change", [dict(codes=P, x=P), dict(scales=P, x=P), dict(codes=3 * P, scales=3 * P)])
def test_quantize_refuses_shared_memory(change):
    a = {**QUANTIZE, "x": P, "codes": 2 * P, "scales": 3 * P, **change}
    assert dg.lib.dist_gemm_mx_quantize(a["x"], a["ldx"], a["elem"], a["rows"], a["cols"], a["format"], a["codes"],
                                        a["scales"], None) == INVALID
    assert b"alias" in dg.lib.dist_gemm_mx_last_error(None)
    if a["codes"] != a["scales"]:      # (both are inputs there)
        assert dg.lib.dist_gemm_mx_dequantize(a["codes"], a["scales"], a["format"], a["rows"], a["cols"], a["x"],
                                              a["ldx"], a["elem"], None) == INVALID
        assert b"alias" in dg.lib.dist_gemm_mx_last_error(None)


@pytest.mark.parametrize("what,where", [(w, o) for w in ("rstd", "scales")
                                        for o in ("x", "residual", "weight", "y", "h")] + [("rstd", "scales")])
def test_rms_norm_refuses_shared_memory(what, where):
    a = {**NORM, "out": 3, "residual": 4 * P, "ldr": 64, "h": 5 * P, "ldh": 64, "scales": 6 * P, "rstd": 7 * P}
    a[what] = a[where]
    assert dg.lib.dist_gemm_rms_norm(*(a[k] for k in NORM), None) == INVALID
    assert b"alias" in dg.lib.dist_gemm_mx_last_error(None)


@pytest.mark.parametrize("where", ["dy", "h", "dh", "rstd", "weight", "dx", "dweight"])
def test_rms_norm_backward_refuses_a_workspace_on_an_operand(where):
    a = {**BACKWARD, "dh": 8 * P, "lddh": 64}
    a["workspace"] = a[where]
    assert dg.lib.dist_gemm_rms_norm_backward(*(a[k] for k in BACKWARD), None) == INVALID
    assert b"alias" in dg.lib.dist_gemm_mx_last_error(None)
