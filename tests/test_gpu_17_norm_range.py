"""GPU tests of the RMS norm and its gradient away from unit scale and ordinary
row counts, against the fp64 oracle.  Bars as in test_gpu_12_rms_norm.py, whose
helpers these are."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import mx
from test_gpu_12_rms_norm import NORM, OUT_STEP, U, draw, empty, f64, torch_type

pytestmark = pytest.mark.gpu


def check_backward(h, h64, rstd, typ, seed):
    """The gradient of these rows; h64's rows times rstd are within fp32, as is all that the formula forms."""
    import torch
    rows, cols = h64.shape
    dy, dy64 = draw(rows, cols, typ, seed + 1)
    dh, dh64 = draw(rows, cols, typ, seed + 2)
    w, w64 = draw(1, cols, typ, seed + 3)
    s = f64(rstd)
    for d, d64 in ((None, None), (dh, dh64)):
        dx, dw = empty(rows, cols, torch_type(typ)), torch.full((cols,), 7.0, device="cuda")
        ws = torch.empty(dg.dist_gemm_rms_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
        dg.dist_gemm_rms_norm_backward(dy, h, rstd, w[0], dx, dw, ws, dh=d)
        ref, refw = mx.rms_norm_backward(dy64, h64, w64[0], s, d64)
        n, g = h64 * s[:, None], dy64 * w64
        size = s[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(-1, keepdims=True))
        if d is not None:
            size = size + np.abs(d64)
        assert np.all(np.abs(f64(dx) - ref) <= OUT_STEP[typ] * np.abs(ref) + 2 * NORM * size)
        assert np.all(np.abs(f64(dw) - refw) <= (rows / 2 + 24) * U * np.abs(dy64 * n).sum(0) + 1e-30)


# every number of pieces per lane; 1e15: rstd cubed is below fp32, 1e-14 (eps = 0): above it
@pytest.mark.parametrize("size", [1e15, 1e-14])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("rows,cols", [(9, 96), (5, 5123), (3, 16384), (4, 20000)])
def test_gradient_of_large_and_small_rows(rows, cols, typ, size):
    import torch
    log("norm gradient", rows, cols, typ, size)
    h, h64 = draw(rows, cols, typ, cols, scale=size)
    w = torch.ones(cols, dtype=torch_type(typ), device="cuda")
    y, rstd = torch.empty_like(h), torch.empty(rows, device="cuda")
    dg.dist_gemm_rms_norm(h, w, y, eps=0.0, rstd=rstd)
    ref = mx.rms_norm(h64, np.ones(cols), 0.0)
    assert np.all(np.abs(f64(rstd) - ref[1]) <= NORM * ref[1])
    assert np.all(np.abs(f64(y) - ref[0]) <= (OUT_STEP[typ] + 2 * NORM) * np.abs(ref[0]))
    check_backward(h, h64, rstd, typ, cols)


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("cols", [96, 5123, 16384, 20000])
def test_gradient_of_rows_of_zeros(cols, typ):
    """Such a row has rstd = 1 / sqrt(eps) and dx = rstd dy w, finite for any eps that keeps rstd finite."""
    import torch
    log("norm gradient of zeros", cols, typ)
    h, h64 = draw(4, cols, typ, 3)
    h[1], h64[1] = 0, 0
    h[3], h64[3] = 0, 0
    y, rstd = torch.empty_like(h), torch.empty(4, device="cuda")
    dg.dist_gemm_rms_norm(h, torch.ones(cols, dtype=torch_type(typ), device="cuda"), y, eps=1e-28, rstd=rstd)
    assert abs(rstd[1].item() - 1e14) <= NORM * 1e14 and not y[1].any()
    check_backward(h, h64, rstd, typ, 3)


# more rows than a launch has threads along x for, four to a workgroup (norms per head of a long batch), up to as many as are
# accepted
@pytest.mark.parametrize("rows,cols,typ,out", [((1 << 26) + 13, 128, "BF16", "SAME"), ((1 << 26) + 3, 64, "BF16", "MX_E4M3"),
                                               ((1 << 26) + 5, 512, "BF16", "E4M3"), ((1 << 31) - 1, 1, "F32", "SAME")])
def test_many_rows_equal_their_parts(rows, cols, typ, out):
    import torch
    log("many rows", rows, cols, typ, out)
    t = torch_type(typ)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.empty((rows, cols), dtype=t, device="cuda").normal_(generator=g)
    w = torch.randn(cols, generator=g, device="cuda").to(t)

    def run(x):
        n = x.size(0)
        y = torch.full((n, cols), 77, dtype=t if out == "SAME" else torch.uint8, device="cuda")
        s = torch.full((n, mx.scale_pitch(cols)), 77, dtype=torch.uint8, device="cuda") if out.startswith("MX") else None
        rstd = torch.full((n,), -1.0, device="cuda")
        dg.dist_gemm_rms_norm(x, w, y, output=out, rstd=rstd, scales=s, scale=0.1)
        return [v for v in (y, rstd, s) if v is not None]

    whole = run(x)
    assert bool((whole[1] > 0).all())                 # every row was reached
    for lo in sorted({0, rows // 2, 1 << 21, 1 << 23, 1 << 24, 1 << 26, rows - 3000}):
        lo = max(0, min(lo - 1500, rows - 3000))
        assert all(torch.equal(p, v[lo:lo + 3000]) for p, v in zip(run(x[lo:lo + 3000]), whole))
    x64 = f64(x[rows - 20:])
    ref = mx.rms_norm(x64, f64(w), 1e-6)
    assert np.all(np.abs(f64(whole[1][rows - 20:]) - ref[1]) <= NORM * ref[1])
    if out == "SAME":
        assert np.all(np.abs(f64(whole[0][rows - 20:]) - ref[0]) <= (OUT_STEP[typ] + 2 * NORM) * np.abs(ref[0]))
    del x, whole
    torch.cuda.empty_cache()      # 70 to 110 GB
