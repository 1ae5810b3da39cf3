"""GPU tests of what the header says of the ends of fp32's range: the largest
fp32 values through an F8 tensor and its transpose, and rows whose squares
vanish or overflow without an eps."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from oracle import f8

pytestmark = pytest.mark.gpu


def room(rows, cols):
    import torch
    return (torch.full((rows, f8.pitch(cols)), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((rows, f8.scale_pitch(cols)), 0xA5, dtype=torch.uint8, device="cuda"))


def test_the_largest_values_transposed():
    """fp32's largest value rounds to 256 * 2^120 = 2^128, which fp32 does not have: quantised it is
    kept, back in fp32 it is an infinity, and read transposed its block is NaN.  248 * 2^120 is halfway from 240 to 256 and goes to
    the even one, 256; below it everything stays."""
    import torch
    rows, cols = 130, 140
    v = np.random.default_rng(1).standard_normal((rows, cols)).astype(np.float32)
    v[3, 7], v[5, 9] = np.finfo(np.float32).max, 248 * 2.0 ** 120
    v[7, 11], v[128, 13] = np.nextafter(np.float32(248 * 2.0 ** 120), np.float32(0)), -240 * 2.0 ** 120
    x = torch.from_numpy(v).cuda()
    a, b, c = room(rows, cols), room(cols, rows), room(cols, rows)
    dg.dist_gemm_f8_quantize(x, *a, *b)
    for (codes, scales), of in ((a, v), (b, v.T)):
        want = f8.quantize(of.astype(np.float64))
        assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
    back = torch.empty_like(x)
    dg.dist_gemm_f8_dequantize(*a, back)
    back = back.cpu().numpy()
    values = f8.values(a[0].cpu().numpy(), a[1].cpu().numpy(), cols)
    assert values[3, 7] == 2.0 ** 128 == values[5, 9] and values[7, 11] == 240 * 2.0 ** 120
    past = np.abs(values) >= 2.0 ** 128
    assert np.array_equal(np.isinf(back), past) and np.array_equal(back[~past], values[~past].astype(np.float32))
    dg.dist_gemm_f8_transpose(*a, *c)
    want = f8.quantize(np.where(past, np.inf, values).T)
    assert np.array_equal(c[0].cpu().numpy(), want[0]) and np.array_equal(c[1].cpu().numpy(), want[1])
    s = c[1].cpu().numpy()
    assert s[7, 0] == s[9, 0] == 255 and s[11, 0] == 247 == s[13, 1] and (s == 255).sum() == 2


@pytest.mark.parametrize("cols", [64, 200, 1000, 5123, 20000])
def test_rows_past_the_range_without_eps(cols):
    import torch
    x = torch.ones((5, cols), device="cuda")
    x[:, 1::2] = -1
    x *= torch.tensor([1.0, 1e-25, 1e20, 0.0, 1e-10], device="cuda")[:, None]
    w, b = torch.full((cols,), 0.5, device="cuda"), torch.full((cols,), 0.25, device="cuda")
    mean, rstd, y = torch.empty(5, device="cuda"), torch.empty(5, device="cuda"), torch.empty_like(x)
    dg.dist_gemm_layer_norm(x, w, b, y, eps=0.0, mean=mean, rstd=rstd)
    got, m, s = y.double().cpu().numpy(), mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    h = x.double().cpu().numpy()
    want, _, wm, ws = f8.layer_norm(h, w.double().cpu().numpy(), b.double().cpu().numpy(), 0.0)
    tol = 64 * 2.0 ** -24                                    # as in the norm's tests; mean|h| rstd is 1
    for i in (0, 4):
        assert abs(m[i] - wm[i]) <= tol * abs(h[i, 0]) and abs(s[i] - ws[i]) <= 3 * tol * ws[i]
        assert (np.abs(got[i] - want[i]) <= 0.5 * (4 * tol * np.abs(h[i, 0]) * ws[i] + tol)).all()
    assert np.isinf(s[1]) and np.isinf(got[1]).all()         # its squares vanish
    assert s[2] == 0 and (got[2] == 0.25).all()              # they overflow: the bias alone
    assert np.isinf(s[3]) and np.isnan(got[3]).all()         # equal values


def test_fewer_rows_may_need_a_workspace():
    """K in parts is for few tiles: where M varies the workspace is the largest over M."""
    need = [dg.dist_gemm_f8_product_workspace(M, 512, 16384) for M in (1, 128, 100000)]
    assert need[0] == 0 and need[1] > 0 and need[2] == 0
