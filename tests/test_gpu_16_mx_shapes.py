"""GPU tests of the MX products at sizes whose workgroups do not come out even,
with offsets that are not in order and at the ends of the scales' range.

Bars as in test_gpu_13_mx_products.py, whose helpers these are."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import codecs, mx
from test_gpu_13_mx_products import check_on_gpu, dense, f64, random_codes, up

pytestmark = pytest.mark.gpu


# row tiles of 32 that do not divide the CUs, at widths where a column tile's even share is more than the 32
# columns of a workgroup (on 256 CUs 33 to 41): every column has to be written
@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("M,N,K", [(96, 2730, 512), (200, 1168, 256), (400, 624, 96), (640, 400, 1024), (900, 280, 256),
                                   (3200, 81, 96), (160, 1638, 544), (96, 5456, 4640), (1365, 547, 4128)])
def test_row_tiles_that_do_not_divide_the_cus(M, N, K, a_format):
    log("uneven row tiles", M, N, K, a_format)
    dense(M, N, K, a_format, "BF16")
    dense(M, N, K, a_format, "F32", alpha=0.5, beta=2.0, with_bias=True, pitch=N + 5)


# few rows to a group, 128 x 128 tiles, their K split over two groups of waves, 256 x 256 tiles, more than 64 groups
@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("rows,N,K,offsets", [
    (20, 100, 544, [0, 10, 5, 20]),
    (40, 272, 96, [3, 40, 0, 40, 0, 40, -7, 1000]),
    (100, 70, 512, [50, 20, 70, 60, 100]),
    (900, 720, 544, [0, 900, 0, 900, 0, 900]),
    (900, 1500, 544, [10, 700, 300, 850, 400]),
    (900, 1500, 4640, [0, 900, 100, 900, 200, 900]),
    (6000, 3000, 288, [5, 4000, 20, 5990, 4000]),
    (300, 100, 96, [0] * 40 + [200, 100] + [50] * 70 + [290, 250]),
    (9000, 200, 96, [0] * 30 + [6000, 100, 5000] + [8000] * 60 + [9000, 20, 9000])])
def test_offsets_that_fall(rows, N, K, offsets, a_format):
    """An offset outside 0 .. rows is clamped to it, one below an earlier one counts as that one."""
    import torch
    log("falling offsets", rows, N, K, len(offsets), a_format)
    E = len(offsets) - 1
    A, As, a = random_codes(rows, K, a_format, 1)
    B, Bs, b = random_codes(E * N, K, "E2M1", 2)
    D = torch.full((rows, N), -5.0, dtype=torch.bfloat16, device="cuda")
    with dg.MxPlan(rows, N, K, groups=E, a_format=a_format) as p:
        p.run(A, As, B, Bs, D, offsets=up(np.array(offsets, dtype=np.int32)))
        torch.cuda.synchronize()
    at = np.maximum.accumulate(np.clip(offsets, 0, rows))
    for e in range(E):
        if at[e + 1] > at[e]:
            check_on_gpu(D[at[e]:at[e + 1]], a[at[e]:at[e + 1]], b[e * N:(e + 1) * N], "BF16")
    assert bool((D[:at[0]] == -5.0).all()) and bool((D[at[-1]:] == -5.0).all())


@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("M,N", [(16, 255), (64, 255), (1100, 1100), (2304, 1100)])
def test_scales_over_their_whole_range(M, N, a_format):
    """One product per element, 2^(a - 127) 2^(b - 127) for all scale bytes a and b but NaN: exact down to the smallest
    subnormal, zero below, infinite above."""
    import torch
    log("all scales", M, N, a_format)
    K = 512
    a, b = np.zeros((M, K)), np.zeros((N, K))
    a[:, 5], b[:, 5] = 1.0, 1.0
    A = mx.pack(mx.f64_to_e2m1(a)) if a_format == "E2M1" else codecs.f64_to_e4m3(a)
    As, Bs = np.zeros((M, mx.scale_pitch(K)), dtype=np.uint8), np.zeros((N, mx.scale_pitch(K)), dtype=np.uint8)
    As[:, 0], Bs[:, 0] = np.arange(M) * 7 % 255, np.arange(N) % 255
    D = torch.empty((M, N), device="cuda")
    with dg.MxPlan(M, N, K, a_format=a_format, out_dtype="F32") as p:
        p.run(up(A), up(As), up(mx.pack(mx.f64_to_e2m1(b))), up(Bs), D)
    e = As[:, :1].astype(int) + Bs[:, 0].astype(int)[None] - 254
    want = np.where(e > 127, np.inf, np.where(e < -149, 0.0, np.ldexp(1.0, np.clip(e, -149, 127))))
    # halfway between zero and the smallest subnormal goes to zero (even)
    assert np.array_equal(f64(D), want)
