"""GPU tests of the MX products between a few rows and large ones: tiles where a
launch has some dozens of them, their K split between two groups of waves, and
many rows by the kernel of few where the tiles would leave most CUs idle.

Bars as in test_gpu_13_mx_products.py, whose helpers these are."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from test_gpu_13_mx_products import check, dense, f64, grouped, make, torch_out, up

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])


# 72 to 90 tiles of 128 x 128: one block of K, less than a slab, one slab, ragged, several chunks of scales
@BOTH
@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,K", [(1100, 1000, 32), (1100, 1000, 96), (1090, 1003, 256), (1025, 1100, 800), (1100, 1101, 1184)])
def test_some_tiles(M, N, K, a_format, out):
    dense(M, N, K, a_format, out)


# K above 4096, not a multiple of a chunk or slab, the second half shorter by none to several slabs
@BOTH
@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("K", [4128, 4608, 4736, 5632, 6144, 8224])
def test_split_k(K, a_format, out):
    dense(1100, 1090, K, a_format, out)


@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("K", [544, 4640])
def test_epilogue_forms(K, out):
    dense(1100, 1024, K, "E4M3", out, alpha=0.375, beta=-1.5, with_bias=True)
    dense(1090, 1024, K, "E2M1", out, alpha=2.0, with_bias=True)          # whole columns, a last row tile of 66
    dense(1100, 1024, K, "E2M1", out, beta=1.0, in_place=True)
    dense(1100, 1024, K, "E2M1", out, pitch=1037)
    dense(1100, 1024, K, "E4M3", out, pitch=1032, rows=1057)


@BOTH
@pytest.mark.parametrize("M,N,K", [(1100, 1000, 1120), (1100, 1100, 4128), (300, 113, 4640), (126, 113, 15168)])
def test_scale_bytes_past_k_and_nan_blocks(M, N, K, a_format):
    """Bytes past K / 32 hold the NaN scale and do not count; a NaN block reaches its row, or its column, alone."""
    import torch
    log("past k", M, N, K, a_format)
    A, As, a = make(M, K, a_format, 5)
    B, Bs, b = make(N, K, "E2M1", 6)
    As[:, K // 32:], Bs[:, K // 32:] = 255, 255
    As[M - 1, K // 32 - 1], Bs[N - 1, 0] = 255, 255
    D = torch.full((M, N), -5.0, dtype=torch.bfloat16, device="cuda")
    with dg.MxPlan(M, N, K, a_format=a_format) as p:
        p.run(up(A), up(As), up(B), up(Bs), D)
        torch.cuda.synchronize()
    got = f64(D)
    assert np.isnan(got[M - 1]).all() and np.isnan(got[:, N - 1]).all()
    check(got[:M - 1, :N - 1], a[:M - 1], b[:N - 1], "BF16")


@BOTH
@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,K", [(126, 113, 15168), (300, 70, 4640), (200, 1000, 544), (65, 4, 32), (500, 1000, 4608), (1000, 1, 96)])
def test_many_rows_few_tiles(M, N, K, a_format, out):
    dense(M, N, K, a_format, out)
    dense(M, N, K, a_format, out, alpha=0.5, beta=2.0, with_bias=True, pitch=N + 3)


@BOTH
@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("counts,N,K", [
    ([300, 0, 77, 500, 1, 129, 260], 720, 544),     # 128 x 128 tiles, ragged
    ([300, 0, 77, 500, 1, 129, 260], 720, 4640),    # ... with K split
    ([0, 520, 0, 90], 100, 1184),                   # few tiles: 32 rows at a time
    ([0] * 70 + [900, 3, 4000], 160, 288)])         # more than 64 groups
def test_groups(counts, N, K, a_format, out):
    grouped(counts, N, K, a_format, out, lead=2, tail=1, with_bias=True)


def test_split_k_is_the_same_every_time():
    """Two groups' sums are added in a fixed order: bit for bit, with other products between."""
    import torch
    A, As, _ = make(700, 4640, "E4M3", 1)
    B, Bs, _ = make(1600, 4640, "E2M1", 2)
    args = up(A), up(As), up(B), up(Bs)
    one = up(A[:1]), up(As[:1]), *args[2:]
    with dg.MxPlan(700, 1600, 4640, a_format="E4M3", out_dtype="F32") as p:
        D = [torch.empty(700, 1600, dtype=torch_out("F32"), device="cuda") for _ in range(3)]
        for i in range(3):
            p.run(*args, D[i])
            p.run(*one, torch.empty(1, 1600, dtype=torch_out("F32"), device="cuda"))
        torch.cuda.synchronize()
    assert torch.equal(D[0], D[1]) and torch.equal(D[0], D[2])
