"""GPU tests of the MX products at the ends of their range: as many columns and
rows as a plan takes, K of one block.

Bars as in test_gpu_13_mx_products.py, whose helpers these are."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import mx
from test_gpu_13_mx_products import check_on_gpu, random_codes, up

pytestmark = pytest.mark.gpu

K = 32
MOST = (1 << 31) - 1


@pytest.fixture(scope="module")
def large():
    """A tensor of MOST rows of 32 in E2M1, 34 GB of codes and 34 of scales."""
    import torch
    log("large tensor")
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.empty((MOST, K // 2), dtype=torch.uint8, device="cuda")
    codes.view(torch.int64).random_(generator=g)
    scales = torch.randint(120, 130, (MOST, mx.scale_pitch(K)), generator=g, dtype=torch.uint8, device="cuda")
    yield codes, scales
    del codes, scales
    torch.cuda.empty_cache()


def values(large, lo, hi):
    import torch
    c, s = large[0][lo:hi], large[1][lo:hi]
    table = torch.from_numpy(mx.e2m1_to_f64(np.arange(16))).cuda()
    v = table[torch.stack((c & 15, c >> 4), -1).reshape(hi - lo, K).long()]
    return v * torch.exp2(s[:, :K // 32].double() - 127).repeat_interleave(K, -1)


def windows(n):
    """Where a launch's parts meet (2^21 workgroups of 16 and 32 columns) and the two ends."""
    at = {0, n // 2, n - 3000} | {k << 25 for k in (1, 2, 3)} | {k << 26 for k in (1, 5, 31)}
    return [(max(p - 1500, 0), min(p + 3000, n)) for p in sorted(at) if p < n]


@pytest.mark.parametrize("rows,N", [(1, (1 << 25) + 5), (40, (1 << 26) + 77), (1, MOST), (3, MOST - 100)])
def test_columns(large, rows, N):
    import torch
    log("columns", rows, N)
    A, As, a = random_codes(rows, K, "E2M1", 1)
    D = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    with dg.MxPlan(rows, N, K) as p:
        p.run(A, As, large[0][:N], large[1][:N], D)
        torch.cuda.synchronize()
    for r in range(rows):
        assert not bool(torch.isnan(D[r]).any())      # every column was written
    for lo, hi in windows(N):
        check_on_gpu(D[:, lo:hi], a, values(large, lo, hi), "BF16")


@pytest.mark.parametrize("groups", [0, 1, 70])
@pytest.mark.parametrize("M", [MOST, MOST - 130])
def test_rows(large, M, groups):
    import torch
    log("rows", M, groups)
    E = max(groups, 1)
    B, Bs, b = random_codes(E, K, "E2M1", 2)
    off = None
    if groups:       # all rows in the last group but one
        off = up(np.array([0] * max(groups - 1, 1) + [M] * (groups + 1 - max(groups - 1, 1)), dtype=np.int32))
    D = torch.full((M, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    with dg.MxPlan(M, 1, K, groups=groups) as p:
        p.run(large[0][:M], large[1][:M], B, Bs, D, offsets=off)
        torch.cuda.synchronize()
    assert not bool(torch.isnan(D).any())
    one = b[max(groups - 2, 0):][:1]
    for lo, hi in windows(M):
        check_on_gpu(D[lo:hi], values(large, lo, hi), one, "BF16")
