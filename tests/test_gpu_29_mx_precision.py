"""GPU tests of what the MX products' sums lose: fp32 results against fp64, with
the bar and the data of the F8 products' tests (test_gpu_27_f8_precision.py has
its derivation).  E2M1 by E2M1 loses nothing but fp32's own rounding: the cuts are
asserted to be none."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import mx
from test_gpu_27_f8_precision import cuts

pytestmark = pytest.mark.gpu

# few rows, tiles 32 rows at a time, of 128 x 128 (one and two groups of waves) and 256 x 256
SIZES = [(1, 512, 8192), (16, 512, 1024), (64, 520, 2048), (300, 512, 4096), (1024, 4096, 1024), (1000, 4000, 8192), (4096, 8192, 1024)]


@pytest.mark.parametrize("loud", [False, True])
@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sums(M, N, K, fmt, loud):
    import torch
    log("mx precision", M, N, K, fmt, loud)
    g = np.random.default_rng(M + N)
    x, w = g.standard_normal((M, K)), g.standard_normal((N, K))
    if loud:
        x *= 1 + 15 * (g.random(K) < 0.01)
    (A, As), (B, Bs) = mx.quantize(x, fmt), mx.quantize(w, "E2M1")
    up = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()  # noqa: E731
    D = torch.empty((M, N), device="cuda")
    with dg.MxPlan(M, N, K, a_format=fmt, out_dtype="F32") as plan:
        plan.run(up(A), up(As), up(B), up(Bs), D)
        torch.cuda.synchronize()
    # at least 512 results, spread over the rows and columns
    i = np.unique(np.linspace(0, M - 1, 24).astype(int))
    j = np.unique(np.linspace(0, N - 1, max(24, -(-512 // len(i)))).astype(int))
    a, b = up(mx.values(A[i], As[i], fmt, K)), up(mx.values(B[j], Bs[j], "E2M1", K))
    ref = a @ b.t()
    err = (D[i][:, j].double() - ref).abs()
    square, most = torch.empty_like(ref), torch.empty_like(ref)
    for r in range(len(i)):
        square[r], most[r] = cuts(a[r], b)
    if fmt == "E2M1":
        assert not most.any()
    rms = ref.square().mean().sqrt()
    got, bar = err.square().mean().sqrt(), square.mean().sqrt() + (K / 8) ** 0.5 * 2.0 ** -23 * rms
    log("   of the results' rms: off by", (got / rms).item(), "bar", (bar / rms).item())
    assert got <= bar
    assert bool((err <= most + K / 8 * 2.0 ** -23 * (a.abs() @ b.abs().t())).all())
