"""GPU tests of the F8 operators at the ends of their sizes, against fp64 on the
GPU (the operands' values from their bit fields, float64 matmul): the longest
K, millions of rows and of columns, tiles of few slabs in long streams, and
rows of the norm past 2^31 elements."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import codecs, f8

pytestmark = pytest.mark.gpu


def draw(rows, K, seed):
    """Random codes (no NaN) with scales around 1, made on the GPU."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (rows, K), dtype=torch.uint8, device="cuda", generator=g)
    c[(c & 0x7F) == 0x7F] = 0
    s = torch.randint(117, 121, (rows, f8.scale_pitch(K)), dtype=torch.uint8, device="cuda", generator=g)
    return c, s


def values(c, s):
    import torch
    table = torch.from_numpy(codecs.e4m3_to_f64(np.arange(256, dtype=np.uint8))).cuda()
    return table[c.int()] * torch.exp2(s[:, :c.size(1) // 128].double() - 127).repeat_interleave(128, 1)


def workspace(M, N, K):
    import torch
    return torch.empty(dg.dist_gemm_f8_product_workspace(M, N, K), dtype=torch.uint8, device="cuda")


def close(D, a, b):
    """Within 1e-4 of the rows' norms, the bar of the e4m3 products, plus the rounding of a bf16 output."""
    ref = a @ b.t()
    size = a.norm(dim=1)[:, None] * b.norm(dim=1)[None]
    assert bool(((D.double() - ref).abs() <= 1e-4 * size + (2.0 ** -8 * ref.abs() if D.element_size() == 2 else 0)).all())


@pytest.mark.parametrize("M,N", [(3, 20), (40, 70), (70, 300), (300, 40)])
def test_the_longest_k(M, N):
    import torch
    K = 1 << 22
    log("f8 longest", M, N)
    A, B = draw(M, K, 1), draw(N, K, 2)
    D = torch.empty((M, N), device="cuda")
    dg.dist_gemm_f8_product(*A, *B, D, workspace=workspace(M, N, K))
    ref = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    na, nb = torch.zeros(M, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    step = 1 << 19
    for k in range(0, K, step):
        a, b = (values(c[:, k:k + step], s[:, k // 128:(k + step) // 128]) for c, s in (A, B))
        ref += a @ b.t()
        na += a.square().sum(1)
        nb += b.square().sum(1)
    assert bool(((D.double() - ref).abs() <= 1e-4 * na.sqrt()[:, None] * nb.sqrt()[None]).all())


@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,K", [(48, 50000, k) for k in (128, 256, 384, 512, 640, 1920, 2048, 2176, 2304, 2432, 4224)]
                         + [(1000, 9000, k) for k in (128, 256, 384, 2048, 2176, 2304)] + [(130, 40000, 256), (3000, 9000, 2176)])
def test_streams_of_many_tiles(M, N, K, out):
    """Several tiles to a workgroup, of one slab, of the stages' number, and either side of a chunk of scales."""
    import torch
    log("f8 streams", M, N, K, out)
    A, B = draw(M, K, 1), draw(N, K, 2)
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16 if out == "BF16" else torch.float32, device="cuda")
    dg.dist_gemm_f8_product(*A, *B, D, workspace=workspace(M, N, K))
    close(D, values(*A), values(*B))


@pytest.mark.parametrize("M,N", [((1 << 24) + 77, 3), (2, (1 << 24) + 5), (40, (1 << 22) + 9), ((1 << 22) + 1, 200)])
def test_millions_of_rows_or_columns(M, N):
    import torch
    log("f8 millions", M, N)
    K = 128
    A, B = draw(M, K, 1), draw(N, K, 2)
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dist_gemm_f8_product(*A, *B, D, workspace=workspace(M, N, K))
    assert not torch.isnan(D).any()
    g = torch.Generator(device="cuda").manual_seed(3)

    def some(n):
        i = torch.randint(0, n, (min(n, 2000),), device="cuda", generator=g)
        return torch.cat((i, torch.tensor([0, n - 1], device="cuda")))

    i, j = some(M), some(N)
    close(D[i][:, j], values(A[0][i], A[1][i]), values(B[0][j], B[1][j]))


def test_norm_and_gradient_past_32_bits_of_elements():
    """2^31 elements and more: the last rows against the same rows by themselves."""
    import torch
    rows, cols = 270000, 8200
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    w, b = (torch.randn(cols, generator=g, device="cuda").bfloat16() for _ in range(2))
    empty = lambda n: (torch.empty((n, f8.pitch(cols)), dtype=torch.uint8, device="cuda"),  # noqa: E731
                       torch.empty((n, f8.scale_pitch(cols)), dtype=torch.uint8, device="cuda"))

    def run(x):
        n = x.size(0)
        (y, s), (k, ks) = empty(n), empty(n)
        mean, rstd, dx = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x)
        dg.dist_gemm_layer_norm(x, w, b, y, output="F8", scales=s, mean=mean, rstd=rstd, kept=k, kept_scales=ks)
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        ws = torch.empty(dg.dist_gemm_layer_norm_workspace(n, cols), dtype=torch.uint8, device="cuda")
        dg.dist_gemm_layer_norm_backward(x, k, None, rstd, w, dx, dw, db, ws, h_scales=ks)
        return y, s, k, ks, mean, rstd, dx

    whole = [t[-3000:].clone() for t in run(x)]
    assert all(torch.equal(p, q) for p, q in zip(run(x[-3000:]), whole))


def test_long_columns_of_one():
    """One column by millions of rows and the other way round: a block is mostly padding, or one of many."""
    import torch
    n = (1 << 23) + 3
    x = torch.randn(n, 1, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    for v, shape in ((x, (n, 1)), (x.view(1, n), (1, n))):
        rows, cols = shape
        a = (torch.empty((rows, f8.pitch(cols)), dtype=torch.uint8, device="cuda"), torch.empty((rows, f8.scale_pitch(cols)), dtype=torch.uint8, device="cuda"))
        b = (torch.empty((cols, f8.pitch(rows)), dtype=torch.uint8, device="cuda"), torch.empty((cols, f8.scale_pitch(rows)), dtype=torch.uint8, device="cuda"))
        dg.dist_gemm_f8_quantize(v, *a, *b)
        y = torch.empty_like(v)
        dg.dist_gemm_f8_dequantize(*a, y)
        assert bool(((y - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -10).all())
        z = torch.empty((cols, rows), device="cuda")
        dg.dist_gemm_f8_dequantize(*b, z)
        assert bool(((z.t() - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -10).all())
        c = (torch.empty_like(b[0]), torch.empty_like(b[1]))
        dg.dist_gemm_f8_transpose(*a, *c)
        dg.dist_gemm_f8_dequantize(*c, z)
        assert bool(((z.t() - y).abs() <= 2.0 ** -10 * 2.0 ** -5).all())
