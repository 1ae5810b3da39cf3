"""GPU tests of the F8 products against fp64.

Bar: that of the e4m3 GEMM (oracle.parity): the accumulation within 1e-4 of
the rows' norms, plus the rounding of a bf16 output; operands are the same
bytes on both sides.  Products of small whole numbers are exact in fp32: held
to equality there."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import codecs, f8, parity

pytestmark = pytest.mark.gpu


def make(rows, cols, seed, spread=4):
    """An F8 tensor's bytes with blocks of different scales, and its values (padding included)."""
    g = np.random.default_rng(seed)
    blocks = -(-cols // 128)
    x = g.standard_normal((rows, cols)) * np.repeat(np.exp2(g.integers(-spread, spread + 1, (rows, blocks))), 128, axis=1)[:, :cols]
    codes, scales = f8.quantize(x)
    return codes, scales, f8.values(codes, scales)


def up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def torch_out(out):
    import torch
    return torch.bfloat16 if out == "BF16" else torch.float32


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def workspace(M, N, K):
    import torch
    return torch.empty(dg.dist_gemm_f8_product_workspace(M, N, K), dtype=torch.uint8, device="cuda")


def check(got, a, b, out, alpha=1.0, beta=0.0, C=None, bias=None):
    if got.size == 0:
        return
    D = alpha * (a @ b.T)
    if beta:
        D = D + beta * C
    if bias is not None:
        D = D + bias[None]
    ok, worst, tight, _ = parity.check(got, D, np.linalg.norm(a, axis=1), np.linalg.norm(b, axis=1), alpha, beta, C,
                                       "e4m3", "bf16" if out == "BF16" else "f32", bias)
    assert ok and tight, worst


def dense(M, N, K, out, seed=1, alpha=1.0, beta=0.0, with_bias=False, pitch=None, in_place=False):
    import torch
    log("f8 product", M, N, K, out, alpha, beta, with_bias, pitch)
    A, As, a = make(M, K, seed)
    B, Bs, b = make(N, K, seed + 1)
    g = np.random.default_rng(seed + 2)
    t = torch_out(out)
    buf = torch.full((max(M, 1), pitch or N), -5.0, dtype=t, device="cuda")
    D = buf[:M, :N]
    C = c64 = bias = b64 = None
    if beta:
        C = torch.from_numpy(g.standard_normal((M, N)) * 10).to(t).cuda()
        c64 = f64(C)
        if in_place:
            D.copy_(C)
            C = D
    if with_bias:
        bias = torch.from_numpy(g.standard_normal(N) * 10).to(t).cuda()
        b64 = f64(bias)
    dg.dist_gemm_f8_product(up(A), up(As), up(B), up(Bs), D, bias=bias, C=C, alpha=alpha, beta=beta,
                            workspace=workspace(M, N, f8.pitch(K)))
    torch.cuda.synchronize()
    check(f64(D), a, b, out, alpha, beta, c64, b64)
    assert (buf[:, N:] == -5.0).all()
    return f64(D), a, b


SIZES = [(1, 1, 1), (1, 16, 128), (3, 5, 96), (16, 48, 512), (17, 33, 544), (1, 272, 4096), (4, 60, 16384), (15, 70, 4096), (31, 90, 2048), (60, 200, 1100), (31, 100, 992), (33, 64, 1536),
         (2, 100, 16384), (5, 40, 20000), (64, 130, 2080), (65, 257, 160), (100, 300, 1024), (129, 128, 3584), (200, 520, 608),
         (256, 256, 256), (300, 700, 1120), (513, 260, 512), (700, 1030, 2048), (150, 500, 6000), (520, 530, 4224), (140, 900, 128),
         # K in parts
         (70, 130, 20000), (33, 60, 16400), (130, 300, 16500), (513, 700, 12000), (300, 1000, 30000),
         # more than a tile of 64 x 128 per CU
         (2100, 1100, 200), (1000, 3000, 384)]


@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_dense(M, N, K, out):
    dense(M, N, K, out)


@pytest.mark.parametrize("M,N,K", [(2, 40, 96), (24, 100, 544), (60, 33, 1024), (150, 200, 2080), (600, 1000, 640), (130, 260, 5000), (130, 260, 20000), (2200, 1030, 300)])
def test_small_products_are_exact(M, N, K):
    """Scales all 1 and codes of whole numbers up to 8: every sum is a whole number under 2^23, so fp32 holds it exactly."""
    import torch
    g = np.random.default_rng(K)
    a, b = (np.pad(g.integers(-8, 9, (r, K)).astype(np.float64), ((0, 0), (0, f8.pitch(K) - K))) for r in (M, N))
    one = lambda r: up(np.full((r, f8.scale_pitch(K)), 127, dtype=np.uint8))  # noqa: E731
    D = torch.empty((M, N), device="cuda")
    dg.dist_gemm_f8_product(up(codecs.f64_to_e4m3(a)), one(M), up(codecs.f64_to_e4m3(b)), one(N), D,
                            workspace=workspace(M, N, f8.pitch(K)))
    assert np.array_equal(f64(D), a @ b.T)


@pytest.mark.parametrize("M,N,K", [(8, 64, 1024), (3, 50, 4096), (40, 70, 5120), (140, 200, 512), (600, 520, 512), (130, 200, 6400), (130, 200, 20480), (400, 520, 16384)])
def test_every_block_has_its_own_scale(M, N, K):
    """One element of A set per row, another block each: D is that element's
    value times its column of B, so a scale taken from a neighbour shows."""
    import torch
    g = np.random.default_rng(M)
    a = np.zeros((M, K))
    a[np.arange(M), g.integers(0, K, M)] = np.exp2(g.integers(-20, 20, M)) * g.choice([-1.5, 1.0], M)
    A, As = f8.quantize(a)
    B, Bs, b = make(N, K, 3, spread=12)
    D = torch.empty((M, N), device="cuda")
    dg.dist_gemm_f8_product(up(A), up(As), up(B), up(Bs), D, workspace=workspace(M, N, K))
    assert np.array_equal(f64(D), a @ b.T)       # one product per element: exact


@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,K", [(5, 70, 544), (50, 64, 5120), (130, 300, 512), (520, 512, 512), (140, 260, 6400), (140, 262, 20000), (130, 301, 17000)])
def test_alpha_beta_bias(M, N, K, out):
    dense(M, N, K, out, alpha=0.5, beta=-2.0, with_bias=True, pitch=N + 5)
    dense(M, N, K, out, alpha=-1.5, with_bias=True, pitch=N + 8)
    dense(M, N, K, out, alpha=1.0, beta=1.0, in_place=True, pitch=N + 4)
    dense(M, N, K, out, alpha=0.0, beta=1.0)


@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,K", [(40, 128, 256), (130, 256, 512), (300, 512, 256), (2200, 1024, 128), (130, 384, 17000)])
def test_c_and_bias_at_every_alignment(M, N, K, out):
    """Whole blocks of columns with C, bias and D aligned for wide accesses and each of them not."""
    import torch
    log("f8 alignment", M, N, K, out)
    A, As, a = make(M, K, 1)
    B, Bs, b = make(N, K, 2)
    A, As, B, Bs = up(A), up(As), up(B), up(Bs)
    g = np.random.default_rng(5)
    t = torch_out(out)
    c = torch.from_numpy(g.standard_normal((M, N)) * 10).to(t).cuda()
    v = torch.from_numpy(g.standard_normal(N) * 10).to(t).cuda()
    ws = workspace(M, N, f8.pitch(K))

    def at(x, skew, pitch):
        rows, cols = x.shape
        w = torch.full((skew + rows * pitch,), -5.0, dtype=t, device="cuda")[skew:].as_strided((rows, cols), (pitch, 1))
        w.copy_(x)
        return w

    for dc, dv, dd in ((0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1), (2, 2, 0)):
        bias = at(v[None], dv, N)[0]
        for beta in (0.0, 2.0):
            for with_bias in (False, True):
                D, C = at(torch.zeros_like(c), dd, N + dd), at(c, dc, N + dc)
                dg.dist_gemm_f8_product(A, As, B, Bs, D, bias=bias if with_bias else None, C=C, beta=beta, alpha=0.5, workspace=ws)
                check(f64(D), a, b, out, 0.5, beta, f64(c), f64(v) if with_bias else None)


def test_without_beta_c_is_not_read():
    import torch
    A, As, a = make(70, 256, 1)
    B, Bs, b = make(64, 256, 2)
    C = torch.full((70, 64), float("nan"), device="cuda")
    D = torch.empty((70, 64), device="cuda")
    dg.dist_gemm_f8_product(up(A), up(As), up(B), up(Bs), D, C=C, beta=0.0, workspace=workspace(70, 64, 256))
    check(f64(D), a, b, "F32")


@pytest.mark.parametrize("M", [4, 50, 200, 600])
@pytest.mark.parametrize("K", [300, 6400, 24000])
def test_nan_blocks_reach_their_rows_and_columns_alone(M, K):
    import torch
    A, As, a = make(M, K, 1)
    B, Bs, b = make(130, K, 2)
    As[1, 1], Bs[3, 0] = 255, 255
    B[7, 5] = 0x7F
    D = torch.empty((M, 130), device="cuda")
    dg.dist_gemm_f8_product(up(A), up(As), up(B), up(Bs), D, workspace=workspace(M, 130, f8.pitch(K)))
    got = f64(D)
    bad = np.zeros(got.shape, bool)
    bad[1], bad[:, 3], bad[:, 7] = True, True, True
    assert np.array_equal(np.isnan(got), bad)
    rows, cols = np.arange(M) != 1, ~np.isin(np.arange(130), (3, 7))
    check(got[np.ix_(rows, cols)], a[rows], b[cols], "F32")


@pytest.mark.parametrize("M", [3, 40, 200, 520])
@pytest.mark.parametrize("K", [300, 6400, 24000])
def test_scale_bytes_past_the_blocks_do_not_count(M, K):
    import torch
    A, As, a = make(M, K, 1)
    B, Bs, b = make(300, K, 2)
    blocks = f8.pitch(K) // 128
    As[:, blocks:], Bs[:, blocks:] = 255, 255
    D = torch.empty((M, 300), device="cuda")
    dg.dist_gemm_f8_product(up(A), up(As), up(B), up(Bs), D, workspace=workspace(M, 300, f8.pitch(K)))
    check(f64(D), a, b, "F32")


@pytest.mark.parametrize("M", [1, 30, 100, 300])
def test_the_largest_and_smallest_scales(M):
    """Products far below and above 1 whose scales multiply back to the middle."""
    import torch
    A, As, a = make(M, 384, 1, spread=0)
    B, Bs, b = make(70, 384, 2, spread=0)
    As[:, :3], Bs[:, :3] = 1, 253
    D = torch.empty((M, 70), device="cuda")
    dg.dist_gemm_f8_product(up(A), up(As), up(B), up(Bs), D, workspace=workspace(M, 70, 384))
    check(f64(D), codecs.e4m3_to_f64(A), codecs.e4m3_to_f64(B), "F32")


@pytest.mark.parametrize("M,N", [(1, 70000), (70000, 1), (3, 33), (129, 1), (1000, 3), (16, 5000), (4100, 70)])
def test_long_and_thin(M, N):
    dense(M, N, 256, "BF16")


def test_no_rows():
    import torch
    B, Bs, _ = make(64, 128, 2)
    e = torch.empty((0, 128), dtype=torch.uint8, device="cuda")
    dg.dist_gemm_f8_product(e, e[:, :16].contiguous(), up(B), up(Bs), torch.empty((0, 64), device="cuda"))


def test_the_same_from_run_to_run():
    for M, N, K in ((3, 1000, 4096), (200, 1024, 7168), (520, 1024, 1024), (300, 300, 20480)):
        r = [dense(M, N, K, "F32")[0] for _ in range(3)]
        assert np.array_equal(r[0], r[1]) and np.array_equal(r[0], r[2])


@pytest.mark.parametrize("M,N,K", [(7, 300, 1100), (100, 300, 1100), (200, 1024, 7168), (700, 700, 700), (200, 500, 20480)])
def test_on_a_stream_of_its_own_and_in_a_graph(M, N, K):
    import torch
    A, As, a = make(M, K, 1)
    B, Bs, b = make(N, K, 2)
    A, As, B, Bs = up(A), up(As), up(B), up(Bs)
    D = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = workspace(M, N, f8.pitch(K))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dg.dist_gemm_f8_product(A, As, B, Bs, D, workspace=ws)
    side.synchronize()
    want = D.clone()
    check(f64(D), a, b, "BF16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dist_gemm_f8_product(A, As, B, Bs, D, workspace=ws)
    for i in range(3):
        D.fill_(i)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D, want)
        dg.dist_gemm_f8_product(A, As, B, Bs, D, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(D, want)


def test_operands_past_4_gib():
    """B's last rows start past 2^32 bytes; sampled columns against their own product."""
    import torch
    N, K, M = 270000, 16384, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    B = torch.randint(0, 100, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    Bs = torch.randint(120, 130, (N, f8.scale_pitch(K)), dtype=torch.uint8, device="cuda", generator=g)
    A, As, a = make(M, K, 3)
    for rows in (M, 300):
        A2, As2 = (np.resize(t, (rows, t.shape[1])) for t in (A, As))
        D = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
        dg.dist_gemm_f8_product(up(A2), up(As2), B, Bs, D, workspace=workspace(rows, N, K))
        cols = torch.tensor([0, 1, 127, 262143, 262144, 262145, N - 129, N - 1], device="cuda")
        b = f8.values(B[cols].cpu().numpy(), Bs[cols].cpu().numpy())
        check(f64(D[:M, cols]), a, b, "BF16")


def test_refusals_of_tensors():
    import torch
    A, As, _ = make(8, 200, 1)
    B, Bs, _ = make(16, 200, 2)
    good = dict(A=up(A), A_scales=up(As), B=up(B), B_scales=up(Bs), D=torch.empty((8, 16), device="cuda"), workspace=workspace(8, 16, 256))
    dg.dist_gemm_f8_product(**good)
    for bad in (dict(A=good["A"][:, :128].contiguous()), dict(A=good["A"][:7]), dict(B=good["B"][:, :128].contiguous()),
                dict(A_scales=good["A_scales"][:7]), dict(B_scales=good["B_scales"].int()), dict(D=torch.empty((8, 15), device="cuda")),
                dict(D=torch.empty((8, 16), dtype=torch.float16, device="cuda")), dict(D=torch.empty((16, 8), device="cuda").t()),
                dict(bias=torch.empty(15, device="cuda")), dict(bias=torch.empty(16, dtype=torch.bfloat16, device="cuda")),
                dict(C=torch.empty((8, 15), device="cuda")), dict(beta=1.0), dict(alpha=float("nan")), dict(A=good["A"].cpu()),
                dict(A=good["A"].reshape(-1))):
        with pytest.raises((ValueError, dg.DistGemmError)):
            dg.dist_gemm_f8_product(**{**good, **bad})


def test_parts_are_what_these_sizes_take():
    """The sizes above that stand for K in parts have a workspace, and one that is too small, missing or misaligned is refused."""
    import torch
    for M, N, K in ((70, 130, 20096), (33, 60, 16512), (130, 300, 16512), (513, 700, 12032), (200, 130, 24064), (40, 130, 24064)):
        assert dg.dist_gemm_f8_product_workspace(M, N, K) > 0
    assert dg.dist_gemm_f8_product_workspace(64, 64, 100) == 0 and dg.dist_gemm_f8_product_workspace(-1, 64, 128) == 0
    M, N, K = 130, 300, 16512
    A, As, a = make(M, K, 1)
    B, Bs, b = make(N, K, 2)
    n = dg.dist_gemm_f8_product_workspace(M, N, K)
    ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
    D = torch.empty((M, N), device="cuda")
    args = (up(A), up(As), up(B), up(Bs), D)
    for bad in (None, ws[:n - 1], ws[8:], ws[:0], ws.cpu(), ws[::2]):
        with pytest.raises((ValueError, dg.DistGemmError)):
            dg.dist_gemm_f8_product(*args, workspace=bad)
    with pytest.raises(dg.DistGemmError, match="alias"):
        big = torch.empty((n // 1200 + 1) * 300, device="cuda")
        dg.dist_gemm_f8_product(*args[:4], big[:M * N].view(M, N), workspace=big)
    dg.dist_gemm_f8_product(*args, workspace=ws[:n])
    check(f64(D), a, b, "F32")
