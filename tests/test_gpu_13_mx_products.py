"""GPU tests of the MX products, dense and by group of rows, against fp64.

Bar: that of the e4m3 GEMM (oracle.parity): the accumulation within 1e-4 of
the rows' norms, plus the rounding of a bf16 output; operands are the same
bytes on both sides.  The E2M1 x E2M1 product of small sizes is exact in fp32,
since every product is a multiple of a power of two: held to equality there."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import codecs, mx, parity

pytestmark = pytest.mark.gpu


def make(rows, cols, fmt, seed, spread=4):
    """An MX tensor's bytes with blocks of different scales, and its values."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)) * np.repeat(np.exp2(g.integers(-spread, spread + 1, (rows, cols // 32))), 32, axis=1)
    codes, scales = mx.quantize(x, fmt)
    return codes, scales, mx.values(codes, scales, fmt, cols)


def up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def torch_out(out):
    import torch
    return torch.bfloat16 if out == "BF16" else torch.float32


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


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


def dense(M, N, K, a_format, out, seed=1, alpha=1.0, beta=0.0, with_bias=False, pitch=None, rows=None, in_place=False):
    import torch
    log("product", M, N, K, a_format, out, alpha, beta, with_bias, pitch, rows)
    rows = M if rows is None else rows
    A, As, a = make(rows, K, a_format, seed)
    B, Bs, b = make(N, K, "E2M1", seed + 1)
    g = np.random.default_rng(seed + 2)
    t = torch_out(out)
    buf = torch.full((max(rows, 1), pitch or N), -5.0, dtype=t, device="cuda")
    D = buf[:rows, :N]
    C = c64 = bias = b64 = None
    if beta:
        C = torch.from_numpy(g.standard_normal((rows, N)) * 10).to(t).cuda()
        c64 = f64(C)
        if in_place:
            D.copy_(C)
            C = D
    if with_bias:
        bias = torch.from_numpy(g.standard_normal(N) * 10).to(t).cuda()
        b64 = f64(bias)
    with dg.MxPlan(M, N, K, a_format=a_format, out_dtype=out) as p:
        p.run(up(A), up(As), up(B), up(Bs), D, bias=bias, C=C, alpha=alpha, beta=beta)
        torch.cuda.synchronize()
    check(f64(D), a, b, out, alpha, beta, c64, b64)
    assert (buf[:, N:] == -5.0).all()
    return f64(D), a, b


SIZES = [(1, 1, 32), (1, 16, 64), (3, 5, 96), (16, 48, 512), (17, 33, 544), (1, 272, 4096), (31, 100, 992), (33, 64, 1536),
         (64, 130, 2080), (65, 257, 160), (100, 300, 1024), (129, 128, 3584), (200, 520, 608), (256, 256, 256),
         (300, 700, 1120), (513, 260, 512), (700, 1030, 2048)]


@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_dense(M, N, K, a_format, out):
    dense(M, N, K, a_format, out)


@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("M,N,K", [(2, 40, 96), (24, 100, 544), (60, 33, 1024), (150, 200, 2080), (600, 1000, 640)])
def test_small_products_are_exact(M, N, K, a_format):
    """Scales all 1 and e4m3 codes of whole numbers up to 8: every product is a
    multiple of 1/2 and every sum under 2^23, so fp32 holds them exactly."""
    import torch
    g = np.random.default_rng(K)
    b = mx.E2M1_VALUES[g.integers(0, 8, (N, K))] * g.choice([-1, 1], (N, K))
    a = mx.E2M1_VALUES[g.integers(0, 8, (M, K))] * g.choice([-1, 1], (M, K)) if a_format == "E2M1" else \
        g.integers(-8, 9, (M, K)).astype(np.float64)
    A = mx.pack(mx.f64_to_e2m1(a)) if a_format == "E2M1" else codecs.f64_to_e4m3(a)
    one = lambda r: up(np.pad(np.full((r, K // 32), 127, dtype=np.uint8), ((0, 0), (0, mx.scale_pitch(K) - K // 32))))  # noqa: E731
    D = torch.empty((M, N), device="cuda")
    with dg.MxPlan(M, N, K, a_format=a_format, out_dtype="F32") as p:
        p.run(up(A), one(M), up(mx.pack(mx.f64_to_e2m1(b))), one(N), D)
    assert np.array_equal(f64(D), a @ b.T)


@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("M,N,K", [(8, 64, 1024), (140, 200, 512), (600, 520, 512)])
def test_every_block_has_its_own_scale(M, N, K, a_format):
    """One element of A set per row, another block each: D is that element's
    value times its column of B, so a scale taken from a neighbour shows."""
    import torch
    g = np.random.default_rng(M)
    a = np.zeros((M, K))
    at = g.integers(0, K, M)
    a[np.arange(M), at] = np.exp2(g.integers(-20, 20, M)) * g.choice([-1.5, 1.0], M)
    A, As = mx.quantize(a, a_format)
    B, Bs, b = make(N, K, "E2M1", 3, spread=12)
    D = torch.empty((M, N), device="cuda")
    with dg.MxPlan(M, N, K, a_format=a_format, out_dtype="F32") as p:
        p.run(up(A), up(As), up(B), up(Bs), D)
    assert np.array_equal(f64(D), a @ b.T)       # one product per element: exact


@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,K", [(5, 70, 544), (130, 300, 512), (520, 512, 512)])
def test_alpha_beta_bias(M, N, K, out):
    dense(M, N, K, "E4M3", out, alpha=0.375, beta=-1.5, with_bias=True)
    dense(M, N, K, "E2M1", out, alpha=2.0, beta=1.0, in_place=True)
    dense(M, N, K, "E2M1", out, alpha=0.0, beta=0.5, with_bias=True)
    dense(M, N, K, "E4M3", out, with_bias=True)


@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("M,N,pitch", [(9, 64, 65), (140, 130, 132), (300, 256, 259), (520, 256, 264)])
def test_pitch_of_the_output(M, N, pitch, out):
    dense(M, N, 512, "E2M1", out, pitch=pitch, with_bias=True)


@pytest.mark.parametrize("M,N,K", [(4, 64, 1024), (140, 160, 1024), (512, 512, 1024)])
@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
def test_nan_blocks_reach_their_rows_and_columns_alone(M, N, K, a_format):
    import torch
    A, As, a = make(M, K, a_format, 5)
    B, Bs, b = make(N, K, "E2M1", 6)
    As[1, K // 32 - 1] = 255
    Bs[N // 2, 3] = 255
    D = torch.empty((M, N), device="cuda")
    with dg.MxPlan(M, N, K, a_format=a_format, out_dtype="F32") as p:
        p.run(up(A), up(As), up(B), up(Bs), D)
    nan = np.isnan(f64(D))
    want = np.zeros((M, N), dtype=bool)
    want[1], want[:, N // 2] = True, True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("M,N,K", [(4, 40, 544), (70, 100, 96), (600, 520, 1120)])
@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
def test_scale_bytes_past_k_are_not_used(M, N, K, a_format):
    import torch
    A, As, a = make(M, K, a_format, 5)
    B, Bs, b = make(N, K, "E2M1", 6)
    D, E = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    with dg.MxPlan(M, N, K, a_format=a_format, out_dtype="F32") as p:
        p.run(up(A), up(As), up(B), up(Bs), D)
        As[:, K // 32:], Bs[:, K // 32:] = 255, 255
        p.run(up(A), up(As), up(B), up(Bs), E)
    assert torch.equal(D, E)


def random_codes(rows, cols, fmt, seed):
    """Random codes and scales of an MX tensor on the GPU, and its values (fp64)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (rows, cols // 2 if fmt == "E2M1" else cols), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "E4M3":
        codes = codes & 0xB7                 # no NaN, nothing above 2
    scales = torch.randint(120, 130, (rows, mx.scale_pitch(cols)), generator=g, device="cuda", dtype=torch.uint8)
    table = torch.from_numpy(mx.e2m1_to_f64(np.arange(16)) if fmt == "E2M1" else codecs.e4m3_to_f64(np.arange(256))).cuda()
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(rows, cols) if fmt == "E2M1" else codes
    v = table[c.long()] * torch.exp2(scales[:, :cols // 32].double() - 127).repeat_interleave(32, -1)
    return codes, scales, v


def check_on_gpu(D, a, b, out):
    """check() for large products, on the GPU: same bar."""
    ref = a @ b.T
    size = a.norm(dim=1)[:, None] * b.norm(dim=1)[None]
    diff = (D.double() - ref).abs()
    assert bool((diff <= (2.0 ** -8 if out == "BF16" else 2.0 ** -24) * ref.abs() + parity.TIGHT_ACCUM["e4m3"] * size).all())


# more tiles than workgroups, so that each walks several: 256 x 256 and 128 x 128 tiles, one slab of K and more,
# whole and partial ones
@pytest.mark.parametrize("K", [32, 96, 160, 256, 288, 544, 1024, 1184])
@pytest.mark.parametrize("M,N,out", [(5900, 5000, "BF16"), (5888, 5120, "BF16"), (5900, 5000, "F32"), (2500, 4700, "BF16")])
@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
def test_many_tiles(M, N, K, a_format, out):
    import torch
    log("many tiles", M, N, K, a_format, out)
    A, As, a = random_codes(M, K, a_format, 1)
    B, Bs, b = random_codes(N, K, "E2M1", 2)
    D = torch.full((M, N), 7.0, dtype=torch_out(out), device="cuda")
    with dg.MxPlan(M, N, K, a_format=a_format, out_dtype=out) as p:
        p.run(A, As, B, Bs, D)
    check_on_gpu(D, a, b, out)


@pytest.mark.parametrize("E", [5, 100])
@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("K", [96, 544])
def test_many_grouped_tiles(E, K, a_format):
    import torch
    g = np.random.default_rng(E)
    counts = g.multinomial(9000, g.dirichlet(np.full(E, 0.7)))
    counts[E // 2] = 0
    M, N = int(counts.sum()) + 3, 3400
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    log("many grouped tiles", E, K, a_format, M)
    A, As, a = random_codes(M, K, a_format, 1)
    B, Bs, b = random_codes(E * N, K, "E2M1", 2)
    D = torch.full((M, N), -5.0, dtype=torch.bfloat16, device="cuda")
    with dg.MxPlan(M, N, K, groups=E, a_format=a_format) as p:
        p.run(A, As, B, Bs, D, offsets=up(off))
    for e in range(E):
        check_on_gpu(D[off[e]:off[e + 1]], a[off[e]:off[e + 1]], b[e * N:(e + 1) * N], "BF16")
    assert bool((D[off[-1]:] == -5.0).all())


def test_fewer_rows_than_the_plan():
    for rows in (1, 40, 200, 600):
        dense(600, 512, 512, "E4M3", "BF16", rows=rows)


def test_no_rows():
    import torch
    with dg.MxPlan(8, 64, 64) as p:
        z = torch.empty(0, dtype=torch.uint8, device="cuda")
        w = torch.zeros(64 * 32, dtype=torch.uint8, device="cuda")
        s = torch.zeros(64 * 16, dtype=torch.uint8, device="cuda")
        p.run(z, z, w, s, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))


# ---- by group

def grouped(counts, N, K, a_format, out, lead=0, tail=0, with_bias=False, seed=1, M=None):
    """Groups of these row counts, `lead` rows before the first and `tail` after the last that no group has."""
    import torch
    log("grouped", counts if len(counts) < 20 else len(counts), N, K, a_format, out, lead, tail)
    E, rows = len(counts), lead + sum(counts) + tail
    off = lead + np.concatenate([[0], np.cumsum(counts)])
    A, As, a = make(rows, K, a_format, seed)
    B, Bs, b = make(E * N, K, "E2M1", seed + 1)
    t = torch_out(out)
    D = torch.full((rows, N), -5.0, dtype=t, device="cuda")
    bias = b64 = None
    if with_bias:
        bias = torch.from_numpy(np.random.default_rng(seed).standard_normal((E, N)) * 10).to(t).cuda()
        b64 = f64(bias)
    with dg.MxPlan(M or rows, N, K, groups=E, a_format=a_format, out_dtype=out) as p:
        p.run(up(A), up(As), up(B), up(Bs), D, bias=bias, offsets=up(off.astype(np.int32)))
        torch.cuda.synchronize()
    got = f64(D)
    for g in range(E):
        lo, hi = off[g], off[g + 1]
        check(got[lo:hi], a[lo:hi], b[g * N:(g + 1) * N], out, bias=None if b64 is None else b64[g])
    assert (got[:lead] == -5.0).all() and (got[rows - tail:] == -5.0).all()


GROUPS = [[1], [0, 0, 3], [5, 0, 1, 16, 17], [2] * 70, [0] * 64 + [3] + [0] * 80 + [40], [33, 1, 0, 64, 100],
          [256, 0, 255, 257, 1], [600], [130, 300, 20], [0, 900, 0, 0, 70]]


@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("out", ["BF16", "F32"])
@pytest.mark.parametrize("k", range(len(GROUPS)))
def test_grouped(k, a_format, out):
    grouped(GROUPS[k], 100 if k % 2 else 272, 544 if k % 3 else 1024, a_format, out)


def test_grouped_with_bias_and_rows_of_no_group():
    for counts in ([3, 0, 20], [200, 0, 90, 300], [300, 500]):
        grouped(counts, 200, 512, "E4M3", "BF16", lead=5, tail=9, with_bias=True)
        grouped(counts, 200, 512, "E2M1", "F32", lead=1, with_bias=True)


def test_grouped_all_empty():
    grouped([0, 0, 0], 64, 64, "E4M3", "BF16", lead=40)


def test_grouped_equals_dense_per_group():
    """A group's rows come out as the dense product's, whatever the tiles."""
    import torch
    counts, N, K = [70, 200, 5], 256, 1024
    A, As, _ = make(sum(counts), K, "E2M1", 3)
    B, Bs, _ = make(3 * N, K, "E2M1", 4)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    D = torch.empty((sum(counts), N), device="cuda")
    with dg.MxPlan(sum(counts), N, K, groups=3, out_dtype="F32") as p:
        p.run(up(A), up(As), up(B), up(Bs), D, offsets=up(off))
    for g in range(3):
        lo, hi = off[g], off[g + 1]
        d = torch.empty((hi - lo, N), device="cuda")
        with dg.MxPlan(int(hi - lo), N, K, out_dtype="F32") as p:
            p.run(up(A[lo:hi]), up(As[lo:hi]), up(B[g * N:(g + 1) * N]), up(Bs[g * N:(g + 1) * N]), d)
        size = d.abs().max().item()
        assert (d - D[lo:hi]).abs().max().item() <= 1e-5 * size


def test_on_a_stream_of_its_own_and_in_a_graph():
    import torch
    for M, N, K in ((4, 256, 1024), (200, 256, 1024), (600, 768, 512)):
        A, As, a = make(M, K, "E4M3", 7)
        B, Bs, b = make(N, K, "E2M1", 8)
        dev = [up(t) for t in (A, As, B, Bs)]
        D = torch.zeros((M, N), device="cuda")
        with dg.MxPlan(M, N, K, a_format="E4M3", out_dtype="F32") as p:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                p.run(*dev, D)
            s.synchronize()
            first = D.clone()
            check(f64(D), a, b, "F32")
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                p.run(*dev, D)
            for _ in range(3):
                D.zero_()
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(D, first)
                p.run(*dev, D)
                torch.cuda.synchronize()
                assert torch.equal(D, first)


def test_refusals():
    import torch
    A, As, _ = make(4, 64, "E2M1", 1)
    B, Bs, _ = make(32, 64, "E2M1", 2)
    A, As, B, Bs = up(A), up(As), up(B), up(Bs)
    D = torch.empty((4, 32), dtype=torch.bfloat16, device="cuda")
    with dg.MxPlan(4, 32, 64) as p:
        good = dict(A=A, A_scales=As, B=B, B_scales=Bs, D=D)
        p.run(**good)
        for bad in (dict(A=A[:3]), dict(A_scales=As[:, :8]), dict(B=B[:, :31]), dict(B_scales=Bs.float()), dict(D=D.float()),
                    dict(D=D[:, :31]), dict(bias=torch.zeros(31, dtype=torch.bfloat16, device="cuda")), dict(beta=1.0),
                    dict(alpha=float("nan")), dict(offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
                    dict(A=A.cpu()), dict(D=torch.empty((5, 32), dtype=torch.bfloat16, device="cuda"))):
            with pytest.raises((ValueError, dg.DistGemmError)):
                p.run(**{**good, **bad})
    with pytest.raises(ValueError):
        p.run(**good)                       # closed
    with dg.MxPlan(4, 16, 64, groups=2) as p:
        with pytest.raises(dg.DistGemmError):
            p.run(A, As, B, Bs, D[:, :16].contiguous())     # no offsets
        with pytest.raises(ValueError):
            p.run(A, As, B, Bs, D[:, :16].contiguous(), offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(dg.DistGemmError) as ei:
        dg.MxPlan(4, 32, 48)
    assert ei.value.status == -2
