"""GPU tests of the RMS norm and its gradient against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24): a row's sum of squares adds at
most 32 products per lane in a chain, then a tree over 64 lanes and at most 16
waves one after another: under 64 roundings, so under 32 u on the root; the
quotient, the root and two products add 4 u.  NORM = 48 u relative.  The
gradient's row mean is bound the same way, relative to the mean of |g n|.
dweight: a chain over at most rows / 2 + 16 rows of |dy n| each.  Outputs in
fewer bits add half a step: bf16 2^-8 relative, e4m3 2^-4 relative (2^-10
below its normal range)."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import codecs, mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NORM = 48 * U
EPS = 1e-5
OUT_STEP = {"BF16": 2.0 ** -8, "F32": 0.0}


def torch_type(typ):
    import torch
    return torch.bfloat16 if typ == "BF16" else torch.float32


def draw(rows, cols, typ, seed, pitch=None, skew=0, scale=1.0):
    import torch
    pitch = pitch or cols
    v = np.random.default_rng(seed).standard_normal((rows, cols)) * scale
    t = torch.from_numpy(v).to(torch.float32).to(torch_type(typ))
    buf = torch.zeros(skew + max(rows, 1) * pitch, dtype=t.dtype, device="cuda")
    x = buf[skew:].as_strided((rows, cols), (pitch, 1))
    x.copy_(t)
    return x, t.to(torch.float64).numpy()


def empty(rows, cols, dtype, pitch=None, skew=0):
    import torch
    pitch = pitch or cols
    buf = torch.zeros(skew + max(rows, 1) * pitch, dtype=torch.uint8 if dtype is torch.uint8 else dtype, device="cuda")
    return buf[skew:].as_strided((rows, cols), (pitch, 1))


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def sum_stream(x, r, typ):
    """x + residual, rounded to the type: one fp32 addition, then one rounding."""
    import torch
    s = torch.from_numpy((x.astype(np.float32) + r.astype(np.float32)))
    return s.to(torch_type(typ)).to(torch.float64).numpy()


def run_forward(rows, cols, typ, out, residual, seed, pitch=None, skew=0, scale=0.125, x=None):
    import torch
    log("norm", rows, cols, typ, out, residual, pitch, skew)
    x, x64 = draw(rows, cols, typ, seed, pitch, skew) if x is None else x
    w, w64 = draw(1, cols, typ, seed + 1, skew=skew)
    rstd = torch.zeros(rows, device="cuda")
    kw, h64 = {}, x64
    if residual:
        r, r64 = draw(rows, cols, typ, seed + 2, pitch, skew)
        h = empty(rows, cols, torch_type(typ), pitch, skew)
        kw, h64 = dict(residual=r, h=h), sum_stream(x64, r64, typ)
    if out == "SAME":
        y = empty(rows, cols, torch_type(typ), pitch, skew)
    elif out == "E4M3":
        y = empty(rows, cols, torch.uint8, pitch, skew)
    else:
        y = torch.zeros((rows, cols if out == "MX_E4M3" else cols // 2), dtype=torch.uint8, device="cuda")
        kw["scales"] = torch.full((rows, mx.scale_pitch(cols)), 0xA5, dtype=torch.uint8, device="cuda")
    dg.dist_gemm_rms_norm(x, w[0], y, eps=EPS, output=out, rstd=rstd, scale=scale, **kw)
    y64, rstd64 = mx.rms_norm(h64, w64[0], EPS)
    if residual:
        assert np.array_equal(f64(kw["h"]), h64, equal_nan=True)
    with np.errstate(invalid="ignore"):
        assert not np.any(np.abs(f64(rstd) - rstd64) > NORM * rstd64)
        if out == "SAME":
            assert not np.any(np.abs(f64(y) - y64) > (OUT_STEP[typ] + 2 * NORM) * np.abs(y64))
            assert np.array_equal(np.isnan(f64(y)), np.isnan(y64))
        elif out == "E4M3":
            v = np.clip(y64 / scale, -448, 448)
            got = codecs.e4m3_to_f64(y.cpu().numpy())
            assert not np.any(np.abs(got - v) > (2.0 ** -4 + 2 * NORM) * np.abs(v) + 2.0 ** -10)
            assert np.array_equal(np.isnan(got), np.isnan(v))
    return y, kw, y64


FORWARD_SIZES = [(1, 1), (1, 32), (2, 7), (5, 64), (3, 500), (4, 512), (9, 520), (3, 1000), (2, 2048), (5, 5123), (2, 8192),
                 (3, 16384), (2, 20000), (2, 32768), (2100, 96), (2049, 1025), (2050, 4104)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("out", ["SAME", "E4M3"])
@pytest.mark.parametrize("rows,cols", FORWARD_SIZES)
def test_forward(rows, cols, typ, out, residual):
    run_forward(rows, cols, typ, out, residual, rows + cols)


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("out", ["SAME", "E4M3"])
@pytest.mark.parametrize("pitch,skew", [(136, 0), (129, 0), (128, 1), (144, 8)])
def test_forward_pitches_and_bases(typ, out, pitch, skew):
    run_forward(6, 128, typ, out, True, 4, pitch, skew)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (4, 480), (7, 544), (2, 3584), (3, 16384), (2100, 64)])
def test_forward_into_mx_blocks(rows, cols, typ, fmt, residual):
    """Each value within its block's half step of the exact norm: the scale is
    that of the exact block (or, at a power of two within rounding, the
    neighbouring one), the pad bytes are zero."""
    y, kw, y64 = run_forward(rows, cols, typ, "MX_" + fmt, residual, rows + cols)
    scales = kw["scales"].cpu().numpy()
    assert not scales[:, cols // 32:].any()
    b = y64.reshape(rows, cols // 32, 32)
    amax = np.abs(b).max(-1)
    e = np.maximum(np.floor(np.log2(np.maximum(amax, 1e-300))) - mx.EMAX[fmt], -127)
    s = scales[:, :cols // 32].astype(np.int64) - 127
    edge = np.abs(np.log2(np.maximum(amax, 1e-300)) - np.round(np.log2(np.maximum(amax, 1e-300)))) < 1e-5
    assert np.all((s == e) | (edge & (np.abs(s - e) <= 1)))
    v = mx.values(y.cpu().numpy(), scales, fmt, cols).reshape(b.shape)
    top = {"E2M1": 6.0, "E4M3": 448.0}[fmt]
    f = np.exp2(s.astype(np.float64))[..., None]
    q = np.clip(b / f, -top, top)
    rel, low = {"E2M1": (2.0 ** -2, 0.25), "E4M3": (2.0 ** -4, 2.0 ** -10)}[fmt]
    assert np.all(np.abs(v / f - q) <= np.maximum(rel * np.abs(q), low) + 2 * NORM * np.abs(q))


def test_a_row_of_zeros_and_one_of_nan():
    import torch
    x, x64 = draw(4, 256, "F32", 3)
    x[1] = 0
    x64[1] = 0
    x[2, 17] = float("nan")
    x64[2, 17] = np.nan
    x[3, 200] = float("inf")
    x64[3, 200] = np.inf
    with np.errstate(invalid="ignore"):
        for out in ("SAME", "E4M3"):
            y, _, _ = run_forward(4, 256, "F32", out, False, 3, x=(x, x64))
            got = f64(y) if out == "SAME" else codecs.e4m3_to_f64(y.cpu().numpy())
            assert not got[1].any() and np.isnan(got[2]).all() and np.isfinite(got[0]).all()
    y = torch.zeros((4, 256), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((4, 16), dtype=torch.uint8, device="cuda")
    dg.dist_gemm_rms_norm(x, torch.ones(256, device="cuda"), y, output="MX_E4M3", scales=scales)
    s = scales.cpu().numpy()
    assert (s[2, :8] == 255).all() and (s[1, :8] == 0).all() and (s[0, :8] < 200).all()


def test_e4m3_saturates():
    """Everything past the midpoint of 416 and 448 comes out as 448, and nothing as NaN."""
    y, _, y64 = run_forward(5, 512, "BF16", "E4M3", False, 9, scale=1e-4)
    c = y.cpu().numpy() & 0x7F
    past = np.abs(y64 / 1e-4) > 432 * (1 + 2 * NORM)
    assert past.any() and (c[past] == 0x7E).all() and not (c == 0x7F).any()


@pytest.mark.parametrize("where", ["x", "residual"])
def test_stream_kept_in_place(where):
    import torch
    x, x64 = draw(33, 1000, "BF16", 5)
    r, r64 = draw(33, 1000, "BF16", 6)
    w, w64 = draw(1, 1000, "BF16", 7)
    h64 = sum_stream(x64, r64, "BF16")
    y = torch.empty_like(x)
    dg.dist_gemm_rms_norm(x, w[0], y, eps=EPS, residual=r, h=x if where == "x" else r)
    assert np.array_equal(f64(x if where == "x" else r), h64)
    ref = mx.rms_norm(h64, w64[0], EPS)[0]
    assert np.all(np.abs(f64(y) - ref) <= (2.0 ** -8 + 2 * NORM) * np.abs(ref))


def test_output_over_its_input():
    x, x64 = draw(40, 512, "F32", 8)
    w, w64 = draw(1, 512, "F32", 9)
    dg.dist_gemm_rms_norm(x, w[0], x, eps=EPS)
    ref = mx.rms_norm(x64, w64[0], EPS)[0]
    assert np.all(np.abs(f64(x) - ref) <= 2 * NORM * np.abs(ref))


def run_backward(rows, cols, typ, with_dh, seed, pitch=None, skew=0, in_place=None):
    import torch
    log("norm gradient", rows, cols, typ, with_dh, pitch, skew, in_place)
    h, h64 = draw(rows, cols, typ, seed, pitch, skew)
    dy, dy64 = draw(rows, cols, typ, seed + 1, pitch, skew, 0.01)
    dh, dh64 = draw(rows, cols, typ, seed + 2, pitch, skew, 0.01) if with_dh else (None, None)
    w, w64 = draw(1, cols, typ, seed + 3, skew=skew)
    rstd = torch.from_numpy(mx.rms_norm(h64, w64[0], EPS)[1]).float().cuda()
    dx = {"dy": dy, "h": h, "dh": dh, None: None}[in_place]
    if dx is None:
        dx = empty(rows, cols, torch_type(typ), pitch, skew)
    dw = torch.full((cols,), 7.0, device="cuda")
    ws = torch.empty(dg.dist_gemm_rms_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dg.dist_gemm_rms_norm_backward(dy, h, rstd, w[0], dx, dw, ws, dh=dh)
    s = f64(rstd)
    ref, refw = mx.rms_norm_backward(dy64, h64, w64[0], s, dh64)
    n, g = h64 * s[:, None], dy64 * w64
    size = s[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(-1, keepdims=True))
    if with_dh:
        size = size + np.abs(dh64)
    assert np.all(np.abs(f64(dx) - ref) <= OUT_STEP[typ] * np.abs(ref) + 2 * NORM * size)
    assert np.all(np.abs(f64(dw) - refw) <= (rows / 2 + 24) * U * np.abs(dy64 * n).sum(0) + 1e-30)
    return dx, dw


BACKWARD_SIZES = [(1, 1), (1, 8), (3, 7), (5, 64), (4, 512), (1030, 500), (9, 520), (600, 1000), (3, 5123), (700, 8192),
                  (3, 8200), (530, 16384), (3, 20000), (520, 32768)]


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("rows,cols", BACKWARD_SIZES)
def test_backward(rows, cols, typ, with_dh):
    run_backward(rows, cols, typ, with_dh, rows + cols)


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("pitch,skew", [(136, 0), (129, 0), (128, 1)])
def test_backward_pitches_and_bases(typ, pitch, skew):
    run_backward(11, 128, typ, True, 4, pitch, skew)


@pytest.mark.parametrize("in_place", ["dy", "h", "dh"])
@pytest.mark.parametrize("cols", [96, 8192, 20000])
def test_backward_in_place(in_place, cols):
    run_backward(70, cols, "F32", True, 3, in_place=in_place)


def test_backward_is_the_same_from_run_to_run():
    import torch
    a = run_backward(4000, 1024, "BF16", True, 11)
    for _ in range(3):
        b = run_backward(4000, 1024, "BF16", True, 11)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_backward_against_differences():
    """The kernel's own forward pass, in fp32, moved along random directions:
    the central difference of sum(dy * y) over 2t against the gradient's
    product with the direction.  The forward's rounding gives 2 NORM *
    sum|dy y| / 2t, the third derivative about t^2 per unit of the value."""
    import torch
    rows, cols, t = 16, 384, 1e-2
    h, _ = draw(rows, cols, "F32", 1)
    dy, _ = draw(rows, cols, "F32", 2)
    w, _ = draw(1, cols, "F32", 3)
    v, _ = draw(rows, cols, "F32", 4)
    rstd, y = torch.empty(rows, device="cuda"), torch.empty_like(h)

    def value(x):
        dg.dist_gemm_rms_norm(x, w[0], y, eps=EPS, rstd=rstd)
        return (dy.double() * y.double()).sum().item(), (dy.double() * y.double()).abs().sum().item()

    up, size = value(h + t * v)
    down, _ = value(h - t * v)
    value(h)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(dg.dist_gemm_rms_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dg.dist_gemm_rms_norm_backward(dy, h, rstd, w[0], dx, dw, ws)
    want = (dx.double() * v.double()).sum().item()
    assert abs((up - down) / (2 * t) - want) <= 2 * NORM * size / (2 * t) + 4 * t * t * size
    # y is linear in the weight
    assert abs((dw.double() * w[0].double()).sum().item() - value(h)[0]) <= 4 * NORM * size


def test_backward_of_no_rows_clears_dweight():
    import torch
    e = torch.empty((0, 96), device="cuda")
    dw = torch.full((96,), 3.0, device="cuda")
    ws = torch.empty(dg.dist_gemm_rms_norm_workspace(0, 96), dtype=torch.uint8, device="cuda")
    dg.dist_gemm_rms_norm_backward(e, e, torch.empty(0, device="cuda"), torch.ones(96, device="cuda"), e, dw, ws)
    assert not dw.any()


def test_norm_into_the_tensor_parallel_gemm():
    """The E4M3 output is the operand of the all-gather GEMM with scale_a = scale."""
    import torch
    M, N, K, scale = 256, 256, 512, 0.0625
    y, _, y64 = run_forward(M, K, "BF16", "E4M3", True, 21, scale=scale)
    b, b64 = draw(N, K, "F32", 5, scale=0.5)
    B = b.to(torch.float8_e4m3fn)
    D = torch.empty((M, N), device="cuda")
    with dg.Plan(M, N, K, 1, 2, "AG_ROT_A", "E4M3_F32") as p:
        p.set_scales(scale, 1.0)
        p.run(y.contiguous(), B, None, D)
        torch.cuda.synchronize()
    a = codecs.e4m3_to_f64(y.cpu().numpy()) * scale
    ref = a @ f64(B.float()).T
    size = np.linalg.norm(a, axis=1)[:, None] * np.linalg.norm(f64(B.float()), axis=1)[None]
    assert np.all(np.abs(f64(D) - ref) <= 1e-4 * size)     # the e4m3 GEMM's own bar


def test_refusals_of_tensors():
    import torch
    x = torch.zeros((4, 64), device="cuda")
    w, y = torch.ones(64, device="cuda"), torch.empty_like(x)
    good = dict(x=x, weight=w, y=y)
    for bad in (dict(x=x.half()), dict(weight=w[:63]), dict(y=y[:3]), dict(y=y.t()), dict(residual=x), dict(h=y),
                dict(rstd=torch.empty(4, dtype=torch.float64, device="cuda")), dict(output="MX_E4M3"), dict(output="E5M2"),
                dict(output="E4M3"), dict(weight=w.cpu()), dict(x=x.expand(4, 64)[0]),
                dict(x=torch.zeros((1, 64), device="cuda").expand(4, 64))):
        with pytest.raises((ValueError, dg.DistGemmError)):
            dg.dist_gemm_rms_norm(**{**good, **bad})
    with pytest.raises(dg.DistGemmError) as ei:
        ws = torch.empty(16, dtype=torch.uint8, device="cuda")
        dg.dist_gemm_rms_norm_backward(x, x, torch.ones(4, device="cuda"), w, y, torch.empty(64, device="cuda"), ws)
    assert ei.value.status == -1


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("out", ["SAME", "E4M3", "MX_E2M1", "MX_E4M3"])
def test_matrices_past_the_cache_equal_their_parts(typ, out):
    """Above the last-level cache's size the accesses go past the caches: the same bytes."""
    import torch
    rows, cols = 9000, 8224
    t = torch_type(typ)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(rows, cols, generator=g, device="cuda").to(t) for _ in range(2))
    w = torch.randn(cols, generator=g, device="cuda").to(t)

    def run(x, r):
        n = x.size(0)
        y = torch.empty((n, cols // 2 if out == "MX_E2M1" else cols), device="cuda", dtype=t if out == "SAME" else torch.uint8)
        s = torch.empty((n, mx.scale_pitch(cols)), dtype=torch.uint8, device="cuda") if out.startswith("MX") else None
        h, rstd = torch.empty_like(x), torch.empty(n, device="cuda")
        dg.dist_gemm_rms_norm(x, w, y, output=out, residual=r, h=h, rstd=rstd, scales=s, scale=0.1)
        return [v for v in (y, h, rstd, s) if v is not None]

    whole = run(x, r)
    for lo in range(0, rows, 2250):
        part = run(x[lo:lo + 2250], r[lo:lo + 2250])
        assert all(torch.equal(p, v[lo:lo + 2250]) for p, v in zip(part, whole))


@pytest.mark.parametrize("typ", ["BF16", "F32"])
def test_gradients_past_the_cache_equal_their_parts(typ):
    import torch
    rows, cols = 9000, 8224 if typ == "BF16" else 8000
    t = torch_type(typ)
    g = torch.Generator(device="cuda").manual_seed(4)
    h, dy, dh = (torch.randn(rows, cols, generator=g, device="cuda").to(t) for _ in range(3))
    w, rstd = torch.randn(cols, generator=g, device="cuda").to(t), torch.rand(rows, generator=g, device="cuda")

    def run(lo, hi):
        dx, dw = torch.empty_like(h[lo:hi]), torch.empty(cols, device="cuda")
        ws = torch.empty(dg.dist_gemm_rms_norm_workspace(hi - lo, cols), dtype=torch.uint8, device="cuda")
        dg.dist_gemm_rms_norm_backward(dy[lo:hi], h[lo:hi], rstd[lo:hi], w, dx, dw, ws, dh=dh[lo:hi])
        return dx, dw.double()

    dx, dw = run(0, rows)
    total = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for lo in range(0, rows, 1500):
        part, d = run(lo, lo + 1500)
        assert torch.equal(part, dx[lo:lo + 1500])
        total += d
    size = (dy.double() * h.double() * rstd.double()[:, None]).abs().sum(0)
    assert bool(((dw - total).abs() <= (rows / 2 + 24) * U * size).all())
