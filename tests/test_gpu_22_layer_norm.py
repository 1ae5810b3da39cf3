"""GPU tests of the layer norm and its gradient against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24).  A row's mean adds at most 32
values per lane, then a tree over 64 lanes and at most 16 parts one after
another, each part's mean once divided: under 56 roundings, so it is off by at
most N times mean|h|, N = 64 u.  The variance adds squares of differences from
a mean in as many steps (N relative), and a mean that is off by d = N mean|h|
changes it, through the join of the parts, by at most 2 d / s relative to s^2 (s
the standard deviation): with A = mean|h| rstd, rstd is off by N (1 + 2 A)
relative, and n = (h - mean) rstd by that times |n| plus N A.  y adds two
roundings of its terms.  A gradient's row means are bound like the mean,
relative to the mean of the terms' magnitudes.  dweight and dbias: a chain over
at most rows / 2 + 16 rows of |dy n| and |dy| each.  Outputs in fewer bits add
half a step: bf16 2^-8 relative, e4m3 2^-4 relative (2^-10 below its normal
range)."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import codecs, f8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
N = 64 * U
EPS = 1e-5
OUT_STEP = {"BF16": 2.0 ** -8, "F32": 0.0}


def torch_type(typ):
    import torch
    return torch.bfloat16 if typ == "BF16" else torch.float32


def draw(rows, cols, typ, seed, pitch=None, skew=0, scale=1.0, shift=0.0):
    import torch
    pitch = pitch or cols
    v = np.random.default_rng(seed).standard_normal((rows, cols)) * scale + shift
    t = torch.from_numpy(v).to(torch.float32).to(torch_type(typ))
    buf = torch.zeros(skew + max(rows, 1) * pitch, dtype=t.dtype, device="cuda")
    x = buf[skew:].as_strided((rows, cols), (pitch, 1))
    x.copy_(t)
    return x, t.to(torch.float64).numpy()


def empty(rows, cols, dtype, pitch=None, skew=0):
    import torch
    pitch = pitch or cols
    return torch.zeros(skew + max(rows, 1) * pitch, dtype=dtype, device="cuda")[skew:].as_strided((rows, cols), (pitch, 1))


def room(rows, cols, fill=0xA5):
    import torch
    return (torch.full((rows, f8.pitch(cols)), fill, dtype=torch.uint8, device="cuda"),
            torch.full((rows, f8.scale_pitch(cols)), fill, dtype=torch.uint8, device="cuda"))


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def sum_stream(x, r, typ):
    """x + residual, rounded to the type: one fp32 addition, then one rounding."""
    import torch
    return torch.from_numpy((x.astype(np.float32) + r.astype(np.float32))).to(torch_type(typ)).to(torch.float64).numpy()


def check_f8(codes, scales, v, tol, cols):
    """An F8 tensor of values within `tol` of v: every block's scale the least that does for them, every code within
    half a step, nothing past the row."""
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    blocks = -(-cols // 128)
    assert not codes[:, cols:].any() and not scales[:, blocks:].any()
    pad = f8.pitch(cols) - cols
    low, high = (np.pad(np.maximum(np.abs(v) + d * tol, 0), ((0, 0), (0, pad))).reshape(len(v), blocks, 128).max(-1) for d in (-1, 1))
    X = scales[:, :blocks].astype(np.int64) - 127
    assert (low <= 448 * np.exp2(X.astype(float))).all() and ((X == -127) | (high > 224 * np.exp2(X.astype(float)))).all()
    f = np.repeat(np.exp2(X.astype(float)), 128, axis=1)[:, :cols]
    got = codecs.e4m3_to_f64(codes[:, :cols]) * f
    assert (np.abs(got - v) <= tol + np.maximum(2.0 ** -4 * (np.abs(v) + tol), 2.0 ** -10 * f)).all()


def run_forward(rows, cols, typ, out, residual, seed, kept=True, bias=True, pitch=None, skew=0, scale=0.125, shift=0.0, x=None):
    import torch
    log("layer norm", rows, cols, typ, out, residual, kept, bias, pitch, skew, shift)
    x, x64 = draw(rows, cols, typ, seed, pitch, skew, shift=shift) if x is None else x
    w, w64 = draw(1, cols, typ, seed + 1, skew=skew)
    b, b64 = draw(1, cols, typ, seed + 3, skew=skew) if bias else ([None], np.zeros((1, cols)))
    mean, rstd = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    kw, h64 = dict(mean=mean, rstd=rstd), x64
    if residual:
        r, r64 = draw(rows, cols, typ, seed + 2, pitch, skew)
        h = empty(rows, cols, torch_type(typ), pitch, skew)
        kw.update(residual=r, h=h)
        h64 = sum_stream(x64, r64, typ)
    if kept:
        kw["kept"], kw["kept_scales"] = room(rows, cols)
    if out == "SAME":
        y = empty(rows, cols, torch_type(typ), pitch, skew)
    elif out == "E4M3":
        y = empty(rows, cols, torch.uint8, pitch, skew)
    else:
        y, kw["scales"] = room(rows, cols)
    dg.dist_gemm_layer_norm(x, w[0], b[0], y, eps=EPS, output=out, scale=scale, **kw)
    with np.errstate(invalid="ignore"):
        y64, n64, mean64, rstd64 = f8.layer_norm(h64, w64[0], b64[0], EPS)
        if residual:
            assert np.array_equal(f64(kw["h"]), h64, equal_nan=True)
        size = np.abs(h64).mean(-1)
        A = size * rstd64
        assert not np.any(np.abs(f64(mean) - mean64) > N * size)
        assert not np.any(np.abs(f64(rstd) - rstd64) > N * (1 + 2 * A) * rstd64)
        tol = (N * (1 + 2 * A))[:, None] * np.abs(n64) + (N * A)[:, None]
        if kept and np.isfinite(n64).all():
            check_f8(kw["kept"], kw["kept_scales"], n64, tol, cols)
        tol = tol * np.abs(w64) + 2 * U * (np.abs(n64 * w64) + np.abs(b64))
        if out == "SAME":
            assert not np.any(np.abs(f64(y) - y64) > OUT_STEP[typ] * np.abs(y64) + (1 + OUT_STEP[typ]) * tol)
            assert np.array_equal(np.isnan(f64(y)), np.isnan(y64))
        elif out == "E4M3":
            v = np.clip(y64 / scale, -448, 448)
            got = codecs.e4m3_to_f64(y.cpu().numpy())
            t = tol / scale + U * np.abs(y64) / scale
            assert not np.any(np.abs(got - v) > 2.0 ** -4 * (np.abs(v) + t) + 2.0 ** -10 + t)
            assert np.array_equal(np.isnan(got), np.isnan(v))
        elif np.isfinite(y64).all():
            check_f8(y, kw["scales"], y64, tol, cols)
    return y, kw, y64


FORWARD_SIZES = [(1, 1), (1, 32), (2, 7), (5, 64), (3, 500), (4, 512), (9, 520), (3, 1000), (2, 2048), (5, 5123), (2, 8192),
                 (3, 16384), (2, 20000), (2, 32768), (2100, 96), (2049, 1025), (2050, 4104), (70, 128), (131, 129), (67, 250), (1, 256),
                 (300, 3)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("out", ["SAME", "E4M3", "F8"])
@pytest.mark.parametrize("rows,cols", FORWARD_SIZES)
def test_forward(rows, cols, typ, out, residual):
    run_forward(rows, cols, typ, out, residual, rows + cols, kept=(rows + cols) % 2 == 0 or not residual, bias=residual)


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("out", ["SAME", "E4M3", "F8"])
@pytest.mark.parametrize("pitch,skew", [(136, 0), (129, 0), (128, 1), (144, 8)])
def test_forward_pitches_and_bases(typ, out, pitch, skew):
    run_forward(6, 128, typ, out, True, 4, pitch=pitch, skew=skew)


@pytest.mark.parametrize("shift", [30.0, 3e4])
@pytest.mark.parametrize("rows,cols", [(3, 100), (5, 5123), (2100, 1024), (2, 32768)])
def test_means_far_from_zero(rows, cols, shift):
    """The variance is of differences, so a mean of many standard deviations costs its own rounding only."""
    run_forward(rows, cols, "F32", "SAME", False, 5, shift=shift)


def test_rows_of_one_value_of_zeros_and_of_nan():
    import torch
    x, x64 = draw(5, 256, "F32", 3)
    for i, v in ((1, 0.0), (2, 3.5)):
        x[i], x64[i] = v, v
    x[3, 17], x64[3, 17] = float("nan"), np.nan
    x[4, 200], x64[4, 200] = float("inf"), np.inf
    for out in ("SAME", "E4M3"):
        y, kw, _ = run_forward(5, 256, "F32", out, False, 3, x=(x, x64), bias=False)
        got = f64(y) if out == "SAME" else codecs.e4m3_to_f64(y.cpu().numpy())
        assert not got[1:3].any() and np.isnan(got[3:]).all() and np.isfinite(got[0]).all()
    y, s = room(5, 256)
    k, ks = room(5, 256)
    dg.dist_gemm_layer_norm(x, torch.ones(256, device="cuda"), None, y, output="F8", scales=s, kept=k, kept_scales=ks)
    for codes, scales in ((y, s), (k, ks)):
        scales = scales.cpu().numpy()
        assert (scales[3:, :2] == 255).all() and not scales[1:3].any() and (scales[0, :2] < 200).all()
        assert not codes[1:].any()
    # without eps a row of one value has no direction: NaN, as the formula says
    y = torch.empty_like(x)
    dg.dist_gemm_layer_norm(x, torch.ones(256, device="cuda"), None, y, eps=0.0)
    assert torch.isnan(y[1:]).all() and torch.isfinite(y[0]).all()


@pytest.mark.parametrize("where", ["x", "residual"])
def test_stream_kept_in_place(where):
    import torch
    x, x64 = draw(33, 1000, "BF16", 5)
    r, r64 = draw(33, 1000, "BF16", 6)
    w, w64 = draw(1, 1000, "BF16", 7)
    h64 = sum_stream(x64, r64, "BF16")
    y = torch.empty_like(x)
    dg.dist_gemm_layer_norm(x, w[0], None, y, eps=EPS, residual=r, h=x if where == "x" else r)
    assert np.array_equal(f64(x if where == "x" else r), h64)
    ref = f8.layer_norm(h64, w64[0], None, EPS)[0]
    assert np.all(np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 8 * N * np.abs(w64))


def test_output_over_its_input():
    x, x64 = draw(40, 512, "F32", 8)
    w, w64 = draw(1, 512, "F32", 9)
    dg.dist_gemm_layer_norm(x, w[0], None, x, eps=EPS)
    ref = f8.layer_norm(x64, w64[0], None, EPS)[0]
    assert np.all(np.abs(f64(x) - ref) <= 4 * N * np.abs(ref) + 2 * N * np.abs(w64))


def run_backward(rows, cols, typ, kept, with_dh, seed, pitch=None, skew=0, in_place=None, shift=0.5, bias=True):
    import torch
    log("layer norm gradient", rows, cols, typ, kept, with_dh, pitch, skew, in_place)
    h, h64 = draw(rows, cols, typ, seed, pitch, skew, shift=shift)
    dy, dy64 = draw(rows, cols, typ, seed + 1, pitch, skew, 0.01, shift=0.002)
    dh, dh64 = draw(rows, cols, typ, seed + 2, pitch, skew, 0.01) if with_dh else (None, None)
    w, w64 = draw(1, cols, typ, seed + 3, skew=skew)
    _, n64, mean64, rstd64 = f8.layer_norm(h64, w64[0], None, EPS)
    mean, rstd = (torch.from_numpy(t).float().cuda() for t in (mean64, rstd64))
    s = f64(rstd)
    kw = {}
    if kept:
        codes, scales = f8.quantize(n64)
        n64 = f8.values(codes, scales, cols)
        rows_in, kw["h_scales"] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    else:
        rows_in = h
        n64 = (h64 - f64(mean)[:, None]) * s[:, None]
    dx = {"dy": dy, "h": h, "dh": dh, None: None}[in_place]
    if dx is None:
        dx = empty(rows, cols, torch_type(typ), pitch, skew)
    dw, db = torch.full((cols,), 7.0, device="cuda"), torch.full((cols,), 7.0, device="cuda")
    ws = torch.empty(dg.dist_gemm_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dg.dist_gemm_layer_norm_backward(dy, rows_in, None if kept else mean, rstd, w[0], dx, dw, db if bias else None, ws, dh=dh, **kw)
    ref, refw, refb = f8.layer_norm_backward(dy64, n64, w64[0], s, dh64)
    g = dy64 * w64
    size = s[:, None] * (np.abs(g) + np.abs(g).mean(-1, keepdims=True) + np.abs(n64) * np.abs(g * n64).mean(-1, keepdims=True))
    if with_dh:
        size = size + np.abs(dh64)
    assert np.all(np.abs(f64(dx) - ref) <= OUT_STEP[typ] * np.abs(ref) + 2 * N * size)
    chain = (rows / 2 + 24) * U
    assert np.all(np.abs(f64(dw) - refw) <= chain * np.abs(dy64 * n64).sum(0) + 1e-30)
    if bias:
        assert np.all(np.abs(f64(db) - refb) <= chain * np.abs(dy64).sum(0) + 1e-30)
    else:
        assert (db == 7.0).all()
    return dx, dw, db


BACKWARD_SIZES = [(1, 1), (1, 8), (3, 7), (5, 64), (4, 512), (1030, 500), (9, 520), (600, 1000), (3, 5123), (700, 8192),
                  (3, 8200), (530, 16384), (3, 16385), (3, 20000), (520, 32768), (70, 128), (1031, 129), (5000, 250), (20000, 100),
                  (300, 3)]


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("rows,cols", BACKWARD_SIZES)
def test_backward(rows, cols, typ, with_dh, kept):
    run_backward(rows, cols, typ, kept, with_dh, rows + cols, bias=not (with_dh and kept))


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("pitch,skew", [(136, 0), (129, 0), (128, 1)])
def test_backward_pitches_and_bases(typ, pitch, skew, kept):
    run_backward(11, 128, typ, kept, True, 4, pitch, skew)


@pytest.mark.parametrize("in_place", ["dy", "h", "dh"])
@pytest.mark.parametrize("cols", [96, 8192, 20000])
def test_backward_in_place(in_place, cols):
    run_backward(70, cols, "F32", False, True, 3, in_place=in_place)


@pytest.mark.parametrize("cols", [96, 8192, 20000])
def test_backward_from_the_checkpoint_in_place(cols):
    run_backward(70, cols, "BF16", True, True, 3, in_place="dy")


@pytest.mark.parametrize("kept", [False, True])
def test_backward_is_the_same_from_run_to_run(kept):
    import torch
    a = run_backward(4000, 1024, "BF16", kept, True, 11)
    for _ in range(3):
        b = run_backward(4000, 1024, "BF16", kept, True, 11)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_backward_against_differences():
    """The kernel's own forward pass, in fp32, moved along random directions:
    the central difference of sum(dy * y) over 2t against the gradient's
    product with the direction.  The forward's rounding gives 4 N *
    sum|dy y| / 2t, the third derivative about t^2 per unit of the value."""
    import torch
    rows, cols, t = 16, 384, 1e-2
    h, _ = draw(rows, cols, "F32", 1)
    dy, _ = draw(rows, cols, "F32", 2)
    w, _ = draw(1, cols, "F32", 3)
    v, _ = draw(rows, cols, "F32", 4)
    b, _ = draw(1, cols, "F32", 5)
    mean, rstd, y = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(h)

    def value(x, w=w[0], b=b[0]):
        dg.dist_gemm_layer_norm(x, w, b, y, eps=EPS, mean=mean, rstd=rstd)
        return (dy.double() * y.double()).sum().item(), (dy.double() * y.double()).abs().sum().item()

    up, size = value(h + t * v)
    down, _ = value(h - t * v)
    dx, dw, db = torch.empty_like(h), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(dg.dist_gemm_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    at, _ = value(h)
    dg.dist_gemm_layer_norm_backward(dy, h, mean, rstd, w[0], dx, dw, db, ws)
    want = (dx.double() * v.double()).sum().item()
    assert abs((up - down) / (2 * t) - want) <= 4 * N * size / (2 * t) + 4 * t * t * size
    # y is linear in the weight and the bias
    slope = (dw.double() * w[0].double() + db.double() * b[0].double()).sum().item()
    assert abs(slope - at) <= 8 * N * size + 8 * N * (dy.double() * b[0].double()).abs().sum().item()


def test_the_checkpoint_gives_the_gradient_of_its_rows():
    """What the forward pass keeps in 8 bits, taken straight to the backward pass."""
    import torch
    rows, cols = 200, 1000
    x, x64 = draw(rows, cols, "BF16", 1, shift=4.0)
    w, w64 = draw(1, cols, "BF16", 2)
    dy, dy64 = draw(rows, cols, "BF16", 3)
    y, s = room(rows, cols)
    k, ks = room(rows, cols)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dg.dist_gemm_layer_norm(x, w[0], None, y, output="F8", scales=s, mean=mean, rstd=rstd, kept=k, kept_scales=ks)
    ws = torch.empty(dg.dist_gemm_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    got = []
    for h, hs in ((x, None), (k, ks)):
        dx, dw, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        dg.dist_gemm_layer_norm_backward(dy, h, mean, rstd, w[0], dx, dw, db, ws, h_scales=hs)
        got.append((f64(dx), f64(dw), f64(db)))
    n = f8.values(k.cpu().numpy(), ks.cpu().numpy(), cols)
    ref = f8.layer_norm_backward(dy64, n, w64[0], f64(rstd))
    assert np.array_equal(got[0][2], got[1][2])       # dbias does not see n
    size = f64(rstd)[:, None] * (np.abs(dy64 * w64) + np.abs(dy64 * w64).mean(-1, keepdims=True) * (1 + np.abs(n)))
    assert np.all(np.abs(got[1][0] - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + 8 * N * size)
    # half a step of 8 bits per value is what the checkpoint costs
    exact = f8.layer_norm_backward(dy64, f8.layer_norm(x64, w64[0], None, EPS)[1], w64[0], f64(rstd))
    for a, b in zip(got[1][:2], exact[:2]):
        assert np.linalg.norm(a - b) <= 2.0 ** -4 * np.linalg.norm(b)


def test_backward_of_no_rows_clears_the_sums():
    import torch
    e = torch.empty((0, 96), device="cuda")
    dw, db = torch.full((96,), 3.0, device="cuda"), torch.full((96,), 3.0, device="cuda")
    ws = torch.empty(dg.dist_gemm_layer_norm_workspace(0, 96), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, device="cuda")
    dg.dist_gemm_layer_norm_backward(e, e, none, none, torch.ones(96, device="cuda"), e, dw, db, ws)
    assert not dw.any() and not db.any()


def test_refusals_of_tensors():
    import torch
    x = torch.zeros((4, 64), device="cuda")
    w, y = torch.ones(64, device="cuda"), torch.empty_like(x)
    good = dict(x=x, weight=w, bias=w, y=y)
    k, ks = room(4, 64)
    for bad in (dict(x=x.half()), dict(weight=w[:63]), dict(bias=w[:63]), dict(y=y[:3]), dict(y=y.t()), dict(residual=x), dict(h=y),
                dict(rstd=torch.empty(4, dtype=torch.float64, device="cuda")), dict(mean=torch.empty(3, device="cuda")),
                dict(output="F8"), dict(output="F8", y=k), dict(output="MX_E4M3"), dict(output="E4M3"), dict(weight=w.cpu()),
                dict(kept=k), dict(kept_scales=ks), dict(kept=k[:, :64].contiguous(), kept_scales=ks),
                dict(x=torch.zeros((1, 64), device="cuda").expand(4, 64))):
        with pytest.raises((ValueError, dg.DistGemmError)):
            dg.dist_gemm_layer_norm(**{**good, **bad})
    m = torch.ones(4, device="cuda")
    ws = torch.empty(dg.dist_gemm_layer_norm_workspace(4, 64), dtype=torch.uint8, device="cuda")
    good = dict(dy=x, h=y, mean=m, rstd=m.clone(), weight=w, dx=torch.empty_like(x), dweight=torch.empty(64, device="cuda"),
                dbias=torch.empty(64, device="cuda"), workspace=ws)
    dg.dist_gemm_layer_norm_backward(**good)
    for bad in (dict(h=y.bfloat16()), dict(mean=None), dict(h_scales=ks), dict(h=k), dict(rstd=m[:3]), dict(workspace=None),
                dict(workspace=ws[:16]), dict(workspace=ws.cpu()), dict(dbias=w[:3]), dict(dx=x.t()), dict(dh=x[:3])):
        with pytest.raises((ValueError, dg.DistGemmError)):
            dg.dist_gemm_layer_norm_backward(**{**good, **bad})


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("out", ["SAME", "E4M3", "F8"])
def test_matrices_past_the_cache_equal_their_parts(typ, out):
    """Above the last-level cache's size the accesses go past the caches: the same bytes."""
    import torch
    rows, cols = 9000, 8224
    t = torch_type(typ)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(rows, cols, generator=g, device="cuda").to(t) for _ in range(2))
    w, b = (torch.randn(cols, generator=g, device="cuda").to(t) for _ in range(2))

    def run(x, r):
        n = x.size(0)
        s = None
        if out == "F8":
            y, s = room(n, cols)
        else:
            y = torch.empty((n, cols), device="cuda", dtype=t if out == "SAME" else torch.uint8)
        h, mean, rstd = torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        k, ks = room(n, cols)
        dg.dist_gemm_layer_norm(x, w, b, y, output=out, residual=r, h=h, mean=mean, rstd=rstd, scales=s, scale=0.1, kept=k,
                                kept_scales=ks)
        return [v for v in (y, h, mean, rstd, k, ks, s) if v is not None]

    whole = run(x, r)
    for lo in range(0, rows, 2250):
        part = run(x[lo:lo + 2250], r[lo:lo + 2250])
        assert all(torch.equal(p, v[lo:lo + 2250]) for p, v in zip(part, whole))


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
def test_gradients_past_the_cache_equal_their_parts(typ, kept):
    import torch
    rows, cols = 9000, 8224 if typ == "BF16" else 8000
    t = torch_type(typ)
    g = torch.Generator(device="cuda").manual_seed(4)
    h, dy, dh = (torch.randn(rows, cols, generator=g, device="cuda").to(t) for _ in range(3))
    w, rstd = torch.randn(cols, generator=g, device="cuda").to(t), torch.rand(rows, generator=g, device="cuda")
    mean, hs = torch.randn(rows, generator=g, device="cuda"), None
    n = (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    if kept:
        codes, hs = room(rows, cols)
        dg.dist_gemm_f8_quantize(h, codes, hs)
        v = torch.empty(rows, cols, device="cuda")
        dg.dist_gemm_f8_dequantize(codes, hs, v)
        h, n = codes, v.double()

    def run(lo, hi):
        dx = torch.empty_like(dy[lo:hi])
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        ws = torch.empty(dg.dist_gemm_layer_norm_workspace(hi - lo, cols), dtype=torch.uint8, device="cuda")
        dg.dist_gemm_layer_norm_backward(dy[lo:hi], h[lo:hi], mean[lo:hi], rstd[lo:hi], w, dx, dw, db, ws, dh=dh[lo:hi],
                                         h_scales=None if hs is None else hs[lo:hi])
        return dx, dw.double(), db.double()

    dx, dw, db = run(0, rows)
    tw, tb = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for lo in range(0, rows, 1500):
        part, a, b = run(lo, lo + 1500)
        assert torch.equal(part, dx[lo:lo + 1500])
        tw += a
        tb += b
    chain = (rows / 2 + 24) * U
    assert bool(((dw - tw).abs() <= chain * (dy.double() * n).abs().sum(0)).all())
    assert bool(((db - tb).abs() <= chain * dy.double().abs().sum(0)).all())


@pytest.mark.parametrize("kept", [False, True])
def test_on_a_stream_of_its_own_and_in_a_graph(kept):
    """Forward and backward on a side stream, then captured together: every replay equals the eager results."""
    import torch
    rows, cols = 600, 1000
    x, _ = draw(rows, cols, "BF16", 1)
    dy, _ = draw(rows, cols, "BF16", 2)
    w, b = draw(2, cols, "BF16", 3)[0]
    y, s = room(rows, cols)
    k, ks = room(rows, cols)
    mean, rstd, dx = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(dg.dist_gemm_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    out = (y, s, k, ks, mean, rstd, dx, dw, db)

    def step():
        dg.dist_gemm_layer_norm(x, w, b, y, output="F8", scales=s, mean=mean, rstd=rstd, kept=k, kept_scales=ks)
        dg.dist_gemm_layer_norm_backward(dy, k if kept else x, None if kept else mean, rstd, w, dx, dw, db, ws,
                                         h_scales=ks if kept else None)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    for t in out:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(t, v) for t, v in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for t in out:
            t.fill_(i)
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, v) for t, v in zip(out, want))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(t, v) for t, v in zip(out, want))
